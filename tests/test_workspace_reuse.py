"""One zeroed workspace serves decode calls of different sizes in turn: every
result has the bits of a call with a fresh workspace, and every output is written
(`out` is NaN before each call)."""
import numpy as np
import pytest
import torch

import rank_kv_cache_wsvd_b200 as W
from paged_util import cuda, randn, table_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from rank_kv_cache_wsvd_b200 import build
    build.build()
    W.load()


def _lens(B, lo, hi, seed):
    return [int(n) for n in np.random.default_rng(seed).integers(lo, hi + 1, B)]


def _codes(shape, r, bits, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    lat = [torch.randint(0, 256, shape + (r * bits // 8,), generator=g, dtype=torch.uint8, device="cuda") for _ in range(2)]
    return lat + [(torch.rand(shape, generator=g, device="cuda") + 0.5).div(127 if bits == 8 else 7).half() for _ in range(2)]


# Each maker gives (the workspace a call needs, the call: workspace or None -> out, the shape of out).
def _latent_paged(B, H=32, r=32, bits=8, Hd=128, lo=1024, hi=4096, seed=0):
    lens = _lens(B, lo, hi, B + seed)
    table, pool = table_for(lens, 64, B)
    lk, lv, sk, sv = _codes((pool, H, 64), r, bits, B)
    Bk, Bv = (randn((H, r, Hd), "fp16", s) * r ** -0.5 for s in (1, 2))
    q, tab, n = randn((B, H, Hd), "bf16", B), cuda(table), cuda(np.asarray(lens, np.int32))
    return W.wsvd_decode_workspace_size(B, H, r), lambda out, ws: W.wsvd_decode_attention_paged(
        q, lk, lv, sk, sv, Bk, Bv, tab, n, bits, out=out, workspace_buf=ws), (B, H, Hd)


def _latent(B, H=32, r=32, bits=8, Hd=64, L_cap=512):
    lk, lv, sk, sv = _codes((B, H, L_cap), r, bits, B)
    Bk, Bv = (randn((H, r, Hd), "fp16", s) * r ** -0.5 for s in (1, 2))
    q, n = randn((B, H, Hd), "fp16", B), cuda(np.asarray(_lens(B, L_cap // 2, L_cap, B), np.int32))
    assert W.wsvd_decode_launch_count(B, H, Hd, r, bits, L_cap) == 2  # the path that keeps partial results
    return W.wsvd_decode_workspace_size(B, H, r), lambda out, ws: W.wsvd_decode_attention(
        q, lk, lv, sk, sv, Bk, Bv, n, bits, out=out, workspace_buf=ws), (B, H, Hd)


def _dense(B, H=32, Hd=64, L_cap=256):
    K, V = (randn((B, H, L_cap, Hd), "fp16", B + s) for s in (1, 2))
    q, n = randn((B, H, Hd), "fp16", B), cuda(np.asarray(_lens(B, L_cap // 2, L_cap, B), np.int32))
    return W.dense_decode_workspace_size(B, H, Hd), lambda out, ws: W.dense_decode_attention(
        q, K, V, n, out=out, workspace_buf=ws), (B, H, Hd)


def _grouped(B, Tq=1, Hq=32, Hkv=8, r=32, bits=8, Hd=64, L_cap=2048):
    lk, lv, sk, sv = _codes((B, Hkv, L_cap), r, bits, B)
    Bk, Bv = (randn((Hkv, r, Hd), "fp16", s) * r ** -0.5 for s in (1, 2))
    q, n = randn((B, Tq, Hq, Hd), "fp16", B), cuda(np.asarray(_lens(B, L_cap // 2, L_cap, B), np.int32))
    return W.wsvd_decode_multi_workspace_size(B, Tq, Hq, Hkv, r, L_cap), lambda out, ws: W.wsvd_decode_multi(
        q, lk, lv, sk, sv, Bk, Bv, n, bits, out=out, workspace_buf=ws), (B, Tq, Hq, Hd)


def _dense_paged(Tq, G, B=64, Hkv=8, Hd=128, lo=100, hi=600):
    lens = _lens(B, lo, hi, 5)
    table, pool = table_for(lens, 32, 3)
    kp, vp = randn((pool, Hkv, 32, Hd), "bf16", 1), randn((pool, Hkv, 32, Hd), "bf16", 2)
    q, tab, n = randn((B, Tq, G * Hkv, Hd), "bf16", Tq + G), cuda(table), cuda(np.asarray(lens, np.int32))
    return W.paged_decode_workspace_size(B, Tq, G * Hkv, Hkv, Hd), lambda out, ws: W.paged_decode_attention(
        q, kp, vp, tab, n, out=out, workspace_buf=ws), (B, Tq, G * Hkv, Hd)


def _in_turn(calls, order):
    """Every call alone, then all through one buffer that is zeroed once."""
    fresh = [call(torch.full(shape, float("nan"), device="cuda"), None) for _, call, shape in calls]
    assert all(torch.isfinite(t).all() for t in fresh)
    ws = W.workspace(max(need for need, _, _ in calls))
    for i in order:
        _, call, shape = calls[i]
        out = call(torch.full(shape, float("nan"), device="cuda"), ws)
        assert torch.equal(out, fresh[i]), f"call {i}: {int((out != fresh[i]).sum())} of {out.numel()} values differ"


def test_latent_paged_decode_of_a_batch_that_shrinks_and_grows():
    _in_turn([_latent_paged(B) for B in (16, 6, 2, 5)], [0, 1, 2, 0, 3, 1, 0, 0, 2])


@pytest.mark.parametrize("bits,r", [(8, 16), (8, 128), (4, 64)])
def test_latent_paged_decode_of_other_ranks(bits, r):
    _in_turn([_latent_paged(9, r=r, bits=bits), _latent_paged(4), _latent_paged(3, H=7, r=r, bits=bits)], [0, 1, 2, 0, 2, 1, 0])


@pytest.mark.parametrize("G", [4, 8])
def test_dense_paged_decode_of_one_and_several_tokens(G):
    _in_turn([_dense_paged(t, G) for t in (1, 2, 4)], [0, 1, 0, 2, 0, 2, 1, 0])


def test_dense_paged_decode_of_other_head_sizes_and_batches():
    _in_turn([_dense_paged(1, 4), _dense_paged(1, 1, B=300, Hkv=4, Hd=32, lo=1, hi=300),
              _dense_paged(3, 4, B=3, Hkv=2, Hd=256, lo=900, hi=4000), _dense_paged(2, 16, B=5, Hkv=2, Hd=64, hi=5000)],
             [0, 1, 2, 3, 0, 3, 1, 2, 1, 0])


def test_latent_decode_of_a_batch_that_shrinks_and_grows():
    _in_turn([_latent(96), _latent(4, L_cap=8192), _latent(5, L_cap=8192), _latent(6, L_cap=8192), _latent(80)],
             [0, 1, 2, 3, 0, 3, 4, 2, 1, 0])


def test_dense_decode_of_a_batch_that_shrinks_and_grows():
    _in_turn([_dense(96), _dense(4, L_cap=4096), _dense(5, L_cap=4096), _dense(6, L_cap=4096)], [0, 1, 2, 3, 0, 2, 3, 1, 0])


def test_grouped_decode_of_other_batches_and_tokens():
    _in_turn([_grouped(8), _grouped(3), _grouped(2, Tq=4), _grouped(5, Hq=8, L_cap=4096)], [0, 1, 2, 3, 0, 3, 1, 2, 0])


def test_grouped_decode_needs_no_zeroed_workspace():
    need, call, shape = _grouped(4)
    want = call(torch.full(shape, float("nan"), device="cuda"), None)
    ws = torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert torch.equal(call(torch.full(shape, float("nan"), device="cuda"), ws), want)


def test_different_decodes_share_one_workspace():
    _in_turn([_latent_paged(16), _dense_paged(2, 4), _latent(40), _dense(40), _latent_paged(3), _dense_paged(1, 8),
              _latent(4, L_cap=8192)], [0, 1, 2, 3, 4, 5, 6, 2, 0, 6, 3, 1, 5, 4, 3, 0])


def test_every_call_leaves_the_counters_zero():
    """The first 8 KB hold the counters, whatever the sizes."""
    calls = [_latent_paged(16), _dense_paged(2, 4), _dense_paged(1, 4), _dense_paged(4, 8), _latent(40), _dense(40)]
    ws = W.workspace(max(need for need, _, _ in calls))
    for _, call, shape in calls:
        call(torch.empty(shape, device="cuda"), ws)
        assert (ws[:8192] == 0).all()
