"""Calls over pages that the documentation allows and the other tests leave out:
rotations of any multiple of 16, up to 64 queries a head in one token or in many, fp16
activations at both ends of their range, tokens of zeros, the largest E, calls from two
threads, two captured graphs at once."""
import threading

import numpy as np
import pytest
import torch

import rank_kv_cache_wsvd_b200 as W
from oracle import paged_oracle as P
from paged_util import cuda, f64, randn, rope_table, table_for
from test_block_tiles import _check_rows, _rotated
from test_paged_latent_parity import _cache as latent_cache, _factors
from test_paged_parity import LENS, _append_case, _cache, _check_append, _check_decode, _decode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from rank_kv_cache_wsvd_b200 import build
    build.build()
    W.load()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("Hd,rot", [(32, 16), (64, 48), (128, 16), (128, 80), (128, 112), (256, 48), (256, 240)])
@pytest.mark.parametrize("inter", [False, True])
def test_append_rotates_any_multiple_of_sixteen(dtype, Hd, rot, inter):
    B, T, Hq, Hkv, page = 2, 19, 5, 3, 32
    lens = [7, 40]
    q, k, v, kp, vp, table = _append_case(B, T, Hq, Hkv, Hd, page, dtype, lens, seed=Hd + rot)
    cs, n = rope_table(128, rot), cuda(np.asarray(lens, np.int32))
    ref = P.kv_append(f64(k), f64(v), f64(q), f64(kp), f64(vp), table, lens, f64(cs), rot, inter)
    before = kp.clone(), vp.clone()
    qo = W.paged_kv_append(k, v, kp, vp, cuda(table), n, q=q, cos_sin=cs, interleaved=inter)
    mine = (f64(before[0]) != ref[0]).any(axis=-1, keepdims=True)
    _check_append(kp, vp, qo, ref, before, dtype, np.abs(f64(q)).max(), mine)
    assert torch.equal(qo[..., rot:], q[..., rot:]) and n.tolist() == [a + T for a in lens]


@pytest.mark.parametrize("dtype,Hd", [("fp16", 64), ("bf16", 128), ("fp16", 256), ("bf16", 32)])
@pytest.mark.parametrize("Hkv,G,Tq", [(1, 1, 64), (2, 64, 1), (1, 2, 32), (3, 5, 12), (2, 17, 1), (1, 8, 8)])
def test_decode_of_up_to_64_queries_a_head(dtype, Hd, Hkv, G, Tq):
    lens = LENS[:12]
    kp, vp, table = _cache(lens, Hkv, Hd, 16, dtype, seed=Hd + G)
    q = randn((len(lens), Tq, Hkv * G, Hd), dtype, 5)
    out, err = _decode(q, kp, vp, table, lens)
    assert err == 0
    _check_decode(out, q, kp.nan_to_num(0), vp.nan_to_num(0), table, lens, what=f"G{G} Tq{Tq}")
    for b, n in enumerate(lens):  # tokens before the first row see nothing
        assert (out[b, :max(0, min(Tq, Tq - n))] == 0).all()


@pytest.mark.parametrize("B,T,H,E,r,blk", [(1, 1, 3, 256, 32, 128), (2, 1, 4, 1536, 16, 512), (9, 1, 4, 1024, 32, 1024), (1, 70, 5, 256, 64, 64),
                                           (2, 3, 1, 16384, 16, 1024), (1, 1, 2, 16384, 32, 256), (1, 200, 16, 1536, 128, 512)])
def test_latent_append_of_fp16_at_both_ends_of_its_range(B, T, H, E, r, blk):
    """Tokens near the largest fp16 value, among its denormals, of zeros, and ordinary ones, each with
    its own power of two; weights that keep every scale an fp16 number."""
    page, gains = 16, [1.0, 6e4 / 4, 2.0 ** -20, 0.0]
    tokens = torch.randn((B * T, E), generator=torch.Generator().manual_seed(1)).clamp(-4, 4)
    gain = torch.tensor([gains[(b * T + t) % 4] for b in range(B) for t in range(T)])
    x = (tokens * gain[:, None]).half().view(B, T, E).cuda()
    down = [(randn((H, E, r), "fp16", s) * E ** -0.5).contiguous() for s in (4, 5)]
    lens = [5 * b for b in range(B)]
    table, pool = table_for([n + T for n in lens], page, 3)
    lat = [torch.full((pool, H, page, r), 77, dtype=torch.uint8, device="cuda") for _ in range(2)]
    sc = [torch.full((pool, H, page), 3.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    n, tab, err = cuda(np.asarray(lens, np.int32)), cuda(table), torch.zeros(1, dtype=torch.int32, device="cuda")
    W.wsvd_latent_append_paged(x, *down, n, tab, *lat, *sc, 8, blk, err=err)
    assert int(err.item()) == 0
    row = n.long()[:, None] - T + torch.arange(T, device="cuda")
    at = (tab.long().gather(1, row // page), row % page)
    rot = _rotated(x, blk)
    zero, tiny = ((gain == g).view(B, T).cuda() for g in (0.0, 2.0 ** -20))
    for k in range(2):
        c = torch.einsum("bte,her->bthr", rot, down[k].double())
        codes, scale = lat[k][at[0], :, at[1]].view(torch.int8), sc[k][at[0], :, at[1]]
        assert (codes[zero] == 0).all() and (scale[zero] == 0).all()
        # scales of the tiny tokens are fp16 denormals (a few steps of 2^-24), as the definition has them
        want = (c.abs().amax(-1) / 127).half()
        assert (want[tiny] == scale[tiny]).float().mean() > 0.99 or not tiny.any()
        rest = ~zero & ~tiny
        ties = _check_rows(codes[rest], scale[rest], c[rest], 127)
        assert ties <= 4 + B * T * H * (r * 2e-3 + 2.0 ** -8)


@pytest.mark.parametrize("bits,r", [(8, 32), (4, 64)])
def test_latent_decode_of_rows_without_scale(bits, r):
    """All value scales zero: the output is zero; all key scales zero: the mean of the rows."""
    lens, H, Hd = [40, 7], 3, 64
    lk, lv, sk, sv, table = latent_cache(lens, H, r, bits, 16, seed=1, poison=False)
    Bk, Bv = _factors(H, r, Hd, 2)
    q, tab, n = randn((2, H, Hd), "bf16", 3), cuda(table), cuda(np.asarray(lens, np.int32))
    assert (W.wsvd_decode_attention_paged(q, lk, lv, sk, sv * 0, Bk, Bv, tab, n, bits) == 0).all()
    out = W.wsvd_decode_attention_paged(q, lk, lv, sk * 0, sv, Bk, Bv, tab, n, bits)
    codes = P.latent_codes(lv.cpu().numpy(), bits)
    for b, m in enumerate(lens):
        v = P.rows(codes * f64(sv)[..., None], table, b, m)
        want = np.einsum("nhr,hrd->hd", v, f64(Bv)) / m
        mass = np.einsum("nhr,hrd->hd", np.abs(v), np.abs(f64(Bv))) / m
        big = f64(sv).max() * (127 if bits == 8 else 7) * np.abs(f64(Bv)).sum(1)
        assert (np.abs(f64(out[b]) - want) <= P.latent_allowance(mass[None], np.zeros((1, H)), r, Hd, big, m)[0]).all()


def test_calls_from_two_threads():
    """Each thread its stream, its workspaces and its cache; first calls of their kernels among them."""
    def case(seed):
        lens = [900, 20 + seed]
        kp, vp, table = _cache(lens, 2, 64, 16, "bf16", seed=seed)
        lat = latent_cache(lens, 3, 32, 8, 16, seed=seed)
        return dict(kp=kp, vp=vp, tab=cuda(table), n=cuda(np.asarray(lens, np.int32)), q=randn((2, 1, 8, 64), "bf16", seed),
                    lq=randn((2, 3, 64), "bf16", seed), lat=lat[:4], ltab=cuda(lat[4]), up=_factors(3, 32, 64, seed))

    def once(c, **kw):
        return (W.paged_decode_attention(c["q"], c["kp"], c["vp"], c["tab"], c["n"], **kw),
                W.wsvd_decode_attention_paged(c["lq"], *[c["lat"][i] for i in (0, 1, 2, 3)], *c["up"], c["ltab"], c["n"], 8, **kw))

    cases = [case(s) for s in (1, 2)]
    want = [once(c) for c in cases]
    torch.cuda.synchronize()
    wrong, streams = [], [torch.cuda.Stream() for _ in cases]

    def work(i):
        try:
            ws = W.workspace(W.paged_decode_workspace_size(2, 1, 8, 2, 64))
            torch.cuda.synchronize()
            got = [once(cases[i], stream=streams[i], workspace_buf=ws) for _ in range(50)]
            streams[i].synchronize()
            wrong.extend(1 for g in got if not all(torch.equal(a, b) for a, b in zip(g, want[i])))
        except Exception as e:  # a thread's failure is the test's
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_two_captured_steps_at_once():
    """Append and decode captured twice, each graph with its own cache and workspaces, replayed at once."""
    B, Hq, Hkv, Hd, page, steps = 2, 8, 2, 64, 16, 12
    graphs, states, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    cs = rope_table(64, Hd)
    for i in range(2):
        table, pool = table_for([64] * B, page, i)
        s = dict(table=table, tab=cuda(table), n=torch.zeros(B, dtype=torch.int32, device="cuda"), q=randn((B, 1, Hq, Hd), "bf16", i),
                 k=randn((B, 1, Hkv, Hd), "bf16", 7 + i), kp=randn((pool, Hkv, page, Hd), "bf16", 9), vp=randn((pool, Hkv, page, Hd), "bf16", 10),
                 qo=torch.empty((B, 1, Hq, Hd), dtype=torch.bfloat16, device="cuda"), out=torch.empty((B, 1, Hq, Hd), device="cuda"),
                 wa=W.workspace(W.paged_kv_append_workspace_size(B)), wd=W.workspace(W.paged_decode_workspace_size(B, 1, Hq, Hkv, Hd)))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            W.paged_kv_append(s["k"], s["k"], s["kp"], s["vp"], s["tab"], s["n"], q=s["q"], q_out=s["qo"], cos_sin=cs, workspace_buf=s["wa"])
            W.paged_decode_attention(s["qo"], s["kp"], s["vp"], s["tab"], s["n"], out=s["out"], workspace_buf=s["wd"])
        graphs.append(g), states.append(s)
    torch.cuda.synchronize()
    for _ in range(steps):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for s in states:
        assert s["n"].tolist() == [steps] * B
        _check_decode(s["out"], s["qo"], s["kp"], s["vp"], s["table"], [steps] * B, what="two graphs")
        assert (s["wa"] == 0).all() and (s["wd"][:8192] == 0).all()
