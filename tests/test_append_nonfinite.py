"""A token that is not finite stays visible in a latent cache: every head's row of it
gets a scale that is not finite, the decode of its sequence is not finite, and no
other row or sequence changes."""
import numpy as np
import pytest
import torch

import rank_kv_cache_wsvd_b200 as W
from paged_util import cuda, randn, table_for

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from rank_kv_cache_wsvd_b200 import build
    build.build()
    W.load()


def _spoil(x, b, t, how):
    x = x.clone()
    if how == "overflow":  # every value finite, their rotation is not
        x[b, t] = torch.finfo(x.dtype).max
    else:
        x[b, t, 5] = how
    return x


def _paged(x, Ak, Av, bits, blk, page=16):
    B, T, E = x.shape
    H, _, r = Ak.shape
    lens = [3 + 7 * b for b in range(B)]
    table, pool = table_for([n + T for n in lens], page, 2)
    lat = [torch.zeros((pool, H, page, r * bits // 8), dtype=torch.uint8, device="cuda") for _ in range(2)]
    sc = [torch.ones((pool, H, page), dtype=torch.float16, device="cuda") for _ in range(2)]
    n, tab = cuda(np.asarray(lens, np.int32)), cuda(table)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    W.wsvd_latent_append_paged(x, Ak, Av, n, tab, *lat, *sc, bits, blk, err=err)
    assert int(err.item()) == 0
    at = [[(int(table[b, (lens[b] + t) // page]), (lens[b] + t) % page) for t in range(T)] for b in range(B)]
    rows = [torch.stack([torch.stack([a[p, :, i] for p, i in row]) for row in at]) for a in lat + sc]
    q = randn((B, H, 64), "bf16", 4)
    up = (randn((H, r, 64), "fp16", 5) * r ** -0.5).contiguous()
    return rows, W.wsvd_decode_attention_paged(q, *lat, *sc, up, up, tab, n, bits)


def _contiguous(x, Ak, Av, bits, blk):
    B, T, E = x.shape
    H, _, r = Ak.shape
    lat = [torch.zeros((B, H, 64, r * bits // 8), dtype=torch.uint8, device="cuda") for _ in range(2)]
    sc = [torch.ones((B, H, 64), dtype=torch.float16, device="cuda") for _ in range(2)]
    n = cuda(np.asarray([3 + 7 * b for b in range(B)], np.int32))
    at = [int(v) for v in n]
    if T == 1:
        W.wsvd_latent_append(x[:, 0].contiguous(), Ak, Av, n, *lat, *sc, bits, blk)
    else:
        W.wsvd_latent_prefill(x, Ak, Av, n, *lat, *sc, bits, blk)
    rows = [torch.stack([a[b, :, at[b]:at[b] + T].transpose(0, 1) for b in range(B)]) for a in lat + sc]
    q = randn((B, H, 64), "bf16", 4)
    up = (randn((H, r, 64), "fp16", 5) * r ** -0.5).contiguous()
    return rows, W.wsvd_decode_attention(q, *lat, *sc, up, up, n, bits)


@pytest.mark.parametrize("call", [_paged, _contiguous])
@pytest.mark.parametrize("how", [NAN, INF, -INF, "overflow"])
@pytest.mark.parametrize("bits,r", [(8, 16), (8, 32), (8, 128), (4, 32), (4, 64)])
@pytest.mark.parametrize("B,T,blk", [(2, 1, 128), (2, 1, 1), (9, 1, 64), (2, 20, 128), (3, 45, 1)])
def test_a_nonfinite_token_stays_visible(call, how, bits, r, B, T, blk):
    H, E = 3, 256
    x = randn((B, T, E), "bf16", 1)
    Ak, Av = ((randn((H, E, r), "fp16", s) * E ** -0.5).contiguous() for s in (2, 3))
    b, t = B - 1, T // 2
    good, out = call(x, Ak, Av, bits, blk)
    bad, spoilt = call(_spoil(x, b, t, how), Ak, Av, bits, blk)
    assert torch.isfinite(out).all()
    assert not torch.isfinite(bad[2][b, t]).any() and not torch.isfinite(bad[3][b, t]).any()
    assert not torch.isfinite(spoilt[b]).any() and torch.equal(spoilt[:b], out[:b])
    others = torch.ones((B, T), dtype=torch.bool, device="cuda")
    others[b, t] = False
    for g, w in zip(bad, good):
        assert torch.equal(g[others].view(torch.uint8), w[others].view(torch.uint8))
