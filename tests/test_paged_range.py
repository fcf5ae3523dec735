"""Lengths at the end of the range (max_pages * page_size just below 2^31), through
page tables that name a few pages again and again."""
import numpy as np
import pytest
import torch

import rank_kv_cache_wsvd_b200 as W
from oracle import paged_oracle as P
from paged_util import cuda, f64, randn

pytestmark = pytest.mark.gpu
PAGE, MAX_PAGES, CYCLE = 16, (1 << 27) - 1, 64   # rows of a cycle: 1024
CAP = PAGE * MAX_PAGES
N = CAP - 3                                       # 13 rows of the last page, then 3 of nobody


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from rank_kv_cache_wsvd_b200 import build
    build.build()
    W.load()


@pytest.fixture(scope="module")
def table():
    """Pages 0 .. CYCLE - 1 in turn; the last entry is a page of its own."""
    t = (torch.arange(MAX_PAGES, dtype=torch.int32, device="cuda") % CYCLE).view(1, MAX_PAGES)
    t[0, -1] = CYCLE
    yield t
    del t
    torch.cuda.empty_cache()


def _seen(rows):
    """How often each row of the pool counts among the first `rows` rows (the last page apart)."""
    whole = min(rows, CAP - PAGE)
    per = np.full(CYCLE * PAGE, whole // (CYCLE * PAGE), np.float64)
    per[:whole % (CYCLE * PAGE)] += 1
    last = np.zeros(PAGE)
    last[:max(0, rows - (CAP - PAGE))] = 1
    return np.concatenate([per, last])


def _weighted(s, V, count):
    """sum_l count_l 2^.. softmax(s)_l V_l, and sum p |V|."""
    p = count * np.exp(s - s[count > 0].max())
    p /= p.sum()
    return p @ V, p @ np.abs(V)


# Every warp sums its strips one after another; a sequence is cut over at least 148 workers of 6 warps.
PER_WARP = N // (148 * 6)


@pytest.mark.parametrize("G", [1, 8])
def test_dense_decode_of_the_longest_sequence(table, G):
    """Two tokens of one and of eight heads; the last row, which only the second
    token sees, weighs about as much as all others, and rows past it are NaN."""
    Hd, Tq = 32, 2
    kp, vp = randn((CYCLE + 1, 1, PAGE, Hd), "bf16", 1), randn((CYCLE + 1, 1, PAGE, Hd), "bf16", 2)
    q = randn((1, Tq, G, Hd), "bf16", 3)
    q[:, :, 1:] = q[:, :, :1]
    last = (N - 1) % PAGE
    kp[-1, 0, last] = (q[0, 1, 0].float() * (21.5 * Hd ** 0.5 / q[0, 1, 0].float().square().sum())).bfloat16()
    kp[-1, 0, last + 1:], vp[-1, 0, last + 1:] = float("nan"), float("nan")
    lens = torch.tensor([N], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = W.paged_decode_attention(q, kp, vp, table, lens, err=err)
    assert int(err.item()) == 0 and torch.isfinite(out).all()
    K, V = (np.nan_to_num(f64(t[:, 0]).reshape(-1, Hd)) for t in (kp, vp))
    for t in range(Tq):
        qh = f64(q[0, t, 0])
        ref, mass = _weighted(K @ qh * Hd ** -0.5, V, _seen(N - Tq + 1 + t))
        wobble = (np.abs(K) @ np.abs(qh)).max() * Hd ** -0.5
        allow = P.decode_allowance(mass[None], np.asarray([wobble]), Hd, PER_WARP)
        for g in range(G):
            assert (np.abs(f64(out[0, t, g]) - ref) <= allow[0]).all()
    # the last row is there, and once
    assert np.abs(f64(out[0, 1, 0]) - f64(out[0, 0, 0])).max() > 0.2


@pytest.mark.parametrize("bits,r", [(8, 16), (4, 64)])
def test_latent_decode_of_the_longest_sequence(table, bits, r):
    Hd, Q = 32, 127 if bits == 8 else 7
    g = torch.Generator().manual_seed(1)
    lat = [torch.randint(0, 256, (CYCLE + 1, 1, PAGE, r * bits // 8), generator=g, dtype=torch.uint8).cuda() for _ in range(2)]
    sc = [((torch.rand((CYCLE + 1, 1, PAGE), generator=g) + 0.5) / Q).half().cuda() for _ in range(2)]
    Bk, Bv = ((randn((1, r, Hd), "fp16", s) * r ** -0.5).contiguous() for s in (5, 6))
    q = randn((1, 1, Hd), "bf16", 7)
    ck, cv = (P.latent_codes(t.cpu().numpy(), bits).reshape(-1, r) for t in lat)
    qp = f64(Bk[0]) @ f64(q[0, 0]) * Hd ** -0.5
    # the last row's scale gives it a logit of about 21.5
    last = (N - 1) % PAGE
    dot = float(ck.reshape(CYCLE + 1, PAGE, r)[-1, last] @ qp)
    sc[0][-1, 0, last] = 21.5 / dot
    for s in sc:
        s[-1, 0, last + 1:] = float("nan")
    lens = torch.tensor([N], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = lambda: W.wsvd_decode_attention_paged(q, *lat, *sc, Bk, Bv, table, lens, bits, err=err)
    out = call()
    assert int(err.item()) == 0
    sk, sv = (np.nan_to_num(f64(s).reshape(-1, 1)) for s in sc)
    V = (cv * sv) @ f64(Bv[0])
    ref, _ = _weighted(ck * sk @ qp, V, _seen(N))
    p = _seen(N) * np.exp(ck * sk @ qp - 21.5)
    mass = (p / p.sum()) @ (np.abs(cv * sv) @ np.abs(f64(Bv[0])))
    wobble = (np.abs(ck * sk).sum(1).max() * (np.abs(f64(Bk[0])) @ np.abs(f64(q[0, 0]))).max()) * Hd ** -0.5
    big = sv.max() * Q * np.abs(f64(Bv[0])).sum(0)
    allow = P.latent_allowance(mass[None, None], np.asarray([[wobble]]), r, Hd, big, PER_WARP)
    assert (np.abs(f64(out[0, 0]) - ref) <= allow[0, 0]).all()
    lens -= 1
    assert (call() - out).abs().max() > 0.2  # the last row is there


def test_appends_to_the_last_rows(table):
    """Rows up to the capacity are taken, one more is refused."""
    Hkv, Hd, H, E, r = 1, 32, 1, 64, 16
    kp = torch.zeros((CYCLE + 1, Hkv, PAGE, Hd), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    k = randn((1, 3, Hkv, Hd), "bf16", 1)
    for start, want in ((N, 0), (N + 1, W.DEVERR_CACHE_FULL)):
        lens = torch.tensor([start], dtype=torch.int32, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        W.paged_kv_append(k, k, kp, vp, table, lens, err=err)
        assert int(err.item()) == want and int(lens.item()) == (CAP if want == 0 else start)
    assert torch.equal(kp[-1, 0, 13:], k[0, :, 0]) and (kp[:-1] == 0).all() and (kp[-1, 0, :13] == 0).all()
    lat = [torch.zeros((CYCLE + 1, H, PAGE, r), dtype=torch.uint8, device="cuda") for _ in range(2)]
    sc = [torch.zeros((CYCLE + 1, H, PAGE), dtype=torch.float16, device="cuda") for _ in range(2)]
    A = randn((H, E, r), "fp16", 2)
    for T in (1, 3):
        for start, want in ((CAP - T, 0), (CAP - T + 1, W.DEVERR_CACHE_FULL)):
            lens = torch.tensor([start], dtype=torch.int32, device="cuda")
            err = torch.zeros(1, dtype=torch.int32, device="cuda")
            W.wsvd_latent_append_paged(randn((1, T, E), "bf16", 3), A, A, lens, table, *lat, *sc, 8, 64, err=err)
            assert int(err.item()) == want and int(lens.item()) == (CAP if want == 0 else start)
    assert (sc[0][-1, 0, 13:] != 0).all() and (sc[0][:-1] == 0).all() and (sc[0][-1, 0, :13] == 0).all()
