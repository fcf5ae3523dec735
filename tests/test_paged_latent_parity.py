"""GPU parity of the paged latent cache against the float64 oracle: the decode
over pages of codes and scales, at the sizes and contents where it can go wrong."""
import numpy as np
import pytest
import torch

import rank_kv_cache_wsvd_b200 as W
from oracle import paged_oracle as P
from paged_util import cuda, f64, owned, randn, table_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from rank_kv_cache_wsvd_b200 import build
    build.build()
    W.load()


def _cache(lens, H, r, bits, page, seed, caps=None, poison=True, **kw):
    """Pages of random codes; rows of nobody hold arbitrary codes and NaN scales."""
    table, pool = table_for(caps or lens, page, seed, **kw)
    g = torch.Generator().manual_seed(seed)
    mine = torch.from_numpy(owned(table, lens, page, pool))
    out = []
    for _ in range(2):
        top = 127 if bits == 8 else 7
        codes = torch.randint(-top, top + 1, (pool, H, page, r), generator=g, dtype=torch.int8)
        if bits == 4:
            codes = (codes[..., 0::2] & 15) | (codes[..., 1::2] << 4)
        scale = ((torch.rand((pool, H, page), generator=g) + 0.5) / top).half()
        if poison:
            scale = scale.masked_fill(~mine[:, None], float("nan"))
        out += [codes.view(torch.uint8).cuda(), scale.cuda()]
    return out[0], out[2], out[1], out[3], table


def _factors(H, r, Hd, seed):
    return [(randn((H, r, Hd), "fp16", seed + i) * r ** -0.5).contiguous() for i in range(2)]


def _decode(q, cache, Bk, Bv, lens, bits, **kw):
    lk, lv, sk, sv, table = cache
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = W.wsvd_decode_attention_paged(q, lk, lv, sk, sv, Bk, Bv, cuda(table), cuda(np.asarray(lens, np.int32)), bits,
                                        err=err, **kw)
    torch.cuda.synchronize()
    return out, int(err.item())


def _check(out, q, cache, Bk, Bv, lens, bits, scale=None, what=""):
    lk, lv, sk, sv, table = cache
    z = [np.nan_to_num(f64(t)) for t in (sk, sv)]
    ref, mass, wobble = P.latent_decode(f64(q), lk.cpu().numpy(), lv.cpu().numpy(), z[0], z[1], f64(Bk), f64(Bv), table,
                                        lens, bits, scale)
    # the largest value a row may add per column: full codes times the largest scale
    big = z[1].max() * (127 if bits == 8 else 7) * np.abs(f64(Bv)).sum(1)[None]
    n = max(max(lens), 1)
    allow = P.latent_allowance(mass, wobble, Bk.shape[1], q.shape[-1], big, n)
    got = out.double().cpu().numpy()
    assert np.all(np.isfinite(got)), f"{what}: non-finite output"
    worst = float((np.abs(got - ref) / allow).max())
    assert worst <= 1.0, f"{what}: {worst:.3f}x the allowance, largest error {np.abs(got - ref).max():.3e}"


LENS = [0, 1, 15, 16, 17, 31, 32, 33, 63, 65, 127, 128, 129, 300, 1, 0, 517]
RANKS = [(8, 16), (8, 32), (8, 64), (8, 128), (4, 32), (4, 64), (4, 128)]


@pytest.mark.parametrize("bits,r", RANKS)
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("Hd,dtype", [(32, "fp16"), (64, "bf16"), (128, "fp16"), (256, "bf16")])
def test_latent_decode_ragged_lengths(bits, r, page, Hd, dtype):
    H = 3
    cache = _cache(LENS, H, r, bits, page, seed=r + bits)
    Bk, Bv = _factors(H, r, Hd, 7)
    q = randn((len(LENS), H, Hd), dtype, 9)
    out, err = _decode(q, cache, Bk, Bv, LENS, bits)
    assert err == 0
    _check(out, q, cache, Bk, Bv, LENS, bits, what=f"int{bits} r{r} page{page} Hd{Hd}")


@pytest.mark.parametrize("bits,r", RANKS)
@pytest.mark.parametrize("B,H", [(1, 1), (2, 5), (70, 2)])
def test_latent_decode_many_splits_and_many_sequences(bits, r, B, H):
    lens = [6000 + 37 * b for b in range(B)] if B < 10 else [(b * 7) % 190 for b in range(B)]
    cache = _cache(lens, H, r, bits, 32, seed=B + r)
    Bk, Bv = _factors(H, r, 64, 17)
    q = randn((B, H, 64), "bf16", 19)
    out, err = _decode(q, cache, Bk, Bv, lens, bits)
    assert err == 0
    _check(out, q, cache, Bk, Bv, lens, bits, what=f"int{bits} r{r} B{B}")


@pytest.mark.parametrize("scale", [0.02, 2.0, -0.3])
@pytest.mark.parametrize("bits", [8, 4])
def test_latent_decode_softmax_scale(scale, bits):
    lens = [200, 77]
    cache = _cache(lens, 2, 32, bits, 64, seed=4)
    Bk, Bv = _factors(2, 32, 128, 5)
    q = randn((2, 2, 128), "fp16", 6)
    out, err = _decode(q, cache, Bk, Bv, lens, bits, softmax_scale=scale)
    assert err == 0
    _check(out, q, cache, Bk, Bv, lens, bits, scale, f"scale {scale}")


def test_latent_decode_extreme_codes_and_scales():
    """Codes at -128 and -8, zero scales, scales over eight orders of magnitude,
    zero and huge queries: the fixed-point sums neither overflow nor lose rows."""
    for bits, r in ((8, 32), (4, 64)):
        lens = [400, 260, 150]
        cache = _cache(lens, 2, r, bits, 16, seed=3)
        lk, lv, sk, sv, table = cache
        lk[:, :, ::3] = 0x80 if bits == 8 else 0x88
        lv[:, :, ::5] = 0x80 if bits == 8 else 0x88
        sv[:, :, ::2] *= 2.0 ** -12
        sv[:, 0, 1::4] *= 256
        sk[:, :, ::7] = 0
        Bk, Bv = _factors(2, r, 64, 8)
        q = randn((3, 2, 64), "bf16", 9)
        q[1] = 0
        q[2] *= 64
        out, err = _decode(q, cache, Bk, Bv, lens, bits)
        assert err == 0
        _check(out, q, cache, Bk, Bv, lens, bits, what=f"extreme int{bits}")


def test_latent_decode_nan_stays_where_it_is_seen():
    """A NaN query or a NaN scale of a visible row makes that head's output NaN
    and no other's."""
    lens, H = [130, 40], 3
    for bits, r in RANKS:
        cache = _cache(lens, H, r, bits, 16, seed=5, poison=False)
        lk, lv, sk, sv, table = cache
        Bk, Bv = _factors(H, r, 64, 6)
        q = randn((2, H, 64), "bf16", 7)
        good, _ = _decode(q, cache, Bk, Bv, lens, bits)
        q2, sk2, sv2 = q.clone(), sk.clone(), sv.clone()
        q2[0, 1, 5] = float("nan")
        sk2[table[0, 3], 2, 7] = float("nan")
        sv2[table[1, 2], 0, 7] = float("nan")   # row 39 of sequence 1
        bad, err = _decode(q2, (lk, lv, sk2, sv2, table), Bk, Bv, lens, bits)
        assert err == 0
        hit = torch.zeros((2, H), dtype=torch.bool, device="cuda")
        hit[0, 1] = hit[0, 2] = hit[1, 0] = True
        assert torch.isnan(bad[hit]).all() and torch.equal(bad[~hit], good[~hit])


def test_latent_decode_matches_the_contiguous_one():
    """The same rows in pages and contiguous: both agree with the float64 value
    under the framework's rule (1e-3 of the largest output, plus 1e-5)."""
    from gpu_util import assert_attention_close
    lens, H, Hd = [517, 64, 9], 4, 128
    for bits, r in RANKS:
        cache = _cache(lens, H, r, bits, 64, seed=77)
        lk, lv, sk, sv, table = cache
        Bk, Bv = _factors(H, r, Hd, 78)
        q = randn((3, H, Hd), "fp16", 79)
        flat = [torch.zeros((3, H, 520) + t.shape[3:], dtype=t.dtype, device="cuda") for t in (lk, lv, sk, sv)]
        for b, m in enumerate(lens):
            for l in range(m):
                for to, t in zip(flat, (lk, lv, sk, sv)):
                    to[b, :, l] = t[table[b, l // 64], :, l % 64]
        n = cuda(np.asarray(lens, np.int32))
        paged, err = _decode(q, cache, Bk, Bv, lens, bits)
        dense = W.wsvd_decode_attention(q, flat[0], flat[1], flat[2], flat[3], Bk, Bv, n, bits)
        assert err == 0
        assert_attention_close(f64(paged).reshape(-1, Hd), f64(dense).reshape(-1, Hd), f"int{bits} r{r}")


def test_latent_decode_bad_lengths_and_bad_pages():
    lens = [50, 40, 64, 33]
    cache = _cache(lens, 2, 32, 8, 16, seed=6, max_pages=4)
    Bk, Bv = _factors(2, 32, 64, 7)
    q = randn((4, 2, 64), "fp16", 8)
    good, err = _decode(q, cache, Bk, Bv, lens, 8)
    assert err == 0
    for bad in (-1, 65, 2 ** 31 - 1, -2 ** 31):
        out, err = _decode(q, cache, Bk, Bv, [50, bad, 64, 33], 8)
        assert err == 1 and (out[1] == 0).all() and torch.equal(out[[0, 2, 3]], good[[0, 2, 3]])
    for bad in (-1, cache[0].shape[0], 2 ** 31 - 1, -2 ** 31):
        table = cache[4].copy()
        table[2, 1] = bad
        out, err = _decode(q, cache[:4] + (table,), Bk, Bv, lens, 8)
        assert err == W.DEVERR_PAGE_RANGE and torch.equal(out[[0, 1, 3]], good[[0, 1, 3]])


def test_latent_decode_repeats_its_bits_shares_the_contiguous_workspace_and_replays():
    lens, H, r, Hd = [1900, 3, 700], 4, 32, 128
    cache = _cache(lens, H, r, 8, 64, seed=12, caps=[1920] * 3)
    Bk, Bv = _factors(H, r, Hd, 13)
    q = randn((3, H, Hd), "bf16", 14)
    want, _ = _decode(q, cache, Bk, Bv, lens, 8)
    ws = W.workspace(W.wsvd_decode_workspace_size(3, H, r))
    lk, lv, sk, sv, table = cache
    flat = [torch.zeros((3, H, 64) + t.shape[3:], dtype=t.dtype, device="cuda") for t in (lk, lv, sk, sv)]
    n3 = cuda(np.asarray([9, 64, 30], np.int32))
    dense = W.wsvd_decode_attention(q, *flat, Bk, Bv, n3, 8)
    for _ in range(3):
        out, _ = _decode(q, cache, Bk, Bv, lens, 8, workspace_buf=ws)
        assert torch.equal(out, want)
        assert torch.equal(W.wsvd_decode_attention(q, *flat, Bk, Bv, n3, 8, workspace_buf=ws), dense)
    tab, n = cuda(table), cuda(np.asarray(lens, np.int32))
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    outs = [W.wsvd_decode_attention_paged(q, lk, lv, sk, sv, Bk, Bv, tab, n, 8, stream=s) for _ in range(10) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    out, graph = torch.empty_like(want), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        W.wsvd_decode_attention_paged(q, lk, lv, sk, sv, Bk, Bv, tab, n, 8, out=out, workspace_buf=ws)
    for new in ([1900, 3, 700], [17, 0, 1], [640, 2, 129]):
        n.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        want, _ = _decode(q, cache, Bk, Bv, new, 8)
        assert torch.equal(out, want)


# ----------------------------------------------------------------------------- append
def _x(B, T, E, seed, dtype="bf16"):
    return randn((B, T, E), dtype, seed)


def _down(H, E, r, seed):
    return [(randn((H, E, r), "fp16", seed + i) * E ** -0.5).contiguous() for i in range(2)]


def _empty(pool, H, r, bits, page, seed):
    g = torch.Generator().manual_seed(seed)
    lat = [torch.randint(0, 256, (pool, H, page, r * bits // 8), generator=g, dtype=torch.uint8).cuda() for _ in range(2)]
    return lat + [torch.rand((pool, H, page), generator=g).half().cuda() for _ in range(2)]


def _contiguous_rows(x, Ak, Av, lens, bits, blk, one):
    """Codes and scales that the contiguous calls write for x, [B][H][T][..]."""
    B, T, E = x.shape
    H, _, r = Ak.shape
    cap = (max(lens) + T + 7) // 8 * 8
    lat = [torch.zeros((B, H, cap, r * bits // 8), dtype=torch.uint8, device="cuda") for _ in range(2)]
    sc = [torch.zeros((B, H, cap), dtype=torch.float16, device="cuda") for _ in range(2)]
    n = cuda(np.asarray(lens, np.int32))
    if one:
        W.wsvd_latent_append(x[:, 0].contiguous(), Ak, Av, n, *lat, *sc, bits, blk)
    else:
        W.wsvd_latent_prefill(x, Ak, Av, n, *lat, *sc, bits, blk)
    return [torch.stack([t[b, :, lens[b]:lens[b] + T] for b in range(B)]) for t in lat + sc]


def _check_rows(lk, lv, sk, sv, table, lens, x, Ak, Av, bits, page, blk):
    """The new rows against the float64 oracle's latents, with the framework's
    counted-tie rule: codes differ by one only within 1e-3 of a half step, scales
    by one fp16 step only within 2^-20 of its border."""
    import oracle as O
    from gpu_util import compare_codes, unpack
    B, T, E = x.shape
    H, _, r = Ak.shape
    ck, cv = O.latent_project(x.float().cpu().numpy().reshape(B * T, E), Ak.cpu().numpy(), Av.cpu().numpy(), blk)
    ties = 0
    for lat, sc, c in ((lk, sk, ck), (lv, sv, cv)):
        lat, sc = lat.cpu().numpy(), sc.cpu().numpy()
        at = [(table[b, (lens[b] + t) // page], (lens[b] + t) % page) for b in range(B) for t in range(T)]
        got_c = np.stack([unpack(lat[p, :, i], r, bits) for p, i in at])
        got_s = np.stack([sc[p, :, i] for p, i in at])
        want = [[O.quantize(c[m, h], bits) for h in range(H)] for m in range(B * T)]
        want_c = np.stack([[w[0] for w in row] for row in want])
        want_s = np.asarray([[w[1] for w in row] for row in want], np.float16)
        ties += sum(compare_codes(got_c, got_s, want_c, want_s, c, bits))
    # at most 2 * 1e-3 of the codes lie that near a half step, 2^-8 of the scales that near a border
    assert ties <= 4 + 2 * B * T * H * (r * 2e-3 + 2.0 ** -8)


@pytest.mark.parametrize("bits,r", [(8, 16), (8, 32), (8, 64), (8, 128), (4, 32), (4, 64), (4, 128)])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("B,T,H,E,blk", [(1, 1, 4, 256, 128), (5, 1, 3, 512, 64), (20, 1, 4, 256, 128), (2, 1, 8, 1024, 256),
                                         (3, 37, 4, 256, 128), (2, 130, 3, 192, 1), (1, 200, 16, 1024, 128),
                                         (40, 1, 16, 2048, 1024), (1, 70, 1, 64, 16), (9, 1, 2, 272, 16),
                                         (2, 201, 16, 128, 64), (1, 700, 16, 128, 32), (1, 1300, 3, 64, 64),
                                         (1, 300, 32, 256, 128)])
def test_latent_append_writes_its_rows_and_no_others(bits, r, page, B, T, H, E, blk):
    """Both paths (the GEMV; the tensor-core GEMM, whole and with E split over a
    cluster, tiles that run past the last head) against the oracle; one token as
    wsvd_latent_append writes it, bit for bit, where both run the GEMV; every
    other row of the pool keeps its bytes."""
    lens = [(b * 29) % 70 for b in range(B)]
    table, pool = table_for([a + T for a in lens], page, seed=r + B)
    lk, lv, sk, sv = _empty(pool, H, r, bits, page, 5)
    before = [t.clone() for t in (lk, lv, sk, sv)]
    x, (Ak, Av) = _x(B, T, E, 6), _down(H, E, r, 7)
    n = cuda(np.asarray(lens, np.int32))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    W.wsvd_latent_append_paged(x, Ak, Av, n, cuda(table), lk, lv, sk, sv, bits, blk, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and n.tolist() == [a + T for a in lens]
    _check_rows(lk, lv, sk, sv, table, lens, x, Ak, Av, bits, page, blk)
    if T == 1 and B <= 2:
        want = _contiguous_rows(x, Ak, Av, lens, bits, blk, True)
        for got, rows in zip((lk, lv, sk, sv), want):
            for b in range(B):
                assert torch.equal(got[table[b, lens[b] // page], :, lens[b] % page], rows[b, :, 0])
    mine = torch.zeros((pool, page), dtype=torch.bool)
    for b in range(B):
        for l in range(lens[b], lens[b] + T):
            mine[int(table[b, l // page]), l % page] = True
    for got, old in zip((lk, lv, sk, sv), before):
        same = (got.view(torch.uint8) == old.view(torch.uint8)).view(pool, H, page, -1).all(-1).all(1).cpu()
        assert (same | mine).all()


def test_latent_append_refuses_sequences_whole():
    for T in (1, 20):
        H, E, r, page = 2, 256, 16, 16
        lens = [0, 64 - T + 1, -1, 31, 2 ** 31 - 1, 5]
        table, pool = table_for([64] * 6, page, 5)
        table[3, 1 if T == 1 else 2] = pool + 4
        lk, lv, sk, sv = _empty(pool, H, r, 8, page, 8)
        before = [t.clone() for t in (lk, lv, sk, sv)]
        x, (Ak, Av) = _x(6, T, E, 9), _down(H, E, r, 10)
        n = cuda(np.asarray(lens, np.int32))
        to = torch.full_like(n, -7)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        W.wsvd_latent_append_paged(x, Ak, Av, n, cuda(table), lk, lv, sk, sv, 8, 128, seq_lens_out=to, err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 2 | 8
        assert n.tolist() == lens and to.tolist() == [T] + lens[1:5] + [5 + T]
        good = [0, 5]
        _check_rows(lk, lv, sk, sv, table[good], [lens[b] for b in good], x[good], Ak, Av, 8, page, 128)
        mine = torch.zeros((pool, page), dtype=torch.bool)
        for b in good:
            for l in range(lens[b], lens[b] + T):
                mine[int(table[b, l // page]), l % page] = True
        for got, old in zip((lk, lv, sk, sv), before):
            same = (got.view(torch.uint8) == old.view(torch.uint8)).view(pool, H, page, -1).all(-1).all(1).cpu()
            assert (same | mine).all()


def test_latent_append_and_decode_as_used():
    """A prompt block, then one token at a time through one workspace; every
    output against the oracle over the pages' codes, the codes against the
    oracle's latents; then captured steps."""
    B, H, E, r, Hd, page, bits, T = 3, 4, 512, 32, 64, 16, 8, 40
    table, pool = table_for([64] * B, page, 9)
    lk, lv, sk, sv = _empty(pool, H, r, bits, page, 11)
    tab, n = cuda(table), torch.zeros(B, dtype=torch.int32, device="cuda")
    Ak, Av = _down(H, E, r, 12)
    Bk, Bv = _factors(H, r, Hd, 14)
    ws = W.workspace(W.wsvd_latent_append_paged_workspace_size(B, T, E))
    dws = W.workspace(W.wsvd_decode_workspace_size(B, H, r))
    lens = [0] * B
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for i, t in enumerate([T] + [1] * 5):
        x, q = _x(B, t, E, 20 + i), randn((B, H, Hd), "bf16", 40 + i)
        W.wsvd_latent_append_paged(x, Ak, Av, n, tab, lk, lv, sk, sv, bits, 128, workspace_buf=ws, err=err)
        _check_rows(lk, lv, sk, sv, table, lens, x, Ak, Av, bits, page, 128)
        lens = [a + t for a in lens]
        out = W.wsvd_decode_attention_paged(q, lk, lv, sk, sv, Bk, Bv, tab, n, bits, workspace_buf=dws, err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0 and n.tolist() == lens
        _check(out, q, (lk, lv, sk, sv, table), Bk, Bv, lens, bits, what=f"step {i}")
    x, q, out = _x(B, 1, E, 60), randn((B, H, Hd), "bf16", 61), torch.empty((B, H, Hd), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        W.wsvd_latent_append_paged(x, Ak, Av, n, tab, lk, lv, sk, sv, bits, 128, workspace_buf=ws, err=err)
        W.wsvd_decode_attention_paged(q, lk, lv, sk, sv, Bk, Bv, tab, n, bits, out=out, workspace_buf=dws, err=err)
    for i in range(3):
        x.copy_(_x(B, 1, E, 70 + i))
        graph.replay()
        torch.cuda.synchronize()
        lens = [a + 1 for a in lens]
        assert int(err.item()) == 0 and n.tolist() == lens
        _check(out, q, (lk, lv, sk, sv, table), Bk, Bv, lens, bits, what=f"replay {i}")
    assert (ws[:256] == 0).all()


def test_latent_block_append_in_a_graph():
    """A captured block of tokens (two launches, tensor maps among their
    arguments) replays on new contents and lengths, and on two streams at once
    with a workspace each."""
    B, T, H, E, r, page = 2, 24, 8, 512, 32, 16
    table, pool = table_for([128] * B, page, 4)
    Ak, Av = _down(H, E, r, 1)
    x, n = _x(B, T, E, 2), torch.zeros(B, dtype=torch.int32, device="cuda")
    tab = cuda(table)
    ws = W.workspace(W.wsvd_latent_append_paged_workspace_size(B, T, E))
    cache = _empty(pool, H, r, 8, page, 3)
    err, graph = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        W.wsvd_latent_append_paged(x, Ak, Av, n, tab, *cache, 8, 128, workspace_buf=ws, err=err)
    lens = [0] * B
    for i in range(3):
        x.copy_(_x(B, T, E, 10 + i))
        graph.replay()
        torch.cuda.synchronize()
        _check_rows(*cache, table, lens, x, Ak, Av, 8, page, 128)
        lens = [a + T for a in lens]
        assert n.tolist() == lens and int(err.item()) == 0
    other = [t.clone() for t in cache]
    n1, n2 = torch.zeros_like(n), torch.zeros_like(n)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        n1.zero_(), n2.zero_()
        torch.cuda.synchronize()
        W.wsvd_latent_append_paged(x, Ak, Av, n1, tab, *cache, 8, 128, stream=s1)
        W.wsvd_latent_append_paged(x, Ak, Av, n2, tab, *other, 8, 128, stream=s2)
        torch.cuda.synchronize()
        assert n1.tolist() == n2.tolist() == [T] * B
    for a, b in zip(cache, other):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_latent_append_of_no_tokens_copies_the_lengths():
    H, E, r, page = 2, 256, 16, 16
    table, pool = table_for([64] * 2, page, 5)
    lk, lv, sk, sv = _empty(pool, H, r, 8, page, 8)
    Ak, Av = _down(H, E, r, 10)
    n, to = cuda(np.asarray([5, 9], np.int32)), torch.zeros(2, dtype=torch.int32, device="cuda")
    W.wsvd_latent_append_paged(torch.empty((2, 0, E), dtype=torch.bfloat16, device="cuda"), Ak, Av, n, cuda(table), lk, lv,
                               sk, sv, 8, 128, seq_lens_out=to)
    assert to.tolist() == [5, 9]


def _strip_allowance(q, cache, Bk, Bv, lens, bits):
    """How far the cut of the weights to 22 bits may take an output, [B][H][Hd]: a
    weight w_l = p_l s_l is off by half a step of 2^-21 of the largest of its strip
    (128, 64 or 32 rows, for rows of up to 32, 64 and 128 bytes), and meets its codes
    and B_v: sum over strips of 2^-22 max w . sum |code| |B_v|."""
    lk, lv, sk, sv, table = cache
    TS = {16: 128, 32: 128, 64: 64, 128: 32}[lk.shape[-1]]
    ck, cv = (P.latent_codes(t.cpu().numpy(), bits) for t in (lk, lv))
    sk, sv = (np.nan_to_num(f64(t))[..., None] for t in (sk, sv))
    out = np.zeros(q.shape)
    for b, n in enumerate(lens):
        K, C, S = P.rows(ck * sk, table, b, n), np.abs(P.rows(cv, table, b, n)), np.abs(P.rows(sv, table, b, n))
        for h in range(q.shape[1]):
            s = K[:, h] @ f64(Bk[h]) @ f64(q[b, h]) * q.shape[-1] ** -0.5
            p = np.exp(s - s.max())
            w = p / p.sum() * S[:, h, 0]
            for at in range(0, n, TS):
                out[b, h] += 2.0 ** -22 * w[at:at + TS].max() * C[at:at + TS, h].sum(0) @ np.abs(f64(Bv[h]))
    return out


def _uneven(bits, r, seed):
    """Value scales over seven orders of magnitude, by row, by strip and by head."""
    lens, H = [400, 261, 130], 4
    cache = _cache(lens, H, r, bits, 16, seed=seed, poison=False)
    table, sv = cache[4], cache[3]
    sv[:, 0] *= 2.0 ** -9                            # a whole head of small rows beside large ones
    sv[:, 1, ::2] *= 2.0 ** -8                       # every other row
    for b, n in enumerate(lens):
        for l in range(0, n, 2):
            if (l // 32) % 2:                        # whole strips
                sv[table[b, l // 16], 2, l % 16:l % 16 + 2] *= 2.0 ** -7
    sv[:, 3, 5::16] *= 512                           # a few rows far above the others
    return cache, lens, H


@pytest.mark.parametrize("equal", [False, True])
@pytest.mark.parametrize("bits,r", RANKS)
def test_latent_decode_keeps_small_rows_beside_large_ones(bits, r, equal):
    """A row is lost only where it lies 22 bits below the largest of its own strip;
    with a query of zeros (all rows weigh the same) the allowance has no share of the
    logits' rounding and lies below 1e-4 of what each output sums."""
    (cache, lens, H), Hd = _uneven(bits, r, r), 64
    lk, lv, sk, sv, table = cache
    Bk, Bv = _factors(H, r, Hd, 8)
    q = randn((3, H, Hd), "bf16", 9)
    if equal:
        q.zero_()
    out, err = _decode(q, cache, Bk, Bv, lens, bits)
    assert err == 0
    ref, mass, wobble = P.latent_decode(f64(q), lk.cpu().numpy(), lv.cpu().numpy(), f64(sk), f64(sv), f64(Bk), f64(Bv),
                                        table, lens, bits)
    allow = P.latent_allowance(mass, wobble, r, Hd, np.zeros(1), max(lens)) + _strip_allowance(q, cache, Bk, Bv, lens, bits)
    got = f64(out)
    assert np.isfinite(got).all() and (np.abs(got - ref) <= allow).all()
    # 2^-19 + (400 / 16 + 64 + 128) 2^-22 of the mass, and per strip at most 2^-22 x its rows x its largest share
    assert not equal or (allow <= 1e-4 * mass).all()


@pytest.mark.parametrize("bits,r", RANKS)
def test_latent_decode_of_scaled_values_has_scaled_bits(bits, r):
    """Value scales halved some times: every output halves as often, bit for bit, since
    weights are cut relative to their strip."""
    lens, H, Hd = [700, 33], 3, 64
    lk, lv, sk, sv, table = _cache(lens, H, r, bits, 16, seed=r, poison=False)
    Bk, Bv = _factors(H, r, Hd, 8)
    q = randn((2, H, Hd), "bf16", 9)
    sv = (sv.float() * 2.0 ** 8).half()
    want, _ = _decode(q, (lk, lv, sk, sv, table), Bk, Bv, lens, bits)
    by = torch.tensor([2.0 ** -3, 2.0 ** -9, 1.0], device="cuda")
    small = sv * by.half().view(1, H, 1)
    assert torch.equal(small.float() / by.view(1, H, 1), sv.float())  # no scale was rounded
    out, _ = _decode(q, (lk, lv, sk, small, table), Bk, Bv, lens, bits)
    assert torch.equal(out, want * by.view(1, H, 1))
