"""GPU parity of the paged dense cache (paged_kv_append, paged_decode_attention)
against the float64 oracle, at the sizes and contents where it can go wrong."""
import numpy as np
import pytest
import torch

import rank_kv_cache_wsvd_b200 as W
from oracle import paged_oracle as P
from paged_util import TYPES, cuda, f64, owned, randn, rope_table, table_for

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from rank_kv_cache_wsvd_b200 import build
    build.build()
    W.load()


def _cache(lens, Hkv, Hd, page, dtype, seed, caps=None, **kw):
    """Pages whose rows outside the sequences are NaN."""
    table, pool = table_for(caps or lens, page, seed, **kw)
    mine = torch.from_numpy(owned(table, lens, page, pool)).cuda()
    pages = []
    for i in range(2):
        p = randn((pool, Hkv, page, Hd), dtype, 10 * seed + i)
        pages.append(p.masked_fill(~mine[:, None, :, None], NAN))
    return pages[0], pages[1], table


def _check_decode(out, q, kp, vp, table, lens, scale=None, what=""):
    ref, mass, wobble = P.decode(f64(q), f64(kp), f64(vp), table, lens, scale)
    got = out.double().cpu().numpy()
    allow = P.decode_allowance(mass, wobble, q.shape[-1], max(max(lens), 1))
    assert np.all(np.isfinite(got)), f"{what}: non-finite output"
    worst = float((np.abs(got - ref) / allow).max())
    assert worst <= 1.0, f"{what}: {worst:.3f}x the allowance, largest error {np.abs(got - ref).max():.3e}"


def _decode(q, kp, vp, table, lens, **kw):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = W.paged_decode_attention(q, kp, vp, cuda(table), cuda(np.asarray(lens, np.int32)), err=err, **kw)
    torch.cuda.synchronize()
    return out, int(err.item())


LENS = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 130, 300, 1, 0, 517]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("Hd", [32, 64, 128, 256])
@pytest.mark.parametrize("page", [16, 256])
@pytest.mark.parametrize("Hkv,G,Tq", [(2, 1, 1), (1, 4, 1), (3, 7, 1), (1, 16, 1), (2, 4, 4), (1, 9, 7)])
def test_decode_ragged_lengths(dtype, Hd, page, Hkv, G, Tq):
    """Lengths of zero and one, around strips and pages; one to 63 queries a head;
    rows that belong to nobody, and page-table entries that no row reaches, are
    poisoned."""
    kp, vp, table = _cache(LENS, Hkv, Hd, page, dtype, seed=Hd + G + Tq)
    q = randn((len(LENS), Tq, Hkv * G, Hd), dtype, 5)
    out, err = _decode(q, kp, vp, table, LENS)
    assert err == 0
    _check_decode(out, q, kp.nan_to_num(0), vp.nan_to_num(0), table, LENS, what=f"{dtype} Hd{Hd} page{page} G{G} Tq{Tq}")


@pytest.mark.parametrize("page", [32, 64, 128])
@pytest.mark.parametrize("B,Hkv,G", [(1, 1, 8), (3, 2, 5), (70, 1, 2)])
def test_decode_many_splits_and_many_sequences(page, B, Hkv, G):
    """One head cut over the whole grid; more sequences than a warp's lanes."""
    lens = [3000 + 37 * b for b in range(B)] if B < 10 else [(b * 7) % 190 for b in range(B)]
    kp, vp, table = _cache(lens, Hkv, 64, page, "bf16", seed=B)
    q = randn((B, 1, Hkv * G, 64), "bf16", 3)
    out, err = _decode(q, kp, vp, table, lens)
    assert err == 0
    _check_decode(out, q, kp.nan_to_num(0), vp.nan_to_num(0), table, lens, what=f"B{B}")


@pytest.mark.parametrize("scale", [0.03, 1.0, -0.2])
def test_decode_softmax_scale_and_three_dimensional_q(scale):
    lens = [200, 77]
    kp, vp, table = _cache(lens, 2, 128, 64, "fp16", seed=4)
    q = randn((2, 8, 128), "fp16", 6)
    out, err = _decode(q, kp, vp, table, lens, softmax_scale=scale)
    assert err == 0 and out.shape == q.shape
    _check_decode(out[:, None], q[:, None], kp.nan_to_num(0), vp.nan_to_num(0), table, lens, scale, f"scale {scale}")


def test_decode_large_logits_and_outlier_rows():
    """Logits of some hundreds, one row far above the rest: nothing overflows and
    small weights keep their bits."""
    lens = [700]
    kp, vp, table = _cache(lens, 1, 128, 16, "fp16", seed=8)
    kp = kp * 20
    q = randn((1, 1, 4, 128), "fp16", 9)
    q[0, 0, 1] *= 0.01
    out, err = _decode(q, kp, vp, table, lens)
    assert err == 0
    _check_decode(out, q, kp.nan_to_num(0), vp.nan_to_num(0), table, lens, what="large logits")


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("Hd", [32, 64, 128, 256])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), NAN])
def test_decode_rows_a_query_does_not_see_never_reach_it(dtype, Hd, bad):
    """Keys and values of later tokens hold infinities or NaN: only the queries
    that see them may notice."""
    lens, Tq, G = [18, 40, 3, 129], 4, 3
    kp, vp, table = _cache(lens, 2, Hd, 16, dtype, seed=21)
    clean = (kp.clone(), vp.clone())
    for b, n in enumerate(lens):
        for back in (1, 2):  # the last two rows: seen by tokens 3, and by 2 and 3
            l = n - back
            kp[table[b, l // 16], :, l % 16, ::2] = bad
            vp[table[b, l // 16], :, l % 16] = bad
    q = randn((len(lens), Tq, 2 * G, Hd), dtype, 22)
    out, err = _decode(q, kp, vp, table, lens)
    assert err == 0
    # tokens 0 and 1 see rows < n - 3 and < n - 2
    want, _ = _decode(q, clean[0], clean[1], table, lens)
    got, want = out[:, :2], want[:, :2]
    assert torch.isfinite(got).all()
    ref, mass, wobble = P.decode(f64(q), f64(clean[0].nan_to_num(0)), f64(clean[1].nan_to_num(0)), table, lens)
    allow = P.decode_allowance(mass, wobble, Hd, max(lens))[:, :2]
    assert (np.abs(got.double().cpu().numpy() - ref[:, :2]) <= allow).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_decode_nan_stays_where_it_is_seen(dtype):
    """A NaN query makes its own output NaN; a NaN key or value of a visible row
    those of its KV head."""
    lens = [70, 33]
    kp, vp, table = _cache(lens, 3, 64, 16, dtype, seed=5)
    q = randn((2, 1, 12, 64), dtype, 6)
    good, _ = _decode(q, kp, vp, table, lens)
    q2, kp2, vp2 = q.clone(), kp.clone(), vp.clone()
    q2[0, 0, 5, 9] = NAN
    kp2[table[0, 2], 2, 3, 1] = NAN
    vp2[table[1, 2], 0, 0, 17] = NAN  # row 32 of sequence 1
    bad, err = _decode(q2, kp2, vp2, table, lens)
    assert err == 0
    hit = torch.zeros_like(good, dtype=torch.bool)
    hit[0, 0, 5] = hit[0, 0, 8:12] = True
    hit[1, 0, 0:4, 17] = True
    assert torch.isnan(bad[hit]).all() and torch.equal(bad[~hit], good[~hit])


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("Hd", [32, 64, 128, 256])
@pytest.mark.parametrize("G,Tq", [(9, 1), (4, 4), (5, 7)])
@pytest.mark.parametrize("scale", [-0.2, 0.5])
def test_decode_many_queries_a_head_with_either_sign_of_scale(dtype, Hd, G, Tq, scale):
    """Nine queries and more, whose products turn the sign of the scale into the
    queries; logits of some tens, so that the running maximum moves."""
    lens = [200, 77, 2]
    kp, vp, table = _cache(lens, 2, Hd, 16, dtype, seed=31)
    q = randn((3, Tq, 2 * G, Hd), dtype, 32)
    out, err = _decode(q, kp, vp, table, lens, softmax_scale=scale)
    assert err == 0
    _check_decode(out, q, kp.nan_to_num(0), vp.nan_to_num(0), table, lens, scale, f"Hd{Hd} G{G} Tq{Tq} scale {scale}")


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("Hd", [32, 64, 128])
@pytest.mark.parametrize("G,Tq", [(1, 3), (16, 2), (7, 4)])
def test_decode_wild_later_rows_with_few_and_many_queries(dtype, Hd, G, Tq):
    """The last row holds infinities and NaN: only the last token's queries see it."""
    lens = [18, 64, 131]
    kp, vp, table = _cache(lens, 2, Hd, 32, dtype, seed=41)
    clean = (kp.clone(), vp.clone())
    for i, n in enumerate(lens):
        l = n - 1
        kp[table[i, l // 32], :, l % 32] = (float("inf"), float("-inf"), NAN)[i]
        vp[table[i, l // 32], :, l % 32] = (NAN, float("inf"), float("-inf"))[i]
    q = randn((3, Tq, 2 * G, Hd), dtype, 42)
    out, err = _decode(q, kp, vp, table, lens)
    assert err == 0
    got = out[:, : Tq - 1].double().cpu().numpy()
    ref, mass, wobble = P.decode(f64(q), f64(clean[0].nan_to_num(0)), f64(clean[1].nan_to_num(0)), table, lens)
    allow = P.decode_allowance(mass, wobble, Hd, max(lens))[:, : Tq - 1]
    assert np.isfinite(got).all() and (np.abs(got - ref[:, : Tq - 1]) <= allow).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_decode_nan_stays_with_its_query_of_sixteen(dtype):
    """A NaN query among sixteen of a head makes its own output NaN and no other."""
    lens = [70, 33]
    kp, vp, table = _cache(lens, 2, 64, 16, dtype, seed=5)
    q = randn((2, 1, 32, 64), dtype, 6)
    good, _ = _decode(q, kp, vp, table, lens)
    q2 = q.clone()
    q2[0, 0, 5, 9] = q2[1, 0, 29, 60] = NAN
    bad, err = _decode(q2, kp, vp, table, lens)
    assert err == 0
    hit = torch.zeros_like(good, dtype=torch.bool)
    hit[0, 0, 5] = hit[1, 0, 29] = True
    assert torch.isnan(bad[hit]).all() and torch.equal(bad[~hit], good[~hit])


def test_decode_shared_prefix_pages():
    lens = [100, 90, 64]
    table, pool = table_for(lens, 32, 3, shared=2)
    kp, vp = randn((pool, 2, 32, 128), "bf16", 31), randn((pool, 2, 32, 128), "bf16", 32)
    q = randn((3, 1, 8, 128), "bf16", 33)
    out, err = _decode(q, kp, vp, table, lens)
    assert err == 0
    _check_decode(out, q, kp, vp, table, lens, what="shared prefix")


def test_decode_pages_past_32_bit_offsets():
    """The pool holds more than 2^32 values; the rows lie at its end."""
    Hkv, page, Hd = 8, 256, 128
    pool = (1 << 32) // (Hkv * page * Hd) + 8
    kp = torch.zeros((pool, Hkv, page, Hd), dtype=torch.float16, device="cuda")
    vp = torch.zeros_like(kp)
    kp[-4:] = randn((4, Hkv, page, Hd), "fp16", 1)
    vp[-4:] = randn((4, Hkv, page, Hd), "fp16", 2)
    table = np.array([[pool - 1, pool - 3], [pool - 4, pool - 2]], np.int32)
    lens = [300, 511]
    q = randn((2, 1, 16, Hd), "fp16", 3)
    out, err = _decode(q, kp, vp, table, lens)
    assert err == 0
    small = table - (pool - 4)
    _check_decode(out, q, kp[-4:], vp[-4:], small, lens, what="far pages")
    k = randn((2, 3, Hkv, Hd), "fp16", 4)
    new = cuda(np.array([200, 400], np.int32))
    W.paged_kv_append(k, k, kp, vp, cuda(table), new)
    for b, at in enumerate((200, 400)):
        for t in range(3):
            assert torch.equal(kp[table[b, (at + t) // page], :, (at + t) % page], k[b, t])
    assert new.tolist() == [203, 403]


def test_decode_bad_lengths_and_bad_pages():
    """Lengths out of range give zeros and LEN_RANGE, page ids out of range set
    PAGE_RANGE; the other sequences' outputs keep their bits."""
    lens = [50, 40, 64, 33]
    kp, vp, table = _cache(lens, 2, 64, 16, "fp16", seed=6, max_pages=4)
    q = randn((4, 1, 4, 64), "fp16", 7)
    good, err = _decode(q, kp, vp, table, lens)
    assert err == 0
    for bad in (-1, 65, 2 ** 31 - 1, -2 ** 31):
        out, err = _decode(q, kp, vp, table, [50, bad, 64, 33])
        assert err == 1 and (out[1] == 0).all() and torch.equal(out[[0, 2, 3]], good[[0, 2, 3]])
    for bad in (-1, kp.shape[0], 2 ** 31 - 1, -2 ** 31):
        broken = table.copy()
        broken[2, 1] = bad
        out, err = _decode(q, kp, vp, broken, lens)
        assert err == W.DEVERR_PAGE_RANGE and torch.equal(out[[0, 1, 3]], good[[0, 1, 3]])


def test_decode_repeats_its_bits_and_leaves_its_workspace_ready():
    """One workspace serves calls of other sizes in turn; every result has the
    bits of a call with a fresh one; nothing behind `out` is written."""
    shapes = [([1700, 3], 2, 8, 1, 128), ([5, 900, 0, 31], 2, 4, 4, 128), ([2000], 1, 16, 1, 128)]
    ws = W.workspace(max(W.paged_decode_workspace_size(len(n), Tq, Hkv * G, Hkv, Hd) for n, Hkv, G, Tq, Hd in shapes))
    for rep in range(2):
        for i, (lens, Hkv, G, Tq, Hd) in enumerate(shapes):
            kp, vp, table = _cache(lens, Hkv, Hd, 64, "bf16", seed=40 + i)
            q = randn((len(lens), Tq, Hkv * G, Hd), "bf16", 50 + i)
            fresh, _ = _decode(q, kp, vp, table, lens)
            guard = torch.full((fresh.numel() + 64,), 7.0, device="cuda")
            ws_i = ws[:W.paged_decode_workspace_size(len(lens), Tq, Hkv * G, Hkv, Hd)].zero_() if rep == 0 else \
                W.workspace(W.paged_decode_workspace_size(len(lens), Tq, Hkv * G, Hkv, Hd))
            for _ in range(3):
                out, _ = _decode(q, kp, vp, table, lens, workspace_buf=ws_i, out=guard[:fresh.numel()].view(fresh.shape))
                assert torch.equal(out, fresh)
            assert (guard[fresh.numel():] == 7).all()


def test_decode_on_other_streams_and_in_graphs():
    """Two streams with a workspace each at once; a captured call replays on new
    contents and lengths."""
    lens = [1000, 200]
    kp, vp, table = _cache(lens, 2, 128, 64, "bf16", seed=60, caps=[1024, 1024])
    q = randn((2, 1, 16, 128), "bf16", 61)
    want, _ = _decode(q, kp, vp, table, lens)
    tab, n = cuda(table), cuda(np.asarray(lens, np.int32))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [[W.paged_decode_attention(q, kp, vp, tab, n, stream=s) for s in streams] for _ in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for row in outs for o in row)

    ws = W.workspace(W.paged_decode_workspace_size(2, 1, 16, 2, 128))
    out, graph = torch.empty_like(want), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        W.paged_decode_attention(q, kp, vp, tab, n, out=out, workspace_buf=ws)
    for new in ([1000, 200], [17, 0], [640, 199]):
        n.copy_(torch.tensor(new, dtype=torch.int32))
        q.copy_(randn(tuple(q.shape), "bf16", sum(new)))
        graph.replay()
        want, _ = _decode(q, kp, vp, table, new)
        assert torch.equal(out, want)


# ----------------------------------------------------------------------------- append
def _append_case(B, T, Hq, Hkv, Hd, page, dtype, lens, seed, news=None, fused=True, extra=0):
    caps = [max(0, n) + (T if news is None else max(0, m)) for n, m in zip(lens, news or [0] * B)]
    table, pool = table_for(caps, page, seed)
    kp, vp = randn((pool, Hkv, page, Hd), dtype, seed + 1), randn((pool, Hkv, page, Hd), dtype, seed + 2)
    qkv = randn((B, T, (Hq + 2 * Hkv) * Hd + extra), dtype, seed + 3)
    q = qkv[..., :Hq * Hd].unflatten(-1, (Hq, Hd))
    k = qkv[..., Hq * Hd:(Hq + Hkv) * Hd].unflatten(-1, (Hkv, Hd))
    v = qkv[..., (Hq + Hkv) * Hd:(Hq + 2 * Hkv) * Hd].unflatten(-1, (Hkv, Hd))
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    return q, k, v, kp, vp, table


def _check_append(kp, vp, qo, ref, before, dtype, magnitude_q, mine):
    """v, copies and rows not appended keep their bits; rotated values are off by
    half a step of their type (2^-25 at least: fp16 denormals) plus fp32 rounding of
    a product and of a product and sum, each at most 2^-24 of twice the largest."""
    half = torch.finfo(TYPES[dtype]).eps / 2
    rk, rv, rq, _ = ref
    assert np.array_equal(f64(vp), rv)
    big = np.abs(rk).max()
    err = np.abs(f64(kp) - rk)
    assert (err <= half * np.abs(rk) + (2.0 ** -21 * big + 2.0 ** -25) * mine).all()  # mine: 0 where nothing was appended
    if rq is not None:
        assert (np.abs(f64(qo) - rq) <= half * np.abs(rq) + 2.0 ** -21 * magnitude_q + 2.0 ** -25).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("Hd,rot", [(32, 32), (64, 16), (64, 64), (128, 128), (128, 64), (256, 256), (128, 0)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("B,T,Hq,Hkv,page", [(3, 1, 8, 2, 16), (2, 37, 6, 3, 16), (1, 70, 4, 4, 64)])
def test_append_rotates_and_stores(dtype, Hd, rot, inter, B, T, Hq, Hkv, page):
    lens = [5, 31, 0][:B]
    q, k, v, kp, vp, table = _append_case(B, T, Hq, Hkv, Hd, page, dtype, lens, seed=Hd + rot + T, extra=16)
    cs = rope_table(256, rot) if rot else None
    ref = P.kv_append(f64(k), f64(v), f64(q), f64(kp), f64(vp), table, lens, f64(cs) if rot else None, rot, inter)
    before = kp.clone(), vp.clone()
    n = cuda(np.asarray(lens, np.int32))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    qo = W.paged_kv_append(k, v, kp, vp, cuda(table), n, q=q, cos_sin=cs, interleaved=inter, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and n.tolist() == [a + T for a in lens]
    mine = (f64(before[0]) != ref[0]).any(axis=-1, keepdims=True)
    _check_append(kp, vp, qo, ref, before, dtype, np.abs(f64(q)).max(), mine)
    if rot == 0:
        assert torch.equal(qo, q.contiguous())


@pytest.mark.parametrize("out_of_place", [False, True])
def test_append_padded_batch(out_of_place):
    """Ragged blocks: padding is not stored, its q_out rows are zero, its inputs
    may hold NaN; a sequence may get nothing at all."""
    B, T, Hq, Hkv, Hd, page = 5, 150, 4, 2, 64, 32
    lens, news = [0, 7, 100, 3, 64], [150, 0, 1, 77, 149]
    q, k, v, kp, vp, table = _append_case(B, T, Hq, Hkv, Hd, page, "bf16", lens, 70, news, fused=False)
    for b in range(B):
        q[b, news[b]:], k[b, news[b]:], v[b, news[b]:] = NAN, NAN, NAN
    cs = rope_table(512, 64)
    ref = P.kv_append(f64(k), f64(v), f64(q), f64(kp), f64(vp), table, lens, f64(cs), 64, False, news)
    before = kp.clone(), vp.clone()
    n = cuda(np.asarray(lens, np.int32))
    to = torch.full_like(n, -5) if out_of_place else n
    ws = W.workspace(W.paged_kv_append_workspace_size(B))
    qo = W.paged_kv_append(k, v, kp, vp, cuda(table), n, q=q, cos_sin=cs, new_lens=cuda(np.asarray(news, np.int32)),
                           seq_lens_out=to, workspace_buf=ws)
    torch.cuda.synchronize()
    assert to.tolist() == [a + m for a, m in zip(lens, news)]
    assert not out_of_place or n.tolist() == lens
    assert (ws == 0).all()
    mine = (f64(before[0]) != ref[0]).any(axis=-1, keepdims=True)
    _check_append(kp, vp, qo, ref, before, "bf16", 6.0, mine)


def test_append_without_queries_and_with_queries_in_place():
    B, T, Hq, Hkv, Hd, page = 2, 9, 4, 2, 128, 16
    lens = [10, 0]
    q, k, v, kp, vp, table = _append_case(B, T, Hq, Hkv, Hd, page, "fp16", lens, 80, fused=False)
    cs, tab = rope_table(64, 128), cuda(table)
    k1, v1 = kp.clone(), vp.clone()
    qo = W.paged_kv_append(k, v, kp, vp, tab, cuda(np.asarray(lens, np.int32)), q=q, cos_sin=cs)
    assert W.paged_kv_append(k, v, k1, v1, tab, cuda(np.asarray(lens, np.int32)), cos_sin=cs) is None
    assert torch.equal(kp, k1) and torch.equal(vp, v1)
    same = q.clone()
    W.paged_kv_append(k, v, k1, v1, tab, cuda(np.asarray(lens, np.int32)), q=same, q_out=same, cos_sin=cs)
    assert torch.equal(same, qo)


def test_append_refuses_sequences_whole():
    """Full, negative and unplaceable sequences, blocks past the angle table and
    bad counts: nothing of them is stored, q_out is zero, the length is kept; the
    others are appended."""
    B, T, Hkv, Hd, page = 7, 20, 2, 64, 16
    lens = [0, 45, -1, 30, 10, 2 ** 31 - 1, 3]
    news = [20, 20, 20, 20, 21, 20, -1]
    table, pool = table_for([64] * B, page, 5)
    table[3, 2] = pool + 4  # rows 32 .. 47 of sequence 3
    kp, vp = randn((pool, Hkv, page, Hd), "fp16", 1), randn((pool, Hkv, page, Hd), "fp16", 2)
    k, v, q = (randn((B, T, Hkv, Hd), "fp16", 3 + i) for i in range(3))
    before = kp.clone(), vp.clone()
    n = cuda(np.asarray(lens, np.int32))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    qo = W.paged_kv_append(k, v, kp, vp, cuda(table), n, q=q, new_lens=cuda(np.asarray(news, np.int32)), err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 1 | 2 | 8
    assert n.tolist() == [20] + lens[1:]
    assert torch.equal(qo[0], q[0]) and (qo[1:] == 0).all()
    for l in range(20):
        before[0][table[0, l // page], :, l % page] = k[0, l]
        before[1][table[0, l // page], :, l % page] = v[0, l]
    assert torch.equal(kp, before[0]) and torch.equal(vp, before[1])
    # positions without an angle: max_pos 25 holds rows < 25
    n = cuda(np.asarray([6, 5, 5, 5, 5, 5, 5], np.int32))
    err.zero_()
    table[3, 2] = table[3, 1]
    W.paged_kv_append(k, v, kp, vp, cuda(table), n, cos_sin=rope_table(25, 64), err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 2 and n.tolist() == [6] + [25] * 6


def test_append_and_decode_as_used():
    """A prompt in two blocks, then one token at a time: every output and the
    final cache against the oracle; then the same tokens as a captured step."""
    B, Hq, Hkv, Hd, page, steps = 3, 8, 2, 64, 16, 6
    cs = rope_table(512, Hd)
    blocks = [(33, [33, 5, 17]), (20, [1, 20, 0])] + [(1, None)] * steps
    table, pool = table_for([64] * B, page, 9)
    kp, vp = (torch.full((pool, Hkv, page, Hd), NAN, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    tab, n = cuda(table), torch.zeros(B, dtype=torch.int32, device="cuda")
    rk, rv, lens = f64(kp), f64(vp), [0] * B
    for i, (T, news) in enumerate(blocks):
        q, k, v = (randn((B, T, h, Hd), "bf16", 100 * i + j) for j, h in enumerate((Hq, Hkv, Hkv)))
        new = cuda(np.asarray(news, np.int32)) if news else None
        qo = W.paged_kv_append(k, v, kp, vp, tab, n, q=q, cos_sin=cs, new_lens=new)
        rk, rv, rq, lens = P.kv_append(f64(k), f64(v), f64(q), rk, rv, table, lens, f64(cs), Hd, False, news)
        assert n.tolist() == list(lens)
        if T == 1:
            out, err = _decode(qo, kp, vp, table, lens)
            assert err == 0
            _check_decode(out, qo, kp.nan_to_num(0), vp.nan_to_num(0), table, lens, what=f"step {i}")
            # against the fp64 cache: the keys' and queries' rounding (2^-9 relative, 2^-8 of a logit's
            # magnitude for the two) moves a weight by a factor within 4 * 2^-8 * wobble
            ref, mass, wobble = P.decode(rq, np.nan_to_num(rk), np.nan_to_num(rv), table, lens)
            assert (np.abs(out.double().cpu().numpy() - ref) <= 2 * mass * 2.0 ** -6 * wobble[..., None] + 1e-5).all()
    # one more step, captured: the graph appends and attends on every replay
    q, k, v = (randn((B, 1, h, Hd), "bf16", 900 + j) for j, h in enumerate((Hq, Hkv, Hkv)))
    ws = [W.workspace(W.paged_kv_append_workspace_size(B)), W.workspace(W.paged_decode_workspace_size(B, 1, Hq, Hkv, Hd))]
    kept, qo, out = n.clone(), torch.empty_like(q), torch.empty((B, 1, Hq, Hd), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        W.paged_kv_append(k, v, kp, vp, tab, n, q=q, q_out=qo, cos_sin=cs, workspace_buf=ws[0])
        W.paged_decode_attention(qo, kp, vp, tab, n, out=out, workspace_buf=ws[1])
    for i in range(3):
        q.copy_(randn(tuple(q.shape), "bf16", 950 + i))
        graph.replay()
        torch.cuda.synchronize()
        lens = [a + 1 for a in lens]
        assert n.tolist() == lens
        _check_decode(out, qo, kp.nan_to_num(0), vp.nan_to_num(0), table, lens, what=f"replay {i}")


def test_calls_refuse_wrong_tensors():
    """Types, shapes and layouts that do not fit raise before a launch; tensors of
    another device too."""
    lens = [20, 9]
    kp, vp, table = _cache(lens, 2, 64, 16, "fp16", seed=1)
    q, tab, n = randn((2, 4, 64), "fp16", 2), cuda(table), cuda(np.asarray(lens, np.int32))
    out = torch.empty((2, 4, 64), device="cuda")
    call = lambda **kw: W.paged_decode_attention(**{**dict(q=q, k_pages=kp, v_pages=vp, block_table=tab, seq_lens=n), **kw})
    for kw in (dict(q=q.float()), dict(q=q.bfloat16()), dict(k_pages=kp[:, :1]), dict(v_pages=vp.transpose(1, 2)),
               dict(v_pages=vp[:-1]), dict(block_table=tab.long()), dict(block_table=tab[:1]), dict(seq_lens=n[:1]),
               dict(seq_lens=n.long()), dict(out=out[:, :2]), dict(out=out.half()), dict(q=q.cpu()), dict(seq_lens=n.cpu()),
               dict(q=torch.cat([q, q], 2)[..., ::2]), dict(workspace_buf=torch.zeros(4, device="cuda")),
               dict(workspace_buf=W.workspace(64)), dict(softmax_scale=0.0, err=torch.zeros(1, device="cuda"))):
        with pytest.raises(W.WsvdError):
            call(**kw)
    with pytest.raises(W.WsvdError):  # three query heads over two
        call(q=q[:, :3].contiguous())
    k = randn((2, 1, 2, 64), "fp16", 3)
    put = lambda **kw: W.paged_kv_append(**{**dict(k=k, v=k, k_pages=kp, v_pages=vp, block_table=tab, seq_lens=n), **kw})
    before = n.clone(), kp.clone()
    for kw in (dict(v=k[:, :, :1]), dict(v=k.bfloat16()), dict(q=q[:, None].float()), dict(q_out=q[:, None]),
               dict(cos_sin=rope_table(64, 64).half()), dict(cos_sin=rope_table(64, 24)), dict(new_lens=n.long()),
               dict(seq_lens_out=n[:1]), dict(k_pages=kp.float()), dict(q=q[:, None], q_out=kp.view(-1)[:512].view(2, 1, 4, 64))):
        with pytest.raises(W.WsvdError):
            put(**kw)
    torch.cuda.synchronize()
    assert torch.equal(n, before[0]) and torch.equal(kp.view(torch.int16), before[1].view(torch.int16))
    out = call()
    assert torch.isfinite(out).all()


def test_decode_thousands_of_short_sequences():
    B, Hkv = 4500, 1
    lens = [(b * 5) % 23 for b in range(B)]
    kp, vp, table = _cache(lens, Hkv, 32, 16, "fp16", seed=3)
    q = randn((B, 1, 2, 32), "fp16", 4)
    out, err = _decode(q, kp, vp, table, lens)
    assert err == 0
    some = list(range(0, 60)) + list(range(B - 60, B))
    _check_decode(out[some], q[some], kp.nan_to_num(0), vp.nan_to_num(0), table[some], [lens[b] for b in some], what="many")
    assert (out[[b for b in range(B) if lens[b] == 0]] == 0).all()
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("Hd,G,Tq", [(32, 8, 1), (64, 1, 1), (64, 2, 3), (128, 7, 1), (256, 4, 2)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_decode_many_short_sequences(Hd, G, Tq, dtype):
    """Over 512 units of few strips, where every warp works for itself: whole units,
    cut ones, sequences without rows, bad lengths and bad pages among them; the
    same bits again, also when long sequences (CTAs as workers) used the
    workspace in between."""
    B, Hkv = 130, 4
    lens = [(b * 37) % 260 if b % 9 else 0 for b in range(B)]
    lens[5] = 3000
    kp, vp, table = _cache(lens, Hkv, Hd, 32, dtype, seed=Hd + G)
    q = randn((B, Tq, Hkv * G, Hd), dtype, 4)
    ws = W.workspace(W.paged_decode_workspace_size(B, Tq, Hkv * G, Hkv, Hd))
    out, err = _decode(q, kp, vp, table, lens, workspace_buf=ws)
    assert err == 0
    some = list(range(0, 24)) + [60, 99, 129]
    _check_decode(out[some], q[some], kp.nan_to_num(0), vp.nan_to_num(0), table[some], [lens[b] for b in some],
                  what=f"Hd{Hd} G{G} Tq{Tq}")
    assert (out[[b for b in range(B) if lens[b] == 0]] == 0).all() and torch.isfinite(out).all()
    long = [3000] * 4 + [0] * (B - 4)
    big, err = _decode(q, kp, vp, np.repeat(table[5:6], B, 0), long, workspace_buf=ws)
    assert err == 0
    again, _ = _decode(q, kp, vp, table, lens, workspace_buf=ws)
    assert torch.equal(again, out)
    broken, odd = table.copy(), list(lens)
    broken[10, 1], odd[11] = kp.shape[0], -3
    bad, err = _decode(q, kp, vp, broken, odd)
    rest = [b for b in range(B) if b not in (10, 11)]
    assert err == W.DEVERR_PAGE_RANGE | 1 and (bad[11] == 0).all()
    _check_decode(bad[rest[:20]], q[rest[:20]], kp.nan_to_num(0), vp.nan_to_num(0), table[rest[:20]],
                  [lens[b] for b in rest[:20]], what="beside bad ones")


def test_paged_decode_matches_the_contiguous_one():
    """The same rows in pages and in the dense cache: both within the allowance
    of the float64 value."""
    lens, H, Hd = [513, 64, 9], 4, 128
    kp, vp, table = _cache(lens, H, Hd, 64, "fp16", seed=77)
    q = randn((3, H, Hd), "fp16", 78)
    K, V = (torch.zeros((3, H, 520, Hd), dtype=torch.float16, device="cuda") for _ in range(2))
    for b, m in enumerate(lens):
        for l in range(m):
            K[b, :, l], V[b, :, l] = kp[table[b, l // 64], :, l % 64], vp[table[b, l // 64], :, l % 64]
    paged, err = _decode(q, kp, vp, table, lens)
    dense = W.dense_decode_attention(q, K, V, cuda(np.asarray(lens, np.int32)))
    ref, mass, wobble = P.decode(f64(q)[:, None], f64(kp.nan_to_num(0)), f64(vp.nan_to_num(0)), table, lens)
    allow = P.decode_allowance(mass, wobble, Hd, 520)[:, 0]
    assert err == 0 and (np.abs(f64(paged) - ref[:, 0]) <= allow).all() and (np.abs(f64(dense) - ref[:, 0]) <= allow).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("Hd", [32, 64, 128, 256])
@pytest.mark.parametrize("G,Tq", [(2, 1), (16, 1), (3, 2)])
@pytest.mark.parametrize("scale", [0.0, -0.2])
def test_decode_infinite_keys_and_values_that_are_seen(dtype, Hd, G, Tq, scale):
    """Infinite keys go by the formula: a logit of minus infinity weighs nothing, one
    of plus infinity or NaN (and no finite logit at all) makes the output NaN.  An
    infinite value leaves its column not finite, and the others as they were."""
    lens = [40, 70, 33, 2]
    kp, vp, table = _cache(lens, 1, Hd, 16, dtype, seed=51)
    kp, vp = kp.nan_to_num(0), vp.nan_to_num(0)
    q = randn((4, Tq, G, Hd), dtype, 52)
    q[:, :, 0, 3] = 1.0
    q[:, :, 1:, 3] = -1.0
    inf = float("inf")
    kp[table[0, 1], 0, 4, 3] = inf       # row 20 of sequence 0
    kp[table[1, 2], 0, 5, 3] = -inf      # row 37 of sequence 1
    kp[table[3, 0], 0, 0, 3] = inf       # row 0 of sequence 3: all that its token 0 of 2 sees
    clean = vp.clone()
    vp[table[2, 1], 0, 0, 7] = inf       # row 16 of sequence 2
    out, err = _decode(q, kp, vp, table, lens, softmax_scale=scale)
    assert err == 0
    K, Q = f64(kp), f64(q)
    s = scale or Hd ** -0.5
    for b, n in enumerate(lens):
        Kb, Vb = (P.rows(x, table, b, n)[:, 0] for x in (K, f64(clean)))
        for t in range(Tq):
            m = n - Tq + 1 + t
            for g in range(G):
                with np.errstate(invalid="ignore"):
                    logit = (Kb[:m] * Q[b, t, g]).sum(1) * s
                    p = np.exp(logit - logit.max())
                    want = p @ Vb[:m] / p.sum()
                got = f64(out[b, t, g])
                if b == 2:
                    assert not np.isfinite(got[7])
                    want, got = np.delete(want, 7), np.delete(got, 7)
                assert np.array_equal(np.isnan(got), np.isnan(want))
                if not np.isnan(want).any():  # values below six, sums of |q_d k_d| scale below 64
                    assert np.abs(got - want).max() <= P.decode_allowance(np.full(1, 6.0), np.full(1, 64.0), Hd, n).max()
