"""Host-side checks of the paged cache calls: every refusal comes before any
CUDA call (so these run without a GPU), the workspaces hold what the header says,
and the float64 oracle agrees with hand-worked and independent values."""
import ctypes
import math

import numpy as np
import pytest
import torch

import rank_kv_cache_wsvd_b200 as W
from oracle import paged_oracle as P
from rank_kv_cache_wsvd_b200 import _lib

MIB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(_lib.LIB_PATH):
        from rank_kv_cache_wsvd_b200 import build
        build.build()
    return _lib.load()


def _at(mib):
    """A made-up, aligned address; never dereferenced."""
    return ctypes.c_void_p(mib * MIB)


def _append_args(**kw):
    a = dict(B=2, T=3, Hq=4, Hkv=2, Hd=64, rot=64, inter=0, page=16, pages=8, maxp=4, maxpos=64, k=_at(1), ks=128,
             v=_at(2), vs=128, q=_at(3), qs=256, dtype=1, cs=_at(4), news=None, table=_at(5), lens=_at(6), out=_at(6),
             kp=_at(7), vp=_at(8), qo=_at(9), ws=_at(10), wsb=16, err=None, stream=None)
    assert set(kw) <= set(a), kw
    a.update(kw)
    return list(a.values())


def _decode_args(**kw):
    a = dict(B=2, Tq=1, Hq=4, Hkv=2, Hd=64, page=16, pages=8, maxp=4, lens=_at(1), table=_at(2), q=_at(3), kp=_at(4),
             vp=_at(5), dtype=1, scale=0.0, out=_at(6), ws=_at(7), wsb=64 * MIB, err=None, stream=None)
    assert set(kw) <= set(a), kw
    a.update(kw)
    return list(a.values())


def _lat_decode_args(**kw):
    a = dict(B=2, H=4, Hd=64, r=32, bits=8, page=16, pages=8, maxp=4, lens=_at(1), table=_at(2), q=_at(3), dtype=1,
             lk=_at(4), lv=_at(5), sk=_at(6), sv=_at(7), Bk=_at(8), Bv=_at(9), scale=0.0, out=_at(10), ws=_at(11),
             wsb=64 * MIB, err=None, stream=None)
    assert set(kw) <= set(a), kw
    a.update(kw)
    return list(a.values())


def _lat_append_args(**kw):
    a = dict(B=2, T=3, H=4, E=256, r=32, bits=8, page=16, pages=8, maxp=4, blk=128, x=_at(1), dtype=1, Ak=_at(2),
             Av=_at(3), lens=_at(4), out=_at(4), table=_at(5), lk=_at(6), lv=_at(7), sk=_at(8), sv=_at(9), ws=_at(10),
             wsb=64 * MIB, err=None, stream=None)
    assert set(kw) <= set(a), kw
    a.update(kw)
    return list(a.values())


BAD = ctypes.c_void_p(MIB + 8)  # not 16-byte aligned


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), 1), (dict(T=-1), 1), (dict(Hkv=0), 1), (dict(dtype=2), 1), (dict(rot=-16), 1), (dict(rot=80), 1),
    (dict(Hd=48), 1), (dict(Hd=48, rot=16), 2), (dict(Hd=512), 2), (dict(rot=24), 2), (dict(page=8), 2), (dict(page=48), 2), (dict(page=512), 2),
    (dict(B=65536), 2), (dict(maxp=1 << 28, page=16), 2), (dict(k=None), 1), (dict(v=None), 1), (dict(q=None), 1),
    (dict(qo=None), 1), (dict(cs=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(out=None), 1),
    (dict(kp=None), 1), (dict(ws=None), 1), (dict(k=BAD), 1), (dict(q=BAD), 1), (dict(vp=BAD), 1), (dict(cs=BAD), 1),
    (dict(ks=120), 1), (dict(vs=132), 1), (dict(qs=248), 1), (dict(wsb=8), 4), (dict(B=0, k=None, table=None), 0),
    (dict(qo=_at(1)), 1),                                   # q_out over k
    (dict(qo=_at(3), qs=512), 1),                           # in place over a strided q
    (dict(kp=_at(3)), 1), (dict(vp=_at(7)), 1),             # pages over q, both pools one
    (dict(out=ctypes.c_void_p(6 * MIB + 4)), 1),            # lengths shifted by one
    (dict(out=_at(5)), 1), (dict(news=_at(7)), 1),          # lengths over the table, counts inside a pool
])
def test_kv_append_refuses(lib, kw, want):
    assert lib.paged_kv_append(*_append_args(**kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), 1), (dict(Tq=0), 1), (dict(Hkv=0), 1), (dict(Hq=3), 1), (dict(Hq=1), 1), (dict(dtype=-1), 1),
    (dict(Hd=96), 2), (dict(page=24), 2), (dict(page=1024), 2), (dict(Tq=33), 2), (dict(B=70000), 2),
    (dict(lens=None), 1), (dict(table=None), 1), (dict(q=None), 1), (dict(kp=None), 1), (dict(vp=None), 1),
    (dict(out=None), 1), (dict(ws=None), 1), (dict(q=BAD), 1), (dict(kp=BAD), 1), (dict(out=BAD), 1), (dict(ws=BAD), 1),
    (dict(wsb=1024), 4), (dict(B=0, q=None), 0),
])
def test_kv_decode_refuses(lib, kw, want):
    assert lib.paged_decode_attention(*_decode_args(**kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), 1), (dict(H=0), 1), (dict(bits=6), 1), (dict(r=0), 1), (dict(r=3, bits=4), 1), (dict(dtype=3), 1),
    (dict(B=4097), 2), (dict(Hd=48), 2), (dict(page=8), 2), (dict(r=24), 2), (dict(r=16, bits=4), 2), (dict(r=256), 2),
    (dict(lens=None), 1), (dict(table=None), 1), (dict(lk=None), 1), (dict(sv=None), 1), (dict(Bk=None), 1),
    (dict(out=None), 1), (dict(lv=BAD), 1), (dict(Bv=BAD), 1), (dict(ws=BAD), 1), (dict(wsb=1024), 4),
    (dict(B=0, q=None), 0),
])
def test_latent_decode_refuses(lib, kw, want):
    assert lib.wsvd_decode_attention_paged(*_lat_decode_args(**kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), 1), (dict(T=-1), 1), (dict(H=0), 1), (dict(E=0), 1), (dict(bits=5), 1), (dict(dtype=2), 1),
    (dict(page=8), 2), (dict(blk=96), 1), (dict(blk=2048, E=4096), 1), (dict(E=200, blk=128), 1), (dict(r=24), 2),
    (dict(E=272, blk=16), 2), (dict(E=32768), 2), (dict(x=None), 1), (dict(Ak=None), 1), (dict(lens=None), 1),
    (dict(table=None), 1), (dict(sk=None), 1), (dict(ws=None), 1), (dict(x=BAD), 1), (dict(lk=BAD), 1), (dict(ws=BAD), 1),
    (dict(wsb=256), 4), (dict(out=ctypes.c_void_p(4 * MIB + 4)), 1), (dict(out=_at(5)), 1), (dict(B=0, x=None), 0),
    (dict(T=1, r=24), 2), (dict(r=8), 2), (dict(r=16, bits=4), 2), (dict(T=1, blk=96), 1), (dict(T=1, B=17, E=272, blk=16), 2), (dict(T=1, x=None), 1),
])
def test_latent_append_refuses(lib, kw, want):
    assert lib.wsvd_latent_append_paged(*_lat_append_args(**kw)) == want


def test_workspace_sizes(lib):
    a16 = lambda v: (v + 15) // 16 * 16
    assert W.paged_kv_append_workspace_size(1) == 16 and W.paged_kv_append_workspace_size(9) == a16(36)
    assert W.paged_kv_append_workspace_size(-1) == 0
    # two partials per worker (592 CTAs, or 2048 warps with 8 queries a chunk), of O and (m, l) per query of
    # a chunk; a counter per unit
    size = lambda B, Hkv, nq, qc, Hd: (a16(2 * (2048 if qc == 8 else 592) * (min(nq, qc) * Hd + (2 * min(nq, qc) + 3) // 4 * 4) * 4)
                                       + a16(B * Hkv * math.ceil(nq / qc) * 4))
    assert W.paged_decode_workspace_size(3, 1, 32, 8, 128) == size(3, 8, 4, 8, 128)
    assert W.paged_decode_workspace_size(3, 4, 32, 4, 64) == size(3, 4, 32, 16, 64)
    assert W.paged_decode_workspace_size(3, 1, 16, 1, 256) == size(3, 1, 16, 8, 256)
    assert W.paged_decode_workspace_size(3, 1, 30, 8, 128) == 0
    assert W.wsvd_latent_append_paged_workspace_size(2, 3, 256) == 256 + W.wsvd_prefill_workspace_size(2, 3, 256)  # hi, lo, scales


def test_python_refuses_what_it_cannot_pass_on(lib):
    """Host tensors, wrong types and shapes raise before the library is called."""
    z = torch.zeros
    q, kp = z(2, 4, 64, dtype=torch.float16), z(8, 2, 16, 64, dtype=torch.float16)
    table, lens = z(2, 4, dtype=torch.int32), z(2, dtype=torch.int32)
    with pytest.raises(W.WsvdError, match="CUDA"):
        W.paged_decode_attention(q, kp, kp, table, lens)
    with pytest.raises(W.WsvdError, match="CUDA"):
        W.paged_kv_append(z(2, 1, 2, 64, dtype=torch.float16), z(2, 1, 2, 64, dtype=torch.float16), kp, kp, table, lens)
    lat, sc = z(8, 4, 16, 32, dtype=torch.uint8), z(8, 4, 16, dtype=torch.float16)
    up, down = z(4, 32, 64, dtype=torch.float16), z(4, 256, 32, dtype=torch.float16)
    with pytest.raises(W.WsvdError, match="CUDA"):
        W.wsvd_decode_attention_paged(q, lat, lat, sc, sc, up, up, table, lens, 8)
    with pytest.raises(W.WsvdError, match="CUDA"):
        W.wsvd_latent_append_paged(z(2, 1, 256, dtype=torch.bfloat16), down, down, lens, table, lat, lat, sc, sc, 8)


def test_strided_tokens_are_recognised():
    """A slice of a fused projection passes with its token stride; transposed
    heads, uneven batches and broadcast axes are refused."""
    fused = torch.zeros(3, 5, 10 * 32, dtype=torch.float16)
    part = fused[..., 64:128].unflatten(-1, (2, 32))
    ptr, stride = _lib._tokens(part, torch.float16, (3, 5, 2, 32), -1, "k")
    assert (ptr, stride) == (part.data_ptr(), 320)
    one = fused[:, 2:3, 64:128].unflatten(-1, (2, 32))   # one token of each sequence: five tokens apart
    assert _lib._tokens(one, torch.float16, (3, 1, 2, 32), -1, "k")[1] == 1600
    alone = fused[1:2, 2:3, 64:128].unflatten(-1, (2, 32))
    assert _lib._tokens(alone, torch.float16, (1, 1, 2, 32), -1, "k")[1] == 64
    for bad in (part.transpose(0, 1), part[..., ::2], part.transpose(2, 3), fused[:, :4, 64:128].unflatten(-1, (2, 32)),
                part[:, :1].expand(3, 5, 2, 32)):
        with pytest.raises(W.WsvdError):
            _lib._tokens(bad, torch.float16, tuple(bad.shape), -1, "k")


# ----------------------------------------------------------------------------- the oracle itself
def test_oracle_rotation_by_hand_and_as_complex_numbers():
    quarter = np.array([0.0, 0.0, 1.0, 1.0])  # cos, sin of a quarter turn for both pairs
    x = np.array([1.0, 2.0, 3.0, 4.0, 9.0])
    assert np.allclose(P.rotate(x, quarter, 4, False), [-3, -4, 1, 2, 9])
    assert np.allclose(P.rotate(x, quarter, 4, True), [-2, 1, -4, 3, 9])
    rng = np.random.default_rng(0)
    a, x = rng.uniform(0, 6, 8), rng.standard_normal((3, 16))
    cs = np.concatenate([np.cos(a), np.sin(a)])
    z = (x[:, :8] + 1j * x[:, 8:]) * np.exp(1j * a)
    assert np.allclose(P.rotate(x, cs, 16, False), np.concatenate([z.real, z.imag], axis=1))
    z = (x[:, 0::2] + 1j * x[:, 1::2]) * np.exp(1j * a)
    assert np.allclose(P.rotate(x, cs, 16, True), np.stack([z.real, z.imag], axis=-1).reshape(3, 16))


def test_oracle_decode_against_torch():
    rng = np.random.default_rng(1)
    table = np.array([[2, 0], [1, 3]])
    K, V = rng.standard_normal((4, 2, 16, 8)), rng.standard_normal((4, 2, 16, 8))
    q, lens = rng.standard_normal((2, 3, 4, 8)), [20, 2]
    out, mass, _ = P.decode(q, K, V, table, lens)
    for b, n in enumerate(lens):
        Kb, Vb = (torch.from_numpy(P.rows(x, table, b, n)) for x in (K, V))
        for t in range(3):
            m = n - 2 + t
            for h in range(4):
                if m <= 0:
                    assert (out[b, t, h] == 0).all()
                    continue
                p = torch.softmax(Kb[:m, h // 2] @ torch.from_numpy(q[b, t, h]) / math.sqrt(8), 0)
                assert np.allclose(out[b, t, h], (p @ Vb[:m, h // 2]).numpy())
    assert (mass >= np.abs(out) - 1e-12).all()


def test_oracle_latent_decode_against_the_contiguous_oracle():
    import oracle as O
    rng = np.random.default_rng(2)
    H, r, Hd = 2, 16, 32
    for bits in (8, 4):
        lat = [rng.integers(0, 256, (3, H, 16, r * bits // 8), dtype=np.uint8) for _ in range(2)]
        sc = [(rng.random((3, H, 16)) * 0.1).astype(np.float16) for _ in range(2)]
        up = [rng.standard_normal((H, r, Hd)).astype(np.float16) for _ in range(2)]
        table, lens = np.array([[2, 0]]), np.array([21], np.int32)
        q = rng.standard_normal((1, H, Hd))
        flat = [np.concatenate([x[2], x[0]], axis=1)[None] for x in lat + sc]
        want = O.wsvd_decode(q, flat[0], flat[2], flat[1], flat[3], up[0], up[1], lens, r, bits)
        got, _, _ = P.latent_decode(q, lat[0], lat[1], sc[0], sc[1], up[0], up[1], table, lens, bits)
        assert np.allclose(got, want, rtol=1e-9, atol=1e-12)


def test_an_allowance_catches_planted_mistakes():
    """The tolerance of the decode tests refuses a row too many, a row too few,
    a neighbour's page and weights rounded to bf16."""
    rng = np.random.default_rng(3)
    table, lens = np.array([[0, 1, 2, 3]]), [50]
    K, V = rng.standard_normal((5, 1, 16, 64)), rng.standard_normal((5, 1, 16, 64))
    q = rng.standard_normal((1, 1, 2, 64))
    ref, mass, wobble = P.decode(q, K, V, table, lens)
    allow = P.decode_allowance(mass, wobble, 64, 50)
    off = lambda out: float((np.abs(out - ref) / allow).max())
    assert off(P.decode(q, K, V, table, [51])[0]) > 1 and off(P.decode(q, K, V, table, [49])[0]) > 1
    assert off(P.decode(q, K, V, np.array([[0, 1, 4, 3]]), lens)[0]) > 1
    Kr, Vr = P.rows(K, table, 0, 50)[:, 0], P.rows(V, table, 0, 50)[:, 0]
    p = np.exp(Kr @ q[0, 0, 0] / 8 - (Kr @ q[0, 0, 0] / 8).max())
    p16 = torch.from_numpy(p).bfloat16().double().numpy()
    rounded = ref.copy()
    rounded[0, 0, 0] = p16 @ Vr / p.sum()
    assert off(rounded) > 1


def test_latent_append_refuses_blocks_of_too_many_tiles(lib):
    """B * T * H * r past 2^42, each within its own limit."""
    apart = {k: _at((i + 1) << 20) for i, k in enumerate(("x", "Ak", "Av", "table", "lk", "lv", "sk", "sv", "ws"))}
    assert lib.wsvd_latent_append_paged(*_lat_append_args(B=1 << 12, T=1 << 12, H=1 << 14, E=64, blk=64, **apart)) == 2
    assert lib.wsvd_latent_append_paged(*_lat_append_args(B=1 << 12, T=1 << 12, H=1 << 13, E=64, blk=64, **apart)) == 4  # the workspace


@pytest.mark.parametrize("TS", [16, 32, 64, 128])
def test_strips_of_lengths_at_the_end_of_the_range(TS):
    """The decodes' 32-bit sums: strips of a length as large as an int holds, and
    which strips look at their rows' limits (s TS > n - TS, not s TS + TS > n)."""
    wrap = lambda x: (x + 2 ** 31) % 2 ** 32 - 2 ** 31
    for n in (1, TS - 1, TS, TS + 1, 2 ** 31 - TS, 2 ** 31 - TS + 1, 2 ** 31 - 16, 2 ** 31 - 1):
        strips = wrap(((n + TS - 1) % 2 ** 32) // TS)
        assert strips == -(-n // TS)
        s = strips - 1
        assert (wrap(s * TS) > wrap(n - TS)) == (n % TS != 0)
        assert all(wrap(s * TS + i) == s * TS + i for i in (0, TS - 16, TS - 1))


def _lat_pools(at):
    """Every way two of the latent append's outputs, or one and an input, may meet."""
    names = ("lk", "lv", "sk", "sv")
    return [{a: at[b]} for a in names for b in names if a < b] + [{a: at[b]} for a in names for b in ("x", "Ak", "Av", "table", "ws")]


AT = dict(x=_at(1), Ak=_at(2), Av=_at(3), table=_at(5), lk=_at(6), lv=_at(7), sk=_at(8), sv=_at(9), ws=_at(10))


@pytest.mark.parametrize("kw", _lat_pools(AT) + [dict(lens=_at(6), out=_at(6)), dict(out=_at(9)), dict(ws=_at(2)),
                                                 dict(lv=ctypes.c_void_p(6 * MIB + 16)), dict(err=_at(5)), dict(err=_at(8)),
                                                 dict(lens=_at(10), out=_at(10))])
def test_latent_append_refuses_overlaps(lib, kw):
    assert lib.wsvd_latent_append_paged(*_lat_append_args(**kw)) == 1


@pytest.mark.parametrize("kw", [dict(out=_at(i)) for i in (1, 2, 3, 4, 5, 7)] + [dict(ws=_at(i)) for i in range(1, 7)]
                         + [dict(out=ctypes.c_void_p(4 * MIB - 16)), dict(err=_at(2)), dict(err=_at(7))])
def test_kv_decode_refuses_overlaps(lib, kw):
    assert lib.paged_decode_attention(*_decode_args(**kw)) == 1


@pytest.mark.parametrize("kw", [dict(out=_at(i)) for i in (1, 2, 3, 4, 5, 6, 7, 8, 9, 11)] + [dict(ws=_at(i)) for i in range(1, 11)]
                         + [dict(err=_at(10)), dict(err=_at(8))])
def test_latent_decode_refuses_overlaps(lib, kw):
    assert lib.wsvd_decode_attention_paged(*_lat_decode_args(**kw)) == 1


@pytest.mark.parametrize("kw,want", [(dict(ws=_at(i)), 1) for i in (1, 2, 3, 4, 5, 6, 7, 8)] + [
    (dict(err=_at(7)), 1), (dict(err=_at(6)), 1), (dict(ks=1 << 62), 1), (dict(vs=1 << 61), 1), (dict(qs=(1 << 63) - 8), 1),
    (dict(pages=2 ** 31 - 1, Hkv=1 << 18, Hq=0, q=None, qo=None, ks=1 << 26, vs=1 << 26, Hd=256, rot=0, cs=None, page=256), 2)])
def test_kv_append_refuses_more_overlaps_and_impossible_strides(lib, kw, want):
    assert lib.paged_kv_append(*_append_args(**kw)) == want


def test_latent_append_of_more_heads_than_grid_rows_is_refused_where_only_the_append_takes_e(lib):
    """E 272 is the append's alone, whose grid has a row for K and one for V of a head."""
    args = dict(T=1, B=1, E=272, blk=16, r=16, x=_at(1 << 10), Ak=_at(1 << 12), Av=_at(1 << 13), lk=_at(1 << 14), lv=_at(1 << 15),
                sk=_at(1 << 16), sv=_at(1 << 17), wsb=128)
    assert lib.wsvd_latent_append_paged(*_lat_append_args(H=32768, **args)) == 2
    assert lib.wsvd_latent_append_paged(*_lat_append_args(H=32767, **args)) == 4  # the workspace


def test_pools_past_every_address_are_refused(lib):
    big = dict(pages=2 ** 31 - 1, page=256)
    assert lib.paged_decode_attention(*_decode_args(Hq=1 << 20, Hkv=1 << 20, Hd=256, **big)) == 2
    assert lib.wsvd_decode_attention_paged(*_lat_decode_args(H=1 << 20, r=128, **big)) == 2
    assert lib.wsvd_latent_append_paged(*_lat_append_args(H=1 << 20, r=128, **big)) == 2


# ----------------------------------------------------------------------------- how strips are dealt
def _deal(lens, units, TS, count, least, lead):
    """The shares of the decodes' workers: [worker][(sequence * units + unit, first strip, end)], and the holders of a
    unit's strips by the device's formula."""
    sizes = [(b * units + u, -(-n // TS)) for b, n in enumerate(lens) if n > 0 for u in range(units)]
    total = sum(n + lead for _, n in sizes)
    workers = min(count, -(-total // least))
    base, extra = divmod(total, workers)
    begin = lambda c: base * c + min(c, extra)
    worker_of = lambda s: s // (base + 1) if s < extra * (base + 1) else extra + (s - extra * (base + 1)) // base
    shares, holders, at = [[] for _ in range(workers)], {}, 0
    for key, n in sizes:
        first, last = worker_of(at + lead), worker_of(at + lead + n - 1)
        holders[key] = (first, last - first + 1)
        c = worker_of(at)
        while c < workers and begin(c) < at + lead + n:
            s, e = max(begin(c), at + lead), min(begin(c + 1) if c + 1 < workers else total, at + lead + n)
            if e > s:
                shares[c].append((key, s - at - lead, e - at - lead, n))
            c += 1
        at += n + lead
    return shares, holders


@pytest.mark.parametrize("seed", range(40))
def test_a_worker_is_the_first_of_at_most_one_cut_unit(seed):
    """Counters by a unit's first worker, and the slots of the partial results, are each one's own."""
    rng = np.random.default_rng(seed)
    TS, lead, least = int(rng.choice([16, 32, 64, 128])), int(rng.choice([2, 4, 24])), int(rng.choice([1, 6, 12]))
    count = int(rng.choice([148, 1776, 1920, 2016]))
    B, units, top = int(rng.integers(1, 70)), int(rng.integers(1, 40)), int(rng.choice([3, 300, 5000, 40000]))
    lens = [int(n) for n in rng.integers(0, top, B)]
    lens[0] = max(1, lens[0])
    shares, holders = _deal(lens, units, TS, count, least, lead)
    held, counters, slots, two = {}, {}, set(), set()
    for c, segs in enumerate(shares):
        for key, s, e, n in segs:
            held.setdefault(key, []).append((c, s, e))
            if (s, e) == (0, n):
                continue
            counters.setdefault(holders[key][0], set()).add(key)
            assert (c + key) not in slots and c + key < count + B * units  # the latent decode's slot
            slots.add(c + key)
            assert (c, s == 0) not in two                                  # the dense decode's: one that it begins, one within
            two.add((c, s == 0))
    assert all(len(keys) == 1 for keys in counters.values()) and max(counters, default=0) < 2048
    for key, parts in held.items():
        assert [p[0] for p in parts] == list(range(holders[key][0], sum(holders[key])))
        assert parts[0][1] == 0 and all(a[2] == b[1] for a, b in zip(parts, parts[1:]))
    assert sum(p[-1][2] for p in held.values()) == sum(-(-n // TS) for n in lens) * units


def test_workspaces_hold_the_counters_and_the_slots_of_every_worker(lib):
    """8 KB of counters and the partial results of all workers lie within the sizes, from the smallest row to the largest."""
    for B, H in ((1, 1), (3, 7), (4096, 32)):
        for r in (16, 32, 64, 128):
            assert 8192 + (1920 + B * H) * (r + 2) * 4 <= W.wsvd_decode_workspace_size(B, H, r) - B * H * r * 4
        for R in (32, 64, 128, 256):
            assert 8192 + (1920 + B * H) * (R + 2) * 4 <= W.dense_decode_workspace_size(B, H, R) - B * H * R * 4
        for R in (128, 1024):
            assert 8192 + (1920 + B * H) * (R + 2) * 4 <= W.shared_decode_workspace_size(B, H, R) - B * H * R * 4
    for Hd in (32, 64, 128, 256):
        for nq in range(1, 65):
            qc = 16 if nq > 8 and Hd != 256 else 8
            m = min(nq, qc)
            slot = (m * Hd + (2 * m + 3) // 4 * 4) * 4
            assert 8192 + 2 * (2016 if qc == 8 else 588) * slot <= W.paged_decode_workspace_size(1, 1, nq, 1, Hd)
