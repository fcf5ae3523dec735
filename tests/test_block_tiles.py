"""Every tile of the kernel that puts blocks of tokens into latent pages, whole and
with E split over a cluster: a model of the rule that picks the tile shows on the CPU
that the cases reach all of them, and the GPU compares their codes with 64 bits."""
import numpy as np
import pytest
import torch

import rank_kv_cache_wsvd_b200 as W
from paged_util import cuda, randn, table_for

SMS = 148


def _up(a, b):
    return -(-a // b)


def _ranks(tiles, KT, resident):
    """CTAs that split E for one tile."""
    return next((c for c in range(8, 1, -1) if 2 * c <= KT and tiles * c <= SMS and tiles <= resident(c)), 1)


def tile_of(tokens, H, r, E, resident):
    """(columns, tokens of a tile, CTAs a tile) as the host picks them; resident(c): clusters of c CTAs at once."""
    hr, KT, mt = H * r, E // 64, _up(tokens, 64)
    n256 = 2 * _up(hr, 256)
    if mt * 2 * _up(hr, 128) > SMS // 2 and 2 * n256 * 256 <= 5 * hr:
        few, tall = mt * n256, _up(mt, 2) * n256
        span = lambda tiles: _up(tiles * _ranks(tiles, KT, resident), SMS) * _up(KT, _ranks(tiles, KT, resident))
        tiles, rows = (tall, 128) if 8 * span(tall) < 5 * span(few) else (few, 64)
        return 256, rows, _ranks(tiles, KT, resident)
    columns = 64 if hr <= 64 else 128
    return columns, 64, _ranks(mt * 2 * _up(hr, columns), KT, resident)


# (B, T, H, E, r) and the tile; clusters of two need 72 of them resident at most.
CASES = [
    ((1, 70, 3, 64, 16), (64, 64, 1)), ((3, 50, 2, 512, 32), (64, 64, 4)), ((2, 90, 1, 192, 64), (64, 64, 1)),
    ((2, 65, 32, 256, 16), (128, 64, 2)), ((1, 130, 9, 64, 32), (128, 64, 1)), ((5, 1, 32, 512, 64), (128, 64, 4)),
    ((3, 41, 5, 128, 128), (128, 64, 1)), ((2, 10, 3, 512, 128), (128, 64, 4)),
    ((1, 577, 32, 256, 16), (256, 64, 2)), ((3, 769, 32, 192, 16), (256, 64, 1)),
    ((1, 1731, 32, 256, 16), (256, 128, 2)), ((2, 1501, 32, 192, 16), (256, 128, 1)),
    ((1, 300, 32, 256, 32), (256, 64, 2)), ((1, 2307, 32, 128, 32), (256, 64, 1)),
    ((2, 449, 32, 512, 32), (256, 128, 2)), ((2, 577, 32, 256, 32), (256, 128, 1)),
    ((1, 130, 32, 256, 64), (256, 64, 2)), ((1, 130, 32, 512, 64), (256, 128, 4)), ((3, 385, 32, 64, 64), (256, 64, 1)), ((1, 577, 32, 128, 64), (256, 128, 1)),
    ((1, 450, 32, 256, 64), (256, 128, 2)),
    ((1, 577, 32, 64, 128), (256, 64, 1)), ((2, 577, 32, 64, 128), (256, 128, 1)), ((1, 300, 8, 512, 128), (256, 64, 3)),
    ((1, 300, 16, 512, 128), (256, 128, 2)),
]


@pytest.mark.parametrize("case,tile", CASES)
def test_the_rule_gives_each_case_its_tile(case, tile):
    B, T, H, E, r = case
    assert tile_of(B * T, H, r, E, lambda c: {2: 72, 3: 44, 4: 32}.get(c, 16)) == tile


def test_the_cases_reach_every_tile():
    seen = {(r, columns, rows) for (_, _, _, _, r), (columns, rows, _) in CASES}
    assert seen == {(r, c, m) for r in (16, 32, 64, 128) for c, m in ((64, 64), (128, 64), (256, 64), (256, 128))
                    if r <= 64 or c > 64}
    split = {(columns, rows) for _, (columns, rows, ranks) in CASES if ranks > 1}
    assert split == {(64, 64), (128, 64), (256, 64), (256, 128)}


def _rotated(x, blk):
    """x . blockdiag(H / sqrt(blk)) in 64 bits, Sylvester order, by its recursion."""
    y, n = x.double().unflatten(-1, (-1, blk)), 1
    while n < blk:
        y = y.unflatten(-1, (-1, 2, n))
        y = torch.stack([y[..., 0, :] + y[..., 1, :], y[..., 0, :] - y[..., 1, :]], dim=-2).flatten(-3)
        n *= 2
    return (y / blk ** 0.5).flatten(-2)


def _check_rows(codes, scale, c, top):
    """The framework's rule: a code is off by one only within 1e-3 of a half step, a
    scale by one fp16 step only within 2^-20 of its border (its codes then by one)."""
    ratio = c.abs().amax(-1) / top
    want = ratio.half()
    same = want == scale
    lo, hi = torch.minimum(want, scale).double(), torch.maximum(want, scale).double()
    border = (ratio - (lo + hi) / 2).abs() <= 2.0 ** -20 * ratio
    steps = (want.view(torch.int16).int() - scale.view(torch.int16).int()).abs()
    assert (same | (border & (steps == 1))).all()
    v = c / want.double()[..., None]
    off = (codes.double() - torch.round(v).clamp(-top, top)).abs()
    near = ((v.abs() % 1) - 0.5).abs() <= 1e-3
    assert (off <= 1).all() and ((off == 0) | near | ~same[..., None]).all()
    return int((off > 0).sum()) + int((~same).sum())


@pytest.mark.gpu
@pytest.mark.parametrize("case,bits", [(c, b) for c, _ in CASES for b in (8, 4) if c[-1] * b >= 128])
def test_blocks_of_every_tile(case, bits):
    B, T, H, E, r = case
    from rank_kv_cache_wsvd_b200 import build
    build.build()
    page, blk, top = 32, 64, 127 if bits == 8 else 7
    lens = [(b * 29) % 70 for b in range(B)]
    table, pool = table_for([n + T for n in lens], page, seed=r)
    g = torch.Generator(device="cuda").manual_seed(1)
    lat = [torch.randint(0, 256, (pool, H, page, r * bits // 8), generator=g, dtype=torch.uint8, device="cuda") for _ in range(2)]
    sc = [torch.rand((pool, H, page), generator=g, device="cuda").half() for _ in range(2)]
    before = [t.clone() for t in lat + sc]
    x = randn((B, T, E), "bf16", 3)
    down = [(randn((H, E, r), "fp16", s) * E ** -0.5).contiguous() for s in (4, 5)]
    n, tab = cuda(np.asarray(lens, np.int32)), cuda(table)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    need = W.wsvd_latent_append_paged_workspace_size(B, T, E)
    ws = torch.zeros(need + 256, dtype=torch.uint8, device="cuda")
    ws[need:] = 0xA5
    call = lambda: W.wsvd_latent_append_paged(x, *down, n, tab, *lat, *sc, bits, blk, err=err, workspace_buf=ws[:need])
    call()
    assert int(err.item()) == 0 and n.tolist() == [a + T for a in lens] and (ws[need:] == 0xA5).all()
    row = n.long()[:, None] - T + torch.arange(T, device="cuda")
    at = (tab.long().gather(1, row // page), row % page)
    rot, ties = _rotated(x, blk), 0
    for k in range(2):
        c = torch.einsum("bte,her->bthr", rot, down[k].double())
        codes = lat[k][at[0], :, at[1]].view(torch.int8)
        if bits == 4:
            codes = torch.stack([(codes << 4) >> 4, codes >> 4], dim=-1).flatten(-2)
        ties += _check_rows(codes, sc[k][at[0], :, at[1]], c, top)
    assert ties <= 4 + 2 * B * T * H * (r * 2e-3 + 2.0 ** -8)
    # rows of nobody keep their bytes, and the same call again gives the same ones
    mine = torch.zeros((pool, page), dtype=torch.bool, device="cuda")
    mine[at] = True
    for got, old in zip(lat + sc, before):
        same = (got.view(torch.uint8) == old.view(torch.uint8)).view(pool, H, page, -1).all(-1).all(1)
        assert (same | mine).all()
    kept = [t.clone() for t in lat + sc]
    for _ in range(3):
        n.copy_(torch.tensor(lens, dtype=torch.int32))
        call()
    for got, old in zip(lat + sc, kept):
        assert torch.equal(got.view(torch.uint8), old.view(torch.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,E,r,blk", [(1, 4, 256, 128, 128), (3, 32, 512, 64, 128), (4, 32, 1024, 32, 256), (4, 3, 256, 16, 1),
                                         (2, 5, 512, 64, 64), (9, 2, 272, 32, 16), (16, 4, 40, 64, 8)])
def test_one_token_by_the_append_kernel_has_its_bits(B, H, E, r, blk):
    """One token of B <= 4 sequences with B * r <= 192, and any E that only the append
    takes: the codes and scales of wsvd_latent_append, bit for bit."""
    assert (B <= 4 and B * r <= 192) or E % 64
    page, lens = 16, [(b * 29) % 70 for b in range(B)]
    table, pool = table_for([n + 1 for n in lens], page, seed=r)
    x = randn((B, 1, E), "bf16", 3)
    down = [(randn((H, E, r), "fp16", s) * E ** -0.5).contiguous() for s in (4, 5)]
    lat = [torch.zeros((pool, H, page, r), dtype=torch.uint8, device="cuda") for _ in range(2)]
    sc = [torch.zeros((pool, H, page), dtype=torch.float16, device="cuda") for _ in range(2)]
    W.wsvd_latent_append_paged(x, *down, cuda(np.asarray(lens, np.int32)), cuda(table), *lat, *sc, 8, blk)
    flat = [torch.zeros((B, H, 80, r), dtype=torch.uint8, device="cuda") for _ in range(2)]
    fsc = [torch.zeros((B, H, 80), dtype=torch.float16, device="cuda") for _ in range(2)]
    W.wsvd_latent_append(x[:, 0].contiguous(), *down, cuda(np.asarray(lens, np.int32)), *flat, *fsc, 8, blk)
    for got, want in zip(lat + sc, flat + fsc):
        for b, l in enumerate(lens):
            assert torch.equal(got[table[b, l // page], :, l % page], want[b, :, l]) and want[b, :, l].any()


@pytest.mark.gpu
def test_a_prompt_repeats_its_bits_with_other_calls_between():
    """576 tokens of 32 heads, E 4096, again and again with another prompt between and
    nothing awaited: the same bytes each time, and those of a fresh cache."""
    from rank_kv_cache_wsvd_b200 import build
    build.build()
    B, T, H, E, r, page = 1, 576, 32, 4096, 32, 64
    table, pool = table_for([T], page, 1)
    tab, n = cuda(table), torch.zeros(1, dtype=torch.int32, device="cuda")
    to = torch.zeros_like(n)
    x = [randn((B, T, E), "bf16", s) for s in (1, 2)]
    down = [(randn((H, E, r), "fp16", s) * E ** -0.5).contiguous() for s in (4, 5)]
    ws = W.workspace(W.wsvd_latent_append_paged_workspace_size(B, T, E))
    empty = lambda: [torch.zeros((pool, H, page, r), dtype=torch.uint8, device="cuda") for _ in range(2)] + \
        [torch.zeros((pool, H, page), dtype=torch.float16, device="cuda") for _ in range(2)]
    cache, other = empty(), empty()
    call = lambda i, c: W.wsvd_latent_append_paged(x[i], *down, n, tab, *c, 8, 128, seq_lens_out=to, workspace_buf=ws)
    call(0, cache)
    first = [t.clone() for t in cache]
    for _ in range(20):
        call(1, other)
        call(0, cache)
        call(1, cache)
        call(0, cache)
        for got, want in zip(cache, first):
            assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
    fresh = empty()
    call(0, fresh)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(fresh, first))


@pytest.mark.gpu
def test_one_token_of_more_heads_than_the_append_takes():
    """33000 heads: the append's grid has no rows for them, the block kernel takes them."""
    from rank_kv_cache_wsvd_b200 import build
    build.build()
    H, E, r, page = 33000, 64, 16, 16
    x = randn((1, 1, E), "bf16", 3)
    down = [randn((H, E, r), "fp16", s) * E ** -0.5 for s in (4, 5)]
    lat = [torch.zeros((1, H, page, r), dtype=torch.uint8, device="cuda") for _ in range(2)]
    sc = [torch.zeros((1, H, page), dtype=torch.float16, device="cuda") for _ in range(2)]
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    W.wsvd_latent_append_paged(x, *down, n, torch.zeros((1, 1), dtype=torch.int32, device="cuda"), *lat, *sc, 8, 64)
    assert n.tolist() == [1]
    for k in range(2):
        c = torch.einsum("e,her->hr", _rotated(x, 64)[0, 0], down[k].double())
        ties = _check_rows(lat[k][0, :, 0].view(torch.int8), sc[k][0, :, 0], c, 127)
        assert ties <= 4 + H * (r * 2e-3 + 2.0 ** -8)
