"""float64 oracle of the paged cache operators (test infrastructure only).

Row l of sequence b lies in row l % page of page table[b][l // page].  Everything
here walks sequences, tokens and heads one by one and shares no code with the
GPU path.
"""
from __future__ import annotations

import numpy as np


def rotate(x: np.ndarray, cos_sin: np.ndarray, rot: int, interleaved: bool) -> np.ndarray:
    """The rotary rotation of the first `rot` values of x [..., Hd] by one
    position's cosines and sines [rot]."""
    y = np.array(x, np.float64)
    half = rot // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = float(cos_sin[i]), float(cos_sin[half + i])
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def kv_append(k, v, q, k_pages, v_pages, table, lens, cos_sin, rot, interleaved, news=None):
    """New (k_pages, v_pages, q_out, lens) in float64, for sequences that fit."""
    kp, vp = np.array(k_pages, np.float64), np.array(v_pages, np.float64)
    qo = np.zeros(q.shape, np.float64) if q is not None else None
    page = kp.shape[2]
    out = np.array(lens)
    for b in range(k.shape[0]):
        n = k.shape[1] if news is None else int(news[b])
        for t in range(n):
            l = int(lens[b]) + t
            cs = cos_sin[l] if rot else None
            p, r = table[b][l // page], l % page
            kp[p, :, r] = rotate(np.asarray(k[b, t], np.float64), cs, rot, interleaved)
            vp[p, :, r] = v[b, t]
            if q is not None:
                qo[b, t] = rotate(np.asarray(q[b, t], np.float64), cs, rot, interleaved)
        out[b] += n
    return kp, vp, qo, out


def rows(pages: np.ndarray, table, b: int, n: int) -> np.ndarray:
    """Rows [n][H][...] of sequence b."""
    page = pages.shape[2]
    return np.stack([pages[table[b][l // page], :, l % page] for l in range(n)]) if n else \
        np.zeros((0, pages.shape[1]) + pages.shape[3:])


def decode(q, k_pages, v_pages, table, lens, scale=None):
    """(out, mass, wobble) [B][Tq][Hq][Hd]: the attention; sum_l p_l |v_l|; and
    per query [B][Tq][Hq] the largest sum_d |q_d k_d| * scale of its rows.  The
    last two size the rounding allowance of an fp32 computation."""
    B, Tq, Hq, Hd = q.shape
    Hkv = k_pages.shape[1]
    G = Hq // Hkv
    scale = Hd ** -0.5 if scale is None else scale
    out, mass, wobble = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:3])
    for b in range(B):
        n = int(lens[b])
        K = np.asarray(rows(k_pages, table, b, n), np.float64)
        V = np.asarray(rows(v_pages, table, b, n), np.float64)
        for t in range(Tq):
            m = n - Tq + 1 + t
            if m <= 0:
                continue
            for h in range(Hq):
                qh, Kh, Vh = np.asarray(q[b, t, h], np.float64), K[:m, h // G], V[:m, h // G]
                s = Kh @ qh * scale
                p = np.exp(s - s.max())
                p /= p.sum()
                out[b, t, h] = p @ Vh
                mass[b, t, h] = p @ np.abs(Vh)
                wobble[b, t, h] = (np.abs(Kh) @ np.abs(qh)).max() * abs(scale)
    return out, mass, wobble


def decode_allowance(mass, wobble, Hd: int, n: int):
    """How far an fp32 computation of `decode` may be off.  A logit is a sum of
    exact products accumulated over Hd / 16 tensor-core steps, each of which may
    lose up to one fp32 unit (2^-23, truncation) of the sum of magnitudes, and
    is scaled twice (scale, log2 e: 2^-22 more): off by d <= (Hd / 16 + 4) 2^-23
    wobble.  Each weight is then off by a factor within 2 d (its own logit and
    the maximum's), 2^-21 for the exponential and 2^-21 for its cut into parts;
    the two sums (numerator and denominator) lose at most one unit a strip of 16
    rows plus 64 for the joins.  An output is at most twice that, for numerator
    and denominator, times sum p |v|."""
    d = (Hd / 16 + 4) * 2.0 ** -23 * wobble
    return 2 * mass * (2 * d[..., None] + 2.0 ** -20 + (n / 16 + 64) * 2.0 ** -23) + 1e-30


def latent_codes(lat: np.ndarray, bits: int) -> np.ndarray:
    """Integers of code bytes [..., r*bits/8] (4 bits: element 2j in the low half of byte j)."""
    lat = np.asarray(lat, np.uint8)
    if bits == 8:
        return lat.view(np.int8).astype(np.float64)
    both = np.stack([lat & 15, lat >> 4], axis=-1).astype(np.int64)
    return np.where(both > 7, both - 16, both).reshape(lat.shape[:-1] + (-1,)).astype(np.float64)


def latent_decode(q, lat_k, lat_v, scale_k, scale_v, B_k, B_v, table, lens, bits, scale=None):
    """(out, mass, wobble) of the attention over paged latents: K and V rebuilt
    row by row.  mass [B][H][Hd]: sum_l p_l sum_j |code_l,j s_l B_v[j, d]|; wobble
    [B][H]: the largest sum_j |code_l,j s_l| max|q'| * scale, q' = B_k q."""
    B, H, Hd = q.shape
    scale = Hd ** -0.5 if scale is None else scale
    out, mass, wobble = np.zeros(q.shape), np.zeros(q.shape), np.zeros((B, H))
    ck, cv = latent_codes(lat_k, bits), latent_codes(lat_v, bits)
    for b in range(B):
        n = int(lens[b])
        if not n:
            continue
        lk, lv = rows(ck, table, b, n), rows(cv, table, b, n)                      # [n][H][r]
        sk = rows(np.asarray(scale_k, np.float64)[..., None], table, b, n)
        sv = rows(np.asarray(scale_v, np.float64)[..., None], table, b, n)
        for h in range(H):
            K = (lk[:, h] * sk[:, h]) @ np.asarray(B_k[h], np.float64)
            V = (lv[:, h] * sv[:, h]) @ np.asarray(B_v[h], np.float64)
            qh = np.asarray(q[b, h], np.float64)
            s = K @ qh * scale
            p = np.exp(s - s.max())
            p /= p.sum()
            out[b, h] = p @ V
            mass[b, h] = p @ (np.abs(lv[:, h] * sv[:, h]) @ np.abs(np.asarray(B_v[h], np.float64)))
            qp = np.abs(np.asarray(B_k[h], np.float64)) @ np.abs(qh)
            wobble[b, h] = np.abs(lk[:, h] * sk[:, h]).sum(1).max() * qp.max() * abs(scale)
    return out, mass, wobble


def latent_allowance(mass, wobble, r: int, Hd: int, biggest: np.ndarray, n: int):
    """How far an fp32 / fixed-point computation of `latent_decode` may be off.
    q' is an fp32 sum of Hd products (at most (Hd / 32 + 8) 2^-24 of its
    magnitudes) in fixed point to half of 2^-22 of its largest value; a logit is
    an exact integer sum scaled in fp32 (4 roundings): off by
    d <= (Hd / 32 + 16) 2^-23 wobble.  A weight is off by 2 d and 2^-21, and is
    cut to half a step of 2^-21 of the largest weight of its strip, which with
    its codes makes at most 2^-21 * biggest a row, biggest[b, h, d] the largest
    |V| a full code row can give, over the joined mass of all weights: no more
    than `biggest` times 2^-21 a row.  Sums as in decode_allowance, then r more."""
    d = (Hd / 32 + 16) * 2.0 ** -23 * wobble
    return 2 * mass * (2 * d[..., None] + 2.0 ** -20 + (n / 16 + 64 + r) * 2.0 ** -23) + biggest * 2.0 ** -21 + 1e-30
