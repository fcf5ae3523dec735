"""Cases of the paged key-value cache operators: what is measured, their plain form and their 64-bit values.

Four operators over pages of a shared pool (page table [B][max_pages]; row l of sequence b lies in row
l % page_size of page block_table[b][l // page_size]):

  kv_append      new keys and values into dense 16-bit pages, the rotary position rotation applied to k and q
  kv_decode      attention of the newest token(s) over dense pages, grouped query heads
  latent_append  new tokens rotated (Hadamard), projected and quantised into latent pages
  latent_decode  attention of the newest token over latent pages (codes, fp16 row scales, up-projections)

A case is a dict; "spread" fixes the ragged lengths, so that the work of a case does not depend on the inputs' seed.
"""
import math
import random

import torch

own = False


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # one layer of a 7B vision-language model kept dense: 576 image + 1024 text tokens, one new token
        dict(name="kv decode llava layer", op="kv_decode", B=1, Tq=1, Hq=32, Hkv=32, Hd=128, page=64, lo=1600, hi=1600,
             spread=0, dtype="bf16"),
        # a serving batch of ragged lengths, grouped heads
        dict(name="kv decode ragged batch", op="kv_decode", B=16, Tq=1, Hq=32, Hkv=8, Hd=128, page=64, lo=1024,
             hi=4096, spread=1, dtype="fp16"),
        # long documents, grouped heads
        dict(name="kv decode long", op="kv_decode", B=4, Tq=1, Hq=32, Hkv=8, Hd=128, page=128, lo=32768, hi=32768,
             spread=0, dtype="bf16"),
        # four speculated tokens a sequence, short pages, lengths that end anywhere
        dict(name="kv decode four tokens", op="kv_decode", B=9, Tq=4, Hq=28, Hkv=4, Hd=64, page=16, lo=3, hi=8191,
             spread=2, dtype="bf16"),
        # one decode step of a serving batch
        dict(name="kv append one token", op="kv_append", B=16, T=1, Hq=32, Hkv=8, Hd=128, rot=128, inter=False,
             page=64, lo=1024, hi=4096, short=False, spread=1, dtype="bf16"),
        # the image tokens of one prompt
        dict(name="kv append image prompt", op="kv_append", B=1, T=576, Hq=32, Hkv=32, Hd=128, rot=128, inter=False,
             page=64, lo=0, hi=0, short=False, spread=0, dtype="bf16"),
        # a padded batch of prompt chunks behind earlier ones, half of each head rotated, pairs interleaved
        dict(name="kv append ragged prompts", op="kv_append", B=8, T=2047, Hq=32, Hkv=8, Hd=64, rot=32, inter=True,
             page=16, lo=0, hi=4000, short=True, spread=3, dtype="fp16"),
        # one token of the vision-language layer into its latent pages
        dict(name="latent append one token", op="latent_append", B=1, T=1, H=32, E=4096, r=32, bits=8, blk=128,
             page=64, lo=1599, hi=1599, spread=0, dtype="bf16"),
        # its image tokens in one block
        dict(name="latent append prompt", op="latent_append", B=1, T=576, H=32, E=4096, r=32, bits=8, blk=128,
             page=64, lo=0, hi=0, spread=0, dtype="bf16"),
        # one token over its latent pages
        dict(name="latent decode llava layer", op="latent_decode", B=1, H=32, Hd=128, r=32, bits=8, page=64, lo=1600,
             hi=1600, spread=0, dtype="bf16"),
        # a ragged serving batch with 4-bit latents
        dict(name="latent decode ragged int4", op="latent_decode", B=16, H=32, Hd=128, r=32, bits=4, page=64, lo=1024,
             hi=4096, spread=1, dtype="fp16"),
        # long documents, 8-bit latents
        dict(name="latent decode long", op="latent_decode", B=4, H=32, Hd=128, r=64, bits=8, page=128, lo=32768,
             hi=32768, spread=0, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["kv_decode", "kv_decode", "kv_append", "kv_append", "latent_decode", "latent_append"])
    page = rng.choice([16, 32, 64, 128, 256])
    dtype = rng.choice(["fp16", "bf16"])
    spread = rng.randrange(1, 1 << 20)
    if op == "kv_decode":
        Hd, Hkv = rng.choice([32, 64, 128, 128, 256]), rng.choice([1, 2, 3, 4, 8, 32])
        G, Tq = rng.choice([1, 2, 3, 4, 7, 8, 16]), rng.choice([1, 1, 1, 2, 4, 7])
        while G * Tq > 64:
            Tq = (Tq + 1) // 2
        hi = _log_int(rng, 1, 32768)
        most = max(1, (500 << 20) // (Hkv * Hd * 4 * max(hi, page)))
        B = _log_int(rng, 1, min(64, most))
        return dict(op=op, B=B, Tq=Tq, Hq=G * Hkv, Hkv=Hkv, Hd=Hd, page=page, lo=rng.choice([0, 1, hi]), hi=hi,
                    spread=spread, dtype=dtype)
    if op == "kv_append":
        Hd, Hkv, G = rng.choice([32, 64, 128, 128, 256]), rng.choice([1, 2, 3, 4, 8, 32]), rng.choice([1, 2, 4, 7, 8])
        T = rng.choice([1, 1, _log_int(rng, 2, 4096)])
        rot = rng.choice([Hd, Hd, Hd // 2, 0])
        most = max(1, (150 << 20) // ((G + 4) * Hkv * Hd * 4 * T))
        return dict(op=op, B=_log_int(rng, 1, min(128, most)), T=T, Hq=G * Hkv, Hkv=Hkv, Hd=Hd, rot=rot,
                    inter=rng.random() < 0.4, page=page, lo=0, hi=_log_int(rng, 1, 8192), short=rng.random() < 0.4,
                    spread=spread, dtype=dtype)
    H = rng.choice([1, 3, 4, 8, 32])
    if op == "latent_append":
        # 8-bit codes: a 4-bit code on a border between two codes moves by a seventh of its row's largest value,
        # which the outputs' type does not allow for; its rows are the same kernel's
        E, T = rng.choice([256, 1024, 2048, 4096]), rng.choice([1, 1, _log_int(rng, 2, 576)])
        return dict(op=op, B=rng.choice([1, 2, 5, 16]) if T == 1 else rng.choice([1, 2, 3]), T=T, H=H, E=E,
                    r=rng.choice([16, 32, 64]), bits=8, blk=rng.choice([1, 64, 128, 256]), page=page, lo=0,
                    hi=_log_int(rng, 1, 1024), spread=spread, dtype=dtype)
    bits = rng.choice([8, 4])
    r = rng.choice([16, 32, 64, 128]) if bits == 8 else rng.choice([32, 64, 128])
    hi = _log_int(rng, 1, 32768)
    most = max(1, (500 << 20) // (H * max(hi, page) * 2 * (r * bits // 8 + 2)))
    return dict(op=op, B=_log_int(rng, 1, min(32, most)), H=H, Hd=rng.choice([32, 64, 128]), r=r, bits=bits, page=page,
                lo=rng.choice([0, 1, hi]), hi=hi, spread=spread, dtype=dtype)


# ----------------------------------------------------------------------------- sizes of a case
def _lens(c):
    """Cached tokens of each sequence before the call (the decodes: all of them)."""
    rng = random.Random(c["spread"])
    return [rng.randint(min(c["lo"], c["hi"]), c["hi"]) for _ in range(c["B"])]


def _news(c):
    """New tokens of each sequence (at most T; the rest of the block is padding)."""
    rng = random.Random(c["spread"] + 1)
    return [rng.randint(0, c["T"]) if c.get("short") else c["T"] for _ in range(c["B"])]


def work(c):
    if c["op"] == "kv_decode":
        n, q = sum(_lens(c)), c["B"] * c["Tq"] * c["Hq"] * c["Hd"]
        return {"bytes": n * c["Hkv"] * c["Hd"] * 4 + q * 6 + c["B"] * 4, "flops": 4.0 * n * c["Tq"] * c["Hq"] * c["Hd"]}
    if c["op"] == "kv_append":
        n = sum(_news(c))
        rows = n * (2 * c["Hkv"] + c["Hq"]) * c["Hd"]
        return {"bytes": 2 * rows * 2 + n * c["rot"] * 4 + 8 * c["B"],
                "flops": 3.0 * n * (c["Hkv"] + c["Hq"]) * c["rot"]}
    rb = c["r"] * c["bits"] // 8
    if c["op"] == "latent_append":
        m = c["B"] * c["T"]
        return {"bytes": 2 * c["H"] * c["E"] * c["r"] * 2 + m * c["E"] * 2 + m * c["H"] * 2 * (rb + 2) + 8 * c["B"],
                "flops": 4.0 * m * c["E"] * c["H"] * c["r"]}
    n = sum(_lens(c)) * c["H"]
    return {"bytes": n * 2 * (rb + 2) + 2 * c["H"] * c["r"] * c["Hd"] * 2 + c["B"] * c["H"] * c["Hd"] * 6 + 4 * c["B"],
            "flops": 4.0 * n * c["r"] + 4.0 * c["B"] * c["H"] * c["r"] * c["Hd"]}


# ----------------------------------------------------------------------------- inputs
_TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=_TYPES[c["dtype"]], gain=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * gain).to(dtype)

    lens, page, B = _lens(c), c["page"], c["B"]
    after = [a + (c["T"] if "T" in c else 0) for a in lens]
    max_pages = max(1, max(-(-a // page) for a in after))
    used = sum(-(-a // page) for a in after)
    pool = used + 3  # pages of this batch, scattered over the pool, and a few of nobody
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table, at = torch.zeros((B, max_pages), dtype=torch.int32, device="cuda"), 0
    for b, a in enumerate(after):
        n = -(-a // page)
        table[b, :n] = order[at:at + n]
        at += n
    s = dict(case=c, block_table=table, seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    if c["op"].startswith("kv"):
        Hkv, Hd = c["Hkv"], c["Hd"]
        s["k_pages"] = normal(pool, Hkv, page, Hd)
        s["v_pages"] = normal(pool, Hkv, page, Hd)
        if c["op"] == "kv_decode":
            s["q"] = normal(B, c["Tq"], c["Hq"], Hd)
            s["out"] = torch.empty((B, c["Tq"], c["Hq"], Hd), device="cuda")
        else:
            # q, k and v as the fused projection leaves them: one row a token
            qkv = normal(B, c["T"], (c["Hq"] + 2 * Hkv) * Hd)
            s["q"], s["k"], s["v"] = (t.unflatten(-1, (-1, Hd)) for t in
                                      qkv.split([c["Hq"] * Hd, Hkv * Hd, Hkv * Hd], dim=-1))
            s["new_lens"] = torch.tensor(_news(c), dtype=torch.int32, device="cuda") if c["short"] else None
            s["q_out"] = torch.empty((B, c["T"], c["Hq"], Hd), dtype=qkv.dtype, device="cuda")
            s["lens_out"] = torch.empty_like(s["seq_lens"])
            s["cos_sin"] = None
            if c["rot"]:
                half = c["rot"] // 2
                freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
                angle = torch.arange(max_pages * page, dtype=torch.float64, device="cuda")[:, None] * freq
                s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], dim=1).float()
    else:
        H, r, bits = c["H"], c["r"], c["bits"]
        top = 127 if bits == 8 else 7
        for x in "kv":
            codes = torch.randint(-top, top + 1, (pool, H, page, r), generator=g, device="cuda", dtype=torch.int8)
            if bits == 4:
                codes = (codes[..., 0::2] & 15) | (codes[..., 1::2] << 4)
            s["lat_" + x] = codes.view(torch.uint8)
            s["scale_" + x] = (torch.rand((pool, H, page), generator=g, device="cuda") + 1.0).div(top).half()
        if c["op"] == "latent_decode":
            s["q"] = normal(B, H, c["Hd"])
            for x in "kv":
                s["B_" + x] = normal(H, r, c["Hd"], dtype=torch.float16, gain=r ** -0.5)
            s["out"] = torch.empty((B, H, c["Hd"]), device="cuda")
        else:
            s["x"] = normal(B, c["T"], c["E"])
            for x in "kv":
                s["A_" + x] = normal(H, c["E"], r, dtype=torch.float16, gain=c["E"] ** -0.5)
            s["lens_out"] = torch.empty_like(s["seq_lens"])
    if own:  # the scratch that a serving loop keeps
        import rank_kv_cache_wsvd_b200 as W
        if c["op"] == "kv_decode":
            s["ws"] = W.workspace(W.paged_decode_workspace_size(B, c["Tq"], c["Hq"], c["Hkv"], c["Hd"]))
        elif c["op"] == "kv_append":
            s["ws"] = W.workspace(W.paged_kv_append_workspace_size(B))
        elif c["op"] == "latent_decode":
            s["ws"] = W.workspace(W.wsvd_decode_workspace_size(B, c["H"], c["r"]))
        else:
            s["ws"] = W.workspace(W.wsvd_latent_append_paged_workspace_size(B, c["T"], c["E"]))
    return s


# ----------------------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    if own:
        return _own(s)
    return {"kv_decode": _kv_decode, "kv_append": _kv_append, "latent_decode": _latent_decode,
            "latent_append": _latent_append}[c["op"]](s, c)


def _values(s, x):
    """The values that latent pages stand for."""
    return _codes(s["lat_" + x], s["case"]["bits"]) * s["scale_" + x][..., None]


def _codes(lat, bits):
    """The integers of 8- or 4-bit codes (4 bits: element 2j in the low half of byte j)."""
    lat = lat.view(torch.int8)
    return lat if bits == 8 else torch.stack([(lat << 4) >> 4, lat >> 4], dim=-1).flatten(-2)


def _own(s):
    import rank_kv_cache_wsvd_b200 as W
    c = s["case"]
    if c["op"] == "kv_decode":
        return W.paged_decode_attention(s["q"], s["k_pages"], s["v_pages"], s["block_table"], s["seq_lens"],
                                        out=s["out"], workspace_buf=s["ws"])
    if c["op"] == "kv_append":
        W.paged_kv_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["block_table"], s["seq_lens"], q=s["q"],
                          q_out=s["q_out"], cos_sin=s["cos_sin"], interleaved=c["inter"], new_lens=s["new_lens"],
                          seq_lens_out=s["lens_out"], workspace_buf=s["ws"])
        return s["q_out"], s["k_pages"], s["v_pages"], s["lens_out"]
    if c["op"] == "latent_decode":
        return W.wsvd_decode_attention_paged(s["q"], s["lat_k"], s["lat_v"], s["scale_k"], s["scale_v"], s["B_k"],
                                             s["B_v"], s["block_table"], s["seq_lens"], bits=c["bits"], out=s["out"],
                                             workspace_buf=s["ws"])
    W.wsvd_latent_append_paged(s["x"], s["A_k"], s["A_v"], s["seq_lens"], s["block_table"], s["lat_k"], s["lat_v"],
                               s["scale_k"], s["scale_v"], bits=c["bits"], hadamard_block=c["blk"],
                               seq_lens_out=s["lens_out"], workspace_buf=s["ws"])
    return _values(s, "k"), _values(s, "v"), s["lens_out"]


def _rows(pages, table):
    """Pages [N][H][page][...] of each sequence as rows [B][H][max_pages * page][...]."""
    return pages[table.long()].transpose(1, 2).flatten(2, 3)


def _kv_decode(s, c):
    B, Tq, Hkv, Hd = c["B"], c["Tq"], c["Hkv"], c["Hd"]
    G = c["Hq"] // Hkv
    K, V = (_rows(s[x], s["block_table"]).float() for x in ("k_pages", "v_pages"))
    q = s["q"].float().view(B, Tq, Hkv, G, Hd).permute(0, 2, 1, 3, 4).flatten(2, 3)      # [B][Hkv][Tq * G][Hd]
    score = q @ K.transpose(-1, -2) * Hd ** -0.5
    row = torch.arange(K.shape[2], device=K.device)
    sees = s["seq_lens"].long()[:, None] - Tq + 1 + torch.arange(Tq, device=K.device)     # [B][Tq]
    seen = (row < sees[..., None]).repeat_interleave(G, dim=1)[:, None]                   # [B][1][Tq * G][rows]
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top.masked_fill(top == -math.inf, 0))
    V = V.masked_fill(~(row < s["seq_lens"].long()[:, None])[:, None, :, None], 0)
    out = p @ V / p.sum(-1, keepdim=True).clamp_min(1e-37)
    return out.view(B, Hkv, Tq, G, Hd).permute(0, 2, 1, 3, 4).reshape(B, Tq, c["Hq"], Hd)


def _turn(x, cos, sin, rot, inter):
    """The rotation of the first `rot` values of each head, x [B][T][heads][Hd] in fp32."""
    if not rot:
        return x
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
    y, z = a * cos - b * sin, b * cos + a * sin
    return torch.cat([torch.stack([y, z], -1).flatten(-2) if inter else torch.cat([y, z], -1), x[..., rot:]], -1)


def _kv_append(s, c):
    B, T, rot, page = c["B"], c["T"], c["rot"], c["page"]
    dev = s["k"].device
    lens = s["seq_lens"].long()
    t = torch.arange(T, device=dev)
    new = s["new_lens"].long() if s["new_lens"] is not None else torch.full((B,), T, device=dev)
    there = t < new[:, None]                                                              # [B][T]
    row = (lens[:, None] + t).clamp_max(s["block_table"].shape[1] * page - 1)
    cos, sin = s["cos_sin"][row][:, :, None].chunk(2, dim=-1) if rot else (None, None)
    q, k = (_turn(s[x].float(), cos, sin, rot, c["inter"]).to(s[x].dtype) for x in "qk")
    at = (s["block_table"].gather(1, row // page).long(), row % page)
    at = (at[0][there], at[1][there])
    s["k_pages"][at[0], :, at[1]] = k[there]
    s["v_pages"][at[0], :, at[1]] = s["v"][there]
    return q.masked_fill(~there[..., None, None], 0), s["k_pages"], s["v_pages"], (lens + new).int()


def _latent_decode(s, c):
    row = torch.arange(s["block_table"].shape[1] * c["page"], device=s["q"].device)
    seen = (row < s["seq_lens"].long()[:, None])[:, None]                                 # [B][1][rows]
    lat = [_rows(_codes(s["lat_" + x], c["bits"]), s["block_table"]).float()
           * _rows(s["scale_" + x], s["block_table"]).float()[..., None] for x in "kv"]
    K, V = lat[0] @ s["B_k"].float(), lat[1] @ s["B_v"].float()
    score = (K @ s["q"].float()[..., None])[..., 0] * c["Hd"] ** -0.5
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top.masked_fill(top == -math.inf, 0))
    return (p[..., None, :] @ V)[..., 0, :] / p.sum(-1, keepdim=True).clamp_min(1e-37)


def _hadamard(n, device, dtype):
    i = torch.arange(n, device=device)
    both, sign = i[:, None] & i, torch.zeros((n, n), dtype=torch.long, device=device)
    for bit in range(n.bit_length()):
        sign ^= (both >> bit) & 1
    return (1 - 2 * sign).to(dtype) * n ** -0.5


def _latent_append(s, c):
    B, T, page, top = c["B"], c["T"], c["page"], 127 if c["bits"] == 8 else 7
    x = s["x"].float().unflatten(-1, (-1, c["blk"])) @ _hadamard(c["blk"], s["x"].device, torch.float32)
    row = s["seq_lens"].long()[:, None] + torch.arange(T, device=x.device)
    at = (s["block_table"].gather(1, row // page).long(), row % page)
    for k in "kv":
        lat = torch.einsum("bte,her->bthr", x.flatten(-2), s["A_" + k].float())
        scale = (lat.abs().amax(-1) / top).half()
        code = torch.round(lat / scale.float().clamp_min(1e-37)[..., None]).clamp(-top, top).to(torch.int8)
        if c["bits"] == 4:
            code = (code[..., 0::2] & 15) | (code[..., 1::2] << 4)
        s["lat_" + k][at[0], :, at[1]] = code.view(torch.uint8)
        s["scale_" + k][at[0], :, at[1]] = scale
    return _values(s, "k"), _values(s, "v"), (s["seq_lens"] + T).int()


# ----------------------------------------------------------------------------- 64-bit values
def exact(c, seed):
    s = prepare(c, seed)
    lens, page = _lens(c), c["page"]
    table = s["block_table"].tolist()

    def rows(pages, b, n):  # rows [n][heads][...] of sequence b, page by page
        got = [pages[table[b][i]].transpose(0, 1)[:min(page, n - i * page)] for i in range(-(-n // page))]
        return torch.cat(got).double()

    if c["op"] == "kv_decode":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        G = c["Hq"] // c["Hkv"]
        for b, n in enumerate(lens):
            if not n:
                continue
            K, V = (rows(s[x], b, n).transpose(0, 1) for x in ("k_pages", "v_pages"))     # [Hkv][n][Hd]
            for t in range(c["Tq"]):
                m = n - c["Tq"] + 1 + t
                if m > 0:
                    q = s["q"][b, t].double().view(c["Hkv"], G, c["Hd"])
                    p = torch.softmax(torch.einsum("hgd,hnd->hgn", q, K[:, :m]) / math.sqrt(c["Hd"]), dim=-1)
                    out[b, t] = torch.einsum("hgn,hnd->hgd", p, V[:, :m]).reshape(c["Hq"], c["Hd"])
        return out
    if c["op"] == "kv_append":
        rot, half = c["rot"], c["rot"] // 2
        kp, vp = s["k_pages"].double(), s["v_pages"].double()
        q_out = torch.zeros(s["q_out"].shape, dtype=torch.float64, device="cuda")
        news = _news(c)
        for b, n in enumerate(news):
            if not n:
                continue
            turned = []
            for x in "qk":
                z = s[x][b, :n].double().clone()
                if rot:
                    cs = s["cos_sin"][lens[b]:lens[b] + n].double()[:, None]
                    i = torch.arange(half, device="cuda") * (2 if c["inter"] else 1)
                    j = i + (1 if c["inter"] else half)
                    u, w = z[..., i], z[..., j]
                    z[..., i], z[..., j] = u * cs[..., :half] - w * cs[..., half:], w * cs[..., :half] + u * cs[..., half:]
                turned.append(z)
            q_out[b, :n] = turned[0]
            where = torch.tensor([(table[b][l // page], l % page) for l in range(lens[b], lens[b] + n)], device="cuda")
            kp[where[:, 0], :, where[:, 1]] = turned[1]
            vp[where[:, 0], :, where[:, 1]] = s["v"][b, :n].double()
        return q_out, kp, vp, None
    if c["op"] == "latent_decode":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            if not n:
                continue
            lk, lv = (rows(_codes(s["lat_" + x], c["bits"]), b, n) * rows(s["scale_" + x], b, n)[..., None]
                      for x in "kv")                                                        # [n][H][r]
            qp = torch.einsum("hrd,hd->hr", s["B_k"].double(), s["q"][b].double())
            p = torch.softmax(torch.einsum("nhr,hr->hn", lk, qp) / math.sqrt(c["Hd"]), dim=-1)
            out[b] = torch.einsum("hr,hrd->hd", torch.einsum("hn,nhr->hr", p, lv), s["B_v"].double())
        return out
    top, got = 127 if c["bits"] == 8 else 7, []
    x = s["x"].double().view(c["B"], c["T"], -1, c["blk"])
    n = 1
    while n < c["blk"]:  # the Hadamard rotation by its own recursion
        x = x.unflatten(-1, (-1, 2, n))
        x = torch.stack([x[..., 0, :] + x[..., 1, :], x[..., 0, :] - x[..., 1, :]], dim=-2).flatten(-3)
        n *= 2
    x = (x / math.sqrt(c["blk"])).reshape(c["B"], c["T"], c["E"])
    for k in "kv":
        whole = _codes(s["lat_" + k], c["bits"]).double() * s["scale_" + k].double()[..., None]
        for h in range(c["H"]):
            lat = x @ s["A_" + k][h].double()
            scale = (lat.abs().amax(-1, keepdim=True) / top).half().double()
            lat = torch.where(scale > 0, torch.round(lat / scale).clamp(-top, top) * scale, torch.zeros_like(lat))
            for b in range(c["B"]):
                l = torch.arange(lens[b], lens[b] + c["T"], device="cuda")
                whole[s["block_table"][b].long()[l // page], h, l % page] = lat[b]
        got.append(whole)
    return got[0], got[1], None
