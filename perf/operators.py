"""The serving operators around the MXINT K/V cache: rotary positions, writing
new tokens into the cache and reading them back, and attention of drafted
tokens over it.  Each case is one call (or, for the cache, one write and the
read of what it wrote) as a program that serves a model makes it.

With ``own`` false the operators run in plain torch operations; with ``own``
true through this repository's binding.  ``exact`` gives the 64-bit values.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 32


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the query heads of a decode step: a slice of the fused projection's output, one row per sequence
        dict(name="rope_decode", op="rope", T=32, heads=32, d=128, rot=128, half=True, scaling="none", f32=False,
             inverse=False, sliced=True, far=8192),
        # the query heads of a prompt at positions of a context stretched by wavelength
        dict(name="rope_prompt", op="rope", T=8192, heads=32, d=128, rot=128, half=True, scaling="parts", f32=False,
             inverse=False, sliced=False, far=131072),
        # a quarter of wide heads rotated, interleaved pairs, fp32, the gradient's direction (the inverse rotation)
        dict(name="rope_part_back", op="rope", T=4099, heads=16, d=256, rot=64, half=False, scaling="yarn", f32=True,
             inverse=True, sliced=False, far=1000003),
        # the new tokens of a decode step over 16 sequences
        dict(name="cache_step", op="cache", T=16, heads=8, d=128, rot=128, half=True, scaling="none", f32=False, bits=4,
             page=16, slots=131072, far=8192),
        # the K/V tokens of a prompt: the 8192-token, 8-head cache of the decode workload, in pages
        dict(name="cache_prompt", op="cache", T=8192, heads=8, d=128, rot=128, half=True, scaling="parts", f32=False,
             bits=4, page=64, slots=32768, far=131072),
        # 8-bit cache of short heads, fp32 keys with half of each head rotated, an odd number of heads and tokens
        dict(name="cache_kv8", op="cache", T=3001, heads=5, d=64, rot=32, half=False, scaling="linear", f32=True, bits=8,
             page=7, slots=6000, far=65536),
        # a long context read back for a dense kernel
        dict(name="cache_read_long", op="read", T=131072, heads=8, d=128, f32=False, bits=4, page=16, slots=140000),
        # one new token over the 8192-token cache: the framework's decode step
        dict(name="tree_token", op="tree", B=1, L=8192, nq=1, n_qh=32, n_kvh=8, d=128, bits=4, page=64, causal=True,
             f32=True, lse=False),
        # trees of up to 16 drafted tokens over ragged contexts, the usual speculative step of a small batch
        dict(name="tree_draft", op="tree", B=8, L=4096, nq=16, n_qh=32, n_kvh=8, d=128, bits=4, page=16, causal=False,
             f32=False, lse=False),
        # a larger batch over an 8-bit cache of short heads with three query heads each, odd pages, fp32 output
        dict(name="tree_batch_kv8", op="tree", B=32, L=8191, nq=7, n_qh=24, n_kvh=8, d=64, bits=8, page=33, causal=False,
             f32=True, lse=False),
        # 64-token trees over long contexts, eight query heads per K/V head
        dict(name="tree_long", op="tree", B=2, L=65536, nq=64, n_qh=64, n_kvh=8, d=128, bits=4, page=64, causal=False,
             f32=False, lse=True),
        # a further chunk of a prompt (causal among its own tokens) over what the cache holds
        dict(name="tree_chunk", op="tree", B=3, L=3001, nq=211, n_qh=32, n_kvh=8, d=128, bits=4, page=16, causal=True,
             f32=False, lse=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "cache", "read", "tree", "tree"])
    d = rng.choice([64, 128])
    if op == "tree":
        rep = rng.choice([1, 2, 3, 4, 6, 8])
        n_kvh = rng.choice([1, 2, 5, 8])
        L, B, nq = _log(rng, 40, 65536), _log(rng, 1, 32), _log(rng, 1, 192)
        while B * L > 131072 or B * L * nq * rep * n_kvh > 2 * 65536 * 64 * 64:
            L, B, nq = max(40, L * 2 // 3), max(1, B * 2 // 3), max(1, nq * 2 // 3)
        return dict(op=op, B=B, L=max(L, nq + 1), nq=nq, n_qh=rep * n_kvh, n_kvh=n_kvh, d=d, bits=rng.choice([4, 4, 8]),
                    page=rng.choice([1, 5, 16, 33, 64, 128]), causal=rng.random() < 0.4, f32=rng.random() < 0.4,
                    lse=rng.random() < 0.3)
    if op == "rope":
        d = rng.choice([64, 96, 128, 256])
        return dict(op=op, T=_log(rng, 1, 8192), heads=rng.choice([1, 5, 8, 16, 32]), d=d, rot=rng.choice([d, d // 2, d // 4]),
                    half=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "parts", "yarn"]), f32=rng.random() < 0.4,
                    inverse=rng.random() < 0.3, sliced=rng.random() < 0.5, far=_log(rng, 9000, 1 << 20))
    if op == "read":
        T = _log(rng, 1, 100000)
        return dict(op=op, T=T, heads=rng.choice([1, 5, 8]), d=d, f32=rng.random() < 0.3, bits=rng.choice([4, 8]),
                    page=rng.choice([1, 16, 33, 64]), slots=T + 200)
    T = _log(rng, 1, 8192)
    return dict(op=op, T=T, heads=rng.choice([1, 5, 8]), d=d, rot=rng.choice([d, d // 2]), half=rng.random() < 0.5,
                scaling=rng.choice(["none", "linear", "parts", "yarn"]), f32=rng.random() < 0.4, bits=rng.choice([4, 8]),
                page=rng.choice([1, 16, 33, 64]), slots=T + 200, far=_log(rng, 9000, 1 << 20))


THETA = 500000.0
SCALING = {
    "none": None,
    "linear": dict(kind="linear", factor=4.0),
    "parts": dict(kind="parts", factor=8.0, low=1.0, high=4.0, orig_len=8192),
    "yarn": dict(kind="yarn", factor=16.0, orig_len=8192, beta_fast=32.0, beta_slow=1.0),
}


def _counts(case):
    """(context length, drafted tokens) of each sequence: ragged, fixed by the case; the first is the longest."""
    B, L, nq = case["B"], case["L"], case["nq"]
    n = [max(1, nq - (3 * b) % (nq // 2 + 1)) for b in range(B)]
    total = [max(n[b], L - (b * L) // (2 * B)) for b in range(B)]
    return [t - m for t, m in zip(total, n)], n


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _pages(slots_needed, pool, page, g):
    """A table of pages, in random order of the pool, that holds `slots_needed` tokens."""
    return torch.randperm(pool // page, generator=g, device=DEV)[: -(-slots_needed // page)].to(torch.int32)


def _random_cache(rows, d, bits, g):
    """Packed codes and scale bytes of N(0, 1) rows with a few large channels."""
    codes, scales = [], []
    for r0 in range(0, rows, 1 << 19):
        x = torch.randn((min(1 << 19, rows - r0), d), generator=g, device=DEV)
        x[:, :: d // 4] *= 4.0
        c, s = _code(x, bits)
        codes.append(c)
        scales.append(s)
    return torch.cat(codes), torch.cat(scales)


def _tree_masks(n, words, g):
    """Packed masks (32-bit words) of random trees: token i follows a random earlier token, or the context."""
    B, m = len(n), max(n)
    parent = (torch.rand((B, m), generator=g, device=DEV) * (torch.arange(m, device=DEV) + 1)).long() - 1
    reach = torch.eye(m, device=DEV).repeat(B, 1, 1)
    step = torch.zeros((B, m, m + 1), device=DEV).scatter_(2, (parent + 1).unsqueeze(2), 1.0)[:, :, 1:]
    reach = ((reach + step) > 0).float()
    for _ in range(max(1, m.bit_length())):
        reach = (reach @ reach > 0).float()
    bits = torch.zeros((B, m, words * 32), device=DEV, dtype=torch.int64)
    bits[:, :, :m] = reach.long()
    packed = (bits.view(B, m, words, 32) << torch.arange(32, device=DEV)).sum(-1).to(torch.int32)
    return torch.cat([packed[b, : n[b]] for b in range(B)])


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    dt = torch.float32 if case["f32"] else torch.bfloat16
    if own:
        from mx_microscaling_mixed_b200 import capi as c
        s["c"] = c
        if "rot" in case:
            s["plan"] = c.mxs_rope_plan(case["rot"], theta=THETA, layout="half" if case["half"] else "interleaved",
                                        scaling=SCALING[case["scaling"]])
    if case["op"] == "rope":
        T, h, d = case["T"], case["heads"], case["d"]
        x = torch.randn((T, (h + 2 * max(1, h // 4) if case["sliced"] else h) * d), generator=g, device=DEV).to(dt)
        s["x"] = x[:, : h * d].view(T, h, d) if not case["sliced"] else x[:, : h * d].unflatten(1, (h, d))
        start = torch.randint(0, max(1, case["far"] - T), (1,), generator=g, device=DEV)
        s["pos"] = (torch.randint(0, case["far"], (T,), generator=g, device=DEV) if case["sliced"]
                    else start + torch.arange(T, device=DEV))
        return s
    if case["op"] in ("cache", "read"):
        T, h, d = case["T"], case["heads"], case["d"]
        t = torch.arange(T, device=DEV)
        table = _pages(T, case["slots"], case["page"], g).long()
        s["slot"] = table[t // case["page"]] * case["page"] + t % case["page"]
        s["pools"] = [_random_cache(case["slots"] * h, d, case["bits"], g) for _ in range(2)]
        if case["op"] == "cache":
            qkv = torch.randn((T, 4 * h * d), generator=g, device=DEV)                  # 2 h query heads before them
            qkv[:, :: d // 4] *= 4.0
            qkv = qkv.to(dt)
            s["k"] = qkv[:, 2 * h * d: 3 * h * d].unflatten(1, (h, d))
            s["v"] = qkv[:, 3 * h * d:].unflatten(1, (h, d))
            s["pos"] = torch.randint(0, max(1, case["far"] - T), (1,), generator=g, device=DEV) + t
        n_slots, n_kvh = case["slots"], h
    else:
        ctx, n = _counts(case)
        B, d, page, n_kvh = case["B"], case["d"], case["page"], case["n_kvh"]
        rows, s["max_q"], s["max_len"] = sum(n), max(n), max(a + b for a, b in zip(ctx, n))
        per = -(-s["max_len"] // page)
        n_slots = (B * per + 3) * page
        s["pages"] = _pages(B * per * page, n_slots, page, g).view(B, per)
        s["length"] = torch.tensor(ctx, device=DEV, dtype=torch.int32)
        s["q_start"] = torch.tensor([sum(n[:b]) for b in range(B + 1)], device=DEV, dtype=torch.int32)
        s["q"] = torch.randn((rows, case["n_qh"], d), generator=g, device=DEV).to(torch.bfloat16)
        s["mask"] = None if case["causal"] else _tree_masks(n, -(-s["max_q"] // 32), g)
        s["pools"] = [_random_cache(n_slots * n_kvh, d, case["bits"], g) for _ in range(2)]
        s["scale"] = d ** -0.5
    if own:
        s["cache"] = s["c"].kv_cache_empty(n_slots, n_kvh, case["d"], bits=case["bits"])
        seg = 2 if case["bits"] == 4 else 0
        for t, (codes, scales) in zip((s["cache"].K, s["cache"].V), s["pools"]):
            t.code_rows(seg).copy_(codes)
            t.scale_rows(seg).copy_(scales)
        s["pools"] = None
        if case["op"] == "tree":
            s["batch"] = s["c"].tree_batch(s["q_start"], s["length"], s["pages"], page, max_q=s["max_q"],
                                           max_len=s["max_len"], mask=s["mask"])
            s["ws"] = s["c"].attn_tree_workspace(s["q"], s["cache"], s["batch"])
    return s


# ------------------------------------------------------------- plain forms
def _freqs(rot, scaling):
    """(angle per position, 64 bits; factor of cos and sin)."""
    i = torch.arange(rot // 2, device=DEV, dtype=torch.float64)
    f = THETA ** (-2.0 * i / rot)
    p = SCALING[scaling]
    if p is None:
        return f, 1.0
    if p["kind"] == "linear":
        return f / p["factor"], 1.0
    if p["kind"] == "parts":
        turns = p["orig_len"] * f / (2.0 * math.pi)
        keep = ((turns - p["low"]) / (p["high"] - p["low"])).clamp(0.0, 1.0)
        return f * (keep + (1.0 - keep) / p["factor"]), 1.0
    edge = [rot * math.log(p["orig_len"] / (2.0 * math.pi * b)) / (2.0 * math.log(THETA)) for b in (p["beta_fast"], p["beta_slow"])]
    lo, hi = max(0.0, math.floor(edge[0])), min(rot - 1.0, math.ceil(edge[1]))
    keep = 1.0 - ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
    return f * (keep + (1.0 - keep) / p["factor"]), 0.1 * math.log(p["factor"]) + 1.0


def _rotate(x, pos, rot, half, scaling, inverse, work):
    """Rotated heads, computed in `work` (angles always in 64 bits)."""
    f, gain = _freqs(rot, scaling)
    a = pos.double()[:, None, None] * f
    cos, sin = (a.cos() * gain).to(work), (a.sin() * (-gain if inverse else gain)).to(work)
    y = x.to(work)
    u, v = (y[..., : rot // 2], y[..., rot // 2: rot]) if half else (y[..., 0:rot:2], y[..., 1:rot:2])
    ru, rv = u * cos - v * sin, v * cos + u * sin
    turned = torch.cat([ru, rv], -1) if half else torch.stack([ru, rv], -1).flatten(-2)
    return torch.cat([turned, y[..., rot:]], -1)


def _two_to(e):
    """2^e for integers e, exactly: 64 bits, from the exponent field."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _code(x, bits):
    """fp32 rows -> (packed codes, scale bytes), blocks of 32 along the row."""
    b = x.unflatten(-1, (-1, BLOCK))
    byte = (b.abs().amax(-1).view(torch.int32) >> 23)
    step = _two_to(byte - 127 - bits + 2).float()
    top = 2 ** (bits - 1) - 1
    q = (b / step[..., None]).round().clamp(-top, top).flatten(-2).to(torch.int32)
    if bits == 4:
        q = (q[..., 0::2] & 15) | ((q[..., 1::2] & 15) << 4)
    return (q & 255).to(torch.uint8), byte.to(torch.uint8)


def _values(codes, scales, bits):
    """The fp32 values that packed codes and scale bytes stand for."""
    c = codes.to(torch.int32)
    if bits == 4:
        c = torch.stack([c & 15, c >> 4], -1).flatten(-2)
    c = torch.where(c >= 2 ** (bits - 1), c - 2 ** bits, c).float().unflatten(-1, (-1, BLOCK))
    return (c * _two_to(scales.long() - 127 - bits + 2).float()[..., None]).flatten(-2)


def _plain_attention(s):
    B, n_kvh, d, nq, L = s["B"], s["n_kvh"], s["d"], s["max_q"], s["max_len"]
    rep, rows = s["n_qh"] // n_kvh, s["q"].shape[0]
    p = torch.arange(L, device=DEV)
    slot = s["pages"].long()[:, p // s["page"]] * s["page"] + p % s["page"]
    at = slot[..., None] * n_kvh + torch.arange(n_kvh, device=DEV)
    k, v = (_values(c[at], e[at], s["bits"]) for c, e in s["pools"])                # B, L, n_kvh, d
    start, ctx = s["q_start"].long(), s["length"].long()
    i = torch.arange(nq, device=DEV)
    row = (start[:-1, None] + i).clamp(max=rows - 1)                               # B, nq
    q = s["q"][row].float().view(B, nq, n_kvh, rep, d)
    x = torch.einsum("bighd,blgd->bgihl", q, k) * s["scale"]
    j = p - ctx[:, None]                                                           # B, L: drafted token at this place
    if s["mask"] is None:
        see = j[:, None, :] <= i[None, :, None]
    else:
        word = s["mask"].long()[row]                                               # B, nq, words
        t = j.clamp(0, 32 * word.shape[-1] - 1)
        see = (torch.gather(word, 2, (t // 32)[:, None, :].expand(B, nq, L)) >> (t % 32)[:, None, :]) & 1 > 0
        see |= (j < 0)[:, None, :]
    see &= (j < (start[1:] - start[:-1])[:, None])[:, None, :]
    x = x.masked_fill(~see[:, None, :, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    e = (x - torch.where(top.isfinite(), top, 0.0)).exp()
    total = e.sum(-1)                                                              # B, g, i, h
    o = torch.einsum("bgihl,blgd->bighd", e, v) / total.permute(0, 2, 1, 3).clamp(min=1e-38)[..., None]
    of = torch.arange(rows, device=DEV)
    b = torch.bucketize(of, start[1:], right=True)
    o = o.reshape(B, nq, s["n_qh"], d)[b, of - start[b]]
    lse = (top[..., 0] + total.log()).permute(0, 2, 1, 3).reshape(B, nq, s["n_qh"])[b, of - start[b]]
    return o.to(torch.float32 if s["f32"] else torch.bfloat16), lse


def run(s):
    dt = torch.float32 if s["f32"] else torch.bfloat16
    if own:
        c = s["c"]
        if s["op"] == "rope":
            return c.mxs_rope(s["x"], s["pos"], s["plan"], inverse=s["inverse"])
        if s["op"] == "tree":
            if s["lse"]:
                return c.mxs_attn_tree(s["q"], s["cache"], s["batch"], s["scale"], dtype=dt, return_lse=True, workspace=s["ws"])
            return c.mxs_attn_tree(s["q"], s["cache"], s["batch"], s["scale"], dtype=dt, workspace=s["ws"])
        if s["op"] == "cache":
            c.mxs_kv_write(s["k"], s["v"], s["cache"], s["slot"], pos=s["pos"], rope=s["plan"])
        return c.mxs_kv_read(s["cache"], s["slot"], dtype=torch.bfloat16 if s["op"] == "cache" else dt)
    if s["op"] == "rope":
        return _rotate(s["x"], s["pos"], s["rot"], s["half"], s["scaling"], s["inverse"], torch.float32).to(dt)
    if s["op"] == "tree":
        o, lse = _plain_attention(s)
        return (o, lse) if s["lse"] else o
    at = s["slot"][:, None] * s["heads"] + torch.arange(s["heads"], device=DEV)
    if s["op"] == "cache":
        # the keys' codes stand next to borders of the rounding: 64 bits, one rounding to fp32, then the coding
        k = _rotate(s["k"], s["pos"], s["rot"], s["half"], s["scaling"], False, torch.float64).float()
        for (codes, scales), x in zip(s["pools"], (k, s["v"].float())):
            codes[at], scales[at] = _code(x, s["bits"])
        dt = torch.bfloat16
    return tuple(_values(codes[at], scales[at], s["bits"]).to(dt) for codes, scales in s["pools"])


# -------------------------------------------------------------------- work
def work(case):
    if case["op"] == "tree":
        ctx, n = _counts(case)
        d, h, g = case["d"], case["n_qh"], case["n_kvh"]
        row = d * case["bits"] // 8 + d // BLOCK
        cache = sum(a + b for a, b in zip(ctx, n)) * g * 2 * row
        masks = 0 if case["causal"] else sum(n) * (-(-max(n) // 32)) * 4
        own_pairs = [m * (m + 1) // 2 if case["causal"] else m for m in n]
        pairs = sum(a * m for a, m in zip(ctx, n)) + sum(own_pairs)
        io = sum(n) * h * (d * (2 + (4 if case["f32"] else 2)) + (4 if case["lse"] else 0))
        return {"bytes": cache + masks + io, "flops": 4.0 * d * h * pairs}
    T, h, d, size = case["T"], case["heads"], case["d"], 4 if case["f32"] else 2
    if case["op"] == "rope":
        return {"bytes": T * h * d * 2 * size + T * 8, "flops": 3.0 * T * h * case["rot"]}
    row = d * case["bits"] // 8 + d // BLOCK
    if case["op"] == "read":
        return {"bytes": 2 * T * h * (row + d * size) + T * 8, "flops": 2.0 * T * h * d}
    # written from k and v, then read back in bf16
    return {"bytes": 2 * T * h * (d * size + 2 * row + 2 * d) + T * 16, "flops": T * h * (3.0 * case["rot"] + 6.0 * d)}


# -------------------------------------------------- the definition, 64 bits
def _exact_rotation(x, pos, case, inverse):
    """Pairs as complex numbers, turned by exp(i pos f)."""
    rot, p = case["rot"], SCALING[case["scaling"]]
    f, gain = [], 1.0
    for i in range(rot // 2):
        w = THETA ** (-2.0 * i / rot)
        if p is not None and p["kind"] == "linear":
            w = w / p["factor"]
        elif p is not None and p["kind"] == "parts":
            length = 2.0 * math.pi / w
            if length > p["orig_len"] / p["low"]:
                w = w / p["factor"]
            elif length >= p["orig_len"] / p["high"]:
                mix = (p["orig_len"] / length - p["low"]) / (p["high"] - p["low"])
                w = (1.0 - mix) * w / p["factor"] + mix * w
        elif p is not None:
            gain = 0.1 * math.log(p["factor"]) + 1.0
            def place(turns):
                return rot * math.log(p["orig_len"] / (turns * 2.0 * math.pi)) / (2.0 * math.log(THETA))
            lo, hi = max(0, math.floor(place(p["beta_fast"]))), min(rot - 1, math.ceil(place(p["beta_slow"])))
            ramp = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            w = w / p["factor"] * ramp + w * (1.0 - ramp)
        f.append(w)
    angle = torch.outer(pos.to(torch.float64), torch.tensor(f, dtype=torch.float64, device=DEV))
    turn = torch.polar(torch.full_like(angle, gain), -angle if inverse else angle).unsqueeze(1)
    head, rest = x.double()[..., :rot], x.double()[..., rot:]
    pairs = head.unflatten(-1, (2, rot // 2)).transpose(-1, -2) if case["half"] else head.unflatten(-1, (rot // 2, 2))
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    z = z.transpose(-1, -2).flatten(-2) if case["half"] else z.flatten(-2)
    return torch.cat([z, rest], -1)


def _exact_coded(x, bits):
    """What x (64-bit rows) stands for once coded in blocks of 32."""
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    _, e = torch.frexp(b.abs().max(dim=-1, keepdim=True).values)                   # max = m 2^e, m in [0.5, 1)
    scale = torch.tensor([2.0 ** n for n in range(-140, 140)], dtype=torch.float64, device=DEV)[(e - 1 - bits + 2).long() + 140]
    lim = float(2 ** (bits - 1) - 1)
    return (torch.clamp(torch.round(b / scale), -lim, lim) * scale).reshape(x.shape)


def _exact_values(codes, scales, bits):
    n = codes.shape[:-1]
    if bits == 4:
        signed = (torch.arange(16, device=DEV) + 8) % 16 - 8                       # value of each 4-bit code
        q = torch.stack([signed[(codes % 16).long()], signed[(codes // 16).long()]], dim=-1).reshape(*n, -1)
    else:
        q = codes.view(torch.int8)
    step = torch.tensor([2.0 ** (n - 127 - bits + 2) for n in range(256)], dtype=torch.float64, device=DEV)[scales.long()]
    return q.double() * step.repeat_interleave(32, dim=-1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rotation(s["x"], s["pos"], case, case["inverse"])
    if case["op"] == "cache":
        # the operator rounds the rotated keys to fp32 before it codes them
        k = _exact_rotation(s["k"], s["pos"], case, False).float().double()
        return _exact_coded(k, case["bits"]), _exact_coded(s["v"].double(), case["bits"])
    if case["op"] == "read":
        h = torch.arange(case["heads"], device=DEV)
        out = []
        for codes, scales in s["pools"]:
            rows = (s["slot"][:, None] * case["heads"] + h).reshape(-1)
            out.append(_exact_values(codes[rows], scales[rows], case["bits"]).reshape(case["T"], case["heads"], case["d"]))
        return tuple(out)
    ctx, n = _counts(case)
    rep, outs, lses, first = case["n_qh"] // case["n_kvh"], [], [], 0
    for b in range(case["B"]):
        total = ctx[b] + n[b]
        slots = torch.cat([s["pages"][b, i].long() * case["page"] + torch.arange(case["page"], device=DEV)
                           for i in range(-(-total // case["page"]))])[:total] if total <= 4096 else (
            (s["pages"][b].long()[:, None] * case["page"] + torch.arange(case["page"], device=DEV)).reshape(-1)[:total])
        o = torch.empty((n[b], case["n_qh"], case["d"]), dtype=torch.float64, device=DEV)
        l = torch.empty((n[b], case["n_qh"]), dtype=torch.float64, device=DEV)
        see = torch.ones((n[b], total), dtype=torch.bool, device=DEV)
        if case["causal"]:
            see[:, ctx[b]:] = torch.ones((n[b], n[b]), device=DEV).tril() > 0
        else:
            m = s["mask"][first: first + n[b]].long()
            see[:, ctx[b]:] = torch.stack([(m[:, j // 32] // 2 ** (j % 32)) % 2 == 1 if j % 32 < 31 else m[:, j // 32] < 0
                                           for j in range(n[b])], dim=1)
        for gh in range(case["n_kvh"]):
            rows = slots * case["n_kvh"] + gh
            K, V = (_exact_values(c[rows], e[rows], case["bits"]) for c, e in s["pools"])
            for h in range(gh * rep, (gh + 1) * rep):
                x = s["q"][first: first + n[b], h].double() @ K.T * s["scale"]
                x = torch.where(see, x, torch.full_like(x, -math.inf))
                l[:, h] = torch.logsumexp(x, dim=-1)
                o[:, h] = torch.exp(x - l[:, h: h + 1]) @ V
        outs.append(o)
        lses.append(l)
        first += n[b]
    return (torch.cat(outs), torch.cat(lses)) if case["lse"] else torch.cat(outs)
