"""Cases for the low-bit serving operators beside the QK-Norm projection: one
attention block's path with 8-bit weights and activations and a 4-bit cache.

    quant    qknorm_quant_rows     rows to 8-bit integers, one scale a row
    proj     qknorm_qkv_proj_quant     the QKV projection on 8-bit integers, QK-Norm in its epilogue
    cache    qknorm_kv_append/_gather  K and V of fused rows into a paged 4-bit cache, and out of it
    attn     qknorm_kv_attention     attention of fused rows' Q over that cache

``own`` false: elementary torch operations; true: the library's calls.

The cache: uint8 [pages, hkv, 64*D + 256].  One page of one head holds 64
tokens: K codes (token t, byte j: dims 2j in the low and 2j+1 in the high four
bits) at t*D/2 + j; V codes (dims 2j, 2j+1 of token t) at 32*D + 64*j + t; K
scales, bf16, at 64*D + 2*t; V scales at 64*D + 128 + 2*t.  A code is a sign
bit and an index into 0, .5, 1, 1.5, 2, 3, 4, 6 (four-bit floats: one sign, two
exponent and one fraction bits); a scale is amax / 6 rounded to bf16.
"""
import math
import random

import torch

own = False

LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # one decode step's hidden rows of an 8-sequence batch
        {"name": "quant_decode", "op": "quant", "T": 8, "n": 4096, "pad": 0, "dtype": "bf16"},
        # a long prompt's hidden rows (also: a weight, quantised once per output channel)
        {"name": "quant_prefill", "op": "quant", "T": 8192, "n": 4096, "pad": 0, "dtype": "bf16"},
        # one token through a Qwen3-8B layer's QKV projection: the weight is the traffic
        {"name": "proj_decode", "op": "proj", "T": 1, "hidden": 4096, "hq": 32, "hkv": 8, "D": 128, "plain": False,
         "pad": 0, "dtype": "bf16"},
        # a long prompt through the same layer: the product is the work
        {"name": "proj_prefill", "op": "proj", "T": 8192, "hidden": 4096, "hq": 32, "hkv": 8, "D": 128, "plain": False,
         "pad": 0, "dtype": "bf16"},
        # a ragged chunk of tokens, small heads, fp16, rows with a pitch, no norm
        {"name": "proj_ragged", "op": "proj", "T": 333, "hidden": 2048, "hq": 21, "hkv": 3, "D": 64, "plain": True,
         "pad": 64, "dtype": "f16"},
        # one decode step's K and V of 64 sequences, each into its own page
        {"name": "cache_decode", "op": "cache", "T": 64, "hq": 32, "hkv": 8, "D": 128, "run": 1, "skip": 5, "pad": 0,
         "dtype": "bf16"},
        # prompts' K and V, runs of 1000 consecutive slots, some padded rows
        {"name": "cache_prefill", "op": "cache", "T": 8192, "hq": 32, "hkv": 8, "D": 128, "run": 1000, "skip": 0,
         "pad": 0, "dtype": "bf16"},
        # one sequence of a chat, one new token: latency counts
        {"name": "attn_one", "op": "attn", "B": 1, "len": 1000, "ragged": 0, "new": 1, "mix": 1, "hq": 32, "hkv": 8,
         "D": 128, "window": 0, "dtype": "bf16"},
        # a serving batch of ragged lengths, one new token each
        {"name": "attn_batch", "op": "attn", "B": 64, "len": 8192, "ragged": 1, "new": 1, "mix": 2, "hq": 32, "hkv": 8,
         "D": 128, "window": 0, "dtype": "bf16"},
        # four long documents: the work has to be split along the cache
        {"name": "attn_long", "op": "attn", "B": 4, "len": 131071, "ragged": 0, "new": 1, "mix": 3, "hq": 32, "hkv": 8,
         "D": 128, "window": 0, "dtype": "bf16"},
        # chunks of four prompts' tokens over what their caches hold already
        {"name": "attn_chunk", "op": "attn", "B": 4, "len": 5000, "ragged": 1, "new": 512, "mix": 4, "hq": 32, "hkv": 8,
         "D": 128, "window": 0, "dtype": "bf16"},
        # drafts of a few tokens to verify, seven heads a group, a sliding window, some sequences without a token
        {"name": "attn_window", "op": "attn", "B": 33, "len": 3000, "ragged": 2, "new": 5, "mix": 5, "hq": 14, "hkv": 2,
         "D": 64, "window": 1000, "dtype": "f16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("quant", "proj", "cache", "attn"))
    dtype = rng.choice(("bf16", "bf16", "f16"))
    if op == "quant":
        return {"op": op, "T": _log(rng, 1, 8192), "n": 16 * _log(rng, 4, 256), "pad": 16 * rng.choice((0, 0, 1, 5)),
                "dtype": dtype}
    D = rng.choice((64, 128, 128, 256))
    hkv = rng.randint(1, 8)
    group = rng.randint(1, 8)
    if op == "proj":
        hidden = 64 * _log(rng, 4, 64)
        N = (group + 2) * hkv * D
        T = _log(rng, 1, max(1, min(8192, 8192 * 4096 * 6144 // (hidden * max(N, 6144)))))
        return {"op": op, "T": T, "hidden": hidden, "hq": group * hkv, "hkv": hkv, "D": D, "plain": rng.random() < 0.25,
                "pad": 16 * rng.choice((0, 0, 1, 5)), "dtype": dtype}
    if op == "cache":
        return {"op": op, "T": _log(rng, 1, 8192 * 128 // D), "hq": group * hkv, "hkv": hkv, "D": D,
                "run": rng.choice((1, 1, 7, 64, 1000)), "skip": rng.choice((0, 3, 50)), "pad": 16 * rng.choice((0, 0, 1)),
                "dtype": dtype}
    new = rng.choice((1, 1, 1, rng.randint(2, 16), _log(rng, 17, 512)))
    most = 4 * 131072 * 128 // D if new == 1 else 16384 * 128 // D // max(1, new // 128)   # tokens in all caches
    length = _log(rng, 1, 131072 * 128 // D if new == 1 else 8192)
    B = _log(rng, 1, max(1, min(128, most // length)))
    return {"op": op, "B": B, "len": length, "ragged": rng.choice((0, 1, 2)), "new": new, "mix": rng.randint(0, 10 ** 6),
            "hq": group * hkv, "hkv": hkv, "D": D, "window": rng.choice((0, 0, 0, _log(rng, 1, 4096))), "dtype": dtype}


def _lengths(c):
    """Tokens in each sequence's cache and new tokens of each (their last ones)."""
    r = random.Random(c["mix"])
    lens, new = [], []
    for b in range(c["B"]):
        lens.append(c["len"] if c["ragged"] == 0 or b == 0 else _log(r, 1, c["len"]))
        new.append(c["new"] if c["ragged"] < 2 else r.randint(0, c["new"]))
        if c["ragged"] == 2 and b % 8 == 5:
            lens[b] = 0
    return lens, new


def _visible(c):
    """Keys that each new token of each sequence sees, summed."""
    total = 0
    for n, m in zip(*_lengths(c)):
        for i in range(m):
            pos = n - m + i
            total += max(0, min(pos + 1, c["window"] or pos + 1))
    return total


def work(c):
    if c["op"] == "quant":
        return {"bytes": c["T"] * (3 * c["n"] + 4), "flops": 3 * c["T"] * c["n"]}
    if c["op"] == "proj":
        N = (c["hq"] + 2 * c["hkv"]) * c["D"]
        return {"bytes": (c["T"] + N) * (c["hidden"] + 4) + 2 * c["T"] * N, "flops": 2 * c["T"] * N * c["hidden"]}
    if c["op"] == "cache":
        # K and V read, their codes and scales written and read, the values written
        return {"bytes": c["T"] * c["hkv"] * (4 * c["D"] + 2 * (c["D"] + 4) + 4 * c["D"]), "flops": 8 * c["T"] * c["hkv"] * c["D"]}
    held = 0
    for n, m in zip(*_lengths(c)):
        seen = min(n, c["window"] + m - 1) if c["window"] else n
        held += seen if m else 0
    rows = sum(_lengths(c)[1])
    return {"bytes": held * c["hkv"] * (c["D"] + 4) + 4 * rows * c["hq"] * c["D"], "flops": 4 * c["D"] * c["hq"] * _visible(c)}


# ------------------------------------------------------------------ inputs --

def _normed(g, shape, D, dtype):
    """Heads as QK-Norm leaves them: unit mean square, times weights in [0.5, 1.5)."""
    x = torch.randn(*shape, D, generator=g, device="cuda")
    w = torch.rand(D, generator=g, device="cuda") + 0.5
    return (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w).to(dtype)


def _values(g, shape, D, dtype):
    """V as a projection leaves it: tokens of unlike sizes."""
    x = torch.randn(*shape, D, generator=g, device="cuda")
    return (x * (torch.rand(*shape, 1, generator=g, device="cuda") * 2 + 0.1)).to(dtype)


def _pitched(rows, pad):
    """The same rows with `pad` more elements between them."""
    if not pad:
        return rows
    wide = torch.zeros(rows.shape[0], rows.shape[1] + pad, dtype=rows.dtype, device=rows.device)
    wide[:, :rows.shape[1]] = rows
    return wide[:, :rows.shape[1]]


def _empty_cache(pages, hkv, D):
    return torch.zeros(pages, hkv, 64 * D + 256, dtype=torch.uint8, device="cuda")


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["op"] == "quant":
        x = torch.randn(c["T"], c["n"], generator=g, device="cuda")
        x[:, ::97] *= 20                       # a few channels stand out, as hidden states' do
        s["x"] = _pitched((x * (torch.rand(c["T"], 1, generator=g, device="cuda") * 9.9 + 0.1)).to(DT[c["dtype"]]), c["pad"])
        s["q"] = torch.empty(c["T"], c["n"], dtype=torch.int8, device="cuda")
        s["scale"] = torch.empty(c["T"], dtype=torch.float32, device="cuda")
        return s
    dt, D, hq, hkv = DT[c["dtype"]], c["D"], c["hq"], c["hkv"]
    N = (hq + 2 * hkv) * D
    if c["op"] == "proj":
        T, K = c["T"], c["hidden"]
        for name, rows in (("x", T), ("w", N)):
            v = torch.randn(rows, K, generator=g, device="cuda")
            top = v.abs().amax(1, keepdim=True)
            s[name] = _pitched(torch.round(v * (127 / top)).to(torch.int8), c["pad"])
            s[name + "_scale"] = (top[:, 0] / 127 * (1 if name == "x" else K ** -0.5)).contiguous()
        s["gq"] = (torch.rand(D, generator=g, device="cuda") + 0.5).to(dt)
        s["gk"] = (torch.rand(D, generator=g, device="cuda") + 0.5).to(dt)
        s["out"] = _pitched(torch.empty(T, N, dtype=dt, device="cuda"), c["pad"])
        s["space"] = None
        if own:
            import qk_norm_amd as q
            s["space"] = torch.empty(q.qknorm_qkv_proj_quant_workspace_bytes(T, hq, hkv, D), dtype=torch.uint8, device="cuda")
        return s
    if c["op"] == "cache":
        T = c["T"]
        rows = torch.zeros(T, N, dtype=dt, device="cuda")
        rows[:, hq * D:(hq + hkv) * D] = _normed(g, (T, hkv), D, dt).view(T, -1)
        rows[:, (hq + hkv) * D:] = _values(g, (T, hkv), D, dt).view(T, -1)
        s["qkv"] = _pitched(rows, c["pad"])
        runs = (T + c["run"] - 1) // c["run"]
        each = (c["run"] + 63) // 64           # pages of a run, which starts inside its first
        pages = runs * (each + 1) + 1
        at = torch.arange(T, device="cuda")
        first = torch.randint(0, 64, (runs,), generator=g, device="cuda")
        order = torch.randperm(runs, generator=g, device="cuda")
        slots = order[at // c["run"]] * (each + 1) * 64 + first[at // c["run"]] + at % c["run"]
        if c["skip"]:
            slots = torch.where(at % c["skip"] == c["skip"] - 1, -1, slots)     # padded rows
        s["slots"] = slots
        s["cache"] = _empty_cache(pages, hkv, D)
        s["k"] = torch.zeros(T, hkv, D, dtype=dt, device="cuda")
        s["v"] = torch.zeros(T, hkv, D, dtype=dt, device="cuda")
        return s
    lens, new = _lengths(c)
    B, T = c["B"], sum(new)
    width = max(1, max((n + 63) // 64 for n in lens))
    pages = sum((n + 63) // 64 for n in lens) + 1
    cache = _empty_cache(pages, hkv, D)
    step = max(1, (1 << 26) // (64 * hkv * D))
    for p in range(0, pages, step):             # the pool, some pages at a time
        m = min(step, pages - p)
        k = _normed(g, (m, hkv, 64), D, dt)
        v = _values(g, (m, hkv, 64), D, dt)
        cache[p:p + m] = _pack(*_codes(k), *_codes(v))
    table = torch.full((B, width), -1, dtype=torch.int32)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    at = 0
    for b, n in enumerate(lens):
        m = (n + 63) // 64
        table[b, :m] = order[at:at + m]
        at += m
    starts = [0]
    for m in new:
        starts.append(starts[-1] + m)
    rows = torch.zeros(max(T, 1), N, dtype=dt, device="cuda")[:T]
    rows[:, :hq * D] = _normed(g, (T, hq), D, dt).view(T, -1)
    s.update(qkv=rows, cache=cache, table=table.cuda(), lens=torch.tensor(lens, dtype=torch.int32).cuda(),
             starts=torch.tensor(starts, dtype=torch.int32).cuda(), most=max(new), width=width,
             one=all(m == 1 for m in new), out=torch.zeros(T, hq, D, dtype=dt, device="cuda"),
             lse=torch.zeros(T, hq, dtype=torch.float32, device="cuda"), space=None)
    if own:
        import qk_norm_amd as q
        s["space"] = torch.empty(q.qknorm_kv_attention_workspace_bytes(T, B, width, hq, hkv, D), dtype=torch.uint8, device="cuda")
    return s


# -------------------------------------------------------------- plain forms --

def _codes(x):
    """Codes and bf16 scales of the last axis: four-bit floats to nearest, ties to even."""
    x = x.float()
    top = x.abs().amax(-1)
    s = (top / 6).to(torch.bfloat16)
    y = x.abs() / s.float().clamp_min(2.0 ** -120)[..., None]
    code = ((y > 0.25).int() + (y >= 0.75).int() + (y > 1.25).int() + (y >= 1.75).int() + (y > 2.5).int()
            + (y >= 3.5).int() + (y > 5).int())
    return (code + 8 * (x < 0).int()).to(torch.uint8), s


def _bytes(scale):
    return scale.contiguous().view(torch.uint8).flatten(-2) if scale.dim() > 3 else scale.contiguous().view(torch.uint8)


def _pack(kc, ks, vc, vs):
    """[m, hkv, 64, D] codes and [m, hkv, 64] scales as pages."""
    k = kc[..., 0::2] | (kc[..., 1::2] << 4)
    v = (vc[..., 0::2] | (vc[..., 1::2] << 4)).transpose(-1, -2)
    return torch.cat([k.flatten(-2), v.flatten(-2), _bytes(ks), _bytes(vs)], dim=-1)


def _split(b):
    return torch.stack((b & 15, b >> 4), dim=-1).flatten(-2)


def _levels(code):
    table = torch.tensor(LEVELS + tuple(-x for x in LEVELS), device=code.device)
    return table[code.int()]


def _unpack(pages, D):
    """Pages [..., hkv, 64*D + 256] as K and V values, float32 [..., hkv, 64, D]."""
    lead = pages.shape[:-1]
    k = _levels(_split(pages[..., :32 * D].reshape(*lead, 64, D // 2)))
    v = _levels(_split(pages[..., 32 * D:64 * D].reshape(*lead, D // 2, 64).transpose(-1, -2)))
    ks = pages[..., 64 * D:64 * D + 128].contiguous().view(torch.bfloat16).float()
    vs = pages[..., 64 * D + 128:].contiguous().view(torch.bfloat16).float()
    return k * ks[..., None], v * vs[..., None]


def _plain_quant(s):
    x = s["x"].double()                         # quotients next to a half are told apart
    top = x.abs().amax(1, keepdim=True)
    s["q"].copy_(torch.round(x * 127 / top))
    s["scale"].copy_(s["x"].float().abs().amax(1) / 127)
    return {"q": s["q"], "scale": s["scale"]}


def _plain_proj(s):
    c = s["case"]
    D, T, heads = c["D"], c["T"], c["hq"] + c["hkv"]
    # sums of up to hidden * 127 * 127 pass 2^24: kept whole in 64 bits
    y = (s["x"].double() @ s["w"].double().t()).float() * s["w_scale"] * s["x_scale"][:, None]
    if not c["plain"]:
        h = y[:, :heads * D].view(T, heads, D)
        gamma = torch.cat([s["gq"].float().expand(c["hq"], D), s["gk"].float().expand(c["hkv"], D)])
        h = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * gamma
        y = torch.cat([h.reshape(T, -1), y[:, heads * D:]], dim=1)
    s["out"].copy_(y)
    return s["out"]


def _plain_cache(s):
    c = s["case"]
    D, hq, hkv, T = c["D"], c["hq"], c["hkv"], c["T"]
    kv = s["qkv"][:, hq * D:].reshape(T, 2, hkv, D)
    code, scale = _codes(kv)
    byte = code[..., 0::2] | (code[..., 1::2] << 4)
    two = scale.view(torch.uint8).view(T, 2, hkv, 2)
    good = s["slots"] >= 0
    # rows without a slot go to the pool's last page, which nobody reads
    slots = torch.where(good, s["slots"], (s["cache"].shape[0] - 1) * 64)
    page, t = (slots // 64)[:, None, None], (slots % 64)[:, None, None]
    head = torch.arange(hkv, device="cuda")[None, :, None]
    j = torch.arange(D // 2, device="cuda")
    pair = torch.arange(2, device="cuda")
    places = [(page, head, t * (D // 2) + j), (page, head, 32 * D + 64 * j + t),
              (page, head, 64 * D + 2 * t + pair), (page, head, 64 * D + 128 + 2 * t + pair)]
    s["cache"][places[0]] = byte[:, 0]
    s["cache"][places[1]] = byte[:, 1]
    s["cache"][places[2]] = two[:, 0]
    s["cache"][places[3]] = two[:, 1]
    for name, codes, scales in (("k", 0, 2), ("v", 1, 3)):
        value = _levels(_split(s["cache"][places[codes]]))
        value = value * s["cache"][places[scales]].contiguous().view(torch.bfloat16).float()
        s[name].copy_(torch.where(good[:, None, None], value, s[name].float()))
    return {"k": s["k"], "v": s["v"]}


def _plain_attn(s):
    c = s["case"]
    D, hq, hkv, B, T = c["D"], c["hq"], c["hkv"], c["B"], s["qkv"].shape[0]
    if T == 0:
        return {"out": s["out"], "lse": s["lse"]}
    m, L, group = s["most"], s["width"] * 64, hq // hkv
    k, v = _unpack(s["cache"][s["table"].clamp_min(0).long()], D)       # [B, width, hkv, 64, D]
    k = k.transpose(1, 2).reshape(B, hkv, L, D)
    v = v.transpose(1, 2).reshape(B, hkv, L, D)
    i = torch.arange(m, device="cuda")
    start, new = s["starts"][:-1].long(), s["starts"].diff().long()
    row = torch.where(i < new[:, None], start[:, None] + i, T)          # [B, m]; T: no row
    q = torch.cat([s["qkv"][:, :hq * D].float(), torch.zeros(1, hq * D, device="cuda")])[row]
    q = q.view(B, m, hkv, group, D).permute(0, 2, 1, 3, 4).reshape(B, hkv, m * group, D)
    score = q @ k.transpose(-1, -2) * D ** -0.5
    pos = (s["lens"].long() - new)[:, None] + i                         # [B, m]
    at = torch.arange(L, device="cuda")
    see = (at <= pos[..., None]) & (at < s["lens"][:, None, None])
    if c["window"]:
        see &= at > pos[..., None] - c["window"]
    see = see[:, None, :, None].expand(B, 1, m, group, L).reshape(B, 1, m * group, L)
    score = score.masked_fill(~see, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top.masked_fill(top == -math.inf, 0.0))
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / total.masked_fill(total == 0, 1.0)
    lse = (top + torch.log(total))[..., 0]
    back = lambda x: x.view(B, hkv, m, group, -1).permute(0, 2, 1, 3, 4).reshape(B * m, hq, -1)  # noqa: E731
    out = torch.zeros(T + 1, hq, D, device="cuda")
    out[row.flatten()] = back(o)
    far = torch.zeros(T + 1, hq, 1, device="cuda")
    far[row.flatten()] = back(lse)
    s["out"].copy_(out[:T])
    s["lse"].copy_(far[:T, :, 0])
    return {"out": s["out"], "lse": s["lse"]}


# --------------------------------------------------------------------- run --

def _own(s):
    import qk_norm_amd as q
    c = s["case"]
    if c["op"] == "quant":
        q.qknorm_quant_rows(s["x"], s["q"], s["scale"])
        return {"q": s["q"], "scale": s["scale"]}
    if c["op"] == "proj":
        q.qknorm_qkv_proj_quant(s["x"], s["x_scale"], s["w"], s["w_scale"], s["out"], c["hq"], c["hkv"], c["D"], s["gq"],
                               s["gk"], EPS, plain=c["plain"], workspace=s["space"])
        return s["out"]
    if c["op"] == "cache":
        q.qknorm_kv_append(s["qkv"], c["hq"], c["hkv"], c["D"], s["cache"], s["slots"])
        q.qknorm_kv_gather(s["cache"], s["slots"], s["k"], s["v"], c["hkv"], c["D"])
        return {"k": s["k"], "v": s["v"]}
    q.qknorm_kv_attention(s["qkv"], s["cache"], s["table"], s["lens"], s["out"], c["hq"], c["hkv"], c["D"],
                           q_starts=None if s["one"] else s["starts"], window=c["window"], lse=s["lse"],
                           workspace=s["space"])
    return {"out": s["out"], "lse": s["lse"]}


def run(s):
    if own:
        return _own(s)
    return {"quant": _plain_quant, "proj": _plain_proj, "cache": _plain_cache, "attn": _plain_attn}[s["case"]["op"]](s)


# ------------------------------------------------------------------- exact --

def _nearest(x, s):
    """x in units of s to the nearest of the 15 values (halfway: the even code), times s; 64 bits."""
    u = x / torch.where(s > 0, s, 1.0)[..., None]
    lv = torch.tensor(LEVELS, dtype=torch.float64, device=x.device)
    a = u.abs().clamp(max=6.0)
    hi = torch.searchsorted(lv, a).clamp(1, 7)                           # lv[hi-1] < a <= lv[hi], or a = 0
    below, above = a - lv[hi - 1], lv[hi] - a
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return torch.where(up, lv[hi], lv[hi - 1]) * torch.sign(u) * s[..., None]


def _page_values(page, D):
    """One page [hkv, 64*D + 256] as K and V, float64 [hkv, 64, D]."""
    h = page.shape[0]
    lv = torch.tensor([x * y for y in (1, -1) for x in LEVELS], dtype=torch.float64, device=page.device)
    k, v = torch.empty(2, h, 64, D, dtype=torch.float64, device=page.device)
    kb, vb = page[:, :32 * D].view(h, 64, D // 2).long(), page[:, 32 * D:64 * D].view(h, D // 2, 64).long()
    sc = page[:, 64 * D:].contiguous().view(torch.bfloat16).double()
    k[..., 0::2], k[..., 1::2] = lv[kb % 16], lv[kb // 16]
    v[..., 0::2], v[..., 1::2] = lv[vb % 16].mT, lv[vb // 16].mT
    return k * sc[:, :64, None], v * sc[:, 64:, None]


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "quant":
        x = s["x"].double()
        top = torch.linalg.vector_norm(x, ord=math.inf, dim=1)
        return {"q": torch.round(127 * x / top[:, None]).to(torch.int8), "scale": top / 127}
    D, hq, hkv = c["D"], c["hq"], c["hkv"]
    if c["op"] == "proj":
        y = torch.mm(s["x"].double() * s["x_scale"].double()[:, None], (s["w"].double() * s["w_scale"].double()[:, None]).t())
        if not c["plain"]:
            for lo, n, gamma in ((0, hq, s["gq"]), (hq * D, hkv, s["gk"])):
                part = y[:, lo:lo + n * D].unflatten(1, (n, D))
                rms = torch.sqrt(part.square().sum(-1, keepdim=True) / D + EPS)
                y[:, lo:lo + n * D] = (gamma.double() * part / rms).flatten(1)
        return y
    if c["op"] == "cache":
        got = {}
        for name, lo in (("k", hq), ("v", hq + hkv)):
            x = s["qkv"][:, lo * D:(lo + hkv) * D].double().unflatten(1, (hkv, D))
            scale = (torch.linalg.vector_norm(x, ord=math.inf, dim=-1) / 6).to(torch.bfloat16).double()
            got[name] = _nearest(x, scale) * (s["slots"] >= 0)[:, None, None]
        return got
    lens, new = _lengths(c)
    if _visible(c) * hq * D > 4e11:
        return None
    T, group = s["qkv"].shape[0], hq // hkv
    out = torch.zeros(T, hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64, device="cuda")
    t = 0
    for b in range(c["B"]):
        n, m = lens[b], new[b]
        if n and m:
            ids = s["table"][b, :(n + 63) // 64].tolist()
            lo = max(0, (n - m - c["window"] + 1) // 64) if c["window"] else 0     # pages before it are out of all windows
            parts = [_page_values(s["cache"][p], D) for p in ids[lo:]]
            k, v = (torch.cat([part[a] for part in parts], dim=1)[:, :n - 64 * lo] for a in (0, 1))
            at = torch.arange(64 * lo, n, device="cuda")
            for h in range(hq):
                q = s["qkv"][t:t + m, h * D:(h + 1) * D].double()
                x = torch.mm(q, k[h // group].t()) / math.sqrt(D)
                pos = torch.arange(n - m, n, device="cuda")[:, None]
                hidden = at > pos
                if c["window"]:
                    hidden |= at <= pos - c["window"]
                x[hidden] = -math.inf
                lse[t:t + m, h] = torch.logsumexp(x, dim=1)
                ok = lse[t:t + m, h] > -math.inf
                w = torch.where(ok[:, None], torch.exp(x - torch.where(ok, lse[t:t + m, h], 0.0)[:, None]), 0.0)
                out[t:t + m, h] = torch.mm(w, v[h // group])
        t += m
    return {"out": out, "lse": lse}
