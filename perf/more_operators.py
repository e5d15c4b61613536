"""A decoder layer's cache held in 4 bits, and the norms of queries and keys before it, as cases that can be timed:

  norm     RMS norms of q and k for each head with their rotary positions, in one pass
  append   the same, with k and v written into a paged cache of 4-bit codes; then what was written, read back
  read     tokens of such a cache as 16-bit keys and values
  attend   attention of new tokens over such a cache, with a window and first tokens that stay visible

A token and head of the cache holds its D elements as codes 0 .. 15, two a byte, the lower half first, and for each G of
them a scale s and a zero-point z: x = (code - z) s.  s is (hi - lo) / 15 of the group's range, 0 among it, to 7 bits.

``own = False``: elementary torch operations on the same inputs, in fp32; what the codes come from in fp64, since a value
next to a border between two codes would take either.  ``own = True``: the calls of this repository's package.
"""
import math

import torch

own = False

DEVICE = "cuda"
TABLE = 131072          # positions the rotary table covers
EPS = 1e-6
TOP = 57344.0           # what a cache of 4 bits saturates at


def listed():
    return [
        # one new token of one user, for a cache of any kind
        dict(name="norm_token", op="norm", T=1, start=4095, Hq=32, Hkv=8, D=128, rot=128, pairs=False, norm=True, dtype="float16"),
        # a long prompt, far into its context, 70B class
        dict(name="norm_prompt", op="norm", T=8192, start=100000, Hq=64, Hkv=8, D=128, rot=128, pairs=False, norm=True, dtype="bfloat16"),
        # one new token of one user
        dict(name="append4_token", op="append", T=1, start=4095, pad=0, Hq=32, Hkv=8, D=128, G=64, rot=128, pairs=False, norm=True, page=16, dtype="float16"),
        # a batch of new tokens, some of them padding; partial rotation of neighbouring elements, fine groups
        dict(name="append4_ragged", op="append", T=777, start=1000, pad=23, Hq=32, Hkv=8, D=128, G=32, rot=64, pairs=True, norm=False, page=16, dtype="float16"),
        # a long prompt, far into its context, one scale a head and token
        dict(name="append4_prompt", op="append", T=8192, start=100000, pad=0, Hq=64, Hkv=8, D=128, G=128, rot=128, pairs=False, norm=True, page=64, dtype="bfloat16"),
        # a short context taken out of the cache, with places that hold nothing
        dict(name="read_ragged", op="read", T=1001, pad=19, Hkv=4, D=96, G=32, page=16, dtype="bfloat16"),
        # a long context taken out of the cache
        dict(name="read_long", op="read", T=131072, pad=0, Hkv=8, D=128, G=64, page=64, dtype="float16"),
        # one user's next token in a long conversation: a window of 512 and the first 4 tokens
        dict(name="attend4_token", op="attend", B=1, n=1, L=5000, spread=0.0, idle=0, Hq=32, Hkv=8, D=128, G=128, page=16, window=512, sinks=4, dtype="float16", lse=False),
        # a decode batch of users with contexts of all lengths, four idle places
        dict(name="attend4_batch", op="attend", B=64, n=1, L=8192, spread=0.95, idle=4, Hq=32, Hkv=8, D=128, G=64, page=16, window=0, sinks=0, dtype="float16", lse=True),
        # very long contexts
        dict(name="attend4_long", op="attend", B=4, n=1, L=131071, spread=0.3, idle=0, Hq=64, Hkv=8, D=128, G=128, page=64, window=0, sinks=0, dtype="float16", lse=False),
        # chunks of prompts whose beginnings are in the cache, each row with its window and the first tokens
        dict(name="attend4_chunk", op="attend", B=3, n=600, L=32768, spread=0.5, idle=0, Hq=32, Hkv=8, D=128, G=64, page=16, window=4096, sinks=100, dtype="bfloat16", lse=False),
        # whole prompts, one key head for four query heads, fine groups
        dict(name="attend4_prompt", op="attend", B=2, n=4096, L=4096, spread=0.0, idle=0, Hq=32, Hkv=8, D=128, G=32, page=64, window=0, sinks=0, dtype="float16", lse=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "append", "append", "read", "attend", "attend", "attend"))
    Hkv, g = rng.choice((1, 2, 4, 5, 8, 16)), rng.choice((1, 2, 3, 4, 8))
    D = rng.choice((64, 96, 128, 128, 128, 192, 256))
    G = rng.choice([x for x in (32, 64, 128) if D % x == 0])
    page, dtype = rng.choice((1, 16, 32, 64, 100, 256)), rng.choice(("float16", "bfloat16"))
    if op == "read":
        T = _log(rng, 1, 65536)
        return dict(op=op, T=T, pad=rng.randint(0, T // 4), Hkv=Hkv, D=D, G=G, page=page, dtype=dtype)
    if op in ("norm", "append"):
        T, Hq = _log(rng, 1, 4096), Hkv * g
        case = dict(op=op, T=T, start=rng.randint(0, TABLE - 4096), Hq=Hq, Hkv=Hkv, D=D, rot=rng.choice((D, D, D // 32 * 16)), pairs=rng.random() < 0.4,
                    norm=op == "norm" or rng.random() < 0.6, dtype=dtype)
        return case if op == "norm" else dict(case, pad=rng.randint(0, T // 4), G=G, page=page)
    while True:
        n = 1 if rng.random() < 0.5 else _log(rng, 2, 4096)
        B, L = _log(rng, 1, 64), _log(rng, 1, 131072)
        if n <= L and B * n * L * Hkv * g <= 1_800_000_000 and B * n * L * Hkv * g * D <= 128 * 2 * 32 * 4096 * 4096 \
                and B * L * Hkv * D <= 4 * 131072 * 8 * 128:
            break
    window = rng.choice((0, 0, _log(rng, 16, 4096)))
    return dict(op=op, B=B, n=n, L=L, spread=round(rng.uniform(0, 0.99), 3), idle=rng.choice((0, 0, 1)) if B > 1 else 0, Hq=Hkv * g, Hkv=Hkv, D=D, G=G,
                page=page, window=window, sinks=rng.choice((0, 1, 4, _log(rng, 5, 300))) if window else 0, dtype=dtype, lse=rng.random() < 0.5)


def _lengths(c):
    """(new tokens, context length) of each sequence of an attend case; the last `idle` have one query row and no context."""
    got = []
    for i in range(c["B"]):
        if i >= c["B"] - c["idle"]:
            got.append((1, 0))
            continue
        a, b = (i * 0.6180339887) % 1.0, (i * 0.7548776662) % 1.0
        L = max(1, round(c["L"] * (1 - c["spread"] * a)))
        got.append((min(L, max(1, round(c["n"] * (1 - c["spread"] * b)))), L))
    return got


# ---------------------------------------------------------------------------------------------
# inputs

def _filled(shape, G, gen):
    """Codes, scales and zero-points of normal values, a part of the pages at a time."""
    pages, Hkv, page, D = shape
    codes = torch.empty(pages, Hkv, page, D // 2, device=DEVICE, dtype=torch.uint8)
    scale = torch.empty(pages, Hkv, page, D // G, 2, device=DEVICE, dtype=torch.float16)
    step = max(1, 2 ** 26 // (Hkv * page * D))
    for at in range(0, pages, step):
        x = torch.randn(min(step, pages - at), Hkv, page, D, generator=gen, device=DEVICE)
        codes[at:at + step], scale[at:at + step] = _encode(x, G)
    return codes, scale


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEVICE)

    s = dict(case=dict(c))
    dt, Hkv, D = getattr(torch, c["dtype"]), c["Hkv"], c["D"]
    if c["op"] in ("norm", "append"):
        T, Hq, rot = c["T"], c["Hq"], c["rot"]
        # q, k and v are columns of one fused projection
        qkv = normal(T, (Hq + 2 * Hkv) * D).to(dt)
        s["q"] = qkv[:, :Hq * D].unflatten(1, (Hq, D))
        s["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
        s["v"] = qkv[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
        s["q_weight"], s["k_weight"] = ((1 + 0.2 * normal(D)).to(dt) if c["norm"] else None for _ in range(2))
        s["positions"] = torch.arange(T, device=DEVICE, dtype=torch.int32) + c["start"]
        angle = torch.arange(TABLE, device=DEVICE, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(rot // 2, device=DEVICE, dtype=torch.float64) * 2 / rot)
        s["rope"] = torch.cat((angle.cos(), angle.sin()), 1).float()
        s["out"], s["k_out"] = torch.empty(T, Hq, D, device=DEVICE, dtype=dt), torch.empty(T, Hkv, D, device=DEVICE, dtype=dt)
        if c["op"] == "norm":
            return s
    if c["op"] in ("append", "read"):
        T, page = c["T"], c["page"]
        pages = (T + page - 1) // page + 3
        order = torch.randperm(pages, generator=gen, device=DEVICE)
        at = torch.arange(T, device=DEVICE) + c.get("start", 5) % page % 7
        s["slots"] = order[at // page % pages] * page + at % page
        if c["pad"]:
            s["slots"][T - c["pad"]:] = -1
        s["cache"] = _filled((pages, Hkv, page, D), c["G"], gen) + _filled((pages, Hkv, page, D), c["G"], gen)
        s["cache"] = tuple(s["cache"][i] for i in (0, 2, 1, 3))           # codes of k and v, then their scales
        return s
    lens, Hq, page = _lengths(c), c["Hq"], c["page"]
    n, L = [a for a, _ in lens], [b for _, b in lens]
    T, width = sum(n), max(1, -(-max(L) // page))
    s["q"] = normal(T, Hq, D).to(dt)
    cu = [0]
    for a in n:
        cu.append(cu[-1] + a)
    s["cu_q"] = torch.tensor(cu, dtype=torch.int32, device=DEVICE)
    s["kv_lens"] = torch.tensor(L, dtype=torch.int32, device=DEVICE)
    s["max_q"], s["max_kv"] = max(n), max(1, max(L))
    need = torch.tensor([-(-b // page) for b in L], device=DEVICE)
    pages = int(need.sum()) + 3
    order = torch.randperm(pages, generator=gen, device=DEVICE).to(torch.int32)
    col = torch.arange(width, device=DEVICE)
    used = col < need[:, None]
    s["page_table"] = torch.where(used, order[(need.cumsum(0) - need)[:, None] + torch.where(used, col, 0)], 0).to(torch.int32).contiguous()
    k, ks = _filled((pages, Hkv, page, D), c["G"], gen)
    v, vs = _filled((pages, Hkv, page, D), c["G"], gen)
    s["cache"] = (k, v, ks, vs)
    s["scale"] = D ** -0.5
    s["out"] = torch.empty(T, Hq, D, device=DEVICE, dtype=dt)
    s["lse"] = torch.empty(T, Hq, device=DEVICE, dtype=torch.float32) if c["lse"] else None
    return s


# ---------------------------------------------------------------------------------------------
# one pass

def run(state):
    op = state["case"]["op"]
    if op == "norm":
        return _norm_own(state) if own else _norm(state)
    if op == "append":
        return _append_own(state) if own else _append(state)
    if op == "read":
        return _read_own(state) if own else _read(state)
    return _attend_own(state) if own else _attend(state)


def _norm_own(s):
    import bit_weight_quantized_qmm_amd as qmm
    return qmm.qk_norm(s["q"], s["k"], s["q_weight"], s["k_weight"], EPS, s["positions"], s["rope"], pairs=s["case"]["pairs"], q_out=s["out"], k_out=s["k_out"])


def _append_own(s):
    import bit_weight_quantized_qmm_amd as qmm
    q = qmm.kv4_append(s["q"], s["k"], s["v"], s["cache"], s["slots"], s["positions"], s["rope"], pairs=s["case"]["pairs"], q_norm=s["q_weight"], k_norm=s["k_weight"],
                       eps=EPS, out=s["out"])
    return (q,) + tuple(qmm.kv4_read(s["cache"], s["slots"], s["q"].dtype))


def _read_own(s):
    import bit_weight_quantized_qmm_amd as qmm
    return tuple(qmm.kv4_read(s["cache"], s["slots"], getattr(torch, s["case"]["dtype"])))


def _attend_own(s):
    import bit_weight_quantized_qmm_amd as qmm
    out = qmm.kv4_attention(s["q"], s["cache"], s["page_table"], s["cu_q"], s["kv_lens"], s["max_q"], s["max_kv"], scale=s["scale"],
                            window=s["case"]["window"], sinks=s["case"]["sinks"], out=s["out"], lse=s["lse"])
    return out if s["lse"] is None else (out, s["lse"])


def _turned(x, weight, line, c):
    """Norm and rotation in x's type; `line`: each token's cosines and sines."""
    rot = c["rot"]
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.to(x.dtype)
    cos, sin = line[..., :rot // 2].to(x.dtype), line[..., rot // 2:].to(x.dtype)
    if c["pairs"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _norm(s):
    line = s["rope"][s["positions"].long()][:, None, :]
    s["out"].copy_(_turned(s["q"].float(), s["q_weight"], line, s["case"]))
    s["k_out"].copy_(_turned(s["k"].float(), s["k_weight"], line, s["case"]))
    return s["out"], s["k_out"]


def _encode(x, G):
    """[..., D] -> codes [..., D / 2] uint8, scales and zero-points [..., D / G, 2] fp16."""
    x = torch.clamp(x, -TOP, TOP).unflatten(-1, (-1, G))
    lo, hi = torch.clamp(x.amin(-1, keepdim=True), max=0), torch.clamp(x.amax(-1, keepdim=True), min=0)
    s = torch.clamp((hi - lo) / 15, min=2.0 ** -19)
    m, _ = torch.frexp(s)
    s = torch.clamp(torch.round(m * 128) / 128 * (s / m), min=2.0 ** -18)      # (s / m is a power of two)
    z = torch.clamp(torch.round(-lo / s), 0, 15)
    q = torch.clamp(torch.round(x / s) + z, 0, 15).flatten(-2).to(torch.uint8)
    return q[..., 0::2] | (q[..., 1::2] << 4), torch.cat((s, z), -1).half()


def _decode(codes, scale):
    """The inverse, in fp32."""
    x = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float().unflatten(-1, (scale.shape[-2], -1))
    scale = scale.float()
    return ((x - scale[..., 1:]) * scale[..., :1]).flatten(-2)


def _append(s):
    c = s["case"]
    line = s["rope"][s["positions"].long()][:, None, :]
    s["out"].copy_(_turned(s["q"].float(), s["q_weight"], line, c))
    k, v = _turned(s["k"].double(), s["k_weight"], line, c), s["v"].double()
    # padding stands at the end: its values go nowhere
    live = c["T"] - c["pad"]
    at, within = s["slots"][:live] // c["page"], s["slots"][:live] % c["page"]
    k_cache, v_cache, k_scale, v_scale = s["cache"]
    k_cache[at, :, within], k_scale[at, :, within] = _encode(k[:live], c["G"])
    v_cache[at, :, within], v_scale[at, :, within] = _encode(v[:live], c["G"])
    return (s["out"],) + _read(s)


def _read(s):
    c = s["case"]
    page, there = c["page"], (s["slots"] >= 0)[:, None, None]
    at = torch.clamp(s["slots"], min=0)
    k_cache, v_cache, k_scale, v_scale = s["cache"]
    return tuple(torch.where(there, _decode(codes[at // page, :, at % page], scale[at // page, :, at % page]), 0).to(getattr(torch, c["dtype"]))
                 for codes, scale in ((k_cache, k_scale), (v_cache, v_scale)))


def _attend(s):
    c = s["case"]
    Hkv, D, page, g = c["Hkv"], c["D"], c["page"], c["Hq"] // c["Hkv"]
    cu, lens = s["cu_q"].long(), s["kv_lens"].long()
    n, B = cu[1:] - cu[:-1], c["B"]
    i, j = torch.arange(s["max_q"], device=DEVICE), torch.arange(s["max_kv"], device=DEVICE)
    T = s["q"].shape[0]
    k_cache, v_cache, k_scale, v_scale = s["cache"]

    def dense(codes, scale):     # [B, Hkv, max_kv, D]
        at = s["page_table"].long()[:, j // page], j % page
        return _decode(codes[at[0], :, at[1]], scale[at[0], :, at[1]]).transpose(1, 2).contiguous()

    q = s["q"].float()[torch.clamp(cu[:-1, None] + i, max=T - 1)]
    q = q.unflatten(2, (Hkv, g)).permute(0, 2, 3, 1, 4).reshape(B, Hkv, g * i.numel(), D)
    pos = (lens - n)[:, None] + i
    seen = (j <= pos[..., None]) & (j < lens[:, None, None])
    if c["window"]:
        seen = seen & ((j > pos[..., None] - c["window"]) | (j < c["sinks"]))
    x = torch.matmul(q, dense(k_cache, k_scale).transpose(2, 3)).unflatten(2, (g, i.numel()))
    x = torch.where(seen[:, None, None], x * s["scale"], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.flatten(2, 3), dense(v_cache, v_scale)).unflatten(2, (g, i.numel()))
    o = torch.where(total > 0, o / total, 0.0)
    t = torch.arange(T, device=DEVICE)
    seq = torch.searchsorted(cu[1:], t, right=True)
    row = t - cu[seq]
    s["out"].copy_(o.flatten(1, 2)[seq, :, row])
    if s["lse"] is None:
        return s["out"]
    s["lse"].copy_((top + torch.log(total)).squeeze(-1).flatten(1, 2)[seq, :, row])
    return s["out"], s["lse"]


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    c = case
    Hkv, D = c["Hkv"], c["D"]
    if c["op"] == "norm":
        T, H = c["T"], c["Hq"] + Hkv
        return {"bytes": T * (4 * H * D + 4 * c["rot"] + 4) + 4 * D, "flops": T * H * (3 * c["rot"] + 4 * D)}
    cell = 2 * Hkv * (D // 2 + 4 * D // c["G"])          # a token's codes, scales and zero-points of k and v
    if c["op"] == "read":
        live = c["T"] - c["pad"]
        return {"bytes": c["T"] * (8 + 4 * Hkv * D) + live * cell, "flops": live * 4 * Hkv * D}
    if c["op"] == "append":
        T, live, H = c["T"], c["T"] - c["pad"], c["Hq"] + Hkv
        return {"bytes": T * (4 * c["Hq"] * D + 4 * c["rot"] + 12 + 4 * Hkv * D) + live * (4 * Hkv * D + 2 * cell) + 8 * T,
                "flops": T * H * (3 * c["rot"] + (4 * D if c["norm"] else 0)) + live * 12 * Hkv * D}
    read = pairs = rows = 0
    for n, L in _lengths(c):
        W = c["window"] or L + 1
        rows += n
        read += min(L, W + n - 1 + c["sinks"])
        for seen in range(max(0, L - n) + 1, L + 1):     # keys up to each row's own
            pairs += min(seen, W) + min(c["sinks"], max(0, seen - W))
    return {"bytes": read * cell + rows * c["Hq"] * (4 * D + 4 * c["lse"]), "flops": 4 * D * c["Hq"] * pairs}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits

def _exact_group_values(x, G):
    """What x [T, H, D] stands for after 4 bits: for each group the nearest of its 16 levels, halves to the even code."""
    T, H, D = x.shape
    x = x.clamp(-TOP, TOP).reshape(T, H, D // G, G)
    zero = torch.zeros_like(x[..., :1])
    span = torch.cat((x, zero), -1)
    lo, width = span.min(-1, keepdim=True).values, span.max(-1, keepdim=True).values - span.min(-1, keepdim=True).values
    unit = 2.0 ** (torch.floor(torch.log2((width / 15).clamp(min=2.0 ** -30))) - 6)      # 64 units and more, up to 128
    s = (torch.round(width / 15 / unit) * unit).clamp(min=2.0 ** -18)
    z = torch.round(-lo / s).clamp(max=15)
    level = torch.arange(16, device=x.device, dtype=torch.float64)
    value = torch.empty_like(x)
    for a in range(0, T, 512):     # distance to every level; of two alike the one an even number of steps from zero
        steps = level - z[a:a + 512]
        far = (x[a:a + 512, ..., None] / s[a:a + 512, ..., None] - steps[..., None, :]).abs() + (steps.remainder(2) * 1e-13)[..., None, :]
        value[a:a + 512] = torch.gather(steps.expand(*far.shape[:3], 16), -1, far.argmin(-1)) * s[a:a + 512]
    return value.reshape(T, H, D)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    D = c["D"]
    if c["op"] in ("norm", "append"):
        rot = c["rot"]
        lane = torch.arange(rot // 2, device=DEVICE)
        one, two = (2 * lane, 2 * lane + 1) if c["pairs"] else (lane, lane + rot // 2)
        turn = torch.complex(s["rope"][:, :rot // 2].double(), s["rope"][:, rot // 2:].double())[s["positions"].long()][:, None]

        def turned(x, weight):
            x = x.double()
            x = x.clone() if weight is None else x * weight.double() * (x.pow(2).sum(-1, keepdim=True) / D + EPS).rsqrt()
            y = torch.complex(x[..., one], x[..., two]) * turn
            x[..., one], x[..., two] = y.real, y.imag
            return x

        q, k = turned(s["q"], s["q_weight"]), turned(s["k"], s["k_weight"])
        if c["op"] == "norm":
            return q, k
        live = (s["slots"] >= 0)[:, None, None].double()
        return q, _exact_group_values(k, c["G"]) * live, _exact_group_values(s["v"].double(), c["G"]) * live
    k_cache, v_cache, k_scale, v_scale = s["cache"]

    def values(codes, scale, H):
        """[..., page, D] of one head's pages (or tokens), H a head or all."""
        pick = (slice(None),) if H is None else (slice(None), H)
        b = codes[pick].double()
        high = torch.floor(b / 16)
        x = torch.empty(*b.shape[:-1], D, device=DEVICE, dtype=torch.float64)
        x[..., 0::2], x[..., 1::2] = b - 16 * high, high
        sz = scale[pick].double().repeat_interleave(c["G"], -2)
        return (x - sz[..., 1]) * sz[..., 0]

    if c["op"] == "read":
        out = []
        for codes, scale in ((k_cache, k_scale), (v_cache, v_scale)):
            flat = [t.transpose(1, 2).flatten(0, 1) for t in (codes, scale)]
            x = torch.zeros(c["T"], c["Hkv"], D, device=DEVICE, dtype=torch.float64)
            live = s["slots"] >= 0
            x[live] = values(flat[0][s["slots"][live]], flat[1][s["slots"][live]], None)
            out.append(x)
        return tuple(out)
    lens, g = _lengths(c), c["Hq"] // c["Hkv"]
    out, lse, t = [], [], 0
    for b, (n, L) in enumerate(lens):
        q = s["q"][t:t + n].double().transpose(0, 1)            # [Hq, n, D]
        t += n
        if L == 0:
            out.append(torch.zeros(n, c["Hq"], D, dtype=torch.float64, device=DEVICE))
            lse.append(torch.full((n, c["Hq"]), -math.inf, dtype=torch.float64, device=DEVICE))
            continue
        ids = s["page_table"][b, : -(-L // c["page"])].long()
        pos = torch.arange(L - n, L, device=DEVICE)[:, None]
        key = torch.arange(L, device=DEVICE)
        hidden = (key > pos) | ((key <= pos - c["window"]) & (key >= c["sinks"]) if c["window"] else key < 0)
        o, l = [], []
        for h in range(c["Hkv"]):
            k = values(k_cache[ids], k_scale[ids], h).reshape(-1, D)[:L]
            v = values(v_cache[ids], v_scale[ids], h).reshape(-1, D)[:L]
            x = (q[h * g:(h + 1) * g].reshape(g * n, D) @ k.T * s["scale"]).view(g, n, L).masked_fill(hidden, -math.inf)
            o.append(torch.softmax(x, -1).view(g * n, L).matmul(v).view(g, n, D))
            l.append(torch.logsumexp(x, -1))
        out.append(torch.cat(o).transpose(0, 1))
        lse.append(torch.cat(l).transpose(0, 1))
    return torch.cat(out) if not c["lse"] else (torch.cat(out), torch.cat(lse))
