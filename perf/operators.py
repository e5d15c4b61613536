"""What a decoder layer on k-bit weights runs besides the plain product, as cases that can be timed:

  linear   Y = act(X . dequant(Wq) + bias) * mul + residual      (projections of attention and MLP)
  append   rotary positions applied to q and k, k and v written into a paged cache
  attend   attention of a chunk of new tokens (one token and more) over that cache

``own = False``: elementary torch operations in fp32 on the same inputs.  ``own = True``: the
calls of this repository's package.  Sizes are those of the repository's own workloads (7B, 8B and
70B class projections, tokens of 1 to thousands) and generic ones.
"""
import math

import torch

own = False

DEVICE = "cuda"
TABLE = 131072          # positions the rotary table covers


def listed():
    return [
        # gate projection of a gated MLP for one token of one user: silu(x W) * up, 7B class
        dict(name="linear_token", op="linear", M=1, K=4096, N=11008, bits=4, G=128, z=False, bias=False, act="silu", mul=True, residual=False),
        # MLP down projection of a decode batch, added to the residual stream, 70B class
        dict(name="linear_batch", op="linear", M=16, K=28672, N=8192, bits=4, G=128, z=True, bias=False, act="none", mul=False, residual=True),
        # a ragged batch through a small layer with every part of the epilogue, 3-bit codes
        dict(name="linear_ragged", op="linear", M=37, K=2080, N=1000, bits=3, G=32, z=True, bias=True, act="gelu", mul=True, residual=True),
        # gate projection for a prompt of 4096 tokens, 8B class
        dict(name="linear_prompt", op="linear", M=4096, K=4096, N=14336, bits=4, G=128, z=False, bias=False, act="silu", mul=True, residual=False),
        # one new token of one user
        dict(name="append_token", op="append", T=1, start=4095, pad=0, Hq=32, Hkv=8, D=128, rot=128, pairs=False, page=16, dtype="float16", e4m3=False),
        # a batch of new tokens, some of them padding, into an 8-bit cache; partial rotation of neighbouring elements
        dict(name="append_e4m3", op="append", T=777, start=1000, pad=23, Hq=32, Hkv=8, D=128, rot=64, pairs=True, page=16, dtype="float16", e4m3=True),
        # a long prompt, far into its context
        dict(name="append_prompt", op="append", T=8192, start=100000, pad=0, Hq=64, Hkv=8, D=128, rot=128, pairs=False, page=64, dtype="bfloat16", e4m3=False),
        # one user's next token, short context
        dict(name="attend_token", op="attend", B=1, n=1, L=513, spread=0.0, idle=0, Hq=32, Hkv=8, D=128, page=16, window=0, dtype="float16", e4m3=False, lse=False),
        # a decode batch of users with contexts of all lengths, four idle places
        dict(name="attend_batch", op="attend", B=64, n=1, L=8192, spread=0.95, idle=4, Hq=32, Hkv=8, D=128, page=16, window=0, dtype="float16", e4m3=False, lse=True),
        # very long contexts in an 8-bit cache
        dict(name="attend_long", op="attend", B=4, n=1, L=131071, spread=0.3, idle=0, Hq=64, Hkv=8, D=128, page=64, window=0, dtype="float16", e4m3=True, lse=False),
        # chunks of prompts whose beginnings are in the cache already
        dict(name="attend_chunk", op="attend", B=3, n=600, L=32768, spread=0.5, idle=0, Hq=32, Hkv=8, D=128, page=16, window=0, dtype="bfloat16", e4m3=False, lse=False),
        # whole prompts, one key head for each query head
        dict(name="attend_prompt", op="attend", B=2, n=4096, L=4096, spread=0.0, idle=0, Hq=32, Hkv=32, D=128, page=64, window=0, dtype="float16", e4m3=False, lse=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "append", "attend", "attend"))
    if op == "linear":
        G = rng.choice((32, 64, 128))
        while True:
            M, K, N = _log(rng, 1, 4096), G * _log(rng, 1, 28672 // G), _log(rng, 1, 28672)
            if M * K * N <= 4096 * 4096 * 14336 and K * N <= 28672 * 8192:
                break
        return dict(op=op, M=M, K=K, N=N, bits=rng.randint(1, 8), G=G, z=rng.random() < 0.5, bias=rng.random() < 0.5,
                    act=rng.choice(("none", "relu", "silu", "gelu", "gelu_tanh")), mul=rng.random() < 0.5, residual=rng.random() < 0.5)
    Hkv, g = rng.choice((1, 2, 4, 5, 8, 16)), rng.choice((1, 2, 3, 4, 8))
    D = rng.choice((64, 80, 96, 128, 128, 128, 256))
    page, dtype, e4m3 = rng.choice((1, 16, 32, 64, 256)), rng.choice(("float16", "bfloat16")), rng.random() < 0.3
    if op == "append":
        T = _log(rng, 1, 4096)
        return dict(op=op, T=T, start=rng.randint(0, TABLE - 4096), pad=rng.randint(0, T // 4), Hq=Hkv * g, Hkv=Hkv, D=D,
                    rot=rng.choice((D, D, D // 2)), pairs=rng.random() < 0.4, page=page, dtype=dtype, e4m3=e4m3)
    while True:
        n = 1 if rng.random() < 0.4 else _log(rng, 2, 4096)
        B, L = _log(rng, 1, 64), _log(rng, 1, 131072)
        if n <= L and B * n * L * Hkv * g <= 1_800_000_000 and B * n * L * Hkv * g * D <= 128 * 2 * 32 * 4096 * 4096 \
                and B * L * Hkv * D <= 4 * 131072 * 8 * 128:
            break
    return dict(op=op, B=B, n=n, L=L, spread=round(rng.uniform(0, 0.99), 3), idle=rng.choice((0, 0, 1)) if B > 1 else 0, Hq=Hkv * g, Hkv=Hkv, D=D,
                page=page, window=rng.choice((0, 0, 0, _log(rng, 16, 4096))), dtype=dtype, e4m3=e4m3, lse=rng.random() < 0.5)


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

def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEVICE)

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, generator=gen, device=DEVICE) * (hi - lo) + lo

    s = dict(case=dict(c))
    if c["op"] == "linear":
        M, K, N, bits, G = c["M"], c["K"], c["N"], c["bits"], c["G"]
        s["X"] = normal(M, K).half()
        # a random stream is a stream of uniform random codes
        s["wq"] = torch.randint(-2 ** 31, 2 ** 31, (N, K * bits // 32), generator=gen, device=DEVICE, dtype=torch.int64).to(torch.int32)
        s["s"] = (uniform(0.25, 2.0, N, K // G) * (0.09 / 2 ** bits)).half()
        s["z"] = torch.randint(0, 2 ** bits, (N, K // G), generator=gen, device=DEVICE).half() if c["z"] else None
        s["bias"] = normal(N).half() if c["bias"] else None
        s["mul"] = normal(M, N).half() if c["mul"] else None
        s["residual"] = normal(M, N).half() if c["residual"] else None
        return s
    dt = getattr(torch, c["dtype"])
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    cdt = torch.float8_e4m3fn if c["e4m3"] else dt
    s["k_scale"] = uniform(0.01, 0.02, Hkv) if c["e4m3"] else None
    s["v_scale"] = uniform(0.01, 0.02, Hkv) if c["e4m3"] else None
    if c["op"] == "append":
        T, rot = c["T"], c["rot"]
        # q, k and v are columns of one fused projection
        qkv = normal(T, (Hq + 2 * Hkv) * D).to(dt)
        s["q"] = qkv[:, :Hq * D].unflatten(1, (Hq, D))
        s["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
        s["v"] = qkv[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
        pages = (T + page - 1) // page + 3
        order = torch.randperm(pages, generator=gen, device=DEVICE)
        at = torch.arange(T, device=DEVICE) + c["start"] % page % 7
        s["slots"] = order[at // page % pages] * page + at % page
        if c["pad"]:
            s["slots"][T - c["pad"]:] = -1
        s["positions"] = torch.arange(T, device=DEVICE, dtype=torch.int32) + c["start"]
        angle = torch.arange(TABLE, device=DEVICE, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(rot // 2, device=DEVICE, dtype=torch.float64) * 2 / rot)
        s["rope"] = torch.cat((angle.cos(), angle.sin()), 1).float()
        s["k_cache"] = (normal(pages, Hkv, page, D) * (20 if c["e4m3"] else 1)).to(cdt)
        s["v_cache"] = (normal(pages, Hkv, page, D) * (20 if c["e4m3"] else 1)).to(cdt)
        s["out"] = torch.empty(T, Hq, D, device=DEVICE, dtype=dt)
        return s
    lens = _lengths(c)
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
    s["k_cache"] = torch.empty(pages, Hkv, page, D, dtype=cdt, device=DEVICE)
    s["v_cache"] = torch.empty_like(s["k_cache"])
    s["k_cache"].copy_(normal(pages, Hkv, page, D) * (60 if c["e4m3"] else 1))
    s["v_cache"].copy_(normal(pages, Hkv, page, D) * (60 if c["e4m3"] else 1))
    s["scale"] = D ** -0.5
    s["out"] = torch.empty(T, Hq, D, device=DEVICE, dtype=dt)
    s["lse"] = torch.empty(T, Hq, device=DEVICE, dtype=torch.float32) if c["lse"] else None
    return s


# ---------------------------------------------------------------------------------------------
# one pass

def run(state):
    op = state["case"]["op"]
    if op == "linear":
        return _linear_own(state) if own else _linear(state)
    if op == "append":
        return _append_own(state) if own else _append(state)
    return _attend_own(state) if own else _attend(state)


def _linear_own(s):
    import bit_weight_quantized_qmm_amd as qmm
    c = s["case"]
    return qmm.linear(s["X"], s["wq"], s["s"], s["z"], c["bits"], c["G"], bias=s["bias"], act=c["act"], mul=s["mul"], residual=s["residual"])


def _append_own(s):
    import bit_weight_quantized_qmm_amd as qmm
    q = qmm.kv_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], s["positions"], s["rope"], pairs=s["case"]["pairs"],
                      k_scale=s["k_scale"], v_scale=s["v_scale"], out=s["out"])
    return q, s["k_cache"], s["v_cache"]


def _attend_own(s):
    import bit_weight_quantized_qmm_amd as qmm
    out = qmm.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["cu_q"], s["kv_lens"], s["max_q"], s["max_kv"], scale=s["scale"],
                              window=s["case"]["window"], k_scale=s["k_scale"], v_scale=s["v_scale"], out=s["out"], lse=s["lse"])
    return out if s["lse"] is None else (out, s["lse"])


def _linear(s):
    c = s["case"]
    K, bits, G = c["K"], c["bits"], c["G"]
    bit = torch.arange(K, device=DEVICE) * bits
    words = s["wq"].long() & 0xffffffff
    low = words[:, bit // 32]
    high = words[:, torch.clamp(bit // 32 + 1, max=words.shape[1] - 1)]
    codes = ((low >> (bit % 32)) | (high << (32 - bit % 32))) & ((1 << bits) - 1)
    z = float(1 << (bits - 1)) if s["z"] is None else s["z"].float()[:, :, None]
    w = ((codes.float().unflatten(1, (K // G, G)) - z) * s["s"].float()[:, :, None]).flatten(1)
    h = torch.matmul(s["X"].float(), w.t())
    if s["bias"] is not None:
        h = h + s["bias"].float()
    if c["act"] == "relu":
        h = torch.where(h > 0, h, 0.0)
    elif c["act"] == "silu":
        h = h / (1 + torch.exp(-h))
    elif c["act"] == "gelu":
        h = 0.5 * h * (1 + torch.erf(h * math.sqrt(0.5)))
    elif c["act"] == "gelu_tanh":
        h = 0.5 * h * (1 + torch.tanh(math.sqrt(2 / math.pi) * (h + 0.044715 * h * h * h)))
    if s["mul"] is not None:
        h = h * s["mul"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    return h.half()


def _rotate(x, cos, sin, rot, pairs):
    x = x.float()
    if pairs:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _append(s):
    c = s["case"]
    rot, page = c["rot"], c["page"]
    line = s["rope"][s["positions"].long()][:, None, :]
    cos, sin = line[..., :rot // 2], line[..., rot // 2:]
    s["out"].copy_(_rotate(s["q"], cos, sin, rot, c["pairs"]))
    k, v = _rotate(s["k"], cos, sin, rot, c["pairs"]), s["v"].float()
    if c["e4m3"]:
        k = torch.clamp(k / s["k_scale"][None, :, None], -448.0, 448.0)
        v = torch.clamp(v / s["v_scale"][None, :, None], -448.0, 448.0)
    # padding stands at the end: its values go nowhere
    live = c["T"] - c["pad"]
    at, within = s["slots"][:live] // page, s["slots"][:live] % page
    for cache, x in ((s["k_cache"], k), (s["v_cache"], v)):
        x = x[:live].to(cache.dtype)
        if c["e4m3"]:
            cache, x = cache.view(torch.uint8), x.view(torch.uint8)
        cache[at, :, within] = x
    return s["out"], s["k_cache"], s["v_cache"]


def _attend(s):
    c = s["case"]
    Hkv, D, page, g = c["Hkv"], c["D"], c["page"], c["Hq"] // c["Hkv"]
    cu, lens = s["cu_q"].long(), s["kv_lens"].long()
    n, B = cu[1:] - cu[:-1], c["B"]
    i, j = torch.arange(s["max_q"], device=DEVICE), torch.arange(s["max_kv"], device=DEVICE)
    T = s["q"].shape[0]

    def dense(cache, scale):     # [B, Hkv, max_kv, D]
        if c["e4m3"]:
            cache = cache.view(torch.uint8)
        x = cache[s["page_table"].long()[:, j // page], :, j % page]
        if c["e4m3"]:
            x = x.view(torch.float8_e4m3fn)
        x = x.float()
        return (x if scale is None else x * scale[None, None, :, None]).transpose(1, 2).contiguous()

    q = s["q"].float()[torch.clamp(cu[:-1, None] + i, max=T - 1)]
    q = q.unflatten(2, (Hkv, g)).permute(0, 2, 3, 1, 4).reshape(B, Hkv, g * i.numel(), D)
    pos = (lens - n)[:, None] + i
    seen = (j <= pos[..., None]) & (j < lens[:, None, None])
    if c["window"]:
        seen = seen & (j > pos[..., None] - c["window"])
    x = torch.matmul(q, dense(s["k_cache"], s["k_scale"]).transpose(2, 3)).unflatten(2, (g, i.numel()))
    x = torch.where(seen[:, None, None], x * s["scale"], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.flatten(2, 3), dense(s["v_cache"], s["v_scale"])).unflatten(2, (g, i.numel()))
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
    if c["op"] == "linear":
        M, K, N = c["M"], c["K"], c["N"]
        sides = 1 + c["mul"] + c["residual"]
        return {"bytes": N * K * c["bits"] / 8 + 2 * N * (K // c["G"]) * (1 + c["z"]) + 2 * M * K + 2 * M * N * sides + 2 * N * c["bias"], "flops": 2 * M * K * N}
    Hq, Hkv, D, cell = c["Hq"], c["Hkv"], c["D"], 1 if c["e4m3"] else 2
    if c["op"] == "append":
        T, live = c["T"], c["T"] - c["pad"]
        return {"bytes": T * (4 * Hq * D + 4 * c["rot"] + 12) + live * 2 * Hkv * D * (2 + cell), "flops": 3 * c["rot"] * (T * Hq + live * Hkv)}
    read = pairs = rows = 0
    for n, L in _lengths(c):
        W = c["window"] or L + 1
        first, last = max(0, L - n + 1), L            # keys that the first and the last row see, without a window
        rows += n
        read += min(L, W + n - 1)
        if L:
            small = max(0, min(last, W) - first + 1)    # rows that see less than the window
            pairs += small * (first + min(last, W)) // 2 + (n - small) * W if first <= W else n * W
    return {"bytes": read * Hkv * D * 2 * cell + rows * Hq * (4 * D + 4 * c["lse"]), "flops": 4 * D * Hq * pairs}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "linear":
        bits, G, K, N = c["bits"], c["G"], c["K"], c["N"]
        stream = s["wq"].view(torch.uint8).reshape(N, -1)
        w = torch.zeros(N, K, dtype=torch.float64, device=DEVICE)
        for b in range(bits):        # bit b of code i is bit i * bits + b of the column's stream
            p = torch.arange(K, device=DEVICE) * bits + b
            w += ((stream[:, p >> 3] >> (p & 7).to(torch.uint8)) & 1).double() * 2 ** b
        group = torch.arange(K, device=DEVICE) // G
        w -= s["z"].double()[:, group] if c["z"] else 2 ** (bits - 1)
        w *= s["s"].double()[:, group]
        y = s["X"].double() @ w.T
        del w
        if c["bias"]:
            y += s["bias"].double()
        if c["act"] == "relu":
            y = y.clamp(min=0)
        elif c["act"] == "silu":
            y = y * torch.sigmoid(y)
        elif c["act"] == "gelu":
            y = y * torch.special.ndtr(y)
        elif c["act"] == "gelu_tanh":
            y = y * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3))
        if c["mul"]:
            y = y * s["mul"].double()
        if c["residual"]:
            y = y + s["residual"].double()
        return y
    D = c["D"]
    if c["op"] == "append":
        rot, page, T = c["rot"], c["page"], c["T"]
        lane = torch.arange(rot // 2, device=DEVICE)
        one, two = (2 * lane, 2 * lane + 1) if c["pairs"] else (lane, lane + rot // 2)
        turn = torch.complex(s["rope"][:, :rot // 2].double(), s["rope"][:, rot // 2:].double())[s["positions"].long()][:, None]

        def rotated(x):
            x = x.double().clone()
            y = torch.complex(x[..., one], x[..., two]) * turn
            x[..., one], x[..., two] = y.real, y.imag
            return x

        caches = []
        for cache, x, scale in ((s["k_cache"], rotated(s["k"]), s["k_scale"]), (s["v_cache"], s["v"].double(), s["v_scale"])):
            flat = cache.double().transpose(1, 2).reshape(-1, c["Hkv"], D).clone()
            live = s["slots"] >= 0
            if scale is not None:
                x = (x / scale.double()[:, None]).clamp(-448, 448)
            flat[s["slots"][live]] = x[live]
            caches.append(flat.reshape(-1, page, c["Hkv"], D).transpose(1, 2).contiguous())
        return rotated(s["q"]), caches[0], caches[1]
    lens, page, g = _lengths(c), c["page"], c["Hq"] // c["Hkv"]
    out, lse, t = [], [], 0
    for b, (n, L) in enumerate(lens):
        q = s["q"][t:t + n].double().transpose(0, 1)            # [Hq, n, D]
        t += n
        if L == 0:
            out.append(torch.zeros(n, c["Hq"], D, dtype=torch.float64, device=DEVICE))
            lse.append(torch.full((n, c["Hq"]), -math.inf, dtype=torch.float64, device=DEVICE))
            continue
        ids = s["page_table"][b, : -(-L // page)].long()
        pos = torch.arange(L - n, L, device=DEVICE)[:, None]
        key = torch.arange(L, device=DEVICE)
        hidden = (key > pos) | (key <= pos - c["window"] if c["window"] else key < 0)
        o, l = [], []
        for h in range(c["Hkv"]):
            k, v = (x[ids, h].double().reshape(-1, D)[:L] for x in (s["k_cache"], s["v_cache"]))
            if c["e4m3"]:
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            x = (q[h * g:(h + 1) * g].reshape(g * n, D) @ k.T * s["scale"]).view(g, n, L).masked_fill(hidden, -math.inf)
            o.append(torch.softmax(x, -1).view(g * n, L).matmul(v).view(g, n, D))
            l.append(torch.logsumexp(x, -1))
        out.append(torch.cat(o).transpose(0, 1))
        lse.append(torch.cat(l).transpose(0, 1))
    return torch.cat(out) if not c["lse"] else (torch.cat(out), torch.cat(lse))
