"""The operators of a decoder layer around the products (qmm_linear, qmm_kv_append,
qmm_paged_attention) against their formulas in 64 bits, on an MI355X.

Tolerances count roundings.  u is half a step of the output's type (2^-11 for
fp16, 2^-8 for bf16); fp32 sums of n terms are off by at most n 2^-24 of the
sum of magnitudes.  Every bound below is per element.
"""
import math
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import bit_weight_quantized_qmm_amd as qmm
    return qmm


@pytest.fixture(autouse=True)
def _announce(request):
    print(f"\nCASE {request.node.nodeid}", file=sys.stderr, flush=True)
    yield
    torch.cuda.synchronize()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def close(got, want, bound):
    got = got.double()
    assert torch.isfinite(got).all()
    over = (got - want).abs() - bound
    at = int(over.argmax())
    assert over.flatten()[at] <= 0, f"off by {float((got - want).abs().flatten()[at]):.3e}, bound {float(bound.flatten()[at]):.3e}, " \
                                    f"value {float(want.flatten()[at]):.3e} at {at}"


# ------------------------------------------------------------------ linear --
def weights(K, N, bits, G, z, g):
    wq = torch.randint(-2 ** 31, 2 ** 31, (N, K * bits // 32), generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    s = ((torch.rand(N, K // G, generator=g, device=DEV) * 1.75 + 0.25) * (0.09 / 2 ** bits)).half()
    zz = torch.randint(0, 2 ** bits, (N, K // G), generator=g, device=DEV).half() if z else None
    return wq, s, zz


def decoded(wq, K, bits):
    stream = wq.view(torch.uint8).reshape(wq.shape[0], -1)
    w = torch.zeros(wq.shape[0], K, dtype=torch.float64, device=DEV)
    for b in range(bits):
        p = torch.arange(K, device=DEV) * bits + b
        w += ((stream[:, p >> 3] >> (p & 7).to(torch.uint8)) & 1).double() * 2 ** b
    return w


ACTS = {"none": lambda h: h, "relu": lambda h: h.clamp(min=0), "silu": lambda h: h * torch.sigmoid(h),
        "gelu": lambda h: h * torch.special.ndtr(h),
        "gelu_tanh": lambda h: h * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (h + 0.044715 * h ** 3))}


def linear_reference(X, wq, s, z, bits, G, bias, act, mul, residual):
    """(Y, bound): the steepest activation has slope below 1.13; act itself is good to 2^-17 of its value."""
    K, N = X.shape[1], s.shape[0]
    codes, S = decoded(wq, K, bits), s.double().repeat_interleave(G, 1)
    Z = torch.full_like(S, 2.0 ** (bits - 1)) if z is None else z.double().repeat_interleave(G, 1)
    w, x = (codes - Z) * S, X.double()
    h = x @ w.T
    # weights rounded once, fp32 sums; up to 16 rows the codes' offset of 1024 is taken from fp32 sums
    eh = (2.0 ** -11 + K * 2.0 ** -23) * (x.abs() @ w.abs().T)
    if X.shape[0] <= 16:
        eh = eh + 2.0 ** -16 * (x.abs() @ ((1024 + Z) * S).T)
    if bias is not None:
        h = h + bias.double()
    y = ACTS[act](h)
    e = 1.13 * eh + 2.0 ** -17 * y.abs()
    if mul is not None:
        y, e = y * mul.double(), e * mul.double().abs()
    if residual is not None:
        y = y + residual.double()
    return y, e + y.abs() * U[torch.float16] + 2.0 ** -24


LINEAR = [(1, 256, 40, 64), (1, 4096, 1000, 128), (1, 9216, 33, 32), (1, 16384, 70, 128), (2, 96, 19, 32), (3, 1024, 130, 64), (7, 2080, 50, 32),
          (16, 1152, 264, 128), (16, 8320, 17, 128), (17, 256, 8, 32), (37, 2080, 1000, 32), (64, 4224, 4000, 128), (20, 8192, 2001, 64), (33, 28800, 600, 96), (5, 16384, 33, 32), (2, 9344, 130, 64), (50, 512, 28680, 32), (111, 5760, 2001, 64), (130, 8192, 1032, 32), (263, 10240, 700, 128), (129, 512, 264, 128), (300, 128, 777, 64),
          (1100, 256, 1032, 128)]


@pytest.mark.parametrize("M,K,N,G", LINEAR, ids=lambda v: str(v))
@pytest.mark.parametrize("bits", [1, 3, 4, 8])
def test_linear(q, M, K, N, G, bits):
    g = gen(1000 * bits + M + N)
    X = torch.randn(M, K, generator=g, device=DEV).half()
    wq, s, z = weights(K, N, bits, G, bits % 2 == 1, g)
    bias, mul, res = (torch.randn(*sh, generator=g, device=DEV).half() for sh in ((N,), (M, N), (M, N)))
    for act, b, m, r in (("none", None, None, None), ("silu", None, mul, None), ("none", bias, None, res), ("gelu", bias, mul, res),
                         ("gelu_tanh", bias, None, None), ("relu", None, mul, res)):
        Y = q.linear(X, wq, s, z, bits, G, bias=b, act=act, mul=m, residual=r)
        close(Y, *linear_reference(X, wq, s, z, bits, G, b, act, m, r))


@pytest.mark.parametrize("bits", range(1, 9))
@pytest.mark.parametrize("M", [1, 70])
def test_linear_without_epilogue_is_the_product(q, bits, M):
    g = gen(7 + bits)
    X = torch.randn(M, 512, generator=g, device=DEV).half()
    wq, s, z = weights(512, 100, bits, 128, True, g)
    plain = (q.gemv if M <= 16 else q.gemm)(X, wq, s, z, bits, 128)
    assert same(q.linear(X, wq, s, z, bits, 128), plain)


@pytest.mark.parametrize("M,N", [(1, 1000), (9, 136), (70, 136), (70, 137)])
def test_linear_in_place_and_odd_starts(q, M, N):
    """residual and mul as the output itself; operands that stand at 2-byte multiples."""
    g = gen(M + N)
    X = torch.randn(M, 256, generator=g, device=DEV).half()
    wq, s, z = weights(256, N, 4, 64, True, g)
    flat = torch.randn(2 * M * N + N + 3, generator=g, device=DEV).half()
    bias, mul, res = flat[1:1 + N], flat[N + 1:N + 1 + M * N].view(M, N), flat[N + 2 + M * N:N + 2 + 2 * M * N].view(M, N)
    want = linear_reference(X, wq, s, z, 4, 64, bias, "silu", mul, res)
    y = res.clone()
    assert q.linear(X, wq, s, z, 4, 64, bias=bias, act="silu", mul=mul, residual=y, out=y) is y
    close(y, *want)
    y = mul.clone()
    q.linear(X, wq, s, z, 4, 64, bias=bias, act="silu", mul=y, residual=res, out=y)
    close(y, *want)
    buf = torch.full((M * N + 2,), -7.0, device=DEV).half()
    q.linear(X, wq, s, z, 4, 64, bias=bias, act="silu", mul=mul, residual=res, out=buf[1:-1].view(M, N))
    close(buf[1:-1].view(M, N), *want)
    assert buf[0] == -7 and buf[-1] == -7


@pytest.mark.parametrize("M", [1, 4, 40])
def test_linear_far_activations(q, M):
    """Sums far into both tails: gelu and silu keep their relative accuracy, nothing overflows."""
    X = torch.ones(M, 32, device=DEV).half()
    wq, s, _ = weights(32, 64, 1, 32, False, gen(3))
    s.fill_(1e-4)
    bias = torch.linspace(-20, 20, 64, device=DEV).half()
    bias[0], bias[1], bias[2] = 60000, -60000, -30
    for act in ("silu", "gelu", "gelu_tanh", "relu"):
        Y = q.linear(X, wq, s, None, 1, 32, bias=bias, act=act)
        close(Y, *linear_reference(X, wq, s, None, 1, 32, bias, act, None, None))


def test_linear_no_rows(q):
    wq, s, _ = weights(64, 10, 4, 32, False, gen(1))
    assert q.linear(torch.empty(0, 64, dtype=torch.float16, device=DEV), wq, s, None, 4, 32).shape == (0, 10)


# ------------------------------------------------------------------ append --
def rope_table(rows, rot):
    angle = torch.arange(rows, device=DEV, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(rot // 2, device=DEV, dtype=torch.float64) * 2 / rot)
    return torch.cat((angle.cos(), angle.sin()), 1).float()


def turned(x, line, rot, pairs):
    x = x.double().clone()
    lane = torch.arange(rot // 2, device=DEV)
    one, two = (2 * lane, 2 * lane + 1) if pairs else (lane, lane + rot // 2)
    a, b = x[..., one].clone(), x[..., two].clone()
    c, s = line[:, None, :rot // 2].double(), line[:, None, rot // 2:].double()
    x[..., one], x[..., two] = a * c - b * s, b * c + a * s
    size = torch.zeros_like(x)
    size[..., one] = size[..., two] = a.abs() + b.abs()
    return x, size * 2.0 ** -22


def check_append(q, T, Hq, Hkv, D, rot, page, pairs, dtype, e4m3, cut=0, seed=0, layout="fused"):
    g = gen(seed)
    width = (Hq + 2 * Hkv) * D
    if layout == "odd":       # rows that stand at 2-byte multiples
        qkv = torch.randn(T * (width + 1) + 1, generator=g, device=DEV).to(dtype)[1:].view(T, width + 1)[:, :width]
    else:
        qkv = torch.randn(T, width, generator=g, device=DEV).to(dtype)
    xq, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split((Hq * D, Hkv * D, Hkv * D), 1))
    pages = (T + page - 1) // page + 2
    order = torch.randperm(pages * page, generator=g, device=DEV)[:T]
    slots = order.clone()
    if T:
        slots[T - cut:] = -1
    if cut > 1:
        slots[T - 1] = pages * page
        slots[0], slots[T - 2] = -5, slots[0].clone()
    rows = 5000
    positions = torch.randint(0, rows, (T,), generator=g, device=DEV, dtype=torch.int32)
    table = rope_table(rows, rot) if rot else None
    cdt = E4M3 if e4m3 else dtype
    both = (torch.randn(pages, 2, Hkv, page, D, generator=g, device=DEV) * 4).to(cdt)     # one tensor for both caches
    kc, vc = both[:, 0], both[:, 1]
    ksc, vsc = ((torch.rand(Hkv, generator=g, device=DEV) * 0.01 + 0.005) for _ in range(2)) if e4m3 else (None, None)
    before = both.clone()
    out = q.kv_append(xq, k, v, kc, vc, slots, positions if rot else None, table, pairs=pairs, k_scale=ksc, v_scale=vsc)
    line = table[positions.long()] if rot else torch.zeros(T, 0, device=DEV)
    want, size = turned(xq, line, rot, pairs)
    close(out, want, size + want.abs() * U[dtype] + 2.0 ** -25) if T and Hq else None
    live = (slots >= 0) & (slots < pages * page)
    assert int(live.sum()) == T - (0 if cut == 0 else cut if cut == 1 else cut)
    at, within = slots[live] // page, slots[live] % page
    kt, size = turned(k, line, rot, pairs)
    if e4m3:
        for cache, x, sc, extra in ((kc, kt, ksc, size), (vc, v.double(), vsc, torch.zeros_like(size))):
            w = (x / sc.double()[:, None]).clamp(-448, 448)[live]
            close(cache.view(torch.uint8)[at, :, within].view(E4M3).double(), w, w.abs() * 2.0 ** -4 + 2.0 ** -10 + (extra / sc.double()[:, None])[live])
    else:
        if T:
            close(kc[at, :, within], kt[live], (size + kt.abs() * U[dtype])[live] + 2.0 ** -25)
        assert same(vc[at, :, within], v[live])
    rest = torch.ones(pages, page, dtype=torch.bool, device=DEV)
    rest[at, within] = False
    untouched = rest[:, None, None, :, None].expand(both.shape)
    assert torch.equal(both.view(torch.uint8 if e4m3 else torch.int16)[untouched], before.view(torch.uint8 if e4m3 else torch.int16)[untouched])
    return out


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("e4m3", [False, True], ids=["plain", "e4m3"])
@pytest.mark.parametrize("pairs", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,page", [(1, 4, 2, 128, 128, 16), (77, 5, 5, 128, 64, 16), (33, 8, 1, 80, 80, 1), (50, 3, 1, 96, 48, 7),
                                                (19, 2, 2, 64, 20, 32), (65, 2, 1, 256, 256, 256), (130, 1, 1, 80, 40, 3), (700, 16, 4, 64, 64, 64)])
def test_append(q, T, Hq, Hkv, D, rot, page, pairs, dtype, e4m3):
    check_append(q, T, Hq, Hkv, D, rot, page, pairs, dtype, e4m3, cut=min(T // 8, 5), seed=T + D)


@pytest.mark.parametrize("e4m3", [False, True], ids=["plain", "e4m3"])
def test_append_odd_starts(q, e4m3):
    check_append(q, 41, 3, 2, 80, 40, 16, False, torch.float16, e4m3, cut=3, seed=5, layout="odd")
    check_append(q, 41, 3, 2, 128, 128, 16, True, torch.bfloat16, e4m3, cut=3, seed=6, layout="odd")


def test_append_without_positions_and_empty(q):
    check_append(q, 12, 4, 2, 64, 0, 4, False, torch.float16, False, seed=1)
    check_append(q, 0, 4, 2, 64, 64, 4, False, torch.float16, False, seed=2)


def test_append_in_place_and_keys_alone(q):
    g = gen(9)
    xq, k, v = (torch.randn(20, h, 64, generator=g, device=DEV).half() for h in (6, 2, 2))
    table, pos = rope_table(100, 64), torch.arange(20, device=DEV, dtype=torch.int32) + 50
    slots = torch.arange(20, device=DEV)
    kc, vc = (torch.zeros(2, 2, 16, 64, device=DEV).half() for _ in range(2))
    want = q.kv_append(xq, k, v, kc, vc, slots, pos, table)
    kc2, vc2 = torch.zeros_like(kc), torch.zeros_like(vc)
    assert q.kv_append(None, k, v, kc2, vc2, slots, pos, table) is None
    assert same(kc, kc2) and same(vc, vc2)
    assert q.kv_append(xq, k, v, kc2, vc2, slots, pos, table, out=xq) is xq and same(xq, want)


def test_append_e4m3_borders(q):
    """Saturation, ties to even, subnormals, zeros and NaN of the 8-bit store."""
    vals = torch.tensor([0.0, -0.0, 448.0, 449.0, 1e4, -1e4, 17.0, 19.0, 2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -9, -2.5 * 2.0 ** -9, 464.0,
                         float("inf"), -float("inf"), float("nan")], device=DEV)
    v = vals.repeat(1, 1, 4).half()
    kc, vc = (torch.zeros(1, 1, 1, 64, device=DEV).to(E4M3) for _ in range(2))
    one = torch.ones(1, device=DEV)
    q.kv_append(None, v, v, kc, vc, torch.zeros(1, dtype=torch.int64, device=DEV), k_scale=one, v_scale=one)
    want = v.float().clamp(-448, 448).to(E4M3)
    got = vc.float().flatten()
    assert torch.equal(got.nan_to_num(7777), want.float().flatten().nan_to_num(7777)) and same(kc, vc)


# --------------------------------------------------------------- attention --
class Paged:
    """Sequences (n new tokens, L keys) over a paged cache.  Whatever no row may see holds NaN."""

    def __init__(self, seqs, Hq, Hkv, D, page, dtype, e4m3=False, window=0, seed=0, one_tensor=False, spread=1.0):
        g = gen(seed)
        self.seqs, self.page, self.window, self.D, self.g = seqs, page, window, D, Hq // Hkv
        self.Hkv, self.dtype = Hkv, dtype
        T = sum(n for n, _ in seqs)
        fused = torch.randn(T, Hq + 2, D, generator=g, device=DEV).to(dtype)
        self.q = fused[:, :Hq]                                        # rows with a stride of their own
        cu = [0]
        for n, _ in seqs:
            cu.append(cu[-1] + n)
        self.cu_q = torch.tensor(cu, dtype=torch.int32, device=DEV)
        self.kv_lens = torch.tensor([L for _, L in seqs], dtype=torch.int32, device=DEV)
        self.max_q, self.max_kv = max([1] + [n for n, _ in seqs]), max([1] + [L for _, L in seqs])
        need = [-(-L // page) for _, L in seqs]
        width = max([1] + need) + 2
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=g, device=DEV).tolist()
        table = torch.full((len(seqs), width), -1, dtype=torch.int32)
        cdt = E4M3 if e4m3 else dtype
        self.k, self.v = [], []
        shape = (pages, 2, Hkv, page, D) if one_tensor else (2, pages, Hkv, page, D)
        store = torch.full(shape, float("nan"), device=DEV).to(cdt)
        kc, vc = (store[:, 0], store[:, 1]) if one_tensor else (store[0], store[1])
        size = 60.0 if e4m3 else 1.0
        at = 0
        for b, (n, L) in enumerate(seqs):
            k, v = ((torch.randn(L, Hkv, D, generator=g, device=DEV) * size * spread).to(cdt) for _ in range(2))
            first = max(0, L - n - window + 1) if window else 0       # the first key that any row sees
            for p in range(need[b]):
                lo, hi = max(first, p * page), min(L, (p + 1) * page)
                if lo >= hi:
                    continue                                          # a page that has left the window: its entry stays -1
                table[b, p] = order[at]
                for cache, x in ((kc, k), (vc, v)):
                    dst = cache[order[at]].view(torch.uint8) if e4m3 else cache[order[at]]
                    src = x.view(torch.uint8) if e4m3 else x
                    dst[:, lo - p * page:hi - p * page] = src[lo:hi].transpose(0, 1)
                at += 1
            self.k.append(k)
            self.v.append(v)
        self.kc, self.vc, self.table, self.pages = kc, vc, table.to(DEV), pages
        self.ks, self.vs = ((torch.rand(Hkv, generator=g, device=DEV) * 0.01 + 0.01) for _ in range(2)) if e4m3 else (None, None)
        self.scale = D ** -0.5

    def run(self, q, lse=True, **kw):
        out = torch.full((self.q.shape[0], self.q.shape[1], self.D), 7.0, device=DEV).to(self.dtype)
        ls = torch.full(self.q.shape[:2], 7.0, device=DEV) if lse else None
        q.paged_attention(self.q, self.kc, self.vc, self.table, self.cu_q, self.kv_lens, kw.pop("max_q", self.max_q), kw.pop("max_kv", self.max_kv),
                          scale=self.scale, window=self.window, k_scale=self.ks, v_scale=self.vs, out=out, lse=ls, **kw)
        return out, ls

    def check(self, out, lse, hidden=()):
        """hidden: (sequence, page index) whose keys no row sees."""
        u, t = U[self.dtype], 0
        for b, (n, L) in enumerate(self.seqs):
            if n == 0:
                continue
            qs = self.q[t:t + n].double().unflatten(1, (self.Hkv, self.g))
            got, gl = out[t:t + n].double().unflatten(1, (self.Hkv, self.g)), None if lse is None else lse[t:t + n].double().unflatten(1, (self.Hkv, self.g))
            t += n
            pos = torch.arange(L - n, L, device=DEV)[:, None]
            key = torch.arange(L, device=DEV)
            seen = key <= pos
            if self.window:
                seen = seen & (key > pos - self.window)
            for hb, p in hidden:
                if hb == b:
                    seen = seen & ~((key >= p * self.page) & (key < (p + 1) * self.page))
            for h in range(self.Hkv):
                k, v = self.k[b][:, h].double(), self.v[b][:, h].double()
                if self.ks is not None:
                    k, v = k * self.ks[h].double(), v * self.vs[h].double()
                qh = qs[:, h].reshape(n * self.g, self.D)
                mask = seen.repeat_interleave(self.g, 0)
                x = torch.where(mask, qh @ k.T * self.scale, -math.inf)
                l = torch.logsumexp(x, 1) if L else torch.full((n * self.g,), -math.inf, device=DEV, dtype=torch.float64)
                none = torch.isinf(l)
                p = torch.exp(x - torch.where(none, 0.0, l)[:, None])
                o, size = p @ v, p @ v.abs()
                # a score's error: D products summed in fp32, then a few fp32 roundings of it
                dx = ((self.D + 8) * 2.0 ** -24 * (qh.abs() @ k.abs().T) * self.scale).amax(1) if L else torch.zeros_like(l)
                rel = (2 * dx + (L + 64) * 2.0 ** -24 + 2.0 ** -20)[:, None]
                gh = got[:, h].reshape(n * self.g, self.D)
                close(gh, o, (u + rel) * size + u * o.abs() + 2.0 ** -24)
                assert (gh[none] == 0).all()
                if gl is not None:
                    lh = gl[:, h].reshape(-1)
                    assert (lh[none] == -math.inf).all()
                    if (~none).any():
                        close(lh[~none], l[~none], (rel[:, 0] + 2.0 ** -21 * l.abs())[~none])
        assert (out[t:] == 7).all()


SEQS = {
    "decode": [(1, 1), (1, 2), (1, 15), (1, 16), (1, 17), (1, 31), (1, 33), (1, 127), (1, 128), (1, 129), (1, 700), (1, 2049), (1, 0), (1, 5000)],
    "mixed": [(1, 300), (5, 5), (33, 100), (0, 40), (64, 64), (2, 1500), (3, 0), (7, 4), (130, 700)],
    "chunk": [(257, 1025), (100, 4000), (1, 4100)],
}


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("e4m3", [False, True], ids=["plain", "e4m3"])
@pytest.mark.parametrize("seqs", list(SEQS))
@pytest.mark.parametrize("Hq,Hkv,D,page", [(8, 2, 128, 16), (5, 5, 64, 1), (6, 2, 80, 32), (16, 1, 96, 7), (8, 1, 256, 64), (24, 1, 128, 256), (3, 1, 16, 48),
                                           (4, 4, 128, 1)])
def test_attention(q, dtype, e4m3, seqs, Hq, Hkv, D, page):
    c = Paged(SEQS[seqs], Hq, Hkv, D, page, dtype, e4m3, seed=D + page)
    c.check(*c.run(q))


@pytest.mark.parametrize("window", [1, 5, 16, 100, 1000])
@pytest.mark.parametrize("e4m3", [False, True], ids=["plain", "e4m3"])
@pytest.mark.parametrize("seqs,page", [("decode", 16), ("mixed", 16), ("mixed", 5), ("chunk", 64)])
def test_attention_window(q, seqs, page, window, e4m3):
    c = Paged(SEQS[seqs], 4, 2, 64 if page == 5 else 128, page, torch.float16, e4m3, window=window, seed=window)
    c.check(*c.run(q))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
def test_attention_long(q, dtype):
    """Many splits of the keys, one sequence beside very short ones."""
    c = Paged([(1, 70001), (1, 3), (2, 40000)], 8, 2, 128, 16, dtype, seed=4)
    c.check(*c.run(q))


@pytest.mark.parametrize("page", [16, 3])
def test_attention_sharp_rows(q, page):
    """Scores of several hundred: one key takes all, the running maximum moves often."""
    c = Paged([(1, 900), (40, 400)], 4, 2, 128, page, torch.float16, seed=11, spread=30.0)
    c.check(*c.run(q))


@pytest.mark.parametrize("page", [16, 6])
@pytest.mark.parametrize("n", [1, 70])
def test_attention_bad_pages(q, page, n):
    """A page id outside the cache hides its keys: nothing is read through it."""
    c = Paged([(n, 500), (1, 20)], 8, 2, 128, page, torch.float16, seed=2)
    hidden = [(0, 0), (0, 3), (0, 500 // page - 1), (1, 0), (1, 1), (1, 2), (1, 3)]
    for i, (b, p) in enumerate(hidden):
        if p * page < c.seqs[b][1]:
            c.table[b, p] = (-1, c.pages, 2 ** 31 - 1, -2 ** 31)[i % 4]
    c.check(*c.run(q), hidden=hidden)


def test_attention_layouts(q):
    """Both caches in one tensor, loose bounds, no lse, an output with strides."""
    c = Paged(SEQS["mixed"], 8, 2, 128, 16, torch.bfloat16, seed=3, one_tensor=True)
    out, lse = c.run(q)
    c.check(out, lse)
    loose, _ = c.run(q, max_q=4000, max_kv=100000, lse=False)
    c.check(loose, None)
    wide = torch.full((c.q.shape[0], 8, 3, 128), 7.0, device=DEV).to(torch.bfloat16)
    q.paged_attention(c.q, c.kc, c.vc, c.table, c.cu_q, c.kv_lens, c.max_q, c.max_kv, out=wide[:, :, 1])
    assert same(wide[:, :, 1], out) and (wide[:, :, 0] == 7).all() and (wide[:, :, 2] == 7).all()


def test_attention_nothing(q):
    c = Paged([(1, 0), (3, 0)], 4, 1, 64, 16, torch.float16)
    out, lse = c.run(q)
    assert (out == 0).all() and (lse == -math.inf).all()
    empty = q.paged_attention(c.q[:0], c.kc, c.vc, c.table, torch.zeros_like(c.cu_q), c.kv_lens, 1, 10)
    assert empty.shape == (0, 4, 64)


def test_attention_bad_offsets(q):
    """Offsets that do not fit q: the sequence is left out, the others are served."""
    c = Paged([(2, 30), (3, 40), (4, 50)], 4, 1, 64, 16, torch.float16, seed=8)
    good, _ = c.run(q)
    cu = c.cu_q.clone()
    c.cu_q[3] = 10 ** 6
    out, _ = c.run(q)
    assert same(out[:5], good[:5]) and (out[5:] == 7).all()
    c.cu_q = cu


@pytest.mark.parametrize("seqs", list(SEQS))
def test_attention_same_bits_and_streams(q, seqs):
    c = Paged(SEQS[seqs], 8, 2, 128, 16, torch.float16, seed=5)
    out, lse = c.run(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other, lse2 = c.run(q)
    torch.cuda.current_stream().wait_stream(side)
    assert same(out, other) and same(lse, lse2)


def test_far_pages(q):
    """Cache rows beyond 2^32 bytes: pages at the far end of one large tensor."""
    pages, Hkv, page, D = 530000, 2, 16, 128                  # 4.3 GB a cache
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    kc, vc = (torch.empty(pages, Hkv, page, D, dtype=torch.float16, device=DEV) for _ in range(2))
    g = gen(1)
    T = 40
    k, v, xq = (torch.randn(T, h, D, generator=g, device=DEV).half() for h in (Hkv, Hkv, 4))
    ids = torch.tensor([pages - 1, 3, pages - 2], device=DEV)
    t = torch.arange(T, device=DEV)
    slots = ids[t // page] * page + t % page
    q.kv_append(None, k, v, kc, vc, slots)
    assert same(kc[ids[t // page], :, t % page], k) and same(vc[ids[t // page], :, t % page], v)
    table = ids.to(torch.int32)[None].contiguous()
    args = (torch.tensor([0, T], dtype=torch.int32, device=DEV), torch.tensor([T], dtype=torch.int32, device=DEV), T, T)
    far = q.paged_attention(xq, kc, vc, table, *args)
    near = q.paged_attention(xq, kc[ids].contiguous(), vc[ids].contiguous(), torch.arange(3, device=DEV, dtype=torch.int32)[None].contiguous(), *args)
    assert same(far, near)


def test_layer_step_in_a_graph(q):
    """append, attention and two linear calls captured and replayed, with eager work between."""
    g = gen(12)
    Hq, Hkv, D, page, B = 8, 2, 64, 16, 5
    c = Paged([(1, L) for L in (1, 40, 700, 17, 3000)], Hq, Hkv, D, page, torch.float16, seed=6)
    c.kc.nan_to_num_(0.5)
    c.vc.nan_to_num_(0.5)
    K = Hq * D
    wq, s, z = weights(K, K, 4, 64, True, g)
    x = torch.randn(B, (Hq + 2 * Hkv) * D, generator=g, device=DEV).half()
    res = torch.randn(B, K, generator=g, device=DEV).half()
    table = rope_table(4000, D)
    positions = (c.kv_lens - 1).contiguous()
    slots = torch.stack([c.table[b, (L - 1) // page].long() * page + (L - 1) % page for b, (_, L) in enumerate(c.seqs)])

    def step():
        xq, k, v = (t.unflatten(1, (-1, D)) for t in x.split((Hq * D, Hkv * D, Hkv * D), 1))
        t = q.kv_append(xq, k, v, c.kc, c.vc, slots, positions, table)
        o = q.paged_attention(t, c.kc, c.vc, c.table, c.cu_q, c.kv_lens, 1, 3000)
        h = q.linear(o.flatten(1), wq, s, z, 4, 64, residual=res)
        return q.linear(h, wq, s, z, 4, 64, act="silu", mul=h)

    eager = step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        x.copy_(torch.randn(x.shape, generator=g, device=DEV))
        want = step()
        torch.cuda.synchronize()
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, want), i
    assert not same(want, eager)


def test_decoder_layer_example(q):
    """Prompts and graph-replayed decode steps through the paged cache against the layer in fp32.  The
    fp16 roundings on the way (projections, q, k, v, probabilities, outputs) are some ten of 2^-11
    in a row, and weights rounded once; their root sum of squares stays below 2^-8."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_layer.py")
    spec = importlib.util.spec_from_file_location("decoder_layer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    for users, prompt, steps, page in ((3, 75, 6, 16), (1, 1, 3, 1), (5, 300, 2, 64)):
        _, error = example.run(hidden=512, heads=8, kv_heads=2, head_dim=64, inner=1024, users=users, prompt=prompt, steps=steps, page=page)
        assert error < 2.0 ** -8


# -------------------------------------------------------------- refusals --
def test_refusals_on_the_gpu(q):
    """Shapes, types and devices that do not fit, named in the error; nothing is written."""
    c = Paged([(1, 20)], 4, 2, 64, 16, torch.float16)
    out = torch.full((1, 4, 64), 7.0, device=DEV).half()
    ok = dict(q=c.q, k_cache=c.kc, v_cache=c.vc, page_table=c.table, cu_q=c.cu_q, kv_lens=c.kv_lens, max_q=1, max_kv=20, out=out)
    bad = [(dict(q=c.q[:, :3]), ValueError), (dict(q=c.q.float()), TypeError), (dict(k_cache=c.kc[..., :32]), ValueError), (dict(v_cache=c.vc[1:]), ValueError),
           (dict(k_cache=c.kc.transpose(2, 3)), ValueError), (dict(page_table=c.table.long()), TypeError), (dict(cu_q=c.cu_q[:1]), ValueError),
           (dict(kv_lens=c.kv_lens.cpu()), ValueError), (dict(out=out[:, :2]), ValueError), (dict(out=out.to(torch.bfloat16)), TypeError),
           (dict(lse=torch.zeros(1, 3, device=DEV)), ValueError), (dict(k_scale=torch.ones(2, device=DEV)), ValueError), (dict(max_q=0), q.QmmError),
           (dict(window=-1), q.QmmError), (dict(scale=-1.0), q.QmmError), (dict(scale=math.nan), q.QmmError), (dict(max_q=1.5), TypeError),
           (dict(k_cache=c.kc.to(E4M3), v_cache=c.vc.to(E4M3)), ValueError)]
    for change, kind in bad:
        with pytest.raises(kind):
            q.paged_attention(**{**ok, **change})
    k, v = (torch.zeros(1, 2, 64, device=DEV).half() for _ in range(2))
    slots, pos, table = torch.zeros(1, dtype=torch.int64, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV), rope_table(4, 64)
    before = c.kc.clone()
    ok = dict(q=c.q, k=k, v=v, k_cache=c.kc, v_cache=c.vc, slots=slots, positions=pos, rope=table, out=out)
    bad = [(dict(k=k[:, :1]), ValueError), (dict(v=v[..., :32]), ValueError), (dict(slots=slots.int()), TypeError), (dict(positions=None), ValueError),
           (dict(rope=None), ValueError), (dict(rope=table.half()), TypeError), (dict(rope=table[:, ::2]), ValueError), (dict(q=None), ValueError),
           (dict(rope=rope_table(4, 66)), q.QmmError), (dict(k=k.transpose(1, 2)), ValueError), (dict(k_cache=c.kc[:, :1]), ValueError)]
    for change, kind in bad:
        with pytest.raises(kind):
            q.kv_append(**{**ok, **change})
    assert (out == 7).all() and same(c.kc, before)
    X = torch.zeros(2, 64, device=DEV).half()
    wq, s, z = weights(64, 10, 4, 32, True, gen(1))
    y = torch.full((2, 10), 7.0, device=DEV).half()
    ok = dict(X=X, wq=wq, s=s, z=z, bits=4, G=32, out=y)
    bad = [(dict(X=X[0]), ValueError), (dict(X=X.float()), TypeError), (dict(X=torch.zeros(64, 2, device=DEV).half().t()), ValueError), (dict(wq=wq[:9]), ValueError),
           (dict(bits=5), ValueError), (dict(bits=9), ValueError), (dict(G=64), ValueError), (dict(s=s.float()), TypeError), (dict(z=z[:, :1]), ValueError),
           (dict(bias=torch.zeros(9, device=DEV).half()), ValueError), (dict(mul=y[:1]), ValueError), (dict(residual=y.float()), TypeError),
           (dict(act="swish"), ValueError), (dict(out=y.t()), ValueError), (dict(bias=torch.zeros(10).half()), ValueError)]
    for change, kind in bad:
        with pytest.raises(kind):
            q.linear(**{**ok, **change})
    torch.cuda.synchronize()
    assert (y == 7).all()
