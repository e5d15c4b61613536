"""Norms of queries and keys, and the cache of 4-bit codes (qmm_qk_norm, qmm_kv4_append, qmm_kv4_read,
qmm_kv4_attention), against their formulas in 64 bits, on an MI355X.

Tolerances count roundings.  u is half a step of the output's type (2^-11 for fp16, 2^-8 for bf16); fp32
sums of n terms are off by at most n 2^-24 of the sum of magnitudes.  Codes, scales and zero-points are
exact: what fp32 leaves in doubt the kernel decides in fp64 (a value within 2^-40 of a border would be another matter; none of the
inputs is, exact ties apart).
"""
import importlib.util
import math
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16 = torch.float16, torch.bfloat16
U = {F16: 2.0 ** -11, BF16: 2.0 ** -8}
TOP = 57344.0


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


def rope_table(rows, rot):
    angle = torch.arange(rows, device=DEV, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(rot // 2, device=DEV, dtype=torch.float64) * 2 / max(rot, 1))
    return torch.cat((angle.cos(), angle.sin()), 1).float()


# ------------------------------------------------------------ the formulas --
def turned(x, weight, eps, positions, table, pairs):
    """(y, |terms| of y) in 64 bits."""
    x, D = x.double(), x.shape[-1]
    if weight is not None:
        x = x * weight.double() / torch.sqrt(x.square().sum(-1, keepdim=True) / D + eps)
    size = x.abs()
    if table is not None:
        x, size, rot = x.clone(), size.clone(), table.shape[1]
        line = table[positions.long().clamp(0, table.shape[0] - 1)].double()[:, None]
        c, s = line[..., :rot // 2], line[..., rot // 2:]
        lane = torch.arange(rot // 2, device=DEV)
        one, two = (2 * lane, 2 * lane + 1) if pairs else (lane, lane + rot // 2)
        a, b = x[..., one], x[..., two]
        x[..., one], x[..., two] = a * c - b * s, b * c + a * s
        size[..., one], size[..., two] = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    return x, size


def encoded(x, G):
    """[..., D] in 64 bits -> codes [..., D], s and z [..., D / G], by the formulas; a group with NaN has s NaN."""
    x = x.clamp(-TOP, TOP).unflatten(-1, (-1, G))
    bad = x.isnan().any(-1)
    clean = torch.where(bad[..., None], 0.0, x)
    lo, hi = clean.amin(-1).clamp(max=0), clean.amax(-1).clamp(min=0)
    r = ((hi - lo) / 15).clamp(min=2.0 ** -20)
    m, _ = torch.frexp(r)
    step = r / m / 128                                     # (r / m is a power of two)
    # ties of the range against 15 times a middle, exactly: 15 (n + 1/2) step has few bits
    n = torch.floor(r / step)
    rest = (hi - lo) - 15 * (n + 0.5) * step
    n = torch.where(rest > 0, n + 1, torch.where(rest < 0, n, n + n.remainder(2)))
    s = (n * step).clamp(min=2.0 ** -18)
    z = torch.round(-lo / s).clamp(0, 15)
    codes = (torch.round(clean / s[..., None]) + z[..., None]).clamp(0, 15)
    codes[bad] = 0
    return codes.flatten(-2).long(), torch.where(bad, math.nan, s), torch.where(bad, 0.0, z)


def unpacked(codes):
    return torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()


def decoded(codes, scale):
    """uint8 [..., D / 2], fp16 [..., D / G, 2] -> [..., D] in 64 bits."""
    x = unpacked(codes).double().unflatten(-1, (scale.shape[-2], -1))
    return ((x - scale[..., 1:].double()) * scale[..., :1].double()).flatten(-2)


def same_numbers(a, b):
    return torch.equal(a.double().nan_to_num(12345.0), b.double().nan_to_num(12345.0))


# -------------------------------------------------------------------- norms --
def heads(T, Hq, Hkv, D, dtype, g, layout="fused", size=1.0):
    if layout == "fused":
        x = (torch.randn(T, Hq + 2 * Hkv, D, generator=g, device=DEV) * size).to(dtype)
    elif layout == "odd":          # rows at odd places, with a stride of their own
        x = (torch.randn(T, (Hq + 2 * Hkv) * (D + 3) + 1, generator=g, device=DEV) * size).to(dtype)[:, 1:].unflatten(1, (-1, D + 3))[..., :D]
    return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]


def norm_bound(y, size, D, dtype):
    """A sum of D squares, its root and quotient, the products: fp32 roundings; then one to dtype."""
    return y.abs() * U[dtype] + (D + 24) * 2.0 ** -24 * size + 2.0 ** -25


NORMS = [(1, 32, 8, 128, 128), (1, 1, 1, 16, 16), (7, 3, 1, 80, 80), (65, 5, 2, 96, 48), (33, 8, 8, 64, 32), (130, 2, 1, 256, 256), (300, 12, 4, 128, 64),
         (19, 4, 2, 192, 0), (1000, 3, 3, 176, 160)]


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("pairs", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("layout", ["fused", "odd"])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot", NORMS)
def test_qk_norm(q, T, Hq, Hkv, D, rot, layout, pairs, dtype):
    g = gen(T + D)
    xq, xk, _ = heads(T, Hq, Hkv, D, dtype, g, layout)
    wq, wk = ((1 + 0.3 * torch.randn(D, generator=g, device=DEV)).to(dtype) for _ in range(2))
    table = rope_table(2000, rot) if rot else None
    pos = torch.randint(-5, 2010, (T,), generator=g, device=DEV, dtype=torch.int32) if rot else None
    for a, b in ((wq, wk), (None, wk), (wq, None), (None, None)):
        yq, yk = q.qk_norm(xq, xk, a, b, 1e-5, pos, table, pairs)
        for x, w, y in ((xq, a, yq), (xk, b, yk)):
            want, size = turned(x, w, 1e-5, pos, table, pairs)
            close(y, want, norm_bound(want, size, D, dtype))


def test_qk_norm_in_place_and_into_strides(q):
    g = gen(3)
    xq, xk, _ = heads(50, 6, 2, 128, F16, g)
    w, table, pos = torch.rand(128, generator=g, device=DEV).half(), rope_table(60, 128), torch.arange(50, device=DEV, dtype=torch.int32)
    yq, yk = q.qk_norm(xq, xk, w, w, 1e-6, pos, table)
    wide = torch.full((50, 8, 3, 128), 7.0, device=DEV).half()
    oq, ok = q.qk_norm(xq, xk, w, w, 1e-6, pos, table, q_out=wide[:, :6, 1], k_out=wide[:, 6:, 1])
    assert same(oq, yq) and same(ok, yk) and (wide[:, :, ::2] == 7).all()
    third = torch.full((50, 8, 131), 7.0, device=DEV).half()            # odd places: element by element
    q.qk_norm(xq, xk, w, w, 1e-6, pos, table, q_out=third[:, :6, 1:129], k_out=third[:, 6:, 1:129])
    assert same(third[:, :6, 1:129], yq) and same(third[:, 6:, 1:129], yk) and (third[..., 0] == 7).all() and (third[..., 129:] == 7).all()
    a, b = q.qk_norm(xq, xk, w, w, 1e-6, pos, table, q_out=xq, k_out=xk)
    assert a is xq and b is xk and same(xq, yq) and same(xk, yk)


def test_qk_norm_of_nothing_zeros_and_nan(q):
    x = torch.zeros(0, 4, 64, device=DEV).half()
    assert q.qk_norm(x, x)[0].shape == (0, 4, 64)
    x = torch.randn(3, 4, 64, device=DEV).half()
    none = torch.zeros(3, 0, 64, device=DEV).half()
    w = torch.ones(64, device=DEV).half()
    yq, yk = q.qk_norm(x, none, w, w)
    assert yk.shape == (3, 0, 64) and same(yq, q.qk_norm(none, x, None, w)[1])
    x[0], x[1, 1, 5] = 0, math.nan
    y, _ = q.qk_norm(x, none, w, eps=1e-6)
    assert (y[0] == 0).all() and y[1, 1].isnan().all() and torch.isfinite(y[1, 0]).all() and torch.isfinite(y[2]).all()


# ------------------------------------------------------------------- append --
def place(T, pages, page, g, pad=0):
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:T].long()
    if pad:
        slots[T - pad:] = torch.tensor([-1, pages * page, 2 ** 62, -2 ** 62], device=DEV).repeat(pad)[:pad]
    return slots


def filled(q, pages, Hkv, page, D, G, g):
    c = q.kv4_cache(pages, Hkv, page, D, G, DEV)
    for t in c[:2]:
        t.copy_(torch.randint(0, 256, t.shape, generator=g, device=DEV, dtype=torch.uint8))
    for t in c[2:]:
        t.copy_(torch.randn(t.shape, generator=g, device=DEV))
    return c


def check_stored(c, before, k, v, slots, G):
    """The cache holds the codes of k and v [T, Hkv, D] (64 bits) at their slots, and elsewhere what it held."""
    pages, _, page, _ = c.k.shape
    live = (slots >= 0) & (slots < pages * page)
    at, within = slots[live] // page, slots[live] % page
    untouched = torch.ones(pages, page, dtype=torch.bool, device=DEV)
    untouched[at, within] = False
    for codes, scale, old_codes, old_scale, x in ((c.k, c.k_scale, before.k, before.k_scale, k), (c.v, c.v_scale, before.v, before.v_scale, v)):
        want, s, z = encoded(x[live], G)
        assert torch.equal(unpacked(codes[at, :, within]), want)
        got = scale[at, :, within]
        assert same_numbers(got[..., 0], s) and same_numbers(got[..., 1], z)
        keep = untouched[:, None, :, None].expand(codes.shape)
        assert torch.equal(codes[keep], old_codes[keep])
        keep = untouched[:, None, :, None, None].expand(scale.shape)
        assert torch.equal(scale.view(torch.int16)[keep], old_scale.view(torch.int16)[keep])


APPENDS = [(1, 4, 2, 128, 128, 128, 16), (77, 5, 5, 128, 64, 64, 16), (33, 8, 1, 96, 32, 96, 1), (50, 3, 1, 192, 64, 96, 7), (19, 2, 2, 64, 32, 16, 32),
           (65, 2, 1, 256, 128, 256, 256), (130, 1, 1, 32, 32, 32, 3), (700, 16, 4, 64, 64, 64, 64), (40, 4, 2, 224, 32, 32, 100), (12, 1, 3, 256, 32, 0, 16)]


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("norm", [False, True], ids=["plain", "norm"])
@pytest.mark.parametrize("pairs", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("T,Hq,Hkv,D,G,rot,page", APPENDS)
def test_append(q, T, Hq, Hkv, D, G, rot, page, pairs, norm, dtype):
    for layout in ("fused", "odd"):
        g = gen(T + D + G)
        xq, k, v = heads(T, Hq, Hkv, D, dtype, g, layout)
        pages = -(-T // page) + 2
        c = filled(q, pages, Hkv, page, D, G, g)
        before = q.KV4Cache(*(t.clone() for t in c))
        slots = place(T, pages, page, g, pad=min(T // 8, 5))
        table = rope_table(2000, rot) if rot else None
        pos = torch.randint(-5, 2010, (T,), generator=g, device=DEV, dtype=torch.int32) if rot else None
        wq, wk = ((1 + 0.3 * torch.randn(D, generator=g, device=DEV)).to(dtype) for _ in range(2)) if norm else (None, None)
        out = q.kv4_append(xq, k, v, c, slots, pos, table, pairs, wq, wk, 1e-5)
        want, size = turned(xq, wq, 1e-5, pos, table, pairs)
        close(out, want, norm_bound(want, size, D, dtype))
        check_stored(c, before, turned(k, wk, 1e-5, pos, table, pairs)[0], v.double(), slots, G)


@pytest.mark.parametrize("pairs", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("size,eps,turn", [(1e20, 1e-5, 1), (3e37, 1e-5, 1), (1e-25, 0.0, 1), (1e-37, 0.0, 1), (1.0, 1e-5, 300), (2e-3, 0.0, 1e-3), (1e18, 1e-5, 50)])
def test_append_keys_of_any_size(q, size, eps, turn, pairs):
    """Squares beyond fp32's range, tables beyond 1: the codes are the formulas' all the same."""
    g = gen(41)
    _, k, v = heads(40, 0, 3, 128, BF16, g, size=size)
    k[0, 0] = 0
    v = torch.zeros_like(v)
    w, table, pos = (1 + 0.3 * torch.randn(128, generator=g, device=DEV)).to(BF16), rope_table(100, 128) * turn, torch.arange(40, device=DEV, dtype=torch.int32)
    c = q.kv4_cache(6, 3, 16, 128, 64)
    before, slots = q.KV4Cache(*(t.clone() for t in c)), place(40, 6, 16, g)
    q.kv4_append(None, k, v, c, slots, pos, table, pairs, k_norm=w, eps=eps)
    want = turned(k, w, eps, pos, table, pairs)[0]
    assert eps == 0 or torch.isfinite(want).all()
    check_stored(c, before, want, v.double(), slots, 64)


def test_append_in_place_and_keys_alone(q):
    g = gen(9)
    xq, k, v = heads(20, 6, 2, 64, F16, g)
    table, pos, slots = rope_table(100, 64), torch.arange(20, device=DEV, dtype=torch.int32) + 50, torch.arange(20, device=DEV)
    w = torch.rand(64, generator=g, device=DEV).half()
    c, c2 = (q.kv4_cache(2, 2, 16, 64, 32) for _ in range(2))
    want = q.kv4_append(xq, k, v, c, slots, pos, table, q_norm=w, k_norm=w)
    assert q.kv4_append(None, k, v, c2, slots, pos, table, k_norm=w) is None
    assert all(same(a, b) for a, b in zip(c, c2))
    assert q.kv4_append(xq, k, v, tuple(c2), slots, pos, table, q_norm=w, k_norm=w, out=xq) is xq and same(xq, want)
    y, _ = q.qk_norm(*heads(20, 6, 2, 64, F16, gen(9))[:2], w, w, 1e-6, pos, table)
    assert same(y, want)


def test_append_nothing(q):
    c = q.kv4_cache(2, 2, 16, 64)
    x = torch.zeros(0, 2, 64, device=DEV).half()
    assert q.kv4_append(x, x, x, c, torch.zeros(0, dtype=torch.int64, device=DEV)).shape == (0, 2, 64)


def groups_of(dtype, G):
    """Rows of G values on the borders of the mapping."""
    tie = torch.arange(G, dtype=torch.float64)
    rows = [torch.zeros(G, dtype=torch.float64), torch.full((G,), 3.0, dtype=torch.float64), torch.full((G,), -3.0, dtype=torch.float64),
            (tie % 31) / 2,                                # s = 1: halves, up and down to the even code
            (tie % 31) / 2 - 7.5,                          # z = 8 (7.5 to the even one)
            (tie % 31) / 2 - 6.5,                          # z = 6
            torch.where(tie == 0, 65504.0, tie), torch.where(tie == 0, -65504.0, 65504.0), torch.where(tie == 0, math.inf, 1.0), torch.where(tie == 0, -math.inf, tie),
            torch.where(tie == 1, math.nan, tie), torch.where(tie == 0, 2.0 ** -24, 0.0), torch.where(tie == 0, -2.0 ** -20, 2.0 ** -21),
            torch.where(tie == 0, 15.0 * 2.0 ** -18, 0.0), torch.where(tie == 0, 15.0 * 2.0 ** -14, -2.0 ** -14),
            torch.where(tie == 0, -0.0, 0.0)]
    for n in (129, 131, 133, 255, 253):                   # (hi - lo) / 15 halfway between two scales of 7 bits
        if 15 * n < 2 ** 11 or dtype == F16 and 15 * n < 2 ** 11:
            rows.append(torch.where(tie == 0, 15.0 * n / 128, 0.25))
        rows.append(torch.where(tie == 0, 8.0 * n / 128, torch.where(tie == 1, -7.0 * n / 128, 0.0)))     # the range is exact where hi and lo are
    return torch.stack(rows).to(dtype).to(DEV)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("G", [32, 64, 128])
def test_append_borders(q, dtype, G):
    """Ties, saturation, zeros, subnormals and NaN: exact codes; no infinity and no rounding in what they stand for."""
    x = groups_of(dtype, G)
    if dtype == BF16:
        x = torch.cat((x, torch.full((1, G), 3e38, device=DEV).to(dtype), torch.full((1, G), 1e-38, device=DEV).to(dtype)))
    x = torch.cat((x, x.flip(0)), 1)[:, None]                       # two groups a row
    T, D = x.shape[0], 2 * G
    c = q.kv4_cache(1, 1, T, D, G)
    before = q.KV4Cache(*(t.clone() for t in c))
    slots = torch.arange(T, device=DEV)
    q.kv4_append(None, x, x, c, slots)
    check_stored(c, before, x.double(), x.double(), slots, G)
    k, v = q.kv4_read(c, slots)
    values = decoded(c.k[0].transpose(0, 1), c.k_scale[0].transpose(0, 1))
    assert same(k, v) and same_numbers(k, values)                   # fp16 holds them exactly
    bad = x.isnan().unflatten(-1, (2, G)).any(-1, keepdim=True).expand(T, 1, 2, G).flatten(-2)
    assert values[bad].isnan().all() and torch.isfinite(values[~bad]).all()
    # within half a step, or what the shorter scale leaves of 15 of them at the upper end: 15 (2^-7) / 2 steps more
    s = c.k_scale[0, 0, :, :, 0].double().repeat_interleave(G, 1)[:, None]
    off = (values - x.double().clamp(-TOP, TOP)).abs()
    assert (off <= s * (1 + 15 * 2.0 ** -7) / 2 + 2.0 ** -19)[~bad].all()


def test_append_every_scale_is_short(q):
    """Ranges over all of fp16: 7 significant bits, and each of 16 values a number of fp16."""
    g = gen(5)
    T = 4096
    x = torch.randn(T, 1, 128, generator=g, device=DEV) * 2.0 ** torch.randint(-16, 15, (T, 1, 1), generator=g, device=DEV)
    x = x.clamp(-65504, 65504).half()
    c = q.kv4_cache(T // 64, 1, 64, 128, 32)
    before = q.KV4Cache(*(t.clone() for t in c))
    slots = torch.arange(T, device=DEV)
    q.kv4_append(None, x, x, c, slots)
    check_stored(c, before, x.double(), x.double(), slots, 32)
    s = c.k_scale[..., 0].double()
    m, _ = torch.frexp(s)
    assert torch.equal(torch.round(m * 128), m * 128)
    level = torch.arange(-15, 16, device=DEV).double() * s[..., None]
    fine = level.abs() <= 65504
    assert torch.equal(level.half().double()[fine], level[fine])


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
def test_read(q, dtype):
    for T, Hkv, D, G, page in ((1, 1, 32, 32, 16), (100, 3, 96, 32, 7), (333, 2, 256, 64, 64), (5000, 8, 128, 128, 16)):
        g = gen(T)
        pages = -(-T // page) + 1
        c = filled(q, pages, Hkv, page, D, G, g)
        slots = place(T, pages, page, g, pad=min(T // 4, 9))
        slots[: T // 3] = slots[T // 3: 2 * (T // 3)].flip(0)        # the same slot twice
        live = (slots >= 0) & (slots < pages * page)
        at, within = torch.where(live, slots // page, 0), torch.where(live, slots % page, 0)
        out = q.kv4_read(c, slots, dtype)
        odd = torch.full((2, T, Hkv, D + 3), 7.0, device=DEV).to(dtype)
        q.kv4_read(c, slots, dtype, k_out=odd[0, :, :, 1:D + 1], v_out=odd[1, :, :, 1:D + 1])
        assert (odd[..., 0] == 7).all() and (odd[..., D + 1:] == 7).all()
        for y, o, codes, scale in ((out[0], odd[0], c.k, c.k_scale), (out[1], odd[1], c.v, c.v_scale)):
            want = decoded(codes[at, :, within], scale[at, :, within])
            want = torch.where(live[:, None, None], want, 0.0)
            # filled() has scales and zero-points of 11 bits: c - z rounds once in fp32, the product once, then to dtype
            close(y, want, want.abs() * (U[dtype] + 2.0 ** -22) + 2.0 ** -24)
            assert same(o[..., 1:D + 1], y)
    assert q.kv4_read(c, slots[:0])[0].shape == (0, 8, 128)


# ---------------------------------------------------------------- attention --
class Paged:
    """Sequences (n new tokens, L keys) over a paged cache of codes.  Whatever no row may see has scales of NaN."""

    def __init__(self, q, seqs, Hq, Hkv, D, G, page, dtype, window=0, sinks=0, seed=0, one_tensor=False, spread=1.0, q_size=1.0):
        g = gen(seed)
        self.seqs, self.page, self.window, self.sinks, self.D, self.g = seqs, page, window, sinks if window else 0, D, Hq // Hkv
        self.Hkv, self.dtype = Hkv, dtype
        T = sum(n for n, _ in seqs)
        fused = (torch.randn(T, Hq + 2, D, generator=g, device=DEV) * q_size).to(dtype)
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
        if one_tensor:      # k and v of a page side by side
            codes = torch.randint(0, 256, (pages, 2, Hkv, page, D // 2), generator=g, device=DEV, dtype=torch.uint8)
            scale = torch.full((pages, 2, Hkv, page, D // G, 2), math.nan, device=DEV, dtype=F16)
            cache = q.KV4Cache(codes[:, 0], codes[:, 1], scale[:, 0], scale[:, 1])
        else:
            cache = q.kv4_cache(pages, Hkv, page, D, G, DEV)
            for t in cache[:2]:
                t.copy_(torch.randint(0, 256, t.shape, generator=g, device=DEV, dtype=torch.uint8))
            for t in cache[2:]:
                t.fill_(math.nan)
        self.k, self.v = [], []
        at = 0
        for b, (n, L) in enumerate(seqs):
            first = max(0, L - n - window + 1) if window else 0       # the first key that any row sees, but for the sinks
            sides = []
            for _ in range(2):
                codes, s, z = encoded(torch.randn(L, Hkv, D, generator=g, device=DEV).double() * spread, G)
                packed = (codes[..., 0::2] | codes[..., 1::2] << 4).to(torch.uint8)
                sz = torch.stack((s, z), -1).half()
                sides.append((packed, sz))
            for p in range(need[b]):
                lo, hi = p * page, min(L, (p + 1) * page)
                key = torch.arange(lo, hi, device=DEV)
                want = (key >= first) | (key < self.sinks)
                if not bool(want.any()):
                    continue                                          # a page that no row sees: its entry stays -1
                table[b, p] = order[at]
                for codes, scale, (packed, sz) in ((cache.k, cache.k_scale, sides[0]), (cache.v, cache.v_scale, sides[1])):
                    codes[order[at], :, :hi - lo] = packed[lo:hi].transpose(0, 1)
                    scale[order[at], :, :hi - lo] = torch.where(want[None, :, None, None], sz[lo:hi].transpose(0, 1), math.nan)
                at += 1
            self.k.append(decoded(*sides[0]))
            self.v.append(decoded(*sides[1]))
        self.cache, self.table, self.pages = cache, table.to(DEV), pages
        self.scale = D ** -0.5

    def run(self, q, lse=True, **kw):
        out = torch.full((self.q.shape[0], self.q.shape[1], self.D), 7.0, device=DEV).to(self.dtype)
        ls = torch.full(self.q.shape[:2], 7.0, device=DEV) if lse else None
        q.kv4_attention(self.q, self.cache, self.table, self.cu_q, self.kv_lens, kw.pop("max_q", self.max_q), kw.pop("max_kv", self.max_kv), scale=self.scale,
                        window=self.window, sinks=self.sinks, out=out, lse=ls, **kw)
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
                seen = seen & ((key > pos - self.window) | (key < self.sinks))
            for hb, p in hidden:
                if hb == b:
                    seen = seen & ~((key >= p * self.page) & (key < (p + 1) * self.page))
            for h in range(self.Hkv):
                k, v = self.k[b][:, h], self.v[b][:, h]
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
                # probabilities rounded to fp16: half a step, or 2^-36 of the row's largest
                tiny = 2.0 ** -36 * (mask.double() @ v.abs()) * p.amax(1, keepdim=True) if L else 0.0
                close(gh, o, (U[F16] + rel) * size + tiny + u * o.abs() + 2.0 ** -24)
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
    "few": [(2, 2), (3, 70), (4, 1000), (1, 513)],
}


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("seqs", list(SEQS))
@pytest.mark.parametrize("Hq,Hkv,D,G,page", [(8, 2, 128, 128, 16), (5, 5, 64, 64, 1), (6, 2, 96, 32, 32), (16, 1, 32, 32, 7), (8, 1, 256, 64, 64), (24, 1, 128, 32, 256),
                                             (3, 1, 192, 64, 48), (4, 4, 128, 64, 1), (8, 2, 64, 32, 16), (4, 2, 256, 128, 5), (2, 2, 224, 32, 16),
                                             (8, 1, 128, 128, 7), (9, 3, 64, 32, 2), (16, 2, 128, 64, 16), (24, 1, 128, 64, 3), (32, 1, 128, 128, 5), (20, 1, 64, 64, 16)])
def test_attention(q, dtype, seqs, Hq, Hkv, D, G, page):
    c = Paged(q, SEQS[seqs], Hq, Hkv, D, G, page, dtype, seed=D + page)
    c.check(*c.run(q))


@pytest.mark.parametrize("window", [1, 5, 16, 100, 1000])
@pytest.mark.parametrize("sinks", [0, 1, 4, 17, 200, 2 ** 40])
@pytest.mark.parametrize("seqs,page", [("decode", 16), ("mixed", 16), ("mixed", 5), ("chunk", 64), ("few", 100)])
def test_attention_window_and_sinks(q, seqs, page, window, sinks):
    D, G = (64, 32) if page == 5 else (128, 64)
    c = Paged(q, SEQS[seqs], 4, 2, D, G, page, F16, window=window, sinks=sinks, seed=window + sinks % 97)
    c.check(*c.run(q))


def test_attention_window_beyond_the_numbers(q):
    """No window, and one that no sequence reaches, are the same; sinks without a window say nothing."""
    c = Paged(q, SEQS["mixed"], 4, 2, 128, 64, 16, F16, seed=1)
    want, lse = c.run(q)
    c.check(want, lse)
    for window, sinks in ((2 ** 62, 0), (2 ** 62, 4), (0, 100), (5000, 7)):
        c.window, c.sinks = window, sinks
        got, l2 = c.run(q)
        assert same(got, want) and same(lse, l2)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (30000, 100)])
def test_attention_long(q, dtype, window, sinks):
    """Many splits of the keys, one sequence beside very short ones."""
    c = Paged(q, [(1, 70001), (1, 3), (2, 40000)], 8, 2, 128, 128, 16, dtype, window=window, sinks=sinks, seed=4)
    c.check(*c.run(q))


@pytest.mark.parametrize("page", [16, 3])
def test_attention_sharp_rows(q, page):
    """Scores of several hundred: one key takes all, the running maximum moves often."""
    c = Paged(q, [(1, 900), (40, 400)], 4, 2, 128, 64, page, F16, seed=11, spread=30.0)
    c.check(*c.run(q))


@pytest.mark.parametrize("q_size", [1e-30, 1e-4, 3e4, 1e20])
def test_attention_bf16_rows_of_any_size(q, q_size):
    """Rows of q far outside fp16: brought there by their own power of two."""
    c = Paged(q, [(1, 300), (50, 80)], 4, 2, 64, 32, 16, BF16, seed=12, q_size=q_size)
    c.scale = 0.125 / q_size
    c.check(*c.run(q))


def test_attention_large_values(q):
    """Values of the cache's largest size stay finite."""
    c = Paged(q, [(1, 100), (40, 90)], 4, 2, 64, 64, 16, BF16, seed=13, spread=20000.0)
    c.scale = 1e-5
    c.check(*c.run(q))


@pytest.mark.parametrize("page", [16, 6])
@pytest.mark.parametrize("n", [1, 70])
@pytest.mark.parametrize("window,sinks", [(0, 0), (200, 33)])
def test_attention_bad_pages(q, page, n, window, sinks):
    """A page id outside the cache hides its keys: nothing is read through it."""
    c = Paged(q, [(n, 500), (1, 20)], 8, 2, 128, 64, page, F16, window=window, sinks=sinks, seed=2)
    hidden = [(0, 0), (0, 3), (0, 500 // page - 1), (1, 0), (1, 1), (1, 2), (1, 3)]
    for i, (b, p) in enumerate(hidden):
        if p * page < c.seqs[b][1]:
            c.table[b, p] = (-1, c.pages, 2 ** 31 - 1, -2 ** 31)[i % 4]
    c.check(*c.run(q), hidden=hidden)


def test_attention_layouts(q):
    """Both caches in one tensor, loose bounds, no lse, an output with strides."""
    c = Paged(q, SEQS["mixed"], 8, 2, 128, 64, 16, BF16, seed=3, one_tensor=True)
    out, lse = c.run(q)
    c.check(out, lse)
    loose, _ = c.run(q, max_q=4000, max_kv=100000, lse=False)
    c.check(loose, None)
    wide = torch.full((c.q.shape[0], 8, 3, 128), 7.0, device=DEV).to(BF16)
    q.kv4_attention(c.q, tuple(c.cache), c.table, c.cu_q, c.kv_lens, c.max_q, c.max_kv, out=wide[:, :, 1])
    assert same(wide[:, :, 1], out) and (wide[:, :, 0] == 7).all() and (wide[:, :, 2] == 7).all()


def test_strides_of_single_sizes_say_nothing(q):
    """One page, one head, pages of one token: torch leaves any stride there."""
    for pages, heads_, page in ((20, 3, 1), (20, 1, 16), (1, 3, 16), (1, 1, 1)):
        g = gen(pages + heads_)
        T = min(pages * page, 20)
        _, k, v = heads(T, 0, heads_, 64, F16, g)
        slots = place(T, pages, page, g)
        a, b = (q.kv4_cache(pages, heads_, page, 64, 32) for _ in range(2))
        odd = q.KV4Cache(*(t.as_strided(t.shape, [7 if n == 1 else s for n, s in zip(t.shape[:3], t.stride()[:3])] + list(t.stride()[3:])) for t in b))
        q.kv4_append(None, k, v, a, slots)
        q.kv4_append(None, k, v, odd, slots)
        assert all(same(x, y) for x, y in zip(a, b))
        assert all(same(x, y) for x, y in zip(q.kv4_read(a, slots), q.kv4_read(odd, slots)))
        table, cu, lens = torch.arange(pages, device=DEV, dtype=torch.int32)[None], torch.tensor([0, 1], device=DEV, dtype=torch.int32), torch.tensor([T], device=DEV, dtype=torch.int32)
        x = torch.randn(1, 2 * heads_, 64, generator=g, device=DEV).half()
        assert same(q.kv4_attention(x, a, table, cu, lens, 1, T), q.kv4_attention(x, odd, table, cu, lens, 1, T))


def test_attention_nothing(q):
    c = Paged(q, [(1, 0), (3, 0)], 4, 1, 64, 32, 16, F16)
    out, lse = c.run(q)
    assert (out == 0).all() and (lse == -math.inf).all()
    empty = q.kv4_attention(c.q[:0], c.cache, c.table, torch.zeros_like(c.cu_q), c.kv_lens, 1, 10)
    assert empty.shape == (0, 4, 64)


@pytest.mark.parametrize("n", [1, 70])
def test_attention_nan(q, n):
    """A row of NaN, and rows that see a key of NaN, are NaN; rows before that key are not."""
    c = Paged(q, [(n, 100), (n, 100)], 4, 1, 64, 32, 16, F16, seed=7)
    c.q[0, 1] = math.nan
    out, lse = c.run(q)
    assert out[0, 1].isnan().all() and lse[0, 1].isnan() and torch.isfinite(out[0, 0]).all() and torch.isfinite(out[1:]).all() and torch.isfinite(lse[1:]).all()
    c.cache.k_scale[c.table[1, 6].long(), 0, 2, 1, 0] = math.nan        # key 98 of the second sequence: its last two rows see it (or the only one)
    out, lse = c.run(q)
    at = n + max(0, n - 2)
    assert out[at:].isnan().all() and lse[at:].isnan().all() and torch.isfinite(out[1:at]).all() and torch.isfinite(lse[1:at]).all()


def test_attention_bad_offsets(q):
    """Offsets that do not fit q: the sequence is left out, the others are served."""
    c = Paged(q, [(2, 30), (3, 40), (4, 50)], 4, 1, 64, 64, 16, F16, seed=8)
    good, _ = c.run(q)
    c.cu_q[3] = 10 ** 6
    out, _ = c.run(q)
    assert same(out[:5], good[:5]) and (out[5:] == 7).all()


@pytest.mark.parametrize("seqs", list(SEQS))
def test_attention_same_bits_and_streams(q, seqs):
    c = Paged(q, SEQS[seqs], 8, 2, 128, 64, 16, F16, seed=5)
    out, lse = c.run(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other, lse2 = c.run(q)
    torch.cuda.current_stream().wait_stream(side)
    assert same(out, other) and same(lse, lse2)


def test_far_pages(q):
    """Codes beyond 2^32 bytes: pages at the far end of one large tensor."""
    pages, Hkv, page, D, G = 2100000, 2, 16, 128, 32             # 4.3 GB a side
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB")
    codes = [torch.empty(pages, Hkv, page, D // 2, dtype=torch.uint8, device=DEV) for _ in range(2)]
    c = q.KV4Cache(*codes, *(torch.empty(pages, Hkv, page, D // G, 2, dtype=F16, device=DEV) for _ in range(2)))
    g = gen(1)
    T = 40
    k, v, xq = (torch.randn(T, h, D, generator=g, device=DEV).half() for h in (Hkv, Hkv, 4))
    ids = torch.tensor([pages - 1, 3, pages - 2], device=DEV)
    t = torch.arange(T, device=DEV)
    slots = ids[t // page] * page + t % page
    q.kv4_append(None, k, v, c, slots)
    near = q.kv4_cache(3, Hkv, page, D, G)
    q.kv4_append(None, k, v, near, t)
    for a, b in zip(q.kv4_read(c, slots), q.kv4_read(near, t)):
        assert same(a, b) and a.abs().max() > 1
    args = (torch.tensor([0, T], dtype=torch.int32, device=DEV), torch.tensor([T], dtype=torch.int32, device=DEV))
    for n in (T, 1):
        cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
        far = q.kv4_attention(xq[:n], c, ids.to(torch.int32)[None].contiguous(), cu, args[1], n, T)
        assert same(far, q.kv4_attention(xq[:n], near, torch.arange(3, device=DEV, dtype=torch.int32)[None].contiguous(), cu, args[1], n, T))


# ------------------------------------------------------------ run together --
@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
def test_cache_in_4_bits_beside_one_in_16(q, dtype):
    """The same keys and values in a 16-bit cache (what the 4-bit one reads back as) give the same attention."""
    g = gen(21)
    Hq, Hkv, D, G, page, L = 8, 2, 128, 64, 16, 300
    xq, k, v = heads(L, Hq, Hkv, D, F16, g)
    w, table = (1 + 0.2 * torch.randn(D, generator=g, device=DEV)).half(), rope_table(L, D)
    pos, slots = torch.arange(L, device=DEV, dtype=torch.int32), torch.randperm(19 * page, generator=g, device=DEV)[:L]
    pages = torch.arange(19, device=DEV, dtype=torch.int32)[None].contiguous()
    slots = torch.arange(L, device=DEV)
    c = q.kv4_cache(19, Hkv, page, D, G)
    y = q.kv4_append(xq, k, v, c, slots, pos, table, q_norm=w, k_norm=w)
    k16, v16 = (torch.zeros(19, Hkv, page, D, device=DEV).half() for _ in range(2))
    q.kv_append(None, *q.kv4_read(c, slots), k16, v16, slots)
    for n in (1, 5, L):
        args = (pages, torch.tensor([0, n], dtype=torch.int32, device=DEV), torch.tensor([L], dtype=torch.int32, device=DEV), n, L)
        got, want = q.kv4_attention(y[L - n:], c, *args), q.paged_attention(y[L - n:], k16, v16, *args)
        # two results off by their probabilities' and output's roundings each; |v| averages below 4
        close(got, want.double(), 2 * 2.0 ** -11 * (want.double().abs() + 4))


def test_layer_step_in_a_graph(q):
    """Append, attention with a window and sinks, linear and read captured and replayed, with eager work between; two graphs."""
    g = gen(12)
    Hq, Hkv, D, page, B = 8, 2, 64, 16, 5
    c = Paged(q, [(1, L) for L in (1, 40, 700, 17, 3001)], Hq, Hkv, D, 32, page, F16, seed=6)
    for t in c.cache[2:]:
        t.nan_to_num_(0.5)
    K = Hq * D
    wq = torch.randint(-2 ** 31, 2 ** 31, (K, K * 4 // 32), generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    s = (torch.rand(K, K // 64, generator=g, device=DEV) * 0.02).half()
    x = torch.randn(B, (Hq + 2 * Hkv) * D, generator=g, device=DEV).half()
    res, w = torch.randn(B, K, generator=g, device=DEV).half(), (1 + 0.2 * torch.randn(D, generator=g, device=DEV)).half()
    table = rope_table(4000, D)
    positions = (c.kv_lens - 1).contiguous()
    slots = torch.stack([c.table[b, (L - 1) // page].long() * page + (L - 1) % page for b, (_, L) in enumerate(c.seqs)])

    def step(window):
        xq, k, v = (t.unflatten(1, (-1, D)) for t in x.split((Hq * D, Hkv * D, Hkv * D), 1))
        t = q.kv4_append(xq, k, v, c.cache, slots, positions, table, q_norm=w, k_norm=w)
        o = q.kv4_attention(t, c.cache, c.table, c.cu_q, c.kv_lens, 1, 3001, window=window, sinks=4)
        h = q.linear(o.flatten(1), wq, s, None, 4, 64, residual=res)
        y, _ = q.qk_norm(xq, k, w, w, 1e-6, positions, table)
        return (q.linear(h, wq, s, None, 4, 64, act="silu", mul=h), y) + q.kv4_read(c.cache, slots)

    eager = step(0), step(500)
    graphs = []
    for window in (0, 500):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step(window)
        graphs.append((graph, got, window))
    for i in range(4):
        x.copy_(torch.randn(x.shape, generator=g, device=DEV))
        for graph, got, window in graphs:
            want = step(window)
            torch.cuda.synchronize()
            for t in got:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(same(a, b) for a, b in zip(got, want)), i
    assert not same(want[0], eager[1][0]) and not same(eager[0][0], eager[1][0])


# -------------------------------------------------------------- refusals --
def test_decoder_layer_example(q):
    """The example runs on a cache of 4 bits."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_layer.py")
    spec = importlib.util.spec_from_file_location("decoder_layer_4", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    us, error = example.run(hidden=512, heads=8, kv_heads=2, head_dim=64, inner=1024, users=3, prompt=50, steps=4, cache_bits=4)
    assert us > 0 and math.isfinite(error)


def test_refusals_on_the_gpu(q):
    """Shapes, types and devices that do not fit, named in the error; nothing is written."""
    c = Paged(q, [(1, 20)], 4, 2, 64, 32, 16, F16)
    k4, v4, ks, vs = c.cache
    out = torch.full((1, 4, 64), 7.0, device=DEV).half()
    ok = dict(q=c.q, cache=c.cache, page_table=c.table, cu_q=c.cu_q, kv_lens=c.kv_lens, max_q=1, max_kv=20, out=out)
    bad_caches = [((k4, v4, ks), TypeError), (k4, TypeError), (None, TypeError), ((k4, v4[1:], ks, vs), ValueError), ((k4, v4, ks, vs[:, :1]), ValueError),
                  ((k4.view(torch.int8), v4, ks, vs), TypeError), ((k4, v4, ks.float(), vs), TypeError), ((k4, v4.cpu(), ks, vs), ValueError),
                  ((k4, v4, ks[..., :1], vs), ValueError), ((k4.transpose(2, 3), v4, ks, vs), ValueError), ((k4, v4, ks[:, :, :, :1], vs[:, :, :, :1]), ValueError),
                  ((k4, v4, ks.repeat(1, 1, 1, 4, 1), vs.repeat(1, 1, 1, 4, 1)), q.QmmError), ((k4, v4, ks[..., 0], vs), ValueError)]
    bad = [(dict(q=c.q[:, :3], out=None), q.QmmError), (dict(q=c.q.float()), TypeError), (dict(q=c.q[..., :32]), ValueError),
           (dict(page_table=c.table.long()), TypeError), (dict(cu_q=c.cu_q[:1]), ValueError), (dict(kv_lens=c.kv_lens.cpu()), ValueError), (dict(out=out[:, :2]), ValueError),
           (dict(out=out.to(BF16)), TypeError), (dict(lse=torch.zeros(1, 3, device=DEV)), ValueError), (dict(max_q=0), q.QmmError), (dict(window=-1), q.QmmError),
           (dict(sinks=-1), q.QmmError), (dict(sinks=1.5), TypeError), (dict(scale=-1.0), q.QmmError), (dict(scale=math.nan), q.QmmError), (dict(scale="a"), TypeError),
           (dict(max_q=1.5), TypeError)]
    for change, kind in bad + [(dict(cache=x), e) for x, e in bad_caches]:
        with pytest.raises(kind):
            q.kv4_attention(**{**ok, **change})
    k, v = (torch.zeros(1, 2, 64, device=DEV).half() for _ in range(2))
    slots, pos, table, w = torch.zeros(1, dtype=torch.int64, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV), rope_table(4, 64), torch.ones(64, device=DEV).half()
    before = [t.clone() for t in c.cache]
    ok = dict(q=c.q, k=k, v=v, cache=c.cache, slots=slots, positions=pos, rope=table, q_norm=w, k_norm=w, out=out)
    bad = [(dict(k=k[:, :1]), ValueError), (dict(v=v[..., :32]), ValueError), (dict(slots=slots.int()), TypeError), (dict(positions=None), ValueError),
           (dict(rope=None), ValueError), (dict(rope=table.half()), TypeError), (dict(rope=table[:, ::2]), ValueError), (dict(q=None), ValueError),
           (dict(rope=rope_table(4, 40)), q.QmmError), (dict(rope=rope_table(4, 80)), q.QmmError), (dict(k=k.transpose(1, 2)), ValueError), (dict(q_norm=w[:32]), ValueError),
           (dict(k_norm=w.float()), TypeError), (dict(k_norm=torch.ones(72, device=DEV).half()[1:65]), q.QmmError), (dict(eps=-1.0), q.QmmError), (dict(eps=math.nan), q.QmmError),
           (dict(q=None, out=None), ValueError)]
    for change, kind in bad + [(dict(cache=x), e) for x, e in bad_caches]:
        with pytest.raises(kind):
            q.kv4_append(**{**ok, **change})
    bad = [(dict(q_weight=w[:32]), ValueError), (dict(k=k.to(BF16)), TypeError), (dict(k=torch.zeros(2, 2, 64, device=DEV).half()), ValueError), (dict(rope=None), ValueError),
           (dict(q=torch.zeros(1, 2, 40, device=DEV).half(), k=torch.zeros(1, 2, 40, device=DEV).half(), q_weight=None, k_weight=None, rope=None, positions=None, q_out=None), q.QmmError),
           (dict(q_out=out[:, :1]), ValueError), (dict(eps=math.inf), q.QmmError), (dict(eps="a"), TypeError)]
    for change, kind in bad:
        with pytest.raises(kind):
            q.qk_norm(**{**dict(q=c.q, k=k, q_weight=w, k_weight=w, positions=pos, rope=table, q_out=out), **change})
    bad = [(dict(slots=slots.int()), TypeError), (dict(slots=slots[None]), ValueError), (dict(slots=slots.cpu()), ValueError), (dict(dtype=torch.float32), TypeError),
           (dict(k_out=out), ValueError)]
    for change, kind in bad + [(dict(cache=x), e) for x, e in bad_caches]:
        with pytest.raises(kind):
            q.kv4_read(**{**dict(cache=c.cache, slots=slots), **change})
    for kw in (dict(D=40), dict(D=64, G=128), dict(D=64, G=16), dict(D=512), dict(D=0)):
        with pytest.raises(ValueError):
            q.kv4_cache(1, 1, 16, **kw)
    torch.cuda.synchronize()
    assert (out == 7).all() and all(same(a, b) for a, b in zip(before, c.cache))
