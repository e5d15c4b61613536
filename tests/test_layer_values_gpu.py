"""Values at which the decoder-layer calls can go wrong without a fault: NaN and overflow, scales
of any sign, keys far below a row's largest, and products that are exact, so that one lost
code, run, group or slice shows.  On an MI355X.
"""
import math

import pytest
import torch

from test_layer_gpu import DEV, E4M3, SEQS, U, Paged, _announce, close, decoded, gen, q, same, weights  # noqa: F401

pytestmark = pytest.mark.gpu


# --------------------------------------------------------------- attention --
def refill(c):
    """c.k and c.v into the pages of the caches."""
    for b, (_, L) in enumerate(c.seqs):
        ids = c.table[b].tolist()
        for p in range(-(-L // c.page)):
            for cache, x in ((c.kc, c.k[b]), (c.vc, c.v[b])):
                raw = (lambda t: t.view(torch.uint8)) if x.dtype == E4M3 else (lambda t: t)
                part = raw(x)[p * c.page:(p + 1) * c.page].transpose(0, 1)
                raw(cache[ids[p]])[:, :part.shape[1]] = part


def rows_of(c):
    """(row of q, whether it sees a key) of each sequence's first and last new token."""
    t = 0
    for n, L in c.seqs:
        for i in {0, n - 1} if n else ():
            yield t + i, L - n + i >= 0
        t += n


def spoiled(q, c, value, heads):
    """Runs with `value` in the heads of some rows of q: those rows are NaN, or zeros and -inf where they see no key;
    the others are as they would be without."""
    good, good_lse = c.run(q)
    clean = c.q.clone()
    for t, _ in rows_of(c):
        c.q[t, heads, 5 % c.D] = value
    out, lse = c.run(q)
    c.q.copy_(clean)
    for t, sees in rows_of(c):
        if sees:
            assert torch.isnan(out[t, heads]).all() and torch.isnan(lse[t, heads]).all(), t
            out[t, heads], lse[t, heads] = good[t, heads], good_lse[t, heads]
    c.check(out, lse)      # rows without a key among them


@pytest.mark.parametrize("e4m3", [False, True], ids=["plain", "e4m3"])
@pytest.mark.parametrize("seqs", list(SEQS))
@pytest.mark.parametrize("Hq,Hkv,D,page,dtype", [(8, 2, 128, 16, torch.float16), (32, 32, 64, 16, torch.bfloat16), (6, 2, 80, 7, torch.float16),
                                                 (8, 1, 256, 64, torch.bfloat16)])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_attention_keeps_nan(q, seqs, e4m3, Hq, Hkv, D, page, dtype, value):
    spoiled(q, Paged(SEQS[seqs], Hq, Hkv, D, page, dtype, e4m3, seed=D), value, [1, Hq - 1])


@pytest.mark.parametrize("e4m3", [False, True], ids=["plain", "e4m3"])
@pytest.mark.parametrize("page", [16, 7])
@pytest.mark.parametrize("window", [0, 100])
def test_attention_keeps_nan_short_chunks(q, e4m3, page, window):
    """Two blocks of 16 rows a key head, and a window before which pages are gone."""
    spoiled(q, Paged([(5, 5), (4, 300), (8, 2000), (3, 0), (7, 4)], 8, 2, 128, page, torch.float16, e4m3, window=window, seed=2), math.nan, [1, 7])


@pytest.mark.parametrize("seqs", list(SEQS))
def test_attention_overflow_is_nan(q, seqs):
    """Scores that leave fp32 for -inf, all of a row's: not a row without keys."""
    c = Paged(SEQS[seqs], 8, 2, 64, 16, torch.bfloat16, seed=3)
    c.q[..., 5] = 0
    for k in c.k:
        k[..., 5] = -1e30
    refill(c)
    spoiled(q, c, 1e30, [0, 6])


@pytest.mark.parametrize("n", [1, 40])
def test_attention_hidden_pages_of_a_nan_row(q, n):
    """A NaN row whose keys all stand on bad pages sees none; one good page is enough to make it NaN."""
    c = Paged([(n, 500), (n, 90)], 4, 2, 64, 16, torch.float16, seed=7)
    c.q[:] = math.nan
    good = c.table[1, 1].item()
    c.table[:] = -1
    c.table[1, 1] = good
    out, lse = c.run(q)
    assert (out[:n] == 0).all() and (lse[:n] == -math.inf).all()
    sees = torch.arange(90 - n, 90, device=DEV) >= 16
    assert torch.isnan(out[n:][sees]).all() and torch.isnan(lse[n:][sees]).all()


@pytest.mark.parametrize("seqs", list(SEQS))
@pytest.mark.parametrize("page", [16, 7])
@pytest.mark.parametrize("factor", [-1.0, 0.0, -1e-30])
def test_attention_scale_of_any_sign(q, seqs, page, factor):
    """A key stands for its e4m3 value times the scale, whatever its sign."""
    c = Paged(SEQS[seqs], 8, 2, 128, page, torch.float16, True, seed=9)
    c.ks[1] *= factor
    c.vs[0] *= -1
    c.check(*c.run(q))


@pytest.mark.parametrize("seqs", list(SEQS))
def test_attention_nan_scale(q, seqs):
    c = Paged(SEQS[seqs], 8, 2, 128, 16, torch.float16, True, seed=9)
    good, good_lse = c.run(q)
    scale = c.ks[1].clone()
    c.ks[1] = math.nan
    out, lse = c.run(q)
    c.ks[1] = scale
    t = 0
    for n, L in c.seqs:
        for i in range(n):
            if L - n + i >= 0:
                assert torch.isnan(out[t + i, 4:]).all() and torch.isnan(lse[t + i, 4:]).all()
                out[t + i, 4:], lse[t + i, 4:] = good[t + i, 4:], good_lse[t + i, 4:]
        t += n
    c.check(out, lse)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("e4m3", [False, True], ids=["plain", "e4m3"])
@pytest.mark.parametrize("n,B,L,Hkv", [(1, 8, 2000, 32), (20, 8, 2000, 32), (40, 8, 2000, 32), (1, 1, 5000, 32), (300, 1, 5000, 32)])
def test_attention_far_below_the_largest(q, dtype, e4m3, n, B, L, Hkv):
    """One key 11 to 19 above all others in the exponent, its value zero: the output is the others' share alone.

    A probability is rounded once, by half a step of itself or, in fp16, by 2^-36 of the row's largest
    where that is more (2^-25, half the smallest step, of a scale that puts the largest at 2^11 or above)."""
    D, page, u = 64, 16, U[dtype]
    c = Paged([(n, L)] * B, Hkv, Hkv, D, page, dtype, e4m3, seed=1)
    c.q.fill_(1.0)
    far = torch.linspace(11, 19, Hkv, device=DEV)
    one = c.ks if e4m3 else torch.ones(Hkv, device=DEV)
    for k, v in zip(c.k, c.v):
        k.copy_(torch.zeros(L, Hkv, D, device=DEV).to(k.dtype))
        v.copy_(torch.full((L, Hkv, D), 64.0, device=DEV).to(v.dtype))
        k[0] = (far / 8 / one)[:, None].expand(Hkv, D).to(k.dtype)
        v[0] = torch.zeros(Hkv, D, device=DEV).to(v.dtype)
    refill(c)
    out, lse = c.run(q)
    top = c.k[0][0, :, 0].double() * one.double() * D * c.scale                       # [Hkv]
    value = 64.0 * (c.vs.double() if e4m3 else torch.ones_like(top))
    others = torch.arange(L - n, L, device=DEV, dtype=torch.float64)[:, None]         # keys but the first that row i sees
    part = others * torch.exp(-top)
    o = (part / (1 + part) * value).repeat(B, 1)[..., None].expand(B * n, Hkv, D)
    rel = 2 * (D + 8) * 2.0 ** -24 * top + (L + 64) * 2.0 ** -24 + 2.0 ** -20
    floor = L * 2.0 ** -36 * value if dtype is torch.float16 else torch.zeros_like(value)
    close(out, o, (2 * u + rel[:, None]) * o + floor[:, None] + 2.0 ** -24)
    close(lse, (top + torch.log1p(part)).repeat(B, 1), (rel + 2.0 ** -21 * (top + 1)).expand(B * n, Hkv))


# ------------------------------------------------------------------ linear --
# one token; the GEMVs; the streaming kernel with 16, 32 and 64 rows, with groups of 128 and others; the GEMM whole and in slices of K
SHAPES = [(1, 4096, 1000, 128), (1, 16384, 70, 128), (3, 1024, 130, 64), (16, 1152, 264, 128), (7, 2080, 50, 32),
          (2, 8320, 40, 128), (5, 16384, 33, 32), (16, 28672, 264, 128), (16, 8320, 17, 128), (11, 6144, 300, 64),
          (17, 4096, 4100, 128), (32, 8320, 2001, 128), (20, 8192, 2001, 64), (29, 6272, 130, 128), (33, 28800, 600, 96), (64, 4224, 4000, 128), (50, 8192, 130, 128),
          (40, 2080, 1000, 32), (130, 8192, 1032, 32), (111, 5760, 2001, 64), (263, 10240, 700, 128), (300, 4096, 1100, 128), (70, 256, 136, 64),
          (1100, 256, 1032, 128)]


@pytest.mark.parametrize("M,K,N,G", SHAPES, ids=lambda v: str(v))
@pytest.mark.parametrize("bits", range(1, 9))
@pytest.mark.parametrize("z", [False, True], ids=["", "z"])
def test_linear_exact(q, M, K, N, G, bits, z):
    """One +-1 in each run of 32 rows of K, powers of two as scales: every sum is exact in fp32 in
    any order, so Y is the exact value rounded once, bit for bit."""
    g = gen(K + bits)
    runs = K // 32
    assert runs * (1024 + 2 * 2 ** bits) * 8 < 2 ** 24     # in units of the smallest scale, the codes' offset of 1024 with them
    X = torch.zeros(M, runs, 32, device=DEV, dtype=torch.float16)
    at = torch.randint(0, 32, (M, runs, 1), generator=g, device=DEV)
    X.scatter_(2, at, (torch.randint(0, 2, at.shape, generator=g, device=DEV) * 2 - 1).half())
    X = X.view(M, K)
    wq, s, zz = weights(K, N, bits, G, z, g)
    s = 2.0 ** -torch.randint(4, 8, s.shape, generator=g, device=DEV).half()
    w = (decoded(wq, K, bits) - (2.0 ** (bits - 1) if zz is None else zz.double().repeat_interleave(G, 1))) * s.double().repeat_interleave(G, 1)
    h = X.double() @ w.T
    assert same(q.linear(X, wq, s, zz, bits, G), h.half())
    bias, res = (torch.randint(-8, 9, sh, generator=g, device=DEV).half() for sh in ((N,), (M, N)))
    mul = (torch.randint(0, 2, (M, N), generator=g, device=DEV) * 1.5 - 1).half()          # -1 or 1/2
    y = (h + bias.double()).clamp(min=0) * mul.double() + res.double()
    Y = q.linear(X, wq, s, zz, bits, G, bias=bias, act="relu", mul=mul, residual=res)
    assert torch.equal(Y.double(), y.half().double())


@pytest.mark.parametrize("M,K,N,G", [s for s in SHAPES if s[0] > 16 or (s[0] > 1 and s[1] > 8192)], ids=lambda v: str(v))
@pytest.mark.parametrize("bits,z", [(1, False), (2, True), (4, True), (5, False), (8, True)])
def test_linear_rounding(q, M, K, N, G, bits, z):
    """Weights rounded to fp16 once at most and fp32 sums.  X has random signs, so that the sum of the K roundings
    has a standard deviation of 2^-11 (sum x^2 w^2)^(1/2) at most, and that of the sums one of 2^-24 K^(1/2) of
    the same; 8 of them are allowed."""
    g = gen(K + 10 * bits)
    X = torch.randn(M, K, generator=g, device=DEV).half()
    wq, s, zz = weights(K, N, bits, G, z, g)
    w = (decoded(wq, K, bits) - (2.0 ** (bits - 1) if zz is None else zz.double().repeat_interleave(G, 1))) * s.double().repeat_interleave(G, 1)
    h, size = X.double() @ w.T, (X.double() ** 2 @ (w.T ** 2).contiguous()).sqrt()
    close(q.linear(X, wq, s, zz, bits, G), h, 8 * (2.0 ** -11 + 2.0 ** -24 * K ** 0.5) * size + 2.0 ** -11 * h.abs() + 2.0 ** -24)


@pytest.mark.parametrize("M,K,N,G", SHAPES, ids=lambda v: str(v))
def test_linear_keeps_nan(q, M, K, N, G):
    """A NaN activation reaches every output of its row through every epilogue, and no other row."""
    g = gen(M)
    X = torch.randn(M, K, generator=g, device=DEV).half()
    wq, s, z = weights(K, N, 4, G, True, g)
    mul, res = (torch.randn(M, N, generator=g, device=DEV).half() for _ in range(2))
    row = M // 2
    for act, m, r in (("none", None, None), ("relu", None, None), ("silu", mul, None), ("gelu", mul, res), ("gelu_tanh", None, res), ("relu", mul, res)):
        X[row, K - 7] = 0.5
        clean = q.linear(X, wq, s, z, 4, G, act=act, mul=m, residual=r)
        X[row, K - 7] = math.nan
        Y = q.linear(X, wq, s, z, 4, G, act=act, mul=m, residual=r)
        assert torch.isnan(Y[row]).all(), act
        rest = torch.arange(M, device=DEV) != row
        assert same(Y[rest], clean[rest])


@pytest.mark.parametrize("M,K,N,G", [s for s in SHAPES if s[0] > 1], ids=lambda v: str(v))
@pytest.mark.parametrize("what", ["s", "z"])
def test_linear_columns_stand_alone(q, M, K, N, G, what):
    """Scales or zero-points of one column that are infinite or NaN reach no other column."""
    g = gen(N)
    X = torch.randn(M, K, generator=g, device=DEV).half()
    wq, s, z = weights(K, N, 4, G, True, g)
    clean = q.linear(X, wq, s, z, 4, G)
    for col, value in ((N // 2, math.inf), (N // 3, math.nan), (N - 1, math.inf), (0, math.nan)):
        (s if what == "s" else z)[col] = value
        Y = q.linear(X, wq, s, z, 4, G)
        assert not torch.isfinite(Y[:, col]).any()
        clean[:, col] = Y[:, col]
        bad = ~torch.isfinite(Y)
        assert torch.equal(bad, ~torch.isfinite(clean)), torch.unique(bad.nonzero()[:, 1]).tolist()[:8]
        keep = ~bad
        assert torch.equal(Y[keep], clean[keep])
