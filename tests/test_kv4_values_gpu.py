"""Values at which the calls around a cache of 4-bit codes can go wrong without a fault: keys and values of very
different sizes side by side, sums that cancel.  On an MI355X.

Tolerances count roundings, as in test_kv4_gpu.py.
"""
import importlib.util
import math
import os

import pytest
import torch

from test_kv4_gpu import BF16, DEV, F16, U, Paged, _announce, check_stored, close, decoded, encoded, gen, heads, norm_bound, place, q, rope_table, same, turned  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------ attention: sizes far apart --
def refill(c, k=None, v=None):
    """k and v, [L, Hkv, D] for each sequence, into the pages of c; keeps their codes, scales and zero-points."""
    c.parts = []
    for b, (_, L) in enumerate(c.seqs):
        sides = []
        for x, codes, scale, now in ((k, c.cache.k, c.cache.k_scale, c.k), (v, c.cache.v, c.cache.v_scale, c.v)):
            G = c.D // scale.shape[3]
            n, s, z = encoded(now[b] if x is None else x[b].double(), G)
            packed, sz = (n[..., 0::2] | n[..., 1::2] << 4).to(torch.uint8), torch.stack((s, z), -1).half()
            for p in range(-(-L // c.page)):
                at, lo, hi = int(c.table[b, p]), p * c.page, min(L, (p + 1) * c.page)
                if at >= 0:
                    codes[at, :, :hi - lo] = packed[lo:hi].transpose(0, 1)
                    scale[at, :, :hi - lo] = sz[lo:hi].transpose(0, 1)
            now[b] = decoded(packed, sz)
            sides.append((n.double().unflatten(-1, (-1, G)), sz[..., 0].double(), sz[..., 1].double()))      # s and z as they are held
        c.parts.append(sides)


def check(c, out, lse, fed):
    """fed: the codes meet the products as they are, scales and zero-points apart; else as (code - z) s."""
    t = 0
    for b, (n, L) in enumerate(c.seqs):
        if n == 0 or L == 0:
            t += n
            continue
        qs = c.q[t:t + n].double().unflatten(1, (c.Hkv, c.g))
        got, gl = out[t:t + n].double().unflatten(1, (c.Hkv, c.g)), lse[t:t + n].double().unflatten(1, (c.Hkv, c.g))
        t += n
        pos, key = torch.arange(L - n, L, device=DEV)[:, None], torch.arange(L, device=DEV)
        mask = (key <= pos).repeat_interleave(c.g, 0)
        (kn, ks, kz), (vn, vs, vz) = c.parts[b]
        G = kn.shape[-1]
        for h in range(c.Hkv):
            qh, k, v = qs[:, h].reshape(n * c.g, c.D), c.k[b][:, h], c.v[b][:, h]
            x = torch.where(mask, qh @ k.T * c.scale, -math.inf)
            l = torch.logsumexp(x, 1)
            p = torch.exp(x - l[:, None])
            # a score: sums of q c and of q, q on a grid of 6 bits, are exact where they meet so; times s, added, times the
            # scale and in the exponent some ten roundings.  Else D products (code - z) s q summed in fp32.
            size = ((kn[:, h] + kz[:, h, :, None]) * ks[:, h, :, None]).flatten(1)
            dx = ((12 if fed else c.D + 8) * 2.0 ** -24 * c.scale * torch.where(mask, qh.abs() @ size.T, 0.0)).amax(1, keepdim=True)
            rel = 2 * dx + (L + 64) * 2.0 ** -24 + 2.0 ** -20
            o, each = p @ v, p @ v.abs()
            bound = (U[F16] + rel) * each + U[c.dtype] * o.abs() + (2.0 ** -25 if c.dtype == F16 else 0.0)
            if fed:
                # weights p s in fp16: half a step, or 2^-36 of the row's largest in the group, times up to 15 steps;
                # sums of codes and of zero-points in fp32, each for itself
                w = p[:, :, None] * vs[:, h]                                       # [rows, keys, groups]
                tiny = 2.0 ** -36 * 15 * mask.sum(1)[:, None] * w.amax(1)
                step = torch.einsum("rjg,jge->rge", w, vn[:, h] + vz[:, h, :, None])
                bound = bound + ((L + 64) * 2.0 ** -24 * step + tiny[..., None]).flatten(1)
            else:
                bound = bound + 2.0 ** -36 * p.amax(1, keepdim=True) * (mask.double() @ v.abs())
            close(got[:, h].reshape(n * c.g, c.D), o, bound)
            close(gl[:, h].reshape(-1), l, rel[:, 0] + 2.0 ** -21 * l.abs())


def sizes(kind, L, Hkv, D, G, g):
    """(values' exponents [L, Hkv, D / G], what is added to the keys' first 16 elements [L])."""
    e, up = torch.zeros(L, Hkv, D // G, device=DEV), torch.zeros(L, device=DEV)
    at = torch.arange(L, device=DEV)
    if kind == "keys":           # any size beside any other
        e = torch.randint(-11, 14, e.shape, generator=g, device=DEV).float()
    elif kind == "groups":       # one group small, the next large
        e[..., 0::2], e[..., 1::2] = -11, 13
    elif kind == "groups_down":
        e[..., 0::2], e[..., 1::2] = 13, -11
    elif kind == "rare":         # a key in 61 is large, and gets next to no weight
        e -= 11
        e[at % 61 == 17], up[at % 61 == 17] = 13, -4.5
    elif kind == "early":        # large values first, then keys that take all weight from them
        e -= 11
        e[:L // 3], up[L // 3:] = 13, 5.0
    elif kind == "late":
        e -= 11
        e[L // 2:], up[L // 2:] = 13, -5.0
    elif kind == "block":        # in one wave's block alone
        e -= 11
        e[(at >= 32) & (at < 64)] = 13
    return e, up


FED = [(128, 128), (128, 64), (64, 64), (256, 128)]


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("kind", ["keys", "groups", "groups_down", "rare", "early", "late", "block"])
@pytest.mark.parametrize("D,G", FED + [(128, 32), (192, 64), (256, 64)])
def test_attention_of_values_of_very_different_sizes(q, D, G, kind, dtype):
    """Scales of values some 2^24 apart, between keys, groups, blocks, waves and shares: a small value keeps its bits
    wherever no large one has weight beside it in its group."""
    for seqs, Hq, Hkv, page in (([(1, 700), (1, 33), (2, 130)], 4, 2, 16), ([(3, 400), (1, 90)], 8, 1, 3), ([(1, 500), (2, 64)], 4, 2, 1),
                                ([(70, 300), (1, 200)], 4, 2, 16), ([(1, 9000)], 4, 2, 16)):
        c = Paged(q, seqs, Hq, Hkv, D, G, page, dtype, seed=D + G)
        g = gen(D + page)
        c.q.copy_((c.q.clamp(-3.9, 3.9) * 4).round() / 4)
        c.q[..., :16] += 4.0
        k, v = [], []
        for b, (_, L) in enumerate(seqs):
            e, up = sizes(kind, L, Hkv, D, G, g)
            k.append(c.k[b].clone())
            k[b][..., :16] += up[:, None, None]
            v.append(c.v[b] * torch.exp2(e.double()).repeat_interleave(G, 2))
        refill(c, k, v)
        out, lse = c.run(q)
        rows = max(n for n, _ in seqs) * Hq // Hkv
        check(c, out, lse, (D, G) in FED and rows <= (16 if (D, G) == (128, 64) else 32))


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("kind", ["ones", "minus", "mixed", "any"])
@pytest.mark.parametrize("D,G,g", [(64, 64, 16), (64, 64, 32), (128, 64, 16), (128, 128, 16), (128, 128, 32), (256, 128, 16), (128, 32, 16), (96, 32, 32), (256, 64, 8)])
def test_scores_are_sums_of_fp32(q, D, G, g, kind, dtype):
    """One key a sequence: its log sum is its score.  Codes of 1 beside one of 15 in their group, and zero-points of 15, where sums of
    s c, and of z, are far larger than what they differ by.

    32 products of codes of 1 may be off by 2^-18.4 of the sum of their sizes (49 of 2^-24; root mean square 2^-21.6), their sums add a
    rounding each, twelve more are s, z, the scale, the exponent and the logarithm, with 36 at most in the exponent (half a step
    there 2^-19).  Taken together the errors are root mean squares: of the products 2^-21.6, and of twelve roundings in any
    direction 2^-23."""
    B, Hkv = 200, 2
    c = Paged(q, [(1, 1)] * B, g * Hkv, Hkv, D, G, 16, dtype, seed=D + G + g)
    r = gen(g)
    k = torch.ones(B, 1, Hkv, D, device=DEV)
    if kind == "mixed":
        k = torch.randint(-1, 2, k.shape, generator=r, device=DEV).float()
    elif kind == "any":
        k = torch.randint(0, 16, k.shape, generator=r, device=DEV).float()
    k.unflatten(-1, (-1, G))[..., 5] = 15.0
    if kind == "minus":
        k = -k
    refill(c, list(k))
    _, lse = c.run(q)
    square = 0.0
    for b in range(B):
        kn, ks, kz = (x[0] for x in c.parts[b][0])
        qs = c.q[b].double().unflatten(0, (Hkv, g))
        size = ((kn + kz[..., None]) * ks[..., None]).flatten(1)
        want = torch.einsum("hgd,hd->hg", qs, c.k[b][0]) * c.scale
        most = torch.einsum("hgd,hd->hg", qs.abs(), size) * c.scale
        got = lse[b].unflatten(0, (Hkv, g))
        close(got, want, (49 + D // 32 + 12) * 2.0 ** -24 * most + 2.0 ** -19)
        square += float(((got.double() - want) / (most + 0.25)).square().mean()) / B
    assert math.sqrt(square) < 2.0 ** -21


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 7)])
@pytest.mark.parametrize("D,G", FED + [(128, 32), (192, 64), (96, 32), (64, 32)])
def test_values_of_nan_reach_the_rows_that_see_them(q, D, G, window, sinks, dtype):
    """As the formula has it: a scale of NaN at a value makes its group NaN for the rows that see its key, and nothing else: the
    other outputs are those of a value of zeros there.  Up to 32 rows a key head to the bit.  Beyond, the call masks more in its
    second look, which moves the running maxima: fp32 roundings of exponents up to 32 (2^-19 each) and of sums, so
    that each side's probabilities, and its outputs, may round by half a step the other way."""
    for seqs, Hq, Hkv, page in (([(1, 90), (5, 200), (2, 33)], 4, 2, 16), ([(3, 150), (1, 20)], 8, 1, 3), ([(7, 64), (2, 2)], 2, 2, 1),
                                ([(70, 300), (1, 120), (33, 33)], 4, 2, 16), ([(300, 420)], 2, 1, 7), ([(4, 6000), (1, 40)], 4, 2, 16), ([(20, 6000)], 4, 1, 16)):
        c = Paged(q, seqs, Hq, Hkv, D, G, page, dtype, window=window, sinks=sinks, seed=D + G + page)
        g, t = gen(page), 0
        marks = []                                                  # (sequence, key, head, group)
        for b, (n, L) in enumerate(seqs):
            for j in {L - 1, L - 2, L - n, L - n // 2 - 1, 0, 5, L // 2, L - n - 30}:
                if 0 <= j < L and (not window or j < sinks or j > L - n - window):
                    marks.append((b, j, int(torch.randint(0, Hkv, (), generator=g, device=DEV)), int(torch.randint(0, D // G, (), generator=g, device=DEV))))
        for b, j, h, e in marks:
            c.cache.v_scale[c.table[b, j // page].long(), h, j % page, e] = 0
        want, lse = c.run(q)
        for b, j, h, e in marks:
            c.cache.v_scale[c.table[b, j // page].long(), h, j % page, e, 0] = math.nan
        got, lse2 = c.run(q)
        want = want.clone().unflatten(1, (Hkv, -1)).unflatten(3, (-1, G))
        exact = max(n for n, _ in seqs) * Hq // Hkv <= 32
        assert torch.isfinite(want).all()
        if exact:
            assert same(lse, lse2)
        close(lse2, lse.double(), 2.0 ** -18 + 2.0 ** -22 * lse.double().abs() + (max(L for _, L in seqs) + 64) * 2.0 ** -23)
        for b, (n, L) in enumerate(seqs):
            pos = torch.arange(L - n, L, device=DEV)
            for b2, j, h, e in marks:
                if b2 == b:
                    sees = (pos >= j) & ((pos - window < j) | (j < sinks) if window else pos >= j)
                    want[t:t + n, h, :, e][sees] = math.nan
            t += n
        want = want.flatten(3).flatten(1, 2)
        assert torch.equal(got.isnan(), want.isnan())
        got, want = got.nan_to_num(5.0), want.nan_to_num(5.0)
        if exact:
            assert same(got, want)
        most = max(float(v.abs().max()) for v in c.v)
        close(got, want.double(), (2 * U[F16] + 2.0 ** -17 + (max(L for _, L in seqs) + 64) * 2.0 ** -23) * most + 2 * U[dtype] * want.double().abs() + 2.0 ** -24)


# ------------------------------------------------------------------- norms --
@pytest.mark.parametrize("pairs", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("D,rot", [(128, 128), (80, 48), (256, 0)])
@pytest.mark.parametrize("size,eps", [(1e20, 1e-5), (1e20, 0.0), (3e37, 1e-5), (1e-25, 0.0), (1e-37, 0.0), (1e18, 1e-5), (1e-3, 1e-5)])
def test_norms_of_rows_of_any_size(q, size, eps, D, rot, pairs):
    """Squares beyond fp32 on either side: the norm is the formula's all the same, here and where k goes to a cache; rows
    of other sizes and of zeros beside them."""
    g = gen(D)
    xq, xk, v = heads(70, 5, 2, D, BF16, g, size=size)
    xq[3], xk[11] = torch.randn(5, D, generator=g, device=DEV).to(BF16), torch.randn(2, D, generator=g, device=DEV).to(BF16)
    if eps:
        xq[4, 2] = 0
    w, u = ((1 + 0.3 * torch.randn(D, generator=g, device=DEV)).to(BF16) for _ in range(2))
    table, pos = (rope_table(100, rot), torch.arange(70, device=DEV, dtype=torch.int32)) if rot else (None, None)
    yq, yk = q.qk_norm(xq, xk, w, u, eps, pos, table, pairs)
    for x, weight, y in ((xq, w, yq), (xk, u, yk)):
        want, most = turned(x, weight, eps, pos, table, pairs)
        close(y, want, norm_bound(want, most, D, BF16))
    if D % 32 == 0:
        c = q.kv4_cache(8, 2, 16, D)
        assert same(q.kv4_append(xq, xk, v, c, place(70, 8, 16, g), pos, table, pairs, w, u, eps), yq)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("by", [-0.25, 0.0, 0.25])
def test_append_takes_eps_as_it_is(q, dtype, by):
    """Keys whose quotients are ties if eps is rounded to fp32, and 2^-28 beside them by the formula."""
    D = 128
    k = ((torch.arange(D, device=DEV) % 31) / 2 * 2.0 ** -12).to(dtype).expand(5, 3, D).contiguous()
    k[1] *= -1
    mean = float(k[0, 0].double().square().mean())
    eps = 2.0 ** -16 - mean                                          # a number of fp32; the root is then 2^-8
    assert float(torch.tensor(eps, dtype=torch.float32)) == eps
    eps += by * 2.0 ** (math.frexp(eps)[1] - 24)                     # a quarter of its step beside it
    w, slots = torch.ones(D, device=DEV).to(dtype), torch.arange(5, device=DEV)
    c = q.kv4_cache(1, 3, 16, D)
    before = q.KV4Cache(*(t.clone() for t in c))
    v = torch.zeros_like(k)
    q.kv4_append(None, k, v, c, slots, k_norm=w, eps=eps)
    want, _, _ = encoded(turned(k, w, eps, None, None, False)[0], D)
    ties, _, _ = encoded(k.double(), D)
    assert by == 0 or not torch.equal(want, ties)
    check_stored(c, before, turned(k, w, eps, None, None, False)[0], v.double(), slots, D)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("eps", [1e-50, 1e-310])
def test_norms_with_eps_below_fp32(q, dtype, eps):
    """Rows of zeros stay zeros under any eps, however small."""
    x = torch.randn(4, 2, 64, generator=gen(1), device=DEV).to(dtype)
    x[2] = 0
    w = torch.ones(64, device=DEV).to(dtype)
    c = q.kv4_cache(1, 2, 16, 64)
    before = q.KV4Cache(*(t.clone() for t in c))
    y = q.kv4_append(x, x, x, c, torch.arange(4, device=DEV), q_norm=w, k_norm=w, eps=eps)
    want, most = turned(x, w, eps, None, None, False)
    close(y, want, norm_bound(want, most, 64, dtype))
    check_stored(c, before, want, x.double(), torch.arange(4, device=DEV), 64)


# ------------------------------------------------------------ run together --
def test_decoder_layer_example_on_its_cache(q):
    """The example's last output against the layer in fp32 on what the cache of 4 bits holds: the roundings of its 16-bit
    form but for those of k and v, some ten of 2^-11 in a row, whose root sum of squares stays below 2^-8."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_layer.py")
    spec = importlib.util.spec_from_file_location("decoder_layer_4_values", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    for users, prompt, steps, page in ((3, 75, 6, 16), (1, 1, 3, 1), (5, 300, 2, 64)):
        _, error = example.run(hidden=512, heads=8, kv_heads=2, head_dim=64, inner=1024, users=users, prompt=prompt, steps=steps, page=page, cache_bits=4)
        assert error < 2.0 ** -8


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("D,G", [(128, 64), (128, 32), (64, 64)])
def test_cache_in_4_bits_beside_one_in_16_of_its_type(q, D, G, dtype):
    """What the cache reads back as, in a 16-bit cache of the same type at the same shuffled places, gives the same attention.

    Each side rounds its probabilities (4 bits: to fp16, 16 bits: to dtype) and its output, and bf16 rounds the keys and
    values it is handed; scores then differ by 2^-8 of the sum of |q k| in bf16."""
    g = gen(D + G)
    Hq, Hkv, page, L = 8, 2, 16, 300
    xq, k, v = heads(L, Hq, Hkv, D, dtype, g)
    w, table = (1 + 0.2 * torch.randn(D, generator=g, device=DEV)).to(dtype), rope_table(L, D)
    pos, ids = torch.arange(L, device=DEV, dtype=torch.int32), torch.randperm(23, generator=g, device=DEV)
    at = torch.arange(L, device=DEV)
    slots = ids[at // page] * page + at % page
    c = q.kv4_cache(23, Hkv, page, D, G)
    order = torch.randperm(L, generator=g, device=DEV)              # tokens come in any order
    y = torch.empty(L, Hq, D, device=DEV, dtype=dtype)
    y[order] = q.kv4_append(xq[order], k[order], v[order], c, slots[order], pos[order], table, q_norm=w, k_norm=w)
    held = q.kv4_read(c, slots, dtype)
    exact = [t.double() for t in q.kv4_read(c, slots)]              # fp16 holds them as they are
    k16, v16 = (torch.zeros(23, Hkv, page, D, device=DEV, dtype=dtype) for _ in range(2))
    q.kv_append(None, *held, k16, v16, slots)
    more = 0.0 if dtype == F16 else U[BF16]
    pages = ids[:19].to(torch.int32)[None].contiguous()
    for n in (1, 5, L):
        args = (pages, torch.tensor([0, n], dtype=torch.int32, device=DEV), torch.tensor([L], dtype=torch.int32, device=DEV), n, L)
        got, want = q.kv4_attention(y[L - n:], c, *args), q.paged_attention(y[L - n:], k16, v16, *args)
        # the same in 64 bits, for the sizes that the roundings go by
        rows = y[L - n:].double().unflatten(1, (Hkv, -1)).transpose(0, 1).transpose(1, 2)                      # [Hkv, g, n, D]
        seen = torch.arange(L, device=DEV) <= torch.arange(L - n, L, device=DEV)[:, None]
        x = torch.where(seen, rows @ exact[0].permute(1, 2, 0)[:, None].contiguous() * D ** -0.5, -math.inf)
        dx = (rows.abs() @ exact[0].abs().permute(1, 2, 0)[:, None].contiguous() * D ** -0.5 * seen).amax(-1, keepdim=True) * (more + (D + 8) * 2.0 ** -24)
        p = torch.softmax(x, -1)
        size = (p @ exact[1].abs().transpose(0, 1)[:, None].contiguous()) * (U[F16] + U[dtype] + more + torch.exp(2 * dx) - 1 + (L + 64) * 2.0 ** -23)
        o = (p @ exact[1].transpose(0, 1)[:, None].contiguous()).abs()
        bound = (size * (1 + 2.0 ** -6) + 2 * U[dtype] * o + 2.0 ** -24).transpose(1, 2).transpose(0, 1).flatten(1, 2)
        close(got, want.double(), bound)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("G", [32, 64, 128])
def test_append_scales_halfway(q, dtype, G):
    """(hi - lo) / 15 halfway between two scales of 7 bits, to the even one, in numbers that bf16 holds too; a step of the
    range to either side."""
    rows = []
    for n in (129, 131, 133, 253, 255, 187):                       # twice a scale of 7 bits, and one: odd
        hi, lo = 8 * n, 7 * n                                       # hi + lo = 15 n
        fits = [(a, 15 * n - a) for a in range(hi, 15 * n) if all(float(torch.tensor(float(x)).to(BF16)) == x for x in (a, 15 * n - a))]
        assert fits, (n, hi, lo)
        for a, b in (fits[0], fits[len(fits) // 2], fits[-1]):
            for e in (-7, 0, 3):
                rows.append(torch.zeros(G, dtype=torch.float64))
                rows[-1][:4] = torch.tensor([float(a), -float(b), a / 2.0, -b / 4.0], dtype=torch.float64) * 2.0 ** e
                for x, y in ((a * (1 + 2.0 ** -7), b), (a, b * (1 + 2.0 ** -7))):      # not halfway any more
                    rows.append(torch.zeros(G, dtype=torch.float64))
                    rows[-1][:2] = torch.tensor([x, -y], dtype=torch.float64) * 2.0 ** e
    x = torch.stack(rows)
    ties = x[::3]
    assert torch.equal(ties[:, :2].to(dtype).double(), ties[:, :2]) and torch.equal((ties[:, 0] - ties[:, 1]) / 15 * 2, (ties[:, 0] - ties[:, 1]) * 2 / 15)
    x = x.to(dtype).to(DEV)[:, None]
    T = x.shape[0]
    c = q.kv4_cache(1, 1, T, G, G)
    before, slots = q.KV4Cache(*(t.clone() for t in c)), torch.arange(T, device=DEV)
    q.kv4_append(None, x, x, c, slots)
    check_stored(c, before, x.double(), x.double(), slots, G)
    for i in range(0, T, 3):                                        # by whole numbers: the even one of n / 2 - 1/2, n / 2 + 1/2
        n = round(float((x[i].double().max() - x[i].double().min()) / 15 * 2.0 ** 20))
        top = n >> (n.bit_length() - 8)
        assert top % 2 == 1 and n == top << (n.bit_length() - 8)
        even = (top // 2 + (top // 2) % 2) << (n.bit_length() - 7)
        assert float(c.k_scale[0, 0, i, 0, 0]) == even / 2.0 ** 20, i
