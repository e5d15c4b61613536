"""The calls around a cache of 4-bit codes without a GPU: what they refuse, before any HIP call."""
import ctypes
import math

import pytest
import torch

import bit_weight_quantized_qmm_amd as qmm

OK, INVALID, UNSUPPORTED = 0, -1, -2
P, I64, I32, F64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_double
FAKE = 0x10000   # never dereferenced: validation fails first


class Norm(ctypes.Structure):
    _fields_ = [(n, P) for n in ("q", "k", "q_out", "k_out", "q_weight", "k_weight", "positions", "rope")] + \
               [(n, I64 * 2) for n in ("q_stride", "k_stride", "q_out_stride", "k_out_stride")] + \
               [(n, I64) for n in ("T", "Hq", "Hkv", "D", "rot", "table_rows")] + [("eps", F64), ("dtype", I32), ("pairs", I32)]


class Cache(ctypes.Structure):
    _fields_ = [(n, P) for n in ("k", "v", "k_scale", "v_scale")] + [("k_stride", I64 * 3), ("v_stride", I64 * 3), ("k_scale_stride", I64 * 2),
                                                                     ("v_scale_stride", I64 * 2)] + [(n, I64) for n in ("pages", "Hkv", "page", "D", "G")]


class Append(ctypes.Structure):
    _fields_ = [(n, P) for n in ("q", "k", "v", "out", "q_norm", "k_norm", "slots", "positions", "rope")] + [("cache", Cache)] + \
               [(n, I64 * 2) for n in ("q_stride", "k_stride", "v_stride", "out_stride")] + [(n, I64) for n in ("T", "Hq", "rot", "table_rows")] + \
               [("eps", F64), ("dtype", I32), ("pairs", I32)]


class Read(ctypes.Structure):
    _fields_ = [("cache", Cache), ("slots", P), ("k_out", P), ("v_out", P), ("k_out_stride", I64 * 2), ("v_out_stride", I64 * 2), ("T", I64), ("dtype", I32)]


class Attention(ctypes.Structure):
    _fields_ = [(n, P) for n in ("q", "out", "lse", "page_table", "cu_q", "kv_lens")] + [("cache", Cache), ("workspace", P), ("workspace_bytes", I64)] + \
               [("q_stride", I64 * 2), ("out_stride", I64 * 2)] + [(n, I64) for n in ("table_stride", "T", "B", "Hq", "width", "max_q", "max_kv", "window", "sinks")] + \
               [("scale", F64), ("dtype", I32)]


def call(name, args):
    status = getattr(qmm._lib, name)(ctypes.cast(ctypes.pointer(args), P), None)
    return status, qmm._lib.qmm_last_error().decode()


def fill(a, kw):
    for k, v in kw.items():
        if isinstance(v, tuple):
            getattr(a, k)[:] = v
        else:
            setattr(a, k, v)
    return a


def cache(**kw):
    c = Cache(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, pages=3, Hkv=1, page=16, D=64, G=32)
    c.k_stride[:], c.v_stride[:], c.k_scale_stride[:], c.v_scale_stride[:] = (512, 512, 32), (512, 512, 32), (64, 64), (64, 64)
    return fill(c, kw)


def norm(**kw):
    a = Norm(q=FAKE, k=FAKE, q_out=FAKE, k_out=FAKE, positions=FAKE, rope=FAKE, T=4, Hq=2, Hkv=1, D=64, rot=64, table_rows=10, eps=1e-6)
    return fill(a, kw)


def append(c=None, **kw):
    a = Append(q=FAKE, k=FAKE, v=FAKE, out=FAKE, slots=FAKE, positions=FAKE, rope=FAKE, cache=c or cache(), T=4, Hq=2, rot=64, table_rows=10, eps=1e-6)
    return fill(a, kw)


def read(c=None, **kw):
    return fill(Read(cache=c or cache(), slots=FAKE, k_out=FAKE, v_out=FAKE, T=4), kw)


def attention(c=None, **kw):
    a = Attention(q=FAKE, out=FAKE, page_table=FAKE, cu_q=FAKE, kv_lens=FAKE, cache=c or cache(), T=4, B=1, Hq=2, width=2, max_q=4, max_kv=32, scale=0.125, table_stride=2)
    a.q_stride[:], a.out_stride[:] = (128, 64), (128, 64)
    return fill(a, kw)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(Hq=-1), INVALID), (dict(Hkv=-1), INVALID), (dict(D=0), INVALID), (dict(rot=3), INVALID), (dict(rot=80), INVALID), (dict(rot=-2), INVALID),
    (dict(dtype=2), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID), (dict(eps=1e300), INVALID), (dict(q=None), INVALID), (dict(q_out=None), INVALID),
    (dict(k=None), INVALID), (dict(k_out=None), INVALID), (dict(rope=None), INVALID), (dict(positions=None), INVALID), (dict(table_rows=0), INVALID),
    (dict(q_weight=FAKE + 2), INVALID), (dict(k_weight=FAKE + 8), INVALID), (dict(rope=FAKE + 4), INVALID), (dict(D=40, rot=0), UNSUPPORTED), (dict(D=272), UNSUPPORTED),
    (dict(rot=24), UNSUPPORTED), (dict(Hq=65536), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED), (dict(T=1 << 28, Hq=64), UNSUPPORTED)], ids=str)
def test_norm_refuses(kw, want):
    status, text = call("qmm_qk_norm", norm(**kw))
    assert status == want and "qmm_qk_norm" in text


CACHES = [(dict(Hkv=0), INVALID), (dict(page=0), INVALID), (dict(pages=0), INVALID), (dict(D=0), INVALID), (dict(G=0), INVALID), (dict(D=80, G=32), INVALID),
          (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k_scale=None), INVALID), (dict(v_scale=None), INVALID), (dict(k=FAKE + 8), INVALID), (dict(v=FAKE + 4), INVALID),
          (dict(k_scale=FAKE + 2), INVALID), (dict(k_stride=(512, 512, 24)), INVALID), (dict(v_stride=(520, 512, 32)), INVALID), (dict(k_scale_stride=(63, 64)), INVALID),
          (dict(G=16), UNSUPPORTED), (dict(D=48, G=48), UNSUPPORTED), (dict(D=384, G=128), UNSUPPORTED), (dict(D=256, G=256), UNSUPPORTED), (dict(pages=1 << 28), UNSUPPORTED),
          (dict(page=(1 << 20) + 1, pages=1), UNSUPPORTED), (dict(k_stride=(1 << 30, 1 << 30, 1 << 25)), UNSUPPORTED), (dict(v_stride=(512, 512, -32)), UNSUPPORTED)]


@pytest.mark.parametrize("kw,want", CACHES, ids=str)
def test_a_cache_that_does_not_fit_is_refused(kw, want):
    for name, make in (("qmm_kv4_append", append), ("qmm_kv4_read", read), ("qmm_kv4_attention", attention)):
        a = make(cache(**kw))
        if name == "qmm_kv4_append":
            a.rot = 0
        if name == "qmm_kv4_attention" and kw.get("page"):
            a.workspace, a.workspace_bytes = FAKE, 1 << 40
        status, text = call(name, a)
        assert status == want and name in text, name


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(Hq=-1), INVALID), (dict(rot=3), INVALID), (dict(rot=66), INVALID), (dict(dtype=2), INVALID), (dict(q=None), INVALID), (dict(out=None), INVALID),
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(slots=None), INVALID), (dict(rope=None), INVALID), (dict(positions=None), INVALID), (dict(table_rows=0), INVALID),
    (dict(q_norm=FAKE + 2), INVALID), (dict(k_norm=FAKE + 2), INVALID), (dict(eps=-1.0), INVALID), (dict(rot=8), UNSUPPORTED), (dict(Hq=65535), UNSUPPORTED),
    (dict(T=1 << 31), UNSUPPORTED), (dict(T=(1 << 31) - 1, Hq=64), UNSUPPORTED)], ids=str)
def test_append_refuses(kw, want):
    status, text = call("qmm_kv4_append", append(**kw))
    assert status == want and "qmm_kv4_append" in text


@pytest.mark.parametrize("kw,want", [(dict(T=-1), INVALID), (dict(dtype=2), INVALID), (dict(slots=None), INVALID), (dict(k_out=None), INVALID), (dict(v_out=None), INVALID),
                                     (dict(T=1 << 31), UNSUPPORTED), (dict(T=1 << 30), UNSUPPORTED)], ids=str)
def test_read_refuses(kw, want):
    status, text = call("qmm_kv4_read", read(**kw))
    assert status == want and "qmm_kv4_read" in text


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(B=-1), INVALID), (dict(Hq=0), INVALID), (dict(width=0), INVALID), (dict(max_q=0), INVALID), (dict(max_kv=-1), INVALID),
    (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=math.inf), INVALID), (dict(scale=math.nan), INVALID),
    (dict(scale=1e300), INVALID), (dict(dtype=2), INVALID), (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(page_table=None), INVALID), (dict(cu_q=None), INVALID),
    (dict(kv_lens=None), INVALID), (dict(q=FAKE + 8), INVALID), (dict(out=FAKE + 2), INVALID), (dict(q_stride=(100, 64)), INVALID), (dict(out_stride=(128, 60)), INVALID),
    (dict(max_kv=100000), INVALID),                                 # needs a workspace
    (dict(max_kv=100000, workspace=FAKE, workspace_bytes=64), INVALID), (dict(max_kv=100000, workspace=FAKE + 4, workspace_bytes=1 << 40), INVALID),
    (dict(T=1 << 30, max_q=1 << 30), UNSUPPORTED)], ids=str)
def test_attention_refuses(kw, want):
    status, text = call("qmm_kv4_attention", attention(**kw))
    assert status == want and "qmm_kv4_attention" in text
    assert call("qmm_kv4_attention", attention(cache(Hkv=3), Hq=4))[0] == INVALID


@pytest.mark.parametrize("kw", [dict(B=1 << 23, max_kv=64, max_q=40, T=1 << 20, Hq=16), dict(B=1 << 24, max_q=1, T=1 << 20, Hq=1),
                                dict(B=(1 << 31) - 65536, max_q=1 << 20, T=1 << 20, Hq=64)], ids=str)
def test_attention_refuses_more_threads_than_a_launch_has(kw):
    assert call("qmm_kv4_attention", attention(workspace=FAKE, workspace_bytes=1 << 62, **kw))[0] == UNSUPPORTED


def test_nothing_to_do():
    assert call("qmm_qk_norm", norm(T=0, q=None))[0] == OK and call("qmm_qk_norm", norm(Hq=0, Hkv=0, q=None, k=None))[0] == OK
    assert call("qmm_kv4_append", append(T=0, q=None, k=None))[0] == OK and call("qmm_kv4_read", read(T=0, slots=None))[0] == OK
    assert call("qmm_kv4_attention", attention(T=0))[0] == OK and call("qmm_kv4_attention", attention(B=0))[0] == OK
    for name in ("qmm_qk_norm", "qmm_kv4_append", "qmm_kv4_read", "qmm_kv4_attention"):
        assert getattr(qmm._lib, name)(None, None) == INVALID
    assert qmm._lib.qmm_kv4_attention_workspace(None) == 0


def test_attention_workspace():
    need = lambda c=None, **kw: qmm._lib.qmm_kv4_attention_workspace(ctypes.cast(ctypes.pointer(attention(c, **kw)), P))
    assert need(max_q=1, max_kv=100) == 0 and need(T=0) == 0 and need(cache(G=16)) == 0
    one = need(max_q=1, T=1, max_kv=100000)
    assert one > 0 and one % (2 * (64 + 1) * 4) == 0       # whole splits of T * Hq rows of D + 1 floats
    assert need(max_q=1, T=1, max_kv=100000, window=100, sinks=4) == 0     # a short window is one stretch
    assert need(max_q=1, T=1, max_kv=100000, window=100, sinks=90000) > 0


CPU = [(lambda x: qmm.qk_norm(x, x), ValueError), (lambda x: qmm.qk_norm(x.float(), x), TypeError), (lambda x: qmm.qk_norm(x, None), TypeError),
       (lambda x: qmm.kv4_append(None, x, x, (x, x, x, x), x), ValueError), (lambda x: qmm.kv4_append(None, x.int(), x, (x, x, x, x), x), TypeError),
       (lambda x: qmm.kv4_read((x, x, x, x), x), TypeError), (lambda x: qmm.kv4_read(qmm.kv4_cache(1, 1, 16, 64, device="cpu"), x), ValueError),
       (lambda x: qmm.kv4_read(qmm.kv4_cache(1, 1, 16, 64, device="cpu"), x, torch.float32), TypeError), (lambda x: qmm.kv4_attention(x, (x,) * 4, x, x, x, 1, 1), ValueError),
       (lambda x: qmm.kv4_attention([1], (x,) * 4, x, x, x, 1, 1), TypeError)]


@pytest.mark.parametrize("i", range(len(CPU)))
def test_binding_refuses_cpu_tensors(i):
    """Tensors of the host, of other types and no tensors at all: an error of Python, no call."""
    f, kind = CPU[i]
    with pytest.raises(kind):
        f(torch.zeros(2, 64, dtype=torch.float16))


def test_binding_hands_on_an_error_of_pairs():
    x = torch.zeros(2, 1, 64, dtype=torch.float16)
    for f in (lambda p: qmm.qk_norm(x, x, pairs=p), lambda p: qmm.kv4_append(None, x, x, x, x, pairs=p)):
        with pytest.raises(RuntimeError, match="ambiguous"):
            f(torch.tensor([True, False]))


def test_an_empty_cache():
    c = qmm.kv4_cache(3, 2, 16, 192, device="cpu")
    assert c.k.shape == c.v.shape == (3, 2, 16, 96) and c.k_scale.shape == c.v_scale.shape == (3, 2, 16, 3, 2) and isinstance(c, qmm.KV4Cache)
    assert qmm.kv4_cache(1, 1, 1, 256, device="cpu").k_scale.shape[3] == 2 and qmm.kv4_cache(1, 1, 1, 96, device="cpu").k_scale.shape[3] == 3
    for D, G in ((80, None), (96, 64), (64, 16), (512, 128), (0, None)):
        with pytest.raises(ValueError):
            qmm.kv4_cache(1, 1, 16, D, G, device="cpu")
