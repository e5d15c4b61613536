"""The decoder-layer calls without a GPU: what they refuse, before any HIP call, and the
arithmetic of the planner's page division."""
import ctypes
import math
import subprocess
import sys

import pytest
import torch

import bit_weight_quantized_qmm_amd as qmm

OK, INVALID, UNSUPPORTED = 0, -1, -2
P, I64, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
FAKE = 0x10000   # never dereferenced: validation fails first


class Linear(ctypes.Structure):
    _fields_ = [(n, P) for n in ("X", "wq", "s", "z", "Y", "bias", "mul", "residual", "workspace")] + \
               [(n, I64) for n in ("workspace_bytes", "M", "K", "N", "G")] + [("bits", I32), ("act", I32)]


class Append(ctypes.Structure):
    _fields_ = [(n, P) for n in ("q", "k", "v", "out", "k_cache", "v_cache", "slots", "positions", "rope", "k_scale", "v_scale")] + \
               [(n, I64 * 2) for n in ("q_stride", "k_stride", "v_stride", "out_stride")] + \
               [(n, I64 * 3) for n in ("k_cache_stride", "v_cache_stride")] + \
               [(n, I64) for n in ("T", "Hq", "Hkv", "D", "rot", "table_rows", "page", "pages")] + \
               [(n, I32) for n in ("dtype", "cache_dtype", "pairs")]


class Attention(ctypes.Structure):
    _fields_ = [(n, P) for n in ("q", "k_cache", "v_cache", "out", "lse", "page_table", "cu_q", "kv_lens", "k_scale", "v_scale", "workspace")] + \
               [("workspace_bytes", I64), ("q_stride", I64 * 2), ("out_stride", I64 * 2), ("k_cache_stride", I64 * 3),
                ("v_cache_stride", I64 * 3)] + \
               [(n, I64) for n in ("table_stride", "T", "B", "Hq", "Hkv", "D", "page", "pages", "width", "max_q", "max_kv", "window")] + \
               [("scale", ctypes.c_double), ("dtype", I32), ("cache_dtype", I32)]


def lib():
    return qmm._lib


def call(name, args):
    fn = getattr(lib(), name)
    status = fn(ctypes.cast(ctypes.pointer(args), P), None)
    return status, lib().qmm_last_error().decode()


def linear(**kw):
    a = Linear(X=FAKE, wq=FAKE, s=FAKE, Y=FAKE, M=1, K=128, N=64, G=64, bits=4)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def append(**kw):
    a = Append(q=FAKE, k=FAKE, v=FAKE, out=FAKE, k_cache=FAKE, v_cache=FAKE, slots=FAKE, positions=FAKE, rope=FAKE, T=4, Hq=2, Hkv=1, D=64,
               rot=64, table_rows=10, page=16, pages=3)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def attention(**kw):
    a = Attention(q=FAKE, k_cache=FAKE, v_cache=FAKE, out=FAKE, page_table=FAKE, cu_q=FAKE, kv_lens=FAKE, T=4, B=1, Hq=2, Hkv=1, D=64, page=16,
                  pages=3, width=2, max_q=4, max_kv=32, scale=0.125, table_stride=2)
    a.q_stride[:], a.out_stride[:] = (128, 64), (128, 64)
    a.k_cache_stride[:], a.v_cache_stride[:] = (1024, 1024, 64), (1024, 1024, 64)
    for k, v in kw.items():
        if isinstance(v, tuple):
            getattr(a, k)[:] = v
        else:
            setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw", [dict(act=5), dict(act=-1), dict(X=None), dict(wq=None), dict(s=None), dict(Y=None), dict(bits=0), dict(bits=9),
                                dict(K=100), dict(G=48), dict(G=0), dict(M=0), dict(N=0), dict(M=16, K=16384),
                                dict(M=16, K=16384, workspace=FAKE, workspace_bytes=100),
                                dict(M=16, K=16384, workspace=FAKE + 4, workspace_bytes=1 << 30)], ids=str)
def test_linear_refuses(kw):
    status, text = call("qmm_linear", linear(**kw))
    assert status == INVALID and "qmm_linear" in text


SHIM = """
static int calls;
int hipGetDevice(int *d) { (void)d; ++calls; return 100; }
int hipDeviceGetAttribute(int *v, int a, int d) { (void)v, (void)a, (void)d; ++calls; return 100; }
int made(void) { return calls; }
"""
PLAN = """
import ctypes, sys
shim = ctypes.CDLL(sys.argv[1], ctypes.RTLD_GLOBAL)      # its symbols come before the HIP library's
lib = ctypes.CDLL(sys.argv[2])
args = ctypes.create_string_buffer(bytes.fromhex(sys.argv[3]))
lib.qmm_linear_workspace.restype = ctypes.c_int64
print(lib.qmm_linear_workspace(args), lib.qmm_linear(args, None), shim.made())
"""


def test_linear_plans_without_hip_calls(tmp_path):
    """The workspace follows from the sizes alone and a missing one is refused before any HIP call."""
    (tmp_path / "shim.c").write_text(SHIM)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(tmp_path / "shim.so"), str(tmp_path / "shim.c")], check=True)
    for M, K, N in (100, 32768, 64), (300, 4096, 2000):
        text = subprocess.run([sys.executable, "-c", PLAN, str(tmp_path / "shim.so"), qmm.library_path(), bytes(linear(M=M, K=K, N=N)).hex()], check=True,
                              capture_output=True, text=True, timeout=120).stdout
        need, status, calls = map(int, text.split())
        assert need > 0 and status == INVALID and calls == 0


def test_linear_workspace():
    fn = lib().qmm_linear_workspace
    need = lambda **kw: fn(ctypes.cast(ctypes.pointer(linear(**kw)), P))
    assert need(M=1, K=32768) == 0 and need(M=8, K=4096) == 0 and need(M=4, K=100) == 0
    assert need(M=100, K=64) == 0 and need(M=2048, K=4096, N=4096) == 0        # one step of K; a grid that fills the CUs
    for M, K, N in (16, 28672, 8192), (100, 32768, 64):                        # streamed; K cut because one tile would leave CUs idle
        bytes_ = need(M=M, K=K, N=N)
        assert bytes_ > 0 and bytes_ % (M * N * 4) == 0
    assert fn(None) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(Hq=-1), INVALID), (dict(Hkv=0), INVALID), (dict(page=0), INVALID), (dict(pages=0), INVALID),
    (dict(D=63), INVALID), (dict(D=0), INVALID), (dict(rot=3), INVALID), (dict(rot=66), INVALID), (dict(rot=-2), INVALID),
    (dict(dtype=2), INVALID), (dict(dtype=7), INVALID), (dict(dtype=0, cache_dtype=1), INVALID), (dict(cache_dtype=3), INVALID),
    (dict(cache_dtype=2), INVALID),                                # no scales
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k_cache=None), INVALID),
    (dict(v_cache=None), INVALID), (dict(slots=None), INVALID), (dict(rope=None), INVALID), (dict(positions=None), INVALID),
    (dict(table_rows=0), INVALID), (dict(Hq=65536), UNSUPPORTED), (dict(pages=1 << 28), UNSUPPORTED), (dict(T=1 << 30), UNSUPPORTED)], ids=str)
def test_append_refuses(kw, want):
    status, text = call("qmm_kv_append", append(**kw))
    assert status == want and "qmm_kv_append" in text


def test_append_of_nothing():
    assert call("qmm_kv_append", append(T=0, q=None, k=None))[0] == OK
    assert lib().qmm_kv_append(None, None) == INVALID and lib().qmm_linear(None, None) == INVALID and lib().qmm_paged_attention(None, None) == INVALID


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(B=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(Hq=3, Hkv=2), INVALID), (dict(page=0), INVALID),
    (dict(pages=0), INVALID), (dict(width=0), INVALID), (dict(max_q=0), INVALID), (dict(max_kv=-1), INVALID), (dict(window=-1), INVALID),
    (dict(scale=-1.0), INVALID), (dict(scale=math.inf), INVALID), (dict(scale=math.nan), INVALID), (dict(scale=1e300), INVALID),
    (dict(dtype=2), INVALID), (dict(cache_dtype=1), INVALID), (dict(cache_dtype=2), INVALID), (dict(q=None), INVALID), (dict(k_cache=None), INVALID),
    (dict(v_cache=None), INVALID), (dict(out=None), INVALID), (dict(page_table=None), INVALID), (dict(cu_q=None), INVALID), (dict(kv_lens=None), INVALID),
    (dict(q=FAKE + 8), INVALID), (dict(out=FAKE + 2), INVALID), (dict(q_stride=(100, 64)), INVALID), (dict(v_cache_stride=(1024, 1024, 60)), INVALID),
    (dict(max_kv=100000), INVALID),                                 # needs a workspace
    (dict(max_kv=100000, workspace=FAKE, workspace_bytes=64), INVALID),
    (dict(D=40), UNSUPPORTED), (dict(D=272), UNSUPPORTED), (dict(k_cache_stride=(1 << 30, 1 << 30, 1 << 25)), UNSUPPORTED),
    (dict(T=1 << 30, max_q=1 << 30), UNSUPPORTED), (dict(page=1 << 21), UNSUPPORTED)], ids=str)
def test_attention_refuses(kw, want):
    status, text = call("qmm_paged_attention", attention(**kw))
    assert status == want and "qmm_paged_attention" in text


@pytest.mark.parametrize("kw", [
    dict(B=1 << 23, max_kv=64, max_q=40, T=1 << 20, Hq=16),            # 2^23 blocks of 512 threads
    dict(B=1 << 24, max_q=1, T=1 << 20, Hq=1, Hkv=1),                  # 2^24 blocks of 256
    dict(B=1 << 14, max_q=1 << 17, T=1 << 17, Hq=2, Hkv=1, max_kv=64),
    dict(B=1 << 22, max_q=1, T=1 << 20, Hq=16, Hkv=1, max_kv=12000, width=750),           # 2^23 blocks, two shares of the keys; 2^24 of the join
    dict(B=(1 << 31) - 65536, max_q=1 << 20, T=1 << 20, Hq=64, Hkv=64)], ids=str)
def test_attention_refuses_more_threads_than_a_launch_has(kw):
    a = attention(**kw)
    a.workspace, a.workspace_bytes = FAKE, 1 << 62
    fn = lib().qmm_paged_attention
    assert fn(ctypes.cast(ctypes.pointer(a), P), None) == UNSUPPORTED


def test_append_refuses_more_threads_than_a_launch_has():
    a = append(T=1 << 24, D=64, rot=2, Hq=16, Hkv=1)                   # single elements: 2^29 units for each pair of 18 heads
    assert call("qmm_kv_append", a)[0] == UNSUPPORTED


def test_attention_of_nothing():
    assert call("qmm_paged_attention", attention(T=0))[0] == OK
    assert call("qmm_paged_attention", attention(B=0))[0] == OK


def test_attention_workspace():
    fn = lib().qmm_paged_attention_workspace
    need = lambda **kw: fn(ctypes.cast(ctypes.pointer(attention(**kw)), P))
    assert need(max_q=1, max_kv=100) == 0 and need(T=0) == 0 and need(D=40) == 0 and fn(None) == 0
    one = need(max_q=1, T=1, max_kv=100000)
    assert one > 0 and one % (2 * (64 + 1) * 4) == 0       # whole splits of T * Hq rows of D + 1 floats


@pytest.mark.parametrize("page", [1, 2, 3, 5, 7, 16, 17, 48, 100, 255, 256, 1000, 65536, (1 << 20) - 1, 1 << 20])
def test_page_division(page):
    """key / page as the kernels compute it: one product and a shift."""
    lg = max(0, (page - 1).bit_length())
    mul, sh = (1 << (31 + lg)) // page + 1, 31 + lg
    assert mul < 1 << 32
    keys = {0, 1, (1 << 31) - 1, (1 << 31) - 2}
    for q in list(range(0, 2000)) + [(1 << 31) // page - 1, (1 << 31) // page]:
        keys.update(q * page + r for r in (-1, 0, 1))
    for k in keys:
        if 0 <= k < 1 << 31:
            assert k * mul >> sh == k // page


CPU = [(lambda x: qmm.linear(x, x, x, None, 4, 32), ValueError), (lambda x: qmm.linear(x.float(), x, x, None, 4, 32), TypeError),
       (lambda x: qmm.linear(x, x, x, None, 4, 32, act="swish"), ValueError), (lambda x: qmm.linear(None, x, x, None, 4, 32), TypeError),
       (lambda x: qmm.linear(x, x, x, None, 4, 0), ValueError), (lambda x: qmm.linear(x, x, x, None, "4", 32), TypeError),
       (lambda x: qmm.linear(x[0], x, x, None, 4, 32), ValueError), (lambda x: qmm.kv_append(None, x, x, x, x, x), ValueError),
       (lambda x: qmm.kv_append(None, x.int(), x, x, x, x), TypeError), (lambda x: qmm.paged_attention(x, x, x, x, x, x, 1, 1), ValueError),
       (lambda x: qmm.paged_attention(x.float(), x, x, x, x, x, 1, 1), TypeError), (lambda x: qmm.paged_attention(x, x, [1], x, x, x, 1, 1), TypeError)]


def test_binding_hands_on_an_error_of_pairs():
    """A flag without a truth value (an array of several) ends the call with its own error."""
    x = torch.zeros(2, 1, 64, dtype=torch.float16)
    with pytest.raises(RuntimeError, match="ambiguous"):
        qmm.kv_append(None, x, x, x, x, x, pairs=torch.tensor([True, False]))


@pytest.mark.parametrize("i", range(len(CPU)))
def test_binding_refuses_cpu_tensors(i):
    """Tensors of the host, of other types and no tensors at all: an error of Python, no call."""
    f, kind = CPU[i]
    with pytest.raises(kind):
        f(torch.zeros(2, 64, dtype=torch.float16))
