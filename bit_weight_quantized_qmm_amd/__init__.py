"""k-bit weight-quantized matmul on AMD MI355X (gfx950): Python binding of libqmm.so.

This module only marshals arguments: it checks tensor dtypes, shapes and
devices, passes raw device pointers and the current HIP stream to the C ABI
(``include/qmm.h``) and raises :class:`QmmError` on a non-zero status.  Every
step of the computation runs in the library's HIP kernels; there is no
fallback.  Importing the package fails loudly if ``libqmm.so`` has not been
built (``python bit_weight_quantized_qmm_amd/_build.py``).

PyTorch is used for device memory and streams only.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
from typing import NamedTuple

import torch

from ._build import BINDING, LIBRARY

__all__ = ["QmmError", "packed_bytes", "pack", "pack_signed", "unpack", "gemv", "gemv_grouped", "gemv_lut", "gemm", "gemm_fp", "FP4_E2M1",
           "FP8_E4M3", "FP6_E3M2", "FP6_E2M3", "FP3_E1M1", "FP5_E2M2", "FP7_E3M3", "gemm_w4a8", "gemm_wka8", "quantize", "linear", "kv_append",
           "paged_attention", "qk_norm", "KV4Cache", "kv4_cache", "kv4_append", "kv4_read", "kv4_attention", "probe_read", "probe_mfma", "library_path", "SYMBOLS"]

SYMBOLS = ("qmm_packed_bytes", "qmm_pack", "qmm_pack_signed", "qmm_unpack", "qmm_gemv", "qmm_gemv_grouped", "qmm_gemv_lut", "qmm_gemm", "qmm_gemm_fp", "qmm_gemm_w4a8", "qmm_gemm_wka8",
           "qmm_quantize", "qmm_linear", "qmm_linear_workspace", "qmm_kv_append", "qmm_paged_attention", "qmm_paged_attention_workspace",
           "qmm_qk_norm", "qmm_kv4_append", "qmm_kv4_read", "qmm_kv4_attention", "qmm_kv4_attention_workspace", "qmm_status_string", "qmm_last_error", "qmm_last_hip_error", "qmm_probe_read",
           "qmm_probe_mfma")


class QmmError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} (status {status})")
        self.status = status


def _load():
    if not os.path.exists(LIBRARY):
        raise ImportError(f"{LIBRARY} is missing: build it first (python bit_weight_quantized_qmm_amd/_build.py)")
    lib = ctypes.CDLL(LIBRARY)
    P, I64, INT = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    sig = {
        "qmm_packed_bytes": ([I64, I64, INT], ctypes.c_size_t),
        "qmm_pack": ([P, P, I64, I64, INT, P], INT),
        "qmm_pack_signed": ([P, P, I64, I64, INT, P], INT),
        "qmm_unpack": ([P, P, I64, I64, INT, P], INT),
        "qmm_gemv": ([P, P, P, P, P, I64, I64, I64, INT, I64, P], INT),
        "qmm_gemm": ([P, P, P, P, P, I64, I64, I64, INT, I64, P], INT),
        "qmm_gemv_lut": ([P, P, P, P, P, I64, I64, I64, INT, I64, P], INT),
        "qmm_gemv_grouped": ([P, INT, I64, I64, P], INT),
        "qmm_gemm_fp": ([P, P, P, P, I64, I64, I64, INT, I64, P], INT),
        "qmm_gemm_w4a8": ([P, P, P, P, P, P, P, I64, I64, I64, I64, P], INT),
        "qmm_gemm_wka8": ([P, P, P, P, P, P, P, I64, I64, I64, INT, I64, P], INT),
        "qmm_quantize": ([P, P, P, P, I64, I64, INT, I64, P], INT),
        "qmm_linear": ([P, P], INT),
        "qmm_linear_workspace": ([P], I64),
        "qmm_kv_append": ([P, P], INT),
        "qmm_paged_attention": ([P, P], INT),
        "qmm_paged_attention_workspace": ([P], I64),
        "qmm_qk_norm": ([P, P], INT),
        "qmm_kv4_append": ([P, P], INT),
        "qmm_kv4_read": ([P, P], INT),
        "qmm_kv4_attention": ([P, P], INT),
        "qmm_kv4_attention_workspace": ([P], I64),
        "qmm_status_string": ([INT], ctypes.c_char_p),
        "qmm_last_error": ([], ctypes.c_char_p),
        "qmm_last_hip_error": ([], ctypes.c_char_p),
        "qmm_probe_read": ([P, ctypes.c_uint64, P, INT, P], INT),
        "qmm_probe_mfma": ([P, INT, INT, INT, P], INT),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


_lib = _load()


def library_path() -> str:
    return LIBRARY


def _check(status: int):
    if status != 0:
        raise QmmError(status, _lib.qmm_last_error().decode() or _lib.qmm_status_string(status).decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need(t, name, dtype, shape=None, device=None):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def packed_bytes(K: int, N: int, bits: int) -> int:
    return int(_lib.qmm_packed_bytes(K, N, bits))


def pack(codes: torch.Tensor, bits: int, out: torch.Tensor | None = None) -> torch.Tensor:
    """uint8 codes [K, N] -> packed stream as int32 [N, K*bits/32] (bit pattern)."""
    _need(codes, "codes", torch.uint8)
    K, N = codes.shape
    if out is None:
        out = torch.empty((N, K * bits // 32), dtype=torch.int32, device=codes.device)
    _need(out, "out", torch.int32, (N, K * bits // 32), codes.device)
    _check(_lib.qmm_pack(_ptr(codes), _ptr(out), K, N, bits, _stream(codes.device)))
    return out


def pack_signed(codes: torch.Tensor, bits: int, out: torch.Tensor | None = None) -> torch.Tensor:
    """int8 two's-complement codes [K, N] -> packed stream (offset-binary: q + 2^(bits-1))."""
    _need(codes, "codes", torch.int8)
    K, N = codes.shape
    if out is None:
        out = torch.empty((N, K * bits // 32), dtype=torch.int32, device=codes.device)
    _need(out, "out", torch.int32, (N, K * bits // 32), codes.device)
    _check(_lib.qmm_pack_signed(_ptr(codes), _ptr(out), K, N, bits, _stream(codes.device)))
    return out


def unpack(wq: torch.Tensor, K: int, N: int, bits: int, out: torch.Tensor | None = None) -> torch.Tensor:
    """Packed stream [N, K*bits/32] -> uint8 codes [K, N] through the kernels' register unpack."""
    _need(wq, "wq", torch.int32, (N, K * bits // 32))
    if out is None:
        out = torch.empty((K, N), dtype=torch.uint8, device=wq.device)
    _need(out, "out", torch.uint8, (K, N), wq.device)
    _check(_lib.qmm_unpack(_ptr(wq), _ptr(out), K, N, bits, _stream(wq.device)))
    return out


def _product(fn, X, wq, s, z, bits, G, out):
    _need(X, "X", torch.float16)
    M, K = X.shape
    N = s.shape[0] if s.dim() == 2 else -1
    _need(wq, "wq", torch.int32, (N, K * bits // 32), X.device)
    _need(s, "s", torch.float16, (N, K // G), X.device)
    if z is not None:
        _need(z, "z", torch.float16, (N, K // G), X.device)
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=X.device)
    _need(out, "out", torch.float16, (M, N), X.device)
    _check(fn(_ptr(X), _ptr(wq), _ptr(s), _ptr(z), _ptr(out), M, K, N, bits, G, _stream(X.device)))
    return out


def gemv(X, wq, s, z, bits: int, G: int, out=None) -> torch.Tensor:
    """Y [M, N] fp16 = X [M, K] fp16 . dequant(wq); 1 <= M <= 16."""
    return _product(_lib.qmm_gemv, X, wq, s, z, bits, G, out)


class _Problem(ctypes.Structure):
    _fields_ = [("X", ctypes.c_void_p), ("wq", ctypes.c_void_p), ("s", ctypes.c_void_p), ("z", ctypes.c_void_p),
                ("Y", ctypes.c_void_p), ("N", ctypes.c_int64), ("bits", ctypes.c_int)]


def gemv_grouped(problems, G: int, outs=None):
    """Several M = 1 products in one launch.  problems: sequence of (X [1, K], wq, s, z or None,
    bits) sharing K; returns the list of Y [1, N] (or fills outs)."""
    problems = list(problems)
    if not problems:
        raise ValueError("no problems")
    K = problems[0][0].shape[1]
    arr = (_Problem * len(problems))()
    res = []
    for i, (X, wq, s, z, bits) in enumerate(problems):
        _need(X, "X", torch.float16, (1, K))
        N = s.shape[0]
        _need(wq, "wq", torch.int32, (N, K * bits // 32), X.device)
        _need(s, "s", torch.float16, (N, K // G), X.device)
        if z is not None:
            _need(z, "z", torch.float16, (N, K // G), X.device)
        Y = outs[i] if outs is not None else torch.empty((1, N), dtype=torch.float16, device=X.device)
        _need(Y, "out", torch.float16, (1, N), X.device)
        arr[i] = _Problem(X.data_ptr(), wq.data_ptr(), s.data_ptr(), 0 if z is None else z.data_ptr(), Y.data_ptr(),
                          N, bits)
        res.append(Y)
    _check(_lib.qmm_gemv_grouped(ctypes.cast(arr, ctypes.c_void_p), len(problems), K, G,
                                 _stream(problems[0][0].device)))
    return res


def gemv_lut(X, wq, s, z, bits: int, G: int, out=None) -> torch.Tensor:
    """Y [1, N] fp16 = X [1, K] fp16 . dequant(wq) for 1-bit codes by table lookup (K <= 8192)."""
    return _product(_lib.qmm_gemv_lut, X, wq, s, z, bits, G, out)


def gemm(X, wq, s, z, bits: int, G: int, out=None) -> torch.Tensor:
    """Y [M, N] fp16 = X [M, K] fp16 . dequant(wq); any M (f16 MFMA path)."""
    return _product(_lib.qmm_gemm, X, wq, s, z, bits, G, out)


FP4_E2M1, FP8_E4M3, FP6_E3M2, FP6_E2M3, FP3_E1M1, FP5_E2M2, FP7_E3M3 = 0, 1, 2, 3, 4, 5, 6
_FP_BITS = {FP4_E2M1: 4, FP8_E4M3: 8, FP6_E3M2: 6, FP6_E2M3: 6, FP3_E1M1: 3, FP5_E2M2: 5, FP7_E3M3: 7}


def gemm_fp(X, wq, s, fmt: int, G: int, out=None) -> torch.Tensor:
    """Y [M, N] fp16 = X . (value(q) s) for floating-point codes (FP4_E2M1, FP8_E4M3,
    FP6_E3M2, FP6_E2M3, FP3_E1M1, FP5_E2M2 or FP7_E3M3)."""
    if fmt not in _FP_BITS:
        raise ValueError(f"unknown float code format {fmt}: expected one of {sorted(_FP_BITS)}")
    _need(X, "X", torch.float16)
    M, K = X.shape
    N = s.shape[0]
    _need(wq, "wq", torch.int32, (N, K * _FP_BITS[fmt] // 32), X.device)
    _need(s, "s", torch.float16, (N, K // G), X.device)
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=X.device)
    _need(out, "out", torch.float16, (M, N), X.device)
    _check(_lib.qmm_gemm_fp(_ptr(X), _ptr(wq), _ptr(s), _ptr(out), M, K, N, fmt, G, _stream(X.device)))
    return out


def gemm_w4a8(Xq, sx, wq, s, z, G: int, out=None, acc_out=None) -> torch.Tensor:
    """Y [M, N] fp16 for int8 activations Xq [M, K] with per-token fp16 scales sx [M] and
    4-bit weights; acc_out (int32 [M, K/G, N]) optionally receives the exact group sums."""
    return _int8_product(False, Xq, sx, wq, s, z, 4, G, out, acc_out)


def gemm_wka8(Xq, sx, wq, s, z, bits: int, G: int, out=None, acc_out=None) -> torch.Tensor:
    """As gemm_w4a8 for bits-bit weights, bits in 1..8 (8: W8A8)."""
    return _int8_product(True, Xq, sx, wq, s, z, bits, G, out, acc_out)


def _int8_product(any_bits: bool, Xq, sx, wq, s, z, bits: int, G: int, out, acc_out) -> torch.Tensor:
    _need(Xq, "Xq", torch.int8)
    M, K = Xq.shape
    N = s.shape[0]
    _need(sx, "sx", torch.float16, (M,), Xq.device)
    _need(wq, "wq", torch.int32, (N, K * bits // 32), Xq.device)
    _need(s, "s", torch.float16, (N, K // G), Xq.device)
    if z is not None:
        _need(z, "z", torch.float16, (N, K // G), Xq.device)
    if acc_out is not None:
        _need(acc_out, "acc_out", torch.int32, (M, K // G, N), Xq.device)
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=Xq.device)
    _need(out, "out", torch.float16, (M, N), Xq.device)
    ptrs = (_ptr(Xq), _ptr(sx), _ptr(wq), _ptr(s), _ptr(z), _ptr(out), _ptr(acc_out))
    if any_bits:
        _check(_lib.qmm_gemm_wka8(*ptrs, M, K, N, bits, G, _stream(Xq.device)))
    else:
        _check(_lib.qmm_gemm_w4a8(*ptrs, M, K, N, G, _stream(Xq.device)))
    return out


def quantize(W, bits: int, G: int, codes=None, s=None, z=None):
    """(codes uint8 [K, N], s fp16 [N, K/G], z fp16 [N, K/G]) for fp16 weights W [K, N]."""
    _need(W, "W", torch.float16)
    K, N = W.shape
    if codes is None:
        codes = torch.empty((K, N), dtype=torch.uint8, device=W.device)
    if s is None:
        s = torch.empty((N, K // G), dtype=torch.float16, device=W.device)
    if z is None:
        z = torch.empty((N, K // G), dtype=torch.float16, device=W.device)
    _need(codes, "codes", torch.uint8, (K, N), W.device)
    _need(s, "s", torch.float16, (N, K // G), W.device)
    _need(z, "z", torch.float16, (N, K // G), W.device)
    _check(_lib.qmm_quantize(_ptr(W), _ptr(codes), _ptr(s), _ptr(z), K, N, bits, G, _stream(W.device)))
    return codes, s, z


def _load_binding():
    """The C++ side of the calls below: it checks the tensors, fills the library's argument blocks
    and makes the call."""
    if not os.path.exists(BINDING):
        raise ImportError(f"{BINDING} is missing: build it first (python bit_weight_quantized_qmm_amd/_build.py)")
    spec = importlib.util.spec_from_file_location("_binding", BINDING)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    entry = (_lib.qmm_linear, _lib.qmm_linear_workspace, _lib.qmm_kv_append, _lib.qmm_paged_attention, _lib.qmm_paged_attention_workspace,
             _lib.qmm_qk_norm, _lib.qmm_kv4_append, _lib.qmm_kv4_read, _lib.qmm_kv4_attention, _lib.qmm_kv4_attention_workspace)
    mod.connect(*(ctypes.cast(f, ctypes.c_void_p).value for f in entry), _check, torch._C._cuda_getCurrentRawStream,
                torch._C._cuda_getDevice, torch._C._cuda_setDevice)
    return mod


_binding = _load_binding()
_ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}


def linear(X, wq, s, z, bits: int, G: int, bias=None, act: str = "none", mul=None, residual=None, out=None) -> torch.Tensor:
    """Y [M, N] fp16 = act(X [M, K] . dequant(wq) + bias) * mul + residual, any M.

    bias fp16 [N], mul and residual fp16 [M, N], each optional; act: "none", "relu", "silu", "gelu"
    or "gelu_tanh".  The product's fp32 sums go through all of it in fp32 and are rounded once.
    out may be mul or residual itself."""
    code = _ACTS.get(act)
    if code is None:
        raise ValueError(f"unknown activation {act!r}: expected one of {sorted(_ACTS)}")
    return _binding.linear(X, wq, s, z, bits, G, bias, code, mul, residual, out)


def kv_append(q, k, v, k_cache, v_cache, slots, positions=None, rope=None, pairs: bool = False, k_scale=None, v_scale=None, out=None):
    """Rotary positions on q [T, Hq, D] and k [T, Hkv, D], and k and v [T, Hkv, D] into the caches
    [pages, Hkv, page, D] (q's type, or float8_e4m3fn with fp32 scales [Hkv]).  Returns the turned q.

    slots int64 [T]: page id * page + place, or -1 (padding: nothing is stored); positions int32
    [T]: rows of rope, fp32 [rows, rot] with rot/2 cosines and then rot/2 sines (None: no rotation).
    pairs: elements 2i and 2i + 1 turn together (False: i and i + rot/2).  q may be None (k and v
    alone); q, k and v may be slices of one projection, out may be q.  D may be any even number
    here; paged_attention reads caches of D a multiple of 16 up to 256."""
    return _binding.kv_append(q, k, v, k_cache, v_cache, slots, positions, rope, pairs, k_scale, v_scale, out)


def paged_attention(q, k_cache, v_cache, page_table, cu_q, kv_lens, max_q: int, max_kv: int, scale=None, window: int = 0,
                    k_scale=None, v_scale=None, out=None, lse=None) -> torch.Tensor:
    """Causal attention of new tokens q [T, Hq, D] over the paged caches [pages, Hkv, page, D].

    page_table int32 [B, width]; cu_q int32 [B + 1]: sequence b's rows of q; kv_lens int32 [B]: its
    keys, the new tokens' among them; max_q and max_kv: upper bounds of both (host integers: nothing
    is read back).  scale: D ** -0.5 if None; window > 0: a row sees its last `window` keys alone;
    lse fp32 [T, Hq] (written if given): the log of each row's sum.  A row that sees no key gives
    zeros and -inf.  One call serves decode (one row each), chunks and whole prompts mixed; it is
    planned by max_q, so that decode rows on long contexts beside a prompt are quicker in a call of
    their own (one row on 131072 keys, a prompt of 2048: 2429 us in one call, 171 in two)."""
    return _binding.paged_attention(q, k_cache, v_cache, page_table, cu_q, kv_lens, max_q, max_kv, scale, window, k_scale, v_scale, out,
                                    lse)


def qk_norm(q, k, q_weight=None, k_weight=None, eps: float = 1e-6, positions=None, rope=None, pairs: bool = False, q_out=None, k_out=None):
    """RMS norms of q [T, Hq, D] and k [T, Hkv, D] for each head, x / sqrt(mean(x^2) + eps) * weight, and
    their rotary positions, in one pass.  Returns (q, k).

    q_weight and k_weight: [D] of q's type (None: no norm); positions, rope and pairs as in kv_append.
    q and k may be slices of one projection, q_out and k_out may be q and k.  D and rope's width:
    multiples of 16, D up to 256."""
    return _binding.qk_norm(q, k, q_weight, k_weight, eps, positions, rope, pairs, q_out, k_out)


class KV4Cache(NamedTuple):
    """A paged cache of 4-bit codes (any tuple of four such tensors will do where one is asked for).

    The D elements of a token and head are D / 2 bytes, the lower half of each first; x = (code - z) s with
    the s and z of its group of G elements."""
    k: torch.Tensor            # uint8 [pages, heads, page, D / 2]
    v: torch.Tensor
    k_scale: torch.Tensor      # fp16 [pages, heads, page, D / G, 2]: s and z
    v_scale: torch.Tensor


def kv4_cache(pages: int, heads: int, page: int, D: int, G: int | None = None, device="cuda") -> KV4Cache:
    """An empty cache of 4-bit codes: G (32, 64 or 128; None: the largest that divides D) elements share a scale."""
    if G is None:
        G = next((g for g in (128, 64, 32) if D % g == 0), 0)
    if G not in (32, 64, 128) or D % G or not 0 < D <= 256:
        raise ValueError(f"G must be 32, 64 or 128 and D a multiple of it up to 256, got D = {D}, G = {G}")
    codes = [torch.zeros(pages, heads, page, D // 2, dtype=torch.uint8, device=device) for _ in range(2)]
    return KV4Cache(*codes, *(torch.zeros(pages, heads, page, D // G, 2, dtype=torch.float16, device=device) for _ in range(2)))


def kv4_append(q, k, v, cache, slots, positions=None, rope=None, pairs: bool = False, q_norm=None, k_norm=None, eps: float = 1e-6, out=None):
    """qk_norm's norms and rotations of q [T, Hq, D] and k [T, Hkv, D], each where it is asked for, and k and v
    [T, Hkv, D] into a cache of 4-bit codes.  Returns q after them (None without q).

    Each group of G elements is mapped as quantize maps weights, min to max with zero in the range, with
    a scale of 7 significant bits: what the cache then stands for are numbers of fp16.  Elements beyond
    +-57344 are stored as that; a group with NaN reads as NaN.  slots, positions, rope and pairs as in
    kv_append; two tokens of a call must not share a slot.  out may be q."""
    return _binding.kv4_append(q, k, v, cache, slots, positions, rope, pairs, q_norm, k_norm, eps, out)


def kv4_read(cache, slots, dtype: torch.dtype = torch.float16, k_out=None, v_out=None):
    """The keys and values at these slots (int64 [T]) of a cache of 4-bit codes: two tensors [T, Hkv, D] of fp16
    (exactly what kv4_attention multiplies by) or bf16.  A slot outside the cache, as -1, gives zeros."""
    if dtype not in (torch.float16, torch.bfloat16):
        raise TypeError(f"dtype must be float16 or bfloat16, got {dtype}")
    return _binding.kv4_read(cache, slots, dtype == torch.bfloat16, k_out, v_out)


def kv4_attention(q, cache, page_table, cu_q, kv_lens, max_q: int, max_kv: int, scale=None, window: int = 0, sinks: int = 0, out=None,
                  lse=None) -> torch.Tensor:
    """paged_attention over a cache of 4-bit codes.

    window > 0: a row sees its last `window` keys and, of those before them, the sequence's first
    `sinks`.  The other arguments as in paged_attention.  A token with NaN gives NaN to the rows that see it,
    and to no others."""
    return _binding.kv4_attention(q, cache, page_table, cu_q, kv_lens, max_q, max_kv, scale, window, sinks, out, lse)


def probe_read(buf: torch.Tensor, grid: int, sink: torch.Tensor | None = None) -> None:
    """Measurement hook: one streaming read of the whole of buf (any dtype, contiguous,
    byte size a multiple of 16) by `grid` workgroups; computes nothing of the product."""
    if not buf.is_cuda or not buf.is_contiguous():
        raise ValueError("buf must be a contiguous GPU tensor")
    if sink is None:
        sink = torch.empty(grid * 256, dtype=torch.int32, device=buf.device)
    _need(sink, "sink", torch.int32, None, buf.device)
    if sink.numel() < grid * 256:
        raise ValueError("sink needs grid * 256 elements")
    _check(_lib.qmm_probe_read(_ptr(buf), buf.numel() * buf.element_size(), _ptr(sink), grid, _stream(buf.device)))


def probe_mfma(iters: int, grid: int, shape: int = 0, sink: torch.Tensor | None = None,
               device: str = "cuda:0") -> int:
    """Measurement hook: back-to-back f16 MFMAs (shape 0: 16x16x32, 1: 32x32x16) on register
    operands in `grid` workgroups of 8 waves; returns the flops enqueued."""
    if sink is None:
        sink = torch.empty(grid * 512, dtype=torch.float32, device=device)
    _need(sink, "sink", torch.float32)
    if sink.numel() < grid * 512:
        raise ValueError("sink needs grid * 512 elements")
    _check(_lib.qmm_probe_mfma(_ptr(sink), iters, grid, shape, _stream(sink.device)))
    return grid * 8 * iters * 8 * 16384
