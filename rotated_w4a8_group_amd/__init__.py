"""PARO W4A8 linear hot path on AMD Instinct MI355X (gfx950).

Thin Python binding over the C ABI in ``include/pq.h`` (``libpq.so`` in this directory).
It only marshals arguments: every step of the path runs in the library's HIP kernels.
PyTorch supplies device memory and the current HIP stream. There is no fallback: if the
library is missing or fails to load, every call raises.

Calls (same names as the C entry points, without the ``pq_`` prefix):

* ``build_records(pairs, theta)``            host; numpy int16 [8, K], f16 [8, K/2]
* ``pack_weights(qweight, qzeros, scales)``  device; AWQ tensors -> (wpk, sz)
* ``rotate_quant(x, rec, cs)``               device; -> (A, ASG, RS)
* ``rotate(x, rec, cs)``                     device; -> rotated rows of x's type, not quantised
* ``gemm(A, ASG, RS, wpk, sz, N, pb1, pb2)`` device; -> y bf16
* ``gemm_glu(A, ASG, RS, wpk, sz, F)``       device; gate | up projection -> act(gate) * up, f16 or bf16
* ``matvec(x, wpk, sz, N, pb1, pb2)``        device; 16-bit rows (at most 16) -> y of their type
* ``block_norms(x, residual, ...)``           device; -> (new residual, normalised row): the norms before
  and after a block with its gate and residual scale
* ``e4m3_encode(q)``, ``recip_f32(x)``       device verification hooks
"""
import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpq.so")

GROUP = 128
LAYERS = 8
NO_BOUNDARY = 0x7FFFFFFF
INT_MAX = 0x7FFFFFFF

PQ_OK = 0
ERRORS = {
    -1: "PQ_ERR_NULL", -2: "PQ_ERR_SHAPE", -3: "PQ_ERR_ALIGN", -4: "PQ_ERR_PARTITION",
    -5: "PQ_ERR_RECORDS", -6: "PQ_ERR_WORKSPACE", -7: "PQ_ERR_DEVICE",
}

# name -> (restype, argtypes); keep in step with include/pq.h
_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
SIGNATURES = {
    "pq_abi_version": (_I, []),
    "pq_last_error": (ctypes.c_char_p, []),
    "pq_build_records": (_I, [_P, _P, _I, _P]),
    "pq_plan_partitions": (_I, [_I, _P, _P, _P, _P, _I, _P, _P, _P]),
    "pq_packed_weight_bytes": (_SZ, [_I, _I]),
    "pq_pack_weights": (_I, [_P, _P, _P, _I, _I, _P, _P, _P]),
    "pq_rotate_quant": (_I, [_P, _I64, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
    "pq_rotate": (_I, [_P, _I64, _I, _I, _I, _I, _P, _P, _P, _P]),
    "pq_gemm_workspace_bytes": (_SZ, [_I, _I, _I]),
    "pq_gemm": (_I, [_P, _P, _P, _I, _I, _I, _P, _P, _I, _I, _I, _P, _I64, _P, _SZ, _P]),
    "pq_matvec": (_I, [_P, _I64, _I, _I, _I, _I, _P, _P, _I, _I, _I, _P, _I64, _I, _P]),
    "pq_rotate_quant_for_gemm": (_I, [_P, _I64, _I, _I, _I, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "pq_gemm_prepared": (_I, [_P, _P, _P, _I, _I, _I, _P, _P, _I, _I, _I, _P, _I64, _P, _SZ, _P]),
    "pq_gemm_glu": (_I, [_P, _P, _P, _I, _I, _I, _P, _P, _I, _I, _P, _I64, _I, _P, _SZ, _I, _P]),
    "pq_gemm_noalloc_max_scratch_bytes": (_SZ, []),
    "pq_gemm_noalloc": (_I, [_P, _P, _P, _I, _I, _I, _P, _P, _I, _I, _I, _P, _I64, _P]),
    "pq_rotate_quant_tok": (_I, [_P, _I64, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
    "pq_gemm_tok_workspace_bytes": (_SZ, [_I, _I, _I]),
    "pq_gemm_tok": (_I, [_P, _P, _P, _I, _I, _I, _P, _P, _I, _I, _I, _P, _I64, _P, _SZ, _P]),
    "pq_rotate_quant_i8": (_I, [_P, _I64, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
    "pq_gemm_i8": (_I, [_P, _P, _P, _I, _I, _I, _P, _P, _I, _I, _I, _P, _I64, _P, _SZ, _P]),
    "pq_packed_weight5_bytes": (_SZ, [_I, _I]),
    "pq_pack_weights5": (_I, [_P, _P, _P, _P, _P, _I, _I, _P, _P, _P]),
    "pq_gemm5": (_I, [_P, _P, _P, _I, _I, _I, _P, _P, _I, _I, _I, _P, _I64, _P, _SZ, _P]),
    "pq_add_rms_rotate_quant": (_I, [_P, _I64, _P, _I64, _P, ctypes.c_float, _I, _I, _I, _I, _P, _P, _P, _I64,
                                     _P, _P, _P, _P, _P]),
    "pq_block_norms": (_I, [_P, _I64, _I, _P, _I64, _I, _P, _P, _I64, _I, _I, _P, ctypes.c_float, ctypes.c_float,
                            ctypes.c_float, _I, _I, _I, _P, _I64, _P, _I64, _I, _P]),
    "pq_e4m3_encode": (_I, [_P, _P, _I64, _P]),
    "pq_recip_f32": (_I, [_P, _P, _I64, _P]),
    "pq_bf16_round": (_I, [_P, _P, _I64, _P]),
}


class PQError(RuntimeError):
    def __init__(self, fn, code, msg):
        super().__init__(f"{fn}: {ERRORS.get(code, code)}: {msg}")
        self.code = code


_lib = None


def lib():
    """The loaded C library (loaded once). Raises if it is not built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run `python -m rotated_w4a8_group_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


_fast = None


def _native():
    """The compiled calls of rotate, matvec, gemm_glu and block_norms (``_binding.so``), which take the usual call - plain
    tensors that pass every check, on the current device and stream - and answer NotImplemented to any other; False where
    they are not built for this interpreter, torch and library: the functions below then do every call, 2 to 5 us slower each."""
    global _fast
    if _fast is None:
        import torch  # noqa: F401  (its libraries first)
        L = lib()
        try:
            from . import _binding as b
            b.bind(_check, L.pq_abi_version(), *(ctypes.cast(getattr(L, f), _P).value for f in (
                "pq_rotate", "pq_matvec", "pq_gemm_glu", "pq_block_norms", "pq_packed_weight_bytes", "pq_gemm_workspace_bytes")))
            _fast = b
        except ImportError as e:   # not built, or not for this library
            if os.path.exists(os.path.join(_HERE, "_binding.so")):
                import warnings
                warnings.warn(f"_binding.so does not load ({e}): calls go through Python")
            _fast = False
    return _fast


def _check(fn, code):
    if code != PQ_OK:
        raise PQError(fn, code, lib().pq_last_error().decode())


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _nbytes(t):
    """Size in bytes of an optional workspace tensor (0 for None); the library checks it."""
    if t is None:
        return 0
    if not t.is_cuda or not t.is_contiguous():
        raise TypeError("workspace: expected a contiguous CUDA tensor")
    return t.numel() * t.element_size()


def _need(t, dtype, name):
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name}: expected a contiguous CUDA tensor of {dtype}")


def _validate(specs, rows=()):
    """Checks every argument the C ABI cannot see before anything is called.

    specs: (tensor, name, dtype, shape) for contiguous tensors, where shape is a tuple or an int
    (a minimum number of elements). rows: (tensor, name, dtype, (M, K)) for row-strided 2-D
    tensors (unit column stride). Dtypes and shapes of all of them are checked first (TypeError /
    ValueError), then that each is a CUDA tensor on the first one's device (TypeError), so a
    shape mismatch is reported the same way whatever the devices."""
    import torch
    # the usual call passes everything: one cheap look at each tensor, and the ordered checks below
    # only to name what is wrong
    dev, tensor = None, torch.Tensor
    for t, name, dtype, shape in specs:
        if not (isinstance(t, tensor) and t.dtype is dtype and t.is_contiguous() and
                (t.numel() >= shape if type(shape) is int else t.shape == shape)):
            break
        d = t.get_device()
        if d < 0 or (dev is not None and d != dev):
            break
        dev = d
    else:
        for t, name, dtype, shape in rows:
            if not (isinstance(t, tensor) and t.dtype is dtype and t.shape == shape and t.stride()[1] == 1):
                break
            d = t.get_device()
            if d < 0 or (dev is not None and d != dev):
                break
            dev = d
        else:
            return
    for t, name, dtype, shape in list(specs) + list(rows):
        if not isinstance(t, torch.Tensor) or t.dtype != dtype:
            raise TypeError(f"{name}: expected a tensor of {dtype}")
    for t, name, dtype, shape in specs:
        if isinstance(shape, tuple):
            if tuple(t.shape) != tuple(int(d) for d in shape):
                raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
        elif t.numel() < shape:
            raise ValueError(f"{name}: {t.numel()} elements, at least {shape} needed")
    for t, name, dtype, shape in rows:
        if t.dim() != 2 or tuple(t.shape) != tuple(shape) or t.stride(1) != 1:
            raise ValueError(f"{name}: expected a [{shape[0]}, {shape[1]}] tensor with unit column stride, "
                             f"got shape {tuple(t.shape)} strides {t.stride()}")
    devs = set()
    for t, name, dtype, shape in list(specs) + list(rows):
        if not t.is_cuda:
            raise TypeError(f"{name}: expected a CUDA tensor")
        devs.add(t.device)
    if len(devs) > 1:
        raise TypeError(f"tensors on several devices: {sorted(str(d) for d in devs)}")
    for t, name, dtype, shape in specs:
        if not t.is_contiguous():
            raise TypeError(f"{name}: expected a contiguous tensor")


def _too_large(**sizes):
    """Raises for the sizes that the library's 32-bit arguments do not hold (ctypes would wrap them, and the library
    would answer for another size). The callers compare first; this names which."""
    raise ValueError(", ".join(f"{n}={v}" for n, v in sizes.items() if not -INT_MAX <= v <= INT_MAX) + ": at most 2^31 - 1 in one call")


def _partitions(cs, K):
    """P from the channel-scale tensor: [P, K] or [K] (one partition)."""
    if cs.dim() == 2:
        return cs.shape[0]
    if cs.dim() == 1:
        return 1
    raise ValueError(f"cs: expected [P, K] or [K], got shape {tuple(cs.shape)}")


def _prologue_specs(x, rec, cs, K):
    """The inputs every prologue shares: x [M, K] rows, records [P][8][K/2] (8 bytes each),
    channel scales [P, K]; returns (P, specs, rows)."""
    import torch
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x: expected a [M, K] tensor")
    if K <= 0 or K % GROUP:
        raise ValueError(f"x: K={K} must be a positive multiple of {GROUP}")
    if K > INT_MAX or x.shape[0] > INT_MAX:
        _too_large(M=x.shape[0], K=K)
    P = _partitions(cs, K)
    if not 1 <= P <= 3:
        raise ValueError(f"cs: {P} partitions, expected 1..3")
    rec_shape = (P, LAYERS, K // 2, 8) if rec.dim() == 4 else (LAYERS, K // 2, 8)
    if rec.dim() == 3 and P != 1:
        raise ValueError("rec: a [8, K/2, 8] record set serves one partition only")
    cs_shape = (P, K) if cs.dim() == 2 else (K,)
    return P, [(rec, "rec", torch.uint8, rec_shape), (cs, "cs", torch.float16, cs_shape)]


def _addr(t):
    """Address of an optional tensor, as ctypes takes it."""
    return None if t is None else t.data_ptr()


def _pitch(t, M, K):
    """Row stride of a [M, K] tensor in elements; that of a single row is of no consequence."""
    return t.stride()[0] if M > 1 else K


def _new(shape, dtype, device, stream):
    """An output or workspace of a call on ``stream``: from that stream's own memory, so that it is not
    handed out again before the stream has passed the call."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _launch(fn, device, stream, *args):
    """Calls the C entry point ``fn`` on the tensors' device, queued on ``stream`` or that device's current one."""
    import torch
    f = getattr(_lib or lib(), fn)
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(device.index)   # current_stream(device).cuda_stream, without the object
    elif stream.device != device:
        raise ValueError(f"stream: on {stream.device}, the tensors are on {device}")
    else:
        handle = stream.cuda_stream
    if torch._C._cuda_getDevice() == device.index:
        rc = f(*args, handle)
    else:
        with torch.cuda.device(device):
            rc = f(*args, handle)
    if rc != PQ_OK:
        _check(fn, rc)


_codes = {}


def _type_code(dtype, name, allowed=2):
    """The pq_type of a torch dtype: f16, bf16, and f32 where ``allowed`` is 3."""
    if not _codes:
        import torch
        _codes.update({torch.float16: 0, torch.bfloat16: 1, torch.float32: 2})
    code = _codes.get(dtype, 3)
    if code >= allowed:
        raise TypeError(f"{name}: expected a tensor of float16{', bfloat16 or float32' if allowed == 3 else ' or bfloat16'}, got {dtype}")
    return code


# ------------------------------------------------------------------------------------------
def build_records(pairs, theta):
    """pairs int16 [8, K], theta f16 [8, K/2] (numpy, host) -> uint8 [8, K/2, 8] records."""
    pairs = np.ascontiguousarray(pairs, dtype=np.int16)
    theta = np.ascontiguousarray(theta, dtype=np.float16)
    K = pairs.shape[1]
    out = np.zeros((LAYERS, K // 2, 8), dtype=np.uint8)
    _check("pq_build_records", lib().pq_build_records(
        pairs.ctypes.data_as(_P), theta.view(np.uint16).ctypes.data_as(_P), K, out.ctypes.data_as(_P)))
    return out


def plan_partitions(projections):
    """projections: list of (ncols, pairs int16 [8, K], theta f16 [8, K/2], cs f16 [K]) in column
    order (numpy, host). Adjacent projections with identical rotation data merge into one
    partition. Returns (P, pb1, pb2, reps): reps[q] is the projection whose rotation partition q
    uses."""
    J = len(projections)
    arrs = [(np.ascontiguousarray(p, dtype=np.int16), np.ascontiguousarray(t, dtype=np.float16).view(np.uint16),
             np.ascontiguousarray(c, dtype=np.float16).view(np.uint16)) for _, p, t, c in projections]
    K = arrs[0][0].shape[1] if J else 0
    for p, t, c in arrs:
        if p.shape != (LAYERS, K) or t.shape != (LAYERS, K // 2) or c.shape != (K,):
            raise ValueError("plan_partitions: every projection needs pairs [8, K], theta [8, K/2], cs [K]")
    ncols = np.array([n for n, *_ in projections], dtype=np.int32)
    ptrs = [(ctypes.c_void_p * J)(*[a[i].ctypes.data for a in arrs]) for i in range(3)]
    P = ctypes.c_int()
    pb = (ctypes.c_int * 2)()
    rep = (ctypes.c_int * 3)()
    _check("pq_plan_partitions", lib().pq_plan_partitions(
        J, ncols.ctypes.data_as(_P), ptrs[0], ptrs[1], ptrs[2], K, ctypes.byref(P), pb, rep))
    return P.value, pb[0], pb[1], [r for r in rep[:P.value]]


def pack_weights(qweight, qzeros, scales, stream=None):
    """AWQ qweight int32 [K, N/8], qzeros int32 [K/128, N/8], scales f16 [K/128, N] (CUDA)
    -> (wpk uint8 [K*N/2], sz f16 [K/128, N, 2])."""
    import torch
    if not isinstance(qweight, torch.Tensor) or qweight.dim() != 2:
        raise ValueError("qweight: expected an int32 [K, N/8] tensor")
    K, N = qweight.shape[0], qweight.shape[1] * 8
    if K % GROUP or N % 16 or K == 0:
        raise ValueError(f"qweight: K={K} must be a multiple of {GROUP} and N={N} of 16")
    if K > INT_MAX or N > INT_MAX:
        _too_large(K=K, N=N)
    _validate([(qweight, "qweight", torch.int32, (K, N // 8)), (qzeros, "qzeros", torch.int32, (K // GROUP, N // 8)),
               (scales, "scales", torch.float16, (K // GROUP, N))])
    wpk = torch.empty(lib().pq_packed_weight_bytes(K, N), dtype=torch.uint8, device=qweight.device)
    sz = torch.empty((K // GROUP, N, 2), dtype=torch.float16, device=qweight.device)
    _check("pq_pack_weights", lib().pq_pack_weights(
        _ptr(qweight), _ptr(qzeros), _ptr(scales), K, N, _ptr(wpk), _ptr(sz), _stream(stream)))
    return wpk, sz


def pack_weights5(qweight, qweight_hi, qzeros, qzeros_hi, scales, stream=None):
    """int5 bit-plane weights: qweight int32 [K, N/8], qweight_hi int32 [K, N/32], qzeros int32
    [K/128, N/8], qzeros_hi int32 [K/128, N/32], scales f16 [K/128, N] (CUDA)
    -> (wpk5 uint8 [pq_packed_weight5_bytes], sz f16 [K/128, N, 2])."""
    import torch
    if not isinstance(qweight, torch.Tensor) or qweight.dim() != 2:
        raise ValueError("qweight: expected an int32 [K, N/8] tensor")
    K, N = qweight.shape[0], qweight.shape[1] * 8
    if K % GROUP or N % 32 or K == 0:
        raise ValueError(f"qweight: K={K} must be a multiple of {GROUP} and N={N} of 32")
    if K > INT_MAX or N > INT_MAX:
        _too_large(K=K, N=N)
    _validate([(qweight, "qweight", torch.int32, (K, N // 8)), (qweight_hi, "qweight_hi", torch.int32, (K, N // 32)),
               (qzeros, "qzeros", torch.int32, (K // GROUP, N // 8)),
               (qzeros_hi, "qzeros_hi", torch.int32, (K // GROUP, N // 32)),
               (scales, "scales", torch.float16, (K // GROUP, N))])
    wpk = torch.empty(max(1, lib().pq_packed_weight5_bytes(K, N)), dtype=torch.uint8, device=qweight.device)
    sz = torch.empty((K // GROUP, N, 2), dtype=torch.float16, device=qweight.device)
    _check("pq_pack_weights5", lib().pq_pack_weights5(
        _ptr(qweight), _ptr(qweight_hi), _ptr(qzeros), _ptr(qzeros_hi), _ptr(scales), K, N,
        _ptr(wpk), _ptr(sz), _stream(stream)))
    return wpk, sz


def _rotate_quant_common(fn, x, rec, cs, out, stream, a_dtype, tok=False, workspace=False):
    """Checks x [M, K], the records and channel scales, and caller-given outputs (codes [P, M, K],
    scales [P, M, G] or [P, M] with tok, row-sums [P, M, G]); allocates missing outputs.
    workspace (pq_rotate_quant_for_gemm): the GEMM workspace tensor the call also fills, checked
    against gemm_workspace_bytes(M, N, K)."""
    import torch
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x: expected a [M, K] tensor")
    M, K = x.shape
    P, specs = _prologue_specs(x, rec, cs, K)
    G = K // GROUP
    s_shape = (P, M) if tok else (P, M, G)
    if out is not None:
        A, S, R = out
        specs += [(A, "A", a_dtype, (P, M, K)), (S, "AS" if tok else "ASG", torch.float32, s_shape),
                  (R, "RS", torch.float32, (P, M, G))]
    if workspace is not False:
        ws_bytes = gemm_workspace_bytes(M, 0, K)
        if workspace is None:
            if ws_bytes:
                raise ValueError(f"workspace: {ws_bytes} bytes needed at M={M}, K={K}")
        else:
            specs.append((workspace, "workspace", torch.uint8, ws_bytes))
    _validate(specs, rows=[(x, "x", torch.float16, (M, K))])
    ws_args = () if workspace is False else (_ptr(workspace), _nbytes(workspace))
    if out is None:
        A = torch.empty((P, M, K), dtype=a_dtype, device=x.device)
        S = torch.empty(s_shape, dtype=torch.float32, device=x.device)
        R = torch.empty((P, M, G), dtype=torch.float32, device=x.device)
    _check(fn, getattr(lib(), fn)(
        _ptr(x), x.stride(0), M, K, P, _ptr(rec), _ptr(cs), _ptr(A), _ptr(S), _ptr(R), *ws_args, _stream(stream)))
    return A, S, R


def rotate_quant(x, rec, cs, out=None, stream=None):
    """x f16 [M, K] (row stride may exceed K), rec uint8 [P, 8, K/2, 8] (or [8, K/2, 8]),
    cs f16 [P, K] (or [K]) -> (A u8 [P, M, K], ASG f32 [P, M, G], RS f32 [P, M, G])."""
    import torch
    return _rotate_quant_common("pq_rotate_quant", x, rec, cs, out, stream, torch.uint8)


def rotate_quant_for_gemm(x, rec, cs, workspace, out=None, stream=None):
    """pq_rotate_quant_for_gemm: ``rotate_quant`` that also writes, when M > 16, the prefill GEMM's
    activation-side operands into ``workspace`` (uint8, gemm_workspace_bytes(M, N, K) bytes; None
    allowed at M <= 16) for a following ``gemm_prepared`` on the returned (A, ASG, RS)."""
    import torch
    return _rotate_quant_common("pq_rotate_quant_for_gemm", x, rec, cs, out, stream, torch.uint8,
                                workspace=workspace)


def rotate(x, rec, cs, out=None, stream=None):
    """The rotation alone: x f16 or bf16 [M, K] (row stride may exceed K), rec uint8 [P, 8, K/2, 8] (or [8, K/2, 8]),
    cs f16 [P, K] (or [K]) -> y [P, M, K] of x's type, ``rotate_quant``'s rotated rows before their quantisation."""
    f = _native() if _fast is None else _fast
    if f and stream is None:
        done = f.rotate(x, rec, cs, out)
        if done is not NotImplemented:
            return done
    import torch
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x: expected a [M, K] tensor")
    M, K = x.shape
    xt = _type_code(x.dtype, "x")
    P, specs = _prologue_specs(x, rec, cs, K)
    if out is not None:
        specs.append((out, "out", x.dtype, (P, M, K)))
    _validate(specs, rows=[(x, "x", x.dtype, (M, K))])
    if out is None:
        out = _new((P, M, K), x.dtype, x.device, stream)
    _launch("pq_rotate", x.device, stream, x.data_ptr(), _pitch(x, M, K), xt, M, K, P, rec.data_ptr(), cs.data_ptr(), out.data_ptr())
    return out


def gemm_workspace_bytes(M, N, K):
    if M > INT_MAX or N > INT_MAX or K > INT_MAX:
        _too_large(M=M, N=N, K=K)
    return int(lib().pq_gemm_workspace_bytes(M, N, K))


def _gemm_common(fn, A, S, RS, wpk, sz, N, pb1, pb2, out, workspace, stream, *, a_dtype, tok=False, w5=False,
                 prepared=False):
    """Checks every tensor against (P, M, K, N), allocates what is missing, calls `fn`."""
    import torch
    if not isinstance(A, torch.Tensor) or A.dim() != 3:
        raise ValueError("A: expected a [P, M, K] tensor")
    P, M, K = A.shape
    if K == 0 or K % GROUP:
        raise ValueError(f"A: K={K} must be a positive multiple of {GROUP}")
    if M > INT_MAX or K > INT_MAX or N > INT_MAX or not -INT_MAX <= pb1 <= INT_MAX or not -INT_MAX <= pb2 <= INT_MAX:
        _too_large(M=M, K=K, N=N, pb1=pb1, pb2=pb2)
    G = K // GROUP
    L = lib()
    need = L.pq_packed_weight5_bytes(K, N) if w5 else L.pq_packed_weight_bytes(K, N)
    if need == 0:
        raise ValueError(f"N={N}: not a shape the library packs (N % {32 if w5 else 16} == 0 needed)")
    specs = [(A, "A", a_dtype, (P, M, K)), (S, "AS" if tok else "ASG", torch.float32, (P, M) if tok else (P, M, G)),
             (RS, "RS", torch.float32, (P, M, G)), (wpk, "wpk5" if w5 else "wpk", torch.uint8, int(need)),
             (sz, "sz", torch.float16, (G, N, 2))]
    ws_bytes = int(L.pq_gemm_tok_workspace_bytes(M, N, K) if tok else L.pq_gemm_workspace_bytes(M, N, K))
    if workspace is not None:
        specs.append((workspace, "workspace", torch.uint8, ws_bytes))
    elif prepared and ws_bytes:
        raise ValueError("workspace: gemm_prepared reads the workspace rotate_quant_for_gemm filled")
    if out is None:
        _validate(specs)
        out = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    else:
        if not isinstance(out, torch.Tensor) or out.dim() != 2 or out.shape[0] != M or out.shape[1] < N:
            raise ValueError(f"out: expected a bf16 [{M}, >= {N}] tensor")
        _validate(specs, rows=[(out, "out", torch.bfloat16, (M, out.shape[1]))])
    if workspace is None and ws_bytes:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=A.device)
    _check(fn, getattr(L, fn)(
        _ptr(A), _ptr(S), _ptr(RS), M, K, P, _ptr(wpk), _ptr(sz), N, pb1, pb2,
        _ptr(out), out.stride(0), _ptr(workspace), _nbytes(workspace), _stream(stream)))
    return out


def gemm(A, ASG, RS, wpk, sz, N, pb1=NO_BOUNDARY, pb2=NO_BOUNDARY, out=None, workspace=None, stream=None):
    """A u8 [P, M, K], ASG/RS f32 [P, M, G], packed weights (wpk from pack_weights, sz [G, N, 2])
    -> y bf16 [M, N] (or into ``out``, a bf16 [M, ldy >= N] view with unit column stride)."""
    import torch
    return _gemm_common("pq_gemm", A, ASG, RS, wpk, sz, N, pb1, pb2, out, workspace, stream, a_dtype=torch.uint8)


def matvec(x, wpk, sz, N, pb1=NO_BOUNDARY, pb2=NO_BOUNDARY, out=None, dtype=None, stream=None):
    """Products of few 16-bit rows with the packed weights of ``gemm``: x f16 or bf16 [P, M, K] (or [M, K] for one
    partition; row stride may exceed K), M <= 16 -> y [M, N] of ``dtype`` (f16 or bf16; x's type by default), or into
    ``out``, a [M, ldy >= N] view with unit column stride. A row with an infinity or a NaN gives NaN in its whole row of y."""
    f = _native() if _fast is None else _fast
    if f and stream is None:
        done = f.matvec(x, wpk, sz, N, pb1, pb2, out, dtype)
        if done is not NotImplemented:
            return done
    import torch
    if not isinstance(x, torch.Tensor) or x.dim() not in (2, 3):
        raise ValueError("x: expected a [P, M, K] or [M, K] tensor")
    xt = _type_code(x.dtype, "x")
    P, M, K = (1, *x.shape) if x.dim() == 2 else x.shape
    if K == 0 or K % GROUP:
        raise ValueError(f"x: K={K} must be a positive multiple of {GROUP}")
    if M > 16:
        raise ValueError(f"x: M={M} rows, at most 16 (gemm takes more, quantised)")
    if K > INT_MAX or N > INT_MAX or not -INT_MAX <= pb1 <= INT_MAX or not -INT_MAX <= pb2 <= INT_MAX:
        _too_large(K=K, N=N, pb1=pb1, pb2=pb2)
    need = lib().pq_packed_weight_bytes(K, N)
    if need == 0:
        raise ValueError(f"N={N}: not a shape the library packs (N % 16 == 0 needed)")
    specs = [(wpk, "wpk", torch.uint8, need), (sz, "sz", torch.float16, (K // GROUP, N, 2))]
    rows = []
    if x.dim() == 3:
        specs.append((x, "x", x.dtype, (P, M, K)))
        ldx = K
    else:
        rows.append((x, "x", x.dtype, (M, K)))
        ldx = _pitch(x, M, K)
    if out is not None:
        if not isinstance(out, torch.Tensor) or out.dim() != 2 or out.shape[0] != M or out.shape[1] < N:
            raise ValueError(f"out: expected a f16 or bf16 [{M}, >= {N}] tensor")
        if dtype is not None and out.dtype != dtype:
            raise TypeError(f"out: {out.dtype}, dtype says {dtype}")
        rows.append((out, "out", out.dtype, (M, out.shape[1])))
    yt = _type_code(out.dtype if out is not None else dtype or x.dtype, "out")
    _validate(specs, rows=rows)
    if out is None:
        out = _new((M, N), dtype or x.dtype, x.device, stream)
    _launch("pq_matvec", x.device, stream, x.data_ptr(), ldx, xt, M, K, P, wpk.data_ptr(), sz.data_ptr(), N, pb1, pb2,
            out.data_ptr(), _pitch(out, M, N), yt)
    return out


def gemm_prepared(A, ASG, RS, wpk, sz, N, pb1=NO_BOUNDARY, pb2=NO_BOUNDARY, out=None, workspace=None, stream=None):
    """pq_gemm_prepared: ``gemm`` on the workspace that ``rotate_quant_for_gemm`` filled for this same
    (A, ASG, RS) (required when M > 16; nothing may write it in between)."""
    import torch
    return _gemm_common("pq_gemm_prepared", A, ASG, RS, wpk, sz, N, pb1, pb2, out, workspace, stream,
                        a_dtype=torch.uint8, prepared=True)


GLU_ACTS = {"silu": 0, "gelu": 1}


def gemm_glu(A, ASG, RS, wpk, sz, F, act="silu", out=None, dtype=None, workspace=None, prepared=False, stream=None):
    """The gated feed-forward pair in one launch: ``h = act(g) * u`` of ``gemm``'s merged gate | up projection (wpk, sz
    from pack_weights of N = 2 F columns, gate first), g and u not rounded in between. A u8 [P, M, K], ASG/RS f32
    [P, M, G] with P = 1 (one rotation for both) or 2 (the gate's, the up projection's) -> h [M, F] of ``dtype`` (f16 by
    default, what the next prologue takes, or bf16), or into ``out``, a [M, ldh >= F] view with unit column stride.
    act "silu" or "gelu" (tanh form). workspace: gemm_workspace_bytes(M, 2 F, K) bytes; prepared: it holds
    what ``rotate_quant_for_gemm`` wrote for these A, ASG and RS.

    g and u carry what ``gemm``'s products do (the e4m3 matrix instruction drops what lies below 2^-13 of the largest of 8
    neighbours), and in the tiles of long prompts the zero point's bf16 pieces (2^-14 of it): an f16 h shows both, about 1e-4 of the norm."""
    f = _native() if _fast is None else _fast
    if f and stream is None:
        done = f.gemm_glu(A, ASG, RS, wpk, sz, F, GLU_ACTS.get(act), out, dtype, workspace, prepared)
        if done is not NotImplemented:
            return done
    import torch
    if not isinstance(A, torch.Tensor) or A.dim() != 3:
        raise ValueError("A: expected a [P, M, K] tensor")
    P, M, K = A.shape
    if K == 0 or K % GROUP:
        raise ValueError(f"A: K={K} must be a positive multiple of {GROUP}")
    G = K // GROUP
    code = GLU_ACTS.get(act)
    if code is None:
        raise ValueError(f"act: {act!r}, expected one of {', '.join(GLU_ACTS)}")
    if M > INT_MAX or K > INT_MAX or 2 * F > INT_MAX:
        _too_large(M=M, K=K, **{"2 F": 2 * F})
    L = lib()
    need = L.pq_packed_weight_bytes(K, 2 * F) if F % 16 == 0 else 0
    if need == 0:
        raise ValueError(f"F={F}: must be a positive multiple of 16")
    specs = [(A, "A", torch.uint8, (P, M, K)), (ASG, "ASG", torch.float32, (P, M, G)), (RS, "RS", torch.float32, (P, M, G)),
             (wpk, "wpk", torch.uint8, need), (sz, "sz", torch.float16, (G, 2 * F, 2))]
    ws_bytes = L.pq_gemm_workspace_bytes(M, 2 * F, K)
    if workspace is not None:
        specs.append((workspace, "workspace", torch.uint8, ws_bytes))
    elif prepared and ws_bytes:
        raise ValueError("workspace: with prepared, the call reads the workspace rotate_quant_for_gemm filled")
    rows = []
    if out is not None:
        if not isinstance(out, torch.Tensor) or out.dim() != 2 or out.shape[0] != M or out.shape[1] < F:
            raise ValueError(f"out: expected a f16 or bf16 [{M}, >= {F}] tensor")
        if dtype is not None and out.dtype != dtype:
            raise TypeError(f"out: {out.dtype}, dtype says {dtype}")
        rows.append((out, "out", out.dtype, (M, out.shape[1])))
    ht = _type_code(out.dtype if out is not None else dtype or torch.float16, "out")
    _validate(specs, rows=rows)
    if out is None:
        out = _new((M, F), dtype or torch.float16, A.device, stream)
    if workspace is None and ws_bytes:
        workspace = _new((ws_bytes,), torch.uint8, A.device, stream)
    _launch("pq_gemm_glu", A.device, stream, A.data_ptr(), ASG.data_ptr(), RS.data_ptr(), M, K, P, wpk.data_ptr(),
            sz.data_ptr(), F, code, out.data_ptr(), _pitch(out, M, F), ht, _addr(workspace),
            workspace.numel() if workspace is not None else 0, 1 if prepared else 0)
    return out


def gemm_noalloc(A, ASG, RS, wpk, sz, N, pb1=NO_BOUNDARY, pb2=NO_BOUNDARY, out=None, stream=None):
    """pq_gemm_noalloc: the result of ``gemm`` with the library's own per-device scratch in place of
    a workspace (no device allocation in the call; ``out``, a bf16 [M, ldy >= N] tensor, is
    required). Calls that overlap on one device race on that scratch."""
    import torch
    if out is None:
        raise ValueError("out: gemm_noalloc writes into a caller-given bf16 [M, N] tensor")
    if not isinstance(A, torch.Tensor) or A.dim() != 3:
        raise ValueError("A: expected a [P, M, K] tensor")
    P, M, K = A.shape
    if K == 0 or K % GROUP:
        raise ValueError(f"A: K={K} must be a positive multiple of {GROUP}")
    if M > INT_MAX or K > INT_MAX or N > INT_MAX or not -INT_MAX <= pb1 <= INT_MAX or not -INT_MAX <= pb2 <= INT_MAX:
        _too_large(M=M, K=K, N=N, pb1=pb1, pb2=pb2)
    G = K // GROUP
    need = lib().pq_packed_weight_bytes(K, N)
    if need == 0:
        raise ValueError(f"N={N}: not a shape the library packs (N % 16 == 0 needed)")
    if not isinstance(out, torch.Tensor) or out.dim() != 2 or out.shape[0] != M or out.shape[1] < N:
        raise ValueError(f"out: expected a bf16 [{M}, >= {N}] tensor")
    _validate([(A, "A", torch.uint8, (P, M, K)), (ASG, "ASG", torch.float32, (P, M, G)),
               (RS, "RS", torch.float32, (P, M, G)), (wpk, "wpk", torch.uint8, int(need)),
               (sz, "sz", torch.float16, (G, N, 2))], rows=[(out, "out", torch.bfloat16, (M, out.shape[1]))])
    _check("pq_gemm_noalloc", lib().pq_gemm_noalloc(
        _ptr(A), _ptr(ASG), _ptr(RS), M, K, P, _ptr(wpk), _ptr(sz), N, pb1, pb2, _ptr(out), out.stride(0),
        _stream(stream)))
    return out


def gemm5(A, ASG, RS, wpk5, sz, N, pb1=NO_BOUNDARY, pb2=NO_BOUNDARY, out=None, workspace=None, stream=None):
    """int5 bit-plane weights (from pack_weights5) with the e4m3 prologue's A/ASG/RS -> y bf16 [M, N]."""
    import torch
    return _gemm_common("pq_gemm5", A, ASG, RS, wpk5, sz, N, pb1, pb2, out, workspace, stream,
                        a_dtype=torch.uint8, w5=True)


def add_rms_rotate_quant(x, residual, weight, eps, rec, cs, gemma=True, residual_out=None, out=None, stream=None):
    """Fused producer: x, residual f16 [M, K] (row strides multiples of 8), weight f16 [K], rec
    [P, 8, K/2, 8], cs f16 [P, K] -> (residual_out f16 [M, K] (``residual`` itself may be passed to
    update it in place), hs f16 [M, K], A u8 [P, M, K], ASG f32 [P, M, G], RS f32 [P, M, G])."""
    import torch
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x: expected a [M, K] tensor")
    M, K = x.shape
    P, specs = _prologue_specs(x, rec, cs, K)
    G = K // GROUP
    specs.append((weight, "weight", torch.float16, (K,)))
    rows = [(x, "x", torch.float16, (M, K)), (residual, "residual", torch.float16, (M, K))]
    if residual_out is not None:
        rows.append((residual_out, "residual_out", torch.float16, (M, K)))
    if out is not None:
        hs, A, S, R = out
        specs += [(hs, "hs", torch.float16, (M, K)), (A, "A", torch.uint8, (P, M, K)),
                  (S, "ASG", torch.float32, (P, M, G)), (R, "RS", torch.float32, (P, M, G))]
    _validate(specs, rows=rows)
    if residual_out is None:
        residual_out = torch.empty((M, K), dtype=torch.float16, device=x.device)
    if out is None:
        hs = torch.empty((M, K), dtype=torch.float16, device=x.device)
        A = torch.empty((P, M, K), dtype=torch.uint8, device=x.device)
        S = torch.empty((P, M, G), dtype=torch.float32, device=x.device)
        R = torch.empty((P, M, G), dtype=torch.float32, device=x.device)
    _check("pq_add_rms_rotate_quant", lib().pq_add_rms_rotate_quant(
        _ptr(x), x.stride(0), _ptr(residual), residual.stride(0), _ptr(weight), float(eps), 1 if gemma else 0,
        M, K, P, _ptr(rec), _ptr(cs), _ptr(residual_out), residual_out.stride(0), _ptr(hs), _ptr(A), _ptr(S),
        _ptr(R), _stream(stream)))
    return residual_out, hs, A, S, R


def rotate_quant_i8(x, rec, cs, out=None, stream=None):
    """Per-group int8 mode: x f16 [M, K], rec [P, 8, K/2, 8], cs f16 [P, K] -> (A int8 [P, M, K],
    ASG f32 [P, M, G], RS f32 [P, M, G])."""
    import torch
    return _rotate_quant_common("pq_rotate_quant_i8", x, rec, cs, out, stream, torch.int8)


def gemm_i8(A, ASG, RS, wpk, sz, N, pb1=NO_BOUNDARY, pb2=NO_BOUNDARY, out=None, workspace=None, stream=None):
    """Per-group int8 GEMM: A int8 [P, M, K], ASG/RS f32 [P, M, G], packed weights -> y bf16."""
    import torch
    return _gemm_common("pq_gemm_i8", A, ASG, RS, wpk, sz, N, pb1, pb2, out, workspace, stream, a_dtype=torch.int8)


def rotate_quant_tok(x, rec, cs, out=None, stream=None):
    """Per-token path: x f16 [M, K], rec [P, 8, K/2, 8], cs f16 [P, K] -> (A u8 [P, M, K],
    AS f32 [P, M], RS f32 [P, M, G])."""
    import torch
    return _rotate_quant_common("pq_rotate_quant_tok", x, rec, cs, out, stream, torch.uint8, tok=True)


def gemm_tok_workspace_bytes(M, N, K):
    if M > INT_MAX or N > INT_MAX or K > INT_MAX:
        _too_large(M=M, N=N, K=K)
    return int(lib().pq_gemm_tok_workspace_bytes(M, N, K))


def gemm_tok(A, AS, RS, wpk, sz, N, pb1=NO_BOUNDARY, pb2=NO_BOUNDARY, out=None, workspace=None, stream=None):
    """Per-token GEMM: A u8 [P, M, K], AS f32 [P, M], RS f32 [P, M, G], packed weights -> y bf16."""
    import torch
    return _gemm_common("pq_gemm_tok", A, AS, RS, wpk, sz, N, pb1, pb2, out, workspace, stream,
                        a_dtype=torch.uint8, tok=True)


GATE_ACTS = {"none": 0, "sigmoid": 1, "tanh": 2}


def block_norms(x, residual, w_post=None, gate=None, w_pre=None, eps=1e-6, scale=1.0, res_scale=1.0, gate_act="none",
                gemma=False, residual_out=None, out=None, stream=None):
    """The norms before and after a block, its gate and the residual scale in one launch:
    ``n = rmsnorm(x, w_post)`` (``x`` without ``w_post``), ``h = res_scale * residual + scale * a(gate) * n``,
    ``hs = rmsnorm(h, w_pre)`` from the stored ``h`` -> (h, hs), hs None without ``w_pre``.

    x f16 or bf16 [M, K]; residual f16, bf16 or f32 [M, K]; w_post, w_pre [K] of hs's type (f16 or bf16);
    gate of x's type: [K] (one row for every token), [M, K], or [M, 1] (one value per token); gate_act "none",
    "sigmoid" or "tanh". gemma: the norms multiply by 1 + w. residual_out may be ``residual`` itself (in place).
    K a multiple of 8 up to 32768; rows of 2-D tensors start on 16-byte lines."""
    f = _native() if _fast is None else _fast
    if f and stream is None:
        done = f.block_norms(x, residual, w_post, gate, w_pre, eps, scale, res_scale, GATE_ACTS.get(gate_act), gemma, residual_out, out)
        if done is not NotImplemented:
            return done
    import torch
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x: expected a [M, K] tensor")
    if not isinstance(residual, torch.Tensor):
        raise TypeError("residual: expected a tensor")
    M, K = x.shape
    if M > INT_MAX or K > INT_MAX:
        _too_large(M=M, K=K)
    xt = _type_code(x.dtype, "x")
    rt = _type_code(residual.dtype, "residual", 3)
    act = GATE_ACTS.get(gate_act)
    if act is None:
        raise ValueError(f"gate_act: {gate_act!r}, expected one of {', '.join(GATE_ACTS)}")
    specs, rows = [], [(x, "x", x.dtype, (M, K)), (residual, "residual", residual.dtype, (M, K))]
    wt = w_pre.dtype if isinstance(w_pre, torch.Tensor) else w_post.dtype if isinstance(w_post, torch.Tensor) else torch.float16
    ot = _type_code(wt, "w_post" if w_pre is None else "w_pre")
    if w_post is not None:
        specs.append((w_post, "w_post", wt, (K,)))
    if w_pre is not None:
        specs.append((w_pre, "w_pre", wt, (K,)))
    ldg, gcols = 0, K
    if gate is not None:
        if isinstance(gate, torch.Tensor) and gate.dim() == 1:
            specs.append((gate, "gate", x.dtype, (K,)))
        else:
            gcols = 1 if isinstance(gate, torch.Tensor) and gate.dim() == 2 and gate.shape[1] == 1 else K
            if gcols == 1:
                gate = gate.as_strided((M, 1), (gate.stride(0), 1)) if gate.shape[0] == M else gate
            rows.append((gate, "gate", x.dtype, (M, gcols)))
    if residual_out is not None:
        rows.append((residual_out, "residual_out", residual.dtype, (M, K)))
    if out is not None:
        if w_pre is None:
            raise ValueError("out: nothing is written there without w_pre")
        rows.append((out, "out", wt, (M, K)))
    _validate(specs, rows=rows)
    if gate is not None and gate.dim() == 2:
        ldg = _pitch(gate, M, gcols)
    if residual_out is None:
        residual_out = _new((M, K), residual.dtype, x.device, stream)
    if out is None and w_pre is not None:
        out = _new((M, K), wt, x.device, stream)
    _launch("pq_block_norms", x.device, stream,
            x.data_ptr(), _pitch(x, M, K), xt, residual.data_ptr(), _pitch(residual, M, K), rt, _addr(w_post), _addr(gate), ldg, gcols,
            act, _addr(w_pre), float(eps), float(scale), float(res_scale), 1 if gemma else 0, M, K,
            residual_out.data_ptr(), _pitch(residual_out, M, K), _addr(out), K if out is None else _pitch(out, M, K), ot)
    return residual_out, out


def e4m3_encode(q, stream=None):
    """float32 CUDA tensor -> uint8 codes with the prologue's device encoder."""
    import torch
    _need(q, torch.float32, "q")
    out = torch.empty(q.shape, dtype=torch.uint8, device=q.device)
    _check("pq_e4m3_encode", lib().pq_e4m3_encode(_ptr(q), _ptr(out), q.numel(), _stream(stream)))
    return out


def recip_f32(x, stream=None):
    """float32 CUDA tensor -> 1/x with the prologue's device reciprocal."""
    import torch
    _need(x, torch.float32, "x")
    out = torch.empty_like(x)
    _check("pq_recip_f32", lib().pq_recip_f32(_ptr(x), _ptr(out), x.numel(), _stream(stream)))
    return out


def bf16_round(x, stream=None):
    """float32 CUDA tensor -> int16 tensor of bf16 bit patterns with the GEMM's device rounding."""
    import torch
    _need(x, torch.float32, "x")
    out = torch.empty(x.shape, dtype=torch.int16, device=x.device)
    _check("pq_bf16_round", lib().pq_bf16_round(_ptr(x), _ptr(out), x.numel(), _stream(stream)))
    return out
