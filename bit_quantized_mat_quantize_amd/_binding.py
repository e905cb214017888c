"""ctypes binding of libqmm (include/qmm.h): argument marshalling only.

Every computation runs in the HIP kernels of ``libqmm.so``; this module checks
that it was handed torch tensors on the GPU, passes their device pointers and
the current HIP stream, and turns a non-zero status into :class:`QmmError`.
There is no fallback: if ``libqmm.so`` is missing, importing the entry points
raises.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libqmm.so")

# enums of include/qmm.h
Q8_0, Q8_K = 0, 1
Q4_0, Q4_K, Q6_K, Q2_K = 0, 1, 2, 3
CANONICAL, REPACKED = 0, 1
ALGO_AUTO, ALGO_GEMV, ALGO_MFMA, ALGO_SKINNY = 0, 1, 2, 3
F32, F16, BF16 = 0, 1, 2
STATUS = {0: "QMM_OK", 1: "QMM_EINVAL", 2: "QMM_EALIGN", 3: "QMM_EUNSUPPORTED", 4: "QMM_EDEVICE"}

_ACT = {"q8_0": Q8_0, "q8_K": Q8_K}
_WEIGHT = {"q4_0": Q4_0, "q4_K": Q4_K, "q6_K": Q6_K, "q2_K": Q2_K}
_LAYOUT = {"canonical": CANONICAL, "repacked": REPACKED}
_ALGO = {"auto": ALGO_AUTO, "gemv": ALGO_GEMV, "mfma": ALGO_MFMA, "skinny": ALGO_SKINNY}


class _Cache(ctypes.Structure):
    """qmm_cache of include/qmm.h."""
    _fields_ = [("data", ctypes.c_void_p), ("bytes", ctypes.c_size_t), ("pages", ctypes.c_int64),
                ("page", ctypes.c_int64), ("heads", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("table", ctypes.c_void_p), ("seqs", ctypes.c_int64), ("width", ctypes.c_int64),
                ("lens", ctypes.c_void_p), ("starts", ctypes.c_void_p), ("rows", ctypes.c_int64)]


class QmmError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}: {detail}")


_lib = None


def load() -> ctypes.CDLL:
    """Load libqmm.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m bit_quantized_mat_quantize_amd.build`")
    # torch first: its HIP runtime must be the one libqmm binds to (loading
    # libqmm first would bring in the system runtime under the same soname)
    import torch  # noqa: F401
    lib = ctypes.CDLL(LIB_PATH)
    P, I64, SZ, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
    C, D = ctypes.POINTER(_Cache), ctypes.c_double
    sigs = {
        "qmm_act_bytes": (SZ, [I, I64, I64]),
        "qmm_weight_bytes": (SZ, [I, I, I64, I64]),
        "qmm_quantize_row_q8": (I, [I, P, I64, I64, P, SZ, P]),
        "qmm_quantize_weights": (I, [I, P, I64, I64, P, SZ, P]),
        "qmm_repack_weights": (I, [I, P, I64, I64, P, SZ, P]),
        "qmm_mul_mat_q4_0": (I, [P, SZ, I, P, SZ, P, SZ, I64, I64, I64, P]),
        "qmm_mul_mat_q4_K": (I, [P, SZ, I, P, SZ, P, SZ, I64, I64, I64, P]),
        "qmm_mul_mat_q4_K_ex": (I, [P, SZ, I, P, SZ, P, SZ, I64, I64, I64, I, P]),
        "qmm_mul_mat_q6_K": (I, [P, SZ, I, P, SZ, P, SZ, I64, I64, I64, P]),
        "qmm_mul_mat_q6_K_ex": (I, [P, SZ, I, P, SZ, P, SZ, I64, I64, I64, I, P]),
        "qmm_mul_mat_q2_K": (I, [P, SZ, I, P, SZ, P, SZ, I64, I64, I64, P]),
        "qmm_mul_mat_q4_0_ex": (I, [P, SZ, I, P, SZ, P, SZ, I64, I64, I64, I, P]),
        "qmm_mul_mat_id_workspace_bytes": (SZ, [I64, I64, I64]),
        "qmm_mul_mat_id_q4_K": (I, [P, SZ, I64, I, P, SZ, I, P, I64, I64, P, SZ, I64, I64, P, SZ, I, P]),
        "qmm_mul_mat_id": (I, [I, P, SZ, I64, I, P, SZ, I, P, I64, I64, P, SZ, I64, I64, P, SZ, I, P]),
        "qmm_mul_mat_id_noalloc": (I, [I, P, SZ, I64, I, P, SZ, I, P, I64, I64, P, SZ, I64, I64, I, P]),
        "qmm_mul_mat_q2_K_ex": (I, [P, SZ, I, P, SZ, P, SZ, I64, I64, I64, I, P]),
        "qmm_quantize_mul_mat": (I, [I, P, SZ, I, P, P, SZ, P, SZ, I64, I64, I64, P]),
        "qmm_embed_rows": (I, [I, P, SZ, I, P, I64, ctypes.c_float, P, SZ, I64, I64, P]),
        "qmm_lora_workspace_bytes": (SZ, [I64, I64, I64, I64]),
        "qmm_lora_add": (I, [I, P, SZ, P, SZ, I64, I64, P, P, P, SZ, P, P, SZ, I64, P, SZ, I64, I64, I64, I64,
                             P, SZ, P]),
        "qmm_logprobs_workspace_bytes": (SZ, [I64, I64, I64]),
        "qmm_logprobs": (I, [I, P, SZ, I64, I64, I64, ctypes.c_float, P, SZ, I64, P, I64, P, P, I64, P, P,
                             P, SZ, P]),
        "qmm_mul_mat_logprobs_workspace_bytes": (SZ, [I64, I64, I64]),
        "qmm_mul_mat_logprobs": (I, [I, P, SZ, I, P, SZ, I64, I64, I64, ctypes.c_float, P, SZ, I64, P, I64, P, P, I64,
                                     P, P, P, SZ, P]),
        "qmm_rope": (I, [I, P, SZ, I64, I64, P, P, P, SZ, I64, I64, I64, I64, I64, I64, I, D, D, D, D, D, P]),
        "qmm_cache_bytes": (SZ, [I64, I64, I64, I64]),
        "qmm_cache_write": (I, [C, I, P, SZ, I64, P, SZ, I64, P]),
        "qmm_cache_read": (I, [C, I, P, SZ, P, SZ, P]),
        "qmm_cache_attention_workspace_bytes": (SZ, [I, I64, I64, I64, I64, I64, I64, I64, I, I]),
        "qmm_cache_attention": (I, [C, I, P, SZ, I64, I64, P, SZ, I64, ctypes.c_float, I, I64, P, P, I64, P, SZ, P]),
        "qmm_cache_evict": (I, [C, P, I64, I64, I64, P, I64, P, P, I64, P, P]),
        "qmm_debug_block_sums": (I, [I, P, SZ, I, P, SZ, P, SZ, I64, I64, I64, P]),
        "qmm_status_string": (ctypes.c_char_p, [I]),
        "qmm_last_error": (ctypes.c_char_p, []),
        "qmm_version": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(status: int, where: str) -> None:
    if status != 0:
        raise QmmError(status, where, load().qmm_last_error().decode())


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dev(t, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor (got device {t.device})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr()), t.numel() * t.element_size()


def act_bytes(fmt: str, M: int, K: int) -> int:
    return int(load().qmm_act_bytes(_ACT[fmt], M, K))


def weight_bytes(fmt: str, layout: str, N: int, K: int) -> int:
    return int(load().qmm_weight_bytes(_WEIGHT[fmt], _LAYOUT[layout], N, K))


def quantize_row_q8(x, fmt: str = "q8_K", out=None, stream=None):
    """fp32 [M, K] GPU tensor -> uint8 activation blocks (bit-exact Q8_0/Q8_K)."""
    import torch
    M, K = x.shape
    if x.dtype != torch.float32:
        raise ValueError("x must be float32")
    if out is None:
        out = torch.empty(max(act_bytes(fmt, M, K), 1), dtype=torch.uint8, device=x.device)
    px, _ = _dev(x, "x")
    py, ny = _dev(out, "y")
    _check(load().qmm_quantize_row_q8(_ACT[fmt], px, M, K, py, ny, _stream(stream)),
           "qmm_quantize_row_q8")
    return out


def quantize_weights(w, fmt: str = "q4_K", out=None, stream=None):
    """fp32 [N, K] GPU tensor -> canonical uint8 weight blocks."""
    import torch
    N, K = w.shape
    if w.dtype != torch.float32:
        raise ValueError("w must be float32")
    if out is None:
        out = torch.empty(max(weight_bytes(fmt, "canonical", N, K), 1), dtype=torch.uint8,
                          device=w.device)
    pw, _ = _dev(w, "w")
    po, no = _dev(out, "out")
    _check(load().qmm_quantize_weights(_WEIGHT[fmt], pw, N, K, po, no, _stream(stream)),
           "qmm_quantize_weights")
    return out


def repack_weights(w, fmt: str, N: int, K: int, out=None, stream=None):
    import torch
    if out is None:
        out = torch.empty(max(weight_bytes(fmt, "repacked", N, K), 1), dtype=torch.uint8,
                          device=w.device)
    pw, _ = _dev(w, "w_canon")
    po, no = _dev(out, "w_repacked")
    _check(load().qmm_repack_weights(_WEIGHT[fmt], pw, N, K, po, no, _stream(stream)),
           "qmm_repack_weights")
    return out


def mul_mat_q4_0(w, y, M: int, N: int, K: int, layout: str = "canonical", algo: str = "auto",
                 out=None, stream=None):
    import torch
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=y.device)
    pw, nw = _dev(w, "w")
    py, ny = _dev(y, "y")
    po, no = _dev(out, "out")
    _check(load().qmm_mul_mat_q4_0_ex(pw, nw, _LAYOUT[layout], py, ny, po, no, M, N, K,
                                      _ALGO[algo], _stream(stream)), "qmm_mul_mat_q4_0")
    return out


def mul_mat_q4_K(w, y, M: int, N: int, K: int, layout: str = "canonical", algo: str = "auto",
                 out=None, stream=None):
    import torch
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=y.device)
    pw, nw = _dev(w, "w")
    py, ny = _dev(y, "y")
    po, no = _dev(out, "out")
    _check(load().qmm_mul_mat_q4_K_ex(pw, nw, _LAYOUT[layout], py, ny, po, no, M, N, K,
                                      _ALGO[algo], _stream(stream)), "qmm_mul_mat_q4_K")
    return out


def quantize_mul_mat(wfmt: str, w, x, N: int, layout: str = "canonical", y=None, out=None,
                     stream=None):
    """out = mul_mat(w, quantize_row_q8(x)) in one call; returns (out, y).

    x: fp32 [M, K] GPU tensor; y receives the Q8 activation bytes.  For Q4_K
    and M == 1 the quantization runs inside the GEMV launch."""
    import torch
    M, K = x.shape
    if x.dtype != torch.float32:
        raise ValueError("x must be float32")
    afmt = ACT_FOR[wfmt]
    if y is None:
        y = torch.empty(max(act_bytes(afmt, M, K), 1), dtype=torch.uint8, device=x.device)
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=x.device)
    pw, nw = _dev(w, "w")
    px, _ = _dev(x, "x")
    py, ny = _dev(y, "y")
    po, no = _dev(out, "out")
    _check(load().qmm_quantize_mul_mat(_WEIGHT[wfmt], pw, nw, _LAYOUT[layout], px, py, ny, po, no,
                                       M, N, K, _stream(stream)), "qmm_quantize_mul_mat")
    return out, y


def mul_mat_q6_K(w, y, M: int, N: int, K: int, layout: str = "canonical", algo: str = "auto",
                 out=None, stream=None):
    import torch
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=y.device)
    pw, nw = _dev(w, "w")
    py, ny = _dev(y, "y")
    po, no = _dev(out, "out")
    _check(load().qmm_mul_mat_q6_K_ex(pw, nw, _LAYOUT[layout], py, ny, po, no, M, N, K,
                                      _ALGO[algo], _stream(stream)), "qmm_mul_mat_q6_K")
    return out


def mul_mat_q2_K(w, y, M: int, N: int, K: int, layout: str = "canonical", algo: str = "auto",
                 out=None, stream=None):
    import torch
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=y.device)
    pw, nw = _dev(w, "w")
    py, ny = _dev(y, "y")
    po, no = _dev(out, "out")
    _check(load().qmm_mul_mat_q2_K_ex(pw, nw, _LAYOUT[layout], py, ny, po, no, M, N, K,
                                      _ALGO[algo], _stream(stream)), "qmm_mul_mat_q2_K")
    return out


def mul_mat_id_workspace_bytes(T: int, U: int, E: int) -> int:
    return int(load().qmm_mul_mat_id_workspace_bytes(T, U, E))


def mul_mat_id(wfmt: str, w, E: int, y, ids, N: int, K: int, layout: str = "canonical",
               y_per_slot: bool = False, algo: str = "auto", out=None, workspace=None, stream=None):
    """out [T, U, N] fp32: slot u of token t multiplies expert ids[t, u]'s matrix
    in format `wfmt` (w = E matrices back to back) with activation row t (or
    t*U + u)."""
    import torch
    T, U = ids.shape
    if ids.dtype != torch.int32:
        raise ValueError("ids must be int32")
    if out is None:
        out = torch.empty((T, U, N), dtype=torch.float32, device=ids.device)
    if workspace is None:
        workspace = torch.empty(max(mul_mat_id_workspace_bytes(T, U, E), 16), dtype=torch.uint8,
                                device=ids.device)
    pw, nw = _dev(w, "w")
    py, ny = _dev(y, "y")
    pi, _ = _dev(ids, "ids")
    po, no = _dev(out, "out")
    pws, nws = _dev(workspace, "workspace")
    _check(load().qmm_mul_mat_id(_WEIGHT[wfmt], pw, nw, E, _LAYOUT[layout], py, ny, int(bool(y_per_slot)), pi,
                                 T, U, po, no, N, K, pws, nws, _ALGO[algo], _stream(stream)),
           "qmm_mul_mat_id")
    return out


def mul_mat_id_noalloc(wfmt: str, w, E: int, y, ids, N: int, K: int, layout: str = "canonical",
                       y_per_slot: bool = False, algo: str = "auto", out=None, stream=None):
    """mul_mat_id with the expert grouping in the library's own per-GPU scratch
    (no workspace argument; see qmm_mul_mat_id_noalloc)."""
    import torch
    T, U = ids.shape
    if ids.dtype != torch.int32:
        raise ValueError("ids must be int32")
    if out is None:
        out = torch.empty((T, U, N), dtype=torch.float32, device=ids.device)
    pw, nw = _dev(w, "w")
    py, ny = _dev(y, "y")
    pi, _ = _dev(ids, "ids")
    po, no = _dev(out, "out")
    _check(load().qmm_mul_mat_id_noalloc(_WEIGHT[wfmt], pw, nw, E, _LAYOUT[layout], py, ny, int(bool(y_per_slot)),
                                         pi, T, U, po, no, N, K, _ALGO[algo], _stream(stream)),
           "qmm_mul_mat_id_noalloc")
    return out


def mul_mat_id_q4_K(w, E: int, y, ids, N: int, K: int, layout: str = "canonical",
                    y_per_slot: bool = False, algo: str = "auto", out=None, workspace=None,
                    stream=None):
    return mul_mat_id("q4_K", w, E, y, ids, N, K, layout=layout, y_per_slot=y_per_slot, algo=algo,
                      out=out, workspace=workspace, stream=stream)


ACT_FOR = {"q4_0": "q8_0", "q4_K": "q8_K", "q6_K": "q8_K", "q2_K": "q8_K"}  # activation blocks each weight format takes


def mul_mat(wfmt: str, w, y, M: int, N: int, K: int, layout: str = "canonical", out=None,
            stream=None):
    """The mul_mat entry point of weight format `wfmt` (automatic dispatch by M)."""
    fn = {"q4_0": mul_mat_q4_0, "q4_K": mul_mat_q4_K, "q6_K": mul_mat_q6_K, "q2_K": mul_mat_q2_K}[wfmt]
    return fn(w, y, M, N, K, layout=layout, out=out, stream=stream)


def debug_block_sums(wfmt: str, w, y, M: int, N: int, K: int, layout: str = "canonical",
                     out=None, stream=None):
    """int32 [M, N, K/32] per-sub-block (Q4_K) or per-block (Q4_0) sums, or
    [M, N, K/16] per-group sums (Q6_K, Q2_K)."""
    import torch
    if out is None:
        out = torch.empty((M, N, K // (16 if wfmt in ("q6_K", "q2_K") else 32)), dtype=torch.int32,
                          device=y.device)
    pw, nw = _dev(w, "w")
    py, ny = _dev(y, "y")
    po, no = _dev(out, "P")
    _check(load().qmm_debug_block_sums(_WEIGHT[wfmt], pw, nw, _LAYOUT[layout], py, ny, po, no,
                                       M, N, K, _stream(stream)), "qmm_debug_block_sums")
    return out


# ---- the operators beside the projections.  They run on the device of their
# tensors (whichever is current) and on `stream`, by default that device's
# current one; what they allocate belongs to that stream.  A small call costs
# the host more than the GPU (one launch 3.3 us, one tensor 1.3 us by
# empty_strided, 1.7 by empty), so the checks are one expression where nothing is
# wrong, and say what is wrong one by one where something is.  The current stream is
# asked for as the hipStream_t it is (torch.cuda.current_stream builds an object
# first: 2 us).

def _gpu(**tensors) -> int:
    """The index of the one GPU that every tensor is on (None: not given)."""
    index = None
    for name, t in tensors.items():
        if t is None:
            continue
        i = t.get_device()
        if i < 0:
            raise ValueError(f"{name} must be a GPU tensor (got device {t.device})")
        if index is None:
            index = i
        elif i != index:
            raise ValueError(f"{name} is on {t.device}, not on cuda:{index}")
    return index


def _on(index: int, stream):
    """The context to allocate and launch in, where it is not the present one."""
    import torch
    if stream is None:
        return torch.cuda.device(index)
    if stream.device.index != index:
        raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{index}")
    return torch.cuda.stream(stream)


_FLOAT_TYPES = {}


def _float_type(t, name: str) -> int:
    if not _FLOAT_TYPES:
        import torch
        _FLOAT_TYPES.update({torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16})
    i = _FLOAT_TYPES.get(t.dtype)
    if i is None:
        raise ValueError(f"{name} must be float32, float16 or bfloat16 (got {t.dtype})")
    return i


def _is(t, name: str, dtype, *shape) -> None:
    """A contiguous tensor of this type and shape."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, {dtype} and of shape {shape} (got {t.dtype}, {tuple(t.shape)}, "
                         f"strides {t.stride()})")


def _rows(t, name: str, dtype, M: int, N: int):
    """(pointer, bytes from it to the last row's end, row stride) of a matrix with unit column stride."""
    if t.dtype is not dtype or t.shape != (M, N):
        raise ValueError(f"{name} must be {dtype} of shape {(M, N)} (got {t.dtype}, {tuple(t.shape)})")
    step, column = t.stride()
    if N > 1 and column != 1:
        raise ValueError(f"{name} must have unit stride along its rows")
    ld = step if M > 1 else N
    return t.data_ptr(), ((M - 1) * ld + N) * t.element_size() if M and N else 0, ld


def _ptr(t):
    return None if t is None else t.data_ptr()


def _written(torch, out) -> None:
    """Tells autograd that a given out has new values: a backward that saved the old ones raises."""
    torch.autograd.graph.increment_version(out)


def _no_backward(name: str):
    """The operators beside the projections have no backward; a result without one must not look like torch's."""
    return ValueError(f"{name} has no backward and one of its tensors requires a gradient: call it under "
                      "torch.no_grad(), or give it detached tensors")


def _new(torch, M: int, N: int, dtype, device):
    return torch.empty_strided((M, N), (N, 1), dtype=dtype, device=device)


def embed_rows(wfmt: str, w, ids, N: int, K: int, layout: str = "canonical", scale: float = 1.0,
               out=None, stream=None):
    """out [T, K] fp32 = scale * the rows ids (int32 [T]) of the packed table w [N, K], decoded.

    An id outside [0, N) gives a row of NaN.  A slice of ids that does not start on 16 bytes is refused; its
    clone() is not (so for the integer arguments of lora_add and logprobs)."""
    import torch
    if out is not None and out.requires_grad and torch.is_grad_enabled():
        raise _no_backward("embed_rows")
    (T,) = ids.shape
    if ids.dtype is not torch.int32 or not ids.is_contiguous():
        _is(ids, "ids", torch.int32, T)
    if not w.is_contiguous():
        raise ValueError("w must be contiguous")
    index = ids.get_device()
    if index < 0 or w.get_device() != index or (out is not None and out.get_device() != index):
        _gpu(ids=ids, w=w, out=out)
    if stream is not None or torch._C._cuda_getDevice() != index:
        with _on(index, stream):
            return embed_rows(wfmt, w, ids, N, K, layout, scale, out)
    given = out is not None
    if not given:
        out = _new(torch, T, K, torch.float32, ids.device)
    else:
        _is(out, "out", torch.float32, T, K)
    _check(load().qmm_embed_rows(_WEIGHT[wfmt], w.data_ptr(), w.nbytes, _LAYOUT[layout], ids.data_ptr(), T, scale,
                                 out.data_ptr(), T * K * 4, N, K, torch._C._cuda_getCurrentRawStream(index)),
           "qmm_embed_rows")
    if given:
        _written(torch, out)
    return out


def lora_workspace_bytes(M: int, R: int, K: int, E: int) -> int:
    return int(load().qmm_lora_workspace_bytes(M, R, K, E))


def lora_add(base, x, A, B, ids, scales=None, ranks=None, out=None, workspace=None, stream=None):
    """out [M, N] fp32 = base + scales[e] * (x A_e^T) B_e^T with e = ids[m] (int32 [M]; -1: base alone).

    x: fp32 [M, K], the projection's input; A [E, R, K], B [E, N, R]: float32, float16 or bfloat16; scales
    fp32 [E]; ranks int32 [E], each adapter's own rank (at most R).  base and out may be column ranges of
    wider matrices; out=base adds in place.  Without `out` a new tensor is returned.  An id outside
    [-1, E) gives a row of NaN.  There is no backward: tensors that require a gradient are refused
    where gradients are recorded."""
    import torch
    if torch.is_grad_enabled() and (base.requires_grad or x.requires_grad or A.requires_grad or B.requires_grad or
                                    (scales is not None and scales.requires_grad) or
                                    (out is not None and out.requires_grad)):
        raise _no_backward("lora_add")
    (M, N), (E, R, K), t = base.shape, A.shape, A.dtype
    f32, i32 = torch.float32, torch.int32
    if not (x.dtype is f32 and B.dtype is t and ids.dtype is i32 and x.shape == (M, K) and B.shape == (E, N, R) and
            ids.shape == (M,) and x.is_contiguous() and A.is_contiguous() and B.is_contiguous() and
            ids.is_contiguous()):
        _is(x, "x", f32, M, K)
        _is(A, "A", t, E, R, K)
        _is(B, "B", t, E, N, R)
        _is(ids, "ids", i32, M)
    if scales is not None and not (scales.dtype is f32 and scales.shape == (E,) and scales.is_contiguous()):
        _is(scales, "scales", f32, E)
    if ranks is not None and not (ranks.dtype is i32 and ranks.shape == (E,) and ranks.is_contiguous()):
        _is(ranks, "ranks", i32, E)
    pb, nb, ldb = _rows(base, "base", f32, M, N)
    index = base.get_device()
    if not (0 <= index == x.get_device() == A.get_device() == B.get_device() == ids.get_device() and
            (scales is None or scales.get_device() == index) and (ranks is None or ranks.get_device() == index) and
            (out is None or out.get_device() == index) and (workspace is None or workspace.get_device() == index)):
        _gpu(base=base, x=x, A=A, B=B, ids=ids, scales=scales, ranks=ranks, out=out, workspace=workspace)
    if stream is not None or torch._C._cuda_getDevice() != index:
        with _on(index, stream):
            return lora_add(base, x, A, B, ids, scales, ranks, out, workspace)
    given = out is not None
    if not given:
        out = _new(torch, M, N, f32, base.device)
        po, no, ldo = out.data_ptr(), M * N * 4, N
    else:
        po, no, ldo = _rows(out, "out", f32, M, N)
    workspace, nw = _workspace(torch, workspace, load().qmm_lora_workspace_bytes(M, R, K, E), base.device)
    _check(load().qmm_lora_add(_float_type(A, "A"), A.data_ptr(), A.nbytes, B.data_ptr(), B.nbytes, E, R,
                               _ptr(scales), _ptr(ranks), x.data_ptr(), x.nbytes, ids.data_ptr(), pb, nb, ldb,
                               po, no, ldo, M, N, K, _ptr(workspace), nw, torch._C._cuda_getCurrentRawStream(index)),
           "qmm_lora_add")
    if given:
        _written(torch, out)
    return out


def logprobs_workspace_bytes(M: int, V: int, k: int) -> int:
    return int(load().qmm_logprobs_workspace_bytes(M, V, k))


def _logprob_inputs(M: int, V: int, tokens, mask):
    """(tokens per row, words from a mask row to the next, bytes of the mask), checked."""
    import torch
    G, mask_ld, mask_bytes = 0, 0, 0
    if tokens is not None:
        shape = tokens.shape
        if len(shape) not in (1, 2) or shape[0] != M:
            raise ValueError(f"tokens must have shape ({M},) or ({M}, G) (got {tuple(shape)})")
        G = shape[1] if len(shape) == 2 else 1
        if tokens.dtype is not torch.int32 or not tokens.is_contiguous():
            _is(tokens, "tokens", torch.int32, *shape)
    if mask is not None:
        rows, words = (1, mask.shape[0]) if mask.dim() == 1 else mask.shape
        if rows not in (1, M) or words < (V + 31) // 32:
            raise ValueError(f"mask must have 1 or {M} rows of at least {(V + 31) // 32} words (got {tuple(mask.shape)})")
        if mask.dtype is not torch.int32 or not mask.is_contiguous():
            _is(mask, "mask", torch.int32, *mask.shape)
        mask_ld, mask_bytes = words if rows > 1 else 0, mask.nbytes
    return G, mask_ld, mask_bytes


def _logprob_outputs(torch, M: int, k: int, tokens, entropy: bool, device):
    f32, new = torch.float32, torch.empty_strided
    lp = ent = top_ids = top_lp = None
    if tokens is not None:
        shape = tokens.shape
        lp = new(shape, (1,) if len(shape) == 1 else (shape[1], 1), dtype=f32, device=device)
    if entropy:
        ent = new((M,), (1,), dtype=f32, device=device)
    if k > 0:
        top_ids, top_lp = _new(torch, M, k, torch.int32, device), _new(torch, M, k, f32, device)
    return lp, ent, top_ids, top_lp


def _workspace(torch, given, need: int, device):
    """The caller's workspace, or a new one (None where nothing is needed), and its bytes."""
    if given is None:
        return (torch.empty_strided((need,), (1,), dtype=torch.uint8, device=device) if need else None), need
    if not given.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return given, given.nbytes


def logprobs(logits, tokens=None, k: int = 0, scale: float = 1.0, mask=None, entropy: bool = True,
             workspace=None, stream=None):
    """(token_logprobs, entropy, top_ids, top_logprobs) of logits [M, V] (float32, float16 or bfloat16).

    tokens: int32 [M] or [M, G], the tokens whose log probability is asked for (first result, fp32 of the
    same shape); entropy: fp32 [M]; k: that many most likely tokens (int32 and fp32 [M, k], -1 and -inf where
    there are fewer).  mask: int32 words [W], [1, W] or [M, W], W >= ceil(V / 32); bit i % 32 of word i // 32
    allows token i.  scale multiplies the logits (one over the temperature).  What is not asked for is None.
    There is no backward: logits that require a gradient are refused where gradients are recorded."""
    import torch
    if logits.requires_grad and torch.is_grad_enabled():
        raise _no_backward("logprobs")
    M, V = logits.shape
    G, mask_ld, mask_bytes = _logprob_inputs(M, V, tokens, mask)
    px, nx, ld = _rows(logits, "logits", logits.dtype, M, V)
    index = logits.get_device()
    if not (index >= 0 and (tokens is None or tokens.get_device() == index) and
            (mask is None or mask.get_device() == index) and (workspace is None or workspace.get_device() == index)):
        _gpu(logits=logits, tokens=tokens, mask=mask, workspace=workspace)
    if stream is not None or torch._C._cuda_getDevice() != index:
        with _on(index, stream):
            return logprobs(logits, tokens, k, scale, mask, entropy, workspace)
    device = logits.device
    lp, ent, top_ids, top_lp = out = _logprob_outputs(torch, M, k, tokens, entropy, device)
    workspace, nw = _workspace(torch, workspace, load().qmm_logprobs_workspace_bytes(M, V, k), device)
    _check(load().qmm_logprobs(_float_type(logits, "logits"), px, nx, ld, M, V, scale, _ptr(mask), mask_bytes,
                               mask_ld, _ptr(tokens), G, _ptr(lp), _ptr(ent), k, _ptr(top_ids), _ptr(top_lp),
                               _ptr(workspace), nw, torch._C._cuda_getCurrentRawStream(index)), "qmm_logprobs")
    return out


def mul_mat_logprobs_workspace_bytes(rows: int, N: int, k: int) -> int:
    return int(load().qmm_mul_mat_logprobs_workspace_bytes(rows, N, k))


def mul_mat_logprobs(wfmt: str, w, y, M: int, N: int, K: int, tokens=None, k: int = 0, scale: float = 1.0,
                     mask=None, entropy: bool = True, layout: str = "canonical", rows: int = 512, workspace=None,
                     stream=None):
    """logprobs of mul_mat(w, y) [M, N], `rows` rows at a time (or as many as a given workspace holds): the
    logits of all M rows need not exist at once.  w, y, M, N, K, layout as in mul_mat, the rest and the
    results as in logprobs."""
    import torch
    G, mask_ld, mask_bytes = _logprob_inputs(M, N, tokens, mask)
    if not (w.is_contiguous() and y.is_contiguous()):
        raise ValueError("w and y must be contiguous")
    if rows < 1:
        raise ValueError(f"rows = {rows}: at least one at a time")
    index = _gpu(w=w, y=y, tokens=tokens, mask=mask, workspace=workspace)
    if stream is not None or torch._C._cuda_getDevice() != index:
        with _on(index, stream):
            return mul_mat_logprobs(wfmt, w, y, M, N, K, tokens, k, scale, mask, entropy, layout, rows, workspace)
    lp, ent, top_ids, top_lp = out = _logprob_outputs(torch, M, k, tokens, entropy, w.device)
    at_once = min(M, max(rows, 8))
    workspace, nw = _workspace(torch, workspace, mul_mat_logprobs_workspace_bytes(at_once, N, k), w.device)
    _check(load().qmm_mul_mat_logprobs(_WEIGHT[wfmt], w.data_ptr(), w.nbytes, _LAYOUT[layout], y.data_ptr(), y.nbytes,
                                       M, N, K, scale, _ptr(mask), mask_bytes, mask_ld, _ptr(tokens), G, _ptr(lp),
                                       _ptr(ent), k, _ptr(top_ids), _ptr(top_lp), _ptr(workspace), nw,
                                       torch._C._cuda_getCurrentRawStream(index)), "qmm_mul_mat_logprobs")
    return out


# ---- between the projections: rotary positions, the 4-bit cache of keys and values, attention over it, eviction.

def rope_ramp(rot: int, base: float, length: int, factor: float, fast: float = 32.0, slow: float = 1.0):
    """rope's scaling arguments for a model trained on `length` positions and used on `factor` times as many, by the
    published YaRN method (Peng et al., "YaRN: Efficient Context Window Extension", 2023, its ramp over dimensions and its
    attention factor; the ends are whole pairs): pairs that turn more than `fast` times within `length` keep their angles, those of fewer than `slow` turns are slowed by
    `factor`, those between in part, and magnitude = 0.1 ln(factor) + 1."""
    import math

    def pair(turns):  # the pair that turns so often within the length
        return rot * math.log(length / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))
    low, high = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), rot - 1)
    return {"freq_scale": 1.0 / factor, "ramp": (float(low), float(max(high, low + 1))),
            "magnitude": 0.1 * math.log(factor) + 1.0 if factor > 1.0 else 1.0}


def _heads(t, name: str, T: int, H: int, D: int):
    """(bytes from the pointer to the last head's end, elements from a row to the next) of [T, H, D], heads side by side."""
    if t.shape != (T, H, D):
        raise ValueError(f"{name} must have shape {(T, H, D)} (got {tuple(t.shape)})")
    ld, head, one = t.stride()
    if one != 1 or (H > 1 and head != D):
        raise ValueError(f"{name} must have its heads side by side (strides {t.stride()})")
    if T < 2:
        ld = H * D
    return ((T - 1) * ld + H * D) * t.element_size() if T else 0, ld


def rope(x, positions, rot=None, layout: str = "half", base: float = 10000.0, freq_scale: float = 1.0, ramp=None,
         magnitude: float = 1.0, factors=None, out=None, stream=None):
    """Rotary positions of x [T, H, D] (float32, float16 or bfloat16; any strides but along D): out of the same shape.

    positions: int32 [T].  rot: how many elements of a head turn (all).  layout: "half" pairs element i with i + rot/2,
    "interleaved" 2i with 2i + 1.  theta_i = position * base^(-2i/rot), over factors[i] (fp32 [rot/2]) where given, times
    freq_scale for all pairs, or, with ramp = (low, high), from pair `low` to `high` more and more of it (rope_ramp).
    magnitude multiplies what turns.  out may be x.  There is no backward: an x that requires a gradient is refused
    where gradients are recorded."""
    import torch
    if (x.requires_grad or (out is not None and out.requires_grad) or
            (factors is not None and factors.requires_grad)) and torch.is_grad_enabled():
        raise _no_backward("rope")
    T, H, D = x.shape
    rot = D if rot is None else rot
    if layout not in ("half", "interleaved"):
        raise ValueError(f"layout = {layout!r}: half or interleaved")
    low, high = (0.0, 0.0) if ramp is None else ramp
    if ramp is not None and not high > low:
        raise ValueError(f"ramp = {ramp}: low below high")
    if positions.dtype is not torch.int32 or positions.shape != (T,) or not positions.is_contiguous():
        _is(positions, "positions", torch.int32, T)
    if factors is not None:
        _is(factors, "factors", torch.float32, rot // 2)
    ld_x, head_x, one = x.stride()
    if D > 1 and one != 1:
        raise ValueError("x must have unit stride along its heads")
    index = x.get_device()
    if not (0 <= index == positions.get_device() and (factors is None or factors.get_device() == index) and
            (out is None or out.get_device() == index)):
        _gpu(x=x, positions=positions, factors=factors, out=out)
    if stream is not None or torch._C._cuda_getDevice() != index:
        with _on(index, stream):
            return rope(x, positions, rot, layout, base, freq_scale, ramp, magnitude, factors, out)
    given = out is not None
    size = x.element_size()
    if not given:
        out = torch.empty_strided((T, H, D), (H * D, D, 1), dtype=x.dtype, device=x.device)
        ld_o, head_o = H * D, D
    else:
        if out.dtype is not x.dtype or out.shape != x.shape or (D > 1 and out.stride(2) != 1):
            raise ValueError(f"out must be {x.dtype} of shape {(T, H, D)} with unit stride along its heads (got "
                             f"{out.dtype}, {tuple(out.shape)}, strides {out.stride()})")
        ld_o, head_o, _ = out.stride()
    if T and H:
        nx, no = ((T - 1) * ld_x + (H - 1) * head_x + D) * size, ((T - 1) * ld_o + (H - 1) * head_o + D) * size
    else:
        nx = no = 0
    _check(load().qmm_rope(_float_type(x, "x"), x.data_ptr(), nx, ld_x, head_x, positions.data_ptr(), _ptr(factors),
                           out.data_ptr(), no, ld_o, head_o, T, H, D, rot, layout == "interleaved", base, freq_scale,
                           low, high, magnitude, torch._C._cuda_getCurrentRawStream(index)), "qmm_rope")
    if given:
        _written(torch, out)
    return out


def cache_bytes(pages: int, heads: int, dim: int, page: int = 64) -> int:
    return int(load().qmm_cache_bytes(pages, page, heads, dim))


def cache_new(pages: int, heads: int, dim: int, page: int = 64, device="cuda"):
    """A cache for keys and values: uint8 [pages, 2, heads, page, dim * 9 // 16] (the order of the bytes within a page is
    that of include/qmm.h).  It holds anything until rows are written."""
    import torch
    if not cache_bytes(pages, heads, dim, page):
        raise ValueError(f"no cache of {pages} pages of {page} entries, {heads} heads of {dim}: pages of 16, 32, .. 1024, "
                         "heads of 64, 96, 128, 192 or 256")
    return torch.empty((pages, 2, heads, page, dim * 9 // 16), dtype=torch.uint8, device=device)


def _cache(torch, cache, table, lens, starts, T):
    """(struct, heads, dim, sequences, pages of a table, entries of a page) of a cache and its batch, checked."""
    i32 = torch.int32
    if cache.dtype is not torch.uint8 or cache.dim() != 5 or not cache.is_contiguous() or cache.shape[1] != 2:
        raise ValueError(f"cache must be contiguous uint8 [pages, 2, heads, page, dim * 9 // 16] (got {cache.dtype}, "
                         f"{tuple(cache.shape)})")
    pages, _, heads, page, row = cache.shape
    if row % 18:
        raise ValueError(f"cache: {row} bytes an entry are no blocks of 18")
    dim = row * 16 // 9
    if table.dim() != 2 or table.dtype is not i32 or not table.is_contiguous():
        raise ValueError(f"table must be contiguous int32 [sequences, pages] (got {table.dtype}, {tuple(table.shape)})")
    B, W = table.shape
    if lens.dtype is not i32 or lens.shape != (B,) or not lens.is_contiguous():
        _is(lens, "lens", i32, B)
    if starts is not None and (starts.dtype is not i32 or starts.shape != (B + 1,) or not starts.is_contiguous()):
        _is(starts, "starts", i32, B + 1)
    return (_Cache(cache.data_ptr(), cache.nbytes, pages, page, heads, dim, table.data_ptr(), B, W, lens.data_ptr(),
                   None if starts is None else starts.data_ptr(), T), heads, dim, B, W, page)


def cache_write(cache, k, v, table, lens, starts=None, stream=None):
    """Writes rows of keys and values, k and v [T, heads, dim] (float32, float16 or bfloat16; heads side by side), into
    the cache as 4-bit blocks.

    table: int32 [B, pages], the pages of each sequence; lens: int32 [B], its entries with the new rows; starts: int32
    [B + 1], sequence b has the rows starts[b] .. starts[b + 1] - 1 (None: row b is sequence b's).  The last of a
    sequence's rows becomes its entry lens[b] - 1.  Rows of no sequence, and those whose page is not in the cache, are
    left out.  There is no backward: k and v that require a gradient are refused where gradients are recorded."""
    import torch
    if (k.requires_grad or v.requires_grad) and torch.is_grad_enabled():
        raise _no_backward("cache_write")
    T = k.shape[0]
    c, heads, dim, _, _, _ = _cache(torch, cache, table, lens, starts, T)
    nk, ldk = _heads(k, "k", T, heads, dim)
    nv, ldv = _heads(v, "v", T, heads, dim)
    if v.dtype is not k.dtype:
        raise ValueError(f"k is {k.dtype}, v {v.dtype}")
    index = cache.get_device()
    if not (0 <= index == k.get_device() == v.get_device() == table.get_device() == lens.get_device() and
            (starts is None or starts.get_device() == index)):
        _gpu(cache=cache, k=k, v=v, table=table, lens=lens, starts=starts)
    if stream is not None or torch._C._cuda_getDevice() != index:
        with _on(index, stream):
            return cache_write(cache, k, v, table, lens, starts)
    _check(load().qmm_cache_write(c, _float_type(k, "k"), k.data_ptr(), nk, ldk, v.data_ptr(), nv, ldv,
                                  torch._C._cuda_getCurrentRawStream(index)), "qmm_cache_write")
    _written(torch, cache)


def cache_read(cache, rows: int, table, lens, starts=None, dtype=None, stream=None):
    """(k, v) [rows, heads, dim] of `dtype` (float32): the entries that rows of the same table, lens and starts would be
    written to, as numbers.  An entry whose page is not in the cache is NaN; rows of no sequence hold anything."""
    import torch
    c, heads, dim, _, _, _ = _cache(torch, cache, table, lens, starts, rows)
    index = cache.get_device()
    if not (0 <= index == table.get_device() == lens.get_device() and (starts is None or starts.get_device() == index)):
        _gpu(cache=cache, table=table, lens=lens, starts=starts)
    if stream is not None or torch._C._cuda_getDevice() != index:
        with _on(index, stream):
            return cache_read(cache, rows, table, lens, starts, dtype)
    k, v = (torch.empty_strided((rows, heads, dim), (heads * dim, dim, 1), dtype=dtype or torch.float32,
                                device=cache.device) for _ in range(2))
    _check(load().qmm_cache_read(c, _float_type(k, "dtype"), k.data_ptr(), k.nbytes, v.data_ptr(), v.nbytes,
                                 torch._C._cuda_getCurrentRawStream(index)), "qmm_cache_read")
    return k, v


def cache_attention_workspace_bytes(q, heads: int, seqs: int, width: int, page: int, ragged: bool,
                                    mass: bool = False) -> int:
    """For q [T, q_heads, dim] over a cache of `heads` heads, with `seqs` tables of `width` pages; ragged: with starts.  That
    of the largest call serves those with fewer rows, sequences or pages, without lse, without starts and without mass."""
    rows, q_heads, dim = q.shape
    return int(load().qmm_cache_attention_workspace_bytes(_float_type(q, "q"), rows, q_heads, heads, dim, seqs, width, page, ragged, mass))


def cache_attention(q, cache, table, lens, starts=None, scale=None, causal: bool = True, window: int = 0, mass=None,
                    lse: bool = False, out=None, workspace=None, stream=None):
    """Attention of q [T, q_heads, dim] (float32, float16 or bfloat16; heads side by side) over the cache: out of the
    same shape and type, or (out, lse) with lse fp32 [T, q_heads].

    table, lens and starts as in cache_write: lens counts the rows of this call, whose keys and values are in the cache.
    Query heads h * q_heads / heads .. share cache head h.  scale: of the scores (1 / sqrt(dim)).  causal: a row sees
    the entries up to its own position; window > 0: of these the last `window`.  mass: fp32 [B, heads, n] with room for
    a whole table's entries, n >= pages * page: the weights that each entry gets, summed over rows and heads, are added
    to it.  A row that sees nothing gives 0 and lse -inf; one that sees an entry with a NaN, or whose page is not in the
    cache, gives NaN.  Rows of no sequence are left as they are (in a new out: they hold anything).  There is no
    backward: a q that requires a gradient is refused where gradients are recorded."""
    import torch
    if (q.requires_grad or (out is not None and out.requires_grad) or
            (mass is not None and mass.requires_grad)) and torch.is_grad_enabled():
        raise _no_backward("cache_attention")
    T, HQ, dim = q.shape
    c, heads, d, B, W, page = _cache(torch, cache, table, lens, starts, T)
    nq, ldq = _heads(q, "q", T, HQ, d)
    index = cache.get_device()
    if not (0 <= index == q.get_device() == table.get_device() == lens.get_device() and
            (starts is None or starts.get_device() == index) and (mass is None or mass.get_device() == index) and
            (out is None or out.get_device() == index) and (workspace is None or workspace.get_device() == index)):
        _gpu(cache=cache, q=q, table=table, lens=lens, starts=starts, mass=mass, out=out, workspace=workspace)
    if stream is not None or torch._C._cuda_getDevice() != index:
        with _on(index, stream):
            return cache_attention(q, cache, table, lens, starts, scale, causal, window, mass, lse, out, workspace)
    device, given, ld_mass = cache.device, out is not None, 0
    if mass is not None:
        if (mass.dtype is not torch.float32 or mass.dim() != 3 or mass.shape[:2] != (B, heads) or
                mass.shape[2] < W * page or not mass.is_contiguous()):
            raise ValueError(f"mass must be contiguous float32 [{B}, {heads}, {W * page} or more] (got {mass.dtype}, "
                             f"{tuple(mass.shape)}, strides {mass.stride()})")
        ld_mass = mass.shape[2]
    if not given:
        out = torch.empty_strided((T, HQ, dim), (HQ * dim, dim, 1), dtype=q.dtype, device=device)
        no, ldo = T * HQ * dim * q.element_size(), HQ * dim
    else:
        if out.dtype is not q.dtype:
            raise ValueError(f"out must be {q.dtype} (got {out.dtype})")
        no, ldo = _heads(out, "out", T, HQ, dim)
    stats = _new(torch, T, HQ, torch.float32, device) if lse else None
    lib = load()
    workspace, nw = _workspace(torch, workspace, lib.qmm_cache_attention_workspace_bytes(
        _float_type(q, "q"), T, HQ, heads, dim, B, W, page, starts is not None, mass is not None), device)
    _check(lib.qmm_cache_attention(c, _float_type(q, "q"), q.data_ptr(), nq, ldq, HQ, out.data_ptr(), no, ldo,
                                   dim ** -0.5 if scale is None else scale, causal, window, _ptr(stats), _ptr(mass),
                                   ld_mass, _ptr(workspace), nw, torch._C._cuda_getCurrentRawStream(index)),
           "qmm_cache_attention")
    if given:
        _written(torch, out)
    if mass is not None:
        _written(torch, mass)
    return (out, stats) if lse else out


def cache_evict(cache, table, lens, mass, budget: int, recent: int = 0, to=None, stream=None):
    """(lens, mass, ids) after at most `budget` entries of each sequence and head stay: the newest `recent` and, of the
    others, those of the largest mass (fp32 [B, heads, n] as in cache_attention), ties to the lower position.

    They move in their order within the sequences' own pages (to: None; no two sequences may share one then), or into
    those of `to` (int32 [B, pages]), which must be none of the table's: a copy of some of its columns is not refused, and
    entries would be read after others were written over them.  To keep a sequence's first pages alone, let `to` be None and
    cut the table after the call (its entries past lens are nobody's): table[:, :n].contiguous().  ids: int32 [B, heads, budget], where they
    were, -1 behind; mass: fp32 [B, heads, pages of `to` * page], 0 behind; lens: int32 [B]."""
    import torch
    if mass.requires_grad and torch.is_grad_enabled():
        raise _no_backward("cache_evict")
    c, heads, _, B, W, page = _cache(torch, cache, table, lens, None, 0)
    f32, i32 = torch.float32, torch.int32
    if (mass.dtype is not f32 or mass.dim() != 3 or mass.shape[:2] != (B, heads) or mass.shape[2] < W * page or
            not mass.is_contiguous()):
        raise ValueError(f"mass must be contiguous float32 [{B}, {heads}, {W * page} or more] (got {mass.dtype}, "
                         f"{tuple(mass.shape)}, strides {mass.stride()})")
    if to is None:
        to = table
    if to.dim() != 2 or to.shape[0] != B or to.dtype is not i32 or not to.is_contiguous():
        raise ValueError(f"to must be contiguous int32 [{B}, pages] (got {to.dtype}, {tuple(to.shape)})")
    if to.shape[1] * page < budget or not 0 <= recent <= budget or budget < 1:
        raise ValueError(f"budget = {budget}, recent = {recent}: recent <= budget <= the {to.shape[1] * page} entries of `to`")
    index = cache.get_device()
    if not 0 <= index == table.get_device() == lens.get_device() == mass.get_device() == to.get_device():
        _gpu(cache=cache, table=table, lens=lens, mass=mass, to=to)
    if stream is not None or torch._C._cuda_getDevice() != index:
        with _on(index, stream):
            return cache_evict(cache, table, lens, mass, budget, recent, to)
    new, device, wide = torch.empty_strided, cache.device, to.shape[1] * page
    lens_out = new((B,), (1,), dtype=i32, device=device)
    mass_out = new((B, heads, wide), (heads * wide, wide, 1), dtype=f32, device=device)
    ids = new((B, heads, budget), (heads * budget, budget, 1), dtype=i32, device=device)
    _check(load().qmm_cache_evict(c, mass.data_ptr(), mass.shape[2], budget, recent, to.data_ptr(), to.shape[1],
                                  lens_out.data_ptr(), mass_out.data_ptr(), wide, ids.data_ptr(),
                                  torch._C._cuda_getCurrentRawStream(index)), "qmm_cache_evict")
    _written(torch, cache)
    return lens_out, mass_out, ids


def version() -> str:
    return load().qmm_version().decode()
