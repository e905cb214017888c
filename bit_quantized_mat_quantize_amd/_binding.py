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


def version() -> str:
    return load().qmm_version().decode()
