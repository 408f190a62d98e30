"""ctypes binding of librepro_gb300.so (declared in include/repro.h).

Argument marshalling only: every function passes tensor data pointers, sizes
and the current CUDA stream to the C ABI, which does all the work on the GPU.
There is no CPU fallback: if the library is missing, loading raises.
PyTorch supplies device memory and streams.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "librepro_gb300.so")
_lib = None

STATUS = {0: "ok", 1: "invalid argument", 2: "capacity", 3: "overlap", 4: "environment", 5: "cuda",
          6: "device timeout"}


class ReproError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = "%s: %s" % (where, lib().repro_strerror(status).decode())
        if status == 5:
            msg += " (cudaError %d)" % lib().repro_last_cuda_error()
        super().__init__(msg)


class Launch(ctypes.Structure):
    _fields_ = [("block", ctypes.c_int), ("grid", ctypes.c_int)]


def lib():
    """Load the shared library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("librepro_gb300.so is missing: run __graft_entry__.build() "
                               "(or compensated_bit_reproducible_gb300/build.py) first")
        L = ctypes.CDLL(LIB_PATH)
        P, S, I, I64, F = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int64, ctypes.c_float
        sig = {
            "repro_strerror": (ctypes.c_char_p, [I]),
            "repro_last_cuda_error": (I, []),
            "repro_max_count_f32": (ctypes.c_uint64, []),
            "repro_max_count_f64": (ctypes.c_uint64, []),
            "repro_max_k_f32": (I, []),
            "repro_max_k_f64": (I, []),
            "repro_validate_environment": (I, [P]),
            "repro_sum_f32": (I, [P, S, I, P, P]),
            "repro_sum_f64": (I, [P, S, I, P, P]),
            "repro_sum_f32_async": (I, [P, S, I, P, P, P]),
            "repro_sum_f64_async": (I, [P, S, I, P, P, P]),
            "repro_sum_f32_noalloc": (I, [P, S, I, P, P]),
            "repro_cumsum_f32": (I, [P, P, S, I, P]),
            "repro_cumsum_f64": (I, [P, P, S, I, P]),
            "repro_cumsum_f32_ex": (I, [P, P, S, I, P, P]),
            "repro_cumsum_f64_ex": (I, [P, P, S, I, P, P]),
            "repro_segsum_f32": (I, [P, I64, I64, I, I, P, P]),
            "stable_var_f32": (I, [P, I64, I64, I, I, P, P, P]),
            "twoterm_var_f32": (I, [P, I64, I64, I, I, P, P]),
            "stable_var_f64": (I, [P, I64, I64, I, I, P, P, P]),
            "stable_var_c64": (I, [P, I64, I64, I, I, P, P, P]),
            "stable_var_f32_variant": (I, [P, I64, I64, I, I, I, P, P, P]),
            "repro_compensated_chunk": (I, []),
            "repro_state_bytes": (S, [I]),
            "repro_embedding": (I, [P, I64, I64, I64, P, I64, F, I, P, I64, P]),
            "repro_embedding_grad": (I, [P, I64, P, I64, I64, I64, F, I, P, I64, P]),
            "stable_linear_xent": (I, [P, I64, I64, I64, P, I64, I64, P, I, P, P, P]),
            "stable_linear_xent_grad": (I, [P, P, I64, I64, I64, P, I64, I64, P, P, I, P, I64, P, I64, P]),
            "stable_layer_norm": (I, [P, I64, I64, I64, P, P, F, I, P, I64, P, P, P]),
            "stable_layer_norm_grad": (I, [P, I64, P, I64, I64, I64, P, P, P, I, P, I64, P, P, P]),
        }
        for t in ("f32", "f64"):
            sig["repro_state_init_" + t] = (I, [P, I, P])
            sig["repro_state_deposit_" + t] = (I, [P, P, S, I, P])
            sig["repro_state_merge_" + t] = (I, [P, P, I, P])
            sig["repro_state_finalize_" + t] = (I, [P, I, P, P])
            sig["repro_cumsum_from_state_" + t] = (I, [P, P, S, I, P, P])
        for mode in ("naive", "pairwise", "kahan", "neumaier"):
            for t in ("f32", "f64"):
                sig["repro_sum_%s_%s" % (mode, t)] = (I, [P, S, P, P])
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _empty_on(stream):
    """torch.empty for the outputs of a call on `stream`.  They belong to that
    stream, as the call's own work is the first to touch them; where it is not
    the current one, the caller may use and drop them on the current stream
    too, so they are not handed out again before both are past them."""
    return torch.empty if stream is None else functools.partial(_empty_of, stream)


def _empty_of(stream, *shape, dtype, device):
    current = torch.cuda.current_stream(device)
    if stream == current:
        return torch.empty(*shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        out = torch.empty(*shape, dtype=dtype, device=device)
    out.record_stream(current)
    return out


def _ptr(t: torch.Tensor):
    return ctypes.c_void_p(t.data_ptr()) if t.numel() else ctypes.c_void_p(0)


def _check(rc: int, where: str):
    if rc != 0:
        raise ReproError(rc, where)


def _sfx(t: torch.Tensor) -> str:
    if t.dtype == torch.float32:
        return "f32"
    if t.dtype == torch.float64:
        return "f64"
    raise TypeError("float32 or float64 tensor expected, got %s" % t.dtype)


def _launch(block: int = 0, grid: int = 0):
    if not block and not grid:
        return None
    return ctypes.byref(Launch(block, grid))


# ---------------------------------------------------------------- constants
def max_count(dtype) -> int:
    return int(lib().repro_max_count_f32() if dtype == torch.float32 else lib().repro_max_count_f64())


def max_k(dtype) -> int:
    return int(lib().repro_max_k_f32() if dtype == torch.float32 else lib().repro_max_k_f64())


def validate_environment(stream=None) -> None:
    _check(lib().repro_validate_environment(_stream(stream)), "repro_validate_environment")


# ---------------------------------------------------------------- binned sums
def repro_sum(x: torch.Tensor, K: int = 3, stream=None) -> float:
    """Synchronous binned sum of a contiguous 1-D tensor (device or host)."""
    sfx = _sfx(x)
    assert x.is_contiguous()
    out = (ctypes.c_float if sfx == "f32" else ctypes.c_double)()
    st = _stream(stream) if x.is_cuda or stream is not None else _stream()
    _check(getattr(lib(), "repro_sum_" + sfx)(_ptr(x), x.numel(), K, st, ctypes.byref(out)), "repro_sum_" + sfx)
    return out.value


def repro_sum_async(x: torch.Tensor, out: torch.Tensor, K: int = 3, block: int = 0, grid: int = 0,
                    stream=None) -> torch.Tensor:
    """Stream-ordered binned sum into the 1-element device tensor `out`."""
    sfx = _sfx(x)
    assert x.is_cuda and out.is_cuda and out.dtype == x.dtype and x.is_contiguous()
    _check(getattr(lib(), "repro_sum_%s_async" % sfx)(_ptr(x), x.numel(), K, _stream(stream), _ptr(out),
                                                      _launch(block, grid)), "repro_sum_%s_async" % sfx)
    return out


def repro_sum_noalloc(x: torch.Tensor, out: torch.Tensor, K: int = 3, stream=None) -> torch.Tensor:
    """Binned float sum whose workspace is a fixed device array inside the
    library: for callers that cannot allocate device memory (see
    include/repro.h).  Calls on one device must not overlap on the GPU."""
    assert x.is_cuda and out.is_cuda and x.dtype == torch.float32 and out.dtype == torch.float32
    assert x.is_contiguous()
    _check(lib().repro_sum_f32_noalloc(_ptr(x), x.numel(), K, _stream(stream), _ptr(out)), "repro_sum_f32_noalloc")
    return out


def repro_cumsum(x: torch.Tensor, out: torch.Tensor | None = None, K: int = 3, block: int = 0,
                 stream=None) -> torch.Tensor:
    """Binned cumulative sum; out may be x itself (in place).  x and out may
    be CUDA tensors or CPU tensors (plain host memory is copied by the
    library and the call then waits for the result)."""
    sfx = _sfx(x)
    assert x.is_contiguous()
    if out is None:
        out = _empty_on(stream if x.is_cuda else None)(x.shape, dtype=x.dtype, device=x.device)
    assert out.dtype == x.dtype and out.is_contiguous() and out.numel() == x.numel()
    _check(getattr(lib(), "repro_cumsum_%s_ex" % sfx)(_ptr(x), _ptr(out), x.numel(), K, _stream(stream),
                                                      _launch(block, 0)), "repro_cumsum_" + sfx)
    return out


def repro_segsum(x: torch.Tensor, axis: int = 1, K: int = 3, out: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    assert x.is_cuda and x.dtype == torch.float32 and x.dim() == 2 and x.is_contiguous()
    rows, cols = x.shape
    if out is None:
        out = _empty_on(stream)(rows if axis == 1 else cols, dtype=torch.float32, device=x.device)
    _check(lib().repro_segsum_f32(_ptr(x), rows, cols, axis, K, _ptr(out), _stream(stream)), "repro_segsum_f32")
    return out


# ------------------------------------------------------------------ variance
def stable_var(x: torch.Tensor, axis: int = 1, ddof: int = 0, out=None, mean_out=None, with_mean: bool = True,
               stream=None, variant: int = 0):
    """Variance kernel: (var, mean) per slice along `axis` of a 2-D float32,
    float64 or complex64 tensor.  `variant` (float32 only) selects one of the
    section 4 step changes (0 = the kernel)."""
    assert x.is_cuda and x.dim() == 2 and x.is_contiguous()
    rows, cols = x.shape
    ns = rows if axis == 1 else cols
    vdt = {torch.float32: torch.float32, torch.float64: torch.float64, torch.complex64: torch.float32}[x.dtype]
    if out is None:
        out = _empty_on(stream)(ns, dtype=vdt, device=x.device)
    if with_mean and mean_out is None:
        mean_out = _empty_on(stream)(ns, dtype=x.dtype, device=x.device)
    mp = _ptr(mean_out) if with_mean else ctypes.c_void_p(0)
    st = _stream(stream)
    if x.dtype == torch.float32:
        if variant:
            rc = lib().stable_var_f32_variant(_ptr(x), rows, cols, axis, ddof, variant, _ptr(out), mp, st)
            _check(rc, "stable_var_f32_variant")
        else:
            _check(lib().stable_var_f32(_ptr(x), rows, cols, axis, ddof, _ptr(out), mp, st), "stable_var_f32")
    elif x.dtype == torch.float64:
        assert variant == 0
        _check(lib().stable_var_f64(_ptr(x), rows, cols, axis, ddof, _ptr(out), mp, st), "stable_var_f64")
    else:
        assert variant == 0
        _check(lib().stable_var_c64(_ptr(x), rows, cols, axis, ddof, _ptr(out), mp, st), "stable_var_c64")
    return out, mean_out


def twoterm_var(x: torch.Tensor, axis: int = 1, ddof: int = 0, out=None, stream=None) -> torch.Tensor:
    assert x.is_cuda and x.dtype == torch.float32 and x.dim() == 2 and x.is_contiguous()
    rows, cols = x.shape
    if out is None:
        out = _empty_on(stream)(rows if axis == 1 else cols, dtype=torch.float32, device=x.device)
    _check(lib().twoterm_var_f32(_ptr(x), rows, cols, axis, ddof, _ptr(out), _stream(stream)), "twoterm_var_f32")
    return out


# ---------------------------------------------------------- comparison sums
def compare_sum(x: torch.Tensor, mode: str, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """mode in naive / pairwise / kahan / neumaier; result in a 1-element device tensor."""
    sfx = _sfx(x)
    assert x.is_cuda and x.is_contiguous()
    if out is None:
        out = _empty_on(stream)(1, dtype=x.dtype, device=x.device)
    name = "repro_sum_%s_%s" % (mode, sfx)
    _check(getattr(lib(), name)(_ptr(x), x.numel(), _ptr(out), _stream(stream)), name)
    return out


def compensated_chunk() -> int:
    return int(lib().repro_compensated_chunk())


# ------------------------------------------------------------ binned states
def _tsfx(dtype) -> str:
    if dtype == torch.float32:
        return "f32"
    if dtype == torch.float64:
        return "f64"
    raise TypeError("float32 or float64 expected, got %s" % dtype)


def state_bytes(K: int = 3) -> int:
    return int(lib().repro_state_bytes(K))


def state_new(dtype, K: int = 3, device=None, stream=None) -> torch.Tensor:
    """A fresh (empty) binned state for `dtype` sums: a uint8 device tensor."""
    n = state_bytes(K)
    if n == 0:
        raise ReproError(1, "repro_state_bytes")
    st = _empty_on(stream)(n, dtype=torch.uint8, device=device or torch.device("cuda", torch.cuda.current_device()))
    state_init(st, dtype, K, stream)
    return st


def state_init(state: torch.Tensor, dtype, K: int = 3, stream=None) -> None:
    sfx = _tsfx(dtype)
    _check(getattr(lib(), "repro_state_init_" + sfx)(_ptr(state), K, _stream(stream)), "repro_state_init_" + sfx)


def state_deposit(state: torch.Tensor, x: torch.Tensor, K: int = 3, stream=None) -> None:
    sfx = _sfx(x)
    assert x.is_contiguous()
    _check(getattr(lib(), "repro_state_deposit_" + sfx)(_ptr(state), _ptr(x), x.numel(), K, _stream(stream)),
           "repro_state_deposit_" + sfx)


def state_merge(dst: torch.Tensor, src: torch.Tensor, dtype, K: int = 3, stream=None) -> None:
    sfx = _tsfx(dtype)
    _check(getattr(lib(), "repro_state_merge_" + sfx)(_ptr(dst), _ptr(src), K, _stream(stream)),
           "repro_state_merge_" + sfx)


def state_finalize(state: torch.Tensor, dtype, K: int = 3, out: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """Correctly rounded value of the state, as a one-element device tensor."""
    sfx = _tsfx(dtype)
    if out is None:
        out = _empty_on(stream)(1, dtype=dtype, device=state.device)
    _check(getattr(lib(), "repro_state_finalize_" + sfx)(_ptr(state), K, _ptr(out), _stream(stream)),
           "repro_state_finalize_" + sfx)
    return out


def repro_cumsum_from_state(x: torch.Tensor, state: torch.Tensor, K: int = 3, out: torch.Tensor | None = None,
                            stream=None) -> torch.Tensor:
    """Binned cumulative sum of x that starts from a binned state: out[i]
    is the binned sum of the state's contents and x[0..i].  Device tensors
    only; out may be x itself."""
    sfx = _sfx(x)
    assert x.is_contiguous() and state.dtype == torch.uint8
    if out is None:
        out = _empty_on(stream if x.is_cuda else None)(x.shape, dtype=x.dtype, device=x.device)
    assert out.dtype == x.dtype and out.is_contiguous() and out.numel() == x.numel()
    _check(getattr(lib(), "repro_cumsum_from_state_" + sfx)(_ptr(x), _ptr(out), x.numel(), K, _ptr(state),
                                                            _stream(stream)), "repro_cumsum_from_state_" + sfx)
    return out


# ---------------------------------------------------------- model operators
_TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


def _type(t: torch.Tensor) -> int:
    typ = _TYPES.get(t.dtype)
    if typ is None:
        raise TypeError("float32, float16 or bfloat16 tensor expected, got %s" % t.dtype)
    return typ


# These calls are short enough for the lookup of the current stream to show:
# the raw handle skips torch.cuda.Stream's construction (3 us of a 10 us call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


# Every tensor of a call is on one device, the first one's (`dev`), and that is
# the current one, where the C ABI launches.
def _stream_on(dev: int, stream) -> int:
    assert dev == _device()
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(dev)
    return torch.cuda.current_stream(dev).cuda_stream


def _mat(t: torch.Tensor, dev: int):
    """(pointer, rows, columns, row stride) of a 2-D tensor whose rows are
    contiguous.  A single row or none has no stride of its own."""
    assert t.get_device() == dev >= 0 and t.dim() == 2
    rows, cols = t.shape
    ld, one = t.stride()
    assert one == 1 or rows * cols <= 1 or cols <= 1
    return t.data_ptr(), rows, cols, (ld if rows > 1 else max(ld, cols))


def _vec(t: torch.Tensor | None, dtype, n: int, dev: int):
    if t is None:
        return None
    assert t.get_device() == dev and t.dtype == dtype and t.dim() == 1 and t.numel() == n and t.is_contiguous()
    return t.data_ptr()


def _out(out: torch.Tensor | None, rows: int, cols: int, like: torch.Tensor, dev: int, stream):
    """An output of `like`'s type: (tensor, pointer, row stride)."""
    if out is None:
        out = _empty_on(stream)(rows, cols, dtype=like.dtype, device=like.device)
        return out, out.data_ptr(), max(cols, 1)
    p, r, c, ld = _mat(out, dev)
    assert out.dtype == like.dtype and r == rows and c == cols
    return out, p, ld


def repro_embedding(weight: torch.Tensor, tokens: torch.Tensor, scale: float = 1.0, out: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """scale * weight[tokens]: [n, cols] for int64 tokens [n]; a negative
    token gives a zero row, one past the table a row of NaN."""
    dev = weight.get_device()
    w, vocab, cols, ldw = _mat(weight, dev)
    n = tokens.numel()
    out, o, ldo = _out(out, n, cols, weight, dev, stream)
    _check(lib().repro_embedding(w, vocab, cols, ldw, _vec(tokens, torch.int64, n, dev), n, scale, _type(weight), o,
                                 ldo, _stream_on(dev, stream)), "repro_embedding")
    return out


def repro_embedding_grad(dy: torch.Tensor, tokens: torch.Tensor, vocab: int, scale: float = 1.0,
                         out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gradient of repro_embedding to its table: [vocab, cols].  Each element
    is a binned sum (K = 3): its bits do not depend on the tokens' order."""
    dev = dy.get_device()
    y, n, cols, lddy = _mat(dy, dev)
    out, o, ldo = _out(out, vocab, cols, dy, dev, stream)
    _check(lib().repro_embedding_grad(y, lddy, _vec(tokens, torch.int64, n, dev), n, vocab, cols, scale, _type(dy), o,
                                      ldo, _stream_on(dev, stream)), "repro_embedding_grad")
    return out


def stable_layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                      eps: float = 1e-5, out: torch.Tensor | None = None, stream=None):
    """Layer norm of each row of a 2-D tensor: (y, mean, rstd), the last two
    float32.  out may be x itself."""
    dev = x.get_device()
    p, rows, cols, ldx = _mat(x, dev)
    out, o, ldo = _out(out, rows, cols, x, dev, stream)
    empty = _empty_on(stream)
    mean = empty(rows, dtype=torch.float32, device=x.device)
    rstd = empty(rows, dtype=torch.float32, device=x.device)
    _check(lib().stable_layer_norm(p, rows, cols, ldx, _vec(weight, x.dtype, cols, dev),
                                   _vec(bias, x.dtype, cols, dev), eps, _type(x), o, ldo, mean.data_ptr(),
                                   rstd.data_ptr(), _stream_on(dev, stream)), "stable_layer_norm")
    return out, mean, rstd


def stable_layer_norm_grad(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor | None, mean: torch.Tensor,
                           rstd: torch.Tensor, out: torch.Tensor | None = None, stream=None):
    """Gradient of stable_layer_norm: (dx, dweight, dbias).  out (for dx) may
    be dy itself."""
    dev = x.get_device()
    p, rows, cols, ldx = _mat(x, dev)
    y, dy_rows, dy_cols, lddy = _mat(dy, dev)
    assert dy.dtype == x.dtype and dy_rows == rows and dy_cols == cols
    out, o, ldo = _out(out, rows, cols, x, dev, stream)
    empty = _empty_on(stream)
    dweight = empty(cols, dtype=x.dtype, device=x.device)
    dbias = empty(cols, dtype=x.dtype, device=x.device)
    _check(lib().stable_layer_norm_grad(y, lddy, p, rows, cols, ldx, _vec(weight, x.dtype, cols, dev),
                                        _vec(mean, torch.float32, rows, dev), _vec(rstd, torch.float32, rows, dev),
                                        _type(x), o, ldo, dweight.data_ptr(), dbias.data_ptr(),
                                        _stream_on(dev, stream)), "stable_layer_norm_grad")
    return out, dweight, dbias


def stable_linear_xent(h: torch.Tensor, weight: torch.Tensor, labels: torch.Tensor, stream=None):
    """Softmax cross entropy of h @ weight.T (float16 or bfloat16) against
    int64 labels, without keeping the logits: (loss, lse), float32 per row.  A
    negative label gives loss 0."""
    dev = h.get_device()
    p, n, cols, ldh = _mat(h, dev)
    w, vocab, w_cols, ldw = _mat(weight, dev)
    assert weight.dtype == h.dtype and w_cols == cols
    empty = _empty_on(stream)
    loss = empty(n, dtype=torch.float32, device=h.device)
    lse = empty(n, dtype=torch.float32, device=h.device)
    _check(lib().stable_linear_xent(p, n, cols, ldh, w, vocab, ldw, _vec(labels, torch.int64, n, dev), _type(h),
                                    loss.data_ptr(), lse.data_ptr(), _stream_on(dev, stream)), "stable_linear_xent")
    return loss, lse


def stable_linear_xent_grad(dloss: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, labels: torch.Tensor,
                            lse: torch.Tensor, out=None, stream=None):
    """Gradient of stable_linear_xent for dloss (float32 per row): (dh,
    dweight).  out: a pair of tensors to write them to."""
    dev = h.get_device()
    p, n, cols, ldh = _mat(h, dev)
    w, vocab, w_cols, ldw = _mat(weight, dev)
    assert weight.dtype == h.dtype and w_cols == cols
    dh, dweight = out if out is not None else (None, None)
    dh, a, lddh = _out(dh, n, cols, h, dev, stream)
    dweight, b, lddw = _out(dweight, vocab, cols, h, dev, stream)
    _check(lib().stable_linear_xent_grad(_vec(dloss, torch.float32, n, dev), p, n, cols, ldh, w, vocab, ldw,
                                         _vec(labels, torch.int64, n, dev), _vec(lse, torch.float32, n, dev),
                                         _type(h), a, lddh, b, lddw, _stream_on(dev, stream)),
           "stable_linear_xent_grad")
    return dh, dweight
