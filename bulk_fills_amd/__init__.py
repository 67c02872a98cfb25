"""Python binding of libtk (include/tk.h): counter-based random bulk fills on MI355X.

Argument marshalling only: every function has the name of its C entry point, takes the
same arguments in the same order, passes device pointers and the HIP stream through, and
raises TkError on a non-zero status.  All computation happens in the HIP kernels of
libtk.so; there is no CPU fallback, and importing this package without the built library
fails.

A buffer argument may be a torch tensor on a HIP device (its data_ptr is passed after a
check that it holds n elements of the right size) or a raw device address (int).
`stream` defaults to torch's current stream of the tensor's device; pass an int handle or
a torch.cuda.Stream to choose another.
"""
import ctypes as C
import functools
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtk.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'` "
        "(bulk_fills_amd has no CPU fallback)")

# torch ships its own HIP runtime (libamdhip64.so.7).  Loading it first lets libtk bind to
# that same runtime; loading libtk first would bring a second HIP/HSA runtime into the
# process, and one of the two would then find no device.
try:
    import torch  # noqa: F401
except ImportError:  # the C library still loads on its own
    torch = None

lib = C.CDLL(LIB_PATH)

TK_OK, TK_EINVAL, TK_ERANGE, TK_ENOMEM, TK_EHIP = 0, 1, 2, 3, 4
TK_RESIDUAL_F32, TK_PARAMS_F32 = 1, 2  # flags of the row operators
TK_INDEX_I64, TK_ACCUMULATE, TK_INTERLEAVED = 8, 16, 32  # and of those on tokens and heads

_u32, _u64, _i32, _i64, _f32 = C.c_uint32, C.c_uint64, C.c_int32, C.c_int64, C.c_float
_p = C.c_void_p

# C signatures (argument types in declaration order; every fill returns tk_status).
SIGNATURES = {
    "tk_fill_u8": [_u32, _u64, _u64, _p, _p],
    "tk_fill_u16": [_u32, _u64, _u64, _p, _p],
    "tk_fill_u32": [_u32, _u64, _u64, _p, _p],
    "tk_fill_u64": [_u32, _u64, _u64, _p, _p],
    "tk_fill_f16_bits": [_u32, _u64, _u64, _p, _p],
    "tk_fill_f32": [_u32, _u64, _u64, _p, _p],
    "tk_fill_f64": [_u32, _u64, _u64, _p, _p],
    "tk_fill_bool": [_u32, _u64, _u64, _p, _p],
    "tk_fill_u32_below": [_u32, _u64, _u64, _u32, _p, _p],
    "tk_fill_u64_below": [_u32, _u64, _u64, _u64, _p, _p],
    "tk_fill_i32_below": [_u32, _u64, _u64, _i32, _u32, _p, _p],
    "tk_fill_i64_below32": [_u32, _u64, _u64, _i64, _u32, _p, _p],
    "tk_fill_i64_below": [_u32, _u64, _u64, _i64, _u64, _p, _p],
    "tk_fill_normal_f64": [_u32, _u64, _u64, _p, _p],
    "tk_fill_normal_f32": [_u32, _u64, _u64, _p, _p],
    "tk_fill_normal_f32_half_turn": [_u32, _u64, _u64, _p, _p],
    "tk_fill_randn_f32": [_u32, _u64, _u64, _p, _p],
    "tk_fill_exponential_f64": [_u32, _u64, _u64, _p, _p],
    "tk_fill_exponential_f32": [_u32, _u64, _u64, _p, _p],
    "tk_dropout_f32": [_u32, _u64, _u64, _f32, _p, _p, _p, _p],
    "tk_dropout_backward_f32": [_u32, _u64, _u64, _f32, _p, _p, _p],
    "tk_alias_create": [_p, _u32, _p],
    "tk_alias_destroy": [_p],
    "tk_alias_export": [_p, _p, _p],
    "tk_alias_build_host": [_p, _u32, _p, _p],
    "tk_fill_choice_u32": [_u32, _u64, _u64, _p, _p, _p],
    "tk_philox_fill_u32": [_u64, _u64, _u64, _p, _p],
    "tk_philox_fill_u64": [_u64, _u64, _u64, _p, _p],
    "tk_philox_fill_f32": [_u64, _u64, _u64, _p, _p],
    "tk_philox_fill_f64": [_u64, _u64, _u64, _p, _p],
    "tk_philox_fill_u32_below": [_u64, _u64, _u64, _u32, _p, _p],
    "tk_philox_fill_u64_below": [_u64, _u64, _u64, _u64, _p, _p],
    "tk_philox_fill_choice_u32": [_u64, _u64, _u64, _p, _p, _p],
    "tk_philox_fill_normal_f32": [_u64, _u64, _u64, _p, _p],
    "tk_philox_fill_normal_f64": [_u64, _u64, _u64, _p, _p],
    "tk_ziggurat_table": [_p, _p],
    "tk_debug_set_miss_capacity": [_u32, _u64],
    "tk_debug_last_miss_count": [_p],
    "tk_debug_set_normal_f64_mode": [_u32],
    "tk_debug_set_tunable": [C.c_char_p, _i64],
    "tk_debug_fail_allocations": [_u32, _u32],
    "tk_debug_device_bytes": [_p],
    "tk_fill_constant_u32": [_u32, _u64, _p, _p],
    "tk_fill_normal_f64_no_alloc": [_u32, _u64, _u64, _p, _p],
}
for _t in ("f32", "f16", "bf16"):
    SIGNATURES.update({
        f"tk_dropout_add_{_t}": [_u32, _u64, _u64, _u64, _f32, _u32, _p, _u64, _p, _p, _u64, _p, _u64, _p],
        f"tk_dropout_add_backward_{_t}": [_u32, _u64, _u64, _u64, _f32, _u32, _p, _u64, _p, _u64, _p, _p, _u64, _p],
        f"tk_layer_norm_{_t}": [_u64, _u64, _f32, _u32, _p, _u64, _p, _p, _p, _u64, _p, _p, _p],
        f"tk_layer_norm_backward_{_t}": [_u64, _u64, _u32, _p, _u64, _p, _u64, _p, _p, _p, _p, _u64, _p, _p, _p, _u64, _p],
        f"tk_dropout_add_layer_norm_{_t}": [_u32, _u64, _u64, _u64, _f32, _f32, _u32, _p, _u64, _p, _p, _u64, _p, _p, _p,
                                            _u64, _p, _u64, _p, _p, _p],
        f"tk_dropout_add_layer_norm_backward_{_t}": [_u32, _u64, _u64, _u64, _f32, _u32, _p, _u64, _p, _u64, _p, _u64, _p,
                                                     _p, _p, _p, _u64, _p, _u64, _p, _p, _p, _p, _u64, _p],
        f"tk_embedding_{_t}": [_u32, _u64, _u64, _u64, _f32, _f32, _u32, _u64, _p, _p, _u64, _p, _u64, _p],
        f"tk_embedding_backward_{_t}": [_u32, _u64, _u64, _u64, _f32, _f32, _u32, _u64, _p, _p, _u64, _p, _u64, _p, _u64, _p],
        f"tk_head_norm_rotate_{_t}": [_u64] * 5 + [_f32, _u32, _p, _u64, _p, _u64, _p, _p, _p, _u64, _p, _p, _p, _u64, _p,
                                                   _u64, _p],
        f"tk_head_norm_rotate_backward_{_t}": [_u64] * 5 + [_f32, _u32] + [_p, _u64] * 4 + [_p, _p, _p, _u64, _p, _p]
        + [_p, _u64] * 2 + [_p, _p, _p, _u64, _p],
        f"tk_checkpoint_{_t}": [_u32, _u64, _u64, _u64, _u32, _p, _u64, _p, _u64, _p, _p],
        f"tk_checkpoint_restore_{_t}": [_u64, _u64, _u32, _p, _u64, _p, _p, _u64, _p],
        f"tk_layer_norm_backward_checkpoint_{_t}": [_u64, _u64, _u32, _p, _u64, _p, _u64, _p, _p, _p, _p, _p, _u64, _p, _p,
                                                    _p, _u64, _p],
        f"tk_dropout_add_layer_norm_backward_checkpoint_{_t}": [_u32, _u64, _u64, _u64, _f32, _u32, _p, _u64, _p, _u64, _p,
                                                                _u64, _p, _p, _p, _p, _p, _u64, _p, _u64, _p, _p, _p, _p,
                                                                _u64, _p],
    })
SIGNATURES["tk_backward_workspace_bytes"] = [_u64, _u64, _p]
SIGNATURES["tk_embedding_workspace_bytes"] = [_u64, _u64, _u64, _p]
SIGNATURES["tk_head_norm_workspace_bytes"] = [_u64, _u64, _u64, _u64, _p]
for _name, _args in SIGNATURES.items():
    _fn = getattr(lib, _name)
    _fn.argtypes = _args
    _fn.restype = C.c_int
lib.tk_status_string.argtypes = [C.c_int]
lib.tk_status_string.restype = C.c_char_p
lib.tk_last_hip_error.argtypes = []
lib.tk_last_hip_error.restype = C.c_int
lib.tk_alias_size.argtypes = [_p]
lib.tk_alias_size.restype = C.c_uint32


class TkError(RuntimeError):
    def __init__(self, code, where):
        msg = lib.tk_status_string(code).decode()
        if code == TK_EHIP:
            msg += f" (hipError {lib.tk_last_hip_error()})"
        super().__init__(f"{where}: {msg}")
        self.code = code


def _check(code, where):
    if code != TK_OK:
        raise TkError(code, where)


def _buf(x, itemsize, n, where):
    """Device address of a buffer argument (tensor or int), checking size for tensors."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if not x.is_cuda:
        raise ValueError(f"{where}: buffer must live on a HIP device")
    import torch
    if x.device.index != torch.cuda.current_device():
        # the library launches on the calling thread's current device
        raise ValueError(f"{where}: buffer is on {x.device}, the current device is cuda:{torch.cuda.current_device()}")
    if x.element_size() != itemsize:
        raise ValueError(f"{where}: element size {x.element_size()} != {itemsize}")
    if not x.is_contiguous() or x.numel() < n:
        raise ValueError(f"{where}: need a contiguous buffer of at least {n} elements")
    return x.data_ptr()


def _stream(stream, *bufs):
    if isinstance(stream, int):
        return stream
    if stream is not None:
        return stream.cuda_stream
    import torch
    dev = next((b.device for b in bufs if b is not None and not isinstance(b, int)), None)
    return torch.cuda.current_stream(dev).cuda_stream


def _fill(cname, itemsize):
    fn = getattr(lib, cname)

    def call(key, start_draw, n, out, stream=None):
        _check(fn(key, start_draw, n, _buf(out, itemsize, n, cname), _stream(stream, out)), cname)

    call.__name__ = cname
    call.__doc__ = f"{cname}(key, start_draw, n, out, stream=None): see include/tk.h."
    return call


tk_fill_u8 = _fill("tk_fill_u8", 1)
tk_fill_u16 = _fill("tk_fill_u16", 2)
tk_fill_u32 = _fill("tk_fill_u32", 4)
tk_fill_u64 = _fill("tk_fill_u64", 8)
tk_fill_f16_bits = _fill("tk_fill_f16_bits", 2)
tk_fill_f32 = _fill("tk_fill_f32", 4)
tk_fill_f64 = _fill("tk_fill_f64", 8)
tk_fill_bool = _fill("tk_fill_bool", 1)
tk_fill_normal_f64 = _fill("tk_fill_normal_f64", 8)
tk_fill_normal_f32 = _fill("tk_fill_normal_f32", 4)
tk_fill_normal_f64_no_alloc = _fill("tk_fill_normal_f64_no_alloc", 8)
tk_fill_normal_f32_half_turn = _fill("tk_fill_normal_f32_half_turn", 4)
tk_fill_randn_f32 = _fill("tk_fill_randn_f32", 4)
tk_fill_exponential_f64 = _fill("tk_fill_exponential_f64", 8)
tk_fill_exponential_f32 = _fill("tk_fill_exponential_f32", 4)
tk_philox_fill_u32 = _fill("tk_philox_fill_u32", 4)
tk_philox_fill_u64 = _fill("tk_philox_fill_u64", 8)
tk_philox_fill_f32 = _fill("tk_philox_fill_f32", 4)
tk_philox_fill_f64 = _fill("tk_philox_fill_f64", 8)
tk_philox_fill_normal_f32 = _fill("tk_philox_fill_normal_f32", 4)
tk_philox_fill_normal_f64 = _fill("tk_philox_fill_normal_f64", 8)


def tk_fill_constant_u32(value, n, out, stream=None):
    _check(lib.tk_fill_constant_u32(value, n, _buf(out, 4, n, "tk_fill_constant_u32"), _stream(stream, out)),
           "tk_fill_constant_u32")


def tk_philox_fill_u32_below(key, start_draw, n, bound, out, stream=None):
    _check(lib.tk_philox_fill_u32_below(key, start_draw, n, bound, _buf(out, 4, n, "tk_philox_fill_u32_below"),
                                        _stream(stream, out)), "tk_philox_fill_u32_below")


def tk_philox_fill_u64_below(key, start_draw, n, bound, out, stream=None):
    _check(lib.tk_philox_fill_u64_below(key, start_draw, n, bound, _buf(out, 8, n, "tk_philox_fill_u64_below"),
                                        _stream(stream, out)), "tk_philox_fill_u64_below")


def tk_fill_u32_below(key, start_draw, n, bound, out, stream=None):
    _check(lib.tk_fill_u32_below(key, start_draw, n, bound, _buf(out, 4, n, "tk_fill_u32_below"),
                                 _stream(stream, out)), "tk_fill_u32_below")


def tk_fill_u64_below(key, start_draw, n, bound, out, stream=None):
    _check(lib.tk_fill_u64_below(key, start_draw, n, bound, _buf(out, 8, n, "tk_fill_u64_below"),
                                 _stream(stream, out)), "tk_fill_u64_below")


def tk_fill_i32_below(key, start_draw, n, low, bound, out, stream=None):
    _check(lib.tk_fill_i32_below(key, start_draw, n, low, bound, _buf(out, 4, n, "tk_fill_i32_below"),
                                 _stream(stream, out)), "tk_fill_i32_below")


def tk_fill_i64_below32(key, start_draw, n, low, bound, out, stream=None):
    _check(lib.tk_fill_i64_below32(key, start_draw, n, low, bound, _buf(out, 8, n, "tk_fill_i64_below32"),
                                   _stream(stream, out)), "tk_fill_i64_below32")


def tk_fill_i64_below(key, start_draw, n, low, bound, out, stream=None):
    _check(lib.tk_fill_i64_below(key, start_draw, n, low, bound, _buf(out, 8, n, "tk_fill_i64_below"),
                                 _stream(stream, out)), "tk_fill_i64_below")


def tk_dropout_f32(key, start_draw, n, p, x, y, mask=None, stream=None):
    _check(lib.tk_dropout_f32(key, start_draw, n, p, _buf(x, 4, n, "tk_dropout_f32"),
                              _buf(y, 4, n, "tk_dropout_f32"), _buf(mask, 1, n, "tk_dropout_f32"),
                              _stream(stream, y)), "tk_dropout_f32")


def tk_dropout_backward_f32(key, start_draw, n, p, dy, dx, stream=None):
    _check(lib.tk_dropout_backward_f32(key, start_draw, n, p, _buf(dy, 4, n, "tk_dropout_backward_f32"),
                                       _buf(dx, 4, n, "tk_dropout_backward_f32"), _stream(stream, dx)),
           "tk_dropout_backward_f32")


@functools.lru_cache(maxsize=256)
def tk_backward_workspace_bytes(rows, cols):
    """Device bytes that the row operators' backward calls need for their column sums."""
    v = C.c_uint64()
    _check(lib.tk_backward_workspace_bytes(rows, cols, C.byref(v)), "tk_backward_workspace_bytes")
    return v.value


@functools.lru_cache(maxsize=256)
def tk_embedding_workspace_bytes(rows, cols, vocab):
    """Device bytes that the embedding's backward calls need."""
    v = C.c_uint64()
    _check(lib.tk_embedding_workspace_bytes(rows, cols, vocab, C.byref(v)), "tk_embedding_workspace_bytes")
    return v.value


@functools.lru_cache(maxsize=256)
def tk_head_norm_workspace_bytes(rows, heads_q, heads_k, dim):
    """Device bytes that the head norms' backward calls need for their sums."""
    v = C.c_uint64()
    _check(lib.tk_head_norm_workspace_bytes(rows, heads_q, heads_k, dim, C.byref(v)), "tk_head_norm_workspace_bytes")
    return v.value


# The current device and its current stream's handle, as torch.cuda.current_device() and
# torch.cuda.current_stream() give them, without making a Stream object for every call (1.1 of the
# 8.7 us that one row's layer norm took on the host); by those where torch lacks the names.
_get_device = getattr(getattr(torch, "_C", None), "_cuda_getDevice", None)
_raw_stream = getattr(getattr(torch, "_C", None), "_cuda_getCurrentRawStream", None)
_device_ready = False


def _device():
    """The current device's index, or -2 (no tensor's) where there is no device."""
    global _device_ready
    if not _device_ready:
        if not torch.cuda.is_available():
            return -2
        torch.cuda.init()
        _device_ready = True
    return _get_device()


if _get_device is None or _raw_stream is None:
    def _device():
        return torch.cuda.current_device() if torch.cuda.is_available() else -2

    def _raw_stream(dev):
        return torch.cuda.current_stream(dev).cuda_stream


_CODE_BLOCK = 128  # columns of a row that share a checkpoint's scale
_SUMS_ALONE = 8192  # columns up to which a backward call needs its workspace for column sums alone


def _refuse(where, x, dtype, dev, need):
    """Raises what is wrong with a buffer of a row operator."""
    if x.dtype is not dtype:
        raise ValueError(f"{where}: a buffer's type is {x.dtype}, not {dtype}")
    if x.get_device() < 0:
        raise ValueError(f"{where}: buffer must live on a HIP device")
    if x.get_device() != dev:  # the library launches on the calling thread's current device
        raise ValueError(f"{where}: buffer is on {x.device}, the current device is cuda:{dev}")
    raise ValueError(f"{where}: need {need}, got shape {tuple(x.shape)}, strides {x.stride()}")


def _matrix(where, dev, x, ld, rows, cols, dtype):
    """(address, ld) of a row operator's matrix: a tensor of rows x cols on the current device
    `dev` (any shape that flattens to it, or two dimensions with the last contiguous), whose row
    distance is taken where the call gives None for its ld; or a raw address (ld None: cols)."""
    if x is None:
        return None, 0
    if isinstance(x, int):
        return x, cols if ld is None else ld
    if x.dtype is dtype and x.get_device() == dev:
        if x.is_contiguous():
            if x.numel() == rows * cols and (ld is None or ld == cols or rows <= 1):
                return x.data_ptr(), cols if ld is None else ld
        elif x.shape == (rows, cols):
            to_next, within = x.stride()
            own = cols if rows <= 1 else to_next  # one row has no distance to a next
            if (within == 1 or cols == 1) and own >= cols and (ld is None or ld == own or rows <= 1):
                return x.data_ptr(), own if ld is None else ld
    _refuse(where, x, dtype, dev, f"a {rows} x {cols} matrix with contiguous rows that do not overlap (and its own row "
                                  f"distance as ld, or None; here {ld})")


def _vector(where, dev, x, n, dtype):
    """Address of a contiguous vector of n elements on the current device."""
    if x is None or isinstance(x, int):
        return x
    if x.dtype is dtype and x.get_device() == dev and x.numel() == n and x.is_contiguous():
        return x.data_ptr()
    _refuse(where, x, dtype, dev, f"a contiguous vector of {n} elements")


def _on(where, stream, dev):
    """The handle of a call's stream: the current device's current one for None."""
    if stream is None:
        return _raw_stream(dev)
    if isinstance(stream, int):
        return stream
    if stream.device_index != dev:  # the kernels are the current device's, as the buffers are
        raise ValueError(f"{where}: the stream is cuda:{stream.device_index}'s, the current device is cuda:{dev}")
    return stream.cuda_stream


def _workspace(where, dev, x, stream, needed, size, *sizes):
    """(address, bytes, what keeps it alive) of a workspace: a tensor, a pair (address, bytes), or an
    address of as many bytes as `size` names.  None allocates it with torch, in the order of the
    current stream: for a call on another stream the caller passes one."""
    if isinstance(x, tuple):
        return x[0], x[1], None
    if isinstance(x, int):
        return x, size(*sizes), None
    if x is None:
        n = size(*sizes) if needed else 0
        if n == 0:
            return None, 0, None
        if stream is not None and _on(where, stream, dev) != _raw_stream(dev):
            raise ValueError(f"{where}: a call on a stream that is not the current one needs a workspace")
        x = torch.empty(n, dtype=torch.uint8, device=dev)
        return x.data_ptr(), n, x
    if x.get_device() != dev or not x.is_contiguous():
        _refuse(where, x, x.dtype, dev, "a contiguous workspace")
    return x.data_ptr(), x.numel() * x.element_size(), x


def _row_operators(suffix, dtype):
    """The row operators for one element type, under the names of their C entry points."""
    add_fwd, add_bwd = getattr(lib, "tk_dropout_add_" + suffix), getattr(lib, "tk_dropout_add_backward_" + suffix)
    norm_fwd, norm_bwd = getattr(lib, "tk_layer_norm_" + suffix), getattr(lib, "tk_layer_norm_backward_" + suffix)
    both_fwd = getattr(lib, "tk_dropout_add_layer_norm_" + suffix)
    both_bwd = getattr(lib, "tk_dropout_add_layer_norm_backward_" + suffix)
    float32 = torch.float32
    name_dropout_add, name_dropout_add_backward = "tk_dropout_add_" + suffix, "tk_dropout_add_backward_" + suffix
    name_layer_norm, name_layer_norm_backward = "tk_layer_norm_" + suffix, "tk_layer_norm_backward_" + suffix
    name_dropout_add_layer_norm = "tk_dropout_add_layer_norm_" + suffix
    name_dropout_add_layer_norm_backward = "tk_dropout_add_layer_norm_backward_" + suffix

    def dropout_add(key, start_draw, rows, cols, p, flags, x, ldx, bias, residual, ldr, y, ldy, stream=None):
        w, dev = name_dropout_add, _device()
        res, par = float32 if flags & TK_RESIDUAL_F32 else dtype, float32 if flags & TK_PARAMS_F32 else dtype
        px, ldx = _matrix(w, dev, x, ldx, rows, cols, dtype)
        pr, ldr = _matrix(w, dev, residual, ldr, rows, cols, res)
        py, ldy = _matrix(w, dev, y, ldy, rows, cols, res)
        pb = _vector(w, dev, bias, cols, par)
        _check(add_fwd(key, start_draw, rows, cols, p, flags, px, ldx, pb, pr, ldr, py, ldy, _on(w, stream, dev)), w)

    def dropout_add_backward(key, start_draw, rows, cols, p, flags, dy, lddy, dx, lddx, dbias, workspace=None, stream=None):
        w, dev = name_dropout_add_backward, _device()
        res, par = float32 if flags & TK_RESIDUAL_F32 else dtype, float32 if flags & TK_PARAMS_F32 else dtype
        pdy, lddy = _matrix(w, dev, dy, lddy, rows, cols, res)
        pdx, lddx = _matrix(w, dev, dx, lddx, rows, cols, dtype)
        pb = _vector(w, dev, dbias, cols, par)
        ws, n, keep = _workspace(w, dev, workspace, stream, dbias is not None, tk_backward_workspace_bytes, rows, cols)
        _check(add_bwd(key, start_draw, rows, cols, p, flags, pdy, lddy, pdx, lddx, pb, ws, n, _on(w, stream, dev)), w)

    def layer_norm(rows, cols, eps, flags, x, ldx, gamma, beta, y, ldy, mean=None, rstd=None, stream=None):
        w, dev = name_layer_norm, _device()
        res, par = float32 if flags & TK_RESIDUAL_F32 else dtype, float32 if flags & TK_PARAMS_F32 else dtype
        px, ldx = _matrix(w, dev, x, ldx, rows, cols, res)
        py, ldy = _matrix(w, dev, y, ldy, rows, cols, dtype)
        pg, pb = _vector(w, dev, gamma, cols, par), _vector(w, dev, beta, cols, par)
        pm, ps = _vector(w, dev, mean, rows, float32), _vector(w, dev, rstd, rows, float32)
        _check(norm_fwd(rows, cols, eps, flags, px, ldx, pg, pb, py, ldy, pm, ps, _on(w, stream, dev)), w)

    def layer_norm_backward(rows, cols, flags, dy, lddy, x, ldx, gamma, mean, rstd, dx, lddx, dgamma, dbeta,
                            workspace=None, stream=None):
        w, dev = name_layer_norm_backward, _device()
        res, par = float32 if flags & TK_RESIDUAL_F32 else dtype, float32 if flags & TK_PARAMS_F32 else dtype
        pdy, lddy = _matrix(w, dev, dy, lddy, rows, cols, dtype)
        px, ldx = _matrix(w, dev, x, ldx, rows, cols, res)
        pdx, lddx = _matrix(w, dev, dx, lddx, rows, cols, res)
        pg, pdg, pdb = (_vector(w, dev, v, cols, par) for v in (gamma, dgamma, dbeta))
        pm, ps = _vector(w, dev, mean, rows, float32), _vector(w, dev, rstd, rows, float32)
        ws, n, keep = _workspace(w, dev, workspace, stream, cols > _SUMS_ALONE or dgamma is not None or dbeta is not None,
                                 tk_backward_workspace_bytes, rows, cols)
        _check(norm_bwd(rows, cols, flags, pdy, lddy, px, ldx, pg, pm, ps, pdx, lddx, pdg, pdb, ws, n,
                        _on(w, stream, dev)), w)

    def dropout_add_layer_norm(key, start_draw, rows, cols, p, eps, flags, x, ldx, bias, residual, ldr, gamma, beta, sum,
                               lds, y, ldy, mean=None, rstd=None, stream=None):
        w, dev = name_dropout_add_layer_norm, _device()
        res, par = float32 if flags & TK_RESIDUAL_F32 else dtype, float32 if flags & TK_PARAMS_F32 else dtype
        px, ldx = _matrix(w, dev, x, ldx, rows, cols, dtype)
        pr, ldr = _matrix(w, dev, residual, ldr, rows, cols, res)
        pv, lds = _matrix(w, dev, sum, lds, rows, cols, res)
        py, ldy = _matrix(w, dev, y, ldy, rows, cols, dtype)
        pb, pg, pt = (_vector(w, dev, v, cols, par) for v in (bias, gamma, beta))
        pm, ps = _vector(w, dev, mean, rows, float32), _vector(w, dev, rstd, rows, float32)
        _check(both_fwd(key, start_draw, rows, cols, p, eps, flags, px, ldx, pb, pr, ldr, pg, pt, pv, lds, py, ldy, pm, ps,
                        _on(w, stream, dev)), w)

    def dropout_add_layer_norm_backward(key, start_draw, rows, cols, p, flags, dy, lddy, dsum, ldds, sum, lds, gamma, mean,
                                        rstd, dx, lddx, dresidual, lddr, dgamma, dbeta, dbias, workspace=None, stream=None):
        w, dev = name_dropout_add_layer_norm_backward, _device()
        res, par = float32 if flags & TK_RESIDUAL_F32 else dtype, float32 if flags & TK_PARAMS_F32 else dtype
        pdy, lddy = _matrix(w, dev, dy, lddy, rows, cols, dtype)
        pds, ldds = _matrix(w, dev, dsum, ldds, rows, cols, res)
        pv, lds = _matrix(w, dev, sum, lds, rows, cols, res)
        pdx, lddx = _matrix(w, dev, dx, lddx, rows, cols, dtype)
        pdr, lddr = _matrix(w, dev, dresidual, lddr, rows, cols, res)
        pg, pdg, pdb, pdt = (_vector(w, dev, v, cols, par) for v in (gamma, dgamma, dbeta, dbias))
        pm, ps = _vector(w, dev, mean, rows, float32), _vector(w, dev, rstd, rows, float32)
        ws, n, keep = _workspace(w, dev, workspace, stream, cols > _SUMS_ALONE or dgamma is not None or dbeta is not None
                                 or dbias is not None, tk_backward_workspace_bytes, rows, cols)
        _check(both_bwd(key, start_draw, rows, cols, p, flags, pdy, lddy, pds, ldds, pv, lds, pg, pm, ps, pdx, lddx, pdr,
                        lddr, pdg, pdb, pdt, ws, n, _on(w, stream, dev)), w)

    return _named(suffix, dropout_add, dropout_add_backward, layer_norm, layer_norm_backward, dropout_add_layer_norm,
                  dropout_add_layer_norm_backward)


def _named(suffix, *functions):
    """The functions under the names of their C entry points."""
    out = {}
    for f in functions:
        f.__name__ = f.__qualname__ = f"tk_{f.__name__}_{suffix}"
        f.__doc__ = (f"{f.__name__}: see include/tk.h.  Matrices are rows x cols tensors (their ld may be None) or raw "
                     "addresses" + (", and a workspace of None is allocated." if "backward" in f.__name__ else "."))
        out[f.__name__] = f
    return out


def _heads(where, dev, x, ld, rows, heads, dim, dtype):
    """(address, ld) of a matrix of heads: as _matrix takes it, or a view of rows x heads x dim."""
    if x is not None and not isinstance(x, int) and x.dim() == 3 and not x.is_contiguous():
        to_next, apart, within = x.stride()
        if x.shape != (rows, heads, dim) or (heads > 1 and apart != dim) or (dim > 1 and within != 1):
            _refuse(where, x, dtype, dev, f"{rows} x {heads} x {dim} with a row's heads one after the other")
        x = x.as_strided((rows, heads * dim), (to_next, 1))
    return _matrix(where, dev, x, ld, rows, heads * dim, dtype)


def _token_operators(suffix, dtype):
    """The embedding, the head norms and the checkpoints for one element type, under the names of
    their C entry points."""
    emb_fwd, emb_bwd = getattr(lib, "tk_embedding_" + suffix), getattr(lib, "tk_embedding_backward_" + suffix)
    head_fwd = getattr(lib, "tk_head_norm_rotate_" + suffix)
    head_bwd = getattr(lib, "tk_head_norm_rotate_backward_" + suffix)
    pack, unpack = getattr(lib, "tk_checkpoint_" + suffix), getattr(lib, "tk_checkpoint_restore_" + suffix)
    norm_bwd = getattr(lib, "tk_layer_norm_backward_checkpoint_" + suffix)
    both_bwd = getattr(lib, "tk_dropout_add_layer_norm_backward_checkpoint_" + suffix)
    float32, int32, int64, int8 = torch.float32, torch.int32, torch.int64, torch.int8
    name_embedding, name_embedding_backward = "tk_embedding_" + suffix, "tk_embedding_backward_" + suffix
    name_head, name_head_backward = "tk_head_norm_rotate_" + suffix, "tk_head_norm_rotate_backward_" + suffix
    name_checkpoint, name_restore = "tk_checkpoint_" + suffix, "tk_checkpoint_restore_" + suffix
    name_norm_backward = "tk_layer_norm_backward_checkpoint_" + suffix
    name_both_backward = "tk_dropout_add_layer_norm_backward_checkpoint_" + suffix

    def embedding(key, start_draw, rows, cols, p, scale, flags, vocab, ids, table, ldt, y, ldy, stream=None):
        w, dev = name_embedding, _device()
        res, par = float32 if flags & TK_RESIDUAL_F32 else dtype, float32 if flags & TK_PARAMS_F32 else dtype
        pi = _vector(w, dev, ids, rows, int64 if flags & TK_INDEX_I64 else int32)
        pt, ldt = _matrix(w, dev, table, ldt, vocab, cols, par)
        py, ldy = _matrix(w, dev, y, ldy, rows, cols, res)
        _check(emb_fwd(key, start_draw, rows, cols, p, scale, flags, vocab, pi, pt, ldt, py, ldy, _on(w, stream, dev)), w)

    def embedding_backward(key, start_draw, rows, cols, p, scale, flags, vocab, ids, dy, lddy, dtable, lddt, workspace=None,
                           stream=None):
        w, dev = name_embedding_backward, _device()
        res, par = float32 if flags & TK_RESIDUAL_F32 else dtype, float32 if flags & TK_PARAMS_F32 else dtype
        pi = _vector(w, dev, ids, rows, int64 if flags & TK_INDEX_I64 else int32)
        pd, lddy = _matrix(w, dev, dy, lddy, rows, cols, res)
        pt, lddt = _matrix(w, dev, dtable, lddt, vocab, cols, par)
        ws, n, keep = _workspace(w, dev, workspace, stream, True, tk_embedding_workspace_bytes, rows, cols, vocab)
        _check(emb_bwd(key, start_draw, rows, cols, p, scale, flags, vocab, pi, pd, lddy, pt, lddt, ws, n,
                       _on(w, stream, dev)), w)

    def head_norm_rotate(rows, heads_q, heads_k, dim, rotary, eps, flags, q, ldq, k, ldk, gamma_q, gamma_k, positions,
                         table_rows, cosines, sines, yq, ldyq, yk, ldyk, stream=None):
        w, dev = name_head, _device()
        par, turns = float32 if flags & TK_PARAMS_F32 else dtype, table_rows * (rotary // 2)
        pq, ldq = _heads(w, dev, q, ldq, rows, heads_q, dim, dtype)
        pk, ldk = _heads(w, dev, k, ldk, rows, heads_k, dim, dtype)
        pgq, pgk = _vector(w, dev, gamma_q, dim, par), _vector(w, dev, gamma_k, dim, par)
        pp = _vector(w, dev, positions, rows, int64 if flags & TK_INDEX_I64 else int32)
        pc, ps = _vector(w, dev, cosines, turns, float32), _vector(w, dev, sines, turns, float32)
        pyq, ldyq = _heads(w, dev, yq, ldyq, rows, heads_q, dim, dtype)
        pyk, ldyk = _heads(w, dev, yk, ldyk, rows, heads_k, dim, dtype)
        _check(head_fwd(rows, heads_q, heads_k, dim, rotary, eps, flags, pq, ldq, pk, ldk, pgq, pgk, pp, table_rows, pc, ps,
                        pyq, ldyq, pyk, ldyk, _on(w, stream, dev)), w)

    def head_norm_rotate_backward(rows, heads_q, heads_k, dim, rotary, eps, flags, dyq, lddyq, dyk, lddyk, q, ldq, k, ldk,
                                  gamma_q, gamma_k, positions, table_rows, cosines, sines, dq, lddq, dk, lddk, dgamma_q,
                                  dgamma_k, workspace=None, stream=None):
        w, dev = name_head_backward, _device()
        par, turns = float32 if flags & TK_PARAMS_F32 else dtype, table_rows * (rotary // 2)
        pdyq, lddyq = _heads(w, dev, dyq, lddyq, rows, heads_q, dim, dtype)
        pdyk, lddyk = _heads(w, dev, dyk, lddyk, rows, heads_k, dim, dtype)
        pq, ldq = _heads(w, dev, q, ldq, rows, heads_q, dim, dtype)
        pk, ldk = _heads(w, dev, k, ldk, rows, heads_k, dim, dtype)
        pgq, pgk, pdgq, pdgk = (_vector(w, dev, v, dim, par) for v in (gamma_q, gamma_k, dgamma_q, dgamma_k))
        pp = _vector(w, dev, positions, rows, int64 if flags & TK_INDEX_I64 else int32)
        pc, ps = _vector(w, dev, cosines, turns, float32), _vector(w, dev, sines, turns, float32)
        pdq, lddq = _heads(w, dev, dq, lddq, rows, heads_q, dim, dtype)
        pdk, lddk = _heads(w, dev, dk, lddk, rows, heads_k, dim, dtype)
        ws, n, keep = _workspace(w, dev, workspace, stream, dgamma_q is not None or dgamma_k is not None,
                                 tk_head_norm_workspace_bytes, rows, heads_q, heads_k, dim)
        _check(head_bwd(rows, heads_q, heads_k, dim, rotary, eps, flags, pdyq, lddyq, pdyk, lddyk, pq, ldq, pk, ldk, pgq, pgk,
                        pp, table_rows, pc, ps, pdq, lddq, pdk, lddk, pdgq, pdgk, ws, n, _on(w, stream, dev)), w)

    def checkpoint(key, start_draw, rows, cols, flags, x, ldx, codes, ldc, scales, stream=None):
        w, dev = name_checkpoint, _device()
        px, ldx = _matrix(w, dev, x, ldx, rows, cols, float32 if flags & TK_RESIDUAL_F32 else dtype)
        pc, ldc = _matrix(w, dev, codes, ldc, rows, cols, int8)
        ps = _vector(w, dev, scales, rows * -(-cols // _CODE_BLOCK), float32)
        _check(pack(key, start_draw, rows, cols, flags, px, ldx, pc, ldc, ps, _on(w, stream, dev)), w)

    def checkpoint_restore(rows, cols, flags, codes, ldc, scales, y, ldy, stream=None):
        w, dev = name_restore, _device()
        pc, ldc = _matrix(w, dev, codes, ldc, rows, cols, int8)
        ps = _vector(w, dev, scales, rows * -(-cols // _CODE_BLOCK), float32)
        py, ldy = _matrix(w, dev, y, ldy, rows, cols, float32 if flags & TK_RESIDUAL_F32 else dtype)
        _check(unpack(rows, cols, flags, pc, ldc, ps, py, ldy, _on(w, stream, dev)), w)

    def layer_norm_backward_checkpoint(rows, cols, flags, dy, lddy, codes, ldc, scales, gamma, mean, rstd, dx, lddx, dgamma,
                                       dbeta, workspace=None, stream=None):
        w, dev = name_norm_backward, _device()
        res, par = float32 if flags & TK_RESIDUAL_F32 else dtype, float32 if flags & TK_PARAMS_F32 else dtype
        pdy, lddy = _matrix(w, dev, dy, lddy, rows, cols, dtype)
        pc, ldc = _matrix(w, dev, codes, ldc, rows, cols, int8)
        pv = _vector(w, dev, scales, rows * -(-cols // _CODE_BLOCK), float32)
        pdx, lddx = _matrix(w, dev, dx, lddx, rows, cols, res)
        pg, pdg, pdb = (_vector(w, dev, v, cols, par) for v in (gamma, dgamma, dbeta))
        pm, ps = _vector(w, dev, mean, rows, float32), _vector(w, dev, rstd, rows, float32)
        ws, n, keep = _workspace(w, dev, workspace, stream, cols > _SUMS_ALONE or dgamma is not None or dbeta is not None,
                                 tk_backward_workspace_bytes, rows, cols)
        _check(norm_bwd(rows, cols, flags, pdy, lddy, pc, ldc, pv, pg, pm, ps, pdx, lddx, pdg, pdb, ws, n,
                        _on(w, stream, dev)), w)

    def dropout_add_layer_norm_backward_checkpoint(key, start_draw, rows, cols, p, flags, dy, lddy, dsum, ldds, codes, ldc,
                                                   scales, gamma, mean, rstd, dx, lddx, dresidual, lddr, dgamma, dbeta, dbias,
                                                   workspace=None, stream=None):
        w, dev = name_both_backward, _device()
        res, par = float32 if flags & TK_RESIDUAL_F32 else dtype, float32 if flags & TK_PARAMS_F32 else dtype
        pdy, lddy = _matrix(w, dev, dy, lddy, rows, cols, dtype)
        pds, ldds = _matrix(w, dev, dsum, ldds, rows, cols, res)
        pc, ldc = _matrix(w, dev, codes, ldc, rows, cols, int8)
        pv = _vector(w, dev, scales, rows * -(-cols // _CODE_BLOCK), float32)
        pdx, lddx = _matrix(w, dev, dx, lddx, rows, cols, dtype)
        pdr, lddr = _matrix(w, dev, dresidual, lddr, rows, cols, res)
        pg, pdg, pdb, pdt = (_vector(w, dev, v, cols, par) for v in (gamma, dgamma, dbeta, dbias))
        pm, ps = _vector(w, dev, mean, rows, float32), _vector(w, dev, rstd, rows, float32)
        ws, n, keep = _workspace(w, dev, workspace, stream, cols > _SUMS_ALONE or dgamma is not None or dbeta is not None
                                 or dbias is not None, tk_backward_workspace_bytes, rows, cols)
        _check(both_bwd(key, start_draw, rows, cols, p, flags, pdy, lddy, pds, ldds, pc, ldc, pv, pg, pm, ps, pdx, lddx, pdr,
                        lddr, pdg, pdb, pdt, ws, n, _on(w, stream, dev)), w)

    return _named(suffix, embedding, embedding_backward, head_norm_rotate, head_norm_rotate_backward, checkpoint,
                  checkpoint_restore, layer_norm_backward_checkpoint, dropout_add_layer_norm_backward_checkpoint)


if torch is not None:
    for _suffix, _dtype in (("f32", torch.float32), ("f16", torch.float16), ("bf16", torch.bfloat16)):
        globals().update(_row_operators(_suffix, _dtype))
        globals().update(_token_operators(_suffix, _dtype))


class Alias:
    """Owner of a tk_alias handle (tk_alias_create / tk_alias_destroy)."""

    def __init__(self, weights):
        import numpy as np
        w = np.ascontiguousarray(weights, dtype=np.float64)
        h = C.c_void_p()
        _check(lib.tk_alias_create(w.ctypes.data, w.size, C.byref(h)), "tk_alias_create")
        self.handle = h.value
        self.n = w.size

    def export(self):
        import numpy as np
        q = np.empty(self.n, dtype=np.uint32)
        a = np.empty(self.n, dtype=np.uint32)
        _check(lib.tk_alias_export(self.handle, q.ctypes.data, a.ctypes.data), "tk_alias_export")
        return q, a

    def close(self):
        if self.handle:
            _check(lib.tk_alias_destroy(self.handle), "tk_alias_destroy")
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def tk_alias_create(weights):
    return Alias(weights)


def tk_alias_build_host(weights):
    """The library's host alias construction alone: returns (q, alias) numpy arrays."""
    import numpy as np
    w = np.ascontiguousarray(weights, dtype=np.float64)
    q = np.empty(w.size, dtype=np.uint32)
    a = np.empty(w.size, dtype=np.uint32)
    _check(lib.tk_alias_build_host(w.ctypes.data, w.size, q.ctypes.data, a.ctypes.data), "tk_alias_build_host")
    return q, a


def tk_fill_choice_u32(key, start_draw, n, table, out, stream=None):
    _check(lib.tk_fill_choice_u32(key, start_draw, n, table.handle, _buf(out, 4, n, "tk_fill_choice_u32"),
                                  _stream(stream, out)), "tk_fill_choice_u32")


def tk_philox_fill_choice_u32(key, start_draw, n, table, out, stream=None):
    _check(lib.tk_philox_fill_choice_u32(key, start_draw, n, table.handle, _buf(out, 4, n, "tk_philox_fill_choice_u32"),
                                         _stream(stream, out)), "tk_philox_fill_choice_u32")


def tk_ziggurat_table():
    import numpy as np
    x = np.empty(1025, dtype=np.float64)
    f = np.empty(1025, dtype=np.float64)
    _check(lib.tk_ziggurat_table(x.ctypes.data, f.ctypes.data), "tk_ziggurat_table")
    return x, f


def tk_debug_set_miss_capacity(per_group, overflow):
    _check(lib.tk_debug_set_miss_capacity(per_group, overflow), "tk_debug_set_miss_capacity")


def tk_debug_set_normal_f64_mode(mode):
    _check(lib.tk_debug_set_normal_f64_mode(mode), "tk_debug_set_normal_f64_mode")


TUNABLES = ("store_nt", "max_blocks", "unroll", "choice_tiles", "exp_tiles", "zig_tiles", "zig_lds", "zig_fused",
            "philox_lds", "pair_lds", "lds_pad", "zig_lds_pad", "const_work")


def tk_debug_set_tunable(name, value):
    """Sets a launch tunable (see include/tk.h); a negative value restores the environment's."""
    _check(lib.tk_debug_set_tunable(name.encode(), int(value)), "tk_debug_set_tunable")


def tk_debug_fail_allocations(skip, count):
    _check(lib.tk_debug_fail_allocations(skip, count), "tk_debug_fail_allocations")


def tk_debug_device_bytes():
    v = C.c_uint64()
    _check(lib.tk_debug_device_bytes(C.byref(v)), "tk_debug_device_bytes")
    return v.value


def tk_debug_last_miss_count():
    v = C.c_uint64()
    _check(lib.tk_debug_last_miss_count(C.byref(v)), "tk_debug_last_miss_count")
    return v.value
