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
    })
SIGNATURES["tk_backward_workspace_bytes"] = [_u64, _u64, _p]
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
        elif tuple(x.shape) == (rows, cols) and (cols == 1 or x.stride(1) == 1):
            own = cols if rows <= 1 else x.stride(0)  # one row has no distance to a next
            if own >= cols and (ld is None or ld == own or rows <= 1):
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


def _workspace(where, dev, x, stream, rows, cols, needed):
    """(address, bytes, what keeps it alive) of a workspace: a tensor, a pair (address, bytes), or an
    address of as many bytes as tk_backward_workspace_bytes names.  None allocates it with torch, in
    the order of the current stream: for a call on another stream the caller passes one."""
    if isinstance(x, tuple):
        return x[0], x[1], None
    if isinstance(x, int):
        return x, tk_backward_workspace_bytes(rows, cols), None
    if x is None:
        n = tk_backward_workspace_bytes(rows, cols) if needed else 0
        if n == 0:
            return None, 0, None
        if stream is not None and _on(where, stream, dev) != _raw_stream(dev):
            raise ValueError(f"{where}: a call on a stream that is not the current one needs a workspace")
        x = torch.empty(n, dtype=torch.uint8, device="cuda")
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
        ws, n, keep = _workspace(w, dev, workspace, stream, rows, cols, dbias is not None)
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
        ws, n, keep = _workspace(w, dev, workspace, stream, rows, cols,
                                 cols > _SUMS_ALONE or dgamma is not None or dbeta is not None)
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
        ws, n, keep = _workspace(w, dev, workspace, stream, rows, cols, cols > _SUMS_ALONE or dgamma is not None
                                 or dbeta is not None or dbias is not None)
        _check(both_bwd(key, start_draw, rows, cols, p, flags, pdy, lddy, pds, ldds, pv, lds, pg, pm, ps, pdx, lddx, pdr,
                        lddr, pdg, pdb, pdt, ws, n, _on(w, stream, dev)), w)

    out = {}
    for f in (dropout_add, dropout_add_backward, layer_norm, layer_norm_backward, dropout_add_layer_norm,
              dropout_add_layer_norm_backward):
        f.__name__ = f.__qualname__ = f"tk_{f.__name__}_{suffix}"
        f.__doc__ = (f"{f.__name__}: see include/tk.h.  Matrices are rows x cols tensors (their ld may be None) or raw "
                     "addresses" + (", and a workspace of None is allocated." if "backward" in f.__name__ else "."))
        out[f.__name__] = f
    return out


if torch is not None:
    globals().update(_row_operators("f32", torch.float32))
    globals().update(_row_operators("f16", torch.float16))
    globals().update(_row_operators("bf16", torch.bfloat16))


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
