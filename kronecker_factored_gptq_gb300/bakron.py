"""Thin ctypes binding over libbakron.so (argument marshalling only).

Every function here checks tensor devices/dtypes/shapes, allocates outputs
and workspaces with PyTorch (device memory and streams are all PyTorch is used
for), and calls the C entry point of the same name; every step of the solver
runs in the library's CUDA kernels.  There is no CPU path: if the library has
not been built, or no CUDA device is present, the first call raises.
"""

import ctypes
import os

_LIB = None
_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbakron.so")

OK = 0
STATUS = {0: "BAKRON_OK", 1: "BAKRON_ERR_INVALID_ARG", 2: "BAKRON_ERR_NOT_PD",
          3: "BAKRON_ERR_NONFINITE", 4: "BAKRON_ERR_CODE_RANGE", 5: "BAKRON_ERR_TIMEOUT",
          6: "BAKRON_ERR_UNSUPPORTED", 7: "BAKRON_ERR_CUDA"}
INT32_MIN = -(1 << 31)
INT32_MAX = (1 << 31) - 1

EXPORTS = ["bakron_default_opts", "bakron_status_string", "bakron_version", "bakron_kernel_launches",
           "bakron_workspace_size", "bakron_prepare_workspace_size", "bakron_rowscale",
           "bakron_prepare", "bakron_quantize", "bakron_quantize_antidiag",
           "bakron_quantize_noalloc", "bakron_factors_workspace_size", "bakron_factors",
           "bakron_grid_params", "bakron_quantize_grid", "bakron_batch_workspace_size",
           "bakron_quantize_batch", "bakron_schedule_export", "bakron_fma_probe", "bakron_sm_count",
           "bakron_plan_size", "bakron_plan_init", "bakron_async_status", "bakron_pack_size",
           "bakron_pack", "bakron_unpack", "bakron_linear_workspace_size", "bakron_linear",
           "bakron_linear_grad_workspace_size", "bakron_linear_grad", "bakron_moe_workspace_size",
           "bakron_moe", "bakron_layernorm", "bakron_layernorm_grad_workspace_size",
           "bakron_layernorm_grad"]
FACTORS_KFAC = 0
FACTORS_SHAMPOO = 1
F32, BF16, F16 = 0, 1, 2      # bakron_dtype
MOE_TOKENS = 32               # tokens that bakron_moe takes together


class PhaseTimes(ctypes.Structure):
    _fields_ = [("leaf_ms", ctypes.c_double), ("prop1_ms", ctypes.c_double),
                ("prop2_ms", ctypes.c_double), ("other_ms", ctypes.c_double),
                ("prop_flops", ctypes.c_double), ("leaf_launches", ctypes.c_int64),
                ("prop_launches", ctypes.c_int64), ("other_launches", ctypes.c_int64),
                ("near_ms", ctypes.c_double), ("near_launches", ctypes.c_int64)]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


class Opts(ctypes.Structure):
    _fields_ = [("tile", ctypes.c_int), ("leaf_width", ctypes.c_int), ("use_3xtf32", ctypes.c_int),
                ("spin_budget_cycles", ctypes.c_longlong), ("fault_inject", ctypes.c_int),
                ("times", ctypes.POINTER(PhaseTimes)), ("plan", ctypes.c_void_p)]


class Problem(ctypes.Structure):
    _fields_ = [("W", ctypes.c_void_p), ("m", ctypes.c_int64), ("n", ctypes.c_int64),
                ("UA", ctypes.c_void_p), ("UB", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("zero", ctypes.c_void_p), ("group", ctypes.c_int64), ("qmin", ctypes.c_int),
                ("qmax", ctypes.c_int), ("V", ctypes.c_void_p), ("codes", ctypes.c_void_p),
                ("status", ctypes.c_int)]


class Packed(ctypes.Structure):
    _fields_ = [("count", ctypes.c_int64), ("m", ctypes.c_int64), ("n", ctypes.c_int64),
                ("group", ctypes.c_int64), ("qmin", ctypes.c_int), ("has_zero", ctypes.c_int),
                ("data", ctypes.c_void_p), ("bytes", ctypes.c_size_t)]


class BakronError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        msg = lib().bakron_status_string(status).decode()
        super().__init__("%s: %s (%s)" % (where, STATUS.get(status, status), msg))


def lib():
    """Load libbakron.so (raises if it has not been built)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("libbakron.so is not built (%s); run __graft_entry__.build()" % LIB_PATH)
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
    L.bakron_default_opts.argtypes = [ctypes.POINTER(Opts)]
    L.bakron_default_opts.restype = None
    L.bakron_status_string.argtypes = [ctypes.c_int]
    L.bakron_status_string.restype = ctypes.c_char_p
    L.bakron_version.restype = ctypes.c_int
    L.bakron_kernel_launches.restype = ctypes.c_int64
    L.bakron_workspace_size.argtypes = [i64, i64, ctypes.POINTER(Opts), ctypes.POINTER(sz)]
    L.bakron_prepare_workspace_size.argtypes = [i64, i64, ctypes.POINTER(sz)]
    L.bakron_rowscale.argtypes = [vp, i64, i64, ctypes.c_int, vp, vp]
    L.bakron_prepare.argtypes = [vp, i64, ctypes.c_float, vp, i64, ctypes.c_float,
                                 vp, vp, vp, vp, ctypes.POINTER(i64), vp, sz, vp]
    L.bakron_quantize.argtypes = [vp, i64, i64, vp, vp, vp, ctypes.c_int, ctypes.c_int,
                                  vp, vp, vp, ctypes.POINTER(Opts), vp, sz, vp]
    L.bakron_quantize_antidiag.argtypes = [vp, i64, i64, vp, vp, vp, ctypes.c_int, ctypes.c_int,
                                           vp, vp, vp, vp, ctypes.c_float, ctypes.POINTER(i64),
                                           ctypes.POINTER(Opts), vp, sz, vp]
    L.bakron_quantize_noalloc.argtypes = [vp, i64, i64, vp, vp, vp, ctypes.c_int, ctypes.c_int,
                                          vp, vp, vp]
    L.bakron_grid_params.argtypes = [vp, i64, i64, ctypes.c_int, ctypes.c_int, i64, vp, vp,
                                     ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int), vp]
    L.bakron_quantize_grid.argtypes = [vp, i64, i64, vp, vp, vp, vp, i64, ctypes.c_int, ctypes.c_int,
                                       vp, vp, vp, ctypes.POINTER(Opts), vp, sz, vp]
    L.bakron_batch_workspace_size.argtypes = [ctypes.c_int, ctypes.POINTER(Problem),
                                              ctypes.POINTER(Opts), ctypes.POINTER(sz)]
    L.bakron_quantize_batch.argtypes = [ctypes.c_int, ctypes.POINTER(Problem), ctypes.POINTER(Opts),
                                        vp, sz, vp]
    L.bakron_factors_workspace_size.argtypes = [i64, i64, i64, ctypes.POINTER(sz)]
    L.bakron_factors.argtypes = [vp, i64, i64, vp, i64, ctypes.c_int, vp, vp, vp, sz, vp]
    L.bakron_schedule_export.argtypes = [ctypes.c_int, i64, i64, vp, i64, ctypes.POINTER(i64)]
    L.bakron_fma_probe.argtypes = [vp, i64, ctypes.c_int, vp]
    L.bakron_plan_size.argtypes = [i64, i64, ctypes.POINTER(sz)]
    L.bakron_plan_init.argtypes = [i64, i64, vp, sz, vp]
    L.bakron_sm_count.restype = ctypes.c_int
    pk, f32 = ctypes.POINTER(Packed), ctypes.c_float
    L.bakron_async_status.argtypes = [vp]
    L.bakron_pack_size.argtypes = [i64, i64, i64, i64, ctypes.c_int, ctypes.POINTER(sz)]
    L.bakron_pack.argtypes = [vp, vp, vp, i64, i64, i64, i64, ctypes.c_int, ctypes.c_int, vp, sz, vp]
    L.bakron_unpack.argtypes = [pk, vp, vp]
    L.bakron_linear_workspace_size.argtypes = [pk, i64, ctypes.c_int, ctypes.POINTER(sz)]
    L.bakron_linear.argtypes = [vp, i64, ctypes.c_int, pk, vp, vp, sz, vp]
    L.bakron_linear_grad_workspace_size.argtypes = [pk, i64, ctypes.c_int, ctypes.POINTER(sz)]
    L.bakron_linear_grad.argtypes = [vp, i64, ctypes.c_int, pk, vp, vp, sz, vp]
    L.bakron_moe_workspace_size.argtypes = [pk, pk, i64, ctypes.c_int, ctypes.c_int, ctypes.POINTER(sz)]
    L.bakron_moe.argtypes = [vp, i64, ctypes.c_int, vp, pk, pk, ctypes.c_int, ctypes.c_int, vp, vp, sz, vp]
    L.bakron_layernorm.argtypes = [vp, i64, i64, ctypes.c_int, vp, vp, f32, vp, vp, vp, vp]
    L.bakron_layernorm_grad_workspace_size.argtypes = [i64, i64, ctypes.POINTER(sz)]
    L.bakron_layernorm_grad.argtypes = [vp, vp, i64, i64, ctypes.c_int, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    for f in ("bakron_schedule_export", "bakron_workspace_size", "bakron_prepare_workspace_size", "bakron_rowscale",
              "bakron_prepare", "bakron_quantize", "bakron_quantize_antidiag",
              "bakron_quantize_noalloc", "bakron_factors_workspace_size", "bakron_factors",
              "bakron_grid_params", "bakron_quantize_grid", "bakron_batch_workspace_size",
              "bakron_quantize_batch", "bakron_fma_probe", "bakron_plan_size",
              "bakron_plan_init", "bakron_async_status", "bakron_pack_size", "bakron_pack",
              "bakron_unpack", "bakron_linear_workspace_size", "bakron_linear",
              "bakron_linear_grad_workspace_size", "bakron_linear_grad",
              "bakron_moe_workspace_size", "bakron_moe", "bakron_layernorm",
              "bakron_layernorm_grad_workspace_size", "bakron_layernorm_grad"):
        getattr(L, f).restype = ctypes.c_int
    _LIB = L
    return L


def kernel_launches():
    """Kernels the library has launched in this process so far."""
    return int(lib().bakron_kernel_launches())


def sm_count():
    """Streaming multiprocessors of the current CUDA device."""
    return int(lib().bakron_sm_count())


def fma_probe(out, blocks, iters):
    """Enqueue the FP32 FMA throughput probe on the current stream (see
    bakron_fma_probe); ``out`` is a float32 CUDA tensor of blocks * 256
    elements.  Returns the flops it performs."""
    import torch
    assert out.dtype == torch.float32 and out.is_cuda and out.numel() >= blocks * 256
    st = lib().bakron_fma_probe(ctypes.c_void_p(out.data_ptr()), int(blocks), int(iters),
                                ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    if st != OK:
        raise BakronError(st, "bakron_fma_probe")
    return 2.0 * blocks * 256 * iters * 128


SCHEDULE_SOLVE = 0
SCHEDULE_ROWS = 1
SCHEDULE_PREPARE = 2


def schedule_export(kind, M, N=1):
    """The library's work lists for a shape in 128-tiles (host only, no GPU):
    an int32 numpy array in the layout bakron_schedule_export documents."""
    import numpy as np
    n = ctypes.c_int64(0)
    st = lib().bakron_schedule_export(int(kind), int(M), int(N), None, 0, ctypes.byref(n))
    if st != OK:
        raise BakronError(st, "bakron_schedule_export")
    out = np.zeros(max(1, n.value), dtype=np.int32)
    st = lib().bakron_schedule_export(int(kind), int(M), int(N), ctypes.c_void_p(out.ctypes.data),
                                      n.value, ctypes.byref(n))
    if st != OK:
        raise BakronError(st, "bakron_schedule_export")
    return out[:n.value]


def default_opts(**kw):
    o = Opts()
    lib().bakron_default_opts(ctypes.byref(o))
    for k, v in kw.items():
        setattr(o, k, v)
    return o


def _check(st, where):
    if st != OK:
        raise BakronError(st, where)


_TORCH = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        if not torch.cuda.is_available():
            raise RuntimeError("no CUDA device: the BaKron library runs on the GPU only")
        _TORCH = torch
    return _TORCH


_DEVICE = None


def _device():
    """Index of the current CUDA device, on which the library works."""
    global _DEVICE
    if _DEVICE is None:
        _DEVICE = _torch()._C._cuda_getDevice
    return _DEVICE()


def _elsewhere(index, name):
    return ValueError("%s is on cuda:%d, the current device is cuda:%d" % (name, index, _device()))


def _check_stream(stream):
    index = getattr(stream, "device_index", None)
    if index is not None and index != _device():
        raise _elsewhere(index, "stream")


def _dev(t, dtype, shape, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.get_device() != _device():
        raise _elsewhere(t.get_device(), name)
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    else:
        _check_stream(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def workspace_size(m, n, opts=None):
    b = ctypes.c_size_t(0)
    _check(lib().bakron_workspace_size(m, n, ctypes.byref(opts) if opts else None, ctypes.byref(b)),
           "bakron_workspace_size")
    return b.value


def plan_size(m, n):
    b = ctypes.c_size_t(0)
    _check(lib().bakron_plan_size(m, n, ctypes.byref(b)), "bakron_plan_size")
    return b.value


def bakron_plan_init(m, n, plan=None, stream=None):
    """The work-list plan of the m x n shape in a device buffer (uint8 tensor,
    allocated here when ``plan`` is None); pass it as ``opts.plan``."""
    torch = _torch()
    nb = plan_size(m, n)
    if plan is None:
        plan = torch.empty(nb, dtype=torch.uint8, device="cuda")
    elif plan.numel() * plan.element_size() < nb:
        raise ValueError("plan buffer too small: need %d bytes" % nb)
    _check(lib().bakron_plan_init(m, n, ctypes.c_void_p(plan.data_ptr()), nb, _stream(stream)),
           "bakron_plan_init")
    return plan


def prepare_workspace_size(n, m):
    b = ctypes.c_size_t(0)
    _check(lib().bakron_prepare_workspace_size(n, m, ctypes.byref(b)), "bakron_prepare_workspace_size")
    return b.value


def _ws(nbytes, workspace):
    torch = _torch()
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        if workspace.get_device() != _device():
            raise _elsewhere(workspace.get_device(), "workspace")
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError("workspace too small: need %d bytes" % nbytes)
        return workspace
    return torch.empty(nbytes, dtype=torch.uint8, device="cuda")


def bakron_rowscale(W, qmax, out=None, stream=None):
    torch = _torch()
    m, n = W.shape
    if out is None:
        out = torch.empty(m, dtype=torch.float32, device=W.device)
    _check(lib().bakron_rowscale(_dev(W, torch.float32, (m, n), "W"), m, n, int(qmax),
                                 _dev(out, torch.float32, (m,), "scale"), _stream(stream)),
           "bakron_rowscale")
    return out


def bakron_prepare(A, damp_A, B=None, damp_B=0.0, want_L=False, workspace=None, stream=None,
                   out=None):
    """Returns (UA, UB, LA, LB, info); UB/LB are None when B is None."""
    torch = _torch()
    n = A.shape[0]
    m = 0 if B is None else B.shape[0]
    if out is not None:
        UA, UB = out
    else:
        UA = torch.empty((n, n), dtype=torch.float32, device=A.device)
        UB = None if B is None else torch.empty((m, m), dtype=torch.float32, device=A.device)
    LA = torch.empty_like(UA) if want_L else None
    LB = torch.empty_like(UB) if (want_L and B is not None) else None
    nb = prepare_workspace_size(n, m)
    ws = _ws(nb, workspace)
    info = (ctypes.c_int64 * 2)(-1, -1)
    st = lib().bakron_prepare(
        _dev(A, torch.float32, (n, n), "A"), n, float(damp_A),
        None if B is None else _dev(B, torch.float32, (m, m), "B"), m, float(damp_B),
        _dev(UA, torch.float32, (n, n), "UA"),
        None if UB is None else _dev(UB, torch.float32, (m, m), "UB"),
        None if LA is None else _dev(LA, torch.float32, (n, n), "LA"),
        None if LB is None else _dev(LB, torch.float32, (m, m), "LB"),
        info, ctypes.c_void_p(ws.data_ptr()), nb, _stream(stream))
    if st != OK:
        err = BakronError(st, "bakron_prepare")
        err.info = (info[0], info[1])
        raise err
    return UA, UB, LA, LB, (info[0], info[1])


def bakron_quantize(W, UA, UB, scale, qmin, qmax, want_preround=False, opts=None, workspace=None,
                    stream=None, out=None):
    """Returns (V, codes, preround-or-None).  UB=None means B = I: one-sided
    GPTQ with Hessian A for every row, solved by the library's row path."""
    torch = _torch()
    m, n = W.shape
    if out is None:
        V = torch.empty((m, n), dtype=torch.float32, device=W.device)
        codes = torch.empty((m, n), dtype=torch.int8, device=W.device)
    else:
        V, codes = out
    pre = torch.empty((m, n), dtype=torch.float32, device=W.device) if want_preround else None
    nb = workspace_size(m, n, opts)
    ws = _ws(nb, workspace)
    st = lib().bakron_quantize(
        _dev(W, torch.float32, (m, n), "W"), m, n,
        _dev(UA, torch.float32, (n, n), "UA"),
        None if UB is None else _dev(UB, torch.float32, (m, m), "UB"),
        _dev(scale, torch.float32, (m,), "scale"), int(qmin), int(qmax),
        _dev(V, torch.float32, (m, n), "V"), _dev(codes, torch.int8, (m, n), "codes"),
        None if pre is None else _dev(pre, torch.float32, (m, n), "preround"),
        ctypes.byref(opts) if opts is not None else None,
        ctypes.c_void_p(ws.data_ptr()), nb, _stream(stream))
    _check(st, "bakron_quantize")
    return V, codes, pre


def grid_groups(n, group):
    """Number of column groups of a grid (group 0/None or >= n: one per row)."""
    if not group or group >= n:
        return 1
    if group % 32:
        raise ValueError("group must be a multiple of 32 (or cover the whole row)")
    return -(-n // group)


def bakron_grid_params(W, bits, asymmetric=False, group=None, stream=None):
    """Grid of a b-bit base quantizer on the original W: returns
    (scale, zero, qmin, qmax) with scale/zero of shape (m, groups)."""
    torch = _torch()
    m, n = W.shape
    ng = grid_groups(n, group)
    scale = torch.empty((m, ng), dtype=torch.float32, device=W.device)
    zero = torch.empty((m, ng), dtype=torch.float32, device=W.device)
    qmin, qmax = ctypes.c_int(0), ctypes.c_int(0)
    st = lib().bakron_grid_params(_dev(W, torch.float32, (m, n), "W"), m, n, int(bits),
                                  1 if asymmetric else 0, int(group or 0),
                                  ctypes.c_void_p(scale.data_ptr()), ctypes.c_void_p(zero.data_ptr()),
                                  ctypes.byref(qmin), ctypes.byref(qmax), _stream(stream))
    _check(st, "bakron_grid_params")
    return scale, zero, qmin.value, qmax.value


def bakron_quantize_grid(W, UA, UB, scale, zero, group, qmin, qmax, want_preround=False, opts=None,
                         workspace=None, stream=None, out=None):
    """bakron_quantize on a grid (scale/zero of shape (m, groups)); UB=None
    means B = I.  Returns (V, codes, preround-or-None)."""
    torch = _torch()
    m, n = W.shape
    ng = grid_groups(n, group)
    if out is None:
        V = torch.empty((m, n), dtype=torch.float32, device=W.device)
        codes = torch.empty((m, n), dtype=torch.int8, device=W.device)
    else:
        V, codes = out
    pre = torch.empty((m, n), dtype=torch.float32, device=W.device) if want_preround else None
    nb = workspace_size(m, n, opts)
    ws = _ws(nb, workspace)
    st = lib().bakron_quantize_grid(
        _dev(W, torch.float32, (m, n), "W"), m, n, _dev(UA, torch.float32, (n, n), "UA"),
        None if UB is None else _dev(UB, torch.float32, (m, m), "UB"),
        _dev(scale, torch.float32, (m, ng), "scale"),
        None if zero is None else _dev(zero, torch.float32, (m, ng), "zero"),
        int(group or 0), int(qmin), int(qmax),
        _dev(V, torch.float32, (m, n), "V"), _dev(codes, torch.int8, (m, n), "codes"),
        None if pre is None else _dev(pre, torch.float32, (m, n), "preround"),
        ctypes.byref(opts) if opts is not None else None,
        ctypes.c_void_p(ws.data_ptr()), nb, _stream(stream))
    _check(st, "bakron_quantize_grid")
    return V, codes, pre


def bakron_quantize_batch(problems, opts=None, workspace=None, stream=None, outs=None):
    """Several independent solves at once.  ``problems``: sequence of dicts
    with W, UA, UB (None = B = I), scale, zero (None = 0), group (None = per
    row), qmin, qmax.  Returns a list of (V, codes); raises BakronError with
    ``statuses`` (one per problem) if any problem failed."""
    torch = _torch()
    arr = (Problem * len(problems))()
    keep = []
    for k, pr in enumerate(problems):
        W = pr["W"]
        m, n = W.shape
        ng = grid_groups(n, pr.get("group"))
        if outs is None:
            V = torch.empty((m, n), dtype=torch.float32, device=W.device)
            C = torch.empty((m, n), dtype=torch.int8, device=W.device)
        else:
            V, C = outs[k]
        UB, zero = pr.get("UB"), pr.get("zero")
        arr[k] = Problem(
            _dev(W, torch.float32, (m, n), "W"), m, n, _dev(pr["UA"], torch.float32, (n, n), "UA"),
            None if UB is None else _dev(UB, torch.float32, (m, m), "UB"),
            _dev(pr["scale"], torch.float32, (m, ng) if ng > 1 or pr["scale"].dim() == 2 else (m,),
                 "scale"),
            None if zero is None else _dev(zero, torch.float32, (m, ng), "zero"),
            int(pr.get("group") or 0), int(pr["qmin"]), int(pr["qmax"]),
            _dev(V, torch.float32, (m, n), "V"), _dev(C, torch.int8, (m, n), "codes"), 0)
        keep.append((V, C))
    size = ctypes.c_size_t(0)
    o = ctypes.byref(opts) if opts is not None else None
    _check(lib().bakron_batch_workspace_size(len(problems), arr, o, ctypes.byref(size)),
           "bakron_batch_workspace_size")
    ws = _ws(size.value, workspace)
    st = lib().bakron_quantize_batch(len(problems), arr, o, ctypes.c_void_p(ws.data_ptr()),
                                     size.value, _stream(stream))
    if st != OK:
        err = BakronError(st, "bakron_quantize_batch")
        err.statuses = [arr[k].status for k in range(len(problems))]
        raise err
    return keep


def bakron_quantize_antidiag(W, UA, UB, scale, qmin, qmax, guide_codes=None, guide_tol=1e-4,
                             want_preround=False, opts=None, workspace=None, stream=None):
    """Returns (V, codes, preround-or-None, overrides)."""
    torch = _torch()
    m, n = W.shape
    V = torch.empty((m, n), dtype=torch.float32, device=W.device)
    codes = torch.empty((m, n), dtype=torch.int8, device=W.device)
    pre = torch.empty((m, n), dtype=torch.float32, device=W.device) if want_preround else None
    nb = workspace_size(m, n, opts)
    ws = _ws(nb, workspace)
    over = ctypes.c_int64(0)
    st = lib().bakron_quantize_antidiag(
        _dev(W, torch.float32, (m, n), "W"), m, n,
        _dev(UA, torch.float32, (n, n), "UA"), _dev(UB, torch.float32, (m, m), "UB"),
        _dev(scale, torch.float32, (m,), "scale"), int(qmin), int(qmax),
        _dev(V, torch.float32, (m, n), "V"), _dev(codes, torch.int8, (m, n), "codes"),
        None if pre is None else _dev(pre, torch.float32, (m, n), "preround"),
        None if guide_codes is None else _dev(guide_codes, torch.int8, (m, n), "guide_codes"),
        float(guide_tol), ctypes.byref(over),
        ctypes.byref(opts) if opts is not None else None,
        ctypes.c_void_p(ws.data_ptr()), nb, _stream(stream))
    _check(st, "bakron_quantize_antidiag")
    return V, codes, pre, over.value


NOALLOC_MAX_DIM = 512


def bakron_quantize_noalloc(W, UA, UB, scale, qmin, qmax, out=None, stream=None):
    """bakron_quantize without a workspace (the library's fixed scratch array;
    m, n <= 512).  For callers that cannot allocate device memory, pass
    pre-allocated ``out=(V, codes)``; this wrapper then allocates nothing
    either.  Returns (V, codes)."""
    torch = _torch()
    m, n = W.shape
    if out is None:
        V = torch.empty((m, n), dtype=torch.float32, device=W.device)
        codes = torch.empty((m, n), dtype=torch.int8, device=W.device)
    else:
        V, codes = out
    st = lib().bakron_quantize_noalloc(
        _dev(W, torch.float32, (m, n), "W"), m, n,
        _dev(UA, torch.float32, (n, n), "UA"), _dev(UB, torch.float32, (m, m), "UB"),
        _dev(scale, torch.float32, (m,), "scale"), int(qmin), int(qmax),
        _dev(V, torch.float32, (m, n), "V"), _dev(codes, torch.int8, (m, n), "codes"),
        _stream(stream))
    _check(st, "bakron_quantize_noalloc")
    return V, codes


def factors_workspace_size(N, n, m):
    size = ctypes.c_size_t(0)
    _check(lib().bakron_factors_workspace_size(N, n, m, ctypes.byref(size)),
           "bakron_factors_workspace_size")
    return size.value


def bakron_factors(X=None, G=None, mode=FACTORS_KFAC, want_A=True, want_B=True, workspace=None,
                   stream=None):
    """Kronecker factors (A, B) from samples: rows of X (N x n) are input
    activations, rows of G (N x m) output gradients.  mode FACTORS_KFAC or
    FACTORS_SHAMPOO; an unwanted factor comes back as None."""
    torch = _torch()
    ref = X if X is not None else G
    N = ref.shape[0]
    n = 0 if X is None else X.shape[1]
    m = 0 if G is None else G.shape[1]
    A = torch.empty((n, n), dtype=torch.float32, device=ref.device) if (want_A and X is not None) else None
    B = torch.empty((m, m), dtype=torch.float32, device=ref.device) if (want_B and G is not None) else None
    size = ctypes.c_size_t(0)
    _check(lib().bakron_factors_workspace_size(N, n, m, ctypes.byref(size)),
           "bakron_factors_workspace_size")
    ws = _ws(size.value, workspace)
    st = lib().bakron_factors(
        None if X is None else _dev(X, torch.float32, (N, n), "X"), N, n,
        None if G is None else _dev(G, torch.float32, (N, m), "G"), m, int(mode),
        None if A is None else _dev(A, torch.float32, (n, n), "A"),
        None if B is None else _dev(B, torch.float32, (m, m), "B"),
        ctypes.c_void_p(ws.data_ptr()), size.value, _stream(stream))
    _check(st, "bakron_factors")
    return A, B


# ------------------------------------------------ quantised layers in use
#
# A call for one token takes a few microseconds on the GPU, less than careless
# marshalling takes on the host: what these functions look up more than once
# is kept, addresses go to ctypes as plain integers, and the current stream is
# asked for its handle only.
#
# These calls only enqueue (bakron_pack and bakron_unpack excepted) on
# ``stream``, or on the current stream.  Tensors allocated here belong to the
# current stream as far as PyTorch's allocator knows; a caller who passes
# another stream passes ``out`` and ``workspace`` too, or keeps the two
# streams ordered.


_DTYPES = {}


def _dtypes():
    """torch dtype -> bakron_dtype of the activations."""
    if not _DTYPES:
        torch = _torch()
        _DTYPES.update({torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16})
    return _DTYPES


def _handle(stream, index):
    """cudaStream_t of ``stream``, or of the current stream of ``index``, the current device."""
    if stream is not None:
        _check_stream(stream)
        return stream.cuda_stream
    return _torch()._C._cuda_getCurrentRawStream(index)


def _act(t, name, cols=None):
    """Checks an activation matrix; returns (rows, columns, bakron_dtype, device)."""
    if not isinstance(t, _torch().Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    index = t.get_device()
    if index != _device():
        raise _elsewhere(index, name)
    code = (_DTYPES or _dtypes()).get(t.dtype)
    if code is None:
        raise ValueError("%s must be float32, bfloat16 or float16, got %s" % (name, t.dtype))
    shape = t.shape
    if len(shape) != 2 or (cols is not None and shape[1] != cols):
        raise ValueError("%s must have shape (tokens, %s), got %s"
                         % (name, "columns" if cols is None else cols, tuple(shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return shape[0], shape[1], code, index


def _same(t, like, shape, name):
    """Checks a tensor that must have the type and device of ``like``; returns its address."""
    if not isinstance(t, _torch().Tensor) or t.dtype != like.dtype or t.get_device() != like.get_device():
        raise ValueError("%s must be a %s tensor on %s" % (name, like.dtype, like.device))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _out(out, like, shape, name):
    if out is None:
        return _torch().empty(shape, dtype=like.dtype, device=like.device)
    _same(out, like, shape, name)
    return out


def _vec(t, n, like, name):
    """Device address of a float32 vector of n elements, or None."""
    if t is None:
        return None
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or t.get_device() != like.get_device() or \
            t.shape != (n,) or not t.is_contiguous():
        raise ValueError("%s must be a contiguous float32 tensor of shape (%d,) on %s" % (name, n, like.device))
    return t.data_ptr()


class PackedWeight:
    """4-bit codes and their grid in the layout of the products (bakron_pack):
    ``count`` matrices of m x n.  ``data`` is the device buffer."""

    def __init__(self, data, count, m, n, group, qmin, has_zero):
        self.data, self.count, self.m, self.n, self.group = data, count, m, n, group
        self.qmin, self.has_zero = qmin, has_zero
        self.desc = Packed(count, m, n, group, qmin, 1 if has_zero else 0, data.data_ptr(), data.numel())
        self.ref = ctypes.byref(self.desc)
        self.device = data.device
        self._index = data.get_device()
        self._ws = {}

    def _here(self):
        if self._index != _device():
            raise _elsewhere(self._index, "the weight")

    def _check(self, like, name):
        if like.get_device() != self._index:
            raise ValueError("%s must be on %s, the weight's device" % (name, self.device))

    def unpack(self, stream=None):
        """V, float32: (m, n), or (count, m, n) for several matrices."""
        return bakron_unpack(self, stream=stream)


def bakron_pack(codes, scale, qmin, qmax, zero=None, group=None, stream=None):
    """Packs codes (m, n) or (count, m, n), int8 in [qmin, qmax] with
    qmax - qmin <= 15, on a grid as bakron_grid_params returns it: scale and
    zero (m, groups) or (count, m, groups); a scale of one group may be (m,).
    Returns a PackedWeight."""
    torch = _torch()
    if not isinstance(codes, torch.Tensor) or codes.dim() not in (2, 3):
        raise ValueError("codes must be a tensor of shape (m, n) or (count, m, n)")
    lead = tuple(codes.shape[:-1])
    m, n = codes.shape[-2:]
    count = codes.shape[0] if codes.dim() == 3 else 1
    ng = grid_groups(n, group)
    shape = lead if ng == 1 and isinstance(scale, torch.Tensor) and scale.dim() == len(lead) else lead + (ng,)
    size = ctypes.c_size_t(0)
    _check(lib().bakron_pack_size(count, m, n, int(group or 0), 0 if zero is None else 1, ctypes.byref(size)),
           "bakron_pack_size")
    args = (_dev(codes, torch.int8, lead + (n,), "codes"), _dev(scale, torch.float32, shape, "scale"),
            None if zero is None else _dev(zero, torch.float32, zero.shape if zero.shape == lead and ng == 1
                                           else lead + (ng,), "zero"))
    data = torch.empty(size.value, dtype=torch.uint8, device=codes.device)
    _check(lib().bakron_pack(*args, count, m, n, int(group or 0), int(qmin), int(qmax),
                             ctypes.c_void_p(data.data_ptr()), size.value, _stream(stream)), "bakron_pack")
    return PackedWeight(data, count, m, n, int(group or 0), int(qmin), zero is not None)


def bakron_unpack(w, stream=None):
    """V (float32) of a PackedWeight: the values the solver returned."""
    torch = _torch()
    w._here()
    V = torch.empty((w.count, w.m, w.n), dtype=torch.float32, device=w.device)
    _check(lib().bakron_unpack(w.ref, ctypes.c_void_p(V.data_ptr()), _stream(stream)), "bakron_unpack")
    return V[0] if w.count == 1 else V


def bakron_async_status(stream=None):
    """Raises BakronError if an enqueued call left an error on the device."""
    _check(lib().bakron_async_status(_stream(stream)), "bakron_async_status")


def linear_workspace_size(w, T, dtype, grad=False):
    w._here()           # the size depends on the device's SM count
    return _linear_ws_size(w, T, dtype, grad)


def _linear_ws_size(w, T, dtype, grad):
    key = (T, dtype, grad)
    size = w._ws.get(key)
    if size is None:
        code = _dtypes()[dtype]
        f = lib().bakron_linear_grad_workspace_size if grad else lib().bakron_linear_workspace_size
        b = ctypes.c_size_t(0)
        _check(f(w.ref, T, code, ctypes.byref(b)), "bakron_linear_workspace_size")
        size = b.value
        if len(w._ws) > 64:
            w._ws.clear()
        w._ws[key] = size
    return size


def linear_workspace(w, T, dtype, grad=False):
    """A workspace for bakron_linear (or its gradient) of up to T tokens,
    None when none is needed."""
    nb = linear_workspace_size(w, T, dtype, grad)
    return _torch().empty(nb, dtype=_torch().uint8, device=w.device) if nb else None


def _linear(fn, where, grad, x, w, out, workspace, stream):
    name = "dY" if grad else "X"
    T, _, code, dev = _act(x, name, w.m if grad else w.n)
    w._check(x, name)
    if w.count != 1:
        raise ValueError("%s takes a single matrix, got %d" % (where, w.count))
    y = _out(out, x, (T, w.n if grad else w.m), "out")
    nb = _linear_ws_size(w, T, x.dtype, grad)
    ws = _ws(nb, workspace) if nb else None     # alive until the call is enqueued
    st = fn(x.data_ptr(), T, code, w.ref, y.data_ptr(), None if ws is None else ws.data_ptr(), nb,
            _handle(stream, dev))
    if st != OK:
        raise BakronError(st, where)
    return y


def bakron_linear(x, w, out=None, workspace=None, stream=None):
    """Y = X V^T: x (T, n) float32, bfloat16 or float16, w a PackedWeight of
    one m x n matrix; returns (T, m) of x's type."""
    return _linear(lib().bakron_linear, "bakron_linear", False, x, w, out, workspace, stream)


def bakron_linear_grad(dy, w, out=None, workspace=None, stream=None):
    """dX = dY V, the gradient of bakron_linear for its activations: dy
    (T, m); returns (T, n) of dy's type."""
    return _linear(lib().bakron_linear_grad, "bakron_linear_grad", True, dy, w, out, workspace, stream)


def moe_workspace_size(w_in, w_out, T, top_k, dtype):
    w_in._here()
    return _moe_ws_size(w_in, w_out, T, top_k, dtype)


def _moe_ws_size(w_in, w_out, T, top_k, dtype):
    key = (T, dtype, top_k, w_out.n)
    size = w_in._ws.get(key)
    if size is None:
        code = _dtypes()[dtype]
        b = ctypes.c_size_t(0)
        _check(lib().bakron_moe_workspace_size(w_in.ref, w_out.ref, T, int(top_k), code, ctypes.byref(b)),
               "bakron_moe_workspace_size")
        size = b.value
        if len(w_in._ws) > 64:
            w_in._ws.clear()
        w_in._ws[key] = size
    return size


def moe_workspace(w_in, w_out, T, top_k, dtype):
    """A workspace for bakron_moe of up to T tokens."""
    nb = moe_workspace_size(w_in, w_out, T, top_k, dtype)
    return _torch().empty(nb, dtype=_torch().uint8, device=w_in.device)


def bakron_moe(x, router, w_in, w_out, top_k, renormalize=True, out=None, workspace=None, stream=None):
    """A mixture-of-experts layer: x (T, d), router (E, d) of x's type, w_in
    (E matrices of 2f x d: gate rows, then up rows), w_out (E of d x f).
    Returns (T, d) of x's type."""
    T, d, code, dev = _act(x, "X", w_in.n)
    if (w_in.count, w_out.m) != (w_out.count, d) or w_in.m != 2 * w_out.n:
        raise ValueError("w_in must hold E matrices of 2f x d and w_out E of d x f, got %d of %d x %d and "
                         "%d of %d x %d" % (w_in.count, w_in.m, w_in.n, w_out.count, w_out.m, w_out.n))
    w_in._check(x, "X")
    w_out._check(x, "X")
    rp = _same(router, x, (w_in.count, d), "router")
    y = _out(out, x, (T, d), "out")
    nb = _moe_ws_size(w_in, w_out, T, top_k, x.dtype)
    ws = _ws(nb, workspace)
    _check(lib().bakron_moe(x.data_ptr(), T, code, rp, w_in.ref, w_out.ref, int(top_k),
                            1 if renormalize else 0, y.data_ptr(), ws.data_ptr(), nb, _handle(stream, dev)),
           "bakron_moe")
    return y


def bakron_layernorm(x, gamma=None, beta=None, eps=1e-5, out=None, want_stats=True, stream=None):
    """Layer norm of the rows of x (T, d); gamma, beta (d,) float32 or None.
    Returns (y, mean, rstd); mean and rstd (T,) float32 feed the gradient
    (None without want_stats)."""
    T, d, code, dev = _act(x, "X")
    y = _out(out, x, (T, d), "out")
    mean = rstd = mp = rp = None
    if want_stats:
        torch = _torch()
        mean = torch.empty(T, dtype=torch.float32, device=x.device)
        rstd = torch.empty(T, dtype=torch.float32, device=x.device)
        mp, rp = mean.data_ptr(), rstd.data_ptr()
    _check(lib().bakron_layernorm(x.data_ptr(), T, d, code, _vec(gamma, d, x, "gamma"), _vec(beta, d, x, "beta"),
                                  eps, y.data_ptr(), mp, rp, _handle(stream, dev)), "bakron_layernorm")
    return y, mean, rstd


_NORM_WS = {}


def layernorm_grad_workspace_size(T, d):
    """Bytes on the current device (they depend on its SM count)."""
    key = (T, d, _device())
    size = _NORM_WS.get(key)
    if size is None:
        b = ctypes.c_size_t(0)
        _check(lib().bakron_layernorm_grad_workspace_size(T, d, ctypes.byref(b)),
               "bakron_layernorm_grad_workspace_size")
        size = b.value
        if len(_NORM_WS) > 256:
            _NORM_WS.clear()
        _NORM_WS[key] = size
    return size


def layernorm_grad_workspace(T, d):
    """A workspace for bakron_layernorm_grad of up to T rows of d, on the current device."""
    return _torch().empty(layernorm_grad_workspace_size(T, d), dtype=_torch().uint8, device="cuda")


def bakron_layernorm_grad(dy, x, gamma, mean, rstd, want_weight_grads=True, out=None, workspace=None,
                          stream=None):
    """Gradients of bakron_layernorm: returns (dx, dgamma, dbeta), dgamma and
    dbeta (d,) float32 (None without want_weight_grads)."""
    T, d, code, dev = _act(x, "X")
    yp = _same(dy, x, (T, d), "dY")
    dx = _out(out, x, (T, d), "out")
    dg = db = gp = bp = ws = None
    nb = 0
    if want_weight_grads:
        torch = _torch()
        nb = layernorm_grad_workspace_size(T, d)
        # kept until the call is enqueued, then the allocator may reuse it in stream order
        keep = _ws(nb, workspace)
        ws = keep.data_ptr()
        dg = torch.empty(d, dtype=torch.float32, device=x.device)
        db = torch.empty(d, dtype=torch.float32, device=x.device)
        gp, bp = dg.data_ptr(), db.data_ptr()
    _check(lib().bakron_layernorm_grad(yp, x.data_ptr(), T, d, code, _vec(gamma, d, x, "gamma"),
                                       _vec(mean, T, x, "mean"), _vec(rstd, T, x, "rstd"), dx.data_ptr(),
                                       gp, bp, ws, nb, _handle(stream, dev)), "bakron_layernorm_grad")
    return dx, dg, db


class Solver:
    """The whole path on one GPU: row grid, factor preparation, solve.

    Workspaces, the shape's work-list plan and the outputs are allocated once
    per shape and reused, so repeated solves of one shape allocate nothing.
    """

    def __init__(self, m, n, bits=None, qmin=None, qmax=None, opts=None, stream=None):
        torch = _torch()
        self.m, self.n = m, n
        if bits is not None:
            self.qmax = (1 << (bits - 1)) - 1
            self.qmin = -(self.qmax + 1)
        else:
            self.qmin, self.qmax = qmin, qmax
        self.opts = opts if opts is not None else default_opts()
        self.stream = stream
        dev = "cuda"
        self.plan = bakron_plan_init(m, n, stream=stream)
        self.ws_q = torch.empty(workspace_size(m, n, opts), dtype=torch.uint8, device=dev)
        self.ws_p = torch.empty(prepare_workspace_size(n, m), dtype=torch.uint8, device=dev)
        self.scale = torch.empty(m, dtype=torch.float32, device=dev)
        self.UA = torch.empty((n, n), dtype=torch.float32, device=dev)
        self.UB = torch.empty((m, m), dtype=torch.float32, device=dev)
        self.V = torch.empty((m, n), dtype=torch.float32, device=dev)
        self.codes = torch.empty((m, n), dtype=torch.int8, device=dev)

    def rowscale(self, W):
        return bakron_rowscale(W, self.qmax, out=self.scale, stream=self.stream)

    def prepare(self, A, damp_A, B, damp_B):
        bakron_prepare(A, damp_A, B, damp_B, workspace=self.ws_p, stream=self.stream,
                       out=(self.UA, self.UB))
        return self.UA, self.UB

    def quantize(self, W, UA=None, UB=None, scale=None, want_preround=False):
        if self.opts is not None and not self.opts.plan:
            self.opts.plan = self.plan.data_ptr()
        return bakron_quantize(W, self.UA if UA is None else UA, self.UB if UB is None else UB,
                               self.scale if scale is None else scale, self.qmin, self.qmax,
                               want_preround=want_preround, opts=self.opts, workspace=self.ws_q,
                               stream=self.stream, out=(self.V, self.codes))

    def solve(self, W, A, damp_A, B, damp_B):
        """Row grid + factor preparation + BaKron solve; returns (V, codes)."""
        self.rowscale(W)
        self.prepare(A, damp_A, B, damp_B)
        return self.quantize(W)[:2]
