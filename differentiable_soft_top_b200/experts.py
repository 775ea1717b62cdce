"""Operators of a layer of experts behind a router (include/lapsum_experts.h).

Soft top-k memberships train a router; the layer behind it then needs the hard
choice of k experts per token, the exchange between token order and expert
order, and every expert's product with its own weights.  Each operator here
runs in this package's kernels and is differentiable; gradients flow through
the weights of the choice, at fixed choice.

    from differentiable_soft_top_b200 import experts as ex, soft_topk
    w, chosen = ex.route(logits, 8, score="sigmoid", bias=balance)      # scores of the router
    w, chosen = ex.route(soft_topk(logits, 8.0, 0.5), 8, score="identity")  # or LapSum memberships
    out = ex.mlp(x, w, chosen, w_in, w_out, activation="swiglu", residual=x)

mlp() is plan, dispatch, linear, linear, combine in one; each is public.  Like the
rest of the package: CUDA tensors only, the current stream of the tensors'
device, no host synchronisation; every call may be captured into a CUDA graph
(workspaces are allocated per call, never shared).  Gradients are reverse-mode,
once: forward-mode tangents and create_graph=True raise.  Capture a backward pass
only while no eager graph of the same leaves is alive.
"""
from __future__ import annotations

import ctypes
import os
import threading
from dataclasses import dataclass

import torch
import torch.autograd.forward_ad as _forward_ad

from . import LAPSUM_ECUDA, LAPSUM_OK, LapsumError, status_string

__all__ = ["route", "plan", "dispatch", "combine", "linear", "mlp", "Plan", "MAX_EXPERTS", "MAX_K", "MAX_GROUPS",
           "STATUS_TIMEOUT", "library_path"]

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "liblapsum_experts.so")
MAX_EXPERTS, MAX_K, MAX_GROUPS = 1024, 32, 32
STATUS_TIMEOUT = 0x1  # a bounded device wait of a product gave up: what it left undone is NaN

_SCORES = {"softmax": 0, "sigmoid": 1, "identity": 2}
_ACTS = {None: 0, "relu": 1, "silu": 2, "gelu": 3, "swiglu": 4}

_lib = None
_lib_lock = threading.Lock()


def library_path() -> str:
    return _LIB_PATH


class ExpertsError(LapsumError):
    """LapsumError of this library (its own text behind LAPSUM_ECUDA)."""

    def __init__(self, code: int, where: str):
        msg = f"{where}: {status_string(code)} (code {code})"
        if code == LAPSUM_ECUDA:
            msg += f": {_load().lapsum_experts_last_cuda_error().decode()}"
        RuntimeError.__init__(self, msg)
        self.code = code


def _load():
    global _lib
    if _lib is not None:
        return _lib
    with _lib_lock:
        if _lib is None:
            from . import _build
            if _build.stale_experts(_LIB_PATH):
                _build.build_experts()
            if not os.path.exists(_LIB_PATH):
                raise RuntimeError(f"native library missing: {_LIB_PATH}")
            lib = ctypes.CDLL(_LIB_PATH)
            P, i64, i32, sz, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
            for name, args in {
                "route_fwd": [P, i32, i64, i32, i64, i32, i32, P, i32, i32, i32, i32, f32, P, P, P],
                "route_bwd": [P, i32, i64, i32, i64, i32, i32, P, i32, f32, P, P, P, P, i64, P],
                "plan": [P, i64, i32, P, P, P, P, sz, P],
                "dispatch": [P, i32, i64, i32, i64, i64, P, P, i64, P],
                "combine": [P, i32, i64, i32, i64, i64, P, P, P, i64, P, i64, P],
                "combine_bwd": [P, i32, i64, i32, i64, i64, P, i64, P, P, P, P, i64, P, P],
                "linear_fwd": [P, i32, i64, i64, i64, P, i32, i64, P, P, i32, P, i64, P, i64, P, i64, P, P],
                "linear_act_bwd": [P, i32, i64, i64, i64, P, i64, i32, P, i32, P, i64, P, P, sz, P],
                "linear_dx": [P, i32, i64, i64, i64, P, i32, i64, P, P, i64, P, P],
                "linear_dweight": [P, i32, i64, i64, i64, P, i64, i64, i32, P, P, P, P],
                "linear_bwd": [P, i32, i64, i64, i64, P, P, i64, i64, P, i32, P, i32, P, P, P, P, P, sz, P],
                "mlp_fwd": [P, i32, i64, i64, i64, P, P, i32, P, P, i32, i64, i32, P, P, i64, P, i64, P, i64, i32, P, P, sz,
                            P],
                "mlp_bwd": [P, i32, i64, i64, i64, P, i32, P, i32, i64, i32, P, i64, P, i32, P, P, P, P, P, P, P, P, sz, P],
                "trace_collect": [ctypes.c_char_p, sz],
            }.items():
                fn = getattr(lib, "lapsum_experts_" + name)
                fn.argtypes, fn.restype = args, ctypes.c_int
            lib.lapsum_experts_plan_workspace_size.argtypes = [i64, i32]
            lib.lapsum_experts_plan_workspace_size.restype = sz
            lib.lapsum_experts_linear_act_workspace_size.argtypes = [i64, i32, i64]
            lib.lapsum_experts_linear_act_workspace_size.restype = sz
            lib.lapsum_experts_linear_bwd_workspace_size.argtypes = [i64, i32, i64, i32, i32]
            lib.lapsum_experts_linear_bwd_workspace_size.restype = sz
            lib.lapsum_experts_mlp_workspace_size.argtypes = [i64, i32, i32, i64, i64, i32, i64, i32]
            lib.lapsum_experts_mlp_bwd_workspace_size.argtypes = [i64, i32, i32, i64, i64, i32, i64]
            lib.lapsum_experts_mlp_bwd_workspace_size.restype = sz
            lib.lapsum_experts_mlp_workspace_size.restype = sz
            lib.lapsum_experts_last_cuda_error.argtypes = []
            lib.lapsum_experts_last_cuda_error.restype = ctypes.c_char_p
            lib.lapsum_experts_launch_count.argtypes = []
            lib.lapsum_experts_launch_count.restype = ctypes.c_uint64
            lib.lapsum_experts_test_timeout.argtypes = [ctypes.c_uint32]
            lib.lapsum_experts_test_timeout.restype = None
            lib.lapsum_experts_trace_enable.argtypes = [i32]
            lib.lapsum_experts_trace_enable.restype = None
            _lib = lib
    return _lib


# ---------------------------------------------------------------------------
# tensor marshalling
# ---------------------------------------------------------------------------
_F32, _BF16, _F16, _I32 = torch.float32, torch.bfloat16, torch.float16, torch.int32
_DTYPES = {_F32: 0, _BF16: 1, _F16: 2}
_fns: dict = {}  # entry points by name


def _stream_of(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# the same handle without the Stream object around it (3 us of the 5 us a call takes)
_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", _stream_of)


def _call(name, index, *args):
    """lapsum_experts_<name>(*args, stream) on the current stream of device `index`."""
    fn = _fns.get(name)
    if fn is None:
        fn = _fns[name] = getattr(_load(), "lapsum_experts_" + name)
    if torch.cuda.current_device() == index:
        rc = fn(*args, _stream_of(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _stream_of(index))
    if rc != LAPSUM_OK:
        raise ExpertsError(rc, "lapsum_experts_" + name)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _dtype(t, name, *, half_only=False):
    code = _DTYPES.get(t.dtype)
    if code is None or (half_only and code == 0):
        raise TypeError(f"{name} must be {'' if half_only else 'float32, '}bfloat16 or float16, got {t.dtype}")
    return code


def _cuda(t, name, dim=None, dev=None):
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        raise TypeError(f"{name} must be a CUDA tensor (this library has no CPU path)")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name} must be {dim}-D, got shape {tuple(t.shape)}")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    return t


def _rows_of(t):
    """t (2-D) with unit stride along its rows and rows that do not overlap."""
    if t.is_contiguous():
        return t
    r, n = t.shape
    if (t.stride(1) == 1 or n == 1) and (t.stride(0) >= n or r == 1):
        return t
    return t.contiguous()


def _stride(t):
    """Row stride that the C ABI gets (of one row it is never used)."""
    return t.stride(0) if t.shape[0] > 1 else max(1, t.shape[1])


def _rows16(t):
    """t (2-D, 16-bit) with rows that start on 16-byte boundaries, as tiled
    copies need them."""
    t = _rows_of(t)
    if t.data_ptr() % 16 or (t.shape[0] > 1 and t.stride(0) % 8):
        t = t.clone(memory_format=torch.contiguous_format)
    return t


def _dense16(t):
    t = t.contiguous()
    return t.clone() if t.data_ptr() % 16 else t


def _index(t, name, dev):
    if t.dtype != _I32:
        raise TypeError(f"{name} must be int32, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    return t.contiguous()


_functions: dict = {}


def _function(name):
    """The autograd.Function of an operator, made on first use."""
    if not _functions:
        _make_functions()
    return _functions[name]


def _tracked(*ts):
    """Whether the call goes through its autograd.Function: some input wants a
    gradient, or carries a forward-mode tangent (which the function refuses)."""
    if torch.is_grad_enabled():
        for t in ts:
            if t is not None and t.requires_grad:
                return True
    if getattr(_forward_ad, "_current_level", 0) >= 0:  # else no tangents exist
        return any(t is not None and _forward_ad.unpack_dual(t).tangent is not None for t in ts)
    return False


def _once():
    """The gradients' own gradients are not there."""
    if torch.is_grad_enabled():
        raise RuntimeError("the expert operators cannot be differentiated twice (create_graph=True)")


# ---------------------------------------------------------------------------
# operators
# ---------------------------------------------------------------------------
def _route_fwd(scores, k, score, bias, groups, kept, top, renormalize, scale):
    t, e = scores.shape
    w = torch.empty((t, k), dtype=_F32, device=scores.device)
    chosen = torch.empty((t, k), dtype=_I32, device=scores.device)
    if t:
        _call("route_fwd", scores.get_device(), scores.data_ptr(), _dtype(scores, "scores"), t, e, _stride(scores), k, score,
              _ptr(bias), groups, kept, top, int(renormalize), scale, w.data_ptr(), chosen.data_ptr())
    return w, chosen


def route(scores, k: int, *, score: str = "softmax", bias=None, groups: int = 1, groups_kept: int | None = None,
          group_top: int = 1, renormalize: bool = True, scale: float = 1.0):
    """The k experts of every token and their weights, as (weights, chosen):
    fp32 and int32, both [tokens, k].

    scores [tokens, E] (fp32, bf16 or fp16) become s = softmax(scores),
    sigmoid(scores) or, for "identity", scores as they are (memberships, for
    instance soft_topk's).  The experts with the highest s + bias are chosen,
    in descending order, ties to the lowest index; with groups > 1 only from
    the groups_kept (default: all) groups with the highest sum of their
    group_top (1 or 2) highest keys.  weights = scale * s, divided by the sum
    of the chosen s if renormalize.  The bias (fp32 [E]) moves the choice, not
    the weights, and gets no gradient.

    A score or bias of -inf masks an expert.  Where fewer than k are left the
    places get expert -1 and weight 0; a token with a NaN or +inf (unmasked)
    gets expert -1 and weight NaN."""
    _cuda(scores, "scores", 2)
    _dtype(scores, "scores")
    t, e = scores.shape
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, got {score!r}")
    k, groups, group_top, scale = int(k), int(groups), int(group_top), float(scale)
    kept = groups if groups_kept is None else int(groups_kept)
    if not 1 <= e <= MAX_EXPERTS:
        raise ValueError(f"scores must have 1 to {MAX_EXPERTS} experts, got {e}")
    if not 1 <= groups <= MAX_GROUPS or e % groups or not 1 <= kept <= groups or group_top not in (1, 2):
        raise ValueError(f"{groups} groups ({kept} kept, group_top {group_top}) do not fit {e} experts: groups divides "
                         f"them, is at most {MAX_GROUPS}, groups_kept at most groups, group_top 1 or 2")
    if not 1 <= k <= min(MAX_K, e // groups * kept):
        raise ValueError(f"k must be in 1..{min(MAX_K, e // groups * kept)}, got {k}")
    if not 0.0 < scale < float("inf"):
        raise ValueError(f"scale must be finite and positive, got {scale}")
    if bias is not None:
        _cuda(bias, "bias", 1, scores.device)
        if bias.dtype != _F32 or bias.shape[0] != e:
            raise ValueError(f"bias must be float32 [{e}], got {bias.dtype} {tuple(bias.shape)}")
        bias = bias.detach().contiguous()
    args = (k, _SCORES[score], bias, groups, kept, group_top, bool(renormalize), scale)
    if _tracked(scores):
        return _function("route").apply(scores, *args)
    return _route_fwd(_rows_of(scores), *args)


@dataclass
class Plan:
    """Where the slots (token * k + j) of a choice stand in expert order: rows and
    slots are each other's inverse.  A place may be taken away from combine()
    by setting its row to -1."""
    offsets: object   # int32 [experts + 1]: expert e has rows offsets[e] .. offsets[e + 1] - 1
    rows: object      # int32 [tokens, k]: the row of a slot, -1 if its expert is -1
    slots: object     # int32 [tokens * k]: the slot of a row, -1 from offsets[-1] on


def plan(chosen, experts: int) -> Plan:
    """Plan of the exchange for chosen [tokens, k] (int32, from route()); a
    place whose expert is not in 0..experts-1 is dropped.  The rows of one
    expert are in the order of their slots."""
    _cuda(chosen, "chosen", 2)
    experts = int(experts)
    if not 1 <= experts <= MAX_EXPERTS:
        raise ValueError(f"experts must be in 1..{MAX_EXPERTS}, got {experts}")
    if not 1 <= chosen.shape[1] <= MAX_K:
        raise ValueError(f"chosen must have 1 to {MAX_K} places per token, got {chosen.shape[1]}")
    chosen = _index(chosen, "chosen", chosen.device)
    n, dev = chosen.numel(), chosen.device
    if n == 0:
        return Plan(torch.zeros(experts + 1, dtype=_I32, device=dev), torch.empty_like(chosen),
                    torch.empty(0, dtype=_I32, device=dev))
    offsets = torch.empty(experts + 1, dtype=_I32, device=dev)
    rows = torch.empty_like(chosen)
    slots = torch.empty(n, dtype=_I32, device=dev)
    need = int(_load().lapsum_experts_plan_workspace_size(n, experts))
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    _call("plan", chosen.get_device(), chosen.data_ptr(), n, experts, offsets.data_ptr(), rows.data_ptr(), slots.data_ptr(), _ptr(ws),
          need)
    return Plan(offsets, rows, slots)


def _check_plan(p, dev):
    t, k = p.rows.shape
    rows, slots = _index(p.rows, "plan.rows", dev), _index(p.slots, "plan.slots", dev)
    if slots.numel() != t * k:
        raise ValueError(f"plan.slots must hold {t * k} slots, got {slots.numel()}")
    return t, k, rows, slots


def _dispatch(x, slots, t, k):
    out = torch.empty((t * k, x.shape[1]), dtype=x.dtype, device=x.device)
    if out.numel():
        _call("dispatch", x.get_device(), x.data_ptr(), _dtype(x, "x"), t, k, x.shape[1], _stride(x), slots.data_ptr(),
              out.data_ptr(), x.shape[1])
    return out


def dispatch(x, p: Plan):
    """Token order to expert order: row r of the result [tokens * k, dim] is
    the token x[slots[r] // k] (zeros from offsets[-1] on).  fp32, bf16, fp16."""
    _cuda(x, "x", 2)
    _dtype(x, "x")
    t, k, rows, slots = _check_plan(p, x.device)
    if x.shape[0] != t:
        raise ValueError(f"x must have the plan's {t} tokens, got {x.shape[0]}")
    if _tracked(x):
        return _function("dispatch").apply(x, rows, slots)
    return _dispatch(_rows_of(x), slots, t, k)


def _combine(y, weights, rows, residual):
    (t, k), dim = rows.shape, y.shape[1]
    out = torch.empty((t, dim), dtype=y.dtype, device=y.device)
    if out.numel():
        _call("combine", y.get_device(), y.data_ptr(), _dtype(y, "y"), t, k, dim, _stride(y), _ptr(weights), rows.data_ptr(),
              _ptr(residual), _stride(residual) if residual is not None else 0, out.data_ptr(), dim)
    return out


def combine(y, weights, p: Plan, *, residual=None):
    """Expert order to token order: out[t] = residual[t] + sum_j weights[t, j]
    y[rows[t, j]], summed in fp32 in the order of j.  y [tokens * k, dim] (fp32,
    bf16, fp16), weights fp32 [tokens, k], residual [tokens, dim] of y's type."""
    _cuda(y, "y", 2)
    _dtype(y, "y")
    dev = y.device
    t, k, rows, slots = _check_plan(p, dev)
    if y.shape[0] != t * k:
        raise ValueError(f"y must have the plan's {t * k} rows, got {y.shape[0]}")
    _cuda(weights, "weights", 2, dev)
    if weights.dtype != _F32 or tuple(weights.shape) != (t, k):
        raise ValueError(f"weights must be float32 [{t}, {k}], got {weights.dtype} {tuple(weights.shape)}")
    if residual is not None:
        _cuda(residual, "residual", 2, dev)
        if residual.dtype != y.dtype or tuple(residual.shape) != (t, y.shape[1]):
            raise ValueError(f"residual must be {y.dtype} [{t}, {y.shape[1]}], got {residual.dtype} "
                             f"{tuple(residual.shape)}")
    if _tracked(y, weights, residual):
        return _function("combine").apply(y, weights, residual, rows, slots)
    return _combine(_rows_of(y), weights.contiguous(), rows, None if residual is None else _rows_of(residual))


def _linear_fwd(x, weight, offsets, bias, act, residual, keep, status):
    """y and, with keep, the pre-activation; x, weight laid out for the kernels."""
    r, (experts, n, _) = x.shape[0], weight.shape
    width = n // 2 if act == 4 else n
    y = torch.empty((r, width), dtype=x.dtype, device=x.device)
    h = torch.empty((r, n), dtype=x.dtype, device=x.device) if keep else None
    if r:
        _call("linear_fwd", x.get_device(), x.data_ptr(), _dtype(x, "x"), r, x.shape[1], _stride(x), weight.data_ptr(), experts,
              n, _ptr(offsets), _ptr(bias), act, _ptr(residual), _stride(residual) if residual is not None else 0,
              y.data_ptr(), width, _ptr(h), n, _ptr(status))
    return y, h


def _check_linear(x, weight, offsets, bias, activation, residual, status):
    """The activation's number, or an error that says what is wrong."""
    _cuda(x, "x", 2)
    _dtype(x, "x", half_only=True)
    dev = x.device
    if activation not in _ACTS:
        raise ValueError(f"activation must be None or one of {sorted(a for a in _ACTS if a)}, got {activation!r}")
    act = _ACTS[activation]
    _cuda(weight, "weight", 2 if offsets is None else 3, dev)
    n, k = weight.shape[-2:]
    experts = 1 if offsets is None else weight.shape[0]
    if weight.dtype != x.dtype:
        raise TypeError(f"weight must be {x.dtype}, got {weight.dtype}")
    if k != x.shape[1]:
        raise ValueError(f"weight must have x's {x.shape[1]} inputs, got {k}")
    if k % 8 or n % (16 if act == 4 else 8) or not k or not n:
        raise ValueError(f"inputs and outputs must be multiples of 8 (outputs of 16 for swiglu), got {k} and {n}")
    if offsets is not None:
        if not 1 <= experts <= MAX_EXPERTS:
            raise ValueError(f"weight must have 1 to {MAX_EXPERTS} experts, got {experts}")
        _index(_cuda(offsets, "offsets", 1), "offsets", dev)
        if offsets.shape[0] != experts + 1:
            raise ValueError(f"offsets must hold {experts + 1} values, got {offsets.shape[0]}")
    shape = tuple(weight.shape[:-1])
    if bias is not None:
        _cuda(bias, "bias", None, dev)
        if bias.dtype != x.dtype or tuple(bias.shape) != shape:
            raise ValueError(f"bias must be {x.dtype} {list(shape)}, got {bias.dtype} {tuple(bias.shape)}")
    width = n // 2 if act == 4 else n
    if residual is not None:
        _cuda(residual, "residual", 2, dev)
        if residual.dtype != x.dtype or tuple(residual.shape) != (x.shape[0], width):
            raise ValueError(f"residual must be {x.dtype} [{x.shape[0]}, {width}], got {residual.dtype} "
                             f"{tuple(residual.shape)}")
    if status is not None and (_cuda(status, "status", None, dev).dtype != _I32 or status.numel() < 1):
        raise TypeError("status must be an int32 tensor")
    return act


def linear(x, weight, offsets=None, *, bias=None, activation: str | None = None, residual=None, status=None):
    """act(W_e x_r + b_e) + residual_r for the rows offsets[e] <= r < offsets[e + 1]
    of expert e, on the tensor cores with fp32 sums and one rounding.

    x [rows, in] bf16 or fp16; weight [experts, out, in] of that type, with
    offsets int32 [experts + 1] on the device (a Plan's) ascending from 0, or
    [out, in] with offsets None: one matrix for all rows.  in and out are
    multiples of 8.  bias [experts, out] (or [out]) and residual of the type.
    activation: None, "relu", "silu", "gelu" (by erf) or "swiglu" (silu of the
    first half of the outputs times the second: out a multiple of 16, the
    result half as wide).  Rows from offsets[-1] on get the residual (0).
    Gradients take the pre-activation rounded to the type, beyond its range the
    type's largest value.

    status: an int32 [1] tensor into which STATUS_* bits are or'ed (optional)."""
    act = _check_linear(x, weight, offsets, bias, activation, residual, status)
    n, k = weight.shape[-2:]
    experts = 1 if offsets is None else weight.shape[0]
    if offsets is not None:
        offsets = offsets.contiguous()
    if _tracked(x, weight, bias, residual):
        return _function("linear").apply(x, weight, bias, residual, offsets, act, status)
    w = _dense16(weight).view(experts, n, k)
    return _linear_fwd(_rows16(x), w, offsets, None if bias is None else bias.contiguous(), act,
                       None if residual is None else _rows16(residual), False, status)[0]


def _check_weight(weight, bias, name, x, din, act):
    _cuda(weight, name, 3, x.device)
    if weight.dtype != x.dtype:
        raise TypeError(f"{name} must be {x.dtype}, got {weight.dtype}")
    e, n, k = weight.shape
    if k != din:
        raise ValueError(f"{name} must have {din} inputs, got {k}")
    if not 1 <= e <= MAX_EXPERTS:
        raise ValueError(f"{name} must have 1 to {MAX_EXPERTS} experts, got {e}")
    if k % 8 or n % (16 if act == 4 else 8) or not k or not n:
        raise ValueError(f"inputs and outputs must be multiples of 8 (outputs of 16 for swiglu), got {k} and {n}")
    if bias is not None:
        _cuda(bias, "its bias", 2, x.device)
        if bias.dtype != x.dtype or tuple(bias.shape) != (e, n):
            raise ValueError(f"the bias of {name} must be {x.dtype} [{e}, {n}], got {bias.dtype} {tuple(bias.shape)}")
    return e, n


def _mlp_fwd(x, weights, chosen, w_in, w_out, b_in, b_out, act, residual, status, keep):
    """The layer, and its workspace (with keep: what its gradient takes)."""
    t, k = chosen.shape
    (e, up, d), dim = w_in.shape, w_out.shape[1]
    out = torch.empty((t, dim), dtype=x.dtype, device=x.device)
    need = _load().lapsum_experts_mlp_workspace_size(t, k, e, d, up, act, dim, keep)
    ws = torch.empty(need, dtype=torch.uint8, device=x.device)
    if t:
        _call("mlp_fwd", x.get_device(), x.data_ptr(), _DTYPES[x.dtype], t, d, _stride(x), weights.data_ptr(),
              chosen.data_ptr(), k, w_in.data_ptr(), _ptr(b_in), e, up, act, w_out.data_ptr(), _ptr(b_out), dim,
              _ptr(residual), _stride(residual) if residual is not None else 0, out.data_ptr(), dim, keep, _ptr(status),
              ws.data_ptr(), need)
    return out, ws


def mlp(x, weights, chosen, w_in, w_out, *, b_in=None, b_out=None, activation: str | None = "swiglu", residual=None,
        status=None):
    """A layer of experts: every token's weighted sum over its chosen experts of
    W_out act(W_in x + b_in) + b_out, plus residual: plan, dispatch, linear,
    linear and combine in one call (and one gradient).  x [tokens, dim] bf16 or
    fp16; weights and chosen [tokens, k] from route(); w_in [experts, hidden
    (twice for swiglu), dim], w_out [experts, dim_out, hidden]; biases
    [experts, ...]; residual [tokens, dim_out], x itself for instance; status
    as in linear()."""
    _cuda(x, "x", 2)
    _dtype(x, "x", half_only=True)
    dev = x.device
    if activation not in _ACTS:
        raise ValueError(f"activation must be None or one of {sorted(a for a in _ACTS if a)}, got {activation!r}")
    act = _ACTS[activation]
    e, up = _check_weight(w_in, b_in, "w_in", x, x.shape[1], act)
    e2, dim = _check_weight(w_out, b_out, "w_out", x, up // 2 if act == 4 else up, 0)
    if e != e2:
        raise ValueError(f"w_in and w_out must have the same experts, got {e} and {e2}")
    _cuda(chosen, "chosen", 2, dev)
    chosen = _index(chosen, "chosen", dev)
    t, k = chosen.shape
    if t != x.shape[0] or not 1 <= k <= MAX_K:
        raise ValueError(f"chosen must have x's {x.shape[0]} tokens and 1 to {MAX_K} places, got {tuple(chosen.shape)}")
    _cuda(weights, "weights", 2, dev)
    if weights.dtype != _F32 or tuple(weights.shape) != (t, k):
        raise ValueError(f"weights must be float32 [{t}, {k}], got {weights.dtype} {tuple(weights.shape)}")
    if residual is not None:
        _cuda(residual, "residual", 2, dev)
        if residual.dtype != x.dtype or tuple(residual.shape) != (t, dim):
            raise ValueError(f"residual must be {x.dtype} [{t}, {dim}], got {residual.dtype} {tuple(residual.shape)}")
    if status is not None and (_cuda(status, "status", None, dev).dtype != _I32 or status.numel() < 1):
        raise TypeError("status must be an int32 tensor")
    if _tracked(x, weights, w_in, w_out, b_in, b_out, residual):
        own = residual is x  # its gradient joins that of x in one pass
        return _function("mlp").apply(x, weights, w_in, w_out, b_in, b_out, None if own else residual, own, chosen, act,
                                      status)
    return _mlp_fwd(_rows_of(x), weights.contiguous(), chosen, _dense16(w_in), _dense16(w_out),
                    None if b_in is None else b_in.contiguous(), None if b_out is None else b_out.contiguous(), act,
                    None if residual is None else _rows_of(residual), status, 0)[0]


# ---------------------------------------------------------------------------
# gradients
# ---------------------------------------------------------------------------
def _combine_bwd(g, y, weights, rows, slots, need_y, need_w):
    (t, k), dim = rows.shape, y.shape[1]
    gy = torch.empty((t * k, dim), dtype=y.dtype, device=y.device) if need_y else None
    gw = torch.empty_like(weights) if need_w else None
    if (need_y or need_w) and t * dim:
        _call("combine_bwd", y.get_device(), g.data_ptr(), _dtype(y, "y"), t, k, dim, _stride(g), y.data_ptr(), _stride(y),
              weights.data_ptr(), rows.data_ptr(), slots.data_ptr(), _ptr(gy), dim, _ptr(gw))
    elif gw is not None:
        gw.zero_()
    return gy, gw


def _linear_bwd(g, x, w, offsets, h, act, need_x, need_w, need_b, status):
    """(dx, dweight, dbias) for dy = g; h the pre-activation of act != 0."""
    experts, n, k = w.shape
    r, dev = x.shape[0], x.device
    gb = torch.empty((experts, n), dtype=x.dtype, device=dev) if need_b else None
    gx = torch.empty((r, k), dtype=x.dtype, device=dev) if need_x else None
    gw = torch.empty((experts, n, k), dtype=x.dtype, device=dev) if need_w else None
    if r == 0:
        for z in (gb, gw):
            if z is not None:
                z.zero_()
        return gx, gw, gb
    if need_x or need_w or need_b:
        g = _rows16(g)
        need = _load().lapsum_experts_linear_bwd_workspace_size(r, experts, n, act, need_b)
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        _call("linear_bwd", x.get_device(), g.data_ptr(), _DTYPES[x.dtype], r, n, _stride(g), _ptr(h), x.data_ptr(), k,
              _stride(x), w.data_ptr(), experts, _ptr(offsets), act, _ptr(gx), _ptr(gw), _ptr(gb), _ptr(status), _ptr(ws),
              need)
    return gx, gw, gb


def _make_functions():
    class Route(torch.autograd.Function):
        @staticmethod
        def forward(ctx, scores, k, score, bias, groups, kept, top, renormalize, scale):
            x = _rows_of(scores)
            w, chosen = _route_fwd(x, k, score, bias, groups, kept, top, renormalize, scale)
            ctx.save_for_backward(x, bias, w, chosen)
            ctx.rule = (k, score, renormalize, scale)
            ctx.mark_non_differentiable(chosen)
            return w, chosen

        @staticmethod
        def backward(ctx, gw, _):
            _once()
            x, bias, w, chosen = ctx.saved_tensors
            k, score, renormalize, scale = ctx.rule
            t, e = x.shape
            grad = torch.empty((t, e), dtype=x.dtype, device=x.device)
            if t:
                gw = gw.contiguous()
                _call("route_bwd", x.get_device(), x.data_ptr(), _dtype(x, "scores"), t, e, _stride(x), k, score, _ptr(bias),
                      int(renormalize), scale, chosen.data_ptr(), w.data_ptr(), gw.data_ptr(), grad.data_ptr(), e)
            return (grad,) + (None,) * 8

    class Dispatch(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, rows, slots):
            ctx.save_for_backward(rows)
            return _dispatch(_rows_of(x), slots, *rows.shape)

        @staticmethod
        def backward(ctx, g):
            _once()
            (rows,) = ctx.saved_tensors
            return _combine(_rows_of(g), None, rows, None), None, None

    class Combine(torch.autograd.Function):
        @staticmethod
        def forward(ctx, y, weights, residual, rows, slots):
            y2, w2 = _rows_of(y), weights.contiguous()
            ctx.save_for_backward(y2, w2, rows, slots)
            return _combine(y2, w2, rows, None if residual is None else _rows_of(residual))

        @staticmethod
        def backward(ctx, g):
            _once()
            y, w, rows, slots = ctx.saved_tensors
            need_y, need_w, need_r = ctx.needs_input_grad[:3]
            gy, gw = _combine_bwd(_rows_of(g), y, w, rows, slots, need_y, need_w)
            return gy, gw, g if need_r else None, None, None

    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, weight, bias, residual, offsets, act, status):
            x2 = _rows16(x)
            n, k = weight.shape[-2:]
            w2 = _dense16(weight).view(-1, n, k)
            y, h = _linear_fwd(x2, w2, offsets, None if bias is None else bias.contiguous(), act,
                               None if residual is None else _rows16(residual), act != 0, status)
            ctx.save_for_backward(x2, w2, offsets, h)
            ctx.act, ctx.weight_shape, ctx.status = act, weight.shape, status
            return y

        @staticmethod
        def backward(ctx, g):
            _once()
            x, w, offsets, h = ctx.saved_tensors
            need_x, need_w, need_b, need_r = ctx.needs_input_grad[:4]
            gx, gw, gb = _linear_bwd(g, x, w, offsets, h, ctx.act, need_x, need_w, need_b, ctx.status)
            if gw is not None:
                gw = gw.view(ctx.weight_shape)
            if gb is not None:
                gb = gb.view(ctx.weight_shape[:-1])
            return gx, gw, gb, g if need_r else None, None, None, None

    class Mlp(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, weights, w_in, w_out, b_in, b_out, residual, own, chosen, act, status):
            x2, w2, wi, wo = _rows_of(x), weights.contiguous(), _dense16(w_in), _dense16(w_out)
            res = x2 if own else None if residual is None else _rows_of(residual)
            out, kept = _mlp_fwd(x2, w2, chosen, wi, wo, None if b_in is None else b_in.contiguous(),
                                 None if b_out is None else b_out.contiguous(), act, res, status, 1)
            ctx.save_for_backward(w2, wi, wo, kept)
            ctx.act, ctx.own, ctx.status = act, own, status
            return out

        @staticmethod
        def backward(ctx, g):
            _once()
            weights, w_in, w_out, kept = ctx.saved_tensors
            need_x, need_w, need_in, need_out, need_bi, need_bo, need_r = ctx.needs_input_grad[:7]
            (t, k), (e, up, d), dim, act = weights.shape, w_in.shape, w_out.shape[1], ctx.act
            new = w_in.new_zeros if t == 0 else w_in.new_empty
            gx = new((t, d)) if need_x else None
            gw = torch.empty_like(weights) if need_w else None
            gwi = new((e, up, d)) if need_in else None
            gwo = new(w_out.shape) if need_out else None
            gbi = new((e, up)) if need_bi else None
            gbo = new((e, dim)) if need_bo else None
            if t and any(ctx.needs_input_grad[:6]):
                g2 = _rows_of(g)
                need = _load().lapsum_experts_mlp_bwd_workspace_size(t, k, e, d, up, act, dim)
                ws = torch.empty(need, dtype=torch.uint8, device=g.device)
                _call("mlp_bwd", g2.get_device(), g2.data_ptr(), _DTYPES[g2.dtype], t, d, _stride(g2), weights.data_ptr(), k,
                      w_in.data_ptr(), e, up, act, w_out.data_ptr(), dim, kept.data_ptr(), ctx.own, _ptr(gx), _ptr(gw),
                      _ptr(gwi), _ptr(gbi), _ptr(gwo), _ptr(gbo), _ptr(ctx.status), ws.data_ptr(), need)
            return gx, gw, gwi, gwo, gbi, gbo, g if need_r else None, None, None, None, None

    _functions.update(route=Route, dispatch=Dispatch, combine=Combine, linear=Linear, mlp=Mlp)
