"""ctypes binding of ``include/qlora_train.h``: the operators around the
quantized linear in a fine-tuning step.  Argument marshalling only, names as in
the C header; torch supplies device memory and the current HIP stream.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import binding as _b
from .binding import QLoRAError

_DT = _b._DTYPE_ENUM
ADAMW_BLOCK = 256
_c = ctypes
_vp, _i64, _i32, _f32, _f64, _sz = (_c.c_void_p, _c.c_int64, _c.c_int32, _c.c_float, _c.c_double,
                                    _c.c_size_t)


class _Resnorm(_c.Structure):
    _fields_ = [("m", _i64), ("d", _i64), ("act_dtype", _i32), ("res_dtype", _i32),
                ("param_dtype", _i32), ("post", _i32), ("pre", _i32), ("gate_kind", _i32),
                ("scale", _f32), ("eps", _f32), ("w_offset", _f32),
                ("x", _vp), ("y", _vp), ("gate", _vp), ("w_post", _vp), ("w_pre", _vp),
                ("ldx", _i64), ("ldy", _i64), ("ldg", _i64), ("h", _vp), ("z", _vp),
                ("ldh", _i64), ("ldz", _i64)]


class _ResnormGrad(_c.Structure):
    _fields_ = [("m", _i64), ("d", _i64), ("act_dtype", _i32), ("res_dtype", _i32),
                ("param_dtype", _i32), ("post", _i32), ("pre", _i32), ("gate_kind", _i32),
                ("scale", _f32), ("eps", _f32), ("w_offset", _f32),
                ("dz", _vp), ("dh", _vp), ("h", _vp), ("y", _vp), ("gate", _vp), ("w_post", _vp),
                ("w_pre", _vp), ("lddz", _i64), ("lddh", _i64), ("ldh", _i64), ("ldy", _i64),
                ("ldg", _i64), ("dx", _vp), ("dy", _vp), ("dgate", _vp), ("lddx", _i64),
                ("lddy", _i64), ("lddg", _i64), ("dw_post", _vp), ("dw_pre", _vp)]


class _OptTensor(_c.Structure):
    _fields_ = [("p", _vp), ("g", _vp), ("p_out", _vp), ("copy", _vp), ("n", _i64),
                ("lr_mul", _f32), ("wd_mul", _f32)]


class _AdamW(_c.Structure):
    _fields_ = [("table", _vp), ("count", _i32), ("p_dtype", _i32), ("g_dtype", _i32),
                ("copy_dtype", _i32), ("state_bits", _i32), ("blocks", _i64), ("chunks", _i64)]


class _OptState(_c.Structure):
    _fields_ = [("m", _vp), ("v", _vp), ("m_scale", _vp), ("v_scale", _vp)]


class _Hyper(_c.Structure):
    _fields_ = [("step", _i64), ("lr", _f64), ("beta1", _f64), ("beta2", _f64), ("eps", _f64),
                ("weight_decay", _f64), ("seed", _c.c_uint32)]


_lib = None


def lib():
    """The loaded library with this header's entry points declared."""
    global _lib
    if _lib is None:
        L = _b.lib()
        P, int_ = _c.POINTER, _c.c_int
        for name, res, args in (
                ("qlora_embed_fwd", int_, [_vp, int_, _i64, _i64, _i64, _vp, int_, _i64, _f32, _vp,
                                           int_, _i64, _vp]),
                ("qlora_embed_workspace_bytes", _sz, [_i64, _i64, _i64]),
                ("qlora_embed_bwd", int_, [_vp, int_, _i64, _i64, _i64, _vp, int_, _i64, _f32, _vp,
                                           int_, _i64, int_, _vp, _sz, _vp]),
                ("qlora_resnorm_fwd", int_, [P(_Resnorm), _vp]),
                ("qlora_resnorm_workspace_bytes", _sz, [_i64, _i64]),
                ("qlora_resnorm_bwd", int_, [P(_ResnormGrad), _vp, _sz, _vp]),
                ("qlora_adamw_table_bytes", _sz, [P(_i64), int_]),
                ("qlora_adamw_init", int_, [P(_AdamW), P(_OptTensor), int_, int_, int_, int_, int_,
                                            _vp, _sz]),
                ("qlora_grad_norm_workspace_bytes", _sz, [P(_AdamW)]),
                ("qlora_grad_norm", int_, [P(_AdamW), _f32, _vp, _vp, _sz, _vp]),
                ("qlora_adamw_step", int_, [P(_AdamW), P(_OptState), P(_OptState), P(_Hyper), _vp,
                                            _vp])):
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _lib = L
    return _lib


def _check(status, what):
    if status:
        _b._check(status, what)


def _stream(device):
    """The current HIP stream of the tensors' device, which must be the current device.  The raw
    handle is asked for: building a torch.cuda.Stream object takes 2.8 us, as much as a launch.  A torch
    without GPU support lacks these names, but has no tensor that gets to them."""
    i = device.index
    if i is None or i != torch._C._cuda_getDevice():
        raise QLoRAError(f"tensors must be on the current GPU, not on {device}")
    return torch._C._cuda_getCurrentRawStream(i)


def _dt(t, name):
    e = _DT.get(t.dtype)
    if e is None:
        raise QLoRAError(f"{name}: unsupported dtype {t.dtype}")
    return e


def _ld(t, shape, name):
    """Row stride of a 2-D tensor of the given shape with unit column stride."""
    if t.shape != shape:
        raise QLoRAError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    ld, col = t.stride()
    if col == 1 and ld >= shape[1]:
        return ld
    if col != 1 and shape[1] > 1:
        raise QLoRAError(f"{name} must have unit column stride")
    return ld if shape[0] > 1 else shape[1]      # the stride of a single row says nothing


def _vec(t, n, dtypes, name):
    if t.dim() != 1 or t.shape[0] != n or not t.is_contiguous() or t.dtype not in dtypes:
        raise QLoRAError(f"{name} must be a contiguous [{n}] tensor of {' or '.join(map(str, dtypes))}")
    return t.data_ptr()


def _same_device(dev, *tensors):
    for t in tensors:
        if t is not None and t.device != dev:
            raise QLoRAError(f"tensors on different devices: {dev} and {t.device}")


# ------------------------------------------------------------------ embedding

def _ids(ids):
    bits = 64 if ids.dtype == torch.int64 else 32 if ids.dtype == torch.int32 else 0
    if not bits or ids.dim() != 1 or not ids.is_contiguous():
        raise QLoRAError("ids must be a contiguous 1-D int32 or int64 tensor")
    return bits


def qlora_embed_fwd(E: torch.Tensor, ids: torch.Tensor, scale: float = 1.0, out=None,
                    out_dtype=None) -> torch.Tensor:
    """-> [m x d] scale * E[ids], zeros for ids outside the table."""
    bits, m = _ids(ids), ids.shape[0]
    vocab, d = E.shape
    if out is None:
        out = torch.empty((m, d), dtype=out_dtype or E.dtype, device=E.device)
    dev = E.device
    _same_device(dev, ids, out)
    _check(lib().qlora_embed_fwd(E.data_ptr(), _dt(E, "E"), vocab, d, _ld(E, (vocab, d), "E"),
                                 ids.data_ptr(), bits, m, scale, out.data_ptr(), _dt(out, "out"),
                                 _ld(out, (m, d), "out"), _stream(dev)), "qlora_embed_fwd")
    return out


def qlora_embed_workspace_bytes(m: int, vocab: int, d: int) -> int:
    return int(lib().qlora_embed_workspace_bytes(m, vocab, d))


def qlora_embed_bwd(dY: torch.Tensor, ids: torch.Tensor, vocab: int, scale: float = 1.0, out=None,
                    grad_dtype=torch.float32, accumulate: bool = False, workspace=None) -> torch.Tensor:
    """-> dE [vocab x d]; with accumulate the rows are added to `out`."""
    bits = _ids(ids)
    m, d = dY.shape
    if ids.shape[0] != m:
        raise QLoRAError(f"dY has {m} rows for {ids.shape[0]} ids")
    if out is None:
        if accumulate:
            raise QLoRAError("accumulate needs out")
        out = torch.empty((vocab, d), dtype=grad_dtype, device=dY.device)
    if workspace is None:
        workspace = torch.empty(qlora_embed_workspace_bytes(m, vocab, d), dtype=torch.uint8,
                                device=dY.device)
    dev = dY.device
    _same_device(dev, ids, out, workspace)
    _check(lib().qlora_embed_bwd(dY.data_ptr(), _dt(dY, "dY"), m, d, _ld(dY, (m, d), "dY"),
                                 ids.data_ptr(), bits, vocab, scale, out.data_ptr(), _dt(out, "out"),
                                 _ld(out, (vocab, d), "out"), accumulate, workspace.data_ptr(),
                                 workspace.nbytes, _stream(dev)),
           "qlora_embed_bwd")
    return out


# -------------------------------------------------------------- residual norm

def _gate_kind(gate, y, m, d):
    """Kind of a gate: [d] per channel, [m] or [m x 1] per token, [m x d] full.  A [d] gate with
    m == d is per channel."""
    if gate is None or y is None:
        return 0
    shape = gate.shape
    if len(shape) == 2:
        if shape[1] == 1 and d != 1 and shape[0] == m:
            kind = 2
        else:
            if gate.dtype != y.dtype:
                raise QLoRAError("a full gate must have y's dtype")
            return 3
    else:
        kind = 1 if shape == (d,) else 2
        if kind == 2 and shape != (m,):
            raise QLoRAError(f"gate must be [{d}], [{m}], [{m} x 1] or [{m} x {d}], got {tuple(shape)}")
    if not gate.is_contiguous():
        raise QLoRAError("a per-channel or per-token gate must be contiguous")
    return kind


def _params(act, d, w_post, w_pre, gate):
    """Dtype enum of the weights and of a per-channel or per-token gate, which they share."""
    dt = None
    for w, name in ((w_post, "w_post"), (w_pre, "w_pre")):
        if w is not None:
            if w.shape != (d,) or not w.is_contiguous():
                raise QLoRAError(f"{name} must be a contiguous [{d}] tensor")
            if dt is not None and w.dtype != dt:
                raise QLoRAError("weights and gate must share a dtype")
            dt = w.dtype
    if gate is not None:
        if dt is not None and gate.dtype != dt:
            raise QLoRAError("weights and gate must share a dtype")
        dt = gate.dtype
    if dt is None or dt == torch.float32:
        return _b.QLORA_F32
    if dt != act:
        raise QLoRAError(f"weights and gate must be float32 or {act}")
    return _DT[dt]


def _p(t):
    return None if t is None else t.data_ptr()


def qlora_resnorm_fwd(x: torch.Tensor, y=None, gate=None, w_post=None, w_pre=None, post: bool = True,
                      pre: bool = True, scale: float = 1.0, eps: float = 1e-6, w_offset: float = 0.0,
                      h_out=None, z_out=None, act_dtype=None):
    """-> (h, z): h = x + scale * gate * p, p = rms(y) (w_offset + w_post) (y itself without
    post), z = rms(h) (w_offset + w_pre) (None without pre).  Without y: (x, rms(x) ...), z in act_dtype
    (default x's).  gate: [d] per channel, [m] or [m x 1] per token, or [m x d]."""
    shape = x.shape
    m, d = shape
    dev = x.device
    act = y.dtype if y is not None else (z_out.dtype if z_out is not None else act_dtype or x.dtype)
    adt = _DT.get(act)
    if adt is None:
        raise QLoRAError(f"unsupported dtype {act}")
    kind = _gate_kind(gate, y, m, d)
    post = bool(post) and y is not None
    if not post:
        w_post = None
    if not pre:
        w_pre = None
    pdt = _params(act, d, w_post, w_pre, gate if 0 < kind < 3 else None)
    if y is None:
        h, hp, ldh, yp, ldy = x, None, 0, None, 0
    else:
        h = h_out if h_out is not None else torch.empty(shape, dtype=x.dtype, device=dev)
        if h.dtype != x.dtype:
            raise QLoRAError("h must have x's dtype")
        hp, ldh, yp, ldy = h.data_ptr(), _ld(h, shape, "h"), y.data_ptr(), _ld(y, shape, "y")
    z, zp, ldz = None, None, 0
    if pre:
        z = z_out if z_out is not None else torch.empty(shape, dtype=act, device=dev)
        if z.dtype != act:
            raise QLoRAError("z must have y's dtype")
        zp, ldz = z.data_ptr(), _ld(z, shape, "z")
    _same_device(dev, y, gate, w_post, w_pre, h, z)
    a = _Resnorm(m, d, adt, _dt(x, "x"), pdt, post, pre, kind, scale, eps, w_offset, x.data_ptr(), yp,
                 gate.data_ptr() if kind else None, _p(w_post), _p(w_pre), _ld(x, shape, "x"), ldy,
                 _ld(gate, shape, "gate") if kind == 3 else 0, hp, zp, ldh, ldz)
    status = lib().qlora_resnorm_fwd(a, _stream(dev))
    if status:
        _check(status, "qlora_resnorm_fwd")
    return h, z


def qlora_resnorm_workspace_bytes(m: int, d: int) -> int:
    return int(lib().qlora_resnorm_workspace_bytes(m, d))


def qlora_resnorm_bwd(dz, dh, h: torch.Tensor, y=None, gate=None, w_post=None, w_pre=None,
                      post: bool = True, pre: bool = True, scale: float = 1.0, eps: float = 1e-6,
                      w_offset: float = 0.0, outs=None, need=(True, True, True, True),
                      workspace=None):
    """-> (dx, dy, dgate, dw_post, dw_pre), None where there is nothing to compute.  `need` switches
    (dy, dgate, dw_post, dw_pre) off; `outs` gives the five output tensors (None: not computed; one for
    something that the call does not compute is left as it is, and None is returned in its place)."""
    ref = h if h is not None else dh
    shape, res, dev = ref.shape, ref.dtype, ref.device
    m, d = shape
    act = y.dtype if y is not None else dz.dtype if dz is not None else res
    adt = _DT.get(act)
    if adt is None:
        raise QLoRAError(f"unsupported dtype {act}")
    if not pre:
        dz = w_pre = None
    elif dz is None:
        raise QLoRAError("pre needs dz")
    post = bool(post) and y is not None
    if not post:
        w_post = None
    kind = _gate_kind(gate, y, m, d)
    pdt = _params(act, d, w_post, w_pre, gate if 0 < kind < 3 else None)
    f32 = torch.float32
    if outs is None:
        def e(s, dt):
            return torch.empty(s, dtype=dt, device=dev)
        outs = (e(shape, res),
                e(shape, act) if y is not None and need[0] else None,
                None if not kind or not need[1] else e(gate.shape, act if kind == 3 else f32),
                e((d,), f32) if post and need[2] else None,
                e((d,), f32) if pre and need[3] else None)
    dx, dy, dgate, dw_post, dw_pre = outs
    if y is None:
        dy = None
    if not kind:
        dgate = None
    if not post:
        dw_post = None
    if not pre:
        dw_pre = None
    # rows: pointer and stride
    rows = []
    for t, dt, name in ((dz, act, "dz"), (dh, res, "dh"), (h, res, "h"), (y, act, "y"), (dx, res, "dx"), (dy, act, "dy"),
                        (gate if kind == 3 else None, act, "gate"), (dgate if kind == 3 else None, act, "dgate")):
        if t is None:
            rows.append((None, 0))
            continue
        if t.dtype != dt or t.device != dev:
            raise QLoRAError(f"{name} must be {dt} on {dev}")
        rows.append((t.data_ptr(), _ld(t, shape, name)))
    (dzp, lddz), (dhp, lddh), (hp, ldh), (yp, ldy), (dxp, lddx), (dyp, lddy), (gp, ldg), (dgp, lddg) = rows
    if 0 < kind < 3:
        gp = gate.data_ptr()
        if dgate is not None:
            if dgate.dtype != f32 or not dgate.is_contiguous() or dgate.shape != gate.shape:
                raise QLoRAError("dgate must be a contiguous float32 tensor of the gate's shape")
            dgp = dgate.data_ptr()
    for t, name in ((dw_post, "dw_post"), (dw_pre, "dw_pre")):
        if t is not None and (t.dtype != f32 or t.shape != (d,) or not t.is_contiguous()):
            raise QLoRAError(f"{name} must be a contiguous float32 [{d}] tensor")
    if workspace is None:
        workspace = torch.empty(max(16, qlora_resnorm_workspace_bytes(m, d)), dtype=torch.uint8,
                                device=dev)
    _same_device(dev, gate, w_post, w_pre, dgate, dw_post, dw_pre, workspace)
    a = _ResnormGrad(m, d, adt, _DT[res], pdt, post, pre, kind, scale, eps, w_offset, dzp, dhp, hp, yp, gp,
                     _p(w_post), _p(w_pre), lddz, lddh, ldh, ldy, ldg, dxp, dyp, dgp, lddx, lddy, lddg,
                     _p(dw_post), _p(dw_pre))
    status = lib().qlora_resnorm_bwd(a, workspace.data_ptr(), workspace.nbytes, _stream(dev))
    if status:
        _check(status, "qlora_resnorm_bwd")
    return dx, dy, dgate, dw_post, dw_pre


# ---------------------------------------------------------------------- AdamW

@dataclass
class AdamWState:
    """The moments of a plan's tensors (see qlora_opt_state in the C header): float32 [blocks x 256],
    or float8_e4m3fn / float8_e5m2 codes with float32 scales [blocks]."""
    m: torch.Tensor
    v: torch.Tensor
    m_scale: torch.Tensor | None = None
    v_scale: torch.Tensor | None = None

    def moments(self):
        """(m, v) as float32 [blocks x 256]."""
        if self.m_scale is None:
            return self.m, self.v
        return (self.m.float() * self.m_scale[:, None], self.v.float() * self.v_scale[:, None])


class AdamWPlan:
    """A prepared list of tensors; the device table lives in a tensor owned by this object, which
    also keeps the listed tensors alive."""

    def __init__(self, handle, table, keep, device):
        self.handle, self.table, self._keep, self.device = handle, table, keep, device
        self.blocks, self.state_bits = handle.blocks, handle.state_bits
        s = (self.blocks, ADAMW_BLOCK)
        self._fields = ((("m", torch.float32, s), ("v", torch.float32, s)) if self.state_bits == 32 else
                        (("m", torch.float8_e4m3fn, s), ("v", torch.float8_e5m2, s),
                         ("m_scale", torch.float32, (self.blocks,)), ("v_scale", torch.float32, (self.blocks,))))

    def new_state(self) -> AdamWState:
        """Zero moments: the state before the first step."""
        s = (self.blocks, ADAMW_BLOCK)

        def z(shape, dt):
            return torch.zeros(shape, dtype=dt, device=self.device)
        if self.state_bits == 32:
            return AdamWState(z(s, torch.float32), z(s, torch.float32))
        return AdamWState(z(s, torch.uint8).view(torch.float8_e4m3fn),
                          z(s, torch.uint8).view(torch.float8_e5m2),
                          z((self.blocks,), torch.float32), z((self.blocks,), torch.float32))

    def _state(self, st):
        ptrs = []
        for name, dt, shape in self._fields:
            t = getattr(st, name)
            if t is None or t.dtype != dt or t.shape != shape or not t.is_contiguous() or t.device != self.device:
                raise QLoRAError(f"state {name} must be a contiguous {dt} tensor of shape {shape} on {self.device}")
            ptrs.append(t.data_ptr())
        return _OptState(*ptrs)


def qlora_adamw_init(params, grads, copies=None, params_out=None, state_bits: int = 32, lr_mul=None,
                     wd_mul=None) -> AdamWPlan:
    """Plan of one step over lists of tensors: params read, params_out (default: params) written,
    copies (optional, bf16 or fp16) written too.  lr_mul, wd_mul: a number a tensor.  Setup time:
    writes the device table and synchronizes.  The plan holds the tensors and steps on their memory:
    write new gradients into the tensors given here (no new ones in their place), or make another plan."""
    n = len(params)
    outs = params_out if params_out is not None else params
    if not n or len(grads) != n or len(outs) != n or (copies is not None and len(copies) != n):
        raise QLoRAError("params, grads, params_out and copies must be lists of one length, at least 1")
    if any(k is not None and len(k) != n for k in (lr_mul, wd_mul)):
        raise QLoRAError("lr_mul and wd_mul must have a number for every tensor")
    dev = params[0].device
    for name, ts in (("params", params), ("grads", grads), ("params_out", outs), ("copies", copies or [])):
        for t, p in zip(ts, params):
            if t is None and name == "copies":
                continue
            if t.numel() != p.numel() or not t.is_contiguous() or t.device != dev:
                raise QLoRAError(f"{name} must be contiguous, of the parameters' sizes, on {dev}")
    dts = [{t.dtype for t in ts if t is not None} for ts in (params, grads, outs, copies or [])]
    if any(len(s) > 1 for s in dts) or dts[0] != dts[2]:
        raise QLoRAError("the tensors of each list must share a dtype, params_out that of params")
    arr, sizes = (_OptTensor * n)(), (_i64 * n)()
    for i in range(n):
        cp = copies[i] if copies is not None else None
        sizes[i] = params[i].numel()
        arr[i] = _OptTensor(params[i].data_ptr(), grads[i].data_ptr(), outs[i].data_ptr(),
                            cp.data_ptr() if cp is not None else None, sizes[i],
                            1.0 if lr_mul is None else lr_mul[i], 1.0 if wd_mul is None else wd_mul[i])
    nbytes = lib().qlora_adamw_table_bytes(sizes, n)
    if not nbytes:
        raise QLoRAError("qlora_adamw_table_bytes: the tensors are too many or too large")
    ct = next(iter(dts[3]), torch.bfloat16)
    if ct not in _DT:
        raise QLoRAError(f"unsupported copy dtype {ct}")
    _stream(dev)                                 # the table is of the current GPU
    table = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    # the table's memory may be one that work still waiting on this stream writes or reads, and the
    # copy into it is not ordered behind that
    torch.cuda.current_stream(dev).synchronize()
    h = _AdamW()
    _check(lib().qlora_adamw_init(h, arr, n, _dt(params[0], "params"), _dt(grads[0], "grads"), _DT[ct],
                                  state_bits, table.data_ptr(), nbytes), "qlora_adamw_init")
    return AdamWPlan(h, table, (list(params), list(grads), list(outs), list(copies or [])), dev)


def qlora_grad_norm_workspace_bytes(plan: AdamWPlan) -> int:
    return int(lib().qlora_grad_norm_workspace_bytes(plan.handle))


def qlora_grad_norm(plan: AdamWPlan, max_norm: float = 0.0, out=None, workspace=None) -> torch.Tensor:
    """-> float32 [2] on the device: the norm of all gradients, and the factor that brings it to
    max_norm (pass out[1:] to qlora_adamw_step as grad_scale).  Calls on one plan must not overlap on
    the device: on different streams, let one wait for the other."""
    if out is None:
        out = torch.empty(2, dtype=torch.float32, device=plan.device)
    if workspace is None:
        workspace = torch.empty(qlora_grad_norm_workspace_bytes(plan), dtype=torch.uint8,
                                device=plan.device)
    _same_device(plan.device, out, workspace)
    _vec(out, 2, (torch.float32,), "out")
    _check(lib().qlora_grad_norm(plan.handle, max_norm, out.data_ptr(), workspace.data_ptr(),
                                 workspace.nbytes, _stream(plan.device)),
           "qlora_grad_norm")
    return out


def qlora_adamw_step(plan: AdamWPlan, state: AdamWState, step: int, lr: float, betas=(0.9, 0.999),
                     eps: float = 1e-8, weight_decay: float = 0.0, grad_scale=None, seed: int = 0,
                     state_out=None) -> None:
    """One step (step counts from 1) over the plan's tensors; moments from `state` to `state_out`
    (default: in place).  grad_scale: a one-element float32 device tensor multiplying the gradients; a value
    that is not finite skips the step.  A captured step repeats its step count and settings on every replay."""
    s = plan._state(state)
    o = s if state_out is None or state_out is state else plan._state(state_out)
    gs = None
    if grad_scale is not None:
        if grad_scale.dtype != torch.float32 or grad_scale.numel() != 1 or grad_scale.device != plan.device:
            raise QLoRAError(f"grad_scale must be one float32 value on {plan.device}")
        gs = grad_scale.data_ptr()
    h = _Hyper(step, lr, betas[0], betas[1], eps, weight_decay, seed & 0xFFFFFFFF)
    _check(lib().qlora_adamw_step(plan.handle, s, o, h, gs, _stream(plan.device)), "qlora_adamw_step")
