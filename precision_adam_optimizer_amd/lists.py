"""Binding of the list operators (C ABI in ``include/fp8adam_list.h``): AdamW
over mixed tensor lists with moments in 32 or 8 bits, clipping of gradients to a
global norm, and conversion of a list to FP8 with scales and back.

As in the rest of the package, the functions carry the C names and only marshal
arguments, the classes hold the tensors and the plan, and there is no fallback.
"""
from __future__ import annotations

import ctypes

import torch

from . import (_FORMATS, _GRAN, _SMODE, AMP_STATE_DTYPE, BLOCK, AmpConfigArg, SCALE_BLOCK128, _check, _ptr,
               current_stream, load)

F32, BF16, F16 = 0, 1, 2
MOMENTS_32, MOMENTS_8 = 0, 1
MAX_GROUPS = 32
_DTYPES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
_MOMENTS = {32: MOMENTS_32, 8: MOMENTS_8}

LIST_EXPORTS = ("fp8adam_plan_destroy", "fp8adam_adamw_plan", "fp8adam_adamw_step", "fp8adam_adamw_step_amp",
                "fp8adam_clip_plan", "fp8adam_clip_grads", "fp8adam_quant_plan", "fp8adam_quantize",
                "fp8adam_dequantize")


class AdamwTensorArg(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("copy", ctypes.c_void_p),
                ("m", ctypes.c_void_p), ("v", ctypes.c_void_p), ("m_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("numel", ctypes.c_int64), ("param_dtype", ctypes.c_int32),
                ("grad_dtype", ctypes.c_int32), ("copy_dtype", ctypes.c_int32), ("moments", ctypes.c_int32),
                ("group", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class AdamwConfigArg(ctypes.Structure):
    _fields_ = [("n_groups", ctypes.c_int32), ("m_format", ctypes.c_int32), ("v_format", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class AdamwHParamsArg(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double)]


class ClipTensorArg(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("src_dtype", ctypes.c_int32), ("dst_dtype", ctypes.c_int32)]


class QuantTensorArg(ctypes.Structure):
    _fields_ = [("values", ctypes.c_void_p), ("codes", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("numel", ctypes.c_int64), ("dtype", ctypes.c_int32), ("format", ctypes.c_int32)]


class QuantConfigArg(ctypes.Structure):
    _fields_ = [("granularity", ctypes.c_int32), ("scale_mode", ctypes.c_int32)]


_ready = None


def _lib() -> ctypes.CDLL:
    """The library with this header's signatures declared."""
    global _ready
    if _ready is None:
        L = load()
        vp, i32, i64, P = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.POINTER
        L.fp8adam_plan_destroy.argtypes = [vp]
        L.fp8adam_plan_destroy.restype = None
        L.fp8adam_adamw_plan.argtypes = [P(vp), P(AdamwTensorArg), i32, P(AdamwConfigArg), vp]
        # the host structs by address, which the classes below keep: a pointer made for each call costs a small step 0.5 us
        L.fp8adam_adamw_step.argtypes = [vp, vp, i32, i64, vp]
        L.fp8adam_adamw_step_amp.argtypes = [vp, vp, i32, vp, vp, vp]
        L.fp8adam_clip_plan.argtypes = [P(vp), P(ClipTensorArg), i32, vp]
        L.fp8adam_clip_grads.argtypes = [vp, ctypes.c_float, vp, vp]
        L.fp8adam_quant_plan.argtypes = [P(vp), P(QuantTensorArg), i32, P(QuantConfigArg), vp]
        L.fp8adam_quantize.argtypes = [vp, vp]
        L.fp8adam_dequantize.argtypes = [vp, vp]
        for name in LIST_EXPORTS[1:]:
            getattr(L, name).restype = ctypes.c_int
        _ready = L
    return _ready


# ---------------------------------------------------------------- C names

def _plan(fn, *args) -> int:
    h = ctypes.c_void_p()
    _check(fn(ctypes.byref(h), *args))
    return h.value


def fp8adam_plan_destroy(plan: int) -> None:
    _lib().fp8adam_plan_destroy(plan)


def fp8adam_adamw_plan(tensors: list[AdamwTensorArg], cfg: AdamwConfigArg, stream: int | None = None) -> int:
    arr = (AdamwTensorArg * len(tensors))(*tensors)
    return _plan(_lib().fp8adam_adamw_plan, arr, len(tensors), ctypes.byref(cfg),
                 current_stream() if stream is None else stream)


def fp8adam_adamw_step(plan: int, groups: list[AdamwHParamsArg], step: int, stream: int | None = None) -> None:
    arr = (AdamwHParamsArg * len(groups))(*groups)
    _check(_lib().fp8adam_adamw_step(plan, arr, len(groups), step, current_stream() if stream is None else stream))


def fp8adam_adamw_step_amp(plan: int, groups: list[AdamwHParamsArg], amp: AmpConfigArg, state: int,
                           stream: int | None = None) -> None:
    arr = (AdamwHParamsArg * len(groups))(*groups)
    _check(_lib().fp8adam_adamw_step_amp(plan, arr, len(groups), ctypes.byref(amp), state,
                                         current_stream() if stream is None else stream))


def fp8adam_clip_plan(tensors: list[ClipTensorArg], stream: int | None = None) -> int:
    arr = (ClipTensorArg * len(tensors))(*tensors)
    return _plan(_lib().fp8adam_clip_plan, arr, len(tensors), current_stream() if stream is None else stream)


def fp8adam_clip_grads(plan: int, max_norm: float, result: torch.Tensor, stream: int | None = None) -> None:
    assert result.dtype == torch.float32 and result.numel() == 2 and result.is_contiguous()
    _check(_lib().fp8adam_clip_grads(plan, max_norm, _ptr(result), current_stream() if stream is None else stream))


def fp8adam_quant_plan(tensors: list[QuantTensorArg], cfg: QuantConfigArg, stream: int | None = None) -> int:
    arr = (QuantTensorArg * len(tensors))(*tensors)
    return _plan(_lib().fp8adam_quant_plan, arr, len(tensors), ctypes.byref(cfg),
                 current_stream() if stream is None else stream)


def fp8adam_quantize(plan: int, stream: int | None = None) -> None:
    _check(_lib().fp8adam_quantize(plan, current_stream() if stream is None else stream))


def fp8adam_dequantize(plan: int, stream: int | None = None) -> None:
    _check(_lib().fp8adam_dequantize(plan, current_stream() if stream is None else stream))


# ------------------------------------------------------------ torch wrappers

def _order(t: torch.Tensor) -> list:
    """(stride, size) of the dimensions that move, innermost first."""
    return sorted((st, n) for st, n in zip(t.stride(), t.shape) if n != 1)


def _dense(t: torch.Tensor) -> bool:
    """Whether the elements fill one run of memory, in whatever order of the dimensions."""
    if t.is_contiguous():
        return True
    at = 1
    for st, n in _order(t):
        if st != at:
            return False
        at *= n
    return True


def _same_order(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether element by element in memory a and b are the same elements (both dense)."""
    if a.numel() != b.numel():
        return False
    if a.is_contiguous() and b.is_contiguous():
        return True
    return a.shape == b.shape and all(x == y for x, y, n in zip(a.stride(), b.stride(), a.shape) if n != 1)


def _need(ok: bool, i: int, what: str) -> None:
    if not ok:
        raise ValueError(f"tensor {i}: {what}")


def _check_flat(t: torch.Tensor, i: int, what: str, dtype, numel: int, at_least: bool = False) -> None:
    _need(t.dtype == dtype, i, f"{what} must be {str(dtype).replace('torch.', '')}")
    _need(t.numel() == numel or (at_least and t.numel() > numel), i,
          f"{what} must have {'at least ' if at_least else ''}{numel} elements")
    _need(t.is_contiguous(), i, f"{what} must be contiguous")


def _one_gpu(tensors) -> torch.device:
    dev = tensors[0].device
    if any(t.device != dev for t in tensors):
        raise ValueError("every tensor must be on one device")
    if dev.type != "cuda":
        raise ValueError("the tensors must be on a GPU")
    return dev


def _blocks(numel: int) -> int:
    return -(-numel // BLOCK)


def _capturing(device: torch.device) -> bool:
    with torch.cuda.device(device):
        return torch.cuda.is_current_stream_capturing()


_kept: list = []  # objects that were dropped while a graph was captured, with their plans


class _Planned:
    """A plan on its device: calls go to the device's current stream."""
    _plan = None

    def _check_capture(self, tensors) -> None:
        """Before anything is allocated for a plan over these tensors."""
        t = next((t for t in tensors if t.is_cuda), None)
        if t is not None and _capturing(t.device):
            raise RuntimeError("plans cannot be built while a graph is captured: build them before")

    def _build(self, device: torch.device, make) -> None:
        while _kept:
            _kept.pop().close()
        self.device = device
        self._index = device.index
        with torch.cuda.device(device):
            self._plan = make()

    def _call(self, fn, *args) -> None:
        """fn(plan, *args, stream) with the plan's device current."""
        if self._plan is None:
            raise RuntimeError("the plan is closed")
        if torch.cuda.current_device() == self._index:
            rc = fn(self._plan, *args, torch._C._cuda_getCurrentRawStream(self._index))
        else:
            with torch.cuda.device(self._index):
                rc = fn(self._plan, *args, torch._C._cuda_getCurrentRawStream(self._index))
        if rc:
            _check(rc)

    def close(self) -> None:
        """Waits for the device and frees the plan; no graph that captured one of its calls may be
        replayed afterwards."""
        if self._plan:
            if _capturing(self.device):
                raise RuntimeError("a plan cannot be closed while a graph is captured")
            torch.cuda.synchronize(self.device)
            with torch.cuda.device(self.device):
                fp8adam_plan_destroy(self._plan)
            self._plan = None

    def __del__(self):
        try:
            if self._plan and _capturing(self.device):
                _kept.append(self)  # waiting for the device would end the capture: the next plan frees this one
            else:
                self.close()
        except Exception:
            pass


class AdamW(_Planned):
    """AdamW over lists of torch tensors on one GPU, one launch for each kind of
    tensor in the list.

    params: weights in fp32, bf16 or fp16, updated in place; grads: fp32, bf16 or
    fp16 gradients, one for each weight; both may differ from tensor to tensor.
    A weight and its gradient lie in memory in the same order and without gaps
    (contiguous, or both transposed the same way); any alignment will do.
    ``state_bits``: 32 (two fp32 moments) or 8 (FP8 codes in ``m_format`` and
    ``v_format`` with one power-of-two scale per 128 elements each, the state of
    ``FP8AdamW(granularity="block128")``), for the list or a sequence with one for
    each tensor.  ``copies``: for fp32 weights, bf16 or fp16 tensors (or None) that
    every step writes the new weights into as well.  ``groups``: each tensor's
    parameter group, 0 .. n_groups - 1; lr, betas, eps and weight_decay are then
    numbers for all groups, or lists or tuples with one for each.  ``state``: the moments
    to start from, as ``checkpoint()`` and ``converted_state()`` return them ((m, v),
    or (m, v, m_scale, v_scale) with None where moments have 32 bits); fresh ones
    otherwise.  The tensors must stay alive with the same storage while this
    object exists, and none that a step writes may overlap another.

    Steps may be captured into a graph (of this class and of ``GradClip`` and
    ``Quantizer``; the object must outlive it).  A replay takes what is not a
    tensor as it was at the capture: the hyperparameters, ``max_norm`` and ``step``.
    Training by replays therefore takes ``step_amp``, which counts t on the device.
    """

    def __init__(self, params, grads, *, state_bits=32, copies=None, groups=None, n_groups=None, m_format="e4m3",
                 v_format="e5m2", state=None):
        params, grads = list(params), list(grads)
        n = len(params)
        if len(grads) != n or not params:
            raise ValueError("need one gradient per parameter and at least one parameter")
        copies = [None] * n if copies is None else list(copies)
        groups = [0] * n if groups is None else [int(q) for q in groups]
        bits = [state_bits] * n if isinstance(state_bits, int) else list(state_bits)
        if not len(copies) == len(groups) == len(bits) == n:
            raise ValueError("copies, groups and state_bits need one entry per parameter")
        if any(b not in _MOMENTS for b in bits):
            raise ValueError("state_bits must be 32 or 8")
        self._check_capture(params)
        self.n_groups = int(n_groups) if n_groups is not None else max(groups) + 1
        if not 1 <= self.n_groups <= MAX_GROUPS or any(not 0 <= q < self.n_groups for q in groups):
            raise ValueError(f"groups must lie in 0 .. n_groups - 1, with n_groups at most {MAX_GROUPS}")
        for i, (p, g, c) in enumerate(zip(params, grads, copies)):
            _need(p.dtype in _DTYPES, i, "weights must be float32, bfloat16 or float16")
            _need(g.dtype in _DTYPES, i, "gradients must be float32, bfloat16 or float16")
            _need(_dense(p) and _dense(g), i, "weights and gradients must be dense")
            _need(_same_order(p, g), i, "the gradient must have its weight's size and order in memory")
            if c is not None:
                _need(p.dtype == torch.float32 and c.dtype in (torch.bfloat16, torch.float16), i,
                      "a copy must be bfloat16 or float16, of float32 weights")
                _need(_dense(c) and _same_order(p, c), i, "the copy must have its weight's size and order in memory")
        if state is None:
            def zeros(p, b):
                return torch.zeros_like(p, dtype=torch.float32) if b == 32 else p.new_zeros(p.numel(), dtype=torch.uint8)

            def ones(p, b):
                return None if b == 32 else p.new_ones(max(1, _blocks(p.numel())), dtype=torch.float32)
            state = [[zeros(p, b) for p, b in zip(params, bits)] for _ in range(2)]
            state += [[ones(p, b) for p, b in zip(params, bits)] for _ in range(2)]
        state = [list(x) for x in state]
        if len(state) == 2:
            state += [[None] * n, [None] * n]
        if len(state) != 4 or any(len(x) != n for x in state):
            raise ValueError("state must be (m, v) or (m, v, m_scale, v_scale) with one entry per parameter")
        self.m, self.v, self.m_scale, self.v_scale = state
        for i, (p, b) in enumerate(zip(params, bits)):
            for what, t, s in (("m", self.m[i], self.m_scale[i]), ("v", self.v[i], self.v_scale[i])):
                if b == 32:
                    _need(t.dtype == torch.float32 and _dense(t) and (_same_order(p, t) or (
                        t.is_contiguous() and t.dim() == 1 and t.numel() == p.numel())), i,
                          f"32-bit moments ({what}) must be float32 of the weight's size and order in memory")
                else:
                    _check_flat(t, i, f"8-bit moments ({what})", torch.uint8, p.numel())
                    _need(s is not None, i, f"8-bit moments ({what}) need scales")
                    _check_flat(s, i, f"scales of 8-bit moments ({what})", torch.float32, _blocks(p.numel()), True)
        dev = _one_gpu([t for x in (params, grads, copies, *state) for t in x if t is not None])
        self.params, self.grads, self.copies, self.groups, self.state_bits = params, grads, copies, groups, bits
        args = [AdamwTensorArg(_ptr(p), _ptr(g), _ptr(c), _ptr(m), _ptr(v), _ptr(ms) if b == 8 else None,
                               _ptr(vs) if b == 8 else None, p.numel(), _DTYPES[p.dtype], _DTYPES[g.dtype],
                               0 if c is None else _DTYPES[c.dtype], _MOMENTS[b], q, 0)
                for p, g, c, m, v, ms, vs, b, q in zip(params, grads, copies, *state, bits, groups)]
        self.formats = (m_format, v_format)
        cfg = AdamwConfigArg(self.n_groups, _FORMATS[m_format], _FORMATS[v_format], 0)
        self._hp = (AdamwHParamsArg * self.n_groups)()
        self._hp_at = ctypes.addressof(self._hp)
        self._given = None
        self._amp = AmpConfigArg()
        self._amp_at = ctypes.addressof(self._amp)
        self._build(dev, lambda: fp8adam_adamw_plan(args, cfg))

    def _set(self, lr, beta1, beta2, eps, weight_decay) -> None:
        """The groups' hyperparameters into the array that the calls pass (left as it is where
        they are those of the call before)."""
        given = (lr, beta1, beta2, eps, weight_decay)
        if given == self._given:
            return
        self._given = None
        for name, x in zip(("lr", "beta1", "beta2", "eps", "weight_decay"), given):
            if isinstance(x, (list, tuple)):
                if len(x) != self.n_groups:
                    raise ValueError(f"{name} must be a number or one for each of the {self.n_groups} groups")
                for h, y in zip(self._hp, x):
                    setattr(h, name, y)
            else:
                for h in self._hp:
                    setattr(h, name, x)
        flat = [y for x in given for y in (x if type(x) is tuple else (x,))]
        if all(type(y) in (float, int) for y in flat):  # (a list or a tensor could change in place)
            self._given = given

    def step(self, *, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step: int) -> None:
        """One step; ``step`` is the 1-based t of the bias corrections."""
        self._set(lr, beta1, beta2, eps, weight_decay)
        self._call(_lib().fp8adam_adamw_step, self._hp_at, self.n_groups, step)

    def step_amp(self, amp_state: torch.Tensor, *, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0,
                 max_norm: float = 0.0, growth_factor: float = 2.0, backoff_factor: float = 0.5,
                 growth_interval: int = 2000) -> None:
        """A step on gradients of (loss * scale), as ``FP8AdamW.step_amp``: unscale, skip on
        Inf/NaN, clip the global norm to max_norm (if > 0), all on the device.  t is the
        state's count of taken steps (``amp_state()`` starts it at 0).  For gradients that are not
        scaled: a state of scale 1 and growth_interval=2**31 - 1; a skipped step still lowers the scale."""
        if amp_state.dtype != torch.uint8 or amp_state.numel() != AMP_STATE_DTYPE.itemsize:
            raise ValueError("amp_state must be the 32-byte tensor from amp_state()")
        if amp_state.device != self.device or not amp_state.is_contiguous():
            raise ValueError("amp_state must be contiguous and on the weights' device")
        self._set(lr, beta1, beta2, eps, weight_decay)
        a = self._amp
        a.max_norm, a.growth_factor, a.backoff_factor, a.growth_interval = (max_norm, growth_factor, backoff_factor,
                                                                            growth_interval)
        self._call(_lib().fp8adam_adamw_step_amp, self._hp_at, self.n_groups, self._amp_at, amp_state.data_ptr())

    def checkpoint(self) -> list:
        """Copies of the moments in the form ``state=`` takes: [m, v, m_scale, v_scale].
        Together with the weights it resumes bit for bit."""
        with torch.cuda.device(self.device):
            return [[None if t is None else t.clone() for t in x] for x in (self.m, self.v, self.m_scale, self.v_scale)]

    def converted_state(self, state_bits: int, granularity: str = "block128") -> list:
        """The moments in 32 or 8 bits, as new tensors in the form ``state=`` takes: to go on
        with another kind of state.  8 bits with ``granularity="block128"`` suit ``AdamW`` and
        ``FP8AdamW(granularity="block128")``, with ``"tensor"`` FP8AdamW's per-tensor state
        (32-bit moments only)."""
        if state_bits not in _MOMENTS:
            raise ValueError("state_bits must be 32 or 8")
        if granularity == "tensor" and (state_bits != 8 or any(b != 32 for b in self.state_bits)):
            raise ValueError("per-tensor scales are for 32-bit moments going to 8 bits")
        self._check_capture(self.params)
        out = self.checkpoint()
        for k, fmt in enumerate(self.formats):
            idx = [i for i, b in enumerate(self.state_bits) if b != state_bits]
            if not idx:
                continue
            if state_bits == 8:
                q = Quantizer([out[k][i] for i in idx], fmt=fmt, granularity=granularity)
                q.quantize()
            else:
                q = Quantizer([torch.empty_like(self.params[i], dtype=torch.float32) for i in idx], fmt=fmt,
                              codes=[out[k][i] for i in idx], scales=[out[2 + k][i] for i in idx])
                q.dequantize()
            for j, i in enumerate(idx):
                out[k][i], out[2 + k][i] = (q.codes[j], q.scales[j]) if state_bits == 8 else (q.values[j], None)
            q.close()
        return out


class GradClip(_Planned):
    """Clips a list of gradients on one GPU to a global norm, without waiting for it.

    grads: fp32, bf16 or fp16.  ``outs``: None to clip in place, or one entry for each
    gradient: a tensor of any of the three types that takes the clipped gradient, or
    None where the gradient only counts in the norm.  Entries lie in memory in their
    gradient's order, without gaps, at any alignment, and overlap nothing.
    """

    def __init__(self, grads, outs=None):
        grads = list(grads)
        outs = list(grads) if outs is None else list(outs)
        if len(outs) != len(grads) or not grads:
            raise ValueError("need at least one gradient, and one entry of outs per gradient")
        for i, (g, o) in enumerate(zip(grads, outs)):
            _need(g.dtype in _DTYPES and (o is None or o.dtype in _DTYPES), i, "must be float32, bfloat16 or float16")
            _need(_dense(g) and (o is None or _dense(o)), i, "must be dense")
            _need(o is None or _same_order(g, o), i, "the output must have its gradient's size and order in memory")
        self._check_capture(grads)
        dev = _one_gpu([t for x in (grads, outs) for t in x if t is not None])
        self.grads, self.outs = grads, outs
        args = [ClipTensorArg(_ptr(g), _ptr(o), g.numel(), _DTYPES[g.dtype], 0 if o is None else _DTYPES[o.dtype])
                for g, o in zip(grads, outs)]
        self.result = torch.zeros(2, dtype=torch.float32, device=dev)
        self._result_at = self.result.data_ptr()
        self._build(dev, lambda: fp8adam_clip_plan(args))

    def clip(self, max_norm: float) -> torch.Tensor:
        """Clips to max_norm (0 or less: no limit) and returns (norm, coefficient): a tensor on the
        device that the next call overwrites."""
        self._call(_lib().fp8adam_clip_grads, max_norm, self._result_at)
        return self.result


class Quantizer(_Planned):
    """A list of tensors on one GPU in 8 bits with scales, and back.

    values: fp32, bf16 or fp16, dense in any order (a tensor's blocks run over its
    memory).  ``fmt``: "e4m3" or "e5m2", for the list or one for each tensor.
    ``granularity``: one scale per 128 elements ("block128") or per tensor ("tensor");
    ``scale_mode`` "pow2" or "amax", as for the step.  ``codes`` (uint8, one per element)
    and ``scales`` (float32, at least ceil(numel / 128) or 1 each) are allocated unless given.
    """

    def __init__(self, values, *, fmt="e4m3", granularity="block128", scale_mode="pow2", codes=None, scales=None):
        values = list(values)
        if not values:
            raise ValueError("need at least one tensor")
        n = len(values)
        self._check_capture(values)
        fmts = [fmt] * n if isinstance(fmt, str) else list(fmt)
        block = _GRAN[granularity] == SCALE_BLOCK128

        def count(x):
            return _blocks(x.numel()) if block else 1
        if codes is None:
            codes = [x.new_empty(x.numel(), dtype=torch.uint8) for x in values]
        if scales is None:
            # (one, unused, for an empty tensor too, as in FP8AdamW's state)
            scales = [x.new_ones(max(1, count(x)), dtype=torch.float32) for x in values]
        codes, scales = list(codes), list(scales)
        if not len(fmts) == len(codes) == len(scales) == n:
            raise ValueError("fmt, codes and scales need one entry per tensor")
        for i, (x, c, s) in enumerate(zip(values, codes, scales)):
            _need(x.dtype in _DTYPES, i, "values must be float32, bfloat16 or float16")
            _need(_dense(x), i, "values must be dense")
            _check_flat(c, i, "codes", torch.uint8, x.numel())
            _check_flat(s, i, "scales", torch.float32, count(x), True)
        dev = _one_gpu(values + codes + scales)
        self.values, self.codes, self.scales = values, codes, scales
        self.formats, self.granularity, self.scale_mode = fmts, granularity, scale_mode
        args = [QuantTensorArg(_ptr(x), _ptr(c), _ptr(s), x.numel(), _DTYPES[x.dtype], _FORMATS[f])
                for x, c, s, f in zip(values, codes, scales, fmts)]
        cfg = QuantConfigArg(_GRAN[granularity], _SMODE[scale_mode])
        self._build(dev, lambda: fp8adam_quant_plan(args, cfg))

    def quantize(self) -> None:
        """values -> codes and scales"""
        self._call(_lib().fp8adam_quantize)

    def dequantize(self) -> None:
        """codes and scales -> values"""
        self._call(_lib().fp8adam_dequantize)
