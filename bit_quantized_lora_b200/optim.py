"""AdamW over many tensors in one launch: the optimizer step of the adapters
(and of any other bf16 or float32 parameters), with moments in float32 or in
8 bits.

    opt = AdamW(params, grads, lr=1e-4, state_bits=8)
    opt.step()                                   # reads grads, updates params
"""
from __future__ import annotations

import ctypes
import struct

import numpy as np
import torch

from ._lib import FtAdamwTensor, check, load, load_torch
from .blockops import _on_device

_DTYPE = {torch.bfloat16: 0, torch.float32: 1}
_raw_stream = torch._C._cuda_getCurrentRawStream
BLOCK = 256  # consecutive values that share a scale of an 8-bit state
_RECORD = np.dtype([("p", "u8"), ("p16", "u8"), ("grad", "u8"), ("m", "u8"), ("v", "u8"), ("m_scale", "u8"),
                    ("v_scale", "u8"), ("n", "i8"), ("weight_decay", "f4"), ("gt", "i4")])
_HYPER = struct.Struct("@4d")  # ft_adamw_hyper
assert _RECORD.itemsize == ctypes.sizeof(FtAdamwTensor)


def _f32(t, name: str, n: int, dev: int):
    if t is None:
        return None
    if t.dtype is not torch.float32 or t.numel() < n or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous float32 tensor of {n}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the call is on cuda:{dev}")
    return t.data_ptr()


@_on_device(0)
def ft_adamw_decode(codes: torch.Tensor, scales: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """The float32 values that 8-bit moments stand for: codes int8 (first
    moments) or uint8 (second moments), scales float32, one per 256."""
    if codes.dtype not in (torch.int8, torch.uint8) or not codes.is_contiguous():
        raise TypeError("codes must be a contiguous int8 or uint8 tensor")
    n = codes.numel()
    out = torch.empty(codes.shape, dtype=torch.float32, device=codes.device) if out is None else out
    dev = codes.get_device()
    check("ft_adamw_decode", load().ft_adamw_decode(
        codes.data_ptr(), _f32(scales, "scales", -(-n // BLOCK), dev), n, int(codes.dtype == torch.uint8),
        _f32(out, "out", n, dev), _raw_stream(dev)))
    return out


def _check_params(params, dev, dtypes=None, sizes=None) -> None:
    """What a launch takes for granted of the parameters: where they lie, that
    no two share memory, and (once chosen) their types and sizes."""
    for i, p in enumerate(params):
        if not p.is_cuda or p.dtype not in _DTYPE:
            raise TypeError("parameters must be CUDA bfloat16 or float32 tensors")
        if not p.is_contiguous() or p.device != dev:
            raise ValueError("parameters must be contiguous and on one device")
        if dtypes is not None and (p.dtype != dtypes[i] or p.numel() != sizes[i]):
            raise ValueError("a parameter has another type or size than the optimizer was made for")
    used = sorted((p.data_ptr(), p.nbytes) for p in params if p.numel())
    for (a, n), (b, _) in zip(used, used[1:]):
        if a == b:
            raise ValueError("a parameter is listed twice")
        if a + n > b:
            raise ValueError("two parameters share memory")


class AdamW:
    """AdamW on `params`, contiguous bf16 or float32 tensors of one device.

    grads: tensors of the same shapes (bf16 or float32) that step() reads
    every time (a training loop's gradient buffers), unless it is given
    others.  weight_decay: one for all, or one per parameter.  state_bits: 32
    or 8.  master: bf16 parameters are stepped in float32 (`master`) and
    rounded once into the parameter; with master=False they are stepped in
    place.  The state is flat, every parameter's part starting at a multiple
    of 256: master, exp_avg, exp_avg_sq (codes with 8-bit states) and
    exp_avg_scale, exp_avg_sq_scale; step_count is on the device, so a
    captured step counts when it is replayed.  The state's tensors stay the
    optimizer's own (a step holds their addresses): values are exchanged with
    state_dict() and load_state_dict(), and the object is not copied."""

    def __init__(self, params, grads=None, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay=0.01, state_bits: int = 32, master: bool = True):
        self.params = list(params)
        if not self.params:
            raise ValueError("AdamW needs parameters")
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        if not (0.0 <= betas[0] < 1.0 and 0.0 <= betas[1] < 1.0 and eps >= 0.0):
            raise ValueError("betas must lie in [0, 1) and eps must not be negative")
        dev = self.params[0].device
        _check_params(self.params, dev)
        self._dtypes, self._sizes = [p.dtype for p in self.params], [p.numel() for p in self.params]
        self.lr, self.betas, self.eps, self.state_bits = lr, tuple(betas), eps, state_bits
        decay = [float(weight_decay)] * len(self.params) if np.isscalar(weight_decay) else list(weight_decay)
        if len(decay) != len(self.params):
            raise ValueError("one weight_decay, or one per parameter")
        blocks = [-(-p.numel() // BLOCK) for p in self.params]
        starts = np.cumsum([0] + blocks)[:-1]
        total = sum(blocks) * BLOCK
        st = [torch.int8, torch.uint8] if state_bits == 8 else [torch.float32, torch.float32]
        self.exp_avg = torch.zeros(total, dtype=st[0], device=dev)
        self.exp_avg_sq = torch.zeros(total, dtype=st[1], device=dev)
        self.exp_avg_scale = self.exp_avg_sq_scale = None
        if state_bits == 8:
            self.exp_avg_scale = torch.zeros(sum(blocks), device=dev)
            self.exp_avg_sq_scale = torch.zeros(sum(blocks), device=dev)
        self.master = None
        has_master = [master and p.dtype == torch.bfloat16 for p in self.params]
        if any(has_master):
            self.master = torch.zeros(total, device=dev)
            for p, s, own in zip(self.params, starts, has_master):
                if own:
                    self.master[s * BLOCK:s * BLOCK + p.numel()].copy_(p.detach().reshape(-1))
        self._step = torch.zeros(2, dtype=torch.int64, device=dev)
        self.step_count = self._step[:1]
        # the tensors' records; a step looks whether a caller has exchanged one (its memory, type, sizes or strides),
        # checks it as at first and writes the new addresses
        self._starts = starts.astype(np.uint64) * np.uint64(BLOCK)
        self._has_master = np.array(has_master)
        self._is16 = np.array([p.dtype == torch.bfloat16 for p in self.params])
        self._rec = np.zeros(len(self.params), _RECORD)
        self._rec["n"] = [p.numel() for p in self.params]
        self._rec["weight_decay"] = decay
        self._rec_addr = self._rec.ctypes.data
        self._bind()
        self._bind_params(load_torch().layout_of(self.params))
        self._lent, self._seen_grads = True, None  # the records hold no gradients of the optimizer's own yet
        self.grads = None if grads is None else self._checked(grads)

    def _checked(self, grads) -> list:
        grads = list(grads)
        if len(grads) != len(self.params):
            raise ValueError(f"{len(grads)} gradients for {len(self.params)} parameters")
        for g, p in zip(grads, self.params):
            if g.dtype not in _DTYPE:
                raise TypeError("gradients must be bfloat16 or float32")
            if g.shape != p.shape or not g.is_contiguous() or g.device != p.device:
                raise ValueError("a gradient must be contiguous, of its parameter's shape and on its device")
        self._rec["gt"] = [_DTYPE[g.dtype] for g in grads]
        return grads

    def step(self, grads=None, lr=None, grad_scale: torch.Tensor | None = None, stream=None) -> None:
        """One step from `grads` (or the optimizer's own).  lr: a float, or a
        float32 device scalar (a captured step whose rate changes), in place
        of the optimizer's.  grad_scale: a float32 device scalar that
        multiplies the gradients (1 / ranks, a clipping factor)."""
        layout = load_torch().layout_of
        if grads is not None:
            self._lend(grads)
        elif self.grads is None:
            raise ValueError("step() needs gradients")
        else:
            seen = layout(self.grads)
            if self._lent or seen != self._seen_grads:  # the last step read others, or a caller exchanged one
                self._lend(self.grads)
                self._seen_grads, self._lent = seen, False
        held = self._held
        if not (held[0] is self.master and held[1] is self.exp_avg and held[2] is self.exp_avg_sq and
                held[3] is self.exp_avg_scale and held[4] is self.exp_avg_sq_scale):
            raise ValueError("the state's tensors are the optimizer's own: load_state_dict() exchanges their values")
        seen = layout(self.params)
        if seen != self._seen:  # a caller has given a parameter other memory, or another view of its own
            _check_params(self.params, self._step.device, self._dtypes, self._sizes)
            self._bind_params(seen)
        self._launch(self._step, self.lr if lr is None else lr, grad_scale, stream=stream)

    def _lend(self, grads) -> None:
        """The gradients' addresses in the tensors' records."""
        self._lent = True
        self._rec["grad"] = [t.data_ptr() for t in self._checked(grads)]

    def _bind_params(self, seen: bytes) -> None:
        """The parameters' addresses in the tensors' records; seen: their layout."""
        rec, own = self._rec, np.array([p.data_ptr() for p in self.params], np.uint64)
        rec["p16"] = np.where(self._is16, own, 0)
        rec["p"] = np.where(self._has_master, self._master_ptrs, np.where(self._is16, 0, own))
        self._seen = seen

    def _bind(self) -> None:
        """The state's addresses in the tensors' records."""
        rec, at = self._rec, self._starts
        self._master_ptrs = at * np.uint64(4) + np.uint64(0 if self.master is None else self.master.data_ptr())
        size = np.uint64(4 if self.state_bits == 32 else 1)
        rec["m"] = at * size + np.uint64(self.exp_avg.data_ptr())
        rec["v"] = at * size + np.uint64(self.exp_avg_sq.data_ptr())
        if self.state_bits == 8:
            scale_at = at // np.uint64(BLOCK) * np.uint64(4)
            rec["m_scale"] = scale_at + np.uint64(self.exp_avg_scale.data_ptr())
            rec["v_scale"] = scale_at + np.uint64(self.exp_avg_sq_scale.data_ptr())
        self._held = self._state()

    def _state(self) -> tuple:
        return (self.master, self.exp_avg, self.exp_avg_sq, self.exp_avg_scale, self.exp_avg_sq_scale)

    def __reduce_ex__(self, protocol):
        # copies and pickles would carry this object's addresses
        raise TypeError("an AdamW is not copied: make another and load its state_dict()")

    def _launch_here(self, step, lr, grad_scale) -> None:
        dev = step.get_device()
        lr_dev = lr if isinstance(lr, torch.Tensor) else None
        h = _HYPER.pack(0.0 if lr_dev is not None else lr, *self.betas, self.eps)
        check("ft_adamw_step", load().ft_adamw_step(
            self._rec_addr, len(self._rec), h, self.state_bits, step.data_ptr(), _f32(lr_dev, "lr", 1, dev),
            _f32(grad_scale, "grad_scale", 1, dev), _raw_stream(dev)))

    _launch = _on_device(1)(_launch_here)

    def state_values(self):
        """(first, second) moments as flat float32 tensors: the state itself
        with 32-bit states, decoded with 8-bit ones."""
        if self.state_bits == 32:
            return self.exp_avg, self.exp_avg_sq
        return (ft_adamw_decode(self.exp_avg, self.exp_avg_scale),
                ft_adamw_decode(self.exp_avg_sq, self.exp_avg_sq_scale))

    _STATE = ("master", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale", "step_count")

    def state_dict(self) -> dict:
        """Copies of the state, to be saved and loaded again."""
        return {k: None if getattr(self, k) is None else getattr(self, k).clone() for k in self._STATE}

    def load_state_dict(self, state: dict) -> None:
        for k in self._STATE:
            mine, theirs = getattr(self, k), state[k]
            if (mine is None) != (theirs is None) or (mine is not None and (
                    mine.shape != theirs.shape or mine.dtype != theirs.dtype)):
                raise ValueError(f"{k} is not of this optimizer's layout")
        for k in self._STATE:
            if state[k] is not None:
                getattr(self, k).copy_(state[k])
