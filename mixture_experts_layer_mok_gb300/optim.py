"""AdamW over a model's tensors, with 32-bit or MXFP8 states (argument
marshalling only: the step is libmok's ``mok_adamw_step``)."""
from __future__ import annotations

import ctypes as C
import math
from operator import attrgetter

import numpy as np
import torch

from . import _lib
from .ops import _DTYPE, _check, _current_device, _fail, _raw_stream

_STATE = {"fp32": _lib.MOK_ADAMW_STATE_F32, "mxfp8": _lib.MOK_ADAMW_STATE_MXFP8}
_KEPT = {"fp32": ("m", "v"), "mxfp8": ("m", "m_scale", "r", "r_scale")}
_FIELD = {"masters": "master", "m": "m", "v": "v", "r": "v", "m_scale": "m_scale", "r_scale": "v_scale"}
_COUNT, _LR, _SEED_CHANGE = 0, 1, 2   # the counter's 64-bit fields
_capturing = torch._C._cuda_isCurrentStreamCapturing
# over a list, map() of these takes a third less time than a loop's body
_data_ptr, _is_contiguous, _device = torch.Tensor.data_ptr, torch.Tensor.is_contiguous, torch.Tensor.get_device
_dtype, _shape = attrgetter("dtype"), attrgetter("shape")


class AdamW:
    """Decoupled-weight-decay Adam over ``params`` (contiguous CUDA tensors of
    one device, bf16 or fp32, updated in place), all of them in one launch per
    kind.

    ``state``: "fp32" keeps m and v in 32 bits; "mxfp8" keeps m and
    r = sqrt(v) as E4M3 codes with one E8M0 scale per 32 elements, rounded
    stochastically with bits that ``seed``, the step, the tensor's place in
    ``params`` and the element's index determine (give two
    optimisers over one model two seeds).  ``master``: bf16 parameters
    also get an fp32 copy that takes the update; the parameter is its rounding.

    ``buffers`` hands in state tensors instead of fresh zeros: a dict of lists
    (one entry per parameter, None for a master of an fp32 parameter) with the
    keys of ``state_dict()["buffers"]``; ``step`` is the count they stand at.

    A step may be captured in a CUDA graph: each replay is the step that is due,
    and ``step_count`` and ``state_dict()`` (which then wait for the device)
    count it.  Replays follow ``lr``, ``step_count``, ``seed`` and
    ``load_state_dict`` as these are set between them; betas, eps, the weight
    decay and an ``lr`` given to the captured ``step`` itself stay as they were."""

    def __init__(self, params, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.01,
                 state: str = "fp32", master: bool = False, seed: int = 0, step: int = 0, buffers: dict | None = None):
        self.params = list(params)
        if state not in _STATE:
            raise ValueError(f"state must be one of {sorted(_STATE)}")
        self._dev = None
        for i, p in enumerate(self.params):
            self._dev = _check(p, f"params[{i}]", None, (torch.bfloat16, torch.float32), self._dev)
        # the host's share of what a step reads; from the first captured step on
        # `_counter` on the device holds the count of the steps since, and what
        # replaces lr and seed
        self._base_lr, self._base_seed, self._base_step = lr, int(seed), int(step)
        self._captured, self._device_lr, self._seed_change = False, None, 0
        self._counter = None
        if self.params:
            self._counter = torch.zeros(_lib.MOK_ADAMW_COUNTER_BYTES // 8, dtype=torch.int64, device=self.params[0].device)
            self._counter.view(torch.float64)[_LR].fill_(float("nan"))
        self.betas, self.eps, self.weight_decay, self.state = tuple(betas), eps, weight_decay, state
        if buffers is None:
            buffers = self._fresh(master)
        self._take(buffers)

    def _fresh(self, master):
        def zeros(p, n, dtype):
            return torch.zeros(n, dtype=dtype, device=p.device)

        out = {}
        for name in _KEPT[self.state]:
            if name.endswith("_scale"):   # the scale of a block of zeros is 2^0
                out[name] = [torch.full(((p.numel() + 31) // 32,), 127, dtype=torch.uint8, device=p.device)
                             for p in self.params]
            else:
                dtype = torch.float32 if self.state == "fp32" else torch.uint8
                out[name] = [zeros(p, p.numel(), dtype) for p in self.params]
        if master:
            out["masters"] = [p.detach().reshape(-1).float() if p.dtype == torch.bfloat16 else None
                              for p in self.params]
        return out

    def _take(self, buffers):
        want = set(_KEPT[self.state])
        if not want <= set(buffers) or set(buffers) - want - {"masters"}:
            raise ValueError(f"buffers: expected {sorted(want)} and optionally masters, got {sorted(buffers)}")
        for name, ts in buffers.items():
            if len(ts) != len(self.params):
                raise ValueError(f"buffers[{name!r}]: expected {len(self.params)} tensors, got {len(ts)}")
            for i, (p, t) in enumerate(zip(self.params, ts)):
                if name == "masters" and p.dtype == torch.float32 and t is None:
                    continue
                n = (p.numel() + 31) // 32 if name.endswith("_scale") else p.numel()
                dtype = torch.float32 if name == "masters" or self.state == "fp32" else torch.uint8
                _check(t, f"buffers[{name!r}][{i}]", None, (dtype,), self._dev)
                if t.numel() != n or (name == "masters" and p.dtype == torch.float32):
                    raise ValueError(f"buffers[{name!r}][{i}]: expected {n} elements for a "
                                     f"{p.dtype} parameter of {p.numel()}, got {t.numel()}")
        self.buffers = {k: list(v) for k, v in buffers.items()}
        # one launch list per parameter type (master copies belong to the bf16
        # ones), with the fields that a step changes as arrays over it
        self._groups = []
        for dtype in (torch.bfloat16, torch.float32):
            idx = [i for i, p in enumerate(self.params) if p.dtype == dtype]
            if not idx:
                continue
            arr = (_lib.MokAdamwTensor * len(idx))()
            for a, i in zip(arr, idx):
                a.p, a.n, a.index = self.params[i].data_ptr(), self.params[i].numel(), i
                for name, ts in self.buffers.items():
                    if ts[i] is not None:
                        setattr(a, _FIELD[name], ts[i].data_ptr())
            fields = np.frombuffer(arr, dtype=np.dtype(_lib.MokAdamwTensor))
            params = [self.params[i] for i in idx]
            self._groups.append((dtype, idx, params, [p.shape for p in params], arr, fields, fields["p"].tolist(),
                                 fields["n"].tolist()))

    @property
    def lr(self) -> float:
        return self._base_lr if self._device_lr is None else self._device_lr

    @lr.setter
    def lr(self, value: float) -> None:
        if self._captured:
            if not math.isfinite(value):
                raise ValueError("lr must be finite")
            self._counter.view(torch.float64)[_LR].fill_(value)
            self._device_lr = value
        else:
            self._base_lr = value

    @property
    def seed(self) -> int:
        return self._base_seed ^ self._seed_change

    @seed.setter
    def seed(self, value: int) -> None:
        if self._captured:
            self._seed_change = self._base_seed ^ int(value)
            low = self._seed_change & (2 ** 64 - 1)
            self._counter[_SEED_CHANGE].fill_(low - 2 ** 64 if low >> 63 else low)
        else:
            self._base_seed = int(value)

    @property
    def step_count(self) -> int:
        return self._base_step + (int(self._counter[_COUNT]) if self._captured else 0)

    @step_count.setter
    def step_count(self, value: int) -> None:
        if self._captured:
            self._counter[_COUNT].fill_(int(value) - self._base_step)
        else:
            self._base_step = int(value)

    def state_dict(self) -> dict:
        """The step count, the state kind and the state tensors themselves."""
        return {"step": self.step_count, "state": self.state, "seed": self.seed, "buffers": self.buffers}

    def load_state_dict(self, sd: dict) -> None:
        """Copies another optimiser's state (of the same kind and shapes) into this one's."""
        if sd["state"] != self.state or set(sd["buffers"]) != set(self.buffers):
            raise ValueError("the state is of another kind")
        pairs = []
        for name, ts in self.buffers.items():
            if len(sd["buffers"][name]) != len(ts):
                raise ValueError(f"{name}: another number of tensors")
            for i, (mine, other) in enumerate(zip(ts, sd["buffers"][name])):
                if (mine is None) != (other is None) or (mine is not None and
                                                         (mine.dtype != other.dtype or mine.numel() != other.numel())):
                    raise ValueError(f"{name}[{i}]: another type or length")
                if mine is not None:
                    pairs.append((mine, other))
        for mine, other in pairs:
            mine.copy_(other.reshape(mine.shape))
        self.step_count, self.seed = int(sd["step"]), int(sd["seed"])

    def _gradients(self, grads, idx, params, shapes, at):
        """The set of the gradients' types, and each one's type and address (None and 0: no gradient)."""
        own = grads if len(idx) == len(grads) else [grads[i] for i in idx]
        try:
            kinds, ptrs = list(map(_dtype, own)), list(map(_data_ptr, own))
            found = set(kinds)
            if (found <= _DTYPE.keys() and list(map(_shape, own)) == shapes and set(map(_device, own)) == {self._dev}
                    and all(map(_is_contiguous, own)) and list(map(_data_ptr, params)) == at):
                return found, kinds, ptrs
        except (AttributeError, TypeError):   # not all of them are tensors
            pass
        kinds, ptrs = [None] * len(idx), [0] * len(idx)
        for k, (i, g) in enumerate(zip(idx, own)):
            if g is None:
                continue
            _check(g, f"grads[{i}]", shapes[k], tuple(_DTYPE), self._dev)
            if params[k].data_ptr() != at[k]:
                raise ValueError(f"params[{i}] moved to other memory: build the optimiser again")
            kinds[k], ptrs[k] = g.dtype, g.data_ptr()
        return set(kinds), kinds, ptrs

    def step(self, grads=None, grad_scale=None, lr: float | None = None, stream=None) -> None:
        """One step.  ``grads``: one gradient per parameter, of its shape, bf16
        or fp32 (default: each ``param.grad``); None entries are skipped.
        ``grad_scale``: a one-element fp32 CUDA tensor that multiplies every
        gradient (clipping, loss scaling).  ``lr`` replaces the learning rate
        for this step."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.step(grads, grad_scale, lr)
        if grads is None:
            grads = [p.grad for p in self.params]
        if len(grads) != len(self.params):
            raise ValueError(f"expected {len(self.params)} gradients, got {len(grads)}")
        if self.params and self._dev != _current_device():
            raise ValueError(f"the parameters are on cuda:{self._dev}, but the current device (or the stream's) is "
                             f"cuda:{_current_device()}")
        scale = None
        if grad_scale is not None:
            _check(grad_scale, "grad_scale", None, (torch.float32,), self._dev)
            if grad_scale.numel() != 1:
                raise ValueError("grad_scale: expected one element")
            scale = grad_scale.data_ptr()
        # the launches: (parameter type, gradient type, list, its fields, addresses, lengths)
        launches, changed = [], []
        for dtype, idx, params, shapes, arr, fields, at, lengths in self._groups:
            found, kinds, ptrs = self._gradients(grads, idx, params, shapes, at)
            if len(found) == 1 and None not in found:
                launches.append((dtype, kinds[0], arr, fields, ptrs, lengths))
            else:   # a length of 0 leaves a tensor out: no gradient, or one of another type
                launches += [(dtype, kind, arr, fields, ptrs, [n if t is kind else 0 for n, t in zip(lengths, kinds)])
                             for kind in found - {None}]
                params = [p for p, kind in zip(params, kinds) if kind is not None]
            changed += params
        lib = _lib.load()
        if not self._captured and self.params and _capturing():
            self._captured = True   # for good: only the device knows how often the graph runs
        counted = self._captured
        cfg = _lib.MokAdamwConfig(state=_STATE[self.state], lr=self._base_lr if lr is None else lr, beta1=self.betas[0],
                                  beta2=self.betas[1], eps=self.eps, weight_decay=self.weight_decay,
                                  step=self._base_step + (not counted), seed=self._base_seed & (2 ** 64 - 1))
        handle = _raw_stream(self._dev) if self.params else None
        # several calls make one step: what any of them would refuse is refused
        # before the first one moves anything
        if counted or len(launches) > 1:
            self._call(lib.mok_adamw_check, cfg, launches)
        if counted:
            counter = self._counter.data_ptr()
            st = lib.mok_adamw_advance(C.byref(cfg), lr is not None, counter, handle)
            if st:
                _fail(st, "mok_adamw_advance")
            self._call(lib.mok_adamw_step_counted, cfg, launches, scale, counter, handle)
        else:
            self._call(lib.mok_adamw_step, cfg, launches, scale, handle)
            self._base_step += 1
        # the parameters changed under autograd's eyes: a backward that saved
        # them before this step has to notice (and only those: a parameter
        # without a gradient is what it was)
        torch.autograd.graph.increment_version(changed)

    @staticmethod
    def _call(fn, cfg, launches, *args):
        for dtype, kind, arr, fields, ptrs, lengths in launches:
            cfg.param_dtype, cfg.grad_dtype = _DTYPE[dtype], _DTYPE[kind]
            fields["g"], fields["n"] = ptrs, lengths
            st = fn(C.byref(cfg), arr, len(arr), *args)
            if st:
                _fail(st, fn.__name__)
