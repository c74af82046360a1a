"""The optimizer of a training step on one GPU: gradient norm, clipping and AdamW.

Buffers and argument checks around ``moe_grad_norm`` and ``moe_adamw_step``; the
arithmetic is in the library's kernels.  Every call runs on the current CUDA stream of
the tensors' device, reads nothing back, and can be captured in a CUDA graph (the step
count lives on the device: a replay is the next step).

    opt = layer.optimizer(lr=1e-4, state="e4m3", ema_decay=0.9999)   # masters from the layer's weights
    out = layer.forward(x)
    opt.step(layer.backward(x, dout), max_norm=1.0)                  # the layer's weights are the new ones
"""
from __future__ import annotations

from typing import Optional, Sequence

import torch

from . import binding as B

ALIGN = 16             # bytes: the kernels' vectors start at each tensor's first element
BLOCK = 256            # elements that share a scale of 8-bit moments; each tensor's state starts on such a block
_DTYPE = {torch.float32: B.MOE_F32, torch.bfloat16: B.MOE_BF16, torch.float16: B.MOE_F16}


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _check(t, what, dtypes, device, n=None):
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes:
        raise ValueError(f"{what} must be a tensor of {' or '.join(str(d) for d in dtypes)}")
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, not on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if t.numel() and t.data_ptr() % ALIGN:
        raise ValueError(f"{what} starts at an address that is not {ALIGN}-byte aligned")
    if n is not None and t.numel() != n:
        raise ValueError(f"{what} has {t.numel()} elements, not {n}")


class _Control:
    """The 256-byte control block on the device and views of its words."""

    def __init__(self, device):
        self.device = torch.device(device)
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.ctl = torch.zeros(256, dtype=torch.uint8, device=self.device)
        self._step = self.ctl[0:8].view(torch.int64)
        self.lr_scale = self.ctl[24:28].view(torch.float32)      # factor of lr; write it between replays of a graph
        self.grad_norm = self.ctl[28:32].view(torch.float32)     # of the last norm: [1] tensors on the device
        self.grad_scale = self.ctl[32:36].view(torch.float32)
        self.nonfinite = self.ctl[36:40].view(torch.int32)
        self.skipped = self.ctl[40:48].view(torch.int64)         # steps that a non-finite gradient left out
        self._ctl_ptr, self._ws_for = self.ctl.data_ptr(), -1
        self._ws = []                                            # the last is the one in use; a captured graph may hold another

    def _init(self, step, betas):
        with torch.cuda.device(self.device):
            B.moe_optim_init(self.ctl, step, betas[0], betas[1], _stream(self.device))

    def _norm(self, tensors, n, max_norm, grad_mult, stream):
        if self._ws_for < n:
            need = B.moe_grad_norm_workspace_size(n)
            if not self._ws or self._ws_bytes < need:
                self._ws.append(torch.empty(need, dtype=torch.uint8, device=self.device))
                self._ws_ptr, self._ws_bytes = self._ws[-1].data_ptr(), need
            self._ws_for = n
        B.moe_grad_norm(tensors, n, grad_mult, max_norm, self._ctl_ptr, self._ws_ptr, self._ws_bytes, stream)

    def _on_device(self, call, *args):
        """The call with the tensors' device current."""
        if torch.cuda.current_device() == self.device.index:
            return call(*args)
        with torch.cuda.device(self.device):
            return call(*args)


class _GradList:
    """The C array of a call's tensors; a call checks its gradients and writes what differs from the last one's."""

    def __init__(self, n, sizes=None):
        self.tensors = (B.MoeAdamwTensor * n)()
        self.sizes = sizes
        self.items = list(self.tensors)              # ctypes makes a new view at every access
        self.held = [None] * n

    def fill(self, grads, device):
        index, sizes, held = device.index, self.sizes, self.held
        for i, g in enumerate(grads):
            if g is None:
                if held[i] is not False:
                    self.items[i].n, held[i] = 0, False   # no gradient: the tensor stays as it is
                continue
            if type(g) is not torch.Tensor or g.get_device() != index or not g.is_contiguous():
                _check(g, f"grads[{i}]", tuple(_DTYPE), device)
            dt, n = _DTYPE.get(g.dtype), g.numel()
            if dt is None or (sizes is not None and n != sizes[i]):
                _check(g, f"grads[{i}]", tuple(_DTYPE), device, None if sizes is None else sizes[i])
            new = (g.data_ptr(), n, dt)
            if held[i] != new:
                if new[0] % ALIGN:
                    _check(g, f"grads[{i}]", tuple(_DTYPE), device)
                t = self.items[i]
                t.grad, t.n, t.grad_dtype = held[i] = new


class GradNorm(_Control):
    """2-norm of a list of gradients (fp32, bf16 or fp16; contiguous, 16-byte aligned) together, and the factor
    that clips them.

    ``norm, scale = GradNorm(device)(grads, max_norm=1.0)``: views of the control block, [1] fp32 each,
    overwritten by the next call.  ``scale`` is 0 and ``nonfinite`` 1 where a gradient is not finite."""

    def __init__(self, device="cuda:0"):
        super().__init__(device)
        self._init(0, (0.0, 0.0))
        self._list = _GradList(0)

    def __call__(self, grads: Sequence[Optional[torch.Tensor]], max_norm: float = 0.0, grad_mult: float = 1.0):
        n = len(grads)
        if len(self._list.items) != n:
            self._list = _GradList(n)
        self._list.fill(grads, self.device)
        self._on_device(self._norm, self._list.tensors, n, max_norm, grad_mult, _stream(self.device))
        return self.grad_norm, self.grad_scale


class AdamW(_Control):
    """AdamW over many tensors in one launch.  Every tensor is contiguous and starts at a 16-byte aligned
    address (slices of a flat buffer: at a multiple of 16 bytes); others are refused.

    ``params``: fp32 tensors, updated in place.  ``weights``: for each its bf16 or fp16 copy, which
    every step rewrites, or None.  ``weight_decay``: one value or one for each tensor.  ``state``:
    "f32" moments, or "e4m3" ones (8 bits, 256 elements to a scale, rounded at random by ``seed``).
    ``ema_decay``: keep a moving average of the params.  ``buffers`` holds the state: one flat tensor
    of each kind ("m", "v", "m_scale", "v_scale", "ema"; "v" holds sqrt(v) for "e4m3"), in which
    ``params[i]``'s part starts at element ``starts[i]``, a multiple of 256 (of 1 in the scales).
    """

    def __init__(self, params: Sequence[torch.Tensor], weights: Optional[Sequence[Optional[torch.Tensor]]] = None, *,
                 lr: float, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay=0.0, state: str = "f32",
                 ema_decay: Optional[float] = None, seed: int = 0):
        params = list(params)
        if not params or not isinstance(params[0], torch.Tensor) or params[0].device.type != "cuda":
            raise ValueError("params must be a list of CUDA tensors")
        super().__init__(params[0].device)
        weights = [None] * len(params) if weights is None else list(weights)
        decay = [float(weight_decay)] * len(params) if isinstance(weight_decay, (int, float)) else list(weight_decay)
        if len(weights) != len(params) or len(decay) != len(params):
            raise ValueError("weights and weight_decay need one entry for each tensor")
        if state not in ("f32", "e4m3"):
            raise ValueError(f"state={state!r}: 'f32' or 'e4m3'")
        if not (0.0 <= betas[0] < 1.0 and 0.0 <= betas[1] < 1.0):
            raise ValueError(f"betas={betas} outside [0, 1)")
        spans = []
        for i, (p, w) in enumerate(zip(params, weights)):
            _check(p, f"params[{i}]", (torch.float32,), self.device)
            spans.append((p.data_ptr(), p.numel() * 4, f"params[{i}]"))
            if w is not None:
                _check(w, f"weights[{i}]", (torch.bfloat16, torch.float16), self.device, p.numel())
                spans.append((w.data_ptr(), w.numel() * 2, f"weights[{i}]"))
        spans = sorted(s for s in spans if s[1])
        for a, b in zip(spans, spans[1:]):
            if a[0] + a[1] > b[0]:
                raise ValueError(f"{a[2]} and {b[2]} overlap")
        self.params, self.weights, self.betas = params, weights, (float(betas[0]), float(betas[1]))
        self.sizes = [p.numel() for p in params]
        self.starts, total = [], 0
        for n in self.sizes:
            self.starts.append(total)
            total += -(-n // BLOCK) * BLOCK
        z = lambda n, dt: torch.zeros(n, dtype=dt, device=self.device)  # noqa: E731
        q8 = state == "e4m3"
        self.buffers = {k: z(total, torch.float8_e4m3fn if q8 else torch.float32) for k in ("m", "v")}
        if q8:
            self.buffers.update({k: z(total // BLOCK, torch.float32) for k in ("m_scale", "v_scale")})
        if ema_decay is not None:
            self.buffers["ema"] = z(total, torch.float32)
            for p, at in zip(params, self.starts):
                self.buffers["ema"][at:at + p.numel()].copy_(p.reshape(-1))
        self.settings = B.MoeAdamw(lr, self.betas[0], self.betas[1], eps, 0.0 if ema_decay is None else ema_decay, 1.0,
                                   seed % (1 << 64), B.MOE_MOMENTS_E4M3 if q8 else B.MOE_MOMENTS_F32, 0)
        self._list = _GradList(len(params), self.sizes)
        at = {k: b.data_ptr() for k, b in self.buffers.items()}
        for t, p, w, wd, s in zip(self._list.items, params, weights, decay, self.starts):
            t.param, t.weight_decay = p.data_ptr(), wd
            if w is not None:
                t.weight, t.weight_dtype = w.data_ptr(), _DTYPE[w.dtype]
            size = 1 if q8 else 4
            t.m, t.v = at["m"] + s * size, at["v"] + s * size
            if q8:
                t.m_scale, t.v_scale = (at[k] + s // BLOCK * 4 for k in ("m_scale", "v_scale"))
            if ema_decay is not None:
                t.ema = at["ema"] + s * 4
        self._init(0, self.betas)

    @property
    def lr(self) -> float:
        return self.settings.lr

    @lr.setter
    def lr(self, v: float):
        self.settings.lr = v                         # a captured graph keeps its own: scale that by lr_scale

    def steps_taken(self) -> int:
        """Steps taken so far (waits for the device)."""
        torch.cuda.synchronize(self.device)
        return int(self._step.item())

    def part(self, name: str, i: int) -> torch.Tensor:
        """Tensor i's part of ``buffers[name]``."""
        per = BLOCK if name.endswith("_scale") else 1
        at = self.starts[i] // per
        return self.buffers[name][at:at + -(-self.sizes[i] // per)]

    def step(self, grads: Sequence[Optional[torch.Tensor]], max_norm: Optional[float] = None, grad_mult: float = 1.0):
        """One step.  ``grads``: fp32, bf16 or fp16, one for each tensor (None leaves a tensor as it is),
        taken times ``grad_mult``.  With ``max_norm`` the norm over all of them is formed first
        (``grad_norm``), they are clipped to it (0: not clipped), and a gradient that is not finite
        leaves everything as it is and counts in ``skipped``."""
        if len(grads) != len(self.params):
            raise ValueError(f"{len(grads)} gradients for {len(self.params)} tensors")
        self._list.fill(grads, self.device)
        self._on_device(self._step_now, max_norm, grad_mult, _stream(self.device))

    def _step_now(self, max_norm, grad_mult, stream):
        tensors, n, settings = self._list.tensors, len(self.params), self.settings
        if max_norm is not None:
            self._norm(tensors, n, max_norm, grad_mult, stream)
        settings.clipped = int(max_norm is not None)
        settings.grad_mult = grad_mult
        B.moe_adamw_step(settings, tensors, n, self._ctl_ptr, stream)

    def state_dict(self) -> dict:
        """Copies of the state and the step count: of all steps issued before, on any stream, and of none
        issued later (waits for the device, and for the copies)."""
        step = self.steps_taken()
        state = dict({k: b.clone() for k, b in self.buffers.items()}, step=step)
        torch.cuda.synchronize(self.device)
        return state

    def load_state_dict(self, state: dict):
        """Take up a ``state_dict``, behind all steps issued before and ahead of all issued later (waits for the
        device on both sides).  ``lr_scale`` is 1 and ``skipped`` 0 again."""
        if set(state) != set(self.buffers) | {"step"}:
            raise ValueError(f"state has {sorted(state)}, not {sorted(self.buffers) + ['step']}")
        for k, b in self.buffers.items():
            if state[k].shape != b.shape or state[k].dtype != b.dtype:
                raise ValueError(f"state[{k!r}] is {tuple(state[k].shape)} {state[k].dtype}, not {tuple(b.shape)} {b.dtype}")
        if int(state["step"]) < 0:
            raise ValueError(f"state['step'] is {state['step']}")
        torch.cuda.synchronize(self.device)
        for k, b in self.buffers.items():
            b.copy_(state[k])
        self._init(int(state["step"]), self.betas)
        torch.cuda.synchronize(self.device)


class LayerAdamW(AdamW):
    """AdamW of a ``MoELayer``'s weights: fp32 masters made from them (an fp32 weight is its own), the
    layer's tensors rewritten by every step.  ``weight_decay`` (one value) is for the matrices; biases
    have none.  ``step`` takes what ``MoELayer.backward`` returns."""

    NAMES = (("wg", "dwg"), ("w1", "dw1"), ("w2", "dw2"), ("ws1", "dws1"), ("ws2", "dws2"),
             ("router_bias", "dbias"), ("b1", "db1"), ("b2", "db2"), ("bs1", "dbs1"), ("bs2", "dbs2"))

    def __init__(self, layer, *, weight_decay: float = 0.0, **settings):
        self.grad_names, params, weights, decay = [], [], [], []
        for name, grad in self.NAMES:
            w = getattr(layer, name)
            if w is None:
                continue
            own = w.dtype == torch.float32
            self.grad_names.append(grad)
            params.append(w if own else w.float())
            weights.append(None if own else w)
            decay.append(0.0 if "b" in name else weight_decay)
        super().__init__(params, weights, weight_decay=decay, **settings)

    def step(self, grads: dict, max_norm: Optional[float] = None, grad_mult: float = 1.0):
        super().step([grads[n] for n in self.grad_names], max_norm, grad_mult)

    def state_dict(self) -> dict:
        """Copies of the state, the step count and the masters (waits for the device)."""
        state = dict(super().state_dict(), params=[p.clone() for p in self.params])
        torch.cuda.synchronize(self.device)
        return state

    def load_state_dict(self, state: dict):
        """Take up a ``state_dict``: the layer's weights become those of its masters."""
        state = dict(state)
        params = state.pop("params", ())
        if [p.shape for p in params] != [p.shape for p in self.params]:
            raise ValueError("state['params'] does not fit the layer's weights")
        super().load_state_dict(state)
        for p, w, saved in zip(self.params, self.weights, params):
            p.copy_(saved)
            if w is not None:
                w.copy_(p)
        torch.cuda.synchronize(self.device)
