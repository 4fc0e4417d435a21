"""The AdamW step and the gradient norm (include/wtconv_optim.h) on PyTorch tensors.

``AdamW`` is the object a training program builds once over its parameters and their gradient
buffers: it checks them, keeps their states and the descriptors that the library reads, and every
step is one call of the compiled binding.  The update runs in the library's CUDA kernels.
"""
from __future__ import annotations

import ctypes

import torch

from .wtconv import DTYPE_CODE, _on, load, load_binding

ADAMW_BLOCK = 256  # WTCONV_ADAMW_BLOCK

EXPORTED = ("wtconv_adamw_step", "wtconv_adamw_state_values", "wtconv_grad_norm", "wtconv_grad_norm_workspace_size")


class OptimTensor(ctypes.Structure):
    """wtconv_optim_tensor."""

    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "grad", "m", "v", "m_max", "v_max", "copy")] + \
        [("n", ctypes.c_longlong)]


class AdamWConfig(ctypes.Structure):
    """wtconv_adamw_config."""

    _fields_ = [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps", "weight_decay")] + \
        [("step", ctypes.c_longlong)] + [(n, ctypes.c_int) for n in ("state_bits", "grad_dtype", "copy_dtype")]


_lib = None


def _load() -> ctypes.CDLL:
    """The library with this header's signatures."""
    global _lib
    if _lib is None:
        lib = load()
        i, vp, sz = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
        tensors = ctypes.POINTER(OptimTensor)
        lib.wtconv_adamw_step.restype = i
        lib.wtconv_adamw_step.argtypes = [i, tensors, ctypes.POINTER(AdamWConfig), vp, vp]
        lib.wtconv_adamw_state_values.restype = i
        lib.wtconv_adamw_state_values.argtypes = [i, tensors, ctypes.POINTER(vp), ctypes.POINTER(vp), vp]
        lib.wtconv_grad_norm_workspace_size.restype = sz
        lib.wtconv_grad_norm_workspace_size.argtypes = [i, tensors]
        lib.wtconv_grad_norm.restype = i
        lib.wtconv_grad_norm.argtypes = [i, tensors, i, ctypes.c_double, vp, vp, sz, vp]
        _lib = lib
    return _lib


class AdamW:
    """AdamW over many tensors in one call per step.

    params: contiguous fp32 CUDA tensors, updated in place; one that layers share is given once.
    grads: one contiguous tensor per parameter, of its size and one dtype (fp32, bf16 or fp16); the
    buffers that the backward writes each step (``set_grads`` for other tensors).  copies: optional
    16-bit working copies of the parameters, rewritten by each step (None entries: no copy).  Each of
    these may be given other memory between steps (``p.data = ...``); a ``detach()`` of it would not
    follow.  state_bits: 32 or 8.
    states: adopt existing ones, as ``state_dict`` gives them (they are used in place), ``count``
    steps having been taken.

    A method's ``stream`` (default: the current one) is where its work is queued.  The caller orders it
    after the work that writes the gradients, and keeps this object until that work has ended.
    """

    def __init__(self, params, grads, state_bits=32, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01,
                 copies=None, states=None, count=0):
        self.params = list(params)
        if not self.params:
            raise ValueError("no parameters")
        if state_bits not in (32, 8):
            raise ValueError(f"state_bits must be 32 or 8, not {state_bits}")
        self.state_bits, self.count, self.lr = state_bits, int(count), lr
        self.device = self.params[0].device
        n = len(self.params)
        self._tensors = (OptimTensor * n)()
        self._ext = load_binding()
        self._table = self._ext.TensorTable(n, ctypes.addressof(self._tensors), self.device)
        self._fill("param", self.params, torch.float32, "params", params=True)
        self.copies = [None] * n if copies is None else list(copies)
        kinds = {c.dtype for c in self.copies if c is not None}
        if len(kinds) > 1 or kinds - {torch.bfloat16, torch.float16}:
            raise ValueError(f"copies must all be bf16 or all fp16, not {kinds}")
        copy_dtype = kinds.pop() if kinds else torch.bfloat16
        self._fill("copy", self.copies, copy_dtype, "copies", may_be_none=True)
        if states is None:
            states = self._new_states()
        self.states = {name: list(ts) for name, ts in states.items()}
        want = self._state_layout()
        if set(self.states) != set(want):
            raise ValueError(f"states hold {sorted(self.states)}, expected {sorted(want)}")
        for name, (dtype, per) in want.items():
            self._fill(name, self.states[name], dtype, f"states[{name!r}]", per)
        self._config = AdamWConfig(lr, betas[0], betas[1], eps, weight_decay, 0, state_bits, 0, DTYPE_CODE[copy_dtype])
        self._scalars = ctypes.addressof(self._config)
        self.set_grads(grads)

    def _fill(self, field, tensors, dtype, name, per=1, params=False, may_be_none=False):
        self._table.fill(tensors, getattr(OptimTensor, field).offset, dtype, per, name, params, may_be_none)

    def _state_layout(self):
        if self.state_bits == 32:
            return {"m": (torch.float32, 1), "v": (torch.float32, 1)}
        return {"m": (torch.int8, 1), "v": (torch.uint8, 1), "m_max": (torch.float32, ADAMW_BLOCK),
                "v_max": (torch.float32, ADAMW_BLOCK)}

    def _new_states(self):
        return {name: [torch.zeros(-(-p.numel() // per), dtype=dtype, device=self.device) for p in self.params]
                for name, (dtype, per) in self._state_layout().items()}

    def set_grads(self, grads):
        """Take the gradients from these buffers from now on."""
        grads = list(grads)
        if len(grads) != len(self.params):
            raise ValueError(f"{len(grads)} gradients for {len(self.params)} parameters")
        dtype = grads[0].dtype
        if dtype not in DTYPE_CODE:
            raise ValueError(f"gradients have unsupported dtype {dtype}")
        self._fill("grad", grads, dtype, "grads")
        self.grads = grads
        self._config.grad_dtype = self._grad_dtype = DTYPE_CODE[dtype]
        self._norm_bytes = _load().wtconv_grad_norm_workspace_size(len(self.params), self._tensors)

    def state_dict(self):
        return {"states": self.states, "count": self.count}

    def grad_norm(self, max_norm=float("inf"), out=None, workspace=None, stream=None) -> torch.Tensor:
        """Device tensor (norm, factor): the norm over every gradient and the factor that limits it
        to max_norm (NaN where the norm is not finite), for ``step(clip=...)``."""
        return self._ext.grad_norm(self._table, self._grad_dtype, max_norm, out, workspace, self._norm_bytes, stream)

    def step(self, clip=None, lr=None, count=None, stream=None) -> None:
        """One update of every parameter.  clip: what ``grad_norm`` returned (a factor that is not
        finite leaves everything as it is).  lr: the rate from this step on.  count: the step's
        number, from 1 (default: the next).  A captured graph replays this step's number."""
        lr = self.lr if lr is None else lr
        count = self.count + 1 if count is None else count
        self._ext.adamw_step(self._table, self._scalars, lr, count, clip, stream)
        self.count, self.lr = count, lr

    def state_values(self, m_out=None, v_out=None, stream=None):
        """The averages (m, v) as lists of fp32 tensors.  m_out, v_out: lists of fp32 tensors to write
        them to.  Where a list is not given, the states themselves in 32 bits, in 8 new tensors of what
        the codes stand for."""
        if self.state_bits == 8:
            m, v = self._ext.state_values(self._table, m_out, v_out, stream)
            return m_out if m is None else m, v_out if v is None else v
        lists = []
        for name, kind, out in (("m_out", "m", m_out), ("v_out", "v", v_out)):
            states = self.states[kind]
            if out is not None and len(out) != len(states):
                raise ValueError(f"{len(out)} tensors in {name} for {len(states)} parameters")
            for i, (t, s) in enumerate(zip(out or (), states)):
                if t.dtype != torch.float32 or t.device != self.device or t.numel() != s.numel() or not t.is_contiguous():
                    raise ValueError(f"{name}[{i}] must be a contiguous fp32 tensor of {s.numel()} elements on {self.device}")
            lists.append(states if out is None else out)
        with _on(self.device, stream, None, [t for out in (m_out, v_out) for t in out or ()]):
            for out, kind in zip(lists, "mv"):
                for t, s in zip(out, self.states[kind]):
                    if t is not s:
                        t.view(-1).copy_(s.view(-1))
        return tuple(lists)
