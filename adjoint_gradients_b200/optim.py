"""AdamW over many tensors on one GPU (qml_opt_* of include/qml.h).

Argument marshalling only, as in qml.py: torch tensors provide device memory and
streams, the update runs in the library's CUDA kernels.

    opt = AdamW([theta], lr=1e-2)                   # full-precision states
    opt = AdamW(params, lr=1e-3, state="8bit")      # states in 8 bits with block scales
    norm = opt.step(grads, max_norm=1.0)            # clip to norm 1 and update in place
"""
from __future__ import annotations

import ctypes
import operator
from array import array

from . import qml

STATE = {"full": 0, "8bit": 1}
_DTYPE = operator.attrgetter("dtype")
BLOCK = 256  # QML_OPT_BLOCK: elements that share a scale; tensors start at multiples of it in the flat states


def _dtypes():
    import torch

    return {torch.float32: 0, torch.float64: 1, torch.bfloat16: 2, torch.float16: 3}


def _per_tensor(value, n, what):
    if not hasattr(value, "__len__"):
        return [float(value)] * n
    value = [float(x) for x in value]
    if len(value) != n:
        raise ValueError(f"{what}: {len(value)} values for {n} tensors")
    return value


class AdamW:
    """Adam with decoupled weight decay over a list of contiguous CUDA tensors.

    params        tensor or list of tensors (fp32, bf16, fp16; or all fp64), updated in place
    lr            default learning rate of step()
    weight_decay  one value, or one per tensor; lr_scale likewise: factors of lr
    state         "full": fp32 (fp64 parameters: fp64) moments; "8bit": e4m3 codes with a
                  float scale for every 256 elements (see QML_STATE_8BIT)
    grad_dtype    type of the gradients: the parameters' (default), or float32 for
                  bf16 / fp16 parameters
    master        for bf16 / fp16 parameters: True (fp32 copies made here) or a list of
                  contiguous fp32 tensors that the parameters are rounded copies of
    seed          of the random rounding of the 8-bit states

    The states are flat buffers in which tensor i takes numel elements from
    offsets[i] (a multiple of 256): m and v, and with "8bit" m_scale and v_scale (a
    float for every 256 elements), v then holding sqrt(v) / scale.

    One object serves one stream at a time (see include/qml.h).
    """

    def __init__(self, params, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay=0.01,
                 state: str = "full", grad_dtype=None, master=None, lr_scale=1.0, seed: int = 0):
        import torch

        if isinstance(params, torch.Tensor):
            params = [params]
        params = list(params)
        if not params:
            raise ValueError("no parameters")
        if state not in STATE:
            raise ValueError(f"state must be one of {tuple(STATE)}")
        n = len(params)
        types = _dtypes()
        self.device = params[0].device
        self._index = self.device.index
        for p in params:
            if p.dtype not in types:
                raise ValueError(f"parameters of type {p.dtype} are not supported")
            self._check_buffer(p, p.dtype, p.numel(), "a parameter")
        f64 = [p.dtype == torch.float64 for p in params]
        if any(f64) and not all(f64):
            raise ValueError("fp64 parameters take an optimiser of their own")
        if all(f64) and state == "8bit":
            raise ValueError("fp64 parameters have no 8-bit states")
        self.params, self.lr, self.betas, self.eps, self.state = params, lr, tuple(betas), eps, state
        self.real_dtype = torch.float64 if all(f64) else torch.float32
        gt = [grad_dtype or p.dtype for p in params]
        for p, g in zip(params, gt):
            if g != p.dtype and not (g == torch.float32 and p.dtype in (torch.bfloat16, torch.float16)):
                raise ValueError(f"gradients of type {g} for parameters of type {p.dtype}")
        if master is True:
            master = [p.float() if p.dtype in (torch.bfloat16, torch.float16) else None for p in params]
        self.master = list(master) if master is not None else [None] * n
        if len(self.master) != n:
            raise ValueError(f"master: {len(self.master)} tensors for {n}")
        for p, w in zip(params, self.master):
            if w is None:
                continue
            if p.dtype not in (torch.bfloat16, torch.float16):
                raise ValueError("master weights are for bf16 and fp16 parameters")
            self._check_buffer(w, torch.float32, p.numel(), "a master weight")
        lrs, wds = _per_tensor(lr_scale, n, "lr_scale"), _per_tensor(weight_decay, n, "weight_decay")

        self.offsets, total = [], 0
        for p in params:
            self.offsets.append(total)
            total += -(-p.numel() // BLOCK) * BLOCK
        new = lambda count, dt: torch.zeros(count, dtype=dt, device=self.device)  # noqa: E731
        st = torch.float8_e4m3fn if state == "8bit" else self.real_dtype
        self.m, self.v = new(total, st), new(total, st)
        self.m_scale = self.v_scale = None
        if state == "8bit":
            self.m_scale, self.v_scale = new(total // BLOCK, torch.float32), new(total // BLOCK, torch.float32)

        table = (qml._OptTensor * n)()
        size = self.m.element_size()
        for i, (p, off) in enumerate(zip(params, self.offsets)):
            w = self.master[i]
            sc = [None if s is None else s.data_ptr() + off // BLOCK * 4 for s in (self.m_scale, self.v_scale)]
            table[i] = qml._OptTensor(p.data_ptr(), None if w is None else w.data_ptr(), self.m.data_ptr() + off * size,
                                      self.v.data_ptr() + off * size, sc[0], sc[1], p.numel(), types[p.dtype],
                                      types[gt[i]], lrs[i], wds[i])
        cfg = qml._OptConfig(STATE[state], self.betas[0], self.betas[1], eps, seed & (2 ** 64 - 1))
        self.lib = qml.load_library()
        h = ctypes.c_void_p()
        qml._check(self.lib.qml_opt_create(ctypes.byref(cfg), n, table, self.device.index, ctypes.byref(h)),
                   "qml_opt_create")
        self._h = h
        T = torch.Tensor
        self._calls = T.numel, T.is_contiguous, T.get_device, T.data_ptr
        self._one_by_one = (ctypes.c_void_p * n)()
        self._at = ctypes.addressof(self._one_by_one)
        self._one = torch.empty(1, dtype=self.real_dtype, device=self.device)
        self._norms, self._norms_of = [], None
        # (the functions below torch's own of the same meaning, where it has them: 0.2 us less)
        self._capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", torch.cuda.is_current_stream_capturing)
        self._on_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        self._numels, self._dtypes = [p.numel() for p in params], gt
        self._written = params + [w for w in self.master if w is not None]
        self._increment_version = getattr(torch._C, "_increment_version", torch.autograd.graph.increment_version)
        nbytes = int(self.lib.qml_opt_workspace_bytes(h))
        self.ws = torch.empty(nbytes + 256, dtype=torch.uint8, device=self.device)
        qml._check(self.lib.qml_opt_set_workspace(h, (self.ws.data_ptr() + 255) // 256 * 256, nbytes, self._stream(None)),
                   "qml_opt_set_workspace")

    def _check_buffer(self, t, dtype, numel, what):
        if not t.is_cuda or t.device != self.device:
            raise ValueError(f"{what} is on {t.device}: all tensors belong on one CUDA device")
        if t.dtype != dtype or t.numel() != numel or not t.is_contiguous():
            raise ValueError(f"{what} must be a contiguous {dtype} tensor of {numel} elements")

    def _stream(self, stream):
        if stream is None:
            return qml._current_stream(self._index)
        return getattr(stream, "cuda_stream", stream)

    def close(self):
        if getattr(self, "_h", None):
            self.lib.qml_opt_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ------------------------------------------------------------------ calls
    def _take(self, grads):
        """Address of the array of the gradients' pointers, checked."""
        if not isinstance(grads, (list, tuple)):
            grads = [grads]
        if len(grads) != len(self._numels):
            raise ValueError(f"{len(grads)} gradients for {len(self._numels)} tensors")
        if len(grads) > 3 and self._take_many(grads):
            return self._many.buffer_info()[0]
        out, dev = self._one_by_one, self._index
        for i, (g, numel, dtype) in enumerate(zip(grads, self._numels, self._dtypes)):
            if g is None:
                out[i] = None
            elif g.dtype is dtype and g.numel() == numel and g.is_contiguous() and g.get_device() == dev:
                out[i] = g.data_ptr()
            else:
                raise ValueError(f"gradient {i} must be a contiguous {dtype} tensor of {numel} elements on "
                                 f"{self.device}")
        return self._at

    def _take_many(self, grads) -> bool:
        """Many gradients checked all at once (a quarter less time); False when one of
        them is absent or not as it should be."""
        numel, contiguous, device, data_ptr = self._calls
        try:
            if (list(map(numel, grads)) == self._numels and list(map(_DTYPE, grads)) == self._dtypes
                    and all(map(contiguous, grads)) and set(map(device, grads)) == {self._index}):
                self._many = array("Q", map(data_ptr, grads))
                return True
        except (TypeError, AttributeError):  # not a tensor
            pass
        return False

    def _norm_out(self, norm, stream):
        """The norm's tensor, by default a new one that belongs to the launch's stream."""
        if norm is None and stream is None:
            # a captured call's is the graph's: replays write it when eager calls' norms may be long gone
            if self._capturing() or self._on_device() != self._index:
                return self._one.new_empty(1)
            # eager calls' are made some at a time (6,000 elements, clipped: one by one 7.5 us a call, so 7.1)
            here = qml._current_stream(self._index)
            if not self._norms or self._norms_of != here:
                self._norms_of, self._norms = here, list(self._one.new_empty((64, 1)).unbind(0))
            return self._norms.pop()
        if norm is None:
            return qml._run_on(stream, self._index, lambda: self._one.new_empty(1))
        self._check_buffer(norm, self.real_dtype, 1, "the norm")
        return norm

    def step(self, grads, lr=None, max_norm: float | None = None, grad_scale: float = 1.0, norm=None, stream=None):
        """One step in place; grads: a tensor for each parameter, or None for one that
        stays as it is.  lr: the object's by default, a number, or a one-element device
        tensor (for captured steps).  max_norm clips the gradients' common 2-norm and
        makes a step with a norm that is not finite change nothing (sync() then raises);
        the norm before clipping is returned, as a one-element tensor."""
        lr_dev = None
        lr = self.lr if lr is None else lr
        if hasattr(lr, "data_ptr"):
            self._check_buffer(lr, self.real_dtype, 1, "lr")
            lr, lr_dev = 0.0, lr.data_ptr()
        if max_norm is None:
            if norm is not None:
                raise ValueError("the norm comes with max_norm (math.inf to measure only)")
            max_norm, norm_ptr = 0.0, None
        else:
            if not max_norm > 0.0:
                raise ValueError("max_norm must be positive")
            norm = self._norm_out(norm, stream)
            norm_ptr = norm.data_ptr()
        qml._check(self.lib.qml_opt_step(self._h, self._take(grads), lr, lr_dev, grad_scale, max_norm, norm_ptr,
                                         self._stream(stream)), "qml_opt_step")
        self._increment_version(self._written)  # so that autograd notices tensors saved before the step
        return norm

    def grad_norm(self, grads, grad_scale: float = 1.0, norm=None, stream=None):
        """The 2-norm of all gradients together, as a one-element tensor."""
        norm = self._norm_out(norm, stream)
        qml._check(self.lib.qml_opt_grad_norm(self._h, self._take(grads), grad_scale, norm.data_ptr(),
                                              self._stream(stream)), "qml_opt_grad_norm")
        return norm

    def sync(self, stream=None):
        qml._check(self.lib.qml_opt_sync(self._h, self._stream(stream)), "qml_opt_sync (device status)")

    @property
    def step_count(self) -> int:
        t = ctypes.c_longlong()
        qml._check(self.lib.qml_opt_get_step(self._h, ctypes.byref(t), self._stream(None)), "qml_opt_get_step")
        return t.value

    @step_count.setter
    def step_count(self, t: int):
        qml._check(self.lib.qml_opt_set_step(self._h, t, self._stream(None)), "qml_opt_set_step")

    @property
    def launch_count(self) -> int:
        return int(self.lib.qml_opt_launch_count(self._h))

    # ----------------------------------------------------------------- states
    def moments(self, i: int):
        """(m, v) of tensor i, in the shape of its parameter, as real numbers (new tensors)."""
        p, off = self.params[i], self.offsets[i]
        out = []
        for flat, scale, square in ((self.m, self.m_scale, False), (self.v, self.v_scale, True)):
            if scale is None:
                x = flat[off:off + p.numel()].clone()
            else:
                pad = -(-p.numel() // BLOCK) * BLOCK
                x = flat[off:off + pad].float().view(-1, BLOCK) * scale[off // BLOCK:(off + pad) // BLOCK, None]
                x = x.view(-1)[:p.numel()].clone()
                x = x.square_() if square else x
            out.append(x.view(p.shape))
        return tuple(out)

    def state_dict(self) -> dict:
        """Copies of the states, the master weights (None for tensors without) and the step
        count, for load_state."""
        d = {"step": self.step_count, "m": self.m.clone(), "v": self.v.clone()}
        if self.state == "8bit":
            d |= {"m_scale": self.m_scale.clone(), "v_scale": self.v_scale.clone()}
        d["master"] = [None if w is None else w.clone() for w in self.master]
        return d

    def load_state(self, d: dict):
        """Take the states, the master weights and the step count of state_dict() (on the
        current stream).  Parameters with master weights become their rounded copies; a
        dict without "master" leaves those as they are.  One that does not fit is refused
        (ValueError) and changes nothing."""
        import torch

        have = {"m": self.m, "v": self.v, "m_scale": self.m_scale, "v_scale": self.v_scale}
        for key, mine in have.items():
            x = d.get(key)
            if (x is None) != (mine is None):
                raise ValueError(f"{key}: states of another kind")
            if mine is not None and (x.shape != mine.shape or x.dtype != mine.dtype):
                raise ValueError(f"{key}: states of other tensors")
        master = list(d.get("master", self.master))
        if len(master) != len(self.master):
            raise ValueError(f"master: {len(master)} tensors for {len(self.master)}")
        for mine, x in zip(self.master, master):
            if (x is None) != (mine is None):
                raise ValueError("master: weights of a handle with other master weights")
            if mine is not None and (x.shape != mine.shape or x.dtype != mine.dtype):
                raise ValueError("master: weights of other tensors")
        step = int(d["step"])
        if step < 0:
            raise ValueError("step: a count of steps")
        with torch.no_grad():
            for key, mine in have.items():
                if mine is not None:
                    mine.copy_(d[key])
            if "master" in d:
                for p, mine, x in zip(self.params, self.master, master):
                    if mine is not None:
                        mine.copy_(x)
                        p.copy_(mine.view(p.shape))
        self.step_count = step
