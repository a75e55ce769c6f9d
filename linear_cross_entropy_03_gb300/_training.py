"""What a training step runs around the fused linear cross entropy: the norm in
front of the head, the gradients' norm, and the optimiser's step.

``ln_fwd``, ``ln_bwd``, ``grad_norm_raw`` and ``adamw_step`` marshal their
arguments for the C entry points; ``layer_norm``, ``layer_norm_backward``,
``grad_norm`` and ``AdamW`` take tensors, check them, allocate what is not given
and raise on an error status (in csrc/binding.cpp).  Memory that a call allocates belongs to the
stream that the call runs on; as with any torch operation, a tensor that was
written on another stream has to be waited for by the caller.

None of the calls records anything for autograd: their results have no graph, also
where their inputs require gradients, and ``layer_norm_backward`` is called by
the program that wants them.  What a call writes (``out`` and the like, an
optimiser's parameters and copies) counts as changed in place, so a graph that
had saved it refuses its backward pass.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import math
import os

from . import FlceError, _dt, _ptr, _stream, lib

NORM_KINDS = {"layer": 0, "rms": 1}
ADAMW_BLOCK = 256


class TensorEntry(ctypes.Structure):
    """flce_tensor_t"""
    _fields_ = [("data", ctypes.c_void_p), ("n", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class AdamWEntry(ctypes.Structure):
    """flce_adamw_tensor_t"""
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("exp_avg", ctypes.c_void_p),
                ("exp_avg_sq", ctypes.c_void_p), ("exp_avg_scale", ctypes.c_void_p),
                ("exp_avg_sq_scale", ctypes.c_void_p), ("copy", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("lr_scale", ctypes.c_float), ("weight_decay", ctypes.c_float), ("param_dtype", ctypes.c_int32),
                ("grad_dtype", ctypes.c_int32), ("copy_dtype", ctypes.c_int32), ("moment_bits", ctypes.c_int32)]


class AdamWNumbers(ctypes.Structure):
    """flce_adamw_t"""
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("step", ctypes.c_int64), ("step_dev", ctypes.c_void_p),
                ("lr_dev", ctypes.c_void_p), ("grad_scale_dev", ctypes.c_void_p), ("grad_scale", ctypes.c_float),
                ("skip_nonfinite", ctypes.c_int32), ("stochastic", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("seed", ctypes.c_uint64)]


# ------------------------------------------------------------------ raw ABI

def _kind(kind) -> int:
    return NORM_KINDS.get(kind, -1) if isinstance(kind, str) else int(kind)


def ln_workspace_size(N: int, H: int) -> int:
    return lib().ln_workspace_size(N, H)


def ln_fwd(kind, dtype, x, ld_x, residual, ld_residual, weight, bias, param_dtype, N, H, eps, y, ld_y, sum, ld_sum,
           mean, rstd, stream=None) -> int:
    return lib().ln_fwd(_kind(kind), _dt(dtype), _ptr(x), ld_x, _ptr(residual), ld_residual, _ptr(weight), _ptr(bias),
                        _dt(param_dtype), N, H, float(eps), _ptr(y), ld_y, _ptr(sum), ld_sum, _ptr(mean), _ptr(rstd),
                        _stream(stream))


def ln_bwd(kind, dtype, grad_y, ld_grad_y, x, ld_x, weight, param_dtype, mean, rstd, grad_sum, ld_grad_sum, N, H,
           grad_x, ld_grad_x, grad_weight, grad_bias, accumulate, workspace, workspace_bytes, stream=None) -> int:
    return lib().ln_bwd(_kind(kind), _dt(dtype), _ptr(grad_y), ld_grad_y, _ptr(x), ld_x, _ptr(weight),
                        _dt(param_dtype), _ptr(mean), _ptr(rstd), _ptr(grad_sum), ld_grad_sum, N, H, _ptr(grad_x),
                        ld_grad_x, _ptr(grad_weight), _ptr(grad_bias), int(accumulate), _ptr(workspace),
                        int(workspace_bytes), _stream(stream))


def grad_norm_workspace_size(count: int) -> int:
    return lib().grad_norm_workspace_size(count)


def grad_norm_raw(tensors, count, grad_scale, max_norm, eps, out, workspace, workspace_bytes, stream=None) -> int:
    """The C entry point grad_norm; `tensors` is an array of TensorEntry."""
    return lib().grad_norm(tensors, count, float(grad_scale), float(max_norm), float(eps), _ptr(out), _ptr(workspace),
                           int(workspace_bytes), _stream(stream))


def adamw_step(tensors, count, numbers, stream=None) -> int:
    """The C entry point; `tensors` is an array of AdamWEntry, `numbers` an AdamWNumbers."""
    return lib().adamw_step(tensors, count, None if numbers is None else ctypes.byref(numbers), _stream(stream))


# ------------------------------------------------------------------ tensors

_binding = None


def _native():
    """The extension that checks tensors and calls the library; raises if it has not been built."""
    global _binding
    if _binding is None:
        from . import _build
        lib()
        path = _build.binding_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`")
        loader = importlib.machinery.ExtensionFileLoader("flce_torch", path)
        spec = importlib.util.spec_from_file_location("flce_torch", path, loader=loader)
        module = importlib.util.module_from_spec(spec)
        loader.exec_module(module)
        module.set_error(FlceError)
        _binding = module
    return _binding


def _on(stream):
    """Makes `stream` torch's current one for a call, so that what it allocates is that stream's."""
    import torch
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


# ------------------------------------------------------------------ layer norm

def layer_norm(x, weight=None, bias=None, *, kind="layer", eps: float = 1e-5, residual=None, out=None, sum_out=None,
               row_stats: bool = True, stream=None) -> dict:
    """Layer norm over the last dimension of x (+ residual), or with ``kind="rms"`` its form without the mean.

    x [..., H] bf16, fp16 or fp32, its rows contiguous and one stride apart;
    residual of its shape and type, added first; weight and bias [H], each or
    both, of one of the three types.  Returns a dict with ``y``, ``sum`` (x +
    residual in the type of x, or None without residual), ``mean`` (fp32, None
    for rms) and ``rstd``, one a row (both None with ``row_stats=False``).
    ``out`` and ``sum_out`` may be x or residual.
    """
    if stream is not None:
        with _on(stream):
            return layer_norm(x, weight, bias, kind=kind, eps=eps, residual=residual, out=out, sum_out=sum_out,
                              row_stats=row_stats)
    y, total, mean, rstd = _native().layer_norm(x, weight, bias, _kind(kind), eps, residual, out, sum_out, row_stats)
    return {"y": y, "sum": total, "mean": mean, "rstd": rstd}


def layer_norm_backward(grad_y, x, weight=None, *, mean=None, rstd, kind="layer", grad_sum=None, grad_x: bool = True,
                        grad_weight: bool = True, grad_bias: bool = True, out=None, grad_weight_out=None,
                        grad_bias_out=None, accumulate: bool = False, workspace=None, stream=None) -> dict:
    """Gradients of layer_norm.

    x is what was normalised (``sum`` where there was a residual), mean and rstd
    are layer_norm's; ``grad_sum`` is the gradient that reaches ``sum`` from
    elsewhere.  Returns a dict with ``grad_x`` (the residual's gradient too),
    ``grad_weight`` and ``grad_bias`` (fp32 [H]; None where switched off).
    ``accumulate`` adds to ``grad_weight_out`` and ``grad_bias_out``.  ``out``
    may be grad_y, grad_sum or x.
    """
    if stream is not None:
        with _on(stream):
            return layer_norm_backward(grad_y, x, weight, mean=mean, rstd=rstd, kind=kind, grad_sum=grad_sum,
                                       grad_x=grad_x, grad_weight=grad_weight, grad_bias=grad_bias, out=out,
                                       grad_weight_out=grad_weight_out, grad_bias_out=grad_bias_out,
                                       accumulate=accumulate, workspace=workspace)
    gx, gw, gb = _native().layer_norm_backward(grad_y, x, weight, mean, rstd, _kind(kind), grad_sum, grad_x,
                                               grad_weight, grad_bias, out, grad_weight_out, grad_bias_out, accumulate,
                                               workspace)
    return {"grad_x": gx, "grad_weight": gw, "grad_bias": gb}


# ------------------------------------------------------------------ optimiser

def grad_norm(grads, *, max_norm=None, grad_scale: float = 1.0, eps: float = 1e-6, out=None, workspace=None,
              stream=None) -> dict:
    """The 2-norm of all of ``grads`` together, times ``grad_scale``, and the factor that clips it to ``max_norm``.

    Returns ``norm`` and ``scale``, one fp32 element each on the device: scale =
    grad_scale * min(1, max_norm / (norm + eps)), or NaN where the norm is not
    finite.  ``AdamW.step`` takes ``scale`` as it is, so nothing waits for the
    host.  Gradients may be bf16, fp16 or fp32 in any mixture; None is passed
    over.
    """
    if stream is not None:
        with _on(stream):
            return grad_norm(grads, max_norm=max_norm, grad_scale=grad_scale, eps=eps, out=out, workspace=workspace)
    max_norm = math.inf if max_norm is None else max_norm
    norm, scale = _native().grad_norm(grads, grad_scale, max_norm, eps, out, workspace)
    return {"norm": norm, "scale": scale}


def _each(value, count, where):
    """A number for every tensor, from one or from a sequence."""
    if isinstance(value, (int, float)):
        return [float(value)] * count
    value = [float(v) for v in value]
    if len(value) != count:
        raise FlceError(1, f"{where}: {len(value)} numbers for {count} tensors")
    return value


class AdamW:
    """AdamW over many tensors at once, with decoupled weight decay.

    params        contiguous bf16, fp16 or fp32 tensors, updated in place.  One that
                  is given other memory (``p.data = ...``, a model that was moved)
                  is followed, as is another tensor put into ``params``,
                  ``copies`` or the lists of moments; a captured step is not: it
                  goes on with the memory that it was captured with.
    weight_decay, lr_scale  one number, or one for each tensor.
    moments       "fp32", or "8bit": e4m3 numbers with an fp32 scale for each
                  block of 256; tensors below ``min_8bit_size`` elements keep
                  fp32 moments.
    seed          rounds 8-bit moments stochastically, so that changes smaller
                  than a number's spacing are kept on average; None: to nearest.
    copies        for each tensor another of its size that gets the rounded new
                  parameter (the 16-bit weight that products read), or None.
    state, step   moments and the number of steps already taken, from
                  ``state_dict()``; without them the moments start at 0.
    capturable    keeps the step's number on the device, so that ``step`` can be
                  captured in a graph and replayed.
    """

    def __init__(self, params, *, lr: float, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay=0.01, lr_scale=1.0,
                 moments: str = "fp32", min_8bit_size: int = 4096, copies=None, seed=None, state=None, step=None,
                 capturable: bool = False):
        import torch
        self.params = list(params)
        count = len(self.params)
        if moments not in ("fp32", "8bit"):
            raise FlceError(1, f"AdamW: moments {moments!r}")
        if not (0 <= betas[0] < 1 and 0 <= betas[1] < 1) or not 0 <= eps < math.inf or not math.isfinite(lr):
            raise FlceError(1, "AdamW: betas lie in [0, 1), eps is at least 0 and lr finite")
        if seed is not None and not 0 <= seed < 1 << 64:
            raise FlceError(1, "AdamW: seed is a whole number of 64 bits")
        decay, scale = _each(weight_decay, count, "AdamW: weight_decay"), _each(lr_scale, count, "AdamW: lr_scale")
        copies = [None] * count if copies is None else list(copies)
        if len(copies) != count:
            raise FlceError(1, f"AdamW: {len(copies)} copies for {count} tensors")
        self.lr, self.copies = lr, copies
        names = ("exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale")
        if state is not None:
            given = [list(state.get(k) or [None] * count) for k in names]
            if any(len(v) != count for v in given):
                raise FlceError(1, f"AdamW: state of another number of tensors than {count}")
            step = state.get("step", 0) if step is None else step
        else:
            given = [[None] * count for _ in names]
        step = 0 if step is None else int(step)
        if step < 0:
            raise FlceError(1, "AdamW: a negative step")
        if state is None:
            for i, p in enumerate(self.params):
                small = moments == "8bit" and p.numel() >= min_8bit_size
                kind = torch.float8_e4m3fn if small else torch.float32
                given[0][i], given[1][i] = (torch.zeros(p.shape, dtype=kind, device=p.device) for _ in range(2))
                if small:
                    blocks = -(-p.numel() // ADAMW_BLOCK)
                    given[2][i], given[3][i] = (torch.zeros(blocks, device=p.device) for _ in range(2))
        self.exp_avg, self.exp_avg_sq, self.exp_avg_scale, self.exp_avg_sq_scale = given
        self._table = (AdamWEntry * count)()
        self._numel = (ctypes.c_int64 * count)()
        _native().adamw_table(ctypes.addressof(self._table), ctypes.addressof(self._numel), self.params, *given, copies,
                              decay, scale)
        self._numbers = AdamWNumbers(beta1=betas[0], beta2=betas[1], eps=eps, stochastic=int(seed is not None),
                                     seed=seed or 0)
        self._addresses = (ctypes.addressof(self._table), ctypes.addressof(self._numel), count,
                           ctypes.addressof(self._numbers))
        self._steps = step
        self._step_dev = torch.full((1,), step, dtype=torch.int64, device="cuda") if capturable else None
        if capturable:
            self._numbers.step_dev = self._step_dev.data_ptr()

    @property
    def steps(self) -> int:
        """Steps taken; with ``capturable`` this reads the device and waits for it."""
        return self._steps if self._step_dev is None else int(self._step_dev.item())

    def state_dict(self) -> dict:
        """The moments (the tensors themselves) and the number of steps: what ``state`` takes."""
        return dict(step=self.steps, exp_avg=self.exp_avg, exp_avg_sq=self.exp_avg_sq,
                    exp_avg_scale=self.exp_avg_scale, exp_avg_sq_scale=self.exp_avg_sq_scale)

    def step(self, grads, *, lr=None, grad_scale=None, skip_nonfinite: bool = False, stream=None) -> None:
        """One step.  ``grads``: a contiguous tensor of each parameter's size, or None to leave it out.

        lr           a number (default: the constructor's) or a device fp32 element.
        grad_scale   what the gradients are multiplied by: a number or a device
                     fp32 element, as ``grad_norm`` leaves it.
        skip_nonfinite  writes nothing when that factor is not finite.  Such a
                     step does not count, unless the factor lies on the device
                     and the step's number does not (``capturable``): the host
                     cannot know then.
        """
        import torch
        if stream is not None:
            with _on(stream):
                return self.step(grads, lr=lr, grad_scale=grad_scale, skip_nonfinite=skip_nonfinite)
        lr = self.lr if lr is None else lr
        if skip_nonfinite and grad_scale is not None and not isinstance(grad_scale, torch.Tensor) and \
                not math.isfinite(grad_scale):
            return
        if self._step_dev is not None:
            if self._step_dev.get_device() != torch.cuda.current_device():
                raise FlceError(1, "AdamW.step: its number of steps lies on another GPU")
            # counted on the device, and not at all where the step is skipped; taken back if the call is refused
            on_device = skip_nonfinite and isinstance(grad_scale, torch.Tensor)
            one = torch.isfinite(grad_scale).reshape(-1)[:1].to(torch.int64) if on_device else 1
            self._step_dev.add_(one)
        try:
            _native().adamw(*self._addresses, grads, lr, grad_scale, skip_nonfinite, self._steps + 1, self.params,
                            self.exp_avg, self.exp_avg_sq, self.exp_avg_scale, self.exp_avg_sq_scale, self.copies)
        except Exception:
            if self._step_dev is not None:
                self._step_dev.sub_(one)
            raise
        self._steps += 1
