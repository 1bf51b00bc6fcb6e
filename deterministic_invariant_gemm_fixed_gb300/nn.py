"""PyTorch layer over the C ABI: a linear layer whose three matmuls and bias
gradient run in libbi's deterministic kernels.

Sources: sgemm-bi 0.1.1.post2, "Use" -- a drop-in `Linear(in, out, ...,
tensor_cores=...)` whose weight is stored [in, out], `Linear.from_torch` for
converting existing layers, and the functional `deterministic_linear(x,
weight, bias, tensor_cores)`; ViperLLM ffma.py, `_FFMAAddmm` -- an autograd
function that saves the original x and W and returns gx = gy W^T, gW = x^T gy
and gb = column sums of gy.

Everything numeric happens in the library: this module only reshapes tensors,
allocates outputs with torch and passes pointers and the current stream.  The
bias gradient comes from bi_bias_grad (fixed-order column sum) instead of
torch's reduction, so a whole training step is bit-reproducible.

FP8 route (AstrAI csrc/kernels/fp8_mm.cu, fp8_linear_forward_scaled and
fp8_linear_backward_scaled): with `fp8=Fp8Scales(...)`, the forward quantizes
x and the weight to e4m3 with the caller's per-tensor scales (codes =
e4m3(value / scale)), multiplies the codes on the tensor cores and scales the
f32 product by scale_x * scale_w, then adds the bias and rounds once; the
backward quantizes the output gradient with scale_g and computes dX and dW from
the saved codes the same way.  The bias gradient is the fixed-order column sum
of the unquantized output gradient.

FP4 route: with `fp4=True` the three matmuls run on MXFP4 codes of x, the weight and
the output gradient, each operand quantized along that product's contraction (blocks
of 32 with a power-of-two scale taken from the block, so there are no scales to pass);
the backward keeps codes of x and the weight in place of the tensors.

Beside the layer: `adapter_linear` (a shared projection with the low-rank adapter
of each row), `route` (a router's expert choice, weights, counts and balance
loss, whose ids the grouped matmul takes), `clip_grad_norm_` (global gradient
norm and clipping of a parameter list) and `moe` (router and experts of a decoding
step, with weights of x's type or in MXFP4), each over its own entry points of the
library, so a program made of them is bit-reproducible too.

Calls are asynchronous.  A kernel whose wait for its own copies ran out stops with its
results unfinished; no function here asks for that, which would synchronize:
`engine_for(device).check()` does, and raises BiError.
"""
from __future__ import annotations

import dataclasses
import math
import threading

import torch
from torch.autograd.function import once_differentiable

from . import Engine, TensorSet, fp4_buffers

_engines: dict[int, Engine] = {}
_engines_lock = threading.Lock()


def engine_for(device: torch.device) -> Engine:
    """One engine per CUDA device, created on first use."""
    idx = device.index if device.index is not None else torch.cuda.current_device()
    with _engines_lock:
        eng = _engines.get(idx)
        if eng is None:
            eng = Engine(idx)
            _engines[idx] = eng
        return eng


def _check(x: torch.Tensor, weight: torch.Tensor, bias):
    if not (x.is_cuda and weight.is_cuda):
        raise ValueError("deterministic_linear needs CUDA tensors")
    if x.dtype != weight.dtype or (bias is not None and bias.dtype != x.dtype):
        raise TypeError("x, weight and bias must share one dtype (float32, bfloat16 or float16)")
    if weight.dim() != 2 or x.shape[-1] != weight.shape[0]:
        raise ValueError(f"weight must be [in, out] with in = x.shape[-1]; got {tuple(weight.shape)}")
    if bias is not None and bias.shape != (weight.shape[1],):
        raise ValueError("bias must be [out]")


class _DeterministicLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, tensor_cores):
        _check(x, weight, bias)
        k, n = weight.shape
        x2 = x.reshape(-1, k).contiguous()
        w = weight.contiguous()
        b = bias.contiguous() if bias is not None else None
        m = x2.shape[0]
        y = torch.empty(m, n, dtype=x.dtype, device=x.device)
        eng = engine_for(x.device)
        eng.forward(y, x2, w, b, m, k, n, x.dtype, torch.cuda.current_stream(x.device), int(tensor_cores))
        ctx.save_for_backward(x2, w)
        ctx.has_bias = bias is not None
        ctx.tensor_cores = int(tensor_cores)
        ctx.x_shape = x.shape
        return y.reshape(*x.shape[:-1], n)

    @staticmethod
    def backward(ctx, gy):
        x2, w = ctx.saved_tensors
        k, n = w.shape
        gy2 = gy.reshape(-1, n).to(w.dtype).contiguous()
        m = gy2.shape[0]
        eng = engine_for(w.device)
        stream = torch.cuda.current_stream(w.device)
        tc = ctx.tensor_cores
        gx = gw = gb = None
        if ctx.needs_input_grad[0]:
            gx = torch.empty(m, k, dtype=w.dtype, device=w.device)
            eng.backward_dx(gx, gy2, w, m, k, n, w.dtype, stream, tc)
            gx = gx.reshape(ctx.x_shape)
        if ctx.needs_input_grad[1]:
            gw = torch.empty(k, n, dtype=w.dtype, device=w.device)
            eng.backward_dw(gw, int(w.dtype == torch.float32), x2, gy2, m, k, n, w.dtype, stream, tc)
        if ctx.has_bias and ctx.needs_input_grad[2]:
            gb = torch.empty(n, dtype=w.dtype, device=w.device)
            eng.bias_grad(gb, int(w.dtype == torch.float32), gy2, m, n, w.dtype, stream)
        return gx, gw, gb, None


@dataclasses.dataclass
class Fp8Scales:
    """Per-tensor scales of the FP8 route: a value v is stored as the e4m3 code
    of v / scale.  Each scale is a float or a one-element float32 CUDA tensor.
    `amax`, if given, is a float32 CUDA tensor of 3 elements that receives the
    maximum |value| of x and of the weight (forward) and of the output gradient
    (backward), for a caller that derives the next step's scales from them."""
    scale_x: float | torch.Tensor
    scale_w: float | torch.Tensor
    scale_g: float | torch.Tensor
    amax: torch.Tensor | None = None


def _scale_pair(s, device):
    """(scale, 1 / scale) as one-element f32 tensors on device (the reciprocal is
    taken by torch on the device; power-of-two scales have exact reciprocals)."""
    t = (s if isinstance(s, torch.Tensor) else torch.tensor([float(s)])).to(device=device, dtype=torch.float32)
    t = t.reshape(1).contiguous()
    return t, torch.reciprocal(t)


def _amax_slot(amax, i, device):
    if amax is None:
        return torch.empty(1, dtype=torch.float32, device=device)
    if not (amax.is_cuda and amax.dtype == torch.float32 and amax.numel() == 3 and amax.is_contiguous()):
        raise ValueError("Fp8Scales.amax must be a contiguous float32 CUDA tensor of 3 elements")
    return amax[i:i + 1]


class _DeterministicLinearFp8(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, fp8):
        _check(x, weight, bias)
        if x.dtype not in (torch.bfloat16, torch.float16):
            raise TypeError("the FP8 route takes bfloat16 or float16 x and weight")
        k, n = weight.shape
        x2 = x.reshape(-1, k).contiguous()
        w = weight.contiguous()
        b = bias.contiguous() if bias is not None else None
        m = x2.shape[0]
        dev = x.device
        eng = engine_for(dev)
        stream = torch.cuda.current_stream(dev)
        sx, sx_inv = _scale_pair(fp8.scale_x, dev)
        sw, sw_inv = _scale_pair(fp8.scale_w, dev)
        xq = torch.empty(m, k, dtype=torch.uint8, device=dev)
        wq = torch.empty(k, n, dtype=torch.uint8, device=dev)
        eng.fp8_quantize(xq, _amax_slot(fp8.amax, 0, dev), x2, sx_inv, m * k, x.dtype, stream)
        eng.fp8_quantize(wq, _amax_slot(fp8.amax, 1, dev), w, sw_inv, k * n, x.dtype, stream)
        y = torch.empty(m, n, dtype=x.dtype, device=dev)
        eng.fp8_forward(y, xq, wq, b, sx, sw, m, k, n, x.dtype, stream)
        ctx.save_for_backward(xq, wq, sx, sw)
        ctx.fp8 = fp8
        ctx.dtype = x.dtype
        ctx.has_bias = bias is not None
        ctx.x_shape = x.shape
        return y.reshape(*x.shape[:-1], n)

    @staticmethod
    def backward(ctx, gy):
        xq, wq, sx, sw = ctx.saved_tensors
        k, n = wq.shape
        dt = ctx.dtype
        gy2 = gy.reshape(-1, n).to(dt).contiguous()
        m = gy2.shape[0]
        dev = wq.device
        eng = engine_for(dev)
        stream = torch.cuda.current_stream(dev)
        sg, sg_inv = _scale_pair(ctx.fp8.scale_g, dev)
        gq = torch.empty(m, n, dtype=torch.uint8, device=dev)
        eng.fp8_quantize(gq, _amax_slot(ctx.fp8.amax, 2, dev), gy2, sg_inv, m * n, dt, stream)
        gx = gw = gb = None
        if ctx.needs_input_grad[0]:
            gx = torch.empty(m, k, dtype=dt, device=dev)
            eng.fp8_backward_dx(gx, gq, wq, sg, sw, m, k, n, dt, stream)
            gx = gx.reshape(ctx.x_shape)
        if ctx.needs_input_grad[1]:
            gw = torch.empty(k, n, dtype=dt, device=dev)
            eng.fp8_backward_dw(gw, xq, gq, sx, sg, m, k, n, dt, stream)
        if ctx.has_bias and ctx.needs_input_grad[2]:
            gb = torch.empty(n, dtype=dt, device=dev)
            eng.bias_grad(gb, 0, gy2, m, n, dt, stream)
        return gx, gw, gb, None


class _DeterministicLinearFp4(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        _check(x, weight, bias)
        k, n = weight.shape
        x2 = x.reshape(-1, k).contiguous()
        w = weight.contiguous()
        b = bias.contiguous() if bias is not None else None
        m, dt, dev = x2.shape[0], x.dtype, x.device
        eng, stream = engine_for(dev), torch.cuda.current_stream(dev)
        need_x, need_w = ctx.needs_input_grad[0], ctx.needs_input_grad[1]
        xq, wq = fp4_buffers(m, k, dev), fp4_buffers(n, k, dev)
        xt = fp4_buffers(k, m, dev) if need_w else (None, None)
        wt = fp4_buffers(k, n, dev) if need_x else (None, None)
        eng.fp4_quantize(*xq, *xt, x2, m, k, dt, stream)
        eng.fp4_quantize(*wt, *wq, w, k, n, dt, stream)
        y = torch.empty(m, n, dtype=dt, device=dev)
        eng.fp4_forward(y, *xq, *wq, b, m, k, n, dt, stream)
        ctx.save_for_backward(*xt, *wt)
        ctx.sizes, ctx.dtype, ctx.has_bias, ctx.x_shape = (m, k, n), dt, bias is not None, x.shape
        return y.reshape(*x.shape[:-1], n)

    @staticmethod
    @once_differentiable  # a second derivative is refused, not left out
    def backward(ctx, gy):
        xt, xts, wt, wts = ctx.saved_tensors
        (m, k, n), dt = ctx.sizes, ctx.dtype
        gy2 = gy.reshape(-1, n).to(dt).contiguous()
        dev = gy2.device
        eng, stream = engine_for(dev), torch.cuda.current_stream(dev)
        gq = fp4_buffers(m, n, dev) if wt is not None else (None, None)
        gt = fp4_buffers(n, m, dev) if xt is not None else (None, None)
        if wt is not None or xt is not None:
            eng.fp4_quantize(*gq, *gt, gy2, m, n, dt, stream)
        gx = gw = gb = None
        if wt is not None:
            gx = torch.empty(m, k, dtype=dt, device=dev)
            eng.fp4_backward_dx(gx, *gq, wt, wts, m, k, n, dt, stream)
            gx = gx.reshape(ctx.x_shape)
        if xt is not None:
            gw = torch.empty(k, n, dtype=dt, device=dev)
            eng.fp4_backward_dw(gw, xt, xts, *gt, m, k, n, dt, stream)
        if ctx.has_bias and ctx.needs_input_grad[2]:
            gb = torch.empty(n, dtype=dt, device=dev)
            eng.bias_grad(gb, int(dt == torch.float32), gy2, m, n, dt, stream)
        return gx, gw, gb


def deterministic_linear(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None,
                         tensor_cores: bool = True, fp8: Fp8Scales | None = None, fp4: bool = False) -> torch.Tensor:
    """y = x @ weight (+ bias) with weight [in, out]; bit-reproducible forward and
    backward (scalar tier with tensor_cores=False, tcgen05 tier otherwise).
    With fp8 (Fp8Scales), the three matmuls run on e4m3 codes of x, the weight
    and the output gradient, quantized with the given per-tensor scales, on the
    tensor cores (tensor_cores is then ignored).  With fp4, on MXFP4 codes of them
    (any sizes and types; likewise).  The gradients are those of the products, with
    the rounding to codes passed through."""
    if fp4:
        if fp8 is not None:
            raise ValueError("deterministic_linear: fp8 and fp4 exclude each other")
        return _DeterministicLinearFp4.apply(x, weight, bias)
    if fp8 is not None:
        return _DeterministicLinearFp8.apply(x, weight, bias, fp8)
    return _DeterministicLinear.apply(x, weight, bias, tensor_cores)


class Linear(torch.nn.Module):
    """Linear layer with the weight stored [in, out] (the layout the library's
    matmuls read without a transpose)."""

    def __init__(self, in_features: int, out_features: int, bias: bool = True, device=None,
                 dtype=None, tensor_cores: bool = True):
        super().__init__()
        self.in_features, self.out_features = in_features, out_features
        self.tensor_cores = tensor_cores
        self.weight = torch.nn.Parameter(torch.empty(in_features, out_features, device=device, dtype=dtype))
        self.bias = torch.nn.Parameter(torch.empty(out_features, device=device, dtype=dtype)) if bias else None
        self.reset_parameters()

    def reset_parameters(self):
        # the usual uniform(-1/sqrt(in), 1/sqrt(in)) initialisation of a linear layer
        bound = 1.0 / math.sqrt(self.in_features)
        with torch.no_grad():
            self.weight.uniform_(-bound, bound)
            if self.bias is not None:
                self.bias.uniform_(-bound, bound)

    @classmethod
    def from_torch(cls, layer: torch.nn.Linear, tensor_cores: bool = True) -> "Linear":
        """Convert a torch.nn.Linear (weight [out, in]) into this layout."""
        new = cls(layer.in_features, layer.out_features, bias=layer.bias is not None,
                  device=layer.weight.device, dtype=layer.weight.dtype, tensor_cores=tensor_cores)
        with torch.no_grad():
            new.weight.copy_(layer.weight.t())
            if layer.bias is not None:
                new.bias.copy_(layer.bias)
        return new

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return deterministic_linear(x, self.weight, self.bias, self.tensor_cores)

    def extra_repr(self) -> str:
        return (f"in_features={self.in_features}, out_features={self.out_features}, "
                f"bias={self.bias is not None}, tensor_cores={self.tensor_cores}")


class _AdapterLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, a, b, scales, ids, tensor_cores):
        _check(x, weight, bias)
        k, n = weight.shape
        if a.dim() != 3 or b.dim() != 3 or a.shape[2] != k or b.shape != (a.shape[0], a.shape[1], n):
            raise ValueError("a must be [adapters, rank, in] and b [adapters, rank, out]")
        if a.dtype != x.dtype or b.dtype != x.dtype:
            raise TypeError("x, weight, a and b must share one dtype")
        g, r, _ = a.shape
        if ids.dtype not in (torch.int32, torch.uint32) or ids.shape != x.shape[:-1]:
            raise ValueError("ids must be int32 or uint32, one per row of x")
        if scales is not None and (scales.dtype != torch.float32 or scales.shape != (g,)):
            raise ValueError("scales must be float32 [adapters]")
        if not all(t is None or (t.is_cuda and t.device == x.device) for t in (a, b, scales, ids)):
            raise ValueError("adapter_linear needs all tensors on x's CUDA device")
        x2, w, a, b = x.reshape(-1, k).contiguous(), weight.contiguous(), a.contiguous(), b.contiguous()
        ids2 = ids.reshape(-1).contiguous()
        sc = scales.contiguous() if scales is not None else None
        m = x2.shape[0]
        y = torch.empty(m, n, dtype=x.dtype, device=x.device)
        h = torch.empty(m, r, dtype=torch.float32, device=x.device)
        engine_for(x.device).adapter_forward(y, h, x2, w, bias.contiguous() if bias is not None else None, a, b, sc, ids2,
                                             m, k, n, r, g, x.dtype, torch.cuda.current_stream(x.device), int(tensor_cores))
        ctx.save_for_backward(x2, w, a, b, sc, ids2, h)
        ctx.has_bias, ctx.tensor_cores, ctx.x_shape = bias is not None, int(tensor_cores), x.shape
        return y.reshape(*x.shape[:-1], n)

    @staticmethod
    @once_differentiable  # a second derivative is refused, not left out
    def backward(ctx, gy):
        x2, w, a, b, sc, ids2, h = ctx.saved_tensors
        (k, n), (g, r, _) = w.shape, a.shape
        dt, dev, m = w.dtype, w.device, x2.shape[0]
        gy2 = gy.reshape(-1, n).to(dt).contiguous()
        eng, stream, tc = engine_for(dev), torch.cuda.current_stream(dev), ctx.tensor_cores
        need = ctx.needs_input_grad
        gx = torch.empty(m, k, dtype=dt, device=dev) if need[0] else None
        ga = torch.empty(g, r, k, dtype=torch.float32, device=dev) if need[3] else None
        gb = torch.empty(g, r, n, dtype=torch.float32, device=dev) if need[4] else None
        eng.adapter_backward(gx, ga, gb, x2, h, w, gy2, a, b, sc, ids2, m, k, n, r, g, dt, stream, tc)
        gw = gbias = None
        f32 = int(dt == torch.float32)
        if need[1]:
            gw = torch.empty(k, n, dtype=dt, device=dev)
            eng.backward_dw(gw, f32, x2, gy2, m, k, n, dt, stream, tc)
        if ctx.has_bias and need[2]:
            gbias = torch.empty(n, dtype=dt, device=dev)
            eng.bias_grad(gbias, f32, gy2, m, n, dt, stream)
        return (gx.reshape(ctx.x_shape) if gx is not None else None, gw, gbias, ga.to(dt) if ga is not None else None,
                gb.to(dt) if gb is not None else None, None, None, None)


def adapter_linear(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None, a: torch.Tensor, b: torch.Tensor,
                   scales: torch.Tensor | None, ids: torch.Tensor, tensor_cores: bool = True) -> torch.Tensor:
    """y = x @ weight (+ bias) + scales[g] * (x @ a[g].T) @ b[g] with g = ids[row]:
    weight [in, out] shared by all rows, adapters a [G, rank, in] and b [G, rank,
    out], scales [G] float32 (None: 1), ids int32 or uint32 of x's leading shape;
    a row whose id is outside [0, G) gets the shared projection alone.  Gradients
    for x, weight, bias, a and b; a row's y and dx do not depend on other rows.
    scales are constants: one that requires a gradient is refused (fold a trained
    scale into b instead)."""
    if scales is not None and scales.requires_grad and torch.is_grad_enabled():
        raise ValueError("adapter_linear has no gradient for scales: pass scales.detach(), or fold them into b")
    return _AdapterLinear.apply(x, weight, bias, a, b, scales, ids, tensor_cores)


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, normalize, valid):
        if not logits.is_cuda:
            raise ValueError("route needs CUDA tensors")
        e = logits.shape[-1]
        x = logits.reshape(-1, e).contiguous()
        t, dev = x.shape[0], x.device
        if valid is not None:
            if valid.shape != logits.shape[:-1] or valid.dtype not in (torch.bool, torch.uint8) or valid.device != dev:
                raise ValueError("valid must be bool or uint8, one per row of logits")
            valid = valid.reshape(-1).contiguous()
        def new(*shape, dtype=torch.float32):
            return torch.empty(*shape, dtype=dtype, device=dev)
        ids, weights, lse = new(t, k, dtype=torch.int32), new(t, k), new(t)
        counts, rows, mean, loss = new(e, dtype=torch.int32), new(1, dtype=torch.int32), new(e), new(1)
        engine_for(dev).router_forward(ids, weights, counts, rows, mean, loss, lse, x, valid, t, e, k, normalize, x.dtype,
                                       torch.cuda.current_stream(dev))
        ctx.save_for_backward(x, lse, ids, weights, counts, rows)
        ctx.k, ctx.normalize, ctx.shape = k, normalize, logits.shape
        ids_out, counts_out = ids.reshape(*logits.shape[:-1], k), counts.clone()
        ctx.mark_non_differentiable(ids_out, counts_out)
        return ids_out, weights.clone().reshape(*logits.shape[:-1], k), loss.reshape(()), counts_out

    @staticmethod
    @once_differentiable
    def backward(ctx, _ids, gweights, gloss, _counts):
        x, lse, ids, weights, counts, rows = ctx.saved_tensors
        t, e = x.shape
        d = torch.empty_like(x)
        gw = gweights.reshape(t, ctx.k).float().contiguous() if gweights is not None else None
        gl = gloss.reshape(1).float().contiguous() if gloss is not None else None
        engine_for(x.device).router_backward(d, x, lse, ids, weights, counts, rows, gw, gl, t, e, ctx.k, ctx.normalize,
                                             x.dtype, torch.cuda.current_stream(x.device))
        return d.reshape(ctx.shape), None, None, None


def route(logits: torch.Tensor, k: int, normalize: bool = True, valid: torch.Tensor | None = None):
    """A softmax router's choice of k experts per row of logits [..., E]: (ids int32
    [..., k], weights float32 [..., k], balance loss [], counts int32 [E]).  ids of
    rows with valid = 0 are E, which the grouped matmul takes as padding; the loss is
    E * sum_e (counts_e / kV) * mean_t p_te over the V rows that take part.
    Gradients of the weights and the loss reach the logits."""
    return _Route.apply(logits, k, normalize, valid)


@dataclasses.dataclass
class Fp4Weight:
    """Expert weights [E, rows, length] kept in MXFP4 along their last dimension."""
    codes: torch.Tensor
    scales: torch.Tensor
    shape: tuple[int, int, int]

    @classmethod
    def quantize(cls, w: torch.Tensor) -> "Fp4Weight":
        if w.dim() != 3 or not w.is_cuda:
            raise ValueError("Fp4Weight needs a CUDA tensor [experts, rows, length]")
        e, r, n = w.shape
        q, s = fp4_buffers(e * r, n, w.device)
        engine_for(w.device).fp4_quantize(q, s, None, None, w.detach().contiguous(), e * r, n, w.dtype,
                                          torch.cuda.current_stream(w.device))
        return cls(q, s, (e, r, n))

    def dequantize(self, dtype=torch.float32) -> torch.Tensor:
        out = torch.empty(self.shape, dtype=dtype, device=self.codes.device)
        e, r, n = self.shape
        engine_for(out.device).fp4_dequantize(out, self.codes, self.scales, e * r, n, dtype,
                                              torch.cuda.current_stream(out.device))
        return out


def moe(x: torch.Tensor, logits: torch.Tensor, w_gate, w_up, w_down, k: int, normalize: bool = True,
        valid: torch.Tensor | None = None, activation: str = "silu") -> torch.Tensor:
    """A mixture-of-experts layer on the tokens x [..., in] of a decoding step, routed by
    logits [..., E] (see `route`): y = sum over the k chosen experts of their weight times
    (act(x w_gate[e].T) * (x w_up[e].T)) w_down[e].T, with w_gate and w_up [E, hidden, in]
    (w_gate None: act(x w_up[e].T)) and w_down [E, out, hidden], all tensors of x's dtype
    or all Fp4Weight.  activation: "silu", "gelu" (the tanh form) or "relu".  Rows with
    valid = 0 get zeros.  A row's y does not depend on the rows beside it; more than
    2048 / k tokens go in several calls, where `route` and the grouped matmul are
    faster.  Forward only: tensors that require a gradient are refused.  A device-side
    error is raised by engine_for(x.device).check(), after one call or many."""
    weights = [w for w in (w_gate, w_up, w_down) if w is not None]
    fp4 = isinstance(w_up, Fp4Weight)
    if any(isinstance(w, Fp4Weight) != fp4 for w in weights):
        raise ValueError("moe: the expert weights must be all tensors or all Fp4Weight")
    if not x.is_cuda or not logits.is_cuda or logits.device != x.device:
        raise ValueError("moe needs CUDA tensors on one device")
    if torch.is_grad_enabled() and any(isinstance(t, torch.Tensor) and t.requires_grad for t in (x, logits, *weights)):
        raise ValueError("moe has no backward: train with route and the grouped matmul, or call it under no_grad")
    (e, f, n_in), (_, n_out, _) = w_up.shape, w_down.shape
    if tuple(w_down.shape) != (e, n_out, f) or (w_gate is not None and tuple(w_gate.shape) != (e, f, n_in)):
        raise ValueError("moe: w_gate and w_up must be [E, hidden, in] and w_down [E, out, hidden]")
    if x.shape[-1] != n_in or logits.shape != (*x.shape[:-1], e):
        raise ValueError("moe: x must be [..., in] and logits [..., E]")
    if any((w.codes if fp4 else w).device != x.device for w in weights) or (not fp4 and any(w.dtype != x.dtype for w in weights)):
        raise ValueError("moe: the expert weights must be on x's device and, unless quantized, of its dtype")
    dev, dt = x.device, x.dtype
    x2, l2 = x.reshape(-1, n_in).contiguous(), logits.reshape(-1, e).contiguous()
    t = x2.shape[0]
    if valid is not None:
        if valid.shape != x.shape[:-1] or valid.dtype not in (torch.bool, torch.uint8) or valid.device != dev:
            raise ValueError("valid must be bool or uint8, one per row of x")
        valid = valid.reshape(-1).contiguous()
    eng, stream = engine_for(dev), torch.cuda.current_stream(dev)
    def new(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device=dev)
    ids, p = new(t, k, dtype=torch.int32), new(t, k)
    eng.router_forward(ids, p, new(e, dtype=torch.int32), new(1, dtype=torch.int32), new(e), new(1), new(t), l2, valid, t, e, k,
                       normalize, l2.dtype, stream)
    y = new(t, n_out, dtype=dt)
    if fp4:
        args = [v for w in (w_gate, w_up, w_down) for v in ((w.codes, w.scales) if w is not None else (None, None))]
        call = eng.moe_forward_fp4
    else:
        args = [w.contiguous() if w is not None else None for w in (w_gate, w_up, w_down)]
        call = eng.moe_forward
    step = max(1, 2048 // k)
    for i in range(0, t, step):
        rows = slice(i, min(t, i + step))
        call(y[rows], x2[rows], ids[rows], p[rows], *args, rows.stop - i, k, n_in, f, n_out, e, activation, dt, stream)
    return y.reshape(*x.shape[:-1], n_out)


def clip_grad_norm_(parameters, max_norm: float) -> torch.Tensor:
    """Scale the gradients of `parameters` in place so that their global norm is at
    most max_norm; returns the norm before (a float32 tensor of one element, on the
    device; nothing synchronises).  The gradients must be contiguous, on one device,
    and each parameter is given once."""
    params = [parameters] if isinstance(parameters, torch.Tensor) else list(parameters)
    grads = [p.grad for p in params if p.grad is not None]
    if not grads:
        return torch.zeros(1, device=params[0].device if params else None)
    dev = grads[0].device
    if any(g.device != dev for g in grads):
        raise ValueError("clip_grad_norm_: gradients must be on one device")
    norm = torch.empty(1, dtype=torch.float32, device=dev)
    s = TensorSet(grads)
    engine_for(dev).clip_gradients(s, s, norm, max_norm, torch.cuda.current_stream(dev))
    return norm
