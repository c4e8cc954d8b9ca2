"""PyTorch modules over the library: a quantize-once convolution for training and inference.

``MQConv2d`` is a drop-in ``nn.Conv2d`` (groups 1, dilation 1, no bias) whose three GEMMs run
through the library, following the onedev.kr MicroQonv digest (sections "How it works" and "How it
differs"):

  forward   X (NCHW) -> quantized channel-batch-first squares  } one batched call
            W (OIHW) -> quantized tap-major squares             } (quantize once, RNE)
            Y = conv_fwd(Xq, Wq), back to NCHW
  backward  G_Y (NCHW) -> quantized channel-batch-first squares, one call (quantize once, SR)
            G_W = conv_wgrad(G_Yq, Xq) (the forward's Xq is kept, not re-quantized)
            G_X = conv_dgrad(Wq, G_Yq)   (the forward's Wq is kept)

so each of X, W and G_Y is quantized exactly once per step and reused by both GEMMs that read it.
Every layout change, quantization and GEMM is a library call on torch's current stream; the
module only allocates buffers and marshals arguments. Batch norm, activations, residual adds,
pooling and the first and last layers stay in PyTorch fp32, the precision policy the digest's
experiments use for the layers it does not quantize.

Stochastic rounding draws its bits from a seed per call: ``seed_base + layer_index +
layers * step`` with ``step`` counted by the module (one per training forward), so a run is
reproducible, and no two layers or steps share a stream of random bits where every layer of a model
has a number of its own in 0 .. ``layers`` - 1. An ``MXGatedMLP`` takes two: block i of ``layers``
blocks is numbers 2i and 2i + 1 of 2 ``layers``. ``number_layers`` numbers a model of several kinds.
A captured step replays the seeds that it was captured with.

In eval mode with ``cache_weight=True`` the weight is quantized once and reused until the
parameter changes (its version counter moves): the inference path then quantizes only
activations. (The modules on 4 bits: until one of the other changes that ``_MXModule`` names,
too, and not in a captured graph, which quantizes the weight in every replay.)

``MXLinear`` and ``MXGatedMLP`` are the linear layer and the gated feed-forward block of a
transformer on microscaled 4-bit operands (E2M1, a power-of-two scale per 32 elements along the
contracted dimension). A training step reads each weight once for both of its directions, and the
forward pass keeps the input in 4 bits along its columns instead of itself:

  forward   W -> rows and columns (one call); Y = mq_mx4_linear(X, W rows), which also leaves X's columns
  backward  G_Y -> rows and columns (one call, SR); G_X from W's columns, G_W from X's
"""
from __future__ import annotations

from typing import List, Optional, Sequence, Tuple

import torch
from torch import nn

from . import (MQ_NVFP4, MX4, MQ_QUANTIZE_WS_BYTES, MQ_ROLE_ACT, MQ_ROLE_GRAD, MQ_ROLE_WEIGHT,
               MQ_RNE, MQ_SR, MQ_SRC_NCHW, MQ_SRC_OIHW, QTensor, mq_conv_backward,
               mq_conv_dgrad, mq_conv_fwd, mq_conv_wgrad, mq_quantize_batch, mq_quantize_nchw, mq_quantize_weight,
               mq_mx4_gated, mq_mx4_gated_backward, mq_mx4_linear, mq_mx4_linear_backward,
               mq_mx4_quantize, mq_relayout_cbf, mq_relayout_weight, mq_wgrad_workspace_bytes,
               mx4_gated_backward_workspace, mx4_gated_workspace, mx4_linear_backward_workspace,
               mx4_linear_workspace, out_hw, quant_job)


def _check_input(t: torch.Tensor, what: str, ndim: int = 4):
    if not t.is_cuda or t.dtype != torch.float32 or t.dim() != ndim:
        raise ValueError(f"{what}: expected a {ndim}-D float32 CUDA tensor, got "
                         f"{tuple(t.shape)} {t.dtype} on {t.device}")


def quantize_weight(weight: torch.Tensor, fmt: int, ws: torch.Tensor) -> QTensor:
    """OIHW fp32 weight -> quantized tap-major weight (RNE), one library call."""
    Cout, Cin, Kh, Kw = weight.shape
    qw = QTensor(Kh, Kw, Cout, Cin, fmt, MQ_ROLE_WEIGHT, weight.device)
    mq_quantize_weight(weight, qw, MQ_RNE, 0, ws)
    return qw


def quantize_activation(x: torch.Tensor, fmt: int, rnd: int, seed: int, role: int,
                        ws: torch.Tensor) -> QTensor:
    """NCHW fp32 tensor -> quantized channel-batch-first tensor with the given rounding (one
    library call: amax pass, then a pass that reads NCHW and writes squares)."""
    N, C, H, W = x.shape
    q = QTensor(H, W, C, N, fmt, role, x.device)
    mq_quantize_nchw(x, q, rnd, seed, ws)
    return q


class MQConv2dFunction(torch.autograd.Function):
    """Autograd function: forward and backward of one convolution through the library."""

    @staticmethod
    def forward(ctx, x: torch.Tensor, weight: torch.Tensor, stride: int, padding: int, fmt: int,
                sr_seed: int, qw_cached: Optional[QTensor]):
        _check_input(x, "input")
        _check_input(weight, "weight")
        x = x.contiguous()
        weight = weight.contiguous()
        N, Cin, H, W = x.shape
        Cout, Cin_w, Kh, Kw = weight.shape
        if Cin_w != Cin:
            raise ValueError(f"input has {Cin} channels, weight expects {Cin_w}")
        conv = (N, Cin, H, W, Cout, Kh, Kw, stride, stride, padding, padding)
        Ho, Wo = out_hw(conv)
        dev = x.device
        ws = torch.empty(2 * MQ_QUANTIZE_WS_BYTES, dtype=torch.uint8, device=dev)
        if qw_cached is not None:
            qx = quantize_activation(x, fmt, MQ_RNE, 0, MQ_ROLE_ACT, ws[:MQ_QUANTIZE_WS_BYTES])
            qw = qw_cached
        else:  # X and W together: one amax launch and one quantizing launch
            qx = QTensor(H, W, Cin, N, fmt, MQ_ROLE_ACT, dev)
            qw = QTensor(Kh, Kw, Cout, Cin, fmt, MQ_ROLE_WEIGHT, dev)
            mq_quantize_batch([
                quant_job(x, MQ_SRC_NCHW, qx, MQ_RNE, 0, ws[:MQ_QUANTIZE_WS_BYTES]),
                quant_job(weight, MQ_SRC_OIHW, qw, MQ_RNE, 0, ws[MQ_QUANTIZE_WS_BYTES:])])
        yc = torch.empty(Ho * Wo * Cout * N, dtype=torch.float32, device=dev)
        mq_conv_fwd(conv, qx, qw, yc)
        y = torch.empty((N, Cout, Ho, Wo), dtype=torch.float32, device=dev)
        mq_relayout_cbf(yc, y, N, Cout, Ho, Wo, 1)
        ctx.conv, ctx.fmt, ctx.sr_seed = conv, fmt, sr_seed
        ctx.qx, ctx.qw = qx, qw
        return y

    @staticmethod
    def backward(ctx, gy: torch.Tensor):
        conv, fmt = ctx.conv, ctx.fmt
        N, Cin, H, W, Cout, Kh, Kw = conv[:7]
        Ho, Wo = out_hw(conv)
        gy = gy.contiguous().float()
        dev = gy.device
        ws = torch.empty(MQ_QUANTIZE_WS_BYTES, dtype=torch.uint8, device=dev)
        qg = quantize_activation(gy, fmt, MQ_SR, ctx.sr_seed, MQ_ROLE_GRAD, ws)
        gx = gw = None
        need_x, need_w = ctx.needs_input_grad[0], ctx.needs_input_grad[1]
        if need_w:
            gwk = torch.empty(Kh * Kw * Cout * Cin, dtype=torch.float32, device=dev)
            wsb = torch.empty(max(1, mq_wgrad_workspace_bytes(conv)), dtype=torch.uint8,
                              device=dev)
        if need_x:
            gxc = torch.empty(H * W * Cin * N, dtype=torch.float32, device=dev)
        if need_w and need_x:  # both gradients in one call (their launches overlap)
            mq_conv_backward(conv, ctx.qw, qg, ctx.qx, gwk, gxc, wsb)
        elif need_w:
            mq_conv_wgrad(conv, qg, ctx.qx, gwk, wsb)
        elif need_x:
            mq_conv_dgrad(conv, ctx.qw, qg, gxc)
        if need_w:
            gw = torch.empty((Cout, Cin, Kh, Kw), dtype=torch.float32, device=dev)
            mq_relayout_weight(gwk, gw, Cout, Cin, Kh, Kw, 1)
        if need_x:
            gx = torch.empty((N, Cin, H, W), dtype=torch.float32, device=dev)
            mq_relayout_cbf(gxc, gx, N, Cin, H, W, 1)
        ctx.qx = ctx.qw = None
        return gx, gw, None, None, None, None, None


class MQConv2d(nn.Module):
    """Square-kernel convolution (stride s, zero padding p, no bias) whose forward and backward
    GEMMs run on quantized operands (NVFP4 or NVFP6); fp32 master weight."""

    def __init__(self, in_channels: int, out_channels: int, kernel_size: int, stride: int = 1,
                 padding: int = 0, fmt: int = MQ_NVFP4, layer_index: int = 0, layers: int = 1,
                 seed_base: int = 1, cache_weight: bool = False):
        super().__init__()
        self.in_channels, self.out_channels = in_channels, out_channels
        self.kernel_size, self.stride, self.padding = kernel_size, stride, padding
        self.fmt = fmt
        self.layer_index, self.layers, self.seed_base = layer_index, layers, seed_base
        self.cache_weight = cache_weight
        self.weight = nn.Parameter(torch.empty(out_channels, in_channels, kernel_size,
                                               kernel_size))
        nn.init.kaiming_normal_(self.weight, mode="fan_in", nonlinearity="relu")
        self.step = 0
        self._qw: Optional[QTensor] = None
        self._qw_key: Optional[Tuple[int, int]] = None

    def sr_seed(self) -> int:
        return self.seed_base + self.layer_index + self.layers * self.step

    def _cached_weight(self) -> Optional[QTensor]:
        if self.training or not self.cache_weight:
            return None
        key = (self.weight.data_ptr(), self.weight._version)
        if self._qw is None or self._qw_key != key:
            ws = torch.empty(MQ_QUANTIZE_WS_BYTES, dtype=torch.uint8, device=self.weight.device)
            with torch.no_grad():
                self._qw = quantize_weight(self.weight.detach().contiguous(), self.fmt, ws)
            self._qw_key = key
        return self._qw

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        seed = self.sr_seed()
        if self.training:
            self.step += 1
        return MQConv2dFunction.apply(x, self.weight, self.stride, self.padding, self.fmt, seed,
                                      self._cached_weight())

    def extra_repr(self) -> str:
        return (f"{self.in_channels}, {self.out_channels}, kernel_size={self.kernel_size}, "
                f"stride={self.stride}, padding={self.padding}, fmt=NVFP{self.fmt}")


# ---- linear layers and the gated feed-forward block on microscaled 4-bit operands --------------

def _rows_of(x: torch.Tensor, cols: int, what: str) -> torch.Tensor:
    """x [...][cols] as a matrix with contiguous rows."""
    if not x.is_cuda or x.dtype not in (torch.float16, torch.bfloat16, torch.float32) or x.dim() < 1:
        raise ValueError(f"{what}: expected a float16, bfloat16 or float32 CUDA tensor, got "
                         f"{tuple(x.shape)} {x.dtype} on {x.device}")
    if x.shape[-1] != cols:
        raise ValueError(f"{what} has {x.shape[-1]} features, the weight expects {cols}")
    return x.reshape(x.shape[:-1].numel(), cols).contiguous()  # (-1 cannot be told where cols is 0)


def quantize_linear_weight(weight: torch.Tensor, columns: bool) -> Tuple[MX4, Optional[MX4]]:
    """A weight [out][in] along its rows and, if asked, its columns, from one read (RNE)."""
    n, k = weight.shape
    row = MX4.empty(n, k, weight.device)
    col = MX4.empty(k, n, weight.device) if columns else None
    mq_mx4_quantize(weight, row, col)
    return row, col


class _NoGraph:
    """The context of a forward pass that no graph records: nothing needs a gradient, nothing is kept."""
    needs_input_grad = (False,) * 5

    def save_for_backward(self, *tensors):
        pass


class _MXFunction(torch.autograd.Function):
    """What the 4-bit functions share."""

    @classmethod
    def apply(cls, *args):
        # ctx.needs_input_grad asks the inputs alone, so that a parameter needs a gradient also where no
        # graph is recorded: there, nothing is to be made for a backward pass
        return super().apply(*args) if torch.is_grad_enabled() else cls.forward(_NoGraph(), *args)

    @staticmethod
    def save(ctx, matrices: Sequence[Optional[MX4]], *tensors: Optional[torch.Tensor]):
        """Keep 4-bit matrices and tensors as saved tensors: the backward pass frees them, hooks see them."""
        ctx.held = [None if q is None else q.shape for q in matrices]
        ctx.save_for_backward(*tensors, *(t for q in matrices if q is not None for t in (q.codes, q.scales)))

    @staticmethod
    def saved(ctx, tensors: int) -> Tuple[Sequence[torch.Tensor], List[Optional[MX4]]]:
        saved = ctx.saved_tensors
        parts = iter(saved[tensors:])
        return saved[:tensors], [None if shape is None else MX4(*shape, next(parts), next(parts)) for shape in ctx.held]


class MXLinearFunction(_MXFunction):
    """Autograd function: y = x weight^T and its gradients through the library."""

    @staticmethod
    def forward(ctx, x: torch.Tensor, weight: torch.Tensor, sr_seed: int, held: Optional[MX4]):
        n, k = weight.shape
        rows = _rows_of(x, k, "input")
        m, dev = rows.shape[0], x.device
        need_x, need_w = ctx.needs_input_grad[:2]
        with torch.cuda.device(dev):
            w_row, w_col = (held, None) if held is not None else quantize_linear_weight(
                weight.detach().contiguous(), need_x)
            if need_x and w_col is None:
                w_col = MX4.empty(k, n, dev)
                mq_mx4_quantize(weight.detach().contiguous(), None, w_col)
            x_col = MX4.empty(k, m, dev) if need_w else None
            y = torch.empty((m, n), dtype=x.dtype, device=dev)
            mq_mx4_linear(rows, w_row, y, mx4_linear_workspace(m, n, k, dev), x_col)
        _MXFunction.save(ctx, (x_col, w_col))
        ctx.sr_seed = sr_seed
        ctx.sizes, ctx.shape, ctx.w_dtype = (m, n, k), x.shape, weight.dtype
        return y.view(*x.shape[:-1], n)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, gy: torch.Tensor):
        m, n, k = ctx.sizes
        rows, dev = _rows_of(gy, n, "gradient"), gy.device
        _, (x_col, w_col) = _MXFunction.saved(ctx, 0)
        dx = dw = None
        with torch.cuda.device(dev):
            if w_col is not None:
                dx = torch.empty((m, k), dtype=gy.dtype, device=dev)
            if x_col is not None:
                dw = torch.empty((n, k), dtype=ctx.w_dtype, device=dev)
            if dx is not None or dw is not None:
                mq_mx4_linear_backward(rows, x_col, w_col, dx, dw,
                                       mx4_linear_backward_workspace(m, n, k, dev), MQ_SR, ctx.sr_seed)
        return None if dx is None else dx.view(ctx.shape), dw, None, None


class MXGatedFunction(_MXFunction):
    """Autograd function: silu(x gate^T) * (x up^T) and its gradients through the library."""

    @staticmethod
    def forward(ctx, x: torch.Tensor, gate: torch.Tensor, up: torch.Tensor, sr_seed: int,
                held: Optional[Tuple[MX4, MX4]]):
        f, k = gate.shape
        rows = _rows_of(x, k, "input")
        m, dev = rows.shape[0], x.device
        need_x, need_w = ctx.needs_input_grad[0], any(ctx.needs_input_grad[1:3])
        with torch.cuda.device(dev):
            new = lambda: torch.empty((m, f), dtype=x.dtype, device=dev)
            if held is not None:
                row = held
                col = [None, None]
                if need_x:
                    col = [MX4.empty(k, f, dev) for _ in row]
                    for w, q in zip((gate, up), col):
                        mq_mx4_quantize(w.detach().contiguous(), None, q)
            else:
                row, col = zip(*(quantize_linear_weight(w.detach().contiguous(), need_x)
                                 for w in (gate, up)))
            x_col = MX4.empty(k, m, dev) if need_w else None
            g, u = (new(), new()) if need_x or need_w else (None, None)
            h = new()
            mq_mx4_gated(rows, row[0], row[1], h, mx4_gated_workspace(m, f, k, dev), g, u, x_col)
        _MXFunction.save(ctx, (x_col, *col), g, u)
        ctx.sr_seed = sr_seed
        ctx.sizes, ctx.shape, ctx.w_dtype = (m, f, k), x.shape, gate.dtype
        return h.view(*x.shape[:-1], f)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dh: torch.Tensor):
        m, f, k = ctx.sizes
        rows, dev = _rows_of(dh, f, "gradient"), dh.device
        need_x, need_w = ctx.needs_input_grad[0], any(ctx.needs_input_grad[1:3])
        (g, u), (x_col, wg_col, wu_col) = _MXFunction.saved(ctx, 2)
        dx = dwg = dwu = None
        with torch.cuda.device(dev):
            if need_x:
                dx = torch.empty((m, k), dtype=dh.dtype, device=dev)
            if need_w:
                dwg, dwu = (torch.empty((f, k), dtype=ctx.w_dtype, device=dev) for _ in range(2))
            if need_x or need_w:
                mq_mx4_gated_backward(rows, g, u, x_col, wg_col, wu_col, dx, dwg, dwu,
                                      mx4_gated_backward_workspace(m, f, k, dev), MQ_SR, ctx.sr_seed)
        return None if dx is None else dx.view(ctx.shape), dwg, dwu, None, None


class _MXModule(nn.Module):
    """What the 4-bit modules share: seeds of the stochastic rounding, and weights held in 4 bits
    from one evaluation to the next (``cache_weight``) until a parameter changes: its version counter moves,
    another takes its place, or the module is moved, cast, or told ``train()`` or ``eval()`` (changes through
    ``.data`` are not counted: they need one of these)."""

    # the matrices, what they were made of, the stream that made them and an event behind that: in one
    # piece, which a call on another thread sees whole
    _kept: Optional[Tuple[List[MX4], list, torch.cuda.Stream, torch.cuda.Event]] = None

    def __init__(self, layer_index: int, layers: int, seed_base: int, cache_weight: bool):
        super().__init__()
        self.layer_index, self.layers, self.seed_base = layer_index, layers, seed_base
        self.cache_weight = cache_weight
        self.step = 0
        self._release()

    def _release(self):
        """Let go of the weights held in 4 bits."""
        self._kept = None

    @property
    def _held(self) -> Optional[List[MX4]]:
        return None if self._kept is None else self._kept[0]

    def __getstate__(self) -> dict:
        # copies and pickles quantize their own weights
        return {**self.__dict__, "_kept": None}

    def train(self, mode: bool = True):
        self._release()
        return super().train(mode)

    def _apply(self, *args, **kwargs):
        self._release()
        return super()._apply(*args, **kwargs)

    def _next_seed(self) -> int:
        seed = self.seed_base + self.layer_index + self.layers * self.step
        if self.training:
            self.step += 1
        return seed

    def _cached(self, *weights: torch.Tensor) -> Optional[List[MX4]]:
        # (changes of tensors made in inference mode are not counted)
        if self.training or not self.cache_weight or any(w.is_inference() for w in weights):
            return None
        # the parameters themselves, not their addresses: another tensor may come to lie at one
        now = [(w, w._version, w.data_ptr(), w.dtype) for w in weights]
        with torch.cuda.device(weights[0].device):
            if torch.cuda.is_current_stream_capturing():
                # quantized inside the graph: a replay reads the weights as they are then, no memory that is
                # let go of when they change, and an eager call holds nothing that only a replay fills
                return None
            stream, kept = torch.cuda.current_stream(), self._kept
            if kept is None or any(a[0] is not b[0] or a[1:] != b[1:] for a, b in zip(now, kept[1])):
                held = [quantize_linear_weight(w.detach().contiguous(), False)[0] for w in weights]
                self._kept = held, now, stream, stream.record_event()
                return held
            held, _, made_on, made = kept
            if stream != made_on:
                # another stream than the one that quantized them: it waits for that, and their memory is
                # not used again before it has read them
                stream.wait_event(made)
                for t in (t for q in held for t in (q.codes, q.scales)):
                    t.record_stream(stream)
        return held


class MXLinear(_MXModule):
    """Linear layer (no bias) whose forward and backward products run on 4-bit operands; fp32 master
    weight. Inputs [...][in_features] in float16, bfloat16 or float32; outputs of their type."""

    def __init__(self, in_features: int, out_features: int, layer_index: int = 0, layers: int = 1,
                 seed_base: int = 1, cache_weight: bool = False):
        super().__init__(layer_index, layers, seed_base, cache_weight)
        self.in_features, self.out_features = in_features, out_features
        self.weight = nn.Parameter(torch.empty(out_features, in_features))
        nn.init.normal_(self.weight, std=in_features ** -0.5)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        held = self._cached(self.weight)
        return MXLinearFunction.apply(x, self.weight, self._next_seed(), None if held is None else held[0])

    def extra_repr(self) -> str:
        return f"{self.in_features}, {self.out_features}"


class MXGatedMLP(_MXModule):
    """Gated feed-forward block: down(silu(x gate^T) * (x up^T)), all three products on 4-bit
    operands; fp32 master weights."""

    def __init__(self, features: int, hidden: int, layer_index: int = 0, layers: int = 1,
                 seed_base: int = 1, cache_weight: bool = False):
        super().__init__(2 * layer_index, 2 * layers, seed_base, cache_weight)
        self.features, self.hidden = features, hidden
        self.gate = nn.Parameter(torch.empty(hidden, features))
        self.up = nn.Parameter(torch.empty(hidden, features))
        for w in (self.gate, self.up):
            nn.init.normal_(w, std=features ** -0.5)
        self.down = MXLinear(hidden, features, 2 * layer_index + 1, 2 * layers, seed_base, cache_weight)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        held = self._cached(self.gate, self.up)
        h = MXGatedFunction.apply(x, self.gate, self.up, self._next_seed(),
                                  None if held is None else tuple(held))
        return self.down(h)

    def extra_repr(self) -> str:
        return f"{self.features}, {self.hidden}"


def number_layers(model: nn.Module, seed_base: int = 1) -> int:
    """Number a model's quantized layers through (``MQConv2d``, ``MXLinear``, and the two products of each
    ``MXGatedMLP``), in the order of ``model.modules()``, so that no two of them round their gradients by
    the same bits in any step. Returns how many there are."""
    layers = [m for m in model.modules() if isinstance(m, (MQConv2d, _MXModule))]
    for i, m in enumerate(layers):
        m.layer_index, m.layers, m.seed_base = i, len(layers), seed_base
    return len(layers)


# ---- ResNet-18 with the 19 body convolutions quantized ---------------------------------------

class BasicBlock(nn.Module):
    def __init__(self, cin: int, cout: int, stride: int, convs: List[MQConv2d]):
        super().__init__()
        self.conv1 = convs[0]
        self.bn1 = nn.BatchNorm2d(cout)
        self.conv2 = convs[1]
        self.bn2 = nn.BatchNorm2d(cout)
        self.down = None
        if len(convs) == 3:
            self.down = convs[2]
            self.bn_down = nn.BatchNorm2d(cout)

    def forward(self, x):
        out = torch.relu(self.bn1(self.conv1(x)))
        out = self.bn2(self.conv2(out))
        sc = x if self.down is None else self.bn_down(self.down(x))
        return torch.relu(out + sc)


class ResNet18MQ(nn.Module):
    """ResNet-18 whose 19 body convolutions (layer1..layer4, downsample 1x1 included) are
    MQConv2d; the 7x7 stem, batch norms, pooling and the classifier stay fp32 PyTorch."""

    BODY = ([(64, 64, 1)] * 2 + [(64, 128, 2), (128, 128, 1)] + [(128, 256, 2), (256, 256, 1)] +
            [(256, 512, 2), (512, 512, 1)])

    def __init__(self, num_classes: int = 1000, fmt: int = MQ_NVFP4, seed_base: int = 1):
        super().__init__()
        self.stem = nn.Conv2d(3, 64, 7, 2, 3, bias=False)
        self.bn = nn.BatchNorm2d(64)
        self.pool = nn.MaxPool2d(3, 2, 1)
        specs = []  # (cin, cout, k, stride, pad) of every quantized conv, network order
        for cin, cout, s in self.BODY:
            specs.append((cin, cout, 3, s, 1))
            specs.append((cout, cout, 3, 1, 1))
            if s != 1 or cin != cout:
                specs.append((cin, cout, 1, s, 0))
        n = len(specs)
        convs = [MQConv2d(ci, co, k, s, p, fmt, i, n, seed_base) for i, (ci, co, k, s, p)
                 in enumerate(specs)]
        self.mq_convs = nn.ModuleList(convs)
        blocks, i = [], 0
        for cin, cout, s in self.BODY:
            k = 3 if (s != 1 or cin != cout) else 2
            blocks.append(BasicBlock(cin, cout, s, convs[i:i + k]))
            i += k
        self.blocks = nn.Sequential(*blocks)
        self.fc = nn.Linear(512, num_classes)

    def forward(self, x):
        x = self.pool(torch.relu(self.bn(self.stem(x))))
        x = self.blocks(x)
        return self.fc(torch.flatten(nn.functional.adaptive_avg_pool2d(x, 1), 1))
