"""torch modules over libkron: the Kronecker-factored layer, its gated form, adapters beside a
projection, the Kronecker-sparse layer, the losses over a vocabulary and the tutorial's MLP training
step.  Marshalling only; every step runs in libkron.
"""
from __future__ import annotations

import math
from typing import Optional

import torch
from torch import nn
from torch.autograd.function import once_differentiable

from . import api
from ._lib import KRON_ADAPTERS_MAX_RANK, KRON_GLU_MAX_RANK, KRON_GLU_MAX_SIDE


class _KronLinearFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, S, A, B, bias, relu: bool, sparse_rows: bool, save_z: bool = False):
        x = x.contiguous()
        # Z_i = X B_i saved for the backward where the shape has that path (else recomputed)
        zc = api.new_zcache(x, S, A, B) if save_z and not sparse_rows else None
        y = api.kron_linear_fwd(x, S, A, B, bias, relu=relu, sparse_rows=sparse_rows, zcache=zc)
        ctx.zc = zc
        ctx.relu = relu
        ctx.sparse_rows = sparse_rows
        ctx.save_for_backward(x, S, A, B, y if relu else None)
        ctx.has_S = S is not None
        ctx.has_bias = bias is not None
        return y

    @staticmethod
    def backward(ctx, dy):
        x, S, A, B, y = ctx.saved_tensors
        dy = dy.contiguous()
        if ctx.relu:
            dy = api.kron_relu_bwd(y, dy)
        g = api.kron_linear_bwd(x, S, A, B, dy, want_dx=ctx.needs_input_grad[0],
                                want_dbias=ctx.has_bias, sparse_rows=ctx.sparse_rows, zcache=ctx.zc)
        ctx.zc = None
        return g["dx"], g["dS"], g["dA"], g["dB"], g["dbias"], None, None, None


class KronLinear(nn.Module):
    """y = x W + bias, W = sum_i kron(S o A_i, B_i) (Kronecker layer tutorial,
    "Build W, then multiply": S p x q initialised to ones, A_i ~ randn/sqrt(p),
    B_i ~ randn/sqrt(m), bias zeros; p = in/m, q = out/n).  sparse_rows: S is expected
    to have whole rows zero (e.g. after l1 pruning) and the forward skips them.  save_z: the
    forward keeps Z_i = X B_i of the first ranks (kron_linear_zcache_bytes per batch) for the
    backward instead of the backward recomputing it, where the shape has that path."""

    def __init__(self, in_features: int, out_features: int, m: int, r: int, n: Optional[int] = None,
                 with_S: bool = True, relu: bool = False, device=None, sparse_rows: bool = False,
                 save_z: bool = False):
        super().__init__()
        n = m if n is None else n
        if in_features % m or out_features % n:
            raise ValueError("in_features must be a multiple of m and out_features of n")
        p, q = in_features // m, out_features // n
        dev = device
        self.S = nn.Parameter(torch.ones(p, q, device=dev)) if with_S else None
        self.A = nn.Parameter(torch.randn(r, p, q, device=dev) / math.sqrt(p))
        self.B = nn.Parameter(torch.randn(r, m, n, device=dev) / math.sqrt(m))
        self.bias = nn.Parameter(torch.zeros(out_features, device=dev))
        self.relu = relu
        self.sparse_rows = sparse_rows
        self.save_z = save_z

    def forward(self, x):
        return _KronLinearFn.apply(x, self.S, self.A, self.B, self.bias, self.relu, self.sparse_rows, self.save_z)

    def l1_penalty(self):
        """sum|S| as a 0-dim tensor with autograd (sign(S) times the upstream gradient)."""
        return _L1Fn.apply(self.S) if self.S is not None else 0.0


class _L1Fn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, S):
        ctx.save_for_backward(S)
        return api.kron_l1_penalty([S.contiguous()], 1.0).view(())

    @staticmethod
    def backward(ctx, g):
        (S,) = ctx.saved_tensors
        return api.kron_l1_penalty_grad(S.contiguous(), 1.0, g.reshape(1).contiguous())


def _whole(t: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    """t contiguous and at a 16-byte boundary, as libkron takes it: a slice of a batch, or a gradient that
    autograd cut out of a larger one, may start anywhere."""
    if t is None:
        return None
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class _KronGLUFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, S, A, B, bias, act: str):
        rows = _whole(x.reshape(-1, x.shape[-1]))
        params = (S, A, B, bias)
        ctx.types = [None if t is None else t.dtype for t in params]
        if rows.dtype == torch.bfloat16:      # (float32 parameters: the block runs in the input's type)
            params = [t.to(rows.dtype) if t is not None and t.dtype == torch.float32 else t for t in params]
        ctx.save_for_backward(rows, *params)
        ctx.act, ctx.shape = act, x.shape
        y = api.kron_glu_fwd(rows, *params, act=act)
        return y.view(*x.shape[:-1], y.shape[1])

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, S, A, B, bias = ctx.saved_tensors
        g = api.kron_glu_bwd(x, S, A, B, bias, _whole(dy.reshape(x.shape[0], dy.shape[-1])), act=ctx.act,
                             want_dx=ctx.needs_input_grad[0])
        dx = g["dx"]
        # the parameters' gradients come in float32, which parameters in float32 get as they are
        to = [None if g[k] is None else g[k].to(t) for k, t in zip(("dS", "dA", "dB", "dbias"), ctx.types)]
        return (None if dx is None else dx.view(ctx.shape), *to, None)


class KronGLU(nn.Module):
    """y = act(x W_0 + b_0) o (x W_1 + b_1) with W_f = sum_i kron(S_f o A_fi, B_fi): the gated half
    of a feed-forward block, both projections Kronecker layers of one shape in one kernel.  Parameters
    as KronLinear's with a leading 2 (gate, up).  x: [..., in_features], float32 or bfloat16 like the
    parameters, or bfloat16 with float32 parameters: they are rounded to bfloat16 for the products, and their
    gradients stay float32.  m, n, in_features / m and out_features / n are at most 64, r at most 16.  act: silu,
    gelu, gelu_tanh or relu.  The backward recomputes the projections.
    A backward captured into a graph has to be the only autograd graph of the parameters alive (or
    taken with torch.autograd.grad): torch ends the process otherwise, for this module as for any."""

    def __init__(self, in_features: int, out_features: int, m: int, r: int, n: Optional[int] = None, act: str = "silu",
                 with_S: bool = True, bias: bool = True, device=None, dtype=None):
        super().__init__()
        n = m if n is None else n
        if in_features % m or out_features % n:
            raise ValueError("in_features must be a multiple of m and out_features of n")
        if act not in api.KRON_ACTS:
            raise ValueError(f"act must be one of {sorted(api.KRON_ACTS)}, got {act!r}")
        p, q = in_features // m, out_features // n
        if not 1 <= min(p, q, m, n) <= max(p, q, m, n) <= KRON_GLU_MAX_SIDE or not 1 <= r <= KRON_GLU_MAX_RANK:
            raise ValueError(f"the factors' sides p = {p}, q = {q}, m = {m}, n = {n} must be in 1..{KRON_GLU_MAX_SIDE} "
                             f"and r = {r} in 1..{KRON_GLU_MAX_RANK}")
        kw = dict(device=device, dtype=dtype)
        self.S = nn.Parameter(torch.ones(2, p, q, **kw)) if with_S else None
        self.A = nn.Parameter(torch.randn(2, r, p, q, **kw) / math.sqrt(p))
        self.B = nn.Parameter(torch.randn(2, r, m, n, **kw) / math.sqrt(m))
        self.bias = nn.Parameter(torch.zeros(2, out_features, **kw)) if bias else None
        self.act = act

    def forward(self, x):
        return _KronGLUFn.apply(x, self.S, self.A, self.B, self.bias, self.act)


class _KronDistillFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, teacher, teacher_lse, labels, weights, temperature: float, alpha: float):
        ctx.kw = dict(temperature=temperature, alpha=alpha)
        loss, stats = api.kron_distill_fwd(logits, ids, teacher, teacher_lse, labels, weights, **ctx.kw)
        ctx.save_for_backward(logits, ids, teacher, teacher_lse, labels, weights, stats)
        return loss.view(())

    @staticmethod
    @once_differentiable
    def backward(ctx, gout):
        logits, ids, teacher, lse, labels, weights, stats = ctx.saved_tensors
        dz = api.kron_distill_bwd(logits, ids, teacher, stats, _whole(gout.reshape(1)), lse, labels, weights, **ctx.kw)
        return (dz,) + (None,) * 7


class KronDistillLoss(nn.Module):
    """Distillation from a teacher's top logits (kron_topk_logits), mixed with the cross-entropy on
    labels: alpha T^2 KD + (1 - alpha) CE over the rows, weighted (weights None: their mean, weight 0: a
    padded position).  logits [..., V] with ids and teacher [..., k], the others [...] (nothing: one row); the
    gradient goes to the logits alone.  Logits whose leading dimensions are not one stride apart are copied:
    give a batch's last positions weight 0 rather than cutting them off (logits[:, :-1])."""

    def __init__(self, temperature: float = 1.0, alpha: float = 1.0):
        super().__init__()
        if not (temperature > 0 and 0 <= alpha <= 1):
            raise ValueError(f"temperature must be positive and alpha in [0, 1], got {temperature} and {alpha}")
        self.temperature, self.alpha = float(temperature), float(alpha)

    def forward(self, logits, ids=None, teacher=None, teacher_lse=None, labels=None, weights=None):
        def rows(t, last):
            if t is None or t.dim() == 1 + last:
                return t
            return t.flatten(0, -1 - last) if t.dim() > 1 + last else t.unsqueeze(0)
        other = [_whole(rows(t, last)) for t, last in ((ids, 1), (teacher, 1), (teacher_lse, 0), (labels, 0), (weights, 0))]
        return _KronDistillFn.apply(rows(logits, 1), *other, self.temperature, self.alpha)


class _KronVocabCEFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, W, labels, weights):
        ctx.type = W.dtype
        w = _whole(W if W.dtype == h.dtype or h.dtype != torch.bfloat16 else W.to(h.dtype))
        loss, nll, stats = api.kron_vocab_ce_fwd(h, w, labels, weights)
        ctx.save_for_backward(h, w, labels, weights, stats, nll if ctx.needs_input_grad[3] else None)
        return loss.view(())

    @staticmethod
    @once_differentiable
    def backward(ctx, gout):
        h, W, labels, weights, stats, nll = ctx.saved_tensors
        g = api.kron_vocab_ce_bwd(h, W, labels, stats, _whole(gout.reshape(1)), weights,
                                  want_dh=ctx.needs_input_grad[0], want_dW=ctx.needs_input_grad[1])
        return g["dh"], None if g["dW"] is None else g["dW"].to(ctx.type), None, None if nll is None else nll * gout


class KronVocabCE(nn.Module):
    """The cross-entropy of the logits h W^T on labels, without the logits in memory: sum_n weights[n] nll[n]
    (weights None: the mean over the rows; weight 0: a padded position, or one of a prompt, that is left out).  h [..., K], W [V, K]
    (an embedding table; a float32 one with bfloat16 h is rounded to bfloat16), labels and weights [...].  The
    backward computes the logits once more.  The gradient of weights is nll (0 for a row that is left out)."""

    def forward(self, h, W, labels, weights=None):
        rows = _whole(h.reshape(-1, h.shape[-1]))
        labels = _whole(labels.reshape(-1))
        return _KronVocabCEFn.apply(rows, W, labels, None if weights is None else _whole(weights.reshape(-1)))


class _KronAdaptersFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, base, down, up, ids, starts, scales):
        ctx.types = (down.dtype, up.dtype)
        d, u = (_whole(t.to(x.dtype)) for t in (down, up))
        ctx.save_for_backward(x, d, u, ids, starts, scales)
        return api.kron_adapters_fwd(x, base, d, u, ids, starts, scales)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, down, up, ids, starts, scales = ctx.saved_tensors
        dy = _whole(dy)
        dx = None
        dd = du = None
        if any(ctx.needs_input_grad[i] for i in (0, 2, 3)):
            g = api.kron_adapters_bwd(x, dy, down, up, ids, starts, scales, want_dx=ctx.needs_input_grad[0])
            dx, dd, du = g["dx"], g["ddown"].to(ctx.types[0]), g["dup"].to(ctx.types[1])
        return dx, dy if ctx.needs_input_grad[1] else None, dd, du, None, None, None


class KronAdapters(nn.Module):
    """Low-rank adapters beside a projection (a KronLinear, or any module of rows): y = projection(x) + scale (x
    down[e]^T) up[e]^T, for each request with its own adapter e.  down ~ randn / sqrt(in), up zeros, scale = alpha /
    rank (alpha None: rank).  forward(x, ids, starts): x [N, in] (or [..., in] without ids: adapter 0 everywhere), request
    i the rows starts[i] to starts[i + 1] (int32; None: one row each) with adapter ids[i] (int32, negative: none).
    down and up are rounded to x's type for the products; their gradients are computed in float32.  The scales are
    float32 whatever type the module is converted to."""

    def __init__(self, projection: nn.Module, in_features: int, out_features: int, rank: int, adapters: int = 1,
                 alpha: Optional[float] = None, device=None, dtype=None):
        super().__init__()
        if not 1 <= rank <= KRON_ADAPTERS_MAX_RANK:
            raise ValueError(f"rank must be in 1..{KRON_ADAPTERS_MAX_RANK}, got {rank}")
        kw = dict(device=device, dtype=dtype)
        self.projection = projection
        self.down = nn.Parameter(torch.randn(adapters, rank, in_features, **kw) / math.sqrt(in_features))
        self.up = nn.Parameter(torch.zeros(adapters, out_features, rank, **kw))
        scale = 1.0 if alpha is None else alpha / rank
        self.register_buffer("scales", torch.full((adapters,), scale, device=device, dtype=torch.float32))

    def _apply(self, fn, recurse=True):
        scales = self.scales
        super()._apply(fn, recurse)
        if self.scales.dtype != torch.float32:      # .bfloat16() and the like convert floating buffers too
            self.scales = scales.to(self.scales.device)
        return self

    def forward(self, x, ids=None, starts=None):
        base = self.projection(x)
        rows, wide = _whole(x.reshape(-1, x.shape[-1])), _whole(base.reshape(-1, base.shape[-1]))
        if ids is None:
            if starts is not None:
                raise ValueError("starts needs ids")
            ids = torch.zeros(1, dtype=torch.int32, device=x.device)
            starts = torch.arange(2, dtype=torch.int32, device=x.device) * rows.shape[0]
        return _KronAdaptersFn.apply(rows, wide, self.down, self.up, ids, starts, self.scales.float()).view(base.shape)


class KSLinear(nn.Module):
    """Y = X K with K Kronecker-sparse of support I_a (x) 1_{b x c} (x) I_d ("Fast Inference
    with Kronecker-Sparse Matrices"); values a x d x b x c ~ N(0, 1/b).  Forward only."""

    def __init__(self, a: int, b: int, c: int, d: int, dtype=torch.float32, device=None):
        super().__init__()
        self.abcd = (a, b, c, d)
        self.vals = nn.Parameter((torch.randn(a, d, b, c, device=device) / math.sqrt(b)).to(dtype),
                                 requires_grad=False)

    def forward(self, x):
        a, b, c, d = self.abcd
        return api.ks_matmul(x.contiguous(), self.vals, a, b, c, d)


class KronMLPStep:
    """The tutorial's training step (Kronecker layer tutorial, "Setup"): MLP
    in -> hidden -> hidden -> classes with ReLU, both hidden layers Kronecker, a dense
    head, mean cross-entropy + lam * sum|S|, backward, and one fused Adam update.

    Parameters live in flat lists of device tensors in the order
    S1, A1, B1, bias1, S2, A2, B2, bias2, head_w (hidden x classes), head_b.
    One step is 10 kernel launches plus the column reductions, independent of r.

    optimizer "muon": the factors A and B (matrices of p x q and m x n) take an orthogonalised update
    of rate muon_lr and momentum beta1 instead of Adam's, everything else Adam's.
    """

    MUON = (1, 2, 5, 6)      # A1, B1, A2, B2

    def __init__(self, layers, head_w, head_b, lam: float, lr: float, device,
                 beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8, optimizer: str = "adam",
                 muon_lr: float = 0.02):
        if optimizer not in ("adam", "muon"):
            raise ValueError(f"optimizer must be adam or muon, got {optimizer!r}")

        def t(a):
            return torch.as_tensor(a, dtype=torch.float32, device=device).contiguous()
        self.params = []
        for L in layers:
            self.params += [t(L["S"]), t(L["A"]), t(L["B"]), t(L["bias"])]
        self.params += [t(head_w), t(head_b)]
        self.m = [torch.zeros_like(p) for p in self.params]
        self.v = [torch.zeros_like(p) for p in self.params]
        self.l1 = [lam, 0.0, 0.0, 0.0, lam, 0.0, 0.0, 0.0, 0.0, 0.0]
        self.lam, self.lr = lam, lr
        self.beta1, self.beta2, self.eps = beta1, beta2, eps
        self.optimizer, self.muon_lr = optimizer, muon_lr
        self.step_count = 0
        self.device = device
        self._ws = {}

    def _workspace(self, key, nbytes):
        w = self._ws.get(key)
        if w is None or w.numel() < nbytes:
            w = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=self.device)
            self._ws[key] = w
        return w

    def grads(self, x: torch.Tensor, labels: torch.Tensor):
        """Forward + backward; returns (loss tensor, gradient list, activations).  The loss is
        the mean cross-entropy plus lam * (sum|S1| + sum|S2|); the l1 subgradient of the
        penalty is applied inside the Adam step."""
        S1, A1, B1, b1, S2, A2, B2, b2, hw, hb = self.params
        h1 = api.kron_linear_fwd(x, S1, A1, B1, b1, relu=True)
        h2 = api.kron_linear_fwd(h1, S2, A2, B2, b2, relu=True)
        head = api.kron_head_ce(h2, hw, hb, labels, want_dh=True, relu_mask=True)
        api.kron_l1_penalty([S1, S2], self.lam, loss=head["loss"], accumulate=True)
        shape2 = api.layer_shape(h1.shape[0], S2, A2, B2)
        g2 = api.kron_linear_bwd(h1, S2, A2, B2, head["dh"], want_dx=True, relu_mask=True,
                                 workspace=self._workspace("l2", api.kron_linear_bwd_workspace_bytes(shape2)))
        shape1 = api.layer_shape(x.shape[0], S1, A1, B1)
        g1 = api.kron_linear_bwd(x, S1, A1, B1, g2["dx"], want_dx=False,
                                 workspace=self._workspace("l1", api.kron_linear_bwd_workspace_bytes(shape1)))
        grads = [g1["dS"], g1["dA"], g1["dB"], g1["dbias"], g2["dS"], g2["dA"], g2["dB"], g2["dbias"],
                 head["dW"], head["db"]]
        return head["loss"], grads, dict(h1=h1, h2=h2, dh2=head["dh"], dh1=g2["dx"])

    def step(self, x: torch.Tensor, labels: torch.Tensor):
        """One full training step; returns the loss (cross-entropy + l1 penalty, device tensor)."""
        loss, grads, _ = self.grads(x, labels)
        self.step_count += 1
        rest = range(len(self.params))
        if self.optimizer == "muon":
            api.kron_muon_step(*([ts[i] for i in self.MUON] for ts in (self.params, grads, self.m)), lr=self.muon_lr,
                               momentum=self.beta1)
            rest = [i for i in rest if i not in self.MUON]
        api.kron_adam_l1_step(*([ts[i] for i in rest] for ts in (self.params, grads, self.m, self.v)), self.step_count,
                              self.lr, self.beta1, self.beta2, self.eps, l1=[self.l1[i] for i in rest])
        return loss
