"""A pre-norm sequence block on the library's kernels, fp32:

    y = x + dropout(W_out scan(conv(W_in layer_norm(x))))

Rows x [S, L, C] (or packed [T, C] with cu_seqlens).  W_in gives the
convolution's input and the scan's gate (halves of one buffer); the
convolution's output u gives, through W_x, a low-rank step size and the scan's
input and output weights B and C.  The projections are mlp_linear_*, the rest
are the operators of recurrent_cell_amd.seq.  Torch's own elementwise kernels
form A = -exp(A_log) (for every call, single tokens too) and its gradient, the
residual sums of prefill, step and backward, u's gradient from its two uses, and
the copies that bring W_x's parts side by side.

forward / backward are a training pass, prefill / step serve the same weights:
a whole prompt in one pass from empty states, then a token at a time.
"""
import math
from dataclasses import dataclass

import torch

from . import cfc as _cfc
from . import mlp as _mlp
from . import seq as _seq


@dataclass
class Cache:
    """What single tokens carry on: the convolution's last inputs and the scan's
    state."""
    conv: torch.Tensor   # [S, K - 1, D]
    h: torch.Tensor      # [S, N, D]


class SequenceBlock:
    """C channels in and out, D inside, N states, K taps, rank R of the step
    size's projection, dropout p."""

    def __init__(self, C, D, N=16, K=4, R=None, p=0.0, eps=1e-5, device="cuda", seed=0):
        self.C, self.D, self.N, self.K, self.p, self.eps = C, D, N, K, p, eps
        self.R = R = R or max(1, -(-C // 16))
        g = torch.Generator().manual_seed(seed)

        def uniform(fan_in, *shape):
            return ((torch.rand(shape, generator=g) * 2 - 1) / math.sqrt(fan_in)).to(device)

        delta = torch.exp(torch.rand(D, generator=g) * (math.log(0.1) - math.log(1e-3)) + math.log(1e-3))
        self.params = {
            "ln_w": torch.ones(C, device=device), "ln_b": torch.zeros(C, device=device),
            "W_in": uniform(C, 2 * D, C), "conv_w": uniform(K, D, K), "conv_b": torch.zeros(D, device=device),
            "W_x": uniform(D, R + 2 * N, D), "W_dt": uniform(R, D, R),
            "dt_bias": (delta + torch.log(-torch.expm1(-delta))).to(device),   # softplus of it is delta
            "A_log": torch.log(torch.arange(1, N + 1, dtype=torch.float32))[:, None].repeat(1, D).to(device),
            "skip": torch.ones(D, device=device), "W_out": uniform(D, C, D),
        }

    def _inner(self, x, cu=None, state=None, conv_out=None, h0=None, save=False):
        """Everything up to W_out's output, and what the backward pass reads."""
        P, D, R, N, rows = self.params, self.D, self.R, self.N, x.shape[:-1]
        t = {"x": x, "cu": cu}
        t["n"], t["mean"], t["rstd"] = _seq.layer_norm_fwd(x, P["ln_w"], P["ln_b"], eps=self.eps)
        xz = _mlp.mlp_linear_fwd(t["n"].view(-1, self.C), P["W_in"], None, relu=False).view(*rows, 2 * D)
        t["xc"], t["z"] = xz[..., :D], xz[..., D:]
        t["u"] = _seq.causal_conv_fwd(t["xc"], P["conv_w"], P["conv_b"], state=state, cu_seqlens=cu, state_out=conv_out)
        w = _mlp.mlp_linear_fwd(t["u"].view(-1, D), P["W_x"], None, relu=False).view(*rows, R + 2 * N)
        t["low"] = w[..., :R].reshape(-1, R).contiguous()
        t["B"], t["C"] = w[..., R:R + N], w[..., R + N:]
        t["dt"] = _mlp.mlp_linear_fwd(t["low"], P["W_dt"], None, relu=False).view(*rows, D)
        t["A"] = -torch.exp(P["A_log"])
        t["scan"] = _seq.selective_scan_fwd(t["u"], t["dt"], t["A"], t["B"], t["C"], skip=P["skip"], z=t["z"],
                                            dt_bias=P["dt_bias"], h0=h0, cu_seqlens=cu, save=save)
        out = _mlp.mlp_linear_fwd(t["scan"].y.view(-1, D), P["W_out"], None, relu=False).view(*rows, self.C)
        return out, t

    def forward(self, x, seed=0, offset=0, cu_seqlens=None):
        """(y, saved): a training pass; seed and offset choose the dropout's mask."""
        out, t = self._inner(x, cu_seqlens, save=True)
        t["seed"], t["offset"] = seed, offset
        return _seq.dropout_fwd(out, self.p, seed, offset, residual=x), t

    def backward(self, dy, t):
        """(dx, gradients of every parameter) from forward's saved values."""
        P, D, R, C = self.params, self.D, self.R, self.C
        rows, g = dy.shape[:-1], {}
        dout = _seq.dropout_bwd(dy, self.p, t["seed"], t["offset"]).view(-1, C)
        g["W_out"] = _mlp.mlp_linear_bwd_weight(dout, t["scan"].y.view(-1, D), with_bias=False)[0]
        ds = _mlp.mlp_linear_bwd_data(dout, P["W_out"]).view(*rows, D)
        dxz = torch.empty((*rows, 2 * D), dtype=torch.float32, device=dy.device)
        d = _seq.selective_scan_bwd(ds, t["u"], t["dt"], t["A"], t["B"], t["C"], t["scan"].hist, skip=P["skip"], z=t["z"],
                                    dt_bias=P["dt_bias"], cu_seqlens=t["cu"], dz=dxz[..., D:])
        g["skip"], g["dt_bias"], g["A_log"] = d.dskip, d.ddt_bias, d.dA * t["A"]
        g["W_dt"] = _mlp.mlp_linear_bwd_weight(d.ddt.view(-1, D), t["low"], with_bias=False)[0]
        dlow = _mlp.mlp_linear_bwd_data(d.ddt.view(-1, D), P["W_dt"]).view(*rows, R)
        dw = torch.cat([dlow, d.dB, d.dC], -1).view(-1, R + 2 * self.N)
        g["W_x"] = _mlp.mlp_linear_bwd_weight(dw, t["u"].view(-1, D), with_bias=False)[0]
        du = d.du + _mlp.mlp_linear_bwd_data(dw, P["W_x"]).view(*rows, D)
        _, g["conv_w"], g["conv_b"] = _seq.causal_conv_bwd(du, t["xc"], P["conv_w"], P["conv_b"], cu_seqlens=t["cu"],
                                                           dx=dxz[..., :D])
        dxz = dxz.view(-1, 2 * D)
        g["W_in"] = _mlp.mlp_linear_bwd_weight(dxz, t["n"].view(-1, C), with_bias=False)[0]
        dn = _mlp.mlp_linear_bwd_data(dxz, P["W_in"]).view(*rows, C)
        dx, g["ln_w"], g["ln_b"] = _seq.layer_norm_bwd(dn, t["x"], P["ln_w"], t["mean"], t["rstd"])
        return dx + dy, g

    def prefill(self, x, cu_seqlens=None):
        """(y, Cache) of whole prompts, without dropout."""
        S = x.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1
        conv = torch.empty((S, self.K - 1, self.D), dtype=torch.float32, device=x.device)
        out, t = self._inner(x, cu_seqlens, conv_out=conv)
        return x + out, Cache(conv, t["scan"].h_last)

    def step(self, x, cache):
        """y [S, C] of one token x [S, C] per sequence; the cache moves on."""
        P, D, R, N = self.params, self.D, self.R, self.N
        n, _, _ = _seq.layer_norm_fwd(x, P["ln_w"], P["ln_b"], eps=self.eps)
        xz = _mlp.mlp_linear_fwd(n, P["W_in"], None, relu=False)
        u = _seq.causal_conv_step(xz[:, :D], cache.conv, P["conv_w"], P["conv_b"])
        w = _mlp.mlp_linear_fwd(u, P["W_x"], None, relu=False)
        dt = _mlp.mlp_linear_fwd(w[:, :R].contiguous(), P["W_dt"], None, relu=False)
        y = _seq.selective_scan_step(cache.h, u, dt, -torch.exp(P["A_log"]), w[:, R:R + N], w[:, R + N:], skip=P["skip"],
                                     z=xz[:, D:], dt_bias=P["dt_bias"])
        return x + _mlp.mlp_linear_fwd(y, P["W_out"], None, relu=False)


class AdamW:
    """cfc_adamw_step over a dict of parameters, four tensors a launch."""

    def __init__(self, params, lr=1e-3, weight_decay=0.0):
        self.params, self.lr, self.weight_decay, self.t = params, lr, weight_decay, 0
        self.m = {k: torch.zeros_like(v) for k, v in params.items()}
        self.v = {k: torch.zeros_like(v) for k, v in params.items()}

    def step(self, grads):
        self.t += 1
        names = list(self.params)
        for i in range(0, len(names), 4):
            part = names[i:i + 4]
            _cfc.cfc_adamw_step([self.params[k] for k in part], [grads[k] for k in part], [self.m[k] for k in part],
                                [self.v[k] for k in part], self.lr, weight_decay=self.weight_decay, step=self.t)
