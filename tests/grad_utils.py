"""64-bit definitions of the forward passes in torch, whose autograd gives the gradients that the kernels are held to.

The rule runs token by token (``rule``), so it shares nothing with the kernels' chunkwise algebra.  The CPU
tests hold these definitions to the C oracle and their gradients to central differences of that oracle.
"""
from __future__ import annotations

import math

import torch


def rule(q, k, v, g, beta, s0, lens, qk_l2norm=True, scale=0.0):
    """(out, final_state) of the gated delta rule over packed sequences, in the inputs' precision."""
    nqk, dk = q.shape[1:]
    nv, dv = v.shape[1:]
    group = nv // nqk
    scale = scale if scale > 0 else 1.0 / math.sqrt(dk)
    if qk_l2norm:
        q, k = (x / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-6) for x in (q, k))
    q, k = (x.repeat_interleave(group, 1) for x in (q * scale, k))
    outs, finals, t = [], [], 0
    for n, length in enumerate(lens):
        s = s0[n] if s0 is not None else torch.zeros(nv, dk, dv, dtype=q.dtype, device=q.device)
        for _ in range(length):
            s = s * torch.exp(g[t])[:, None, None]
            delta = beta[t][:, None] * (v[t] - torch.einsum("hdc,hd->hc", s, k[t]))
            s = s + k[t][:, :, None] * delta[:, None, :]
            outs.append(torch.einsum("hdc,hd->hc", s, q[t]))
            t += 1
        finals.append(s)
    out = torch.stack(outs) if outs else torch.zeros(0, nv, dv, dtype=q.dtype, device=q.device)
    return out, torch.stack(finals)


def rule_grads(q, k, v, g, beta, s0, dout, ds, lens, **kw):
    """(dq, dk, dv, dg, dbeta, ds0) in 64 bits on the CPU; s0 and ds may be None."""
    x = [t.detach().cpu().double().requires_grad_() for t in (q, k, v, g, beta)]
    n, nv, dk, dv = len(lens), v.shape[1], q.shape[2], v.shape[2]
    st = (s0.detach().cpu().double() if s0 is not None else torch.zeros(n, nv, dk, dv).double()).requires_grad_()
    out, fin = rule(*x, st, lens, **kw)
    seeds = [dout.detach().cpu().double(), ds.detach().cpu().double() if ds is not None else torch.zeros_like(fin)]
    return torch.autograd.grad([out, fin], x + [st], seeds)


def gate(a, b, A_log, dt_bias):
    """(g, beta) of the layer's gate."""
    u = a + dt_bias
    return (-torch.exp(A_log) * (torch.clamp(u, min=0) + torch.log1p(torch.exp(-u.abs()))), torch.sigmoid(b))


def norm(o, z, w, eps):
    return o / torch.sqrt((o * o).mean(-1, keepdim=True) + eps) * w * (z * torch.sigmoid(z))


def conv(x, w, b, state, lens):
    """(y [T, C], new state [N, C, K]) of the causal conv + SiLU over packed sequences."""
    k, rows, states, t = w.shape[1], [], [], 0
    for n, length in enumerate(lens):
        window = state[n].t() if state is not None else torch.zeros(k, x.shape[1], dtype=x.dtype, device=x.device)
        line = torch.cat([window, x[t:t + length]])
        pre = sum(w[:, i] * line[1 + i:1 + i + length] for i in range(k))
        pre = pre + b if b is not None else pre
        rows.append(pre * torch.sigmoid(pre))
        states.append(line[len(line) - k:].t())
        t += length
    return torch.cat(rows), torch.stack(states)


def assert_close(got, want, io, what, floor=0.0):
    """Every element within the rounding of its type and the arithmetic of the path.

    fp32: operands are pairs hi + lo, each product within 2^-22 of its value, and sums run over at
    most 128 terms in fp32 (2^-24 sqrt(128) < 2^-20); a gradient passes through at most about 16 such
    products, so 16 * 2^-20 = 2^-16 of the largest element bounds it.  bf16: the same plus one rounding of
    the output, half a step = 2^-8 of the element, and operands that may be held to fp16's 2^-12 in place of
    pairs: through 4 of them, 2^-10 of the largest element.
    """
    got, want = got.detach().cpu().double(), want.detach().cpu().double()
    assert got.shape == want.shape, what
    assert torch.isfinite(got).all(), what
    if want.numel() == 0:
        return
    top = max(want.abs().max().item(), floor)
    bound = 2.0 ** -16 * top if io == torch.float32 else 2.0 ** -8 * want.abs() + 2.0 ** -10 * top
    over = ((got - want).abs() - bound).max().item()
    assert over <= 0, "%s: %g over its bound (largest element %g)" % (what, over, top)
