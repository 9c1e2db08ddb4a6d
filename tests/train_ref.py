"""Plain 64-bit forms of the training operators, for the tests. Every function
takes and returns float64 tensors (or the tensors' own bits where nothing is
computed); `inv` [T, K] holds each pair's row, negative for a dropped pair."""

import torch

F64 = torch.float64
BF16_HALF = torch.finfo(torch.bfloat16).eps / 2  # largest relative error of one rounding to bf16
F32_HALF = torch.finfo(torch.float32).eps / 2


def half(dtype):
    return BF16_HALF if dtype == torch.bfloat16 else F32_HALF


def routing(T, K, E, seed, drop=0.0, drop_token=None, skew=1.1):
    """Distinct experts per token under a Zipf prior, weights, and the sort of the kept pairs (CPU tensors)."""
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(T, E, generator=g, dtype=F64) - skew * torch.log(1.0 + torch.arange(E, dtype=F64))
    top = torch.topk(logits, K, dim=1)
    idx = top.indices
    key = idx.clone()
    key[torch.rand(T, K, generator=g) < drop] = E
    if drop_token is not None:
        key[drop_token] = E
    flat = key.reshape(-1)
    order = torch.argsort(flat, stable=True)
    inv = torch.empty(T * K, dtype=torch.int64)
    inv[order] = torch.arange(T * K)
    inv[flat >= E] = -1
    offsets = torch.zeros(E + 1, dtype=torch.int64)
    offsets[1:] = torch.cumsum(torch.bincount(flat, minlength=E + 1)[:E], 0)
    n = int(offsets[E])
    perm_src, perm_k = order // K, order % K
    perm_src[n:] = 2 ** 30  # nothing reads the places behind the kept pairs
    perm_k[n:] = 2 ** 30
    i32 = torch.int32
    return dict(idx=idx.to(i32), w=torch.softmax(top.values, 1).float(), inv=inv.view(T, K).to(i32),
                offsets=offsets.to(i32), perm_src=perm_src.to(i32), perm_k=perm_k.to(i32), n=n)


def gathered(rows, inv):
    """rows[inv] with zeros for dropped pairs, whatever the rows behind them hold: [T, K, H]."""
    kept = (inv >= 0)[..., None]
    return torch.where(kept, rows[inv.clamp(min=0).long()].to(F64), torch.zeros((), dtype=F64, device=rows.device))


def dispatch_bwd(rows, inv, dl=None, idx=None, wr=None):
    """(dx, sum of the terms' absolute values)."""
    g = gathered(rows, inv)
    dx, mag = g.sum(1), g.abs().sum(1)
    if dl is not None:
        r = dl.to(F64)[..., None] * wr.to(F64)[idx.long()]
        dx, mag = dx + r.sum(1), mag + r.abs().sum(1)
    return dx, mag


def combine(y, w, inv):
    g = gathered(y, inv) * w.to(F64)[..., None]
    return g.sum(1), g.abs().sum(1)


def combine_bwd(dout, y, w, inv):
    """(w dout per pair [T, K, H], dw [T, K], sum of |terms| of dw)."""
    d = dout.to(F64)[:, None]
    g = gathered(y, inv) * d
    return w.to(F64)[..., None] * d, g.sum(-1), g.abs().sum(-1)


def decode(q, s):
    """Values of an e4m3 checkpoint: codes (uint8) times scales."""
    v = q.view(torch.float8_e4m3fn).to(F64).view(*q.shape[:-1], -1, 128) * s.to(F64)[..., None]
    return v.view(q.shape)


def silu_parts(g):
    sig = 1.0 / (1.0 + torch.exp(-g))
    return sig, g * sig


def swiglu_bwd(g, u, dh, w):
    """(dg, du, h, dw) with a weight per row (all float64)."""
    sig, silu = silu_parts(g)
    h = silu * u
    wd = w[:, None] * dh
    return wd * u * sig * (1 + g * (1 - sig)), wd * silu, h, (dh * h).sum(1)


def route_bwd(x, w, dw, idx, inv, E):
    """(dlogit, dWr, dbias, and the sums of |terms| of each)."""
    w, dw = w.to(F64), dw.to(F64)
    dot, mag_dot = (w * dw).sum(1, keepdim=True), (w * dw).abs().sum(1, keepdim=True)
    dl = w * (dw - dot)
    mag = w * (dw.abs() + mag_dot)
    kept = (inv >= 0).to(F64)
    full = torch.zeros(x.shape[0], E, dtype=F64, device=x.device).scatter_add_(1, idx.long(), dl * kept)
    fmag = torch.zeros_like(full).scatter_add_(1, idx.long(), mag * kept)
    return dl, full.t() @ x.to(F64), full.sum(0), mag, fmag.t() @ x.to(F64).abs(), fmag.sum(0)


def route_bwd_by_autograd(x, wr, w, dw, idx, rows, inv):
    """(dx, dWr, dbias) in float64, by autograd, of a loss that sees the routing weights and the kept rows:
    sum over kept pairs of softmax(l)[t,k] * dw[t,k] + <x[t], rows[inv[t,k]]>, where l = x Wr^T + b over the K chosen
    logits is shifted by constants so that softmax(l) is w. Dropped pairs are in the softmax and nowhere else."""
    x, wr = x.to(F64).clone().requires_grad_(), wr.to(F64).clone().requires_grad_()
    b = torch.zeros(wr.shape[0], dtype=F64, device=x.device, requires_grad=True)
    kept = inv >= 0
    upstream = torch.where(kept, dw.to(F64), torch.zeros((), dtype=F64, device=x.device))
    logits = torch.gather(x @ wr.t() + b, 1, idx.long())
    weights = torch.softmax(logits + (torch.log(w.to(F64)) - logits).detach(), 1)
    ((weights * upstream).sum() + (x[:, None] * gathered(rows, inv)).sum()).backward()
    return x.grad, wr.grad, b.grad


def products(a, w, offsets, transposed):
    """(out, sum of |terms|) of the kept rows."""
    cut = offsets.tolist()
    f = (lambda m: m.to(F64)) if transposed else (lambda m: m.to(F64).t())
    parts = [(a[i:j].to(F64) @ f(m), a[i:j].to(F64).abs() @ f(m).abs()) for i, j, m in zip(cut, cut[1:], w)]
    return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])


def wgrads(dy, a, offsets):
    cut = offsets.tolist()
    d, b = dy.to(F64), a.to(F64)
    return (torch.stack([d[i:j].t() @ b[i:j] for i, j in zip(cut, cut[1:])]),
            torch.stack([d[i:j].abs().t() @ b[i:j].abs() for i, j in zip(cut, cut[1:])]))


def layer_loss(x, wr, bias, w_gu, w_dn, dout, idx, gu_at=None):
    """<out, dout> of the layer with the given choice of experts, in float64 and differentiable. gu_at: the gate/up
    values of every pair [T, K, 2I] to use in place of the products' own values (their gradient passes through)."""
    K, I = idx.shape[1], w_dn.shape[2]
    logits = x @ wr.t() + bias
    w = torch.softmax(torch.gather(logits, 1, idx.long()), 1)
    out = 0
    for k in range(K):
        gu = torch.einsum("toh,th->to", w_gu[idx[:, k].long()], x)
        if gu_at is not None:
            gu = gu + (gu_at[:, k] - gu).detach()
        g, u = gu[:, :I], gu[:, I:]
        out = out + w[:, k, None] * torch.einsum("thi,ti->th", w_dn[idx[:, k].long()], g * torch.sigmoid(g) * u)
    return (out * dout).sum()
