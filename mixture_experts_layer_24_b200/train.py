"""One training step of a routed MoE layer: forward with 8-bit checkpoints, and
the gradients of its input, router and experts.

Forward (``forward``), on T tokens x [T, H] bf16:

1. ``route`` and ``permute`` as in serving;
2. ``dispatch``: the tokens' rows in expert order;
3. ``expert_product`` with w_gu [E, 2I, H]; ``swiglu_ckpt``: h, and the gate/up
   values kept as e4m3 codes with one scale per 128 columns;
4. ``expert_product`` with w_dn [E, H, I]; ``combine_weighted``: out [T, H].

Kept for the backward pass: the routing, the gate/up checkpoint (1 byte per
value), and x -- the caller's own tensor, or (``ckpt_x=True``) an e4m3
checkpoint of it. Neither h nor any expert row is kept.

Backward (``backward``), from dout [T, H] bf16:

1. ``dispatch`` of dout; ``expert_product`` with w_dn transposed: the gradient
   that reaches h before the routing weight;
2. ``swiglu_ckpt_bwd``: the gate/up gradient, w * h, and the weights' gradient
   <dh, h> (so the down product's output is not needed);
3. ``expert_wgrad`` for w_dn (dout rows, w * h) and w_gu (gate/up gradient, x
   rows);
4. ``expert_product`` with w_gu transposed, ``route_bwd``, and ``dispatch_bwd``,
   which sums each token's rows and adds the router's share.

The gate/up values round to bf16 between the product and the activation, and
the experts' outputs before the combine, so ``forward`` agrees with
``MoeLayer.forward`` to bf16 accuracy, not to the bit. Gradients are those of
the layer at the checkpointed gate/up values. Weights are stacked per expert;
views of them can be registered with the same ``MoeLayer`` for serving.

All arithmetic runs in libmoe's kernels, on the current stream; nothing reads
the device from the host, so both passes may be captured in a CUDA graph.
"""

from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

import torch

from .binding import _rows, _want, check_tensor, moe_permute, moe_quantize_e4m3, moe_route, moe_workspace_size


@dataclass
class Saved:
    """What one forward keeps for its backward."""
    x: torch.Tensor                    # [T, H] bf16, or uint8 e4m3 codes
    x_scales: Optional[torch.Tensor]   # [T, H/128] fp32 with codes, else None
    topk_idx: torch.Tensor             # [T, K] int32
    topk_w: torch.Tensor               # [T, K] fp32
    offsets: torch.Tensor              # [E+1] int32
    perm_src: torch.Tensor             # [T*K] int32
    perm_k: torch.Tensor               # [T*K] int32
    inv: torch.Tensor                  # [T, K] int32
    gu_q: torch.Tensor                 # [T*K, 2I] uint8 e4m3 codes
    gu_s: torch.Tensor                 # [T*K, 2I/128] fp32


@dataclass
class Grads:
    """Gradients of one step."""
    x: torch.Tensor                    # [T, H] bf16
    w_router: torch.Tensor             # [E, H] fp32
    logit_bias: torch.Tensor           # [E] fp32
    w_gu: torch.Tensor                 # [E, 2I, H]
    w_dn: torch.Tensor                 # [E, H, I]


def _check_weights(layer, w_gu, w_dn):
    check_tensor(w_gu, "w_gu", torch.bfloat16, (layer.E, 2 * layer.I, layer.H), layer.device)
    check_tensor(w_dn, "w_dn", torch.bfloat16, (layer.E, layer.H, layer.I), layer.device)


def _check_backward(layer, s, dout, w_router, w_gu, w_dn, w_dtype, into):
    """All that a call of ``backward`` could refuse, before its first launch: a step that was half done would have added
    to one of ``into`` and not to the other."""
    H, E, K, I, d = layer.H, layer.E, layer.K, layer.I, layer.device
    bf16, f32, i32, u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
    _check_weights(layer, w_gu, w_dn)
    T = _rows(dout, "dout")
    ckpt_x = s.x_scales is not None
    wanted = [("dout", dout, bf16, (T, H)), ("w_router", w_router, f32, (E, H)),
              ("saved.x", s.x, u8 if ckpt_x else bf16, (T, H)), ("saved.topk_idx", s.topk_idx, i32, (T, K)),
              ("saved.topk_w", s.topk_w, f32, (T, K)), ("saved.offsets", s.offsets, i32, (E + 1,)),
              ("saved.perm_src", s.perm_src, i32, (T * K,)), ("saved.perm_k", s.perm_k, i32, (T * K,)),
              ("saved.inv", s.inv, i32, (T, K)), ("saved.gu_q", s.gu_q, u8, (T * K, 2 * I)),
              ("saved.gu_s", s.gu_s, f32, (T * K, 2 * I // 128))]
    if ckpt_x:
        wanted.append(("saved.x_scales", s.x_scales, f32, (T, H // 128)))
    if into is not None:
        if w_dtype is not None and w_dtype != f32:
            raise TypeError(f"w_dtype: {w_dtype}, but gradients are added to fp32 tensors")
        into_gu, into_dn = into
        wanted += [("into[0]", into_gu, f32, w_gu.shape), ("into[1]", into_dn, f32, w_dn.shape)]
    elif w_dtype not in (None, bf16, f32):
        raise TypeError(f"w_dtype: {w_dtype}, expected bf16 or fp32")
    for name, t, dtype, shape in wanted:
        _want(t, name, dtype, shape, d)
    for name, t in (("w_gu", w_gu), ("w_dn", w_dn), ("w_router", w_router), ("dout", dout), ("saved.x", s.x),
                    ("saved.gu_q", s.gu_q), ("into[0]", into and into[0]), ("into[1]", into and into[1])):
        if t is not None and t.data_ptr() % 16:
            raise ValueError(f"{name}: must be 16-byte aligned")


def _route_and_permute(layer, x, w_router, logit_bias):
    """layer.route and layer.permute on a workspace of this call's own: a captured step must not share the layer's,
    which a later, larger call replaces."""
    T, K, d = layer._check_route_inputs(x, w_router, logit_bias), layer.K, layer.device
    ws = torch.empty(max(moe_workspace_size(layer.ctx, T), 256), dtype=torch.uint8, device=d)

    def ints(*shape):
        return torch.empty(shape, dtype=torch.int32, device=d)

    idx, w = ints(T, K), torch.empty((T, K), dtype=torch.float32, device=d)
    moe_route(layer.ctx, x, w_router, logit_bias, T, idx, w, ws)
    counts, offsets, perm_src, perm_k, inv = ints(layer.E), ints(layer.E + 1), ints(T * K), ints(T * K), ints(T, K)
    moe_permute(layer.ctx, idx, T, counts, offsets, perm_src, perm_k, inv, ws)
    return idx, w, offsets, perm_src, perm_k, inv


def forward(layer, x, w_router, w_gu, w_dn, logit_bias=None, ckpt_x=False):
    """(out [T, H] bf16, Saved) of one training forward on the layer's context.

    With ckpt_x the router's gradient and that of w_gu use x as its e4m3
    checkpoint holds it; otherwise x is kept by reference and must not change
    before ``backward``."""
    _check_weights(layer, w_gu, w_dn)
    with layer._on(None):
        topk_idx, topk_w, offsets, perm_src, perm_k, inv = _route_and_permute(layer, x, w_router, logit_bias)
        gu = layer.expert_product(layer.dispatch(x, inv), w_gu, offsets)
        h, gu_q, gu_s = layer.swiglu_ckpt(gu, inv)
        del gu
        out = layer.combine_weighted(layer.expert_product(h, w_dn, offsets), topk_w, inv)
        kept, scales = x, None
        if ckpt_x:
            T, H = x.shape
            kept = torch.empty((T, H), dtype=torch.uint8, device=layer.device)
            scales = torch.empty((T, H // 128), dtype=torch.float32, device=layer.device)
            moe_quantize_e4m3(x, T, H, 1, kept, scales)
    return out, Saved(kept, scales, topk_idx, topk_w, offsets, perm_src, perm_k, inv, gu_q, gu_s)


def backward(layer, saved, dout, w_router, w_gu, w_dn, w_dtype=None, into=None):
    """Grads of one step from dout [T, H] bf16 and the forward's Saved.

    The experts' weight gradients come in w_dtype (bf16, the default, or fp32);
    ``into``, a pair of fp32 tensors (w_gu's, w_dn's), has them added to what it
    holds (gradient accumulation) and returned instead. Arguments are checked
    before anything is launched or added to."""
    s = saved
    _check_backward(layer, s, dout, w_router, w_gu, w_dn, w_dtype, into)
    into_gu, into_dn = into if into is not None else (None, None)
    add = into is not None
    with layer._on(None):
        xs = layer.dispatch(s.x, s.inv, x_scales=s.x_scales)
        dys = layer.dispatch(dout, s.inv)
        dh = layer.expert_product(dys, w_dn, s.offsets, transposed=True)
        dgu, hw, dtopk_w = layer.swiglu_ckpt_bwd(s.gu_q, s.gu_s, dh, topk_w=s.topk_w, inv=s.inv)
        del dh
        dw_dn = layer.expert_wgrad(dys, hw, s.offsets, dtype=w_dtype, out=into_dn, accumulate=add)
        del dys, hw
        dw_gu = layer.expert_wgrad(dgu, xs, s.offsets, dtype=w_dtype, out=into_gu, accumulate=add)
        del xs
        dxs = layer.expert_product(dgu, w_gu, s.offsets, transposed=True)
        del dgu
        dlogit, dw_router, dbias = layer.route_bwd(s.x, s.topk_w, dtopk_w, s.offsets, s.perm_src, s.perm_k,
                                                   x_scales=s.x_scales)
        dx = layer.dispatch_bwd(dxs, s.inv, dlogit=dlogit, topk_idx=s.topk_idx, w_router=w_router)
    return Grads(dx, dw_router, dbias, dw_gu, dw_dn)
