"""Training operators without a GPU: what the entry points refuse, and the
gradient formulas against differences of the forward."""

import pytest
import torch

import train_ref as R

F64 = torch.float64


@pytest.fixture(scope="module")
def lib():
    from mixture_experts_layer_24_b200 import build as B
    B.build()
    import mixture_experts_layer_24_b200 as M
    return M.lib()


def test_null_contexts_are_refused(lib):
    N = None
    assert lib.moe_dispatch(N, N, N, 0, N, 1, N, N) == 1
    assert lib.moe_dispatch_bwd(N, N, 0, N, N, N, N, 1, N, N) == 1
    assert lib.moe_combine_weighted(N, N, 0, N, N, 1, N, N) == 1
    assert lib.moe_combine_weighted_bwd(N, N, N, 0, N, N, 1, N, N, N) == 1
    assert lib.moe_swiglu_ckpt(N, N, N, 1, N, N, N, N) == 1
    assert lib.moe_swiglu_ckpt_bwd(N, N, N, N, N, N, 1, N, N, N, N) == 1
    assert lib.moe_route_bwd_workspace_size(N, 4) == 0
    assert lib.moe_route_bwd(N, N, N, N, N, N, N, N, 1, N, N, N, N, 0, N) == 1
    assert lib.moe_expert_product(N, N, N, N, 1, 128, 128, 0, N, N) == 1
    assert lib.moe_expert_wgrad(N, N, N, N, 1, 128, 128, 0, 0, N, N) == 1
    assert b"NULL context" in lib.moe_last_error()


CALLS = ("moe_dispatch", "moe_dispatch_bwd", "moe_combine_weighted", "moe_combine_weighted_bwd", "moe_swiglu_ckpt",
         "moe_swiglu_ckpt_bwd", "moe_route_bwd", "moe_expert_product", "moe_expert_wgrad", "moe_route", "moe_permute",
         "moe_quantize_e4m3")


@pytest.fixture
def host_layer(monkeypatch):
    """A layer on the host whose C calls only note that they were reached: argument checks and allocation run."""
    from mixture_experts_layer_24_b200 import binding as B
    from mixture_experts_layer_24_b200 import train
    calls = []
    for mod in (B, train):
        for name in CALLS:
            if hasattr(mod, name):
                monkeypatch.setattr(mod, name, lambda *a, _n=name, **k: calls.append(_n))
        monkeypatch.setattr(mod, "moe_workspace_size", lambda ctx, T: 4096)
    monkeypatch.setattr(B, "moe_route_bwd_workspace_size", lambda ctx, T: 64)
    L = object.__new__(B.MoeLayer)
    L.H, L.E, L.K, L.I, L.wdtype = 256, 8, 2, 128, B.MOE_BF16
    L.device, L.ctx, L.slots, L._keep, L._ws = torch.device("cpu"), None, None, {}, None
    return L, calls


def _args(T=5):
    H, E, K, I = 256, 8, 2, 128
    z = torch.zeros
    bf, i32 = torch.bfloat16, torch.int32
    return dict(x=z((T, H), dtype=bf), rows=z((T * K, H), dtype=bf), inv=z((T, K), dtype=i32),
                idx=z((T, K), dtype=i32), w=z((T, K)), wr=z((E, H)), offsets=z((E + 1,), dtype=i32),
                perm=z((T * K,), dtype=i32), gu=z((T * K, 2 * I), dtype=bf), dh=z((T * K, I), dtype=bf),
                q=z((T * K, 2 * I), dtype=torch.uint8), s=z((T * K, 2 * I // 128)),
                w_gu=z((E, 2 * I, H), dtype=bf), w_dn=z((E, H, I), dtype=bf))


def test_layer_methods_take_valid_arguments(host_layer):
    L, calls = host_layer
    for T in (5, 0):
        a = _args(T)
        assert L.dispatch(a["x"], a["inv"]).shape == (2 * T, 256)
        assert L.dispatch(a["x"].float(), a["inv"]).dtype == torch.float32
        assert L.dispatch(a["x"].to(torch.uint8), a["inv"], x_scales=torch.zeros(T, 2)).dtype == torch.bfloat16
        assert L.dispatch_bwd(a["rows"], a["inv"]).shape == (T, 256)
        assert L.dispatch_bwd(a["rows"], a["inv"], a["w"], a["idx"], a["wr"], out=a["x"]) is a["x"]
        assert L.combine_weighted(a["rows"].float(), a["w"], a["inv"]).dtype == torch.float32
        dy, dw = L.combine_weighted_bwd(a["x"], a["rows"], a["w"], a["inv"])
        assert dy.shape == (2 * T, 256) and dw.shape == (T, 2)
        h, q, s = L.swiglu_ckpt(a["gu"], a["inv"])
        assert h.shape == (2 * T, 128) and q.shape == (2 * T, 256) and s.shape == (2 * T, 2)
        dgu, hw, dw = L.swiglu_ckpt_bwd(a["q"], a["s"], a["dh"], topk_w=a["w"], inv=a["inv"])
        assert dgu.shape == (2 * T, 256) and hw.shape == (2 * T, 128) and dw.shape == (T, 2)
        assert L.swiglu_ckpt_bwd(a["q"], a["s"], a["dh"])[1:] == (None, None)
        dl, dwr, db = L.route_bwd(a["x"], a["w"], a["w"], a["offsets"], a["perm"], a["perm"])
        assert dl.shape == (T, 2) and dwr.shape == (8, 256) and db.shape == (8,)
        assert L.expert_product(a["rows"], a["w_gu"], a["offsets"]).shape == (2 * T, 256)
        assert L.expert_product(a["rows"], a["w_dn"], a["offsets"], transposed=True).shape == (2 * T, 128)
        assert L.expert_wgrad(a["gu"], a["rows"], a["offsets"], dtype=torch.float32).shape == (8, 256, 256)
    L.swiglu_ckpt(torch.zeros((3, 256), dtype=torch.bfloat16))  # rows that are no whole number of tokens, without inv
    assert len(set(calls)) == 9


def test_layer_methods_refuse_bad_arguments_before_any_call(host_layer):
    L, calls = host_layer
    a = _args()
    half = torch.float16
    bad = [
        lambda: L.dispatch(a["x"].to(half), a["inv"]),
        lambda: L.dispatch(a["x"], a["inv"].long()),
        lambda: L.dispatch(a["x"], a["inv"][:, :1].contiguous()),
        lambda: L.dispatch(a["x"][:, :128], a["inv"]),
        lambda: L.dispatch(a["x"], a["inv"], x_scales=torch.zeros(5, 2)),             # bf16 rows with scales
        lambda: L.dispatch(a["x"].to(torch.uint8), a["inv"]),                         # codes without scales
        lambda: L.dispatch(a["x"].to(torch.uint8), a["inv"], x_scales=torch.zeros(5, 1)),
        lambda: L.dispatch(a["x"], a["inv"], out=a["x"]),
        lambda: L.dispatch_bwd(a["rows"][:-1], a["inv"]),
        lambda: L.dispatch_bwd(a["rows"].t().contiguous().t(), a["inv"]),              # not row-major
        lambda: L.dispatch_bwd(a["rows"], a["inv"], dlogit=a["w"]),                   # the router's three go together
        lambda: L.dispatch_bwd(a["rows"], a["inv"], a["w"], a["idx"], a["wr"][:4]),
        lambda: L.combine_weighted(a["rows"], a["w"].double(), a["inv"]),
        lambda: L.combine_weighted(a["rows"], a["w"], a["inv"], out=a["x"].float()),
        lambda: L.combine_weighted_bwd(a["x"].float(), a["rows"], a["w"], a["inv"]),   # two row types
        lambda: L.swiglu_ckpt(a["gu"].float(), a["inv"]),
        lambda: L.swiglu_ckpt(a["gu"][:-1].contiguous(), a["inv"]),
        lambda: L.swiglu_ckpt(a["dh"], a["inv"]),
        lambda: L.swiglu_ckpt_bwd(a["q"].to(torch.int8), a["s"], a["dh"]),
        lambda: L.swiglu_ckpt_bwd(a["q"], a["s"][:, :1].contiguous(), a["dh"]),
        lambda: L.swiglu_ckpt_bwd(a["q"], a["s"], a["dh"], topk_w=a["w"][:2]),
        lambda: L.swiglu_ckpt_bwd(a["q"], a["s"], a["dh"], out=(a["gu"], a["dh"])),   # hw without weights
        lambda: L.route_bwd(a["x"].float(), a["w"], a["w"], a["offsets"], a["perm"], a["perm"]),
        lambda: L.route_bwd(a["x"], a["w"], a["w"], a["offsets"][:-1], a["perm"], a["perm"]),
        lambda: L.route_bwd(a["x"], a["w"], a["w"], a["offsets"], a["perm"][:-1], a["perm"]),
        lambda: L.route_bwd(a["x"], a["w"], a["w"], a["offsets"], a["perm"], a["perm"], x_scales=torch.zeros(5, 2)),
        lambda: L.expert_product(a["rows"], a["w_gu"][:4], a["offsets"]),
        lambda: L.expert_product(a["rows"], a["w_gu"][0], a["offsets"]),
        lambda: L.expert_product(a["rows"], a["w_dn"], a["offsets"]),                  # K does not match
        lambda: L.expert_product(a["rows"].float(), a["w_gu"], a["offsets"]),
        lambda: L.expert_wgrad(a["gu"], a["rows"][:-1], a["offsets"]),
        lambda: L.expert_wgrad(a["gu"], a["rows"], a["offsets"], dtype=half),
        lambda: L.expert_wgrad(a["gu"], a["rows"], a["offsets"], accumulate=True),     # nothing to add to
        lambda: L.expert_wgrad(a["gu"], a["rows"], a["offsets"], out=torch.zeros(8, 256, 128)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((TypeError, ValueError)):
            f()
        assert not calls, f"bad call {i} reached the C ABI"


def test_router_gradient_takes_the_choice_or_a_list_of_pairs(host_layer, monkeypatch):
    from mixture_experts_layer_24_b200 import binding as B
    L, calls = host_layer
    monkeypatch.setattr(B, "moe_route_bwd_topk_workspace_size", lambda ctx, T: 64)
    monkeypatch.setattr(B, "moe_route_bwd_topk", lambda *a, **k: calls.append("moe_route_bwd_topk"))
    a = _args()
    bad = [
        lambda: L.route_bwd(a["x"], a["w"], a["w"]),
        lambda: L.route_bwd(a["x"], a["w"], a["w"], a["offsets"], a["perm"], a["perm"], topk_idx=a["idx"]),
        lambda: L.route_bwd(a["x"], a["w"], a["w"], perm_k=a["perm"], topk_idx=a["idx"]),
        lambda: L.route_bwd(a["x"], a["w"], a["w"], topk_idx=a["idx"].long()),
        lambda: L.route_bwd(a["x"], a["w"], a["w"], topk_idx=a["idx"][:-1]),
        lambda: L.route_bwd(a["x"], a["w"][:, :1], a["w"], topk_idx=a["idx"]),
    ]
    for f in bad:
        with pytest.raises((TypeError, ValueError)):
            f()
    assert not calls
    dl, dwr, db = L.route_bwd(a["x"], a["w"], a["w"], topk_idx=a["idx"])
    assert dl.shape == (5, 2) and dwr.shape == (8, 256) and db.shape == (8,) and calls == ["moe_route_bwd_topk"]


def test_router_gradient_of_a_null_context_is_refused(lib):
    N = None
    assert lib.moe_route_bwd_topk_workspace_size(N, 4) == 0
    assert lib.moe_route_bwd_topk(N, N, N, N, N, N, 1, N, N, N, N, 0, N) == 1


def test_train_step_order_of_calls(host_layer):
    from mixture_experts_layer_24_b200 import train
    L, calls = host_layer
    a = _args()
    out, saved = train.forward(L, a["x"], a["wr"], a["w_gu"], a["w_dn"], ckpt_x=True)
    assert out.shape == a["x"].shape and saved.x.dtype == torch.uint8
    g = train.backward(L, saved, a["x"], a["wr"], a["w_gu"], a["w_dn"], w_dtype=torch.float32)
    assert g.w_gu.shape == a["w_gu"].shape and g.w_dn.shape == a["w_dn"].shape and g.w_gu.dtype == torch.float32
    assert calls == ["moe_route", "moe_permute", "moe_dispatch", "moe_expert_product", "moe_swiglu_ckpt",
                     "moe_expert_product", "moe_combine_weighted", "moe_quantize_e4m3", "moe_dispatch", "moe_dispatch",
                     "moe_expert_product", "moe_swiglu_ckpt_bwd", "moe_expert_wgrad", "moe_expert_wgrad",
                     "moe_expert_product", "moe_route_bwd", "moe_dispatch_bwd"]
    with pytest.raises((TypeError, ValueError)):
        train.forward(L, a["x"], a["wr"], a["w_dn"], a["w_gu"])


def test_train_backward_refuses_before_any_call(host_layer):
    """A backward pass that is refused has launched nothing: a gradient it should add to is never half updated."""
    from dataclasses import replace
    from mixture_experts_layer_24_b200 import train
    L, calls = host_layer
    a, half, f32 = _args(), torch.float16, torch.float32
    _, saved = train.forward(L, a["x"], a["wr"], a["w_gu"], a["w_dn"], ckpt_x=True)
    _, plain = train.forward(L, a["x"], a["wr"], a["w_gu"], a["w_dn"])
    into = (torch.zeros(a["w_gu"].shape), torch.zeros(a["w_dn"].shape))
    odd = lambda t: torch.zeros(t.numel() + 1, dtype=t.dtype)[1:].view(t.shape)  # noqa: E731  not 16-byte aligned
    calls.clear()

    def back(s=saved, dout=a["x"], wr=a["wr"], w_gu=a["w_gu"], w_dn=a["w_dn"], **more):
        return train.backward(L, s, dout, wr, w_gu, w_dn, **more)

    bad = [
        lambda: back(into=(into[0][:, :-1], into[1])),
        lambda: back(into=(into[0].to(torch.bfloat16), into[1])),
        lambda: back(into=(into[0], into[1].to(torch.bfloat16))),
        lambda: back(into=(into[0].transpose(1, 2).contiguous().transpose(1, 2), into[1])),
        lambda: back(into=(odd(into[0]), into[1])),
        lambda: back(into=(into[1], into[0])),
        lambda: back(into=(None, into[1])),
        lambda: back(into=into, w_dtype=torch.bfloat16),
        lambda: back(w_dtype=half),
        lambda: back(into=into, dout=a["x"][:-1]),
        lambda: back(into=into, dout=a["x"].float()),
        lambda: back(into=into, wr=a["wr"].double()),
        lambda: back(into=into, wr=odd(a["wr"])),
        lambda: back(into=into, w_gu=odd(a["w_gu"])),
        lambda: back(into=into, w_gu=a["w_dn"]),
        lambda: back(into=into, s=replace(saved, x_scales=None)),
        lambda: back(into=into, s=replace(saved, topk_w=saved.topk_w[:-1])),
        lambda: back(into=into, s=replace(plain, perm_k=plain.perm_k.long())),
        lambda: back(into=into, s=replace(saved, gu_q=saved.gu_q[:, :-1])),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((TypeError, ValueError)):
            f()
        assert not calls, f"bad call {i} reached the C ABI"
    for s in (saved, plain):
        g = back(s=s, into=into, w_dtype=f32)
        assert g.w_gu is into[0] and g.w_dn is into[1]
        assert back(s=s, into=into).w_gu is into[0]
        assert back(s=s).w_gu.dtype == torch.bfloat16 and back(s=s, w_dtype=f32).w_dn.dtype == f32


def test_weight_gradient_of_another_type_than_its_output_is_refused(host_layer):
    L, calls = host_layer
    a, f32, bf16 = _args(), torch.float32, torch.bfloat16
    out = torch.zeros((8, 256, 256))
    for kw in (dict(dtype=bf16, out=out), dict(dtype=f32, out=out.to(bf16)), dict(out=out.to(bf16), accumulate=True),
               dict(out=out.double()), dict(out=[0])):
        with pytest.raises((TypeError, ValueError)):
            L.expert_wgrad(a["gu"], a["rows"], a["offsets"], **kw)
    assert not calls
    assert L.expert_wgrad(a["gu"], a["rows"], a["offsets"]).dtype == bf16
    assert L.expert_wgrad(a["gu"], a["rows"], a["offsets"], out=out) is out
    assert L.expert_wgrad(a["gu"], a["rows"], a["offsets"], dtype=f32, out=out, accumulate=True) is out


def _difference(f, v, i, step=1e-6):
    """Central difference of f at flat place i of v (float64: error about step^2 + eps/step, 1e-10 of f's scale)."""
    keep = v.reshape(-1)[i].item()
    v.reshape(-1)[i] = keep + step
    up = f().item()
    v.reshape(-1)[i] = keep - step
    down = f().item()
    v.reshape(-1)[i] = keep
    return (up - down) / (2 * step)


def test_gradient_formulas_against_differences():
    """The formulas the kernels are held to (train_ref), chained as one backward pass, against central differences
    of the layer's loss in 64 bits: input, router, bias and both expert weights."""
    T, H, E, K, I = 6, 8, 5, 3, 4
    r = R.routing(T, K, E, seed=3)
    g = torch.Generator().manual_seed(4)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=F64)  # noqa: E731
    x, wr, bias, w_gu, w_dn, dout = rnd(T, H), rnd(E, H), rnd(E), rnd(E, 2 * I, H), rnd(E, H, I), rnd(T, H)
    idx = r["idx"]
    loss = lambda: R.layer_loss(x, wr, bias, w_gu, w_dn, dout, idx)  # noqa: E731
    # the backward pass from the formulas
    w = torch.softmax(torch.gather(x @ wr.t() + bias, 1, idx.long()), 1)
    src, pk, inv, offsets = r["perm_src"].long(), r["perm_k"].long(), r["inv"], r["offsets"]
    xs, dys = x[src], dout[src]
    gu, _ = R.products(xs, w_gu, offsets, False)
    dh, _ = R.products(dys, w_dn, offsets, True)
    dg, du, h, dw_rows = R.swiglu_bwd(gu[:, :I], gu[:, I:], dh, w[src, pk])
    dgu = torch.cat((dg, du), 1)
    dw = dw_rows[inv.long()]
    d_dn, _ = R.wgrads(dys, w[src, pk][:, None] * h, offsets)
    d_gu, _ = R.wgrads(dgu, xs, offsets)
    dxs, _ = R.products(dgu, w_gu, offsets, True)
    dl, d_wr, d_bias = R.route_bwd(x, w, dw, idx, inv, E)[:3]
    dx, _ = R.dispatch_bwd(dxs, inv, dl, idx, wr)
    # the same weights' gradient through the combine
    y, _ = R.products(h, w_dn, offsets, False)
    assert torch.allclose(R.combine_bwd(dout, y, w, inv)[1], dw, rtol=1e-10, atol=1e-12)
    for value, grad in ((x, dx), (wr, d_wr), (bias, d_bias), (w_gu, d_gu), (w_dn, d_dn)):
        at = torch.randperm(value.numel(), generator=g)[:12].tolist()
        for i in at:
            d = _difference(loss, value, i)
            assert abs(d - grad.reshape(-1)[i].item()) <= 1e-6 * (1 + abs(d)), i


def test_router_gradient_formula_with_dropped_pairs():
    """The router's gradient sums over every chosen pair: with pairs and a whole token dropped, the formula over all
    pairs is autograd's, and the formula over the kept ones is not."""
    T, K, E, H = 9, 3, 7, 16
    r = R.routing(T, K, E, seed=5, drop=0.3, drop_token=4)
    g = torch.Generator().manual_seed(6)
    x, wr, dw = (torch.randn(*s, generator=g, dtype=F64) for s in ((T, H), (E, H), (T, K)))
    rows = torch.randn(T * K, H, generator=g, dtype=F64)
    dx_ref, dwr_ref, db_ref = R.route_bwd_by_autograd(x, wr, r["w"], dw, r["idx"], rows, r["inv"])
    kept = r["inv"] >= 0
    assert 3 < int((~kept).sum()) < T * K
    dw = torch.where(kept, dw, torch.zeros((), dtype=F64))
    w = r["w"].to(F64) / r["w"].to(F64).sum(1, keepdim=True)
    everyone = torch.zeros_like(r["inv"])  # no pair marked as dropped
    dl, dwr, db = R.route_bwd(x, w, dw, r["idx"], everyone, E)[:3]
    dx, _ = R.dispatch_bwd(rows, r["inv"], dl, r["idx"], wr)
    for got, ref in ((dx, dx_ref), (dwr, dwr_ref), (db, db_ref)):
        assert torch.allclose(got, ref, rtol=1e-12, atol=1e-12)
    listed = R.route_bwd(x, w, dw, r["idx"], r["inv"], E)[1]
    assert (listed - dwr_ref).norm() > 0.1 * dwr_ref.norm()


def test_oracle_quantiser_is_the_checkpoint_rule():
    """The e4m3 rule of the checkpoint against its statement, and how far a decoded value may be off: half a step
    of e4m3 relative to the value (2^-4), or of its subnormals (2^-10 of the scale), and fp32's roundings."""
    import oracle
    g = torch.Generator().manual_seed(7)
    v = (torch.randn(9, 512, generator=g) * torch.logspace(-3, 3, 9)[:, None]).to(torch.bfloat16)
    v[4, :128] = 0
    q, s = oracle.quant_e4m3(oracle.as_u16(v), 1)
    q, s = torch.from_numpy(q), torch.from_numpy(s)
    back, x = R.decode(q, s), v.to(F64)
    step = s.to(F64).repeat_interleave(128, 1)
    assert ((back - x).abs() <= (2 ** -4 * x.abs()).maximum(2 ** -10 * step) * (1 + 2 ** -20)).all()
    assert (s[4, 0] == 1) and (q[4, :128] == 0).all()
