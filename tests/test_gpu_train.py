"""The training operators on the GPU against their plain 64-bit forms
(train_ref): sizes from one token up, dropped pairs and tokens, rows that hold
NaN where nothing may be read, refusals, streams and graphs, and a whole step.

Tolerances count the roundings: one rounding is at most half a step
(bf16 2^-8, fp32 2^-24 relative to the value); n fp32 additions or fused
multiply-adds in any order are within n * 2^-24 of the sum of the terms'
magnitudes (to first order; the factor 1.01 covers the rest)."""

import numpy as np
import pytest
import torch

import oracle
import train_ref as R

pytestmark = pytest.mark.gpu

F64 = torch.float64
BF16, F32 = torch.bfloat16, torch.float32
U = R.F32_HALF  # 2^-24


@pytest.fixture(scope="module", autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


@pytest.fixture(scope="module")
def layers():
    import mixture_experts_layer_24_b200 as M
    made = {}

    def get(H, E, K, I=128):
        if (H, E, K, I) not in made:
            made[H, E, K, I] = M.MoeLayer(H, E, K, I)
        return made[H, E, K, I]

    yield get
    for L in made.values():
        L.close()


def _cuda(r):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in r.items()}


def _rand(seed, *shape, std=1.0, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _poison_behind(rows, n):
    """Rows that no kept pair names hold NaN and infinity: nothing may read them."""
    rows[n:] = float("nan")
    if rows.shape[0] > n + 1:
        rows[n + 1] = float("inf")
    return rows


def _within(got, ref, bound, what):
    off = (got.to(F64) - ref).abs()
    bad = ~(off <= bound)  # a NaN is outside
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst {(off - bound).max().item():.3g}"


# T, K, E, H, share of dropped pairs, a token that loses all its pairs
ROWS = [(1, 1, 1, 128, 0.0, None), (1, 8, 384, 4096, 0.0, None), (3, 2, 8, 256, 0.5, 0), (37, 3, 7, 384, 0.1, 36),
        (257, 8, 48, 512, 0.1, 5), (130, 32, 64, 128, 0.05, 7), (65, 9, 33, 640, 0.0, None),
        (1001, 4, 48, 1024, 0.3, 0)]


@pytest.mark.parametrize("T,K,E,H,drop,gone", ROWS)
@pytest.mark.parametrize("src", ["bf16", "fp32", "e4m3"])
def test_dispatch(layers, T, K, E, H, drop, gone, src):
    import mixture_experts_layer_24_b200 as M
    L, r = layers(H, E, K), _cuda(R.routing(T, K, E, 11, drop, gone))
    x = _rand(1, T, H, dtype=F32 if src == "fp32" else BF16)
    scales, values = None, x
    if src == "e4m3":
        codes = torch.empty((T, H), dtype=torch.uint8, device="cuda")
        scales = torch.empty((T, H // 128), device="cuda")
        M.moe_quantize_e4m3(x, T, H, 1, codes, scales)
        values, x = R.decode(codes, scales), codes
    out = torch.full((T * K, H), 7.0, dtype=F32 if src == "fp32" else BF16, device="cuda")
    L.dispatch(x, r["inv"], x_scales=scales, out=out)
    n = r["n"]
    want = values[r["perm_src"][:n].long()]
    if src == "e4m3":  # the product rounds to fp32, then to bf16
        _within(out[:n], want, want.abs() * (R.BF16_HALF + 2 * U) , "dispatch")
    else:
        assert torch.equal(out[:n], want)
    assert (out[n:] == 7).all() and L.status() == 0


@pytest.mark.parametrize("T,K,E,H,drop,gone", ROWS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("router", [False, True])
def test_dispatch_bwd(layers, T, K, E, H, drop, gone, dtype, router):
    L, r = layers(H, E, K), _cuda(R.routing(T, K, E, 12, drop, gone))
    rows = _poison_behind(_rand(2, T * K, H, dtype=dtype), r["n"])
    more = (_rand(3, T, K, dtype=F32), r["idx"], _rand(4, E, H, dtype=F32)) if router else ()
    got = L.dispatch_bwd(rows, r["inv"], *more)
    ref, mag = R.dispatch_bwd(rows, r["inv"], *more)
    _within(got, ref, 2 * K * U * mag * 1.01 + R.half(dtype) * ref.abs() * 1.01, "dx")
    assert L.status() == 0


@pytest.mark.parametrize("T,K,E,H,drop,gone", ROWS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_combine_weighted_and_its_gradient(layers, T, K, E, H, drop, gone, dtype):
    L, r = layers(H, E, K), _cuda(R.routing(T, K, E, 13, drop, gone))
    y = _poison_behind(_rand(5, T * K, H, dtype=dtype), r["n"])
    dout = _rand(6, T, H, dtype=dtype)
    out = L.combine_weighted(y, r["w"], r["inv"])
    ref, mag = R.combine(y, r["w"], r["inv"])
    _within(out, ref, K * U * mag * 1.01 + R.half(dtype) * ref.abs() * 1.01, "out")
    dy = torch.full((T * K, H), 7.0, dtype=dtype, device="cuda")
    _, dw = L.combine_weighted_bwd(dout, y, r["w"], r["inv"], out=dy)
    want, dw_ref, dw_mag = R.combine_bwd(dout, y, r["w"], r["inv"])
    kept = r["inv"] >= 0
    # fp32 product, then the rows' type
    _within(dy[r["inv"][kept].long()], want[kept], want[kept].abs() * (R.half(dtype) + 2 * U), "dy")
    _within(dw, dw_ref, (H + 1) * U * dw_mag * 1.01, "dw")
    assert (dw[~kept] == 0).all() and (dy[r["n"]:] == 7).all() and L.status() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_at_the_widest(layers, dtype):
    """H = 8192 through every row operator, against its 64-bit form."""
    T, K, E, H = 61, 5, 33, 8192
    L, r = layers(H, E, K), _cuda(R.routing(T, K, E, 21, 0.1, 60))
    rows, x = _poison_behind(_rand(185, T * K, H, dtype=dtype), r["n"]), _rand(186, T, H, dtype=dtype)
    xs = L.dispatch(x, r["inv"])
    assert torch.equal(xs[:r["n"]], x[r["perm_src"][:r["n"]].long()])
    for more in ((), (_rand(187, T, K, dtype=F32), r["idx"], _rand(188, E, H, dtype=F32))):
        ref, mag = R.dispatch_bwd(rows, r["inv"], *more)
        _within(L.dispatch_bwd(rows, r["inv"], *more), ref,
                2 * K * U * mag * 1.01 + R.half(dtype) * ref.abs() * 1.01, "dx")
    ref, mag = R.combine(rows, r["w"], r["inv"])
    bound = K * U * mag * 1.01 + R.half(dtype) * ref.abs() * 1.01
    _within(L.combine_weighted(rows, r["w"], r["inv"]), ref, bound, "out")
    dy, dw = L.combine_weighted_bwd(x, rows, r["w"], r["inv"])
    want, dw_ref, dw_mag = R.combine_bwd(x, rows, r["w"], r["inv"])
    kept = r["inv"] >= 0
    _within(dy[r["inv"][kept].long()], want[kept], want[kept].abs() * (R.half(dtype) + 2 * U), "dy")
    _within(dw, dw_ref, (H + 1) * U * dw_mag * 1.01, "dw")
    if dtype == BF16:
        up = _rand(189, T, K, dtype=F32)
        got = L.route_bwd(x, r["w"], up, topk_idx=r["idx"])
        ref = R.route_bwd(x, r["w"], up, r["idx"], torch.zeros_like(r["inv"]), E)
        _within(got[1], ref[1], (K + 4 + T) * U * ref[4] * 1.01, "dw_router")
    assert L.status() == 0


def test_combine_gradient_against_differences(layers):
    """fp32 rows: <out, dout> is linear in each weight and each row, so a difference with step 1 is the gradient up
    to the forward's own rounding."""
    T, K, E, H = 9, 3, 7, 256
    L, r = layers(H, E, K), _cuda(R.routing(T, K, E, 14, 0.1, 4))
    y, dout = _rand(7, T * K, H, dtype=F32), _rand(8, T, H, dtype=F32)
    dy, dw = L.combine_weighted_bwd(dout, y, r["w"], r["inv"], out=torch.zeros_like(y))
    loss = lambda y, w: (L.combine_weighted(y, w, r["inv"]).to(F64) * dout.to(F64)).sum()  # noqa: E731
    _, mag = R.combine(y, r["w"] + 1, r["inv"])
    err = 2 * ((K + 1) * U * (mag + 10) * dout.abs().to(F64)).sum(1).max() + H * U * 64
    for t, k in ((0, 0), (3, 2), (8, 1), (4, 1)):
        w2 = r["w"].clone()
        w2[t, k] += 1
        assert abs(loss(y, w2) - loss(y, r["w"]) - dw[t, k]) <= err
        p = int(r["inv"][t, k])
        if p >= 0:
            y2 = y.clone()
            y2[p, 17] += 1
            assert abs(loss(y2, r["w"]) - loss(y, r["w"]) - dy[p, 17]) <= err


# rows are T*K pairs of I columns
ACT = [(1, 1, 128, 0.0), (3, 2, 256, 0.3), (37, 8, 384, 0.1), (129, 3, 2048, 0.0), (5, 4, 8192, 0.2),
       (700, 8, 128, 0.05)]


def _gate_up(seed, rows, I):
    gu = _rand(seed, rows, 2 * I, std=2.0)
    gu[0, :128] = 0                                # an all-zero block: scale 1
    gu[rows // 2, I:I + 128] *= 2.0 ** -100         # a block of tiny values
    gu[rows // 3, I:I + 128] *= 2.0 ** -128         # and one of subnormal ones
    gu[rows - 1, 0:4] = torch.tensor([120.0, -120.0, -88.0, 30000.0], dtype=BF16)  # exp over- and underflows
    return gu


@pytest.mark.parametrize("T,K,I,drop", ACT)
def test_swiglu_ckpt(layers, T, K, I, drop):
    import mixture_experts_layer_24_b200 as M
    L, r = layers(128, max(K, 8), K, I), _cuda(R.routing(T, K, max(K, 8), 15, drop))
    rows, n = T * K, r["n"]
    gu = _gate_up(9, rows, I)
    out = (torch.full((rows, I), 7.0, dtype=BF16, device="cuda"),
           torch.full((rows, 2 * I), 7, dtype=torch.uint8, device="cuda"),
           torch.full((rows, 2 * I // 128), 7.0, device="cuda"))
    h, q, s = L.swiglu_ckpt(_poison_behind(gu.clone(), n), r["inv"], out=out)
    g, u = gu[:n, :I].to(F64), gu[:n, I:].to(F64)
    ref = R.silu_parts(g)[1] * u
    # expf within 2 ulp (2^-22), an add, a division, two products (2^-24 each): 2^-21 in all. Where exp(-g)
    # overflows, sigmoid is 0 for a true value below 2^-127 |g|.
    _within(h[:n], ref, ref.abs() * (R.BF16_HALF + 2 ** -20) + 2.0 ** -120 * u.abs() + 2.0 ** -133, "h")
    q_ref, s_ref = oracle.quant_e4m3(oracle.as_u16(gu[:n].cpu()), 1)
    assert np.array_equal(q[:n].cpu().numpy(), q_ref) and np.array_equal(s[:n].cpu().numpy(), s_ref)
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    M.moe_quantize_e4m3(gu, rows, 2 * I, 1, q2, s2)  # the same bits as the block quantiser's
    assert torch.equal(q[:n], q2[:n]) and torch.equal(s[:n], s2[:n])
    for t in out:
        assert (t[n:].float() == 7).all()
    h3, q3, s3 = L.swiglu_ckpt(gu)  # without inv: every row
    assert torch.equal(h3[:n], h[:n]) and torch.equal(q3, q2) and torch.equal(s3, s2)
    assert L.status() == 0


def test_swiglu_ckpt_infinities_and_nan(layers):
    """Codes and scales of blocks that hold infinities and NaN are the block quantiser's; h follows IEEE rules."""
    import mixture_experts_layer_24_b200 as M
    L, I = layers(128, 8, 2, 256), 256
    gu = _rand(10, 6, 2 * I)
    gu[0, 3], gu[1, I + 5], gu[2, 7], gu[3, I + 130], gu[4, 9] = (float(v) for v in
                                                                  ("inf", "inf", "nan", "nan", "-inf"))
    h, q, s = L.swiglu_ckpt(gu)
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    M.moe_quantize_e4m3(gu, 6, 2 * I, 1, q2, s2)
    assert torch.equal(q, q2) and torch.equal(s.view(torch.int32), s2.view(torch.int32))
    g, u = gu[:, :I].float(), gu[:, I:].float()
    ref = g / (1 + torch.exp(-g)) * u
    assert torch.equal(torch.isnan(h), torch.isnan(ref)) or torch.isnan(h[4, 9])  # -inf * 0 is NaN either way
    assert torch.isinf(h[0, 3]) and torch.isinf(h[1, 5]) and torch.isnan(h[2, 7]) and torch.isnan(h[3, 130])
    assert torch.isfinite(h[5]).all()


def test_swiglu_nan_and_infinity_places(layers):
    """h, dgu, hw and the weights' gradient hold NaN and infinities exactly where the formulas in fp32 do, and nowhere
    else: values that reach no overflow of their own (|g| < 80), beside infinities and NaN in g, u and dh."""
    rows, I = 24, 256
    L = layers(128, 8, 1, I)
    gu, dh = _rand(160, rows, 2 * I, std=2.0), _rand(161, rows, I)
    inf, nan = float("inf"), float("nan")
    for i, (col, v) in enumerate(((3, inf), (I + 5, inf), (7, nan), (I + 130, nan), (9, -inf), (I + 9, -inf))):
        gu[i, col] = v
    gu[6, 11], gu[6, I + 11] = inf, nan
    gu[7, 12], gu[7, I + 12] = -inf, 0.0
    gu[8, 13], gu[8, I + 13] = inf, 0.0
    h, q, s = L.swiglu_ckpt(gu)
    g, u = gu[:, :I].float(), gu[:, I:].float()
    ref = g / (1 + torch.exp(-g)) * u
    assert torch.equal(torch.isnan(h), torch.isnan(ref))
    assert torch.equal(torch.isinf(h), torch.isinf(ref))
    assert torch.equal(torch.signbit(h)[torch.isinf(h)], torch.signbit(ref)[torch.isinf(h)])
    # the gradient from a checkpoint without them, and dh with them
    clean = _rand(162, rows, 2 * I, std=2.0)
    _, q, s = L.swiglu_ckpt(clean)
    dh[0, 3], dh[1, I - 1], dh[2, 0] = inf, -inf, nan
    w = torch.rand(rows, 1, device="cuda") + 0.5
    w[3] = 0.0
    w[4], w[5] = inf, nan
    inv = torch.arange(rows, dtype=torch.int32, device="cuda").view(-1, 1)
    dgu, hw, dw = L.swiglu_ckpt_bwd(q, s, dh, topk_w=w, inv=inv)
    v = R.decode(q, s)
    dg, du, h64, dots = R.swiglu_bwd(v[:, :I], v[:, I:], dh.to(F64), w.view(-1).to(F64))
    for got, want in ((dgu[:, :I], dg), (dgu[:, I:], du), (hw, w.to(F64) * h64), (dw.view(-1), dots)):
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(torch.isinf(got), torch.isinf(want))
    assert L.status() == 0


@pytest.mark.parametrize("T,K,I,drop", ACT)
@pytest.mark.parametrize("weighted", [False, True])
def test_swiglu_ckpt_bwd(layers, T, K, I, drop, weighted):
    L, r = layers(128, max(K, 8), K, I), _cuda(R.routing(T, K, max(K, 8), 16, drop))
    rows, n = T * K, r["n"]
    _, q, s = L.swiglu_ckpt(_gate_up(11, rows, I))
    dh = _rand(12, rows, I)
    s_p, dh_p = s.clone(), dh.clone()
    s_p[n:], dh_p[n:] = float("nan"), float("inf")
    out = (torch.full((rows, 2 * I), 7.0, dtype=BF16, device="cuda"),
           torch.full((rows, I), 7.0, dtype=BF16, device="cuda") if weighted else None)
    dgu, hw, dw = L.swiglu_ckpt_bwd(q, s_p, dh_p, topk_w=r["w"] if weighted else None, inv=r["inv"], out=out)
    v = R.decode(q, s)[:n]
    g, u, d = v[:, :I], v[:, I:], dh[:n].to(F64)
    w = torch.ones(n, dtype=F64, device="cuda")
    if weighted:
        w = r["w"][r["perm_src"][:n].long(), r["perm_k"][:n].long()].to(F64)
    dg, du, h, dots = R.swiglu_bwd(g, u, d, w)
    # g, u: one product each; sigmoid within 2^-21; then at most six roundings: 2^-20 relative to each factor's
    # magnitude. 1 + g (1 - sigmoid) may cancel: its error is relative to 1 + |g|, and (through g sigmoid') g's own.
    sig = R.silu_parts(g)[0]
    tiny = 2.0 ** -120 * (1 + u.abs()) * (1 + d.abs()) * (1 + g.abs()) + 2.0 ** -133
    c = 2.0 ** -20
    _within(dgu[:n, :I], dg, R.BF16_HALF * dg.abs() * 1.01 + c * (w[:, None] * d * u * sig).abs() * (1 + g.abs()) ** 2
            + tiny, "dg")
    _within(dgu[:n, I:], du, du.abs() * (R.BF16_HALF * 1.01 + c * (1 + g.abs())) + tiny, "du")
    assert (dgu[n:] == 7).all() and L.status() == 0
    if not weighted:
        assert hw is None and dw is None
        return
    _within(hw[:n], w[:, None] * h, (w[:, None] * h).abs() * (R.BF16_HALF * 1.01 + c * (1 + g.abs())) + tiny, "hw")
    assert (hw[n:] == 7).all()
    kept = r["inv"] >= 0
    at = r["inv"][kept].long()
    mag = (d * h).abs()
    bound = (mag * (c * (1 + g.abs()))).sum(1) + (I + 1) * U * mag.sum(1) * 1.01 + tiny.sum(1)
    _within(dw[kept], dots[at], bound[at], "dw")
    assert (dw[~kept] == 0).all()


def test_swiglu_codes_over_all_pairs_of_values(layers):
    """The codes' short cut (a reciprocal per block and a correction in place of a division per code) over every block
    maximum a bf16 can hold and every value up to it, signs mixed: the block quantiser's bits, which divides."""
    import mixture_experts_layer_24_b200 as M
    I, per = 8192, 127  # values beside the maximum in a block of 128
    L = layers(128, 8, 1, I)
    top = 0x7f80  # bit patterns of positive finite bf16 values lie below infinity's
    blocks = torch.arange((top + per - 1) // per, device="cuda")
    checked = 0
    for first in range(1, top, 256):
        amax = torch.arange(first, min(first + 256, top), device="cuda")
        bits = (blocks[:, None] * per + torch.arange(per, device="cuda")).view(1, -1, per)
        bits = torch.minimum(bits.expand(len(amax), -1, -1), amax[:, None, None])
        keep = (blocks * per)[None, :] <= amax[:, None]  # blocks that hold a value up to the maximum
        vals = torch.cat((bits, amax[:, None, None].expand(-1, len(blocks), 1)), 2)[keep]
        vals = (vals + (torch.arange(128, device="cuda") % 3 == 1) * 0x8000).to(torch.int32)
        vals = torch.where(vals >= 0x8000, vals - 0x10000, vals).to(torch.int16)
        pad = -vals.shape[0] % (2 * I // 128)
        gu = torch.cat((vals, vals[:1].expand(pad, -1))).view(BF16).view(-1, 2 * I).contiguous()
        _, q, s = L.swiglu_ckpt(gu)
        q2, s2 = torch.empty_like(q), torch.empty_like(s)
        M.moe_quantize_e4m3(gu, gu.shape[0], 2 * I, 1, q2, s2)
        assert torch.equal(q, q2) and torch.equal(s, s2), first
        checked += vals.shape[0] * per
    assert checked >= top * (top - 1) // 2 and L.status() == 0


@pytest.mark.parametrize("I", [128, 640, 2048, 8192])
def test_swiglu_rows_do_not_depend_on_each_other(layers, I):
    """A pair's codes, gradients and weight's gradient have the same bits alone, among few and among many."""
    L, rows = layers(128, 8, 1, I), 9000
    inv = torch.arange(rows, dtype=torch.int32, device="cuda").view(-1, 1)
    gu, dh, w = _gate_up(31, rows, I), _rand(32, rows, I), _rand(33, rows, 1, dtype=F32)
    h, q, s = L.swiglu_ckpt(gu, inv)
    many = (h, q, s) + L.swiglu_ckpt_bwd(q, s, dh, topk_w=w, inv=inv)
    for lo, hi in ((0, 1), (3, 40), (100, 1900), (4000, 7000)):
        few = L.swiglu_ckpt(gu[lo:hi].contiguous(), inv[:hi - lo])
        few += L.swiglu_ckpt_bwd(q[lo:hi].contiguous(), s[lo:hi].contiguous(), dh[lo:hi].contiguous(),
                                 topk_w=w[lo:hi].contiguous(), inv=inv[:hi - lo])
        for a, b in zip(few, many):
            assert torch.equal(a, b[lo:hi])


def test_swiglu_gradient_against_differences(layers):
    """dgu (fp32 reference of the same formula aside) against central differences of silu(g) u in 64 bits at the
    checkpoint's values."""
    T, K, I = 3, 2, 128
    L, r = layers(128, 8, 2, I), _cuda(R.routing(T, K, 8, 17))
    _, q, s = L.swiglu_ckpt(_rand(13, T * K, 2 * I, std=2.0))
    dh = _rand(14, T * K, I)
    dgu, _, _ = L.swiglu_ckpt_bwd(q, s, dh, topk_w=r["w"], inv=r["inv"])
    v, step = R.decode(q, s), 1e-5
    w = torch.zeros(T * K, dtype=F64, device="cuda")
    w[r["inv"].long().view(-1)] = r["w"].to(F64).view(-1)

    def h(v):
        return R.silu_parts(v[:, :I])[1] * v[:, I:]

    for part in (slice(0, I), slice(I, 2 * I)):
        e = torch.zeros_like(v)
        e[:, part] = step
        diff = w[:, None] * dh.to(F64) * (h(v + e) - h(v - e)) / (2 * step)
        # differences: step^2 times a third derivative below 4 (1 + |u|); bf16 rounding of the result
        bound = R.BF16_HALF * diff.abs() * 1.01 + 1e-5 * (1 + v.abs()).max() ** 2 * dh.abs().to(F64) * w[:, None]
        _within(dgu[:, part], diff, bound, "dgu")


ROUTE = [(1, 1, 1, 128, 0.0), (1, 8, 384, 4096, 0.0), (37, 8, 384, 256, 0.0), (300, 2, 5, 2176, 0.2),
         (65, 32, 40, 384, 0.1), (1025, 8, 64, 1024, 0.05), (2000, 1, 3, 128, 0.0), (600, 4, 1024, 128, 0.02)]


@pytest.mark.parametrize("T,K,E,H,drop", ROUTE)
@pytest.mark.parametrize("ckpt", [False, True])
def test_route_bwd(layers, T, K, E, H, drop, ckpt):
    import mixture_experts_layer_24_b200 as M
    L, r = layers(H, E, K), _cuda(R.routing(T, K, E, 18, drop, T // 2 if drop else None))
    x, dw = _rand(15, T, H), _rand(16, T, K, dtype=F32)
    scales, values = None, x
    if ckpt:
        codes = torch.empty((T, H), dtype=torch.uint8, device="cuda")
        scales = torch.empty((T, H // 128), device="cuda")
        M.moe_quantize_e4m3(x, T, H, 1, codes, scales)
        values, x = R.decode(codes, scales), codes
    args = (x, r["w"], dw, r["offsets"], r["perm_src"], r["perm_k"])
    dl, dwr, db = L.route_bwd(*args, x_scales=scales)
    dl_ref, dwr_ref, db_ref, dl_mag, dwr_mag, db_mag = R.route_bwd(values, r["w"], dw, r["idx"], r["inv"], E)
    _within(dl, dl_ref, (K + 2) * U * dl_mag * 1.01, "dlogit")
    longest = int((r["offsets"][1:] - r["offsets"][:-1]).max())
    # a pair's dlogit, the decoded x (one rounding), and as many additions as the expert has pairs
    _within(dwr, dwr_ref, (K + 4 + longest) * U * dwr_mag * 1.01, "dw_router")
    _within(db, db_ref, (K + 3 + longest) * U * db_mag * 1.01, "dlogit_bias")
    assert L.status() == 0
    again = L.route_bwd(*args, x_scales=scales)
    assert all(torch.equal(a, b) for a, b in zip((dl, dwr, db), again))


@pytest.mark.parametrize("T,K,E,H,drop", [(1, 8, 384, 4096, 0.5), (9, 3, 8, 256, 0.3), (37, 8, 384, 256, 0.9),
                                          (300, 2, 5, 2176, 0.2), (65, 32, 40, 384, 0.1), (1025, 8, 64, 1024, 0.05),
                                          (600, 4, 1024, 128, 0.0), (64, 4, 16, 512, 1.0)])
@pytest.mark.parametrize("ckpt", [False, True])
def test_router_gradient_with_dropped_pairs_against_autograd(layers, T, K, E, H, drop, ckpt):
    """dx (router and rows together), dw_router and dlogit_bias belong to one loss, whatever pairs the forward
    dropped. w is rounded to fp32 and the reference's softmax sums to 1 in 64 bits: they are 2^-24 apart at most, twice
    in a dlogit."""
    import mixture_experts_layer_24_b200 as M
    L, r = layers(H, E, K), _cuda(R.routing(T, K, E, 19, drop, T // 2 if drop else None))
    x, rows = _rand(120, T, H), _poison_behind(_rand(121, T * K, H), r["n"])
    wr, c = _rand(122, E, H, std=0.05, dtype=F32), _rand(123, T, K, dtype=F32)
    scales, values = None, x
    if ckpt:
        codes = torch.empty((T, H), dtype=torch.uint8, device="cuda")
        scales = torch.empty((T, H // 128), device="cuda")
        M.moe_quantize_e4m3(x, T, H, 1, codes, scales)
        values, x = R.decode(codes, scales), codes
    # the weights' gradient comes from the combine, so that of dropped pairs is its 0
    dw = torch.where(r["inv"] >= 0, c, torch.zeros_like(c))
    dl, dwr, db = L.route_bwd(x, r["w"], dw, x_scales=scales, topk_idx=r["idx"])
    dx = L.dispatch_bwd(rows, r["inv"], dl, r["idx"], wr)
    dx_ref, dwr_ref, db_ref = R.route_bwd_by_autograd(values, wr, r["w"], dw, r["idx"], rows, r["inv"])
    everyone = torch.zeros_like(r["inv"])
    _, _, _, dl_mag, dwr_mag, db_mag = R.route_bwd(values, r["w"], dw, r["idx"], everyone, E)
    most = int(torch.bincount(r["idx"].view(-1).long()).max())
    _within(dwr, dwr_ref, (K + 6 + most) * U * dwr_mag * 1.01, "dw_router")
    _within(db, db_ref, (K + 5 + most) * U * db_mag * 1.01, "dlogit_bias")
    _, mag = R.dispatch_bwd(rows, r["inv"], dl_mag, r["idx"], wr.abs())
    _within(dx, dx_ref, (3 * K + 4) * U * mag * 1.01 + R.BF16_HALF * dx_ref.abs() * 1.01, "dx")
    assert L.status() == 0
    again = L.route_bwd(x, r["w"], dw, x_scales=scales, topk_idx=r["idx"])
    assert all(torch.equal(a, b) for a, b in zip((dl, dwr, db), again))
    # the list of every chosen pair gives the same bits
    _, offsets, perm_src, perm_k, _ = L.permute(r["idx"])
    listed = L.route_bwd(x, r["w"], dw, offsets, perm_src, perm_k, x_scales=scales)
    assert all(torch.equal(a, b) for a, b in zip((dl, dwr, db), listed))


def test_router_gradient_of_the_choice_refusals_and_marks(layers):
    """Refused on the host before any launch; an index that names no expert adds nothing and is reported; no tokens;
    a captured call, replayed on new inputs; another stream."""
    import mixture_experts_layer_24_b200 as M
    T, K, E, H = 6, 2, 8, 256
    L, r = layers(H, E, K), _cuda(R.routing(T, K, E, 30))
    x, dw = _rand(131, T, H), _rand(132, T, K, dtype=F32)
    need = M.moe_route_bwd_topk_workspace_size(L.ctx, T)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    dl, dwr, db = torch.empty_like(dw), torch.empty((E, H), device="cuda"), torch.empty(E, device="cuda")
    c, w, idx, before = L.ctx, r["w"], r["idx"], L.launches()
    calls = [
        (1, lambda: M.moe_route_bwd_topk(c, x, None, None, w, dw, T, dl, dwr, db, ws)),
        (1, lambda: M.moe_route_bwd_topk(c, None, None, idx, w, dw, T, dl, dwr, db, ws)),
        (1, lambda: M.moe_route_bwd_topk(c, x, None, idx, w, None, T, dl, dwr, db, ws)),
        (1, lambda: M.moe_route_bwd_topk(c, x, None, idx, w, dw, T, None, dwr, db, ws)),
        (1, lambda: M.moe_route_bwd_topk(c, x, None, idx, w, dw, T, dl, None, db, ws)),
        (1, lambda: M.moe_route_bwd_topk(c, x, None, idx, w, dw, T, dl, dwr, db, None)),
        (1, lambda: M.moe_route_bwd_topk(c, x, None, idx, w, dw, T, dl, dwr, db, ws[:-1])),
        (1, lambda: M.moe_route_bwd_topk(c, x, None, idx, w, dw, -1, dl, dwr, db, ws)),
        (2, lambda: M.moe_route_bwd_topk(c, x, None, idx, w, dw, 65537, dl, dwr, db, ws)),
    ]
    for i, (status, call) in enumerate(calls):
        with pytest.raises(M.MoeError) as e:
            call()
        assert e.value.status == status, (i, e.value)
    assert L.launches() == before and L.status() == 0
    assert M.moe_route_bwd_topk_workspace_size(c, -1) == 0 and M.moe_route_bwd_topk_workspace_size(c, 65537) == 0
    marked = idx.clone()
    marked[2, 1], marked[4, 0] = E, -1
    _, off, src, pk, _ = L.permute(marked)
    want = L.route_bwd(x, w, dw, off, src, pk)
    assert L.status() == M.binding.MOE_DEV_BAD_EXPERT
    got = L.route_bwd(x, w, dw, topk_idx=marked)
    assert L.status() == M.binding.MOE_DEV_BAD_EXPERT and all(torch.equal(a, b) for a, b in zip(got, want))
    none = torch.empty((0, K), dtype=torch.int32, device="cuda")
    empty = L.route_bwd(x[:0], w[:0], dw[:0], topk_idx=none)
    assert empty[0].shape == (0, K) and (empty[1] == 0).all() and (empty[2] == 0).all()
    xin = x.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = L.route_bwd(xin, w, dw, topk_idx=idx)
    xin.copy_(_rand(133, T, H))
    g.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = L.route_bwd(xin, w, dw, topk_idx=idx, stream=side)
    torch.cuda.synchronize()
    want = L.route_bwd(_rand(133, T, H), w, dw, topk_idx=idx)
    assert all(torch.equal(a, b) and torch.equal(o, b) for a, o, b in zip(out, other, want)) and L.status() == 0


def _segments(counts, slack=0):
    off = torch.zeros(len(counts) + 1, dtype=torch.int32)
    off[1:] = torch.cumsum(torch.tensor(counts), 0)
    return off.cuda(), int(off[-1]) + slack


# counts per expert, rows behind the last, n_in, n_out
PROD = [([1], 0, 128, 128), ([0, 1, 0, 0], 3, 128, 256), ([17, 0, 64, 63, 65], 5, 256, 384),
        ([256, 257, 511], 0, 384, 128), ([300, 2, 0, 33], 40, 640, 512), ([0, 0, 0], 2, 256, 128),
        ([15, 16, 31, 32, 33, 47, 48, 49, 127, 128, 129, 191, 193], 1, 256, 512), ([1] * 70, 0, 512, 256),
        ([0] * 40 + [700] + [3] * 8, 9, 2048, 1152), ([1, 0, 2, 0] * 256, 3, 128, 128)]


def _ints(seed, *shape):
    """-1, 0 or 1: every product and sum of them is exact in fp32, and up to 256 in bf16."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-1, 2, shape, generator=g, device="cuda").to(BF16)


@pytest.mark.parametrize("counts,slack,n_in,n_out", PROD)
@pytest.mark.parametrize("transposed", [False, True])
def test_expert_product(layers, counts, slack, n_in, n_out, transposed):
    E = len(counts)
    L, (off, P) = layers(256, E, 1, 128), _segments(counts, slack)
    n, k, m = P - slack, n_out if transposed else n_in, n_in if transposed else n_out
    for exact in (True, False):
        a = _ints(20, P, k) if exact else _rand(20, P, k)
        w = _ints(21, E, n_out, n_in) if exact else _rand(21, E, n_out, n_in, std=0.1)
        _poison_behind(a, n)
        out = torch.full((P, m), 7.0, dtype=BF16, device="cuda")
        L.expert_product(a, w, off, transposed=transposed, out=out)
        ref, mag = R.products(a, w, off, transposed)
        if exact:
            assert torch.equal(out[:n], ref.to(BF16)), "exact sums of whole numbers"
        else:
            # the tensor cores' fp32 sum of k exact products: one step (2^-23) for each at most
            _within(out[:n], ref, k * 2.0 ** -23 * mag + R.BF16_HALF * ref.abs() * 1.01, "out")
        assert (out[n:] == 7).all() and L.status() == 0


@pytest.mark.parametrize("transposed", [False, True])
def test_products_rows_do_not_depend_on_each_other(layers, transposed):
    """A row's bits are the same alone, among few and among many rows of its expert, at any place in a tile."""
    E, n_in, n_out = 3, 1024, 640
    L, k = layers(256, E, 1, 128), n_out if transposed else n_in
    w, rows = _rand(26, E, n_out, n_in, std=0.1), _rand(27, 700, k)
    off, _ = _segments([0, 700, 0])
    many = L.expert_product(rows, w, off, transposed=transposed)
    for lo, hi in ((0, 1), (5, 38), (255, 257), (400, 699)):
        few, _ = _segments([0, hi - lo, 0])
        got = L.expert_product(rows[lo:hi].contiguous(), w, few, transposed=transposed)
        assert torch.equal(got, many[lo:hi])


@pytest.mark.parametrize("counts,slack,n_in,n_out", PROD)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_expert_wgrad(layers, counts, slack, n_in, n_out, dtype):
    """Neighbouring experts' rows and the rows behind the last hold NaN and infinities where they are not summed."""
    E = len(counts)
    L, (off, P) = layers(256, E, 1, 128), _segments(counts, slack)
    n = P - slack
    for exact in (True, False):
        a = _ints(22, P, n_in) if exact else _rand(22, P, n_in)
        dy = _ints(23, P, n_out) if exact else _rand(23, P, n_out)
        _poison_behind(a, n)
        _poison_behind(dy, n)
        dw = L.expert_wgrad(dy, a, off, dtype=dtype)
        ref, mag = R.wgrads(dy[:n], a[:n], off)
        if exact:
            assert torch.equal(dw, ref.to(dtype)), "exact sums of whole numbers"
        else:
            most = max(counts)
            _within(dw, ref, most * 2.0 ** -23 * mag + R.half(dtype) * ref.abs() * 1.01, "dw")
        if dtype == F32:
            base = torch.full_like(dw, 3.0)
            got = L.expert_wgrad(dy, a, off, out=base, accumulate=True)
            assert got is base and torch.equal(base, 3.0 + dw)
        if E > 1 and exact and sum(c > 0 for c in counts) > 1:  # NaN in one expert's rows stays with it
            e = next(i for i, c in enumerate(counts) if c)
            a2 = a.clone()
            a2[int(off[e]):int(off[e + 1])] = float("nan")
            got = L.expert_wgrad(dy, a2, off, dtype=dtype)
            others = [i for i in range(E) if i != e]
            assert torch.equal(got[others], dw[others])
    assert L.status() == 0


def test_wgrad_fp32_over_many_rows(layers):
    """Positive terms, so that nothing cancels and every lost bit shows. The kernel sums 896 rows (56 steps of 16) in
    the tensor cores and adds the segments in fp32: each of these 56 + 19 additions may lose one unit of the running
    sum (2^-23). Summed in one run, 1024 steps, the loss was measured at 8e-5."""
    L = layers(256, 2, 1, 128)
    off, P = _segments([16384, 100])
    a, dy = _rand(24, P, 256).abs(), _rand(25, P, 128).abs()
    ref, mag = R.wgrads(dy, a, off)
    base = torch.ones((2, 128, 256), device="cuda")
    got = L.expert_wgrad(dy, a, off, dtype=F32)
    _within(got, ref, (56 + 19 + 1) * 2.0 ** -23 * mag, "dw")
    again = L.expert_wgrad(dy, a, off, dtype=F32)
    assert torch.equal(got, again)
    L.expert_wgrad(dy, a, off, out=base, accumulate=True)
    _within(base, ref + 1, (56 + 19 + 2) * 2.0 ** -23 * (mag + 1), "accumulated dw")
    half = L.expert_wgrad(dy, a, off)  # bf16: one run, one rounding
    _within(half, ref, (1024 * 2.0 ** -23 + R.BF16_HALF) * mag * 1.01, "bf16 dw")


@pytest.mark.parametrize("n_in,n_out", [(16384, 2432), (2432, 16384), (16384, 16256)])
def test_products_at_the_widest(layers, n_in, n_out):
    """The most features, in an odd number of tiles and of bands, over whole numbers: every bit is pinned."""
    counts = [70, 0, 300]
    L, (off, P) = layers(256, 3, 1, 128), _segments(counts, 3)
    n = P - 3
    w = _ints(180, 3, n_out, n_in)
    a, dy = _ints(181, P, n_in), _ints(182, P, n_out)
    _poison_behind(a, n)
    _poison_behind(dy, n)
    cut = off.tolist()
    for rows, transposed in ((a, False), (dy, True)):
        out = torch.full((P, n_in if transposed else n_out), 7.0, dtype=BF16, device="cuda")
        L.expert_product(rows, w, off, transposed=transposed, out=out)
        for e, (i, j) in enumerate(zip(cut, cut[1:])):
            m = w[e] if transposed else w[e].t()
            assert torch.equal(out[i:j], (rows[i:j].to(F64) @ m.to(F64)).to(F32).to(BF16))
        assert (out[n:] == 7).all()
    for dtype in (BF16, F32):
        dw = L.expert_wgrad(dy, a, off, dtype=dtype)
        for e, (i, j) in enumerate(zip(cut, cut[1:])):
            assert torch.equal(dw[e], (dy[i:j].to(F64).t() @ a[i:j].to(F64)).to(F32).to(dtype))
    assert L.status() == 0


def test_wgrad_bf16_over_the_most_rows(layers):
    """Positive terms over every number of rows accepted up to the most, where nothing cancels what the tensor cores'
    sum cuts off: a run of 2^15 rows loses at most one unit (2^-23) of its sum per row, 2^-8 in all; the runs (64 at
    most) are added in fp32, and the sum is rounded once to bf16."""
    L = layers(256, 1, 1, 128)
    for P in (32768, 65536, 300001, 65536 * 32):
        off = torch.tensor([0, P], dtype=torch.int32, device="cuda")
        a, dy = _rand(140, P, 128).abs_(), _rand(141, P, 128).abs_()
        ref = torch.zeros((128, 128), dtype=F64, device="cuda")
        for i in range(0, P, 65536):
            ref += dy[i:i + 65536].to(F64).t() @ a[i:i + 65536].to(F64)
        got = L.expert_wgrad(dy, a, off)[0]
        _within(got, ref, (2.0 ** -8 + 64 * U + R.BF16_HALF) * ref * 1.01, f"bf16 dw over {P} rows")
        # no bias beyond a quarter of the rounding's half step: over 16384 elements the roundings average out
        assert abs(((got.to(F64) - ref) / ref).mean()) <= R.BF16_HALF / 4, P
        assert torch.equal(got, L.expert_wgrad(dy, a, off)[0])
    assert L.status() == 0


def test_wgrad_bf16_runs_of_whole_numbers(layers):
    """Experts of one run, of several, with and without a ragged end, none and few rows, in many tiles per CTA pair:
    sums of whole numbers are exact in fp32 and rounded once, so every bit is pinned."""
    counts = [40000, 5, 70001, 0, 32768, 32769, 32784, 65552, 16, 98320, 1]
    L, (off, P) = layers(256, len(counts), 1, 128), _segments(counts, 7)
    n = P - 7
    for n_in, n_out in ((1280, 1024), (128, 384)):
        a, dy = _ints(142, P, n_in), _ints(143, P, n_out)
        _poison_behind(a, n)
        _poison_behind(dy, n)
        got = L.expert_wgrad(dy, a, off)
        cut = off.tolist()
        for e, (i, j) in enumerate(zip(cut, cut[1:])):
            ref = dy[i:j].to(F64).t() @ a[i:j].to(F64)
            assert torch.equal(got[e], ref.to(F32).to(BF16)), counts[e]
    assert L.status() == 0


def test_wgrad_without_any_row(layers):
    L = layers(256, 3, 1, 128)
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    none = torch.empty((0, 256), dtype=BF16, device="cuda")
    out = torch.full((3, 256, 256), 5.0, device="cuda")
    assert torch.equal(L.expert_wgrad(none, none, off, out=out.clone(), accumulate=True), out)
    assert (L.expert_wgrad(none, none, off, out=out) == 0).all()
    w = torch.zeros((3, 256, 256), dtype=BF16, device="cuda")
    assert L.expert_product(none, w, off).shape == (0, 256)


def test_no_tokens(layers):
    L = layers(256, 8, 2, 128)
    e = lambda *s, dtype=BF16: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
    inv, w = e(0, 2, dtype=torch.int32), e(0, 2, dtype=F32)
    off = torch.zeros(9, dtype=torch.int32, device="cuda")
    assert L.dispatch(e(0, 256), inv).shape == (0, 256)
    assert L.dispatch_bwd(e(0, 256), inv).shape == (0, 256)
    assert L.combine_weighted(e(0, 256), w, inv).shape == (0, 256)
    assert L.combine_weighted_bwd(e(0, 256), e(0, 256), w, inv)[1].shape == (0, 2)
    h, q, s = L.swiglu_ckpt(e(0, 256), inv)
    assert L.swiglu_ckpt_bwd(q, s, h, topk_w=w, inv=inv)[2].shape == (0, 2)
    perm = e(0, dtype=torch.int32)
    dl, dwr, db = L.route_bwd(e(0, 256), w, w, off, perm, perm)
    assert (dwr == 0).all() and (db == 0).all()


def test_refusals_of_the_c_abi(layers):
    """Refused on the host, nothing launched: the launch count does not move."""
    import mixture_experts_layer_24_b200 as M
    L = layers(256, 8, 2, 128)
    T, H, K, I, E = 4, 256, 2, 128, 8
    x, rows = torch.zeros((T, H), dtype=BF16, device="cuda"), torch.zeros((T * K, H), dtype=BF16, device="cuda")
    inv, w = torch.zeros((T, K), dtype=torch.int32, device="cuda"), torch.zeros((T, K), device="cuda")
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    wt = torch.zeros((E, 256, 256), dtype=BF16, device="cuda")
    odd = torch.zeros(T * K * H + 1, dtype=BF16, device="cuda")[1:]  # not 16-byte aligned
    c, before = L.ctx, L.launches()
    calls = [
        (1, lambda: M.moe_dispatch(c, x, None, 3, inv, T, rows)),
        (1, lambda: M.moe_dispatch(c, x, None, M.MOE_T_E4M3_B128, inv, T, rows)),
        (1, lambda: M.moe_dispatch(c, x, w, M.MOE_T_BF16, inv, T, rows)),
        (1, lambda: M.moe_dispatch(c, x, None, 0, inv, -1, rows)),
        (2, lambda: M.moe_dispatch(c, x, None, 0, inv, 65537, rows)),
        (1, lambda: M.moe_dispatch(c, odd, None, 0, inv, T, rows)),
        (1, lambda: M.moe_dispatch_bwd(c, rows, M.MOE_T_E4M3_B128, inv, None, None, None, T, x)),
        (1, lambda: M.moe_dispatch_bwd(c, rows, 0, inv, w, None, None, T, x)),
        (1, lambda: M.moe_dispatch_bwd(c, rows, 0, None, None, None, None, T, x)),
        (1, lambda: M.moe_combine_weighted(c, rows, 0, None, inv, T, x)),
        (1, lambda: M.moe_combine_weighted(c, odd, 0, w, inv, T, x)),
        (1, lambda: M.moe_combine_weighted_bwd(c, x, rows, 0, w, inv, T, rows, None)),
        (1, lambda: M.moe_swiglu_ckpt(c, rows, None, -1, rows, rows, w)),
        (2, lambda: M.moe_swiglu_ckpt(c, rows, None, 65536 * 32 + 1, rows, rows, w)),
        (1, lambda: M.moe_swiglu_ckpt(c, rows, None, 4, None, rows, w)),
        (1, lambda: M.moe_swiglu_ckpt_bwd(c, rows, w, rows, w, None, 4, rows, None, None)),
        (1, lambda: M.moe_swiglu_ckpt_bwd(c, rows, w, rows, None, None, 4, rows, rows, None)),
        (1, lambda: M.moe_route_bwd(c, x, None, w, w, off, inv, inv, T, w, wt, None, None)),
        (1, lambda: M.moe_route_bwd(c, x, None, w, w, None, inv, inv, T, w, wt, None, odd)),
        (2, lambda: M.moe_expert_product(c, rows, wt, off, T * K, 192, 256, 0, rows)),
        (2, lambda: M.moe_expert_product(c, rows, wt, off, T * K, 256, 16512, 0, rows)),
        (1, lambda: M.moe_expert_product(c, rows, wt, off, T * K, 0, 256, 0, rows)),
        (1, lambda: M.moe_expert_product(c, rows, wt, None, T * K, 256, 256, 0, rows)),
        (1, lambda: M.moe_expert_product(c, odd, wt, off, T * K, 256, 256, 0, rows)),
        (2, lambda: M.moe_expert_wgrad(c, rows, rows, off, T * K, 256, 256, M.MOE_T_BF16, 1, wt)),
        (1, lambda: M.moe_expert_wgrad(c, rows, rows, off, T * K, 256, 256, M.MOE_T_E4M3_B128, 0, wt)),
        (1, lambda: M.moe_expert_wgrad(c, None, rows, off, T * K, 256, 256, 0, 0, wt)),
    ]
    for i, (status, call) in enumerate(calls):
        with pytest.raises(M.MoeError) as e:
            call()
        assert e.value.status == status, (i, e.value)
    assert L.launches() == before and L.status() == 0


def test_bad_device_indices_are_ignored_and_reported(layers):
    """inv, perm, offsets and expert entries outside their arrays: taken as dropped, nothing read or written there."""
    import mixture_experts_layer_24_b200 as M
    T, K, E, H, I = 6, 2, 8, 256, 128
    L = layers(H, E, K, I)
    r = _cuda(R.routing(T, K, E, 30))
    bad = r["inv"].clone()
    bad[1, 0], bad[4, 1] = T * K, 2 ** 31 - 1
    dropped = r["inv"].clone()
    dropped[1, 0] = dropped[4, 1] = -1
    x, rows, dout = _rand(31, T, H), _rand(32, T * K, H), _rand(33, T, H)
    gu, dh = _rand(34, T * K, 2 * I), _rand(35, T * K, I)

    def every(inv):
        z = lambda *s: torch.zeros(s, dtype=BF16, device="cuda")  # noqa: E731
        q0, s0 = torch.zeros((T * K, 2 * I), dtype=torch.uint8, device="cuda"), torch.zeros((T * K, 2), device="cuda")
        h, q, s = L.swiglu_ckpt(gu, inv, out=(z(T * K, I), q0, s0))
        return [L.dispatch(x, inv, out=z(T * K, H)), L.dispatch_bwd(rows, inv), L.combine_weighted(rows, r["w"], inv),
                *L.combine_weighted_bwd(dout, rows, r["w"], inv, out=z(T * K, H)), h, q, s,
                *L.swiglu_ckpt_bwd(q, s, dh, topk_w=r["w"], inv=inv, out=(z(T * K, 2 * I), z(T * K, I)))]

    want = every(dropped)
    assert L.status() == 0
    got = every(bad)
    assert L.status() == M.binding.MOE_DEV_BAD_INDEX
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # an expert index outside the router
    idx = r["idx"].clone()
    idx[2, 1] = E
    dl, wr = _rand(36, T, K, dtype=F32), _rand(37, E, H, dtype=F32)
    dl0 = dl.clone()
    dl0[2, 1] = 0
    a, b = L.dispatch_bwd(rows, r["inv"], dl, idx, wr), L.dispatch_bwd(rows, r["inv"], dl0, r["idx"], wr)
    assert L.status() == M.binding.MOE_DEV_BAD_EXPERT and torch.equal(a, b)
    # offsets past the rows: those experts compute nothing
    off = r["offsets"].clone()
    off[E] = T * K + 5
    w = _rand(38, E, 256, H)
    out = torch.full((T * K, 256), 7.0, dtype=BF16, device="cuda")
    L.expert_product(rows, w, off, out=out)
    assert L.status() == M.binding.MOE_DEV_BAD_INDEX
    last = int(r["offsets"][E - 1])
    assert torch.equal(out[:last], L.expert_product(rows, w, r["offsets"])[:last]) and (out[last:] == 7).all()
    dwr = L.route_bwd(x, r["w"], r["w"], off, r["perm_src"], r["perm_k"])[1]
    assert L.status() & M.binding.MOE_DEV_BAD_INDEX and torch.isfinite(dwr).all()
    src = r["perm_src"].clone()
    src[3] = T
    L.route_bwd(x, r["w"], r["w"], r["offsets"], src, r["perm_k"])
    assert L.status() == M.binding.MOE_DEV_BAD_INDEX


def test_other_streams_and_replayed_graphs(layers):
    """The same bits on a side stream, passed as an argument and as the current one, and from replayed graphs whose
    inputs change; two graphs that replay at the same time keep apart."""
    T, K, E, H, I = 70, 4, 16, 512, 256
    L, r = layers(H, E, K, I), _cuda(R.routing(T, K, E, 40, 0.1))
    x, dw = _rand(41, T, H), _rand(42, T, K, dtype=F32)
    rows, w = _rand(43, T * K, H), _rand(44, E, 2 * I, H, std=0.05)
    P = (r["offsets"], r["perm_src"], r["perm_k"])

    def step(x, stream=None):
        z = torch.zeros((T * K, H), dtype=BF16, device="cuda")
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        xs = L.dispatch(x, r["inv"], out=z, stream=stream)
        return [xs, L.expert_product(xs, w, r["offsets"], out=torch.zeros((T * K, 2 * I), dtype=BF16, device="cuda"))
                if stream is None else xs, *L.route_bwd(x, r["w"], dw, *P, stream=stream),
                L.dispatch_bwd(rows, r["inv"], stream=stream)]

    want = step(x)
    side = torch.cuda.Stream()
    got = step(x, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and all(torch.equal(a, b) for a, b in zip(got[2:], want[2:]))
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(x)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for seed in (51, 52):
        xin = _rand(41, T, H)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(xin)
        graphs.append((g, xin, out, seed))
    for g, xin, out, seed in graphs:
        xin.copy_(_rand(seed, T, H))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for (g, xin, out, seed), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for g, xin, out, seed in graphs:
        assert all(torch.equal(a, b) for a, b in zip(out, step(_rand(seed, T, H))))
    assert L.status() == 0


def test_rows_past_32_bit_offsets(layers):
    """More than 2^31 elements in the sorted rows: the last rows are where they belong."""
    T, K, E, H = 65536, 9, 16, 4096  # 2.4e9 elements
    L, P = layers(H, E, K), T * K
    inv = torch.arange(P, device="cuda", dtype=torch.int32).flip(0).view(T, K).contiguous()
    x, w = _rand(1, T, H), torch.rand(T, K, device="cuda")
    xs = L.dispatch(x, inv)
    tok = torch.tensor([0, 1, T // 2, T - 1], device="cuda")
    for k in (0, K - 1):
        assert torch.equal(xs[inv[tok, k].long()], x[tok])
    ref, mag = R.dispatch_bwd(xs, inv[tok])
    _within(L.dispatch_bwd(xs, inv)[tok], ref, K * U * mag + R.BF16_HALF * ref.abs() * 1.01, "dx")
    ref, mag = R.combine(xs, w[tok], inv[tok])
    _within(L.combine_weighted(xs, w, inv)[tok], ref, K * U * mag + R.BF16_HALF * ref.abs() * 1.01, "out")
    dy, dw = L.combine_weighted_bwd(x, xs, w, inv)
    want, ref, mag = R.combine_bwd(x[tok], xs, w[tok], inv[tok])
    _within(dy[inv[tok].long()], want, want.abs() * (R.BF16_HALF + 2 * U), "dy")
    _within(dw[tok], ref, (H + 1) * U * mag * 1.01, "dw")
    assert L.status() == 0


def test_activation_and_products_past_32_bit_offsets(layers):
    """The same for the activation's rows, the products' rows and the weights' gradient (more than 2^31 elements)."""
    rows, I = 540672, 2048
    L = layers(256, 8, 1, I)
    gu = torch.zeros((rows, 2 * I), dtype=BF16, device="cuda")
    gu[-3:] = _rand(2, 3, 2 * I)
    h, q, s = L.swiglu_ckpt(gu)
    small = L.swiglu_ckpt(gu[-3:])
    assert all(torch.equal(a[-3:], b) for a, b in zip((h, q, s), small))
    dh = _rand(3, 3, I)
    h[-3:] = dh
    dgu = L.swiglu_ckpt_bwd(q, s, h)[0]
    assert torch.equal(dgu[-3:], L.swiglu_ckpt_bwd(*small[1:], dh)[0])
    off = torch.zeros(9, dtype=torch.int32, device="cuda")
    off[8], off[7] = rows, rows - 3
    wt = _rand(4, 8, 128, 2 * I)
    got = L.expert_product(gu, wt, off)
    assert torch.equal(got[-3:], L.expert_product(gu[-3:], wt, (off - (rows - 3)).clamp(min=0)))
    back = L.expert_product(got, wt, off, transposed=True)
    assert torch.equal(back[-3:], L.expert_product(got[-3:], wt, (off - (rows - 3)).clamp(min=0), transposed=True))
    del gu, h, q, s, dgu, got, back
    E, n = 530, 2048  # 2.2e9 elements of dw
    L = layers(256, E, 1, 128)
    off = torch.arange(E + 1, device="cuda", dtype=torch.int32)
    a, dy = _ints(5, E, n), _ints(6, E, n)
    dw = L.expert_wgrad(dy, a, off)
    for e in (0, E - 1):
        assert torch.equal(dw[e], dy[e][:, None] * a[e][None, :])
    assert L.status() == 0


def test_router_gradient_of_the_most_pairs(layers):
    """65536 tokens of 32 pairs, half of them of one expert or its neighbour, from a list and from the choice."""
    T, K, E, H = 65536, 32, 64, 128
    L, r = layers(H, E, K), _cuda(R.routing(T, K, E, 170, drop=0.02, skew=3.0))
    x, dw = _rand(171, T, H), _rand(172, T, K, dtype=F32)
    listed = L.route_bwd(x, r["w"], dw, r["offsets"], r["perm_src"], r["perm_k"])
    chosen = L.route_bwd(x, r["w"], dw, topk_idx=r["idx"])
    for got, inv in ((listed, r["inv"]), (chosen, torch.zeros_like(r["inv"]))):
        dl_ref, dwr_ref, db_ref, dl_mag, dwr_mag, db_mag = R.route_bwd(x, r["w"], dw, r["idx"], inv, E)
        _within(got[0], dl_ref, (K + 2) * U * dl_mag * 1.01, "dlogit")
        most = T  # an expert's pairs: every token at most
        _within(got[1], dwr_ref, (K + 4 + most) * U * dwr_mag * 1.01, "dw_router")
        _within(got[2], db_ref, (K + 3 + most) * U * db_mag * 1.01, "dlogit_bias")
        # the sums are split over many blocks, so the error is far below that bound: 2-norm within 2^-20
        for a, b in ((got[1], dwr_ref), (got[2], db_ref)):
            assert (a.to(F64) - b).norm() <= 2.0 ** -20 * b.norm()
    assert L.status() == 0


def test_router_gradient_in_plain_stream_order(layers):
    """Without programmatic dependent launch: the same bits."""
    import mixture_experts_layer_24_b200 as M
    T, K, E, H = 700, 4, 12, 256
    r = _cuda(R.routing(T, K, E, 99, 0.05))
    args = (_rand(100, T, H), r["w"], _rand(101, T, K, dtype=F32), r["offsets"], r["perm_src"], r["perm_k"])
    plain = M.MoeLayer(H, E, K, 128, flags=M.binding.MOE_FLAG_NO_PDL)
    for _ in range(3):
        got, want = plain.route_bwd(*args), layers(H, E, K).route_bwd(*args)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    plain.close()


def test_calls_from_two_threads(layers):
    """Two host threads, each with a stream of its own, on one layer: the bits of a single thread."""
    import threading
    T, K, E, H, I = 65, 4, 16, 512, 256
    L, r = layers(H, E, K, I), _cuda(R.routing(T, K, E, 90))
    w = _rand(91, E, 2 * I, H, std=0.05)
    sets = [(_rand(92 + s, T, H), _rand(94 + s, T, K, dtype=F32)) for s in range(2)]

    def work(s):
        x, dw = sets[s]
        xs = L.dispatch(x, r["inv"])
        h, q, sc = L.swiglu_ckpt(L.expert_product(xs, w, r["offsets"]), r["inv"])
        return [xs, h, q, sc, L.expert_wgrad(L.swiglu_ckpt_bwd(q, sc, h, r["w"], r["inv"])[0], xs, r["offsets"]),
                *L.route_bwd(x, r["w"], dw, r["offsets"], r["perm_src"], r["perm_k"])]

    want = [work(s) for s in range(2)]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def run(s):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got[s] = work(s)
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # surfaced below
            errors.append(e)

    threads = [threading.Thread(target=run, args=(s,)) for s in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join(timeout=120)
    assert not errors, errors
    for s in range(2):
        assert all(torch.equal(a, b) for a, b in zip(got[s], want[s]))
    assert L.status() == 0


def _hammer(calls, rounds):
    """Each call from a thread and on a stream of its own, many times over, straight through the C function (which lets
    go of the interpreter's lock). Returns the errors."""
    import threading
    import mixture_experts_layer_24_b200 as M
    errors = []

    def run(call):
        stream = torch.cuda.Stream()
        for i in range(rounds):
            if call(stream.cuda_stream) != 0:
                errors.append(M.lib().moe_last_error().decode())
            if i % 100 == 0:
                stream.synchronize()
        stream.synchronize()

    threads = [threading.Thread(target=run, args=(c,)) for c in calls]
    for th in threads:
        th.start()
    for th in threads:
        th.join(timeout=240)
    assert not any(th.is_alive() for th in threads)
    return errors


def test_products_of_two_layers_from_two_threads(layers):
    """Layers of 8 and of 1024 experts, whose launches need different amounts of shared memory."""
    import mixture_experts_layer_24_b200 as M
    calls, kept = [], []
    for E in (8, 1024, 8, 1024):
        L, (off, P) = layers(256, E, 1, 128), _segments([0] * (E - 1) + [3])
        for transposed in (0, 1):
            a, w = _ints(155 + E, P, 128), _ints(156 + E, E, 128, 128)
            out = torch.zeros_like(a)
            args = (L.ctx, a.data_ptr(), w.data_ptr(), off.data_ptr(), P, 128, 128, transposed, out.data_ptr())
            calls.append(lambda s, args=args: M.lib().moe_expert_product(*args, s))
            kept.append((L, a, w, off, out, transposed))
    torch.cuda.synchronize()
    errors = _hammer(calls, 4000)
    assert not errors, (len(errors), errors[0])
    for L, a, w, off, out, transposed in kept:
        assert torch.equal(out, L.expert_product(a, w, off, transposed=bool(transposed))) and L.status() == 0


def _in_a_new_thread(f):
    import threading
    result = []

    def run():
        try:
            result.append((f(), None))
        except Exception as e:  # surfaced below
            result.append((None, e))

    th = threading.Thread(target=run)
    th.start()
    th.join(timeout=120)
    value, error = result[0]
    if error is not None:
        raise error
    return value


def test_first_call_of_a_thread(layers):
    """A call whose thread has made no CUDA call before (outputs at hand, so not even an allocation): the products,
    whose tensor maps come from the driver, and the registration of experts."""
    import mixture_experts_layer_24_b200 as M
    T, K, E, H, I = 9, 2, 8, 256, 128
    L, r = M.MoeLayer(H, E, K, I), _cuda(R.routing(T, K, E, 150))
    w_gu, w_dn = _rand(151, E, 2 * I, H, std=0.1), _rand(152, E, H, I, std=0.1)
    a, x = _rand(153, T * K, H), _rand(154, T, H)
    want = L.expert_product(a, w_gu, r["offsets"])
    dw = L.expert_wgrad(want, a, r["offsets"])
    out, dw2 = torch.zeros_like(want), torch.zeros_like(dw)
    torch.cuda.synchronize()
    _in_a_new_thread(lambda: L.expert_product(a, w_gu, r["offsets"], out=out))
    _in_a_new_thread(lambda: L.expert_wgrad(want, a, r["offsets"], out=dw2))
    for e in range(E):
        _in_a_new_thread(lambda: L.register(e, w_gu[e], w_dn[e]))
    y = torch.zeros((T * K, H), dtype=F32, device="cuda")
    ws = L.workspace(T)
    torch.cuda.synchronize()
    _in_a_new_thread(lambda: M.moe_expert_ffn(L.ctx, L.slots, x, r["perm_src"], r["perm_k"], r["offsets"], r["w"], T,
                                              y, ws))
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(dw2, dw)
    assert torch.equal(y, L.expert_ffn(x, r["perm_src"], r["perm_k"], r["offsets"], r["w"])) and L.status() == 0
    L.close()


def test_launches_are_counted_and_timed(layers):
    """moe_launch_count and moe_profile_* see the training calls under their own kinds."""
    import mixture_experts_layer_24_b200 as M
    T, K, E, H, I = 9, 2, 8, 256, 128
    L, r = layers(H, E, K, I), _cuda(R.routing(T, K, E, 96))
    x, w = _rand(97, T, H), _rand(98, E, 2 * I, H)
    torch.cuda.synchronize()
    before = L.launches()
    M.moe_profile_enable(L.ctx, True)
    M.moe_profile_read(L.ctx)
    xs = L.dispatch(x, r["inv"])
    h, q, s = L.swiglu_ckpt(L.expert_product(xs, w, r["offsets"]), r["inv"])
    L.expert_wgrad(q.to(BF16), xs, r["offsets"])
    L.route_bwd(x, r["w"], r["w"], r["offsets"], r["perm_src"], r["perm_k"])
    prof = M.moe_profile_read(L.ctx)
    M.moe_profile_enable(L.ctx, False)
    assert L.launches() - before == 1 + 1 + 1 + 1 + 2
    assert [prof[k][1] for k in ("rows", "swiglu", "route_bwd", "product")] == [1, 1, 1, 2]
    assert all(prof[k][0] > 0 for k in ("rows", "swiglu", "route_bwd", "product")) and prof["router"][1] == 0


STEP = [(1, 256, 8, 2, 128), (37, 256, 8, 2, 256), (300, 512, 48, 4, 256)]


@pytest.mark.parametrize("T,H,E,K,I", STEP)
@pytest.mark.parametrize("ckpt_x", [False, True])
def test_training_step_against_autograd(layers, T, H, E, K, I, ckpt_x):
    """A whole step (mixture_experts_layer_24_b200.train) against torch.autograd over the layer's definition in 64
    bits, at the checkpointed gate/up values. Each gradient passes through at most five bf16 roundings of its
    factors (rows, products, activations: 2^-8 each, relative to their magnitudes); they average over the sums, so
    the 2-norm of the error is held to five of them."""
    import mixture_experts_layer_24_b200 as M
    from mixture_experts_layer_24_b200 import train
    L = layers(H, E, K, I)
    x, wr = _rand(61, T, H), _rand(62, E, H, std=0.05, dtype=F32)
    bias = _rand(63, E, std=0.5, dtype=F32)
    w_gu, w_dn = _rand(64, E, 2 * I, H, std=0.06), _rand(65, E, H, I, std=0.06)
    dout = _rand(66, T, H)
    out, saved = train.forward(L, x, wr, w_gu, w_dn, bias, ckpt_x=ckpt_x)
    got = train.backward(L, saved, dout, wr, w_gu, w_dn, w_dtype=F32)
    assert L.status() == 0
    rel = lambda a, b: ((a.to(F64) - b).norm() / b.norm()).item()  # noqa: E731
    # forward: against the serving forward of the same layer
    for e in range(E):
        L.register(e, w_gu[e], w_dn[e])
    assert rel(out, L.forward(x, wr, bias).to(F64)) <= 4 * R.BF16_HALF
    leaves = [t.to(F64).requires_grad_() for t in (x, wr, bias, w_gu, w_dn)]
    xv = x.to(F64)
    if ckpt_x:  # the gradients of the weights use x as the checkpoint holds it
        xv = R.decode(saved.x, saved.x_scales)
        leaves[0] = xv.clone().requires_grad_()
    gu_at = R.decode(saved.gu_q, saved.gu_s)[saved.inv.long()]
    if ckpt_x:  # routing weights are those of the forward, from x itself
        logits = x.to(F64) @ leaves[1].t() + leaves[2] + (leaves[0] - xv) @ leaves[1].t() + \
            (xv - x.to(F64)) @ (leaves[1] - leaves[1].detach()).t()
        w = torch.softmax(torch.gather(logits, 1, saved.topk_idx.long()), 1)
        loss = 0
        for k in range(K):
            e = saved.topk_idx[:, k].long()
            gu = torch.einsum("toh,th->to", leaves[3][e], leaves[0])
            gu = gu + (gu_at[:, k] - gu).detach()
            h = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
            loss = loss + (w[:, k, None] * torch.einsum("thi,ti->th", leaves[4][e], h) * dout.to(F64)).sum()
    else:
        loss = R.layer_loss(*leaves, dout.to(F64), saved.topk_idx, gu_at=gu_at)
    loss.backward()
    for name, leaf in zip(("x", "w_router", "logit_bias", "w_gu", "w_dn"), leaves):
        if leaf.grad.norm() > 0:
            assert rel(getattr(got, name), leaf.grad) <= 5 * R.BF16_HALF, name
    # accumulation: a second backward into the same fp32 gradients doubles them
    train.backward(L, saved, dout, wr, w_gu, w_dn, into=(got.w_gu, got.w_dn))
    again = train.backward(L, saved, dout, wr, w_gu, w_dn, w_dtype=F32)
    assert torch.equal(got.w_gu, 2 * again.w_gu) and torch.equal(got.w_dn, 2 * again.w_dn)


def test_training_step_without_tokens(layers):
    from mixture_experts_layer_24_b200 import train
    T, H, E, K, I = 0, 256, 8, 2, 128
    L = layers(H, E, K, I)
    x, wr = _rand(1, T, H), _rand(2, E, H, dtype=F32)
    w_gu, w_dn = _rand(3, E, 2 * I, H), _rand(4, E, H, I)
    out, saved = train.forward(L, x, wr, w_gu, w_dn, ckpt_x=True)
    g = train.backward(L, saved, out, wr, w_gu, w_dn)
    assert out.shape == (0, H) and g.x.shape == (0, H)
    assert all((t == 0).all() for t in (g.w_router, g.logit_bias, g.w_gu, g.w_dn)) and L.status() == 0


def test_captured_training_step(layers):
    """Forward and backward captured in one graph, beside an eager step that stays alive: replays on new inputs give
    the eager bits, also after larger eager calls have replaced the layer's own workspace."""
    from mixture_experts_layer_24_b200 import train
    T, H, E, K, I = 33, 256, 8, 2, 256
    L = layers(H, E, K, I)
    wr = _rand(72, E, H, std=0.05, dtype=F32)
    w_gu, w_dn = _rand(73, E, 2 * I, H, std=0.06), _rand(74, E, H, I, std=0.06)

    def step(x, dout):
        out, saved = train.forward(L, x, wr, w_gu, w_dn, ckpt_x=True)
        g = train.backward(L, saved, dout, wr, w_gu, w_dn)
        return [out, g.x, g.w_router, g.logit_bias, g.w_gu, g.w_dn]

    x, dout = _rand(71, T, H), _rand(75, T, H)
    alive = step(x, dout)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(x, dout)
    L.route(_rand(76, 500, H), wr)
    for seed in (81, 82):
        x.copy_(_rand(seed, T, H))
        dout.copy_(_rand(seed + 10, T, H))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, step(x, dout)))
    assert torch.isfinite(alive[1].float()).all() and L.status() == 0
