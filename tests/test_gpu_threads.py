"""Layers of different sizes served from several host threads at once. A
kernel's limits (cudaFuncSetAttribute) belong to the kernel and not to a call,
so what one call sets must do for every other one."""

import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def _layer(wdtype, H, E, I, seed):
    """A layer whose experts share one set of weights."""
    import mixture_experts_layer_24_b200 as M
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: (torch.randn(*s, generator=gen, device="cuda") * 0.05).to(torch.bfloat16)  # noqa: E731
    gu, dn = rnd(2 * I, H), rnd(H, I)
    weights = (gu, dn)
    if wdtype == M.MOE_FP8_E4M3_B128:
        byte = lambda *s: torch.empty(s, dtype=torch.uint8, device="cuda")  # noqa: E731
        weights = (byte(2 * I, H), byte(H, I), torch.empty((2 * I // 128, H // 128), device="cuda"),
                   torch.empty((H // 128, I // 128), device="cuda"))
        M.moe_quantize_e4m3(gu, 2 * I, H, 128, weights[0], weights[2])
        M.moe_quantize_e4m3(dn, H, I, 128, weights[1], weights[3])
    L = M.MoeLayer(H, E, 1, I, wdtype=wdtype)
    for e in range(E):
        L.register(e, *weights)
    return L, rnd(E, H).float()


@pytest.mark.parametrize("fp8,T,rounds", [(False, 1, 3000), (False, 64, 1000), (True, 300, 500)])
def test_forwards_of_two_layers_from_two_threads(fp8, T, rounds):
    import mixture_experts_layer_24_b200 as M
    wdtype = M.MOE_FP8_E4M3_B128 if fp8 else M.MOE_BF16
    cases = []
    for i, (H, E) in enumerate(((256, 4), (4096, 1024), (256, 4), (4096, 1024))):
        L, wr = _layer(wdtype, H, E, 256, seed=i)
        x = torch.randn(T, H, device="cuda").to(torch.bfloat16)
        out, ws = torch.zeros_like(x), torch.empty(M.moe_workspace_size(L.ctx, T), dtype=torch.uint8, device="cuda")
        args = (L.ctx, L.slots, x.data_ptr(), wr.data_ptr(), None, T, out.data_ptr(), ws.data_ptr(), ws.numel())
        cases.append((L, x, wr, out, ws, args))
    torch.cuda.synchronize()
    errors = []

    def run(args):
        stream = torch.cuda.Stream()
        for i in range(rounds):
            if M.lib().moe_forward(*args, stream.cuda_stream) != 0:
                errors.append(M.lib().moe_last_error().decode())
            if i % 50 == 0:
                stream.synchronize()
        stream.synchronize()

    threads = [threading.Thread(target=run, args=(c[-1],)) for c in cases]
    for th in threads:
        th.start()
    for th in threads:
        th.join(timeout=240)
    assert not any(th.is_alive() for th in threads)
    assert not errors, (len(errors), errors[0])
    for L, x, wr, out, ws, args in cases:
        assert torch.equal(out, L.forward(x, wr)) and L.status() == 0
        L.close()


def _stacked(H, E, I, seed, std=0.05):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda") * std  # noqa: E731
    return rnd(E, 2 * I, H).to(torch.bfloat16), rnd(E, H, I).to(torch.bfloat16), rnd(E, H)


def _tokens(T, H, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(T, H, generator=gen, device="cuda").to(torch.bfloat16)


def test_few_tokens_routed_beside_each_other():
    """Up to 4 tokens the router's last CTA takes the top-k, found by an arrival counter: calls of one layer on several
    streams, each with a workspace of its own, and replayed graphs among them, must not count each other's CTAs. The
    layer is used further afterwards."""
    import mixture_experts_layer_24_b200 as M
    H, E, K = 4096, 384, 8
    L = M.MoeLayer(H, E, K, 128)
    wr = torch.randn(E, H, device="cuda")

    def case(T, seed):
        x = _tokens(T, H, seed)
        ws = torch.empty(M.moe_workspace_size(L.ctx, T), dtype=torch.uint8, device="cuda")
        idx, w = torch.zeros((T, K), dtype=torch.int32, device="cuda"), torch.zeros((T, K), device="cuda")
        return x, idx, w, ws, T

    def want(x):  # a layer of its own, one call at a time
        alone = M.MoeLayer(H, E, K, 128)
        got = alone.route(x, wr)
        torch.cuda.synchronize()
        alone.close()
        return got

    cases = [case(T, 10 + T) for T in (1, 2, 3, 4, 1, 4)]
    replayed = [case(T, 20 + T) for T in (1, 4)]
    wanted = [want(c[0]) for c in cases + replayed]
    torch.cuda.synchronize()
    graphs = []
    for x, idx, w, ws, T in replayed:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(20):
                M.moe_route(L.ctx, x, wr, None, T, idx, w, ws)
        graphs.append(g)

    def eager(c):
        x, idx, w, ws, T = c
        args = (L.ctx, x.data_ptr(), wr.data_ptr(), None, T, idx.data_ptr(), w.data_ptr(), ws.data_ptr(), ws.numel())
        return lambda stream: M.lib().moe_route(*args, stream.cuda_stream)

    def replay(g):
        def call(stream):
            with torch.cuda.stream(stream):
                g.replay()
            return 0
        return call

    calls = [(eager(c), 1500) for c in cases] + [(replay(g), 100) for g in graphs]
    errors = []

    def run(call, rounds):
        stream = torch.cuda.Stream()
        for i in range(rounds):
            if call(stream) != 0:
                errors.append(M.lib().moe_last_error().decode())
            if i % 50 == 0:
                stream.synchronize()
        stream.synchronize()

    threads = [threading.Thread(target=run, args=c) for c in calls]
    for th in threads:
        th.start()
    for th in threads:
        th.join(timeout=240)
    assert not any(th.is_alive() for th in threads) and not errors, errors[:1]
    for (x, idx, w, ws, T), (idx0, w0) in zip(cases + replayed, wanted):
        assert torch.equal(idx, idx0) and torch.equal(w, w0), T
    for c in cases:
        assert all(torch.equal(a, b) for a, b in zip(L.route(c[0], wr), want(c[0])))
    assert L.status() == 0
    L.close()


def test_captured_forwards_replayed_beside_each_other():
    """Two graphs of one layer (MoeLayer.capture: a workspace each), one token each, on two streams."""
    import mixture_experts_layer_24_b200 as M
    H, E, K, I = 512, 64, 4, 256
    w_gu, w_dn, wr = _stacked(H, E, I, 3)
    L = M.MoeLayer(H, E, K, I)
    for e in range(E):
        L.register(e, w_gu[e], w_dn[e])
    xs = [_tokens(T, H, 30 + T) for T in (1, 3)]
    wanted = [L.forward(x, wr) for x in xs]
    graphs = [L.capture(x, wr) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(200):
        for (g, _), stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                for _ in range(5):
                    g.replay()
        torch.cuda.synchronize()
        for (_, out), ref in zip(graphs, wanted):
            assert torch.equal(out, ref)
            out.zero_()
        torch.cuda.synchronize()
    assert L.status() == 0
    L.close()


def test_training_forwards_of_few_tokens_from_two_threads():
    import mixture_experts_layer_24_b200 as M
    from mixture_experts_layer_24_b200 import train
    H, E, K, I = 512, 64, 4, 256
    w_gu, w_dn, wr = _stacked(H, E, I, 4)
    L = M.MoeLayer(H, E, K, I)
    xs = [_tokens(T, H, 40 + T) for T in (1, 2, 4)]
    wanted = [train.forward(L, x, wr, w_gu, w_dn)[0] for x in xs]
    torch.cuda.synchronize()
    got, errors = [None] * len(xs), []

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(100):
                    out, _ = train.forward(L, xs[i], wr, w_gu, w_dn)
                    if not torch.equal(out, wanted[i]):
                        errors.append(i)
                got[i] = out
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # surfaced below
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(xs))]
    for th in threads:
        th.start()
    for th in threads:
        th.join(timeout=240)
    assert not any(th.is_alive() for th in threads) and not errors, errors[:3]
    assert all(torch.equal(a, b) for a, b in zip(got, wanted)) and L.status() == 0
    L.close()


def test_more_captured_routes_than_counters():
    """A captured launch keeps its counter. Where none is left the top-k is a launch of its own: the same bits."""
    import mixture_experts_layer_24_b200 as M
    H, E, K = 256, 8, 2
    L = M.MoeLayer(H, E, K, 128)
    wr, xs = torch.randn(E, H, device="cuda"), [_tokens(T, H, 50 + T) for T in (1, 2, 4)]
    wanted = [L.route(x, wr) for x in xs]
    torch.cuda.synchronize()
    ws = torch.empty(M.moe_workspace_size(L.ctx, 4), dtype=torch.uint8, device="cuda")
    outs = [(torch.zeros_like(i), torch.zeros_like(w)) for i, w in wanted]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for n in range(4200):
            x, (idx, w) = xs[n % 3], outs[n % 3]
            M.moe_route(L.ctx, x, wr, None, x.shape[0], idx, w, ws)
    g.replay()
    torch.cuda.synchronize()
    for (idx, w), (idx0, w0) in zip(outs, wanted):
        assert torch.equal(idx, idx0) and torch.equal(w, w0)
    with torch.cuda.stream(torch.cuda.Stream()):  # a stream without a counter
        late = [L.route(x, wr) for x in xs]
        torch.cuda.current_stream().synchronize()
    for got, ref in zip(late, wanted):
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    assert L.status() == 0
    L.close()
