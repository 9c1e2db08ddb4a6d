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
