"""Calls on a stream that is not the current one, with the outputs allocated by
the call, while the current stream still has work queued on memory that the
program has already let go of."""
import pytest

torch = pytest.importorskip("torch")
import fp32_gemm_tuning_amd as sg  # noqa: E402

pytestmark = pytest.mark.gpu

M, F, K = 300, 512, 256


@pytest.fixture(scope="module")
def job():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    dev = torch.device("cuda:0")
    gen = torch.Generator().manual_seed(41)
    t = torch.bfloat16
    X, dH, Wg, Wu = (torch.randn(s, generator=gen).to(dev, t) for s in ((M, K), (M, F), (F, K), (F, K)))
    P = torch.empty(M, 2 * F, device=dev)
    sg.glu(X, Wg, Wu, preact=P)
    wg, wu = sg.w4_quantize(Wg, 64), sg.w4_quantize(Wu, 64)
    slow = torch.zeros(1 << 28, device=dev)                      # 1 GiB: a pass takes 0.4 ms
    calls = {
        "glu": lambda s: [sg.glu(X, Wg, Wu, stream=s)],
        "glu_backward": lambda s: list(sg.glu_backward(dH, X, Wg, Wu, P, stream=s)),
        "w4_quantize": lambda s: list(sg.w4_quantize(Wg, 64, zeros=True, stream=s)[:3]),
        "w4_dequantize": lambda s: [sg.w4_dequantize(wg, stream=s)],
        "w4_matmul": lambda s: [sg.w4_matmul(X, wg, stream=s)],
        "w4_glu": lambda s: [sg.w4_glu(X, wg, wu, stream=s)],
    }
    return dev, calls, slow


@pytest.mark.parametrize("address", [False, True], ids=["stream", "address"])
@pytest.mark.parametrize("name", ["glu", "glu_backward", "w4_quantize", "w4_dequantize", "w4_matmul", "w4_glu"])
def test_memory_still_in_use_is_not_taken(job, name, address):
    dev, calls, slow = job
    call = calls[name]
    print("[gpu] memory in use", name, address, flush=True)
    alone = call(None)
    workspace = sg.glu_backward_workspace(torch.empty(M, K, dtype=torch.bfloat16, device=dev), F)
    sizes = [v.numel() * v.element_size() for v in alone] + [workspace]
    torch.cuda.synchronize()
    s = torch.cuda.Stream(dev)
    for _ in range(3):
        # temporaries of the sizes that the call allocates, read after slow work ...
        held = [torch.full((n,), i + 1, dtype=torch.uint8, device=dev) for i, n in enumerate(sizes)]
        torch.cuda.synchronize()
        for _ in range(10):
            slow.add_(1)
        copies = [h.clone() for h in held]
        # ... which the call, on another stream, does not wait for
        del held
        got = call(s.cuda_stream if address else s)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, alone))
        torch.cuda.synchronize()
        for i, c in enumerate(copies):
            assert (c == i + 1).all()


def test_results_outlive_their_use_on_the_current_stream(job):
    # The call's output is read by slow work on the current stream and let go of;
    # further calls on its stream must not write over it before.
    dev, calls, slow = job
    print("[gpu] output in use", flush=True)
    s = torch.cuda.Stream(dev)
    alone = calls["glu"](None)[0].clone()
    torch.cuda.synchronize()
    for _ in range(3):
        got = calls["glu"](s)[0]
        torch.cuda.current_stream().wait_stream(s)
        for _ in range(10):
            slow.add_(1)
        copy = got.clone()
        del got
        junk = [calls[n](s) for n in ("w4_matmul", "glu_backward", "w4_matmul", "w4_glu")]
        torch.cuda.synchronize()
        assert torch.equal(copy, alone)
        del junk


def test_the_default_streams_address(job):
    dev, calls, _ = job
    for name, call in calls.items():
        alone = call(None)
        got = call(torch.cuda.default_stream(dev).cuda_stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, alone)), name
