"""Calls from host threads: a thread's first CUDA call may be one of the library's, and several threads
may call on one stream with the binding's own workspace."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    from weight_only_int4_w4_b200 import w4 as mod
    return mod


def layer(w4, N, K, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return w4.w4_quantize(torch.randn((N, K), generator=gen, device="cuda") / K ** 0.5), gen


@pytest.mark.parametrize("M", [1, 4, 16, 100])
def test_the_first_call_of_a_thread(w4, M):
    """Every entry point as the first thing that a thread does with CUDA, outputs and workspace
    given, so that nothing else has made a context current there."""
    N, K = 512, 1024
    w, gen = layer(w4, N, K, 1)
    X = torch.randn((M, K), generator=gen, device="cuda").to(torch.bfloat16)
    dY = torch.randn((M, N), generator=gen, device="cuda").to(torch.bfloat16)
    Y = [torch.empty((M, N), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    H, dX = torch.empty((M, N // 2), dtype=torch.bfloat16, device="cuda"), torch.empty_like(X)
    dX2 = torch.empty_like(X)
    dH = dY[:, :N // 2].contiguous()
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    X_host, Y_host = X.cpu().pin_memory(), torch.empty((M, N), dtype=torch.bfloat16).pin_memory()
    stream = torch.cuda.current_stream()
    kw = dict(ws=ws, stream=stream)
    calls = [lambda: w4.w4a16_gemm(X, *w, out=Y[0], **kw),
             lambda: w4.w4a16_gemm_host(X_host, X, *w, Y_host, Y[3], **kw),
             lambda: w4.w4a16_linear(X, *w, out=Y[1], **kw),
             lambda: w4.w4a16_gated(X, *w, out=H, **kw),
             lambda: w4.w4a16_linear_grad(dY, *w, out=dX, **kw),
             lambda: w4.w4a16_gated_grad(dH, dY, *w, out=dX2, **kw)]
    if M <= 64:
        calls.append(lambda: w4.w4a16_gemm_decode_static(X, *w, out=Y[2], stream=stream))
    outs = [Y[0], Y_host, Y[1], H, dX, dX2, Y[2]]
    for f in calls:
        f()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs[:len(calls)]]
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    wrong = []
    for f in calls:
        def work():
            try:
                f()
            except Exception as e:  # seen by the test
                wrong.append(e)
        t = threading.Thread(target=work)
        t.start()
        t.join()
    torch.cuda.synchronize()
    assert not wrong, wrong
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_calls_from_threads_on_one_stream(w4):
    """Three threads call every kernel on one stream: the same bits as one call alone."""
    N, K = 2000, 1024
    w, gen = layer(w4, N, K, 1)
    Xs = [torch.randn((M, K), generator=gen, device="cuda").to(torch.bfloat16) for M in (1, 6, 16, 48, 150, 300)]
    want = [w4.w4a16_gemm(X, *w) for X in Xs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    wrong = []

    def work(order):
        try:
            with torch.cuda.stream(side):
                for _ in range(40):
                    got = [(i, w4.w4a16_gemm(Xs[i], *w)) for i in order]
                    wrong.extend(i for i, g in got if not torch.equal(g, want[i]))
        except Exception as e:  # seen by the test
            wrong.append(e)

    ts = [threading.Thread(target=work, args=(o,)) for o in ([0, 1, 2, 3, 4, 5], [5, 4, 3, 2, 1, 0], [2, 5, 3, 0, 4, 1])]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not wrong, wrong[:3]
    assert w4.w4_device_error() == 0


@pytest.mark.parametrize("M", [1, 16, 100])
def test_the_first_call_on_another_stream_finds_its_workspace_zeroed(w4, M):
    """The current stream is busy, and the memory that the new workspace takes was in use."""
    N, K = 4096, 4096
    w, gen = layer(w4, N, K, 2)
    X = torch.randn((M, K), generator=gen, device="cuda").to(torch.bfloat16)
    want = w4.w4a16_gemm(X, *w)
    need = max(w4.w4a16_gemm_workspace_size(M, N, K), 1 << 20)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (torch.cuda.current_stream(), side):
        with torch.cuda.stream(s):
            torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    out = torch.empty_like(want)
    torch.cuda._sleep(20_000_000)  # some 10 ms
    w4.w4a16_gemm(X, *w, out=out, stream=side)
    side.synchronize()
    assert w4.w4_device_error() == 0
    assert torch.equal(out, want)
