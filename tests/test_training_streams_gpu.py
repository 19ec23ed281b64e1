"""Streams given as handles: what a call makes for itself comes from the memory of
the stream that it runs on, since memory of another one may be handed out while the call's
kernels still use it."""
import pytest
import torch

import static_token_routed_b200 as l3

pytestmark = pytest.mark.gpu


def owner(t):
    """The stream whose memory a tensor is."""
    at = [s["stream"] for s in torch.cuda.memory_snapshot()
          if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]]
    assert len(at) == 1
    return at[0]


@pytest.mark.parametrize("which", ["0", "1", "default", "other", "other's handle", "none"])
def test_memory_is_the_streams_own(which):
    current, other = torch.cuda.Stream(), torch.cuda.Stream()
    stream = {"0": 0, "1": 1, "default": torch.cuda.default_stream(), "other": other,
              "other's handle": other.cuda_stream, "none": None}[which]
    want = {"other": other.cuda_stream, "other's handle": other.cuda_stream, "none": current.cuda_stream}.get(which, 0)
    x, W = torch.randn(300, 64, device="cuda"), torch.randn(500, 64, device="cuda")
    t, G = torch.zeros(300, dtype=torch.int32, device="cuda"), torch.randn(200, 300, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(current):
        loss, lse = l3.l3_xent_forward(x, W, t, stream=stream)
        dx, dW = l3.l3_xent_backward(x, W, t, lse, loss, stream=stream)
        O = l3.l3_orthogonalize(G, stream=stream)
        l3.l3_muon_step(G.clone(), torch.zeros_like(G), G, 0.1, stream=current)
    torch.cuda.synchronize()
    for v in (loss, lse, dx, dW, O):
        assert owner(v) == want and torch.isfinite(v).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [1, 200, 300])
def test_the_first_cuda_call_of_a_thread(n, dtype):
    import threading
    x, W = torch.randn(n, 64, device="cuda").to(dtype), torch.randn(500, 64, device="cuda").to(dtype)
    t, G = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.randn(200, 100 + n, device="cuda").to(dtype)
    loss, lse = l3.l3_xent_forward(x, W, t)
    want = (loss, lse) + l3.l3_xent_backward(x, W, t, lse, loss) + (l3.l3_orthogonalize(G),)
    outs = [torch.empty_like(v) for v in want]
    ws = torch.empty(32 << 20, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    calls = [lambda: l3.l3_xent_forward(x, W, t, outs[0], outs[1], ws),
             lambda: l3.l3_xent_backward(x, W, t, want[1], want[0], outs[2], outs[3], ws),
             lambda: l3.l3_orthogonalize(G, outs[4], workspace=ws),
             lambda: l3.l3_workspace_status(ws)]
    failed = []

    def run(call):
        try:
            call()
        except Exception as e:   # noqa: BLE001 (told to the main thread)
            failed.append(e)

    for call in calls:
        th = threading.Thread(target=run, args=(call,))
        th.start()
        th.join()
    torch.cuda.synchronize()
    assert not failed
    for a, b in zip(outs, want):
        assert torch.equal(a, b)


def test_threads_on_one_stream():
    """Calls from several threads, on the default stream, beside threads that allocate and
    fill memory there: every call's results are those it gives alone."""
    import threading
    g = torch.Generator(device="cuda").manual_seed(1)
    jobs = []
    for n, vocab, rows, cols in ((300, 900, 200, 300), (40, 3000, 150, 700), (600, 500, 90, 1000)):
        x = torch.randn(n, 64, generator=g, device="cuda").to(torch.bfloat16)
        W = torch.randn(vocab, 64, generator=g, device="cuda").to(torch.bfloat16)
        t = torch.randint(0, vocab, (n,), generator=g, device="cuda").to(torch.int32)
        w = torch.rand(n, generator=g, device="cuda")
        G = torch.randn(rows, cols, generator=g, device="cuda")
        jobs.append((x, W, t, w, G))

    def run(x, W, t, w, G):
        loss, lse = l3.l3_xent_forward(x, W, t)
        return (loss, lse) + l3.l3_xent_backward(x, W, t, lse, w) + (l3.l3_orthogonalize(G),)

    alone = [run(*j) for j in jobs]
    torch.cuda.synchronize()
    done, bad = threading.Event(), []

    def calls(job, want):
        try:
            for _ in range(30):
                if not all(torch.equal(a, b) for a, b in zip(run(*job), want)):
                    bad.append(want)
        except Exception as e:   # noqa: BLE001 (told to the main thread)
            bad.append(e)

    def fills():
        while not done.is_set():
            for size in (1 << 12, 1 << 16, 1 << 20, 1 << 22):
                torch.full((size,), 255, dtype=torch.uint8, device="cuda")

    workers = [threading.Thread(target=calls, args=a) for a in zip(jobs, alone)]
    others = [threading.Thread(target=fills) for _ in range(2)]
    for th in workers + others:
        th.start()
    for th in workers:
        th.join()
    done.set()
    for th in others:
        th.join()
    torch.cuda.synchronize()
    assert not bad
