"""Calls that follow one another in a stream without waiting: a kernel may start
while the one before drains, and must still see all that it wrote."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev(hm):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


@pytest.mark.parametrize("rows,d", [(500, 256), (700, 1024), (640, 2048), (300, 5120)])
def test_chain_gives_the_bits_of_separate_calls(hm, dev, rows, d):
    """Norm, its transpose by quantization, its gradient, one right behind the other, each
    reading what the one before wrote (rstd; dx as the next step's input) and gamma changed
    between the steps, against the same calls with the GPU idle before each: the
    same bits, twenty times."""
    g = torch.Generator(device=dev)
    g.manual_seed(rows + d)
    x0 = torch.randn(rows, d, generator=g, device=dev)
    dy = torch.randn(rows, d, generator=g, device=dev)
    step = torch.randn(d, generator=g, device=dev) * 0.01
    r32 = -(-rows // 32) * 32

    def run(wait):
        pause = torch.cuda.synchronize if wait else (lambda: None)
        new = lambda *s: torch.zeros(*s, dtype=torch.uint8, device=dev)  # noqa: E731
        x, gamma = x0.clone(), torch.ones(d, device=dev)
        rstd, dx, dg = torch.zeros(rows, device=dev), torch.zeros(rows, d, device=dev), torch.zeros(d, device=dev)
        q, s = new(rows, d), new(hm.mxfp8_tiled_scale_bytes(rows, d))
        qt, st = new(d, r32), new(hm.mxfp8_tiled_scale_bytes(d, r32))
        ws = new(hm.rmsnorm_backward_workspace(rows, d))
        torch.cuda.synchronize()
        stream = torch.cuda.current_stream().cuda_stream
        for _ in range(20):
            hm.rmsnorm_mxfp8(x.data_ptr(), d, 0, 0, 0, hm.HM_F32, rows, d, gamma.data_ptr(), 1e-5, 32, rstd.data_ptr(),
                             q.data_ptr(), s.data_ptr(), stream)
            pause()
            hm.mxfp8_quantize(x.data_ptr(), hm.HM_F32, rows, d, d, rstd.data_ptr(), gamma.data_ptr(), 32, 0, 0, 0,
                              qt.data_ptr(), r32, st.data_ptr(), stream)
            pause()
            hm.rmsnorm_backward(dy.data_ptr(), d, x.data_ptr(), x.data_ptr(), dx.data_ptr(), d, hm.HM_F32, rows, d,
                                gamma.data_ptr(), rstd.data_ptr(), dg.data_ptr(), True, ws.data_ptr(), ws.numel(), stream)
            pause()
            gamma += step
            x, dx = dx, x
        torch.cuda.synchronize()
        assert hm.hm_device_error() == 0
        return [t.cpu().numpy().view(np.uint8) for t in (x, rstd, dg, q, s, qt, st)]

    want = run(True)
    for _ in range(3):
        assert all(np.array_equal(a, b) for a, b in zip(run(False), want))


def _session(dev):
    import workloads
    from head_muon_mxfp8_gb300.session import MuonSession
    cfg = workloads.get("tiny_ragged")
    s = MuonSession.from_config(cfg, device=dev)
    data = workloads.generate(cfg, seed=4)
    s.load("g", data["g"])
    torch.cuda.synchronize()
    return s, np.asarray(data["g"], dtype=np.float64)


def test_clip_on_another_stream_while_the_current_one_is_behind(hm, dev):
    """The current stream is busy, with memory to free and fill behind that: nothing that it
    still has to do reaches the clipping's result or its sums."""
    s, g = _session(dev)
    side = torch.cuda.Stream()
    norm = np.sqrt((g * g).sum())
    held = [torch.ones(64, dtype=torch.uint8, device=dev) for _ in range(64)]   # small blocks to be reused
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    for t in held:
        t.fill_(0xFF)
    del held, t
    stats = s.clip_grad_norm(float(norm) * 0.25, stream=side)
    side.synchronize()
    with torch.cuda.stream(side):
        early = stats.clone()
    torch.cuda.synchronize()
    for got in (early.cpu().numpy(), stats.cpu().numpy()):
        assert abs(got[0] - norm) < 1e-5 * norm and abs(got[1] - 0.25) < 1e-5
    assert np.array_equal(s.fetch("g").numpy(), g.astype(np.float32) * stats.cpu().numpy()[1])
    s.close()


def test_clip_with_two_lists_on_two_streams(hm, dev):
    """Two lists in turn on two streams, nothing waiting in between: every result is its own."""
    s, _ = _session(dev)
    a = torch.randn(300_001, device=dev)
    b = torch.randn(1_700_000, device=dev)
    lists = [[(t.data_ptr(), 0, t.numel(), hm.HM_F32)] for t in (a, b)]
    want = [float(t.double().norm()) for t in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for k in range(20):
        got.append((k % 2, s.clip_grad_norm(1.0, tensors=lists[k % 2], stream=streams[(k // 2) % 2])))
    torch.cuda.synchronize()
    assert len({t.data_ptr() for _, t in got}) == 4
    for which, t in got:
        assert abs(float(t[0]) - want[which]) < 1e-5 * want[which]
    s.close()
