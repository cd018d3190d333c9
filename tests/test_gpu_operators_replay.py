"""A replayed graph of the operators computes: every output is overwritten with
something else before a replay, the inputs are other ones, and the outputs are
those of calls made directly on these inputs."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev(hm):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def test_replay_on_other_inputs(hm, dev):
    g = torch.Generator(device=dev)
    g.manual_seed(9)
    rows, d, n = 70, 256, 384
    new = lambda *s: torch.zeros(*s, dtype=torch.uint8, device=dev)  # noqa: E731
    x = torch.zeros(rows, d, dtype=torch.bfloat16, device=dev)
    w = torch.randn(n, d, generator=g, device=dev)
    gamma, rstd = torch.ones(d, device=dev), torch.zeros(rows, device=dev)
    q, s = new(rows, d), new(hm.mxfp8_tiled_scale_bytes(rows, d))
    qw, sw = new(n, d), new(hm.mxfp8_tiled_scale_bytes(n, d))
    out, dx, dg = torch.zeros(rows, n, device=dev), torch.zeros(rows, d, device=dev), torch.zeros(d, device=dev)
    x32 = torch.zeros(rows, d, device=dev)
    clipped, stats = torch.zeros(rows, n, device=dev), torch.zeros(2, device=dev)
    lst = hm.grad_list([(out.data_ptr(), clipped.data_ptr(), out.numel(), hm.HM_F32)])
    ws, gws = new(max(16, hm.grad_norm_clip_workspace(lst))), new(hm.rmsnorm_backward_workspace(rows, d))
    outputs = (q, s, qw, sw, rstd, out, dx, dg, clipped, stats)

    def step():
        st = torch.cuda.current_stream().cuda_stream
        hm.mxfp8_quantize(w.data_ptr(), hm.HM_F32, n, d, d, 0, 0, 32, qw.data_ptr(), d, sw.data_ptr(), 0, 0, 0, st)
        hm.rmsnorm_mxfp8(x.data_ptr(), d, 0, 0, 0, hm.HM_BF16, rows, d, gamma.data_ptr(), 1e-5, 32, rstd.data_ptr(),
                         q.data_ptr(), s.data_ptr(), st)
        hm.mxfp8_gemm(q.data_ptr(), d, s.data_ptr(), qw.data_ptr(), d, sw.data_ptr(), rows, n, d, out.data_ptr(), n,
                      hm.HM_F32, False, st)
        hm.rmsnorm_backward(out.data_ptr(), n, 0, x32.data_ptr(), dx.data_ptr(), d, hm.HM_F32, rows, d, gamma.data_ptr(),
                            rstd.data_ptr(), dg.data_ptr(), False, gws.data_ptr(), gws.numel(), st)
        hm.grad_norm_clip(lst, 1e-3, 1e-6, stats.data_ptr(), ws.data_ptr(), ws.numel(), st)

    def feed():
        x.copy_(torch.randn(rows, d, generator=g, device=dev))
        x32.copy_(x)
        w.normal_(generator=g)
        gamma.copy_(1 + 0.1 * torch.randn(d, generator=g, device=dev))

    def poison():
        for t in outputs:
            t.view(torch.uint8).fill_(0x5A)

    feed()
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        feed()
        poison()
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in outputs]
        poison()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outputs, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
            assert not bool((a.view(torch.uint8) == 0x5A).all())
        assert torch.isfinite(out).all() and 0 < float(stats[1]) < 1
    assert hm.hm_device_error() == 0
