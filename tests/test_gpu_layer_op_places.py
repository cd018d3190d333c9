"""Outputs in an input's place, the ways that the header allows and other tests do not take: the
gradient of heads over x, and both of a gated pair's gradients crosswise over gate and up, in
every kind of kernel.  The bits of separate outputs."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev(hm):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


@pytest.mark.parametrize("dtype,rows,dim,rot,pairs", [("bf16", 3000, 128, 128, False), ("f32", 37, 80, 24, True), ("bf16", 500, 72, 18, False)])
def test_heads_gradient_over_x(hm, dev, dtype, rows, dim, rot, pairs):
    dt, code = (torch.bfloat16, hm.HM_BF16) if dtype == "bf16" else (torch.float32, hm.HM_F32)
    g = torch.Generator(device=dev)
    g.manual_seed(rows)
    new = lambda: torch.randn(rows, 7, dim, generator=g, device=dev).to(dt)  # noqa: E731
    x, dy, dx = new(), new(), new()
    gamma = torch.rand(dim, generator=g, device=dev) + 0.5
    pos = torch.randint(0, 5000, (rows,), generator=g, device=dev)
    turns, _ = hm.rope_turns(rot)
    table = torch.tensor(turns, dtype=torch.int64, device=dev)
    rotation = hm.hm_rotation(table.data_ptr(), pos.data_ptr(), 1.0, rot, hm.HM_ROPE_PAIRS if pairs else hm.HM_ROPE_HALF)
    at = lambda t, h: (t.data_ptr() + h * dim * t.element_size(), 7 * dim, dim)  # noqa: E731

    def run(to):
        dg = torch.zeros(2, dim, device=dev)
        lst = hm.head_grad_list([(*at(dy, h), *at(x, h), *at(to, h), gamma.data_ptr(), dg[i].data_ptr(), n, False)
                                 for i, (h, n) in enumerate(((0, 5), (5, 2)))])
        ws = torch.empty(hm.head_norm_rope_backward_workspace(lst, rows, dim), dtype=torch.uint8, device=dev)
        hm.head_norm_rope_backward(lst, code, rows, dim, 1e-5, rotation, ws.data_ptr(), ws.numel())
        return dg

    first = run(dx)
    second = run(x)
    assert torch.equal(x, dx) and torch.equal(first, second)


@pytest.mark.parametrize("dtype,m,n,k", [("bf16", 1, 300, 512), ("bf16", 150, 384, 4096), ("bf16", 2311, 1400, 288), ("f32", 33, 256, 2080),
                                         ("f32", 2311, 1400, 2080), ("f32", 2311, 1400, 288), ("bf16", 9, 40, 0)])
@pytest.mark.parametrize("pad", [0, 3])
def test_gated_gradients_crosswise(hm, dev, dtype, m, n, k, pad):
    dt, code = (torch.bfloat16, hm.HM_BF16) if dtype == "bf16" else (torch.float32, hm.HM_F32)
    g = torch.Generator(device=dev)
    g.manual_seed(m + n)
    ld = n + pad
    operand = lambda rows: torch.randint(0, 0x60, (rows, max(k, 32)), generator=g, device=dev, dtype=torch.uint8)  # noqa: E731
    a, b = operand(m), operand(n)
    sa, sb = (torch.full((hm.mxfp8_tiled_scale_bytes(r, max(k, 32)),), 118, dtype=torch.uint8, device=dev) for r in (m, n))
    gate, up = (torch.randn(m, ld, generator=g, device=dev).to(dt) for _ in range(2))
    p = lambda t: t.data_ptr()  # noqa: E731

    def run(d, out2):
        e = hm.hm_epilogue(hm.HM_EPI_GATED_GRADIENT, hm.HM_ACT_GELU, 0, p(gate), ld, p(up), ld, p(out2), ld)
        hm.mxfp8_gemm_epilogue(p(a), k, p(sa), p(b), k, p(sb), m, n, k, p(d), ld, code, e)

    d, out2 = gate.clone(), up.clone()
    run(d, out2)
    gate0, up0 = gate.clone(), up.clone()
    run(gate, up)                       # d over the gate, out2 over up
    assert torch.equal(gate[:, :n], d[:, :n]) and torch.equal(up[:, :n], out2[:, :n])
    gate.copy_(gate0)
    up.copy_(up0)
    run(up, gate)                       # and the other way round
    assert torch.equal(up[:, :n], d[:, :n]) and torch.equal(gate[:, :n], out2[:, :n])
    assert torch.equal(gate[:, n:], gate0[:, n:]) and torch.equal(up[:, n:], up0[:, n:])
    assert hm.hm_device_error() == 0
