"""How many launches clipping takes at the edges of its one-launch form (16 tensors that are not
empty, 64 chunks of 1024 16-byte vectors, so 1 MB), and that the result does not
depend on it."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
VEC = {"f32": 4, "bf16": 8}   # elements of a 16-byte vector


@pytest.fixture(scope="module")
def dev(hm):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("chunks,tail,lead,launches", [
    (64, 0, 0, 1),     # exactly full
    (64, -1, 0, 1),    # the last vector incomplete
    (64, 1, 0, 2),     # one vector more is one chunk more
    (64, 0, 1, 1),     # off the vector boundary: the ends are outside the vectors
    (64, 2, 1, 2),
    (1, 0, 0, 1),
])
def test_launches_of_one_tensor(hm, dev, dtype, chunks, tail, lead, launches):
    v = VEC[dtype]
    dt, code = (torch.float32, hm.HM_F32) if dtype == "f32" else (torch.bfloat16, hm.HM_BF16)
    n = chunks * 1024 * v + tail * v - (1 if tail < 0 else 0)
    flat = torch.randn(n + lead, device=dev).to(dt)
    _check(hm, dev, [flat[lead:]], code, launches)


@pytest.mark.parametrize("count,empty,launches", [(16, 0, 1), (16, 30, 1), (17, 0, 2), (256, 5, 2), (257, 0, 4), (0, 3, 1)])
def test_launches_of_many_tensors(hm, dev, count, empty, launches):
    grads = [torch.randn(100 + 7 * i, device=dev) for i in range(count)]
    grads += [torch.zeros(0, device=dev)] * empty
    _check(hm, dev, grads, hm.HM_F32, launches)


def _check(hm, dev, grads, code, launches):
    outs = [torch.full_like(g, 3.0) for g in grads]
    lst = hm.grad_list([(g.data_ptr(), o.data_ptr(), g.numel(), code) for g, o in zip(grads, outs)])
    ws = torch.empty(hm.grad_norm_clip_workspace(lst) + 16, dtype=torch.uint8, device=dev)
    stats = torch.zeros(2, device=dev)
    norm = float(torch.sqrt(sum((g.double().square().sum() for g in grads), torch.zeros((), dtype=torch.float64, device=dev))))
    before = hm.hm_kernel_launches()
    hm.grad_norm_clip(lst, max(norm, 1.0) * 0.5, 1e-6, stats.data_ptr(), ws.data_ptr(), ws.numel())
    assert hm.hm_kernel_launches() - before == launches
    torch.cuda.synchronize()
    assert abs(float(stats[0]) - norm) <= 128 * U * norm
    coef = stats[1]
    for g, o in zip(grads, outs):
        assert torch.equal(o, (g.float() * coef).to(g.dtype))
