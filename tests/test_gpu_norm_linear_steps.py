"""NormLinear over several micro-batches per step."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev(hm):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def test_micro_batches_add_up_and_are_clipped_by_their_sum(hm, dev):
    """Two micro-batches: dW and dgamma are the sums of the two passes' own, the step's norm is
    that of the sums, and the next step starts from nothing.  The sums are fp32: the two
    terms' and their sum's roundings, 2^-22 of the terms' size; the norm over 49,408
    elements 128 2^-24 as the clipping's own tests derive, and the sums' 2^-22."""
    from head_muon_mxfp8_gb300.linear import NormLinear
    tokens, d_in, d_out = 96, 256, 192
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    batches = [(rand(tokens, d_in).bfloat16(), rand(tokens, d_out).bfloat16()) for _ in range(2)]
    layer = NormLinear(tokens, d_in, d_out)
    layer.load_weight(rand(d_out, d_in) * d_in ** -0.5)
    alone = []
    for x, dy in batches:
        layer.zero_grad()
        layer.forward(x)
        layer.backward(dy)
        alone.append((layer.g.double().clone(), layer.dgamma.double().clone()))
    layer.zero_grad()
    for x, dy in batches:
        layer.forward(x)
        layer.backward(dy)
    for got, (a, b) in zip((layer.g, layer.dgamma), zip(*alone)):
        assert bool(((got.double() - (a + b)).abs() <= 2.0 ** -22 * (a.abs() + b.abs())).all())
    norm = float(torch.sqrt(sum((a + b).square().sum() for a, b in zip(*alone))))
    hp = hm.hm_muon_hparams(0.01, 0.9, 0.0, 1e-7, 3.4445, -4.7750, 2.0315, 5, 1, 0)
    dgamma = layer.dgamma.clone()
    stats = layer.step(hp, max_norm=0.5 * norm).cpu()
    assert abs(float(stats[0]) - norm) <= (128 * 2.0 ** -24 + 2.0 ** -22) * norm
    assert abs(float(stats[1]) - 0.5) < 1e-4
    assert torch.equal(layer.dgamma, dgamma * stats[1].to(dev))      # clipped, still readable
    assert not layer.g.any()
    x, dy = batches[0]
    layer.forward(x)
    layer.backward(dy)
    after = layer.dgamma.clone()
    layer.zero_grad()
    layer.forward(x)
    layer.backward(dy)
    assert torch.equal(after, layer.dgamma)                          # the step had cleared it too
    layer.close()
    assert hm.hm_device_error() == 0
