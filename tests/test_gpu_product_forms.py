"""Every kernel form of the product, each named by the shape's own dispatch: the CTA-pair
kernel at its three widths, with and without the sums of K's chunks in registers,
stored and added to fp32 (the weight gradient), and the cluster kernel at 128
rows.  If a change of the dispatch moves a shape, its case fails rather than
testing another kernel twice.

Tolerance (by derivation, u = 2^-24): (K / 32 + 33) 2u sum |a b| for the chain of
tensor-core additions (one unit in the last place of the running sum per step, and
one of the largest of a step's 32 addends), 2u |D| for the earlier D's addition, a
bf16 result half of its unit, 2^-8 |D|."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def dev(hm):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def _up(x, k):
    return -(-x // k) * k


def _operand(g, dev, rows, k, block):
    """Codes (no NaN), tiled scales with NaN in their padding, and the values in 64 bits."""
    codes = torch.randint(0, 256, (rows, k), generator=g, device=dev, dtype=torch.uint8)
    codes[codes & 0x7F == 0x7F] = 0x10
    per = block // 32
    sf = torch.randint(120, 131, (rows, _up(k // 32, per) // per), generator=g, device=dev, dtype=torch.uint8)
    sf = sf.repeat_interleave(per, dim=1)[:, :k // 32]
    full = torch.full((_up(rows, 128), _up(k // 32, 4)), 0xFF, dtype=torch.uint8, device=dev)
    full[:rows, :k // 32] = sf
    tiled = full.view(-1, 4, 32, full.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).contiguous()
    val = codes.view(torch.float8_e4m3fn).double().view(rows, -1, 32) * torch.exp2(sf.double() - 127)[:, :, None]
    return codes, tiled, val.view(rows, k)


FORMS = [
    # m, n, k, D, accumulate, block, ldd - n, (tile, parts, sums)
    (2311, 6403, 1056, "f32", True, 32, 5, (256, 0, 0)),     # several tiles per pair, tails in m, n and k, odd pitch
    (2304, 3264, 1056, "f32", True, 128, 0, (256, 0, 0)),
    (1541, 9231, 224, "f32", False, 128, 1, (256, 0, 0)),
    (1030, 6403, 1056, "bf16", False, 128, 3, (256, 0, 0)),
    (130, 9731, 928, "bf16", False, 32, 0, (192, 0, 0)),
    (130, 9731, 928, "f32", True, 128, 1, (192, 0, 0)),
    (2311, 6403, 2208, "f32", True, 128, 1, (192, 0, 1)),    # several tiles per pair, two chunks each
    (1030, 6403, 2208, "f32", True, 32, 6, (192, 0, 1)),
    (1700, 1900, 2080, "f32", False, 32, 0, (192, 0, 1)),
    (617, 9731, 2080, "f32", True, 32, 3, (128, 0, 1)),
    (1541, 4099, 2080, "f32", False, 128, 0, (128, 0, 1)),
    (131, 400, 21024, "f32", True, 32, 0, (128, 0, 1)),      # eleven chunks, the last one short
    (5, 300, 24576, "f32", True, 128, 1, (128, 0, 1)),
    (1000, 2299, 6432, "bf16", False, 32, 2, (128, 0, 0)),
    (515, 1030, 4128, "f32", True, 32, 1, (128, 6, 0)),
    (600, 700, 96, "f32", True, 128, 0, (128, 1, 0)),
    (1900, 2560, 160, "bf16", False, 32, 0, (128, 1, 0)),
]


@pytest.mark.parametrize("m,n,k,out,acc,block,pad,form", FORMS)
def test_product_form(hm, dev, m, n, k, out, acc, block, pad, form):
    g = torch.Generator(device=dev)
    g.manual_seed(m + n + k)
    qa, ta, va = _operand(g, dev, m, k, block)
    qb, tb, vb = _operand(g, dev, n, k, block)
    ref, bound = va @ vb.t(), va.abs() @ vb.abs().t()
    dt, code = (torch.bfloat16, hm.HM_BF16) if out == "bf16" else (torch.float32, hm.HM_F32)
    assert hm.mxfp8_gemm_form(m, n, k, code) == form
    start = torch.full((m + 1, n + pad), 7.0, dtype=dt, device=dev)
    if acc:
        start[:m, :n] = torch.randn(m, n, generator=g, device=dev) * ref.abs().mean()
        ref = ref + start[:m, :n].double()
    runs = []
    for _ in range(2):
        d = start.clone()
        hm.mxfp8_gemm(qa.data_ptr(), k, ta.data_ptr(), qb.data_ptr(), k, tb.data_ptr(), m, n, k, d.data_ptr(), n + pad,
                      code, acc, torch.cuda.current_stream().cuda_stream)
        runs.append(d)
    torch.cuda.synchronize()
    assert hm.hm_device_error() == 0
    d = runs[0]
    tol = (k / 32 + 33) * 2 * U * bound
    if acc:
        tol = tol + 2 * U * ref.abs()
    if out == "bf16":
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs()
    assert bool(((d[:m, :n].double() - ref).abs() <= tol).all())
    assert bool((d[m:] == 7.0).all()) and bool((d[:, n:] == 7.0).all())    # nothing outside m x n is written
    assert torch.equal(runs[0], runs[1])                                   # the same bits every time


def test_every_pair_form_is_covered():
    """The instances that launch_mx_gemm names, and nothing else, appear above."""
    import os
    import re
    src = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "head_muon_mxfp8_gb300", "csrc",
                       "hm_mxgemm.cu")
    named = {(int(b), s == "true") for b, s in re.findall(r"launch_pair<(\d+), (true|false)>\(a", open(src).read())}
    assert named == {(t, bool(s)) for *_, (t, parts, s) in FORMS if not parts}
