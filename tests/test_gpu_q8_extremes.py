"""q8_matmul at the ends of the scales' range: a result that its type holds is
returned even where the sum times one scale alone would be past fp32's range.
The bound is that of test_gpu_q8.py, the rounding of the sum, of two products
and of the output: a factor of a power of two rounds nothing."""
import pytest
import torch

import newton_schulz_04_amd as ns
from test_gpu_q8 import BF16, FP32, check, gen, matmul_bound, product_of, q8_matrix

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ns.lib()


# few tokens; small tiles, whole and in pieces; large tiles
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("t,o,k", [(1, 33, 65), (20, 130, 6144), (70, 96, 200), (64, 64, 8192), (2100, 2064, 1030)])
def test_matmul_of_huge_and_tiny_scales(t, o, k, dtype):
    g = gen(t + o + k)
    x, w = q8_matrix(t, k, g), q8_matrix(o, k, g)
    exponents = torch.tensor([120.0, 100.0, 60.0, 0.0, -60.0, -100.0, -120.0], device="cuda")
    for start in range(7):
        for m, at in ((x, start), (w, 0)):
            n = m[1].numel()
            power = exponents[(torch.arange(n, device="cuda") + at) % 7]
            m[1].copy_(torch.exp2(power) * (1 + torch.rand(n, generator=g, device="cuda")))
        y, = ns.q8_matmul([x], [w], dtype=dtype)
        ref = product_of(x, w)
        assert bool(torch.isinf(y[ref.abs() > 2.0 ** 128.1]).all())
        fine = (ref.abs() < 2.0 ** 127.9) & ((ref.abs() > 2.0 ** -120) | (ref == 0))
        assert bool(fine.any())
        zero = torch.zeros_like(ref)
        check(torch.where(fine, y.double(), zero), torch.where(fine, ref, zero), matmul_bound(ref, dtype).nan_to_num())
