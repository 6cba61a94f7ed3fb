"""8-bit outputs that are small in their group, or small altogether: their codes are those of the 64-bit values."""
import pytest
import torch

import layer_reference as ref
from gated_deltanet_recurrence_gdn_amd import binding as gb
from helpers import DEV
from test_gpu_norm import T, codes_for, normal

pytestmark = pytest.mark.gpu
EXACT = 2.0 ** -40  # what float64 may lose here, far above it, and far below an fp32 step


def halfway(seed, *shape):
    """Values halfway between two e4m3 codes: steps of 2^-9 below 2^-6, and ordinary ones up to 2^-3."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    k = torch.randint(0, 16, shape, generator=g, device=DEV).double() + 0.5
    up = torch.randint(0, 4, shape, generator=g, device=DEV).double()
    return k * 2.0 ** -9 * torch.exp2(torch.where(k >= 8, up, 0))


@pytest.mark.parametrize("width", [128, 200, 1000, 2048, 5120, 16384])
def test_norm_next_to_halves(width):
    """One channel of a group is 300 times a power of two, so that the scale is that power; the weights bring the others
    as near to a half as fp32 comes, where results in fp32 fall to either side."""
    for seed, power in enumerate([0, 40, -40]):
        x = normal(seed, 1, width)
        n = x.double() * (1 / torch.sqrt(x.double().square().mean()))
        y = halfway(seed, width)
        y[::128] = 300.0
        w = (torch.ldexp(y, torch.tensor(power, device=DEV)) / n[0]).float()
        codes, scales = codes_for(1, width)
        gb.gdn_norm_forward(x, w, codes=codes, scales=scales, eps=0.0)
        y, _ = ref.norm(x, w, 0.0)
        ref.check_codes(y, codes, scales, EXACT)


@pytest.mark.parametrize("heads,d", [(3, 16), (2, 64), (1, 48), (48, 128), (2, 96), (3, 256)])
def test_gated_norm_next_to_halves(heads, d):
    """The same by the gates: z with silu(z) = y / (n w), by bisection in float64."""
    rows = 100
    x, w = normal(d, rows, heads, d), 1 + 0.1 * normal(1, d)
    n = x.double() / torch.sqrt(x.double().square().mean(-1, keepdim=True))
    y = halfway(d, rows, heads * d)
    y[:, ::128] = 300.0
    want = y.reshape(rows, heads, d) / (n * w.double()).abs()
    low, high = torch.zeros_like(want), torch.full_like(want, 1e9)
    for _ in range(100):
        z = (low + high) / 2
        over = z * torch.sigmoid(z) > want
        low, high = torch.where(over, low, z), torch.where(over, z, high)
    z = high.float()
    codes, scales = codes_for(rows, heads * d)
    gb.gdn_gated_norm_forward(x, z, w, codes=codes, scales=scales, eps=0.0)
    y, _ = ref.gated(x, z, w, 0.0)
    ref.check_codes(y.reshape(rows, -1), codes, scales, EXACT)


@pytest.mark.parametrize("width", [128, 200, 2048, 5120, 16384])
def test_norm_below_fp32(width):
    """Results below 2^-126, where fp32 has fewer bits."""
    rows = 2000000 // width
    x = normal(1, rows, width)
    w = torch.ldexp(1 + 0.1 * normal(2, width), -118 - torch.arange(width, device=DEV) // 128 % 16)
    codes, scales = codes_for(rows, width)
    gb.gdn_norm_forward(x, w, codes=codes, scales=scales, eps=0.0)
    ref.check_codes(ref.norm(x, w, 0.0)[0], codes, scales, EXACT)


@pytest.mark.parametrize("heads,d", [(3, 16), (2, 64), (1, 48), (48, 128), (2, 96), (3, 256)])
@pytest.mark.parametrize("weight", [0, 30])
def test_gated_norm_below_fp32(heads, d, weight):
    """Gates whose silu is about 2^-118 to 2^-140, by weights about 1 and 2^30."""
    rows = 2000000 // (heads * d)
    x, w = normal(d, rows, heads, d), torch.ldexp(1 + 0.1 * normal(1, d), torch.tensor(weight, device=DEV))
    z = -(86 + 17 * torch.rand(rows, 1, 1, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV)) + 0.5 * normal(4, rows, heads, d)
    codes, scales = codes_for(rows, heads * d)
    gb.gdn_gated_norm_forward(x, z, w, codes=codes, scales=scales, eps=0.0)
    y, _ = ref.gated(x, z, w, 0.0)
    ref.check_codes(y.reshape(rows, -1), codes, scales, EXACT)


@pytest.mark.parametrize("width", [200, 2048, 5120])
def test_zero_rows_beside_small_ones(width):
    x, w = normal(1, 9, width), torch.full((width,), 2.0 ** -130, device=DEV)
    x[::2] = 0
    codes, scales = codes_for(9, width)
    gb.gdn_norm_forward(x, w, codes=codes, scales=scales, eps=1e-6)
    ref.check_codes(ref.norm(x, w, 1e-6)[0], codes, scales, EXACT)
    assert not codes[::2].float().any()
