"""State rows in 8 bits at the ends of fp32: channels up to the largest value, and of the smallest scales."""
import numpy as np
import pytest
import torch

import layer_reference as ref
from gated_deltanet_recurrence_gdn_amd import binding as gb
from helpers import DEV

pytestmark = pytest.mark.gpu


def ints(*x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device=DEV)


def round_trip(x):
    codes, scales = torch.zeros(x.shape, dtype=torch.int8, device=DEV), torch.zeros(x.shape[:-1], device=DEV)
    back, rows = torch.zeros_like(x), ints(*range(x.shape[1]))
    gb.gdn_pool_pack(x, codes, scales, rows, rows)
    gb.gdn_pool_unpack(codes, scales, back, rows, rows)
    return codes, scales, back


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dk", [32, 64, 128])
def test_largest_values(dk, dtype):
    """Channels saturated to the type's largest value, and the next ones below, read back finite and within half a step."""
    x = torch.randn(1, 1, 2, 16, dk, generator=torch.Generator(device=DEV).manual_seed(dk), device=DEV)
    x = (x / x.abs().amax()).double() * torch.finfo(dtype).max * 0.99
    x = x.to(dtype)
    top = torch.full((16,), torch.finfo(dtype).max, dtype=dtype, device=DEV)
    bits = top.view(torch.int32 if dtype is torch.float32 else torch.int16)
    x[0, 0, 0, :, 3] = (bits - torch.arange(16, device=DEV).to(bits.dtype)).view(dtype)
    x[0, 0, 1, :, dk - 1] = -x[0, 0, 0, :, 3]
    codes, scales, back = round_trip(x)
    assert scales.isfinite().all() and back.isfinite().all()
    step = scales.double()[..., None]
    value = codes.double() * step
    # half a step, by a quotient that is rounded once; then the product's rounding and the store's
    assert torch.all((value - x.double()).abs() <= step / 2 * (1 + 2 ** -23))
    ref.near(back, value, value.abs() * ref.U)
    assert torch.all(codes.abs().amax(-1) == 127)
    # the scale is the definition's but where 127 of it would pass fp32's range: the next one down there
    want = ref.pack(x)[1]
    over = (127 * want).isinf()
    assert torch.equal(torch.where(over, torch.nextafter(want, torch.zeros_like(want)), want), scales)
    assert int(over.sum()) == (2 if dtype is torch.float32 else 0)


def test_halves_of_the_smallest_scales():
    """Scales from 2^-126 to 2^-125 with an odd last bit, whose half is no fp32 value: states beside each half of a step."""
    dv, dk = 64, 128
    unit = torch.tensor(-149, device=DEV)
    # the scales in steps of 2^-149, and largest values whose quotient by 127 is the scale
    mantissa = 2 ** 23 + 2 * torch.randint(0, 2 ** 21, (4 * dv,), generator=torch.Generator().manual_seed(7)).to(DEV) + 1
    tops = torch.ldexp((127 * mantissa).double(), unit).float()
    kept = torch.ldexp((tops.double() / 127).float().double(), -unit) == mantissa
    mantissa, tops = mantissa[kept][:dv], tops[kept][:dv]
    x = torch.zeros(1, 2, 1, dv, dk, device=DEV)
    k = torch.arange(dk, device=DEV) - 64
    for row, side in enumerate((0, 1)):  # the steps of 2^-149 below and above the half
        steps = ((2 * k + 1) * mantissa[:, None]) // 2 + side
        x[0, row, 0] = torch.ldexp(steps.double(), unit).float()
    x[..., 0] = tops
    codes, scales, back = round_trip(x)
    want_c, want_s = ref.pack(x)
    assert torch.equal(scales, want_s) and torch.all((scales.view(torch.int32) & 1) == 1)
    assert torch.equal(codes, want_c)
