"""Rows of fp32 and bf16 subnormals with eps = 0: their inverse root is above fp32's range, their results are not."""
import pytest
import torch

import layer_reference as ref
from gated_deltanet_recurrence_gdn_amd import binding as gb
from helpers import DEV
from test_gpu_norm import T, codes_for, like, normal

pytestmark = pytest.mark.gpu
POWERS = {"f32": [-135, 0, -128, -143, -127, -130, -20], "bf16": [-130, 0, -128, -131, -127, -126, -20]}


def rows_of(seed, dtype, *shape):
    """Rows from one power to the next of ordinary and subnormal magnitude, with zeros among their elements."""
    power = torch.tensor(POWERS[dtype], device=DEV)[torch.arange(shape[0], device=DEV) % 7].reshape(-1, *[1] * (len(shape) - 1))
    x = normal(seed, *shape)
    x.flatten(1)[:, ::5] = 0
    x.flatten(1)[:, 1::16] = 1  # no row of zeros
    return torch.ldexp(torch.ldexp(x, power // 2), power - power // 2).to(T[dtype])


# 16 lanes a row, a wave, a workgroup with one, two and four vectors a lane
@pytest.mark.parametrize("width", [16, 200, 256, 264, 2048, 2560, 5120, 16000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm(width, dtype):
    x, w = rows_of(width, dtype, 37, width), 1 + 0.1 * normal(1, width)
    y, _ = ref.norm(x, w, 0.0)
    assert y.isfinite().all()
    plain = like(x)
    gb.gdn_norm_forward(x, w, out=plain, eps=0.0)
    ref.near(plain, y, y.abs() * ref.NORM)
    out, (codes, scales) = like(x), codes_for(37, width)
    gb.gdn_norm_forward(x, w, out=out, codes=codes, scales=scales, eps=0.0)
    ref.near(out, y, y.abs() * ref.NORM)
    ref.check_codes(y, codes, scales, ref.NORM)


@pytest.mark.parametrize("width", [16, 264, 2048, 2560, 5120, 16000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_gradients(width, dtype):
    rows = 1500
    r, w = rows_of(width, dtype, rows, width), 1 + 0.1 * normal(1, width)
    dout = (2.0 ** -30 * normal(2, rows, width)).to(T[dtype])  # dx is about 2^113 at the most
    dx, dw = like(r), torch.empty(width, device=DEV)
    gb.gdn_norm_backward(dout, r, w, dx, dw, eps=0.0)
    want, lost, want_w, lost_w = ref.norm_gradients(dout, r, w, 0.0)
    ref.near(dx, want, lost)
    ref.near(dw, want_w, lost_w)


@pytest.mark.parametrize("heads,d", [(3, 16), (2, 64), (1, 48), (5, 128), (2, 96), (3, 256)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gated_norm(heads, d, dtype):
    rows = 1001
    x = rows_of(d, dtype, rows * heads, d).reshape(rows, heads, d)
    z, w = normal(3, rows, heads, d).to(T[dtype]), 1 + 0.1 * normal(1, d)
    y, _ = ref.gated(x, z, w, 0.0)
    plain = like(z)
    gb.gdn_gated_norm_forward(x, z, w, out=plain, eps=0.0)
    ref.near(plain, y, y.abs() * ref.GATED)
    out, (codes, scales) = like(z), codes_for(rows, heads * d)
    gb.gdn_gated_norm_forward(x, z, w, out=out, codes=codes, scales=scales, eps=0.0)
    ref.near(out, y, y.abs() * ref.GATED)
    ref.check_codes(y.flatten(1), codes, scales, ref.GATED)
    dout = (2.0 ** -30 * normal(4, rows, heads, d)).to(T[dtype])
    dx, dz, dw = like(x), like(z), torch.empty(d, device=DEV)
    gb.gdn_gated_norm_backward(dout, x, z, w, dx, dz, dw, eps=0.0)
    want, lost, want_z, lost_z, want_w, lost_w = ref.gated_gradients(dout, x, z, w, 0.0)
    ref.near(dx, want, lost)
    ref.near(dz, want_z, lost_z)
    ref.near(dw, want_w, lost_w)
