"""Gradients so large that dout w r, whose mean dx needs, is above fp32's range, where dx is not."""
import pytest
import torch

import layer_reference as ref
from gated_deltanet_recurrence_gdn_amd import binding as gb
from helpers import DEV
from test_gpu_norm import EPS, T, like, normal

pytestmark = pytest.mark.gpu
# powers of dout and r in rows next to one another: products of up to 2^208, dx from 2^-20 to 2^100
POWERS = [(0, 0), (100, 0), (100, 28), (80, 50), (0, 0), (90, 118), (20, 120), (100, 5), (-20, 0), (60, 70)]


def rows_of(seed, dtype, *shape):
    """dout and r; exact powers of two, in two steps that stay in range."""
    at = torch.arange(shape[0], device=DEV) % len(POWERS)
    out = []
    for i in (0, 1):
        p = torch.tensor([x[i] for x in POWERS], device=DEV)[at].reshape(-1, *[1] * (len(shape) - 1))
        out.append(torch.ldexp(torch.ldexp(normal(seed + i, *shape), p // 2), p - p // 2).to(T[dtype]))
    return out


@pytest.mark.parametrize("width", [8, 264, 2048, 2560, 5120, 16000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm(width, dtype):
    (dout, r), w = rows_of(width, dtype, 1500, width), 1 + 0.1 * normal(1, width)
    dx, dw = like(r), torch.empty(width, device=DEV)
    gb.gdn_norm_backward(dout, r, w, dx, dw, eps=EPS)
    want, lost, want_w, lost_w = ref.norm_gradients(dout, r, w, EPS)
    ref.near(dx, want, lost)
    ref.near(dw, want_w, lost_w)


@pytest.mark.parametrize("heads,d", [(3, 16), (2, 64), (1, 48), (5, 128), (2, 96), (3, 256)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gated_norm(heads, d, dtype):
    rows = 500
    dout, x = (t.reshape(rows, heads, d) for t in rows_of(d, dtype, rows * heads, d))
    z, w = normal(3, rows, heads, d).to(T[dtype]), 1 + 0.1 * normal(1, d)
    dx, dz, dw = like(x), like(z), torch.empty(d, device=DEV)
    gb.gdn_gated_norm_backward(dout, x, z, w, dx, dz, dw, eps=EPS)
    want, lost, want_z, lost_z, want_w, lost_w = ref.gated_gradients(dout, x, z, w, EPS)
    ref.near(dx, want, lost)
    ref.near(dz, want_z, lost_z)
    ref.near(dw, want_w, lost_w)
