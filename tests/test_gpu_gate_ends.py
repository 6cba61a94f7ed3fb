"""Gates up to their types' largest value: silu(z) is z there, and nothing finite becomes NaN."""
import pytest
import torch

import layer_reference as ref
from gated_deltanet_recurrence_gdn_amd import binding as gb
from helpers import DEV
from test_gpu_norm import EPS, T, codes_for, like, normal

pytestmark = pytest.mark.gpu


def gates(z, seed, *shape):
    """Around 2.36e38, above which z log2(e) leaves fp32's range, the type's largest, and ordinary ones."""
    ends = [3e38, 2.4e38, 2.36e38, 2.3e38, 1e38, 1e30, 1e5, 200.0, 128.0, 104.0, 89.0, 1.0, -1.0]
    far = [torch.finfo(T[z]).max] + [e for e in ends if e < torch.finfo(T[z]).max]
    n = torch.Size(shape).numel()
    order = torch.randperm(n, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)
    return torch.tensor(far, device=DEV).repeat(n // len(far) + 1)[:n][order].reshape(shape).to(T[z])


@pytest.mark.parametrize("heads,d", [(3, 16), (2, 64), (1, 48), (5, 128), (2, 96), (3, 256)])
@pytest.mark.parametrize("z", ["f32", "bf16", "f16"])
def test_largest_gates(heads, d, z):
    rows = 7
    # weights and gradients small enough that products and their sums stay finite
    x, zs, w = normal(d, rows, heads, d), gates(z, d, rows, heads, d), 2.0 ** -10 * (1 + 0.1 * normal(1, d))
    out, (codes, scales) = like(zs), codes_for(rows, heads * d)
    gb.gdn_gated_norm_forward(x, zs, w, out=out, codes=codes, scales=scales, eps=EPS)
    y, _ = ref.gated(x, zs, w, EPS)
    ref.near(out, y, y.abs() * ref.GATED)
    ref.check_codes(y.flatten(1), codes, scales, ref.GATED)
    dout = (2.0 ** -10 * normal(4, rows, heads, d)).to(T[z])
    dx, dz, dw = like(x), like(zs), torch.empty(d, device=DEV)
    gb.gdn_gated_norm_backward(dout, x, zs, w, dx, dz, dw, eps=EPS)
    want, lost, want_z, lost_z, want_w, lost_w = ref.gated_gradients(dout, x, zs, w, EPS)
    ref.near(dx, want, lost)
    # a is 1 in fp32 from z = 18 on, so what is lost of 1 - a is below z e^-z: nothing of the gradient from 104 on
    far = zs.float() >= 104
    ref.near(dz[far], want_z[far], want_z[far].abs() * (ref.HEAD + ref.GATE + 8 * ref.U))
    ref.near(dz[~far], want_z[~far], lost_z[~far])
    ref.near(dw, want_w, lost_w)


@pytest.mark.parametrize("heads,d", [(2, 64), (1, 48)])
def test_infinite_gates(heads, d):
    """silu of +infinity is +infinity: the element's own result only."""
    x, z, w = normal(d, 2, heads, d), normal(2, 2, heads, d), 1 + 0.1 * normal(1, d)
    z[0, 0, 5] = float("inf")
    out = like(z)
    gb.gdn_gated_norm_forward(x, z, w, out=out, eps=EPS)
    y, _ = ref.gated(x, z, w, EPS)
    assert out[0, 0, 5] == y[0, 0, 5] and out[0, 0, 5].isinf()
    fine = z.isfinite()
    ref.near(out[fine], y[fine], y[fine].abs() * ref.GATED)


@pytest.mark.parametrize("heads,d", [(3, 16), (2, 64), (1, 48), (5, 128), (2, 96), (3, 256)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_of_closed_gates(heads, d, dtype):
    """Gates below e^-86, which have few bits in fp32 or none, and gradients of 2^80, which bring them back."""
    rows = 40
    x, w = normal(d, rows, heads, d).to(T[dtype]), 1 + 0.1 * normal(1, d)
    z = -(60 + 70 * torch.rand(rows, heads, d, generator=torch.Generator(device=DEV).manual_seed(d), device=DEV)).to(T[dtype])
    dout = torch.ldexp(normal(4, rows, heads, d), torch.tensor(80, device=DEV)).to(T[dtype])
    dx, dz, dw = like(x), like(z), torch.empty(d, device=DEV)
    gb.gdn_gated_norm_backward(dout, x, z, w, dx, dz, dw, eps=EPS)
    want, lost, want_z, lost_z, want_w, lost_w = ref.gated_gradients(dout, x, z, w, EPS)
    ref.near(dx, want, lost)
    # 1 - a is 1 in fp32 here, so 1 + z (1 - a) is rounded once
    ref.near(dz, want_z, want_z.abs() * (ref.HEAD + ref.GATE + 8 * ref.U))
    ref.near(dw, want_w, lost_w)
    for b in range(rows):  # rows whose gates are all closed: as near in their own size
        one = [t[b:b + 1].clone() for t in (dout, x, z)]
        one[2] = one[2].clamp(max=-90)
        dx, dz = like(one[1]), like(one[2])
        gb.gdn_gated_norm_backward(*one, w, dx, dz, eps=EPS)
        want, lost, want_z, _, _, _ = ref.gated_gradients(*one, w, EPS)
        ref.near(dx, want, lost)
        ref.near(dz, want_z, want_z.abs() * (ref.HEAD + ref.GATE + 8 * ref.U))
