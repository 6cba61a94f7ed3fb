"""The norms over the whole range of their types: rows whose squares leave fp32's range, gates at a type's ends."""
import pytest
import torch

import layer_reference as ref
from gated_deltanet_recurrence_gdn_amd import binding as gb
from helpers import DEV

pytestmark = pytest.mark.gpu
T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
POWERS = [120, 0, -120, 63, 64, -50, 100, -63, -100, 56, -14, 20]  # of the rows' magnitudes, next to one another


def normal(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)


def rows_of(seed, *shape):
    power = torch.tensor(POWERS, device=DEV)[torch.arange(shape[0], device=DEV) % len(POWERS)]
    return torch.ldexp(normal(seed, *shape), power.reshape(-1, *[1] * (len(shape) - 1)))


def codes_for(rows, width):
    codes = torch.empty(rows, width, dtype=torch.float8_e4m3fn, device=DEV)
    return codes, gb.gdn_scales_like(codes)


# 16 lanes a row, a wave, a workgroup with one, two and four vectors a lane
@pytest.mark.parametrize("width", [8, 200, 256, 264, 2048, 2560, 5120, 16000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_norm_of_any_magnitude(width, dtype, eps):
    x, w = rows_of(width, 37, width).to(T[dtype]), 1 + 0.1 * normal(1, width)
    out, (codes, scales) = torch.empty_like(x), codes_for(37, width)
    gb.gdn_norm_forward(x, w, out=out, codes=codes, scales=scales, eps=eps)
    y, _ = ref.norm(x, w, eps)
    ref.near(out, y, y.abs() * ref.NORM)
    ref.check_codes(y, codes, scales, ref.NORM)


@pytest.mark.parametrize("width", [8, 264, 2048, 2560, 5120, 16000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_norm_gradients_of_any_magnitude(width, dtype, eps):
    rows = 1500  # more than one a walker
    r, w = rows_of(width, rows, width).to(T[dtype]), 1 + 0.1 * normal(1, width)
    dout = normal(2, rows, width).to(T[dtype])
    dx, dw = torch.empty_like(r), torch.empty(width, device=DEV)
    gb.gdn_norm_backward(dout, r, w, dx, dw, eps=eps)
    want, lost, want_w, lost_w = ref.norm_gradients(dout, r, w, eps)
    ref.near(dx, want, lost)
    ref.near(dw, want_w, lost_w)


HEADS = [(3, 16), (2, 64), (1, 48), (5, 128), (2, 96), (3, 256)]


@pytest.mark.parametrize("heads,d", HEADS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gated_norm_of_any_magnitude(heads, d, dtype):
    rows, eps = 41, 0.0
    x = rows_of(d, rows * heads, d).reshape(rows, heads, d).to(T[dtype])
    z, w = normal(3, rows, heads, d).to(T[dtype]), 1 + 0.1 * normal(1, d)
    out, (codes, scales) = torch.empty_like(z), codes_for(rows, heads * d)
    gb.gdn_gated_norm_forward(x, z, w, out=out, codes=codes, scales=scales, eps=eps)
    y, _ = ref.gated(x, z, w, eps)
    ref.near(out, y, y.abs() * ref.GATED)
    ref.check_codes(y.flatten(1), codes, scales, ref.GATED)
    dout = normal(4, rows, heads, d).to(T[dtype])
    dx, dz, dw = torch.empty_like(x), torch.empty_like(z), torch.empty(d, device=DEV)
    gb.gdn_gated_norm_backward(dout, x, z, w, dx, dz, dw, eps=eps)
    want, lost, want_z, lost_z, want_w, lost_w = ref.gated_gradients(dout, x, z, w, eps)
    ref.near(dx, want, lost)
    ref.near(dz, want_z, lost_z)
    ref.near(dw, want_w, lost_w)


@pytest.mark.parametrize("heads,d", HEADS)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_gates_at_the_ends(heads, d, dtype):
    """The lowest values, and where e^-z passes fp32's range on either side; z a is nothing far below 0."""
    rows, eps = 23, 1e-6
    ends = [torch.finfo(T[dtype]).min, -1e4, -710.0, -200.0, -104.0, -100.0, -90.0, -88.0, -87.0, -86.5, -86.0, -85.0, -40.0, 0.0, 90.0, 3e4]
    z = torch.tensor(ends, device=DEV).repeat(rows * heads * d // len(ends) + 1)[:rows * heads * d].reshape(rows, heads, d).to(T[dtype])
    z[5] = -90.0  # whole groups of small results
    z[6] = torch.finfo(T[dtype]).min
    x, w = normal(d, rows, heads, d), 1 + 0.1 * normal(1, d)
    out, (codes, scales) = torch.empty_like(z), codes_for(rows, heads * d)
    gb.gdn_gated_norm_forward(x, z, w, out=out, codes=codes, scales=scales, eps=eps)
    y, _ = ref.gated(x, z, w, eps)
    # f16 ends at 65504: a gate of 3e4 times n of 2.2 is over it, and from 65520, half a step on, rounds to infinity
    over = y.abs() >= (65520 if dtype == "f16" else float("inf"))
    assert (out[over] == torch.sign(y[over]) * float("inf")).all()
    ref.near(torch.where(over, 0, out), torch.where(over, 0, y), y.abs() * ref.GATED)
    # below 2^-126 a gate has fewer bits: not compared code by code, nor are rows where such a gate leads a group
    most = y.flatten(1).abs()
    whole = [i for i in range(rows) if i != 6]
    small = (most > 0) & (most < 2.0 ** -124)
    got = torch.where(small, 0, codes.float()).to(torch.float8_e4m3fn)[whole]
    ref.check_codes(torch.where(small, 0, y.flatten(1))[whole], got, scales[whole], ref.GATED)
    assert (codes[6].float() == 0).all() and (scales.view(torch.uint8)[6, :ref.cut(heads * d)] == 1).all()
    dout = normal(4, rows, heads, d).to(T[dtype])
    dx, dz, dw = torch.empty_like(x), torch.empty_like(z), torch.empty(d, device=DEV)
    gb.gdn_gated_norm_backward(dout, x, z, w, dx, dz, dw, eps=eps)
    want, lost, want_z, lost_z, want_w, lost_w = ref.gated_gradients(dout, x, z, w, eps)
    ref.near(dx, want, lost)
    ref.near(dz, want_z, lost_z)
    ref.near(dw, want_w, lost_w)


# 2^-40: what float64 may lose here, far above it, and far below an fp32 step
@pytest.mark.parametrize("rows,width", [(4096, 5120), (20000, 200), (3000, 1024), (5000, 2560), (500, 16000)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_codes_of_the_norm_are_exact(rows, width, dtype):
    x, w = normal(5, rows, width).to(T[dtype]), 1 + 0.1 * normal(1, width)
    codes, scales = codes_for(rows, width)
    gb.gdn_norm_forward(x, w, codes=codes, scales=scales, eps=1e-6)
    ref.check_codes(ref.norm(x, w, 1e-6)[0], codes, scales, 2.0 ** -40)


@pytest.mark.parametrize("heads,d", HEADS)
@pytest.mark.parametrize("x,z", [("f32", "bf16"), ("f16", "f32"), ("bf16", "bf16")])
def test_codes_of_the_gated_norm_are_exact(heads, d, x, z):
    rows = 4000
    x, z, w = normal(5, rows, heads, d).to(T[x]), (3 * normal(6, rows, heads, d)).to(T[z]), 1 + 0.1 * normal(1, d)
    codes, scales = codes_for(rows, heads * d)
    gb.gdn_gated_norm_forward(x, z, w, codes=codes, scales=scales, eps=1e-6)
    ref.check_codes(ref.gated(x, z, w, 1e-6)[0].flatten(1), codes, scales, 2.0 ** -40)


# rows, blocks of rows, tiles
@pytest.mark.parametrize("M", [1, 20, 64, 200, 4000])
@pytest.mark.parametrize("K", [272, 512])
def test_projections_of_any_magnitude(M, K):
    """Activations of 2^108 (2^-110) by fp32 weight scales of 1e-33 (1e33), scales of 0 and below 2^-126."""
    g = torch.Generator(device=DEV).manual_seed(M + K)
    N = 300
    a, w = [(torch.randn(r, K, generator=g, device=DEV) * 60).clamp(-448, 448).to(torch.float8_e4m3fn) for r in (M, N)]
    for power, size in ((235, 1e-33), (17, 1e33), (127, 1e-41), (127, 0.0), (240, 1e-41)):
        sa = torch.full((M, 4 * (K // 512 + 1)), power, dtype=torch.uint8, device=DEV).view(torch.float8_e8m0fnu)
        sw = torch.rand(3, ref.cut(K), generator=g, device=DEV) * size
        sw[1] = -sw[1]
        out = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
        gb.gdn_project(a, sa, w, sw, out)
        y, lost = ref.project(a, sa, w, sw)
        ref.near(out, y, lost)
