"""The gated head norm on the GPU against its formulas in float64."""
import pytest
import torch

import layer_reference as ref
from gated_deltanet_recurrence_gdn_amd import binding as gb
from helpers import DEV
from test_gpu_norm import EPS, T, codes_for, like, normal

pytestmark = pytest.mark.gpu

# every kind of head: 2 to 32 lanes, and those that are no power of two; rows that end inside a group of 128
HEADS = [(1, 16), (3, 16), (5, 32), (2, 48), (7, 64), (4, 80), (3, 96), (1, 112), (48, 128), (6, 128), (3, 144), (2, 208),
         (5, 256), (2, 240)]


def inputs(rows, heads, d, x, z):
    return (normal(1, rows, heads, d, dtype=T[x], scale=0.3), normal(2, rows, heads, d, dtype=T[z], scale=2.0),
            1 + 0.2 * normal(3, d))


@pytest.mark.parametrize("heads,d", HEADS)
@pytest.mark.parametrize("x,z", [("f32", "bf16"), ("f16", "bf16"), ("bf16", "bf16"), ("f32", "f32"), ("bf16", "f16")])
@pytest.mark.parametrize("rows", [1, 17])
def test_forward(rows, heads, d, x, z):
    xs, zs, w = inputs(rows, heads, d, x, z)
    out, (codes, scales) = like(zs), codes_for(rows, heads * d)
    gb.gdn_gated_norm_forward(xs, zs, w, out=out, codes=codes, scales=scales, eps=EPS)
    y, _ = ref.gated(xs, zs, w, EPS)
    ref.near(out, y, ref.GATED * y.abs())
    ref.check_codes(y.reshape(rows, -1), codes, scales, ref.GATED)


@pytest.mark.parametrize("heads,d", HEADS)
@pytest.mark.parametrize("x,z", [("f32", "bf16"), ("bf16", "bf16"), ("f32", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("rows", [1, 37])
def test_backward(rows, heads, d, x, z):
    xs, zs, w = inputs(rows, heads, d, x, z)
    dout = normal(4, rows, heads, d, dtype=T[z])
    dx, dz, dw = like(xs), like(zs), torch.full((d,), float("nan"), device=DEV)
    gb.gdn_gated_norm_backward(dout, xs, zs, w, dx, dz, dw, eps=EPS)
    want_x, lost_x, want_z, lost_z, want_w, lost_w = ref.gated_gradients(dout, xs, zs, w, EPS)
    ref.near(dx, want_x, lost_x)
    ref.near(dz, want_z, lost_z)
    ref.near(dw, want_w, lost_w)
    dx2, dw2 = like(xs), torch.empty_like(dw)
    gb.gdn_gated_norm_backward(dout, xs, zs, w, dx2, None, dw2, eps=EPS)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_many_rows():
    """More pieces than the backward pass has workgroups."""
    xs, zs, w = inputs(3001, 48, 128, "bf16", "bf16")
    dout = normal(4, 3001, 48, 128, dtype=torch.bfloat16)
    dx, dz, dw = like(xs), like(zs), torch.empty(128, device=DEV)
    gb.gdn_gated_norm_backward(dout, xs, zs, w, dx, dz, dw)
    want_x, lost_x, want_z, lost_z, want_w, lost_w = ref.gated_gradients(dout, xs, zs, w, EPS)
    ref.near(dx, want_x, lost_x)
    ref.near(dz, want_z, lost_z)
    ref.near(dw, want_w, lost_w)


def test_rows_apart():
    """x and z are slices of wider projections' rows; a weight in bf16; four dimensions."""
    wide = normal(1, 21, 2000, dtype=torch.bfloat16)
    x, z = wide[:, 104:872].view(21, 6, 128), wide[:, 1000:1768].view(21, 6, 128)
    w = normal(2, 128, dtype=torch.bfloat16)
    out = torch.empty(21, 6, 128, dtype=torch.bfloat16, device=DEV)
    gb.gdn_gated_norm_forward(x, z, w, out=out)
    y, _ = ref.gated(x, z, w, EPS)
    ref.near(out, y, ref.GATED * y.abs())
    x4 = x.contiguous().view(3, 7, 6, 128)
    out4 = torch.empty_like(x4)
    gb.gdn_gated_norm_forward(x4, z.contiguous().view(3, 7, 6, 128), w, out=out4)
    assert torch.equal(out4.view_as(out), out)


def test_extreme_gates():
    """Far gates: the logistic's ends.  |z| up to 80 keeps silu(z) above 2^-126."""
    x = normal(1, 4, 2, 64)
    z = torch.linspace(-80, 80, 4 * 2 * 64, device=DEV).view(4, 2, 64).contiguous()
    w, d = torch.ones(64, device=DEV), normal(2, 4, 2, 64)
    out, dx, dz = like(x), like(x), like(z)
    gb.gdn_gated_norm_forward(x, z, w, out=out)
    gb.gdn_gated_norm_backward(d, x, z, w, dx, dz)
    y, _ = ref.gated(x, z, w, EPS)
    ref.near(out, y, ref.GATED * y.abs())
    want_x, lost_x, want_z, lost_z, _, _ = ref.gated_gradients(d, x, z, w, EPS)
    ref.near(dx, want_x, lost_x)
    ref.near(dz, want_z, lost_z)
    z = torch.full_like(z, -1000.0)
    gb.gdn_gated_norm_forward(x, z, w, out=out)
    assert torch.all(out.abs() < 1e-30)  # 1000 e^-1000 of a few
    z = torch.full_like(z, 1000.0)
    gb.gdn_gated_norm_forward(x, z, w, out=out)
    n, _ = ref.gated(x, z, w, EPS)
    ref.near(out, n, ref.GATED * n.abs())


@pytest.mark.parametrize("where", ["x", "z"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nan_and_infinity_stay_in_their_head(where, bad):
    x, z, w = inputs(3, 4, 64, "f32", "bf16")
    (x if where == "x" else z)[1, 2, 5] = bad
    out, (codes, scales) = like(z), codes_for(3, 256)
    gb.gdn_gated_norm_forward(x, z, w, out=out, codes=codes, scales=scales)
    y, _ = ref.gated(x, z, w, EPS)
    fine = torch.ones(3, 4, dtype=torch.bool, device=DEV)
    fine[1, 2] = False
    ref.near(out[fine], y[fine], ref.GATED * y[fine].abs())
    assert not out[1, 2, 5].isfinite()
    byte = scales.view(torch.uint8)[:, :2]
    assert byte[1, 1] == 255 and (byte == 255).sum() == 1 and codes[1, 128:].float().isnan().all()


def test_empty():
    x, w = torch.empty(0, 4, 64, device=DEV), torch.ones(64, device=DEV)
    dw = torch.full((64,), float("nan"), device=DEV)
    gb.gdn_gated_norm_forward(x, x, w, out=torch.empty_like(x))
    gb.gdn_gated_norm_backward(x, x, x, w, torch.empty_like(x), torch.empty_like(x), dw)
    assert torch.equal(dw, torch.zeros_like(dw))


def test_gradient_against_differences():
    x, z, w, d = normal(1, 2, 3, 48), normal(2, 2, 3, 48), normal(3, 48), normal(4, 2, 3, 48)
    dx, dz, dw = like(x), like(z), torch.empty_like(w)
    gb.gdn_gated_norm_backward(d, x, z, w, dx, dz, dw)
    h = 1e-6
    for seed in range(4):
        u, v, t = normal(10 + seed, 2, 3, 48).double(), normal(20 + seed, 2, 3, 48).double(), normal(30 + seed, 48).double()
        f = lambda s: (ref.gated(x.double() + s * u, z.double() + s * v, w.double() + s * t, EPS)[0] * d.double()).sum()  # noqa: E731
        slope = (f(h) - f(-h)) / (2 * h)
        parts = (dx.double() * u, dz.double() * v, dw.double() * t)
        assert abs(slope - sum(p.sum() for p in parts)) <= 1e-5 * sum(p.abs().sum() for p in parts)


def test_captured():
    x, z, w = inputs(100, 6, 128, "f32", "bf16")
    d = normal(4, 100, 6, 128, dtype=torch.bfloat16)
    (codes, scales), dx, dz, dw = codes_for(100, 768), like(x), like(z), torch.empty(128, device=DEV)
    ws = torch.empty(1024 * 128 * 4, dtype=torch.uint8, device=DEV)

    def step():
        gb.gdn_gated_norm_forward(x, z, w, codes=codes, scales=scales)
        gb.gdn_gated_norm_backward(d, x, z, w, dx, dz, dw, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        x.copy_(normal(50 + seed, 100, 6, 128))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (codes.view(torch.uint8), dx, dz, dw)]
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (codes.view(torch.uint8), dx, dz, dw)):
            assert torch.equal(a, b)
