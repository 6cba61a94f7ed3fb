"""The input norm on the GPU against its formulas in float64: outputs, residual, 8-bit codes and gradients."""
import pytest
import torch

import layer_reference as ref
from gated_deltanet_recurrence_gdn_amd import binding as gb
from helpers import DEV

pytestmark = pytest.mark.gpu
T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


def normal(seed, *shape, dtype=torch.float32, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g, device=DEV)).to(dtype)


def like(t, dtype=None):
    return torch.full_like(t, float("nan"), dtype=dtype)


def codes_for(rows, width):
    codes = torch.full((rows, width), 0x7f, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    return codes, gb.gdn_scales_like(codes)


# widths of part of a wave, a wave, a workgroup of one and of two vectors a lane; odd rows; ragged groups of 128
SIZES = [(1, 8), (3, 128), (7, 200), (33, 256), (5, 264), (2, 512), (9, 1000), (6, 2048), (4, 2056), (1, 5120), (3, 8192),
         (2, 8200), (2, 16384)]


@pytest.mark.parametrize("rows,width", SIZES)
@pytest.mark.parametrize("x,residual,weight,offset", [("bf16", "bf16", "bf16", 1.0), ("f32", None, "f32", 0.0),
                                                      ("bf16", "f32", "f32", 0.0), ("f16", "f16", "f16", 1.0)])
def test_forward(rows, width, x, residual, weight, offset):
    xs, w = normal(1, rows, width, dtype=T[x]), normal(2, width, dtype=T[weight])
    z = None if residual is None else normal(3, rows, width, dtype=T[residual], scale=3.0)
    r = None if z is None else like(z)
    out = like(xs)
    codes, scales = codes_for(rows, width)
    gb.gdn_norm_forward(xs, w, out=out, codes=codes, scales=scales, residual=z, residual_out=r, eps=EPS, weight_offset=offset)
    want = xs if z is None else (xs.float() + z.float()).to(z.dtype)
    if z is not None:
        assert torch.equal(r, want)
    y, _ = ref.norm(want, w.double() + offset, EPS)
    ref.near(out, y, ref.NORM * y.abs())
    ref.check_codes(y, codes, scales, ref.NORM)


@pytest.mark.parametrize("only", ["out", "codes", "residual"])
def test_one_output(only):
    x, z, w = normal(1, 5, 384, dtype=torch.bfloat16), normal(2, 5, 384, dtype=torch.bfloat16), normal(3, 384)
    r, out, (codes, scales) = like(z), like(x), codes_for(5, 384)
    gb.gdn_norm_forward(x, w, residual=z, residual_out=r if only == "residual" else None, out=out if only == "out" else None,
                        codes=codes if only == "codes" else None, scales=scales if only == "codes" else None)
    want = (x.float() + z.float()).bfloat16()
    y, _ = ref.norm(want, w, EPS)
    if only == "residual":
        assert torch.equal(r, want)
    elif only == "out":
        ref.near(out, y, ref.NORM * y.abs())
    else:
        ref.check_codes(y, codes, scales, ref.NORM)


def test_rows_apart_and_in_place():
    """x a slice of wider rows; the residual and the output where their inputs were; nothing written beside them."""
    wide = normal(1, 9, 1000, dtype=torch.bfloat16)
    x, z, w = wide[:, 200:600], normal(2, 9, 400), normal(3, 400)
    want = x.float() + z
    keep = wide.clone()
    gb.gdn_norm_forward(x, w, residual=z, residual_out=z, out=(out := like(z, torch.bfloat16)))
    assert torch.equal(z, want) and torch.equal(wide, keep)
    ref.near(out, ref.norm(want, w, EPS)[0], ref.NORM * ref.norm(want, w, EPS)[0].abs())
    x = normal(4, 2, 3, 264, dtype=torch.float16)  # more leading dimensions, the output over x
    y, _ = ref.norm(x.clone(), w[:264], EPS)
    gb.gdn_norm_forward(x, w[:264], out=x)
    ref.near(x, y, ref.NORM * y.abs())


def test_scales_behind_the_last_group_stay():
    x, w = normal(1, 6, 640, dtype=torch.bfloat16), normal(2, 640)
    codes = torch.empty(6, 640, dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.full((6, 12), 0x55, dtype=torch.uint8, device=DEV)
    gb.gdn_norm_forward(x, w, codes=codes, scales=scales.view(torch.float8_e8m0fnu))
    assert torch.all(scales[:, 5:] == 0x55)
    ref.check_codes(ref.norm(x, w, EPS)[0], codes, scales.view(torch.float8_e8m0fnu), ref.NORM)


def test_borders_of_the_scale():
    """Groups whose largest magnitude is 448 2^e exactly, or the next value above: eps 0 and one channel a row make y = w."""
    x = torch.zeros(2, 1024, device=DEV)
    x[:, 0] = 1.0  # s = sqrt(1024) = 32 exactly
    w = torch.zeros(1024, device=DEV)
    for top in (14.0, 14.000001, 28.0, 2.0 ** -100, 1.5):
        w[0] = top
        codes, scales = codes_for(2, 1024)
        gb.gdn_norm_forward(x, w, codes=codes, scales=scales, eps=0.0)
        y = x.double() * 32 * w.double()
        ref.check_codes(y, codes, scales, 0.0)


def test_empty_and_zero_rows():
    w = normal(1, 256)
    x = torch.empty(0, 256, device=DEV)
    dw = torch.full((256,), float("nan"), device=DEV)
    gb.gdn_norm_forward(x, w, out=torch.empty_like(x))
    gb.gdn_norm_backward(torch.empty_like(x), x, w, torch.empty_like(x), dw)
    assert torch.equal(dw, torch.zeros_like(dw))
    x = torch.zeros(3, 256, device=DEV)
    out, (codes, scales) = like(x), codes_for(3, 256)
    gb.gdn_norm_forward(x, w, out=out, codes=codes, scales=scales)
    assert not out.any() and not codes.float().any() and torch.all(scales.view(torch.uint8)[:, :2] == 1)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_nan_and_infinity_stay_in_their_row(bad):
    x, w = normal(1, 8, 1152, dtype=torch.bfloat16), normal(2, 1152)
    x[3, 700] = bad
    out, (codes, scales) = like(x), codes_for(8, 1152)
    gb.gdn_norm_forward(x, w, out=out, codes=codes, scales=scales)
    others = [0, 1, 2, 4, 5, 6, 7]
    y, _ = ref.norm(x[others], w, EPS)
    ref.near(out[others], y, ref.NORM * y.abs())
    ref.check_codes(y, codes[others], scales.view(torch.uint8)[others].view(torch.float8_e8m0fnu), ref.NORM)
    assert out[3, 700].isnan() and scales.view(torch.uint8)[3, 5] == 255 and codes[3, 640:768].float().isnan().all()
    d, dx, dw = normal(3, 8, 1152, dtype=torch.bfloat16), like(x), like(w)
    gb.gdn_norm_backward(d, x, w, dx, dw)
    want, lost, _, _ = ref.norm_gradients(d[others], x[others], w, EPS)
    ref.near(dx[others], want, lost)
    assert dx[3, 700].isnan() and dw[700].isnan()


@pytest.mark.parametrize("rows,width", SIZES + [(1030, 96), (700, 2304), (0, 64)])
@pytest.mark.parametrize("d,r,given,offset", [("bf16", "f32", True, 0.0), ("bf16", "bf16", True, 1.0), ("f32", "f32", False, 0.0),
                                              ("f16", "f16", False, 1.0)])
def test_backward(rows, width, d, r, given, offset):
    dout, rs, w = normal(1, rows, width, dtype=T[d]), normal(2, rows, width, dtype=T[r], scale=2.0), normal(3, width, dtype=torch.bfloat16)
    dres = normal(4, rows, width, dtype=T[r]) if given else None
    dx, dw = like(rs), torch.full((width,), float("nan"), device=DEV)
    gb.gdn_norm_backward(dout, rs, w, dx, dw, dresidual=dres, eps=EPS, weight_offset=offset)
    want, lost, dweight, dlost = ref.norm_gradients(dout, rs, w.double() + offset, EPS, dres)
    ref.near(dx, want, lost)
    ref.near(dw, dweight, dlost)
    again, dw2 = like(rs), torch.empty_like(dw)
    gb.gdn_norm_backward(dout, rs, w, again, dw2, dresidual=dres, eps=EPS, weight_offset=offset)
    assert torch.equal(dx, again) and torch.equal(dw, dw2)


def test_backward_parts():
    """dx over dresidual; each gradient by itself; rows of r apart."""
    wide, d, w = normal(1, 20, 904), normal(2, 20, 320), normal(3, 320)
    r = wide[:, 104:424]
    dres = normal(4, 20, 320)
    want, lost, dweight, dlost = ref.norm_gradients(d, r, w, EPS, dres)
    gb.gdn_norm_backward(d, r, w, dres, None, dresidual=dres)
    ref.near(dres, want, lost)
    dw = torch.empty(320, device=DEV)
    gb.gdn_norm_backward(d, r, w, None, dw)
    ref.near(dw, dweight, dlost)


def test_gradient_against_differences():
    """Central differences of the forward formula in float64 along random directions."""
    r, w, d = normal(1, 3, 64), normal(2, 64), normal(3, 3, 64)
    dx, dw = like(r), torch.empty_like(w)
    gb.gdn_norm_backward(d, r, w, dx, dw)
    h = 1e-6
    for seed in range(4):
        u, v = normal(10 + seed, 3, 64).double(), normal(20 + seed, 64).double()
        f = lambda s: (ref.norm(r.double() + s * u, w.double() + s * v, EPS)[0] * d.double()).sum()  # noqa: E731
        # the difference's own error is about h^2 of the third derivatives, and 2^-53 / h of the sum
        slope, got = (f(h) - f(-h)) / (2 * h), (dx.double() * u).sum() + (dw.double() * v).sum()
        terms = (dx.double() * u).abs().sum() + (dw.double() * v).abs().sum()
        assert abs(slope - got) <= 1e-5 * terms


def test_captured():
    """Forward and backward in a graph, replayed over other inputs, with eager calls between."""
    rows, width = 300, 1536
    x, z, w = normal(1, rows, width, dtype=torch.bfloat16), normal(2, rows, width), normal(3, width)
    d = normal(4, rows, width, dtype=torch.bfloat16)
    r, out, (codes, scales), dx, dw = like(z), like(x), codes_for(rows, width), like(z), torch.empty(width, device=DEV)
    ws = torch.empty(gb.lib().gdn_norm_backward_workspace_bytes(gb.GdnNormShape(rows, width, width, 1, 0, 0, 0, EPS, 0.0)),
                     dtype=torch.uint8, device=DEV)

    def step():
        gb.gdn_norm_forward(x, w, residual=z, residual_out=r, out=out, codes=codes, scales=scales)
        gb.gdn_norm_backward(d, r, w, dx, dw, dresidual=z, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        x.copy_(normal(50 + seed, rows, width, dtype=torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (r, out, codes.view(torch.uint8), dx, dw)]
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (r, out, codes.view(torch.uint8), dx, dw)):
            assert torch.equal(a, b)


def test_another_stream():
    side = torch.cuda.Stream()
    x, w, d = normal(1, 64, 4096, dtype=torch.bfloat16), normal(2, 4096), normal(3, 64, 4096, dtype=torch.bfloat16)
    out, dx, dw = like(x), like(x), torch.empty(4096, device=DEV)
    side.wait_stream(torch.cuda.current_stream())
    gb.gdn_norm_forward(x, w, out=out, stream=side)
    gb.gdn_norm_backward(d, x, w, dx, dw, stream=side)
    side.synchronize()
    y, _ = ref.norm(x, w, EPS)
    want, lost, dweight, dlost = ref.norm_gradients(d, x, w, EPS)
    ref.near(out, y, ref.NORM * y.abs())
    ref.near(dx, want, lost)
    ref.near(dw, dweight, dlost)
