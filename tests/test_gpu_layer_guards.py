"""What lies around the outputs and workspaces of the layer's calls is left as it was."""
import ctypes

import pytest
import torch

import layer_reference as ref
from gated_deltanet_recurrence_gdn_amd import binding as gb
from helpers import DEV
from test_gpu_norm import EPS, normal
from test_gpu_project import operands

pytestmark = pytest.mark.gpu
PAD = 4096  # bytes on either side


class Guarded:
    """Tensors inside larger buffers of 0xA5 bytes."""

    def __init__(self):
        self.all = []

    def __call__(self, shape, dtype):
        n = torch.empty(shape, dtype=dtype, device="meta")
        size = n.numel() * n.element_size()
        whole = torch.full((size + 2 * PAD,), 0xA5, dtype=torch.uint8, device=DEV)
        self.all.append((whole, size))
        return whole[PAD:PAD + size].view(dtype).view(shape)

    def check(self):
        torch.cuda.synchronize()
        for whole, size in self.all:
            assert torch.all(whole[:PAD] == 0xA5) and torch.all(whole[PAD + size:] == 0xA5)


def inside(x):
    """A copy of an input between NaNs: what is read beside it shows."""
    n = x.numel() * x.element_size()
    whole = torch.full((n + 2 * PAD,), 0xFF, dtype=torch.uint8, device=DEV)
    y = whole[PAD:PAD + n].view(x.dtype).view(x.shape)
    y.view(torch.uint8).copy_(x.contiguous().view(torch.uint8))
    return y


@pytest.mark.parametrize("rows,width", [(1, 8), (5, 136), (33, 264), (3, 2056), (700, 1000), (3, 5120)])
def test_norm(rows, width):
    g = Guarded()
    x, z, w, d = inside(normal(1, rows, width, dtype=torch.bfloat16)), inside(normal(2, rows, width)), inside(normal(3, width)), \
        inside(normal(4, rows, width, dtype=torch.bfloat16))
    r, out, codes = g((rows, width), torch.float32), g((rows, width), torch.bfloat16), g((rows, width), torch.float8_e4m3fn)
    scales = g((rows, -(-ref.cut(width) // 4) * 4), torch.float8_e8m0fnu)
    gb.gdn_norm_forward(x, w, out=out, codes=codes, scales=scales, residual=z, residual_out=r, eps=EPS)
    y, _ = ref.norm(x.float() + z, w, EPS)
    ref.near(out, y, ref.NORM * y.abs())
    ref.check_codes(y, codes, scales, ref.NORM)
    need = gb.lib().gdn_norm_backward_workspace_bytes(ctypes.byref(gb.GdnNormShape(rows, width, width, 1, 0, 0, 0, EPS, 0.0)))
    dx, dw, ws = g((rows, width), torch.float32), g((width,), torch.float32), g((need,), torch.uint8)
    gb.gdn_norm_backward(d, r, w, dx, dw, workspace=ws, eps=EPS)
    want, lost, dweight, dlost = ref.norm_gradients(d, r, w, EPS)
    ref.near(dx, want, lost)
    ref.near(dw, dweight, dlost)
    g.check()


@pytest.mark.parametrize("rows,heads,d", [(1, 1, 16), (7, 3, 48), (5, 2, 112), (33, 5, 64), (400, 6, 128), (3, 3, 256)])
def test_gated_norm(rows, heads, d):
    g = Guarded()
    x, z, w, dy = inside(normal(1, rows, heads, d)), inside(normal(2, rows, heads, d, dtype=torch.bfloat16)), inside(normal(3, d)), \
        inside(normal(4, rows, heads, d, dtype=torch.bfloat16))
    out, codes = g((rows, heads, d), torch.bfloat16), g((rows, heads * d), torch.float8_e4m3fn)
    scales = g((rows, -(-ref.cut(heads * d) // 4) * 4), torch.float8_e8m0fnu)
    gb.gdn_gated_norm_forward(x, z, w, out=out, codes=codes, scales=scales, eps=EPS)
    y, _ = ref.gated(x, z, w, EPS)
    ref.near(out, y, ref.GATED * y.abs())
    ref.check_codes(y.reshape(rows, -1), codes, scales, ref.GATED)
    need = gb.lib().gdn_gated_norm_backward_workspace_bytes(
        ctypes.byref(gb.GdnGatedNormShape(rows, heads * d, heads * d, heads, d, 0, 1, 0, 0, EPS)))
    dx, dz, dw, ws = g(x.shape, x.dtype), g(z.shape, z.dtype), g((d,), torch.float32), g((need,), torch.uint8)
    gb.gdn_gated_norm_backward(dy, x, z, w, dx, dz, dw, workspace=ws, eps=EPS)
    want_x, lost_x, want_z, lost_z, want_w, lost_w = ref.gated_gradients(dy, x, z, w, EPS)
    ref.near(dx, want_x, lost_x)
    ref.near(dz, want_z, lost_z)
    ref.near(dw, want_w, lost_w)
    g.check()


@pytest.mark.parametrize("scales", ["f32", "e8m0"])
@pytest.mark.parametrize("M", [1, 17, 33, 65, 200, 300, 66000])
@pytest.mark.parametrize("parts,K", [([5], 16), ([130, 7], 400), ([96, 40], 1040), ([1000, 24, 6], 272)])
def test_project(parts, K, M, scales):
    g = Guarded()
    a, sa, w, sw = (inside(t) for t in operands(1, M, sum(parts), K, scales))
    outs = [g((M, n), torch.bfloat16) for n in parts]
    gb.gdn_project(a, sa, w, sw, outs)
    y, lost = ref.project(a, sa, w, sw)
    ref.near(torch.cat(outs, 1), y, lost)
    g.check()
