"""The layer's calls on arrays past 32-bit offsets and past one launch's threads: the last rows are right, and the first."""
import pytest
import torch

import layer_reference as ref
from gated_deltanet_recurrence_gdn_amd import binding as gb
from helpers import DEV
from test_gpu_norm import EPS, normal
from test_gpu_project import operands

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def noise(seed, rows, width, dtype=torch.bfloat16):
    """Rows of noise, the same 4096 again and again (a large tensor is made quickly so)."""
    return normal(seed, 4096, width, dtype=dtype).repeat(-(-rows // 4096), 1)[:rows]


@pytest.mark.parametrize("rows,width", [((1 << 21) + 5, 8), ((1 << 21) + 5, 1032)])
def test_norm(rows, width):
    """More rows than one launch takes; 2.2 billion elements."""
    x, w = noise(1, rows, width), normal(2, width)
    out, codes = torch.empty_like(x), torch.empty(rows, width, dtype=E4M3, device=DEV)
    scales = gb.gdn_scales_like(codes)
    gb.gdn_norm_forward(x, w, out=out, codes=codes, scales=scales, eps=EPS)
    for part in (slice(0, 9), slice((1 << 21) - 4, rows)):
        y, _ = ref.norm(x[part], w, EPS)
        ref.near(out[part], y, ref.NORM * y.abs())
        ref.check_codes(y, codes[part], scales.view(torch.uint8)[part].view(torch.float8_e8m0fnu), ref.NORM)
    dx = out
    gb.gdn_norm_backward(x, x, w, dx)
    want, lost, _, _ = ref.norm_gradients(x[-9:], x[-9:], w, EPS)
    ref.near(dx[-9:], want, lost)


def test_gated_norm():
    """More workgroups than one launch takes; 2.1 billion elements."""
    rows = (1 << 27) + 3
    x, w = noise(1, rows, 16).view(rows, 1, 16), normal(2, 16)
    z, out = x, torch.empty_like(x)
    gb.gdn_gated_norm_forward(x, z, w, out=out, eps=EPS)
    for part in (slice(0, 9), slice(rows - 9, rows)):
        y, _ = ref.gated(x[part], z[part], w, EPS)
        ref.near(out[part], y, ref.GATED * y.abs())
    dx = out
    gb.gdn_gated_norm_backward(x, x, z, w, dx)
    want, lost, *_ = ref.gated_gradients(x[-9:], x[-9:], z[-9:], w, EPS)
    ref.near(dx[-9:], want, lost)


def test_project():
    """2.3 billion results; weights and activations in rows that lie far apart."""
    M, N, K = 140001, 16384, 128
    a, sa, w, sw = operands(1, 4096, N, K)
    rows = torch.arange(M, device=DEV) % 4096
    big = a.view(torch.uint8)[rows].view(E4M3)
    scales = sa.view(torch.uint8)[rows].view(torch.float8_e8m0fnu)
    out = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    gb.gdn_project(big, scales, w, sw, out)
    for part in (slice(0, 5), slice(M - 5, M)):
        y, lost = ref.project(a.view(torch.uint8)[rows[part]].view(E4M3), sa.view(torch.uint8)[rows[part]].view(torch.float8_e8m0fnu), w, sw)
        ref.near(out[part], y, lost)
    del out, big
    stride = 1 << 22  # the largest: 1030 rows are 4.3 GB
    for M in (3, 1030):
        a, sa, w, sw = operands(2, M, 1030, 144)
        far_a = torch.empty(M, stride, dtype=torch.uint8, device=DEV).view(E4M3)
        far_w = torch.empty(1030, stride, dtype=torch.uint8, device=DEV).view(E4M3)
        far_a.view(torch.uint8)[:, :144], far_w.view(torch.uint8)[:, :144] = a.view(torch.uint8), w.view(torch.uint8)
        out = torch.empty(M, 1030, dtype=torch.bfloat16, device=DEV)
        gb.gdn_project(far_a[:, :144], sa, far_w[:, :144], sw, out)
        y, lost = ref.project(a, sa, w, sw)
        ref.near(out, y, lost)
        del far_a, far_w


def test_pack():
    """A row of states past 4 GiB, to and from a packed row past 2^31 bytes of scales and codes together."""
    slots = 1400
    states = torch.zeros(1, slots, 48, 128, 128, device=DEV)
    states[0, -1] = normal(1, 48, 128, 128)
    codes = torch.zeros(1, 3000, 48, 128, 128, dtype=torch.int8, device=DEV)
    scales = torch.zeros(1, 3000, 48, 128, device=DEV)
    last = torch.tensor([slots - 1, 2999], dtype=torch.int32, device=DEV)
    gb.gdn_pool_pack(states, codes, scales, last[:1], last[1:])
    want_c, want_s = ref.pack(states[0, -1])
    assert torch.equal(codes[0, -1], want_c) and torch.equal(scales[0, -1], want_s) and not codes[0, :-1].any()
    states[0, -1] = 0
    gb.gdn_pool_unpack(codes, scales, states, last[1:], last[:1])
    assert torch.equal(states[0, -1], want_c.float() * want_s[..., None])
