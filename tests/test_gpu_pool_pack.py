"""State rows in 8 bits on the GPU: codes and scales are exactly those of the definition in float64."""
import numpy as np
import pytest
import torch

import layer_reference as ref
from gated_deltanet_recurrence_gdn_amd import binding as gb
from helpers import DEV

pytestmark = pytest.mark.gpu
SLOT = gb.CODES["GDN_ERR_SLOT"]
T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def ints(*x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device=DEV)


def pools(seed, L, slots, packed, H, dv, dk, dtype=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(L, slots, H, dv, dk, generator=g, device=DEV) * torch.exp(2 * torch.randn(L, slots, H, dv, 1, generator=g, device=DEV))
    codes = torch.full((L, packed, H, dv, dk), 99, dtype=torch.int8, device=DEV)
    return x.to(dtype), codes, torch.full((L, packed, H, dv), -5.0, device=DEV)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("L,H,dv,dk", [(1, 1, 16, 32), (3, 2, 32, 32), (2, 3, 48, 64), (2, 6, 128, 128), (1, 5, 16, 128), (48, 1, 16, 64)])
def test_round_trip(L, H, dv, dk, dtype):
    x, codes, scales = pools(1, L, 5, 7, H, dv, dk, T[dtype])
    src, dst = [4, 0, 2, 2], [1, 6, 3, 0]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    gb.gdn_pool_pack(x, codes, scales, ints(*src), ints(*dst), status=status)
    want_c, want_s = ref.pack(x)
    for r in range(7):
        if r in dst:
            s = src[dst.index(r)]
            assert torch.equal(codes[:, r], want_c[:, s]) and torch.equal(scales[:, r], want_s[:, s])
        else:
            assert torch.all(codes[:, r] == 99) and torch.all(scales[:, r] == -5)
    back = torch.full_like(x, -3.0)
    gb.gdn_pool_unpack(codes, scales, back, ints(*dst), ints(3, 1, 4, 0), status=status)
    for d, s in zip((3, 1, 4, 0), src):
        assert torch.equal(back[:, d], (want_c[:, s].float() * want_s[:, s][..., None]).to(x.dtype))
    assert torch.all(back[:, 2] == -3) and status.item() == 0


def test_ties_and_borders():
    """Quotients at and beside halves, scales that are rounded up and down."""
    x, codes, scales = pools(2, 1, 4, 4, 4, 64, 128)
    k = torch.arange(128, device=DEV).float()
    g = torch.Generator(device=DEV).manual_seed(7)
    tops = torch.rand(4, 64, generator=g, device=DEV) + 0.5
    s = (tops.double() / 127).float()
    half = ((k - 64).double() + 0.5) * s.double()[..., None]
    x[0, 0] = half.float()                                        # as near a half as fp32 comes
    x[0, 1] = torch.nextafter(half.float(), torch.full_like(half.float(), 9))
    x[0, 2] = torch.nextafter(half.float(), torch.full_like(half.float(), -9))
    x[0, 3] = (k - 64) + 0.5                                      # exact halves below: the scale is 1
    x[0, :, :, :, 0] = torch.where(torch.arange(4, device=DEV)[:, None, None] == 3, 127.0, tops)
    gb.gdn_pool_pack(x, codes, scales, ints(0, 1, 2, 3), ints(0, 1, 2, 3))
    want_c, want_s = ref.pack(x)
    assert torch.equal(codes, want_c) and torch.equal(scales, want_s)


def test_extreme_channels():
    """Zeros, subnormal and huge channels; NaN and infinities take their own channel only."""
    x, codes, scales = pools(3, 1, 2, 2, 2, 16, 64)
    x[0, 0, 0, 0] = 0
    x[0, 0, 0, 1] = 1e-42
    x[0, 0, 0, 2] *= 1e-36
    x[0, 0, 0, 3] *= 1e37 / x[0, 0, 0, 3].abs().amax()
    x[0, 0, 0, 4, 7] = 3.4e38
    x[0, 0, 0, 5, 1] = float("nan")
    x[0, 0, 1, 6, 2] = float("inf")
    x[0, 0, 1, 7, 63] = -float("inf")
    gb.gdn_pool_pack(x, codes, scales, ints(0, 1), ints(1, 0))
    want_c, want_s = ref.pack(x[:, [1, 0]])
    assert torch.equal(codes, want_c) and torch.equal(scales.nan_to_num(-1), want_s.nan_to_num(-1))
    assert scales.isnan().sum() == 3
    back = torch.zeros_like(x)
    gb.gdn_pool_unpack(codes, scales, back, ints(1, 0), ints(0, 1))
    assert back.isnan().sum() == 3 * 64 and back[0, 0, 0, 5].isnan().all()


def test_bad_rows_and_fresh_ones():
    x, codes, scales = pools(4, 2, 4, 5, 2, 16, 32)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    # out of range, the same destination twice, passed over, and one fresh row
    src, dst = ints(0, 4, -2, 1, 1, 2, -1, 3), ints(0, 1, 1, 2, 2, -1, 3, 5)
    gb.gdn_pool_pack(x, codes, scales, src, dst, status=status)
    assert status.item() == SLOT
    want_c, want_s = ref.pack(x)
    assert torch.equal(codes[:, 0], want_c[:, 0]) and torch.equal(scales[:, 0], want_s[:, 0])
    for r in (1, 2, 4):
        assert torch.all(codes[:, r] == 99) and torch.all(scales[:, r] == -5)
    assert not codes[:, 3].any() and torch.all(scales[:, 3] == 2.0 ** -126)
    back = torch.full_like(x, 2.0)
    status.zero_()
    gb.gdn_pool_unpack(codes, scales, back, ints(0, 5, -1, 3, 0), ints(1, 0, 2, 3, -1), status=status)
    assert status.item() == SLOT
    assert torch.equal(back[:, 1], want_c[:, 0].float() * want_s[:, 0][..., None])
    assert torch.all(back[:, 0] == 2) and not back[:, 2].any() and not back[:, 3].any()


def test_persisted_nodes_and_layers_apart():
    """A verify's persisted f16 nodes as the source; packed pools whose layers lie apart, with guards around."""
    persist = torch.randn(2, 6, 3, 32, 64, device=DEV).half()
    whole_c = torch.full((5, 4, 3, 32, 64), 99, dtype=torch.int8, device=DEV)
    whole_s = torch.full((5, 4, 3, 32), -5.0, device=DEV)
    codes, scales = whole_c[3:4], whole_s[3:4]
    states = persist.flatten(0, 1)[None]
    gb.gdn_pool_pack(states, codes, scales, ints(7, 2), ints(0, 2))
    want_c, want_s = ref.pack(states)
    assert torch.equal(codes[0, 0], want_c[0, 7]) and torch.equal(scales[0, 2], want_s[0, 2])
    whole_c[3, [0, 2]], whole_s[3, [0, 2]] = 99, -5.0
    assert torch.all(whole_c == 99) and torch.all(whole_s == -5)
    x, _, _ = pools(6, 4, 3, 1, 2, 16, 32)
    part = torch.full((8, 3, 2, 16, 32), 99, dtype=torch.int8, device=DEV)
    sc = torch.full((8, 3, 2, 16), -5.0, device=DEV)
    gb.gdn_pool_pack(x, part[::2], sc[::2], ints(2), ints(1))
    want_c, want_s = ref.pack(x)
    assert torch.equal(part[::2, 1], want_c[:, 2]) and torch.equal(sc[::2, 1], want_s[:, 2])
    assert torch.all(part[1::2] == 99) and torch.all(part[::2, [0, 2]] == 99) and torch.all(sc[1::2] == -5)


def test_captured():
    x, codes, scales = pools(5, 3, 4, 4, 2, 64, 64)
    back, src, dst = torch.zeros_like(x), ints(0, 1, 2), ints(3, 2, 1)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        gb.gdn_pool_pack(x, codes, scales, src, dst)
        gb.gdn_pool_unpack(codes, scales, back, dst, src)
    for seed in range(3):
        x.copy_(pools(40 + seed, 3, 4, 4, 2, 64, 64)[0])
        graph.replay()
        torch.cuda.synchronize()
        c, s = ref.pack(x)
        assert torch.equal(back[:, :3], (c.float() * s[..., None])[:, :3])
