"""The projections on the GPU against the product of what the 8-bit operands stand for, in float64."""
import pytest
import torch

import layer_reference as ref
from gated_deltanet_recurrence_gdn_amd import binding as gb
from helpers import DEV

pytestmark = pytest.mark.gpu
T = {"bf16": torch.bfloat16, "f16": torch.float16}


def operands(seed, M, N, K, scales="f32", spread=3):
    """Codes of every size and sign, scales that differ from group to group and from block to block."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    G, B = ref.cut(K), ref.cut(N)
    codes = lambda r: (torch.randn(r, K, generator=g, device=DEV) * 60).clamp(-448, 448).to(torch.float8_e4m3fn)  # noqa: E731
    pad = -(-G // 4) * 4
    powers = lambda r: torch.randint(118 - spread, 119 + spread, (r, pad), generator=g, device=DEV).to(torch.uint8).view(torch.float8_e8m0fnu)  # noqa: E731
    a, sa, w = codes(M), powers(M), codes(N)
    sw = powers(B) if scales == "e8m0" else torch.rand(B, G, generator=g, device=DEV) * 0.01 + 1e-4
    return a, sa, w, sw


def outputs(M, parts, dtype):
    return [torch.full((M, n), float("nan"), dtype=dtype, device=DEV) for n in parts]


def check(a, sa, w, sw, outs):
    y, lost = ref.project(a, sa, w, sw)
    got = torch.cat([o.reshape(o.shape[0], -1) for o in outs], 1)
    ref.near(got, y, lost)


TOKENS = [1, 2, 15, 16, 17, 22, 33, 64, 65, 100, 128, 129, 200, 257, 333]
SHAPES = [(8, 16), (16, 128), (48, 144), (128, 256), (130, 1936), (250, 400), (256, 1024), (1030, 2064)]


@pytest.mark.parametrize("scales", ["f32", "e8m0"])
@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("M", TOKENS)
def test_product(M, N, K, scales):
    x = operands(M + N, M, N, K, scales)
    outs = outputs(M, [N], torch.bfloat16)
    gb.gdn_project(*x, outs[0])
    check(*x, outs)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M", [1, 16, 40, 300, 2200])
@pytest.mark.parametrize("parts", [[256, 256, 768], [777, 6, 6, 250], [1] * 8, [3, 129, 5], [128, 4, 124, 2]])
def test_parts(M, parts, dtype):
    x = operands(M, M, sum(parts), 272)
    outs = outputs(M, parts, T[dtype])
    gb.gdn_project(*x, outs)
    check(*x, outs)


@pytest.mark.parametrize("M", [1, 22, 150, 8300])
def test_rows_apart(M):
    """Operands and outputs that are slices of wider rows; what lies between is left as it was."""
    a, sa, w, sw = operands(3, M, 200, 640)
    wide_a = torch.zeros(M, 1024, dtype=torch.uint8, device=DEV).fill_(0x7f).view(torch.float8_e4m3fn)
    wide_w = torch.zeros(200, 768, dtype=torch.uint8, device=DEV).fill_(0x7f).view(torch.float8_e4m3fn)
    wide_a[:, 128:768], wide_w[:, 64:704] = a, w
    scales = torch.full((M, 12), 0xff, dtype=torch.uint8, device=DEV)
    scales[:, :8] = sa.view(torch.uint8)
    scales[:, 5:] = 0xff  # behind the last group: not used
    out = torch.full((M, 500), 7.0, dtype=torch.bfloat16, device=DEV)
    keep = out.clone()
    parts = [out[:, 3:130], out[:, 200:273]]
    gb.gdn_project(wide_a[:, 128:768], scales.view(torch.float8_e8m0fnu), wide_w[:, 64:704], sw, parts)
    check(a, sa, w, sw, parts)
    keep[:, 3:130], keep[:, 200:273] = out[:, 3:130], out[:, 200:273]
    assert torch.equal(out, keep)


@pytest.mark.parametrize("M", [1, 16, 130, 66000])
@pytest.mark.parametrize("scales", ["f32", "e8m0"])
def test_what_is_behind_the_last_channel_is_not_read(M, scales):
    """K = 144: codes behind the row's end (the next row's) are not part of the last group."""
    a, sa, w, sw = operands(1, M, 40, 144, scales)
    a.view(torch.uint8)[:, :128] = 0
    w.view(torch.uint8)[:, :128] = 0x7f  # NaN codes times zeros
    a.view(torch.uint8)[0, 0] = 0
    w.view(torch.uint8)[1:, :128] = 0
    outs = outputs(M, [40], torch.bfloat16)
    gb.gdn_project(a, sa, w, sw, outs)
    assert outs[0][:, 0].isnan().all()
    y, lost = ref.project(a, sa, w[1:], sw)
    ref.near(outs[0][:, 1:], y, lost)


@pytest.mark.parametrize("M", [1, 20, 140, 4000])
@pytest.mark.parametrize("scales", ["f32", "e8m0"])
def test_nan_scales_and_far_powers(M, scales):
    a, sa, w, sw = operands(2, M, 300, 512, scales)
    sa.view(torch.uint8)[0, 2] = 255
    if scales == "f32":
        sw[1, 1] = float("nan")
    else:
        sw.view(torch.uint8)[1, 1] = 255
    outs = outputs(M, [300], torch.bfloat16)
    gb.gdn_project(a, sa, w, sw, outs)
    assert outs[0][0].isnan().all() and outs[0][:, 128:256].isnan().all()
    fine = [n for n in range(300) if not 128 <= n < 256]
    keep = torch.arange(M, device=DEV) > 0
    y, lost = ref.project(a, sa, w, sw)
    ref.near(outs[0][keep][:, fine], y[keep][:, fine], lost[keep][:, fine])
    # powers far from 1 on one side and the inverse on the other
    a, sa, w, sw = operands(2, M, 300, 512, "e8m0")
    sa.view(torch.uint8)[:] = 217
    sw.view(torch.uint8)[:] = 17
    gb.gdn_project(a, sa, w, sw, outs)
    check(a, sa, w, sw, outs)


def test_no_tokens():
    a, sa, w, sw = operands(1, 4, 64, 128)
    out = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    gb.gdn_project(a[:0], sa.view(torch.uint8)[:0].view(torch.float8_e8m0fnu), w, sw, out)


@pytest.mark.parametrize("M", [4, 200, 2000])
def test_repeats_and_captured(M):
    x = operands(5, M, 520, 1040)
    outs, again = outputs(M, [512, 8], torch.bfloat16), outputs(M, [512, 8], torch.bfloat16)
    gb.gdn_project(*x, outs)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        gb.gdn_project(*x, again)
    for seed in range(3):
        other = operands(60 + seed, M, 520, 1040)
        for t, o in zip(x[:2], other[:2]):
            t.view(torch.uint8).copy_(o.view(torch.uint8))
        graph.replay()
        gb.gdn_project(*x, outs)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(outs, again))
        check(*x, outs)


def test_another_stream():
    side = torch.cuda.Stream()
    x = operands(5, 70, 256, 512)
    outs = outputs(70, [256], torch.bfloat16)
    side.wait_stream(torch.cuda.current_stream())
    gb.gdn_project(*x, outs, stream=side.cuda_stream)
    side.synchronize()
    check(*x, outs)


# sizes that take each of the tiles: 256 x 256, 128 x 128 two and one a CU, 64 x 128; more than 64 groups; blocks of rows
@pytest.mark.parametrize("scales", ["f32", "e8m0"])
@pytest.mark.parametrize("M,parts,K", [(1000, [16000, 380], 272), (300, [16380], 400), (500, [5000, 100], 640), (70, [5100], 384),
                                       (70, [300], 8400), (300, [16384], 8336), (2060, [2300], 272), (256, [1000], 8336), (4100, [60], 2064), (1024, [16384], 8464), (3, [200], 8400), (60, [16400], 1168)])
def test_tiles(M, parts, K, scales):
    x = operands(M, M, sum(parts), K, scales)
    outs = outputs(M, parts, torch.bfloat16)
    gb.gdn_project(*x, outs)
    check(*x, outs)
