"""Projections whose last block of tokens is part of a block, with scales whose rows lie far apart."""
import pytest
import torch

from gated_deltanet_recurrence_gdn_amd import binding as gb
from helpers import DEV
from test_gpu_project import check, operands, outputs

pytestmark = pytest.mark.gpu


# tokens of one, two and three parts of 16 in the last block, in one block and behind whole ones
@pytest.mark.parametrize("M", [17, 33, 40, 47, 65, 100])
@pytest.mark.parametrize("scales", ["f32", "e8m0"])
def test_scales_far_apart(M, scales):
    """Rows of scales 2^20 bytes apart, which end at the tensor's last byte."""
    a, sa, w, sw = operands(M, M, 150, 400, scales)
    far = torch.empty(M, 1 << 20, dtype=torch.uint8, device=DEV)
    far[:, :sa.shape[1]] = sa.view(torch.uint8)
    outs = outputs(M, [150], torch.bfloat16)
    gb.gdn_project(a, far.view(torch.float8_e8m0fnu), w, sw, outs)
    check(a, sa, w, sw, outs)
