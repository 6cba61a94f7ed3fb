"""Prefills whose last chunk is part of one, with NaN behind the last token: it is not read."""
import numpy as np
import pytest
import torch

from gated_deltanet_recurrence_gdn_amd import binding as gb
from helpers import DEV

pytestmark = pytest.mark.gpu


def behind(x, rows, value):
    """A copy of x [tokens][heads][d] with `rows` more tokens of a value behind it."""
    whole = torch.full((x.shape[0] + rows, *x.shape[1:]), value, dtype=x.dtype, device=DEV)
    whole[:x.shape[0]] = x
    return whole[:x.shape[0]]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("Hqk,Hv,dk,dv", [(1, 3, 128, 128), (2, 4, 64, 64), (1, 2, 32, 32)])
@pytest.mark.parametrize("lens", [[1], [17], [33], [47], [65], [100], [64, 30], [70, 1, 129]])
def test_nothing_behind_the_last_token(lens, Hqk, Hv, dk, dv, dtype):
    g = torch.Generator(device=DEV).manual_seed(sum(lens))
    total, cu = sum(lens), np.cumsum([0] + lens).astype(np.int32)
    normal = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    q, k = (torch.nn.functional.normalize(normal(total, Hqk, dk), dim=-1).to(dtype) for _ in range(2))
    v = normal(total, Hv, dv).to(dtype)
    alpha, beta = torch.sigmoid(normal(total, Hv) + 2), torch.sigmoid(normal(total, Hv))
    state = normal(len(lens), Hv, dv, dk)
    results = []
    for value in (0.0, float("nan")):
        out, final = torch.full((total, Hv, dv), 7.0, device=DEV), state.clone()
        args = [behind(t, 64, value) for t in (q, k, v, alpha, beta)]
        gb.gdn_prefill_varlen(cu, *args, final, out, scale=dk ** -0.5)
        results.append((out, final))
    assert results[0][0].isfinite().all() and results[0][1].isfinite().all()
    assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1])
