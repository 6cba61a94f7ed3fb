"""The three-part products of the training scan, on the host: what the parts hold, and that the bar the GPU tests hold
the scan to (scan_model.BAR) is below what any one lost partial product costs."""
import numpy as np
import pytest
import torch

from scan_model import BAR, KEPT, SCALE, Model, case, errors, exact, parts


def test_parts_add_up_and_what_is_left_out_is_below_an_fp32_step():
    g = torch.Generator().manual_seed(1)
    x, y = (1 + torch.rand(1 << 18, generator=g) for _ in range(2))
    edge = torch.tensor([1 + 2.0 ** -7 - 2.0 ** -23, 1.0, 2 - 2.0 ** -23, 1 + 2.0 ** -8 + 2.0 ** -17, 1 + 2.0 ** -8 - 2.0 ** -23])
    x, y = torch.cat([x, edge, edge]), torch.cat([y, edge, edge.flip(0)])
    px, py = parts(x), parts(y)
    assert torch.equal(px[0] + px[1] + px[2], x.double())
    whole = x.double() * y.double()
    lost = (sum(px[i] * py[j] for i, j in KEPT) - whole) / whole
    assert float(lost.abs().max()) < 2.0 ** -23
    assert abs(float(lost.mean())) < 2.0 ** -24 / 50  # of either sign
    # the parts of magnitudes down to where the last one becomes subnormal
    small = x * 2.0 ** -109
    assert torch.equal(sum(parts(small)), small.double())
    assert float(parts(small)[2].abs()[parts(small)[2] != 0].min()) >= float(np.finfo(np.float32).smallest_subnormal)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_every_partial_product_shows(dtype):
    x, dout, dfinal = case(dtype)
    want = exact(x, dout, dfinal)
    model = Model()
    assert max(errors(model.scan(x, SCALE, dout, dfinal), want).values()) < BAR / 4  # the algebra itself
    rounded = errors(Model(rounded=True).scan(x, SCALE, dout, dfinal), want)
    assert max(rounded.values()) < BAR / 2, rounded
    assert len(model.seen) == 21 and sum(map(len, model.seen.values())) == (21 * 6 if dtype == torch.float32 else 77)
    for name, formed in model.seen.items():
        for i, j in formed:
            e = errors(Model((name, i, j)).scan(x, SCALE, dout, dfinal), want)
            assert max(e.values()) > 1.2 * BAR, (name, i, j, e)
