"""The training scan of sequences that all have no tokens: the size queries say that it needs no workspace, so none is
asked for, and the states pass through."""
import numpy as np
import pytest
import torch

from gated_deltanet_recurrence_gdn_amd import binding as gb
from helpers import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("with_state", [True, False])
def test_no_tokens_no_workspace(with_state):
    cu = np.zeros(4, np.int32)
    q, v, gate = (torch.empty(0, *s, device=DEV) for s in ((2, 64), (4, 48), (4,)))
    none = torch.empty(0, dtype=torch.uint8, device=DEV)
    state, final, dfinal, dstate = (torch.randn(3, 4, 48, 64, device=DEV) for _ in range(4))
    tape = torch.empty(gb.gdn_scan_tape_bytes(cu, q, v), dtype=torch.uint8, device=DEV)
    assert tape.numel() > 0
    gb.gdn_scan_forward(cu, q, q, v, gate, gate, torch.empty_like(v), tape=tape, state=state if with_state else None,
                        final_state=final, workspace=none)
    assert torch.equal(final, state) if with_state else not bool(final.any())
    gb.gdn_scan_backward(cu, q, q, v, gate, gate, tape, v, torch.empty_like(q), torch.empty_like(q), torch.empty_like(v),
                         torch.empty_like(gate), torch.empty_like(gate), dfinal=dfinal, dstate=dstate, workspace=none)
    assert torch.equal(dstate, dfinal)
