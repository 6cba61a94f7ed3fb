"""The training scan's entry points on the host: every request here is refused (or empty) before any HIP call."""
import ctypes

import numpy as np
import pytest
import torch

from gated_deltanet_recurrence_gdn_amd import binding as gb

E = gb.CODES
FAKE = 0x1000000  # 16-byte aligned, never dereferenced
BIG = 1 << 40


def shape(**kw):
    d = dict(batch=2, n_nodes=100, h_qk=2, h_v=4, d_k=64, d_v=48, n_slots=3, qkv_dtype=gb.GDN_BF16, out_dtype=gb.GDN_F32,
             persist_dtype=gb.GDN_F16, scale=1.0)
    d.update(kw)
    return gb.GdnShape(*[d[f] for f, _ in gb.GdnShape._fields_])


CU = np.array([0, 30, 100], np.int32)
NAMES_F = ("q", "k", "v", "alpha", "beta", "state", "slot", "out", "final")


def forward(sh=None, cu=CU, tape=FAKE, tape_bytes=BIG, ws=FAKE, ws_bytes=BIG, status=None, **kw):
    p = dict.fromkeys(NAMES_F, FAKE)
    p["final"] = 2 * FAKE
    p.update(kw)
    sh = shape() if sh is None else sh
    return gb.lib().gdn_scan_forward(ctypes.byref(sh), None if cu is None else cu.ctypes.data, *[p[n] for n in NAMES_F], tape,
                                     tape_bytes, ws, ws_bytes, status, None)


NAMES_B = ("dout", "dfinal", "dq", "dk", "dv", "dalpha", "dbeta", "dstate")


def backward(sh=None, cu=CU, tape=FAKE, tape_bytes=BIG, ws=FAKE, ws_bytes=BIG, **kw):
    p = dict.fromkeys(("q", "k", "v", "alpha", "beta") + NAMES_B, FAKE)
    p.update(kw)
    sh = shape() if sh is None else sh
    return gb.lib().gdn_scan_backward(ctypes.byref(sh), None if cu is None else cu.ctypes.data,
                                      *[p[n] for n in ("q", "k", "v", "alpha", "beta")], tape, tape_bytes,
                                      *[p[n] for n in NAMES_B], ws, ws_bytes, None)


@pytest.mark.parametrize("call", [forward, backward])
@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), "GDN_ERR_SHAPE"), (dict(n_nodes=-1), "GDN_ERR_SHAPE"), (dict(n_nodes=99), "GDN_ERR_SHAPE"),
    (dict(h_qk=0), "GDN_ERR_SHAPE"), (dict(h_v=3), "GDN_ERR_SHAPE"), (dict(h_v=0), "GDN_ERR_SHAPE"),
    (dict(d_k=96), "GDN_ERR_SHAPE"), (dict(d_k=256), "GDN_ERR_SHAPE"), (dict(d_v=8), "GDN_ERR_SHAPE"),
    (dict(d_v=40), "GDN_ERR_SHAPE"), (dict(d_v=272), "GDN_ERR_SHAPE"), (dict(scale=float("inf")), "GDN_ERR_SHAPE"),
    (dict(qkv_dtype=gb.GDN_F16), "GDN_ERR_DTYPE"), (dict(out_dtype=7), "GDN_ERR_DTYPE"),
    (dict(batch=0), "GDN_ERR_SHAPE"), (dict(h_qk=1 << 29, h_v=1 << 30), "GDN_ERR_SHAPE"),
])
def test_shapes_are_refused(call, kw, code):
    assert call(shape(**kw)) == E[code]


@pytest.mark.parametrize("call", [forward, backward])
def test_offsets_are_refused(call):
    assert call(cu=None) == E["GDN_ERR_NULL"]
    for cu in ([1, 30, 100], [0, 101, 100], [0, 30, 101], [0, -1, 100]):
        assert call(cu=np.array(cu, np.int32)) == E["GDN_ERR_SHAPE"]


@pytest.mark.parametrize("call,names", [(forward, NAMES_F), (backward, ("q", "k", "v", "alpha", "beta") + NAMES_B)])
def test_pointers_are_refused(call, names):
    for n in names:
        if n not in ("state", "slot", "final", "dfinal", "dstate"):
            assert call(**{n: None}) == E["GDN_ERR_NULL"], n
        assert call(**{n: FAKE + 2}) == E["GDN_ERR_ALIGN"], n
    for n in ("q", "k", "v"):
        assert call(**{n: FAKE + 8}) == E["GDN_ERR_ALIGN"], n


def test_tapes_and_workspaces_are_refused():
    sh, L = shape(), gb.lib()
    p, c = ctypes.byref(sh), CU.ctypes.data
    tape, fwd, alone, bwd = (L.gdn_scan_tape_bytes(p, c), L.gdn_scan_forward_workspace_bytes(p, c, 1),
                             L.gdn_scan_forward_workspace_bytes(p, c, 0), L.gdn_scan_backward_workspace_bytes(p, c))
    units = 1 + 2  # 30 and 70 tokens
    assert tape >= units * 4 * 4 * (64 * 64 + 64 * 48 + 64 * 48) and alone == tape + fwd and bwd > 0
    assert forward(ws=None) == E["GDN_ERR_WORKSPACE"] and forward(ws_bytes=fwd - 1) == E["GDN_ERR_WORKSPACE"]
    assert forward(tape_bytes=tape - 1) == E["GDN_ERR_WORKSPACE"]
    assert forward(tape=None, tape_bytes=0, ws_bytes=alone - 1) == E["GDN_ERR_WORKSPACE"]
    assert forward(ws=FAKE + 4) == E["GDN_ERR_ALIGN"] and forward(tape=FAKE + 4) == E["GDN_ERR_ALIGN"]
    assert backward(tape=None) == E["GDN_ERR_WORKSPACE"] and backward(tape_bytes=tape - 1) == E["GDN_ERR_WORKSPACE"]
    assert backward(ws=None) == E["GDN_ERR_WORKSPACE"] and backward(ws_bytes=bwd - 1) == E["GDN_ERR_WORKSPACE"]
    assert backward(ws=FAKE + 4) == E["GDN_ERR_ALIGN"]


def test_slots_and_empty_calls():
    assert forward(shape(n_slots=0)) == E["GDN_ERR_SHAPE"]
    assert forward(final=FAKE) == E["GDN_ERR_SHAPE"]  # in place through slots
    empty = np.zeros(1, np.int32)
    none = dict.fromkeys(NAMES_F)
    assert forward(shape(batch=0, n_nodes=0), empty, tape=None, ws=None, **none) == 0
    assert backward(shape(batch=0, n_nodes=0), empty, tape=None, ws=None) == 0
    assert gb.lib().gdn_scan_tape_bytes(ctypes.byref(shape(batch=0, n_nodes=0)), empty.ctypes.data) == 0
    assert gb.lib().gdn_scan_tape_bytes(ctypes.byref(shape(d_k=48)), CU.ctypes.data) == 0


def test_binding_checks_tensors():
    bf = torch.bfloat16
    x = dict(q=torch.zeros(6, 2, 32, dtype=bf), k=torch.zeros(6, 2, 32, dtype=bf), v=torch.zeros(6, 4, 16, dtype=bf),
             alpha=torch.zeros(6, 4), beta=torch.zeros(6, 4), out=torch.zeros(6, 4, 16))
    cu = [0, 2, 6]

    def fwd(cu=cu, **kw):
        y = {**x, **{n: kw.pop(n) for n in list(kw) if n in x}}
        return gb.gdn_scan_forward(cu, y["q"], y["k"], y["v"], y["alpha"], y["beta"], y["out"],
                                   workspace=torch.zeros(16, dtype=torch.uint8), **kw)

    with pytest.raises(TypeError, match="device tensor"):
        fwd()
    for bad in (dict(k=torch.zeros(6, 2, 64, dtype=bf)), dict(v=torch.zeros(5, 4, 16, dtype=bf)), dict(alpha=torch.zeros(6, 3)),
                dict(out=torch.zeros(6, 4, 32)), dict(cu=[0, 2, 5]), dict(cu=[[0, 6]]), dict(out=None),
                dict(state=torch.zeros(1, 4, 16, 32)), dict(final_state=torch.zeros(3, 4, 16, 32)),
                dict(state_slot=torch.zeros(2, dtype=torch.int32)), dict(status=torch.zeros(0, dtype=torch.int32))):
        with pytest.raises(ValueError):
            fwd(**bad)
    for bad in (dict(k=torch.zeros(6, 2, 32)), dict(alpha=torch.zeros(6, 4, dtype=bf)), dict(out=torch.zeros(6, 4, 16, dtype=torch.int32)),
                dict(tape=torch.zeros(8)), dict(q=torch.zeros(6, 2, 32, dtype=torch.float16), k=torch.zeros(6, 2, 32, dtype=torch.float16),
                                                v=torch.zeros(6, 4, 16, dtype=torch.float16))):
        with pytest.raises(TypeError):
            fwd(**bad)

    def bwd(**kw):
        y = {**x, "dout": x["out"], "dq": x["q"], "dk": x["k"], "dv": x["v"], "dalpha": x["alpha"], "dbeta": x["beta"],
             "tape": torch.zeros(16, dtype=torch.uint8), **kw}
        return gb.gdn_scan_backward(cu, *(y[n] for n in ("q", "k", "v", "alpha", "beta", "tape", "dout", "dq", "dk", "dv", "dalpha", "dbeta")),
                                    dfinal=y.get("dfinal"), dstate=y.get("dstate"), workspace=torch.zeros(16, dtype=torch.uint8))

    with pytest.raises(TypeError, match="device tensor"):
        bwd()
    for bad in (dict(dq=None), dict(dq=torch.zeros(6, 2, 64, dtype=bf)), dict(dv=torch.zeros(6, 4, 32, dtype=bf)), dict(dout=None),
                dict(dalpha=torch.zeros(6, 2)), dict(dfinal=torch.zeros(1, 4, 16, 32)), dict(dstate=torch.zeros(2, 4, 32, 16))):
        with pytest.raises(ValueError):
            bwd(**bad)
    for bad in (dict(dq=torch.zeros(6, 2, 32)), dict(dbeta=torch.zeros(6, 4, dtype=bf)), dict(dstate=torch.zeros(2, 4, 16, 32, dtype=bf))):
        with pytest.raises(TypeError):
            bwd(**bad)
