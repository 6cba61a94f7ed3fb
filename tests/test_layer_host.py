"""The norms, the projections and the 8-bit rows on the host: every request here is refused (or empty) before any HIP
call."""
import ctypes

import pytest
import torch

from gated_deltanet_recurrence_gdn_amd import binding as gb

E = gb.CODES
FAKE = 0x1000000  # 16-byte aligned, never dereferenced
NAN, INF = float("nan"), float("inf")


def norm(x=FAKE, residual=None, weight=FAKE, residual_out=None, out=FAKE, codes=None, scales=None, rows=4, x_stride=256,
         width=256, dtype=1, residual_dtype=1, weight_dtype=0, scale_stride=4, eps=1e-6, offset=0.0):
    sh = gb.GdnNormShape(rows, x_stride, width, dtype, residual_dtype, weight_dtype, scale_stride, eps, offset)
    return gb.lib().gdn_norm_forward(ctypes.byref(sh), x, residual, weight, residual_out, out, codes, scales, None)


def norm_back(dout=FAKE, r=FAKE, weight=FAKE, dresidual=None, dx=FAKE, dweight=FAKE, ws=FAKE, ws_bytes=1 << 24, rows=4,
              x_stride=256, width=256, dtype=1, residual_dtype=1, weight_dtype=0, eps=1e-6, offset=0.0):
    sh = gb.GdnNormShape(rows, x_stride, width, dtype, residual_dtype, weight_dtype, 0, eps, offset)
    return gb.lib().gdn_norm_backward(ctypes.byref(sh), dout, r, weight, dresidual, dx, dweight, ws, ws_bytes, None)


@pytest.mark.parametrize("call", [norm, norm_back])
@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), "GDN_ERR_SHAPE"), (dict(rows=1 << 31), "GDN_ERR_SHAPE"), (dict(width=0, x_stride=0), "GDN_ERR_SHAPE"),
    (dict(width=252), "GDN_ERR_SHAPE"), (dict(width=16392, x_stride=16392), "GDN_ERR_SHAPE"), (dict(x_stride=248), "GDN_ERR_SHAPE"),
    (dict(x_stride=260), "GDN_ERR_SHAPE"), (dict(x_stride=1 << 40), "GDN_ERR_SHAPE"), (dict(eps=-1.0), "GDN_ERR_SHAPE"),
    (dict(eps=NAN), "GDN_ERR_SHAPE"), (dict(eps=INF), "GDN_ERR_SHAPE"), (dict(offset=NAN), "GDN_ERR_SHAPE"),
    (dict(offset=-INF), "GDN_ERR_SHAPE"), (dict(dtype=3), "GDN_ERR_DTYPE"), (dict(residual_dtype=-1), "GDN_ERR_DTYPE"),
    (dict(weight_dtype=7), "GDN_ERR_DTYPE"), (dict(weight=None), "GDN_ERR_NULL"), (dict(weight=FAKE + 4), "GDN_ERR_ALIGN"),
])
def test_norm_shapes(call, kw, code):
    assert call(**kw) == E[code]


def test_norm_refusals():
    assert gb.lib().gdn_norm_forward(None, *[FAKE] * 7, None) == E["GDN_ERR_NULL"]
    assert norm(x=None) == E["GDN_ERR_NULL"] and norm(out=None) == E["GDN_ERR_NULL"]
    assert norm(codes=FAKE) == E["GDN_ERR_NULL"] and norm(scales=FAKE) == E["GDN_ERR_NULL"]
    assert norm(residual_out=FAKE) == E["GDN_ERR_NULL"]  # nothing to keep without a residual
    for name in ("x", "residual", "residual_out", "out"):
        assert norm(**{"residual": FAKE, name: FAKE + 8}) == E["GDN_ERR_ALIGN"], name
    assert norm(codes=FAKE + 4, scales=FAKE) == E["GDN_ERR_ALIGN"] and norm(codes=FAKE, scales=FAKE + 2) == E["GDN_ERR_ALIGN"]
    assert norm(codes=FAKE, scales=FAKE, scale_stride=6) == E["GDN_ERR_SHAPE"]
    assert norm(codes=FAKE, scales=FAKE, width=640, x_stride=640) == E["GDN_ERR_SHAPE"]
    assert norm(rows=0, x=None, weight=None, out=None) == 0


def test_norm_backward_refusals():
    assert norm_back(dout=None) == E["GDN_ERR_NULL"] and norm_back(r=None) == E["GDN_ERR_NULL"]
    assert norm_back(dx=None, dweight=None) == E["GDN_ERR_NULL"]
    for name in ("dout", "r", "dresidual", "dx", "dweight", "ws"):
        assert norm_back(**{name: FAKE + 8}) == E["GDN_ERR_ALIGN"], name
    need = gb.lib().gdn_norm_backward_workspace_bytes(ctypes.byref(gb.GdnNormShape(4, 256, 256, 1, 1, 0, 0, 1e-6, 0.0)))
    assert need > 0 and need % (4 * 256) == 0
    assert norm_back(ws=None) == E["GDN_ERR_WORKSPACE"] and norm_back(ws_bytes=need - 1) == E["GDN_ERR_WORKSPACE"]
    assert norm_back(rows=0, dweight=None, dout=None, r=None, weight=None, ws=None) == 0
    assert gb.lib().gdn_norm_backward_workspace_bytes(ctypes.byref(gb.GdnNormShape(4, 256, 250, 1, 1, 0, 0, 1e-6, 0.0))) == 0


def gated(x=FAKE, z=FAKE, weight=FAKE, out=FAKE, codes=None, scales=None, rows=4, x_stride=256, z_stride=256, h_v=2, d_v=128,
          x_dtype=0, z_dtype=1, weight_dtype=0, scale_stride=4, eps=1e-6):
    sh = gb.GdnGatedNormShape(rows, x_stride, z_stride, h_v, d_v, x_dtype, z_dtype, weight_dtype, scale_stride, eps)
    return gb.lib().gdn_gated_norm_forward(ctypes.byref(sh), x, z, weight, out, codes, scales, None)


def gated_back(dout=FAKE, x=FAKE, z=FAKE, weight=FAKE, dx=FAKE, dz=FAKE, dweight=FAKE, ws=FAKE, ws_bytes=1 << 24, rows=4,
               x_stride=256, z_stride=256, h_v=2, d_v=128, x_dtype=0, z_dtype=1, weight_dtype=0, eps=1e-6):
    sh = gb.GdnGatedNormShape(rows, x_stride, z_stride, h_v, d_v, x_dtype, z_dtype, weight_dtype, 0, eps)
    return gb.lib().gdn_gated_norm_backward(ctypes.byref(sh), dout, x, z, weight, dx, dz, dweight, ws, ws_bytes, None)


@pytest.mark.parametrize("call", [gated, gated_back])
@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), "GDN_ERR_SHAPE"), (dict(rows=1 << 31), "GDN_ERR_SHAPE"), (dict(h_v=0), "GDN_ERR_SHAPE"),
    (dict(h_v=(1 << 20) + 1, x_stride=1 << 31, z_stride=1 << 31), "GDN_ERR_SHAPE"),
    (dict(d_v=8), "GDN_ERR_SHAPE"), (dict(d_v=120), "GDN_ERR_SHAPE"), (dict(d_v=272, h_v=1, x_stride=272, z_stride=272), "GDN_ERR_SHAPE"),
    (dict(x_stride=248), "GDN_ERR_SHAPE"), (dict(z_stride=260), "GDN_ERR_SHAPE"), (dict(z_stride=0), "GDN_ERR_SHAPE"),
    # more pieces than the kernels count
    (dict(rows=(1 << 31) - 1, h_v=64, x_stride=8192, z_stride=8192), "GDN_ERR_SHAPE"),
    (dict(eps=-1.0), "GDN_ERR_SHAPE"), (dict(eps=NAN), "GDN_ERR_SHAPE"), (dict(x_dtype=3), "GDN_ERR_DTYPE"),
    (dict(z_dtype=3), "GDN_ERR_DTYPE"), (dict(weight_dtype=-1), "GDN_ERR_DTYPE"), (dict(x=None), "GDN_ERR_NULL"),
    (dict(z=None), "GDN_ERR_NULL"), (dict(weight=None), "GDN_ERR_NULL"), (dict(x=FAKE + 8), "GDN_ERR_ALIGN"),
    (dict(z=FAKE + 8), "GDN_ERR_ALIGN"), (dict(weight=FAKE + 4), "GDN_ERR_ALIGN"),
])
def test_gated_norm_shapes(call, kw, code):
    assert call(**kw) == E[code]


def test_gated_norm_refusals():
    assert gated(out=None) == E["GDN_ERR_NULL"] and gated(codes=FAKE) == E["GDN_ERR_NULL"]
    assert gated(out=FAKE + 8) == E["GDN_ERR_ALIGN"] and gated(codes=FAKE + 4, scales=FAKE) == E["GDN_ERR_ALIGN"]
    assert gated(codes=FAKE, scales=FAKE, scale_stride=2) == E["GDN_ERR_SHAPE"]
    assert gated(rows=0, x=None, z=None, weight=None, out=None) == 0
    assert gated_back(dx=None, dz=None, dweight=None) == E["GDN_ERR_NULL"] and gated_back(dout=None) == E["GDN_ERR_NULL"]
    for name in ("dout", "dx", "dz", "dweight", "ws"):
        assert gated_back(**{name: FAKE + 8}) == E["GDN_ERR_ALIGN"], name
    need = gb.lib().gdn_gated_norm_backward_workspace_bytes(ctypes.byref(gb.GdnGatedNormShape(4, 256, 256, 2, 128, 0, 1, 0, 0, 1e-6)))
    assert need > 0 and need % 512 == 0
    assert gated_back(ws=None) == E["GDN_ERR_WORKSPACE"] and gated_back(ws_bytes=need - 1) == E["GDN_ERR_WORKSPACE"]
    assert gated_back(rows=0, dweight=None, dout=None, x=None, z=None, weight=None, ws=None) == 0


def part(data=FAKE, columns=64, stride=None, reserved=0):
    return gb.GdnProjectPart(data, columns if stride is None else stride, columns, reserved)


def project(parts=None, n_parts=None, a=FAKE, a_scales=FAKE, w=FAKE, w_scales=FAKE, tokens=4, a_stride=256, w_stride=256,
            inner=256, a_scale_stride=4, w_scale_stride=4, w_scale_dtype=0, out_dtype=1):
    parts = [part()] if parts is None else parts
    sh = gb.GdnProjectShape(tokens, a_stride, w_stride, inner, a_scale_stride, w_scale_stride, w_scale_dtype, out_dtype)
    return gb.lib().gdn_project(ctypes.byref(sh), a, a_scales, w, w_scales, (gb.GdnProjectPart * max(1, len(parts)))(*parts),
                                len(parts) if n_parts is None else n_parts, None)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), "GDN_ERR_SHAPE"), (dict(tokens=1 << 31), "GDN_ERR_SHAPE"), (dict(inner=0), "GDN_ERR_SHAPE"),
    (dict(inner=-16), "GDN_ERR_SHAPE"), (dict(inner=248), "GDN_ERR_SHAPE"), (dict(a_stride=240), "GDN_ERR_SHAPE"),
    (dict(w_stride=264), "GDN_ERR_SHAPE"), (dict(a_stride=1 << 40), "GDN_ERR_SHAPE"), (dict(a_scale_stride=2), "GDN_ERR_SHAPE"),
    (dict(inner=640, a_stride=640, w_stride=640), "GDN_ERR_SHAPE"), (dict(w_scale_stride=1), "GDN_ERR_SHAPE"),
    (dict(w_scale_stride=6, w_scale_dtype=3), "GDN_ERR_SHAPE"), (dict(w_scale_dtype=1), "GDN_ERR_DTYPE"),
    (dict(out_dtype=0), "GDN_ERR_DTYPE"), (dict(out_dtype=3), "GDN_ERR_DTYPE"), (dict(a=None), "GDN_ERR_NULL"),
    (dict(a_scales=None), "GDN_ERR_NULL"), (dict(w=None), "GDN_ERR_NULL"), (dict(w_scales=None), "GDN_ERR_NULL"),
    (dict(a=FAKE + 8), "GDN_ERR_ALIGN"), (dict(w=FAKE + 8), "GDN_ERR_ALIGN"), (dict(a_scales=FAKE + 1), "GDN_ERR_ALIGN"),
    (dict(w_scales=FAKE + 2), "GDN_ERR_ALIGN"), (dict(n_parts=0), "GDN_ERR_SHAPE"), (dict(parts=[part()] * 9), "GDN_ERR_SHAPE"),
    (dict(parts=[part(), part(columns=0)]), "GDN_ERR_SHAPE"), (dict(parts=[part(stride=63)]), "GDN_ERR_SHAPE"),
    (dict(parts=[part(reserved=1)]), "GDN_ERR_SHAPE"), (dict(parts=[part(data=None)]), "GDN_ERR_NULL"),
    (dict(parts=[part(data=FAKE + 1)]), "GDN_ERR_ALIGN"),
    (dict(parts=[part(columns=1 << 30), part(columns=1 << 30)]), "GDN_ERR_SHAPE"),
    (dict(parts=[part(columns=1 << 27), part(columns=1)]), "GDN_ERR_SHAPE"), (dict(a_scale_stride=1 << 23), "GDN_ERR_SHAPE"),
    (dict(w_stride=(1 << 22) + 16), "GDN_ERR_SHAPE"), (dict(tokens=(1 << 31) - 1, parts=[part(columns=256)]), "GDN_ERR_SHAPE"),
    (dict(tokens=1 << 20, parts=[part(columns=1 << 18)]), "GDN_ERR_SHAPE"),
])
def test_project_refusals(kw, code):
    assert project(**kw) == E[code]


def test_project_empty():
    assert project(tokens=0, a=None, a_scales=None, w=None, w_scales=None, parts=[part(data=None)]) == 0
    assert gb.lib().gdn_project(None, FAKE, FAKE, FAKE, FAKE, None, 1, None) == E["GDN_ERR_NULL"]


def pool(data, row, layers=2, slots=8):
    return gb.GdnPool(data, row, row * slots, layers, slots)


def pack_pools(n=64, dk=32, size=4, **over):
    p = {"states": pool(FAKE, n * dk * size), "codes": pool(4 * FAKE, n * dk), "scales": pool(8 * FAKE, 4 * n)}
    p.update(over)
    return p


def pack(name="gdn_pool_pack", p=None, dk=32, dtype=0, src=FAKE, dst=FAKE, n=3, status=None):
    p = pack_pools() if p is None else p
    refs = {k: None if v is None else ctypes.byref(v) for k, v in p.items()}
    order = ("states", "codes", "scales") if name == "gdn_pool_pack" else ("codes", "scales", "states")
    return getattr(gb.lib(), name)(*[refs[k] for k in order], dk, dtype, src, dst, n, status, None)


@pytest.mark.parametrize("name", ["gdn_pool_pack", "gdn_pool_unpack"])
def test_pack_refusals(name):
    shape, null = E["GDN_ERR_SHAPE"], E["GDN_ERR_NULL"]
    for k in ("states", "codes", "scales"):
        assert pack(name, pack_pools(**{k: None})) == null, k
        assert pack(name, pack_pools(**{k: pool(None, 64)})) == null, k
        assert pack(name, pack_pools(**{k: pool(FAKE + 8, 64)})) == E["GDN_ERR_ALIGN"], k
        assert pack(name, pack_pools(**{k: pool(2 * FAKE, 24)})) == shape, k
    assert pack(name, dk=48) == shape and pack(name, dk=64) == shape and pack(name, dtype=3) == E["GDN_ERR_DTYPE"]
    assert pack(name, dtype=1) == shape  # the rows are those of fp32 states
    assert pack(name, pack_pools(codes=pool(4 * FAKE, 64 * 32, slots=9))) == shape
    assert pack(name, pack_pools(codes=pool(4 * FAKE, 64 * 32, layers=3))) == shape
    assert pack(name, pack_pools(scales=pool(8 * FAKE, 256, layers=1))) == shape
    assert pack(name, pack_pools(scales=pool(8 * FAKE, 512))) == shape
    assert pack(name, pack_pools(codes=pool(FAKE + 64, 64 * 32))) == shape      # overlaps the states
    assert pack(name, pack_pools(scales=pool(4 * FAKE + 16, 256))) == shape     # overlaps the codes
    assert pack(name, n=-1) == shape
    assert pack(name, src=None) == null and pack(name, dst=None) == null
    for k in ("src", "dst", "status"):
        assert pack(name, **{k: FAKE + 2}) == E["GDN_ERR_ALIGN"], k
    assert pack(name, n=0, src=None, dst=None) == 0
    empty = {"states": pool(None, 64 * 32 * 4, layers=0), "codes": pool(None, 64 * 32, layers=0), "scales": pool(None, 256, layers=0)}
    assert pack(name, empty, src=None, dst=None) == 0
    big = {"states": gb.GdnPool(FAKE, 1 << 39, 1 << 39, 1, 1), "codes": gb.GdnPool(1 << 44, 1 << 37, 1 << 37, 1, 1),
           "scales": gb.GdnPool(1 << 45, 1 << 34, 1 << 34, 1, 1)}
    assert pack(name, big, n=1 << 20) == shape  # more tiles than the kernels count


def z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_refuses_host_tensors():
    with pytest.raises(TypeError, match="device tensor"):
        gb.gdn_norm_forward(z(4, 64), z(64), out=z(4, 64))
    with pytest.raises(TypeError, match="device tensor"):
        gb.gdn_norm_backward(z(4, 64), z(4, 64), z(64), z(4, 64))
    with pytest.raises(TypeError, match="device tensor"):
        gb.gdn_gated_norm_forward(z(4, 2, 64), z(4, 2, 64), z(64), out=z(4, 2, 64))
    with pytest.raises(TypeError, match="device tensor"):
        gb.gdn_gated_norm_backward(z(4, 2, 64), z(4, 2, 64), z(4, 2, 64), z(64), z(4, 2, 64))
    with pytest.raises(TypeError, match="device tensor"):
        f8 = z(4, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
        gb.gdn_project(f8, f8[:, :4].contiguous().view(torch.float8_e8m0fnu), f8, z(1, 1), z(4, 4, dtype=torch.bfloat16))
    p, c, s = z(2, 4, 2, 16, 32), z(2, 4, 2, 16, 32, dtype=torch.int8), z(2, 4, 2, 16)
    i = z(1, dtype=torch.int32)
    with pytest.raises(TypeError, match="device tensors"):
        gb.gdn_pool_pack(p, c, s, i, i)
    with pytest.raises(TypeError, match="device tensors"):
        gb.gdn_pool_unpack(c, s, p, i, i)


def test_pack_binding_checks():
    p, c, s = z(2, 4, 2, 16, 32), z(2, 5, 2, 16, 32, dtype=torch.int8), z(2, 5, 2, 16)
    i = z(1, dtype=torch.int32)
    for bad in (dict(p=z(2, 4, 2, 16)), dict(c=c[:, :, :1]), dict(c=c.to(torch.uint8)), dict(s=s[:, :4]), dict(s=s.half()),
                dict(p=p.double()), dict(i=i.long()), dict(p=p.transpose(1, 2))):
        a = {"p": p, "c": c, "s": s, "i": i, **bad}
        with pytest.raises((ValueError, TypeError)):
            gb.gdn_pool_pack(a["p"], a["c"], a["s"], a["i"], i)
        with pytest.raises((ValueError, TypeError)):
            gb.gdn_pool_unpack(a["c"], a["s"], a["p"], a["i"], i)


def test_scales_like():
    codes = z(3, 640, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = gb.gdn_scales_like(codes)
    assert s.shape == (3, 8) and s.dtype is torch.float8_e8m0fnu


def pretend(monkeypatch):
    """Host tensors pass as device tensors where rows are measured: the checks behind that one, on the host."""
    monkeypatch.setattr(gb, "_rows_of", lambda t, name, tail: (t.shape[0], t.stride(0)))


@pytest.mark.parametrize("kw", [dict(weight=z(63)), dict(out=z(4, 65)), dict(out=z(4, 64, dtype=torch.float16)), dict(residual=z(3, 64)),
                                dict(residual=z(4, 64), residual_out=z(4, 64, dtype=torch.bfloat16)),
                                dict(codes=z(4, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)),
                                dict(codes=z(4, 64, dtype=torch.int8), scales=z(4, 4, dtype=torch.uint8).view(torch.float8_e8m0fnu)),
                                dict(codes=z(4, 64, dtype=torch.uint8).view(torch.float8_e4m3fn), scales=z(4, 4, dtype=torch.uint8)),
                                dict(codes=z(4, 64, dtype=torch.uint8).view(torch.float8_e4m3fn),
                                     scales=z(4, 3, dtype=torch.uint8).view(torch.float8_e8m0fnu)),
                                dict(x=z(4, 64, dtype=torch.float64))])
def test_norm_binding_checks(kw, monkeypatch):
    pretend(monkeypatch)
    a = {"x": z(4, 64), "weight": z(64), **kw}
    with pytest.raises((ValueError, TypeError)) as e:
        gb.gdn_norm_forward(a.pop("x"), a.pop("weight"), **a)
    assert "device" not in str(e.value)


@pytest.mark.parametrize("kw", [dict(z=z(4, 2, 32)), dict(weight=z(128)), dict(out=z(4, 2, 64, dtype=torch.float16)), dict(out=z(4, 128))])
def test_gated_norm_binding_checks(kw, monkeypatch):
    pretend(monkeypatch)
    a = {"x": z(4, 2, 64), "z": z(4, 2, 64), "weight": z(64), **kw}
    with pytest.raises((ValueError, TypeError)) as e:
        gb.gdn_gated_norm_forward(a.pop("x"), a.pop("z"), a.pop("weight"), **a)
    assert "device" not in str(e.value)


def f8(*shape):
    return z(*shape, dtype=torch.uint8).view(torch.float8_e4m3fn)


def e8(*shape):
    return z(*shape, dtype=torch.uint8).view(torch.float8_e8m0fnu)


@pytest.mark.parametrize("kw", [dict(a=z(4, 256)), dict(a=f8(4, 128)), dict(w=f8(300, 256).view(torch.uint8)), dict(a_scales=e8(4, 2)),
                                dict(a_scales=e8(3, 4)), dict(a_scales=z(4, 4, dtype=torch.uint8)), dict(w_scales=z(2, 2)),
                                dict(w_scales=z(3, 1)), dict(w_scales=e8(3, 2)), dict(w_scales=z(3, 2).half()), dict(outs=[]),
                                dict(outs=z(4, 300)), dict(outs=z(4, 299, dtype=torch.bfloat16)), dict(outs=z(5, 300, dtype=torch.bfloat16)),
                                dict(outs=[z(4, 150, dtype=torch.bfloat16), z(4, 150, dtype=torch.float16)])])
def test_project_binding_checks(kw, monkeypatch):
    pretend(monkeypatch)
    a = {"a": f8(4, 256), "a_scales": e8(4, 4), "w": f8(300, 256), "w_scales": z(3, 2), "outs": z(4, 300, dtype=torch.bfloat16), **kw}
    with pytest.raises((ValueError, TypeError)) as e:
        gb.gdn_project(*a.values())
    assert "device" not in str(e.value)
