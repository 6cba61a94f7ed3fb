"""The row-pool entry points on the host: every request here is refused (or empty) before any HIP call."""
import pytest
import torch

from gated_deltanet_recurrence_gdn_amd import binding as gb

E = gb.CODES
FAKE = 0x1000000  # 16-byte aligned, never dereferenced


def pool(data=FAKE, row=64, layers=2, slots=8, layer=None):
    return gb.GdnPool(data, row, row * slots if layer is None else layer, layers, slots)


def pools(*p):
    return (gb.GdnPool * max(1, len(p)))(*p)


def copy(dst, src=None, n_pools=None, s=FAKE, d=FAKE, n=3, status=None):
    return gb.lib().gdn_pool_copy(dst, src, len(dst) if n_pools is None else n_pools, s, d, n, status, None)


def fork(p, n_pools=None, table=FAKE, m=4, rows=8, rel=FAKE, n_rel=1, parent=FAKE, child=FAKE, n=2, out=FAKE, ws=FAKE,
         ws_bytes=1 << 20, status=None):
    return gb.lib().gdn_pool_fork(p, len(p) if n_pools is None else n_pools, table, m, rows, rel, n_rel, parent, child, n,
                                  out, ws, ws_bytes, status, None)


def compact(p, n_pools=None, table=FAKE, m=4, rows=8, rel=FAKE, n_rel=1, out=FAKE, count=None, ws=FAKE, ws_bytes=1 << 20,
            status=None):
    return gb.lib().gdn_pool_compact(p, len(p) if n_pools is None else n_pools, table, m, rows, rel, n_rel, out, count, ws,
                                     ws_bytes, status, None)


BAD_POOLS = [
    (pool(row=0), "GDN_ERR_SHAPE"),
    (pool(row=8), "GDN_ERR_SHAPE"),
    (pool(row=24), "GDN_ERR_SHAPE"),
    (pool(row=-16), "GDN_ERR_SHAPE"),
    (pool(slots=0), "GDN_ERR_SHAPE"),
    (pool(layers=-1), "GDN_ERR_SHAPE"),
    (pool(layer=64 * 7), "GDN_ERR_SHAPE"),
    (pool(layer=64 * 8 + 8), "GDN_ERR_SHAPE"),
    (pool(layer=-64 * 8), "GDN_ERR_SHAPE"),
    (pool(data=None), "GDN_ERR_NULL"),
    (pool(data=FAKE + 8), "GDN_ERR_ALIGN"),
]


@pytest.mark.parametrize("call", [copy, fork, compact])
@pytest.mark.parametrize("bad,code", BAD_POOLS)
def test_bad_pools_are_refused(call, bad, code):
    assert call(pools(bad)) == E[code]
    assert call(pools(pool(data=2 * FAKE), bad)) == E[code]


@pytest.mark.parametrize("call", [copy, fork, compact])
def test_pool_sets(call):
    assert call(pools(pool()), n_pools=0) == E["GDN_ERR_SHAPE"]
    assert call(pools(*[pool(data=FAKE * (i + 1)) for i in range(9)])) == E["GDN_ERR_SHAPE"]
    assert call(None, n_pools=1) == E["GDN_ERR_NULL"]
    assert call(pools(pool(), pool(data=2 * FAKE, slots=9))) == E["GDN_ERR_SHAPE"]     # another number of rows
    assert call(pools(pool(), pool(data=FAKE + 64))) == E["GDN_ERR_SHAPE"]             # pools that overlap


def test_copy_refusals():
    p = pools(pool())
    assert copy(p, n=-1) == E["GDN_ERR_SHAPE"]
    assert copy(p, n=0, s=None, d=None) == 0
    assert copy(p, s=None) == E["GDN_ERR_NULL"] and copy(p, d=None) == E["GDN_ERR_NULL"]
    assert copy(p, s=FAKE + 2) == E["GDN_ERR_ALIGN"] and copy(p, status=FAKE + 1) == E["GDN_ERR_ALIGN"]
    far = 4 * FAKE
    assert copy(p, src=pools(pool(data=far, row=128))) == E["GDN_ERR_SHAPE"]
    assert copy(p, src=pools(pool(data=far, layers=1))) == E["GDN_ERR_SHAPE"]
    assert copy(p, src=pools(pool(data=FAKE + 64))) == E["GDN_ERR_SHAPE"]              # overlaps the destination
    assert copy(p, src=p) == E["GDN_ERR_SHAPE"]
    assert copy(p, src=pools(pool(data=None))) == E["GDN_ERR_NULL"]
    # more tiles than the copy counts
    assert copy(pools(pool(row=1 << 30, slots=1)), n=1 << 20) == E["GDN_ERR_SHAPE"]
    # no layers: nothing to read
    assert copy(pools(pool(data=None, layers=0)), n=0) == 0


def test_fork_refusals():
    p = pools(pool())
    assert fork(p, m=-1) == E["GDN_ERR_SHAPE"] and fork(p, m=8193) == E["GDN_ERR_SHAPE"]
    assert fork(p, rows=0) == E["GDN_ERR_SHAPE"] and fork(p, rows=9) == E["GDN_ERR_SHAPE"]
    assert fork(p, n_rel=-1) == E["GDN_ERR_SHAPE"] and fork(p, n=-1) == E["GDN_ERR_SHAPE"]
    assert fork(p, n=8193) == E["GDN_ERR_SHAPE"]
    for name in ("table", "rel", "parent", "child", "out"):
        assert fork(p, **{name: None}) == E["GDN_ERR_NULL"], name
    for name in ("table", "rel", "parent", "child", "out", "status"):
        assert fork(p, **{name: FAKE + 2}) == E["GDN_ERR_ALIGN"], name
    assert fork(p, ws=None) == E["GDN_ERR_WORKSPACE"] and fork(p, ws_bytes=15) == E["GDN_ERR_WORKSPACE"]
    assert fork(p, ws=FAKE + 4) == E["GDN_ERR_ALIGN"]
    assert fork(p, out=FAKE + 4) == E["GDN_ERR_SHAPE"]  # half over the table
    assert fork(p, m=0, n=0, n_rel=0, table=None, rel=None, parent=None, child=None, out=None, ws=None, ws_bytes=0) == 0
    assert fork(pools(pool(row=16, slots=70000)), rows=65537) == E["GDN_ERR_SHAPE"]
    assert gb.lib().gdn_pool_fork_workspace_bytes(5) == 40 and gb.lib().gdn_pool_fork_workspace_bytes(-1) == 0


def test_compact_refusals():
    p = pools(pool())
    for kw in (dict(m=-1), dict(m=8193), dict(rows=0), dict(rows=9), dict(n_rel=-1), dict(out=FAKE + 8)):
        assert compact(p, **kw) == E["GDN_ERR_SHAPE"], kw
    for name in ("table", "rel", "out"):
        assert compact(p, **{name: None}) == E["GDN_ERR_NULL"], name
    for name in ("table", "rel", "out", "count", "status"):
        assert compact(p, **{name: FAKE + 2}) == E["GDN_ERR_ALIGN"], name
    need = gb.lib().gdn_pool_compact_workspace_bytes(8)
    assert need == 16 + 64
    assert compact(p, ws=None) == E["GDN_ERR_WORKSPACE"] and compact(p, ws_bytes=need - 1) == E["GDN_ERR_WORKSPACE"]
    assert compact(p, ws=FAKE + 4) == E["GDN_ERR_ALIGN"]


def i32(*x):
    return torch.tensor(x, dtype=torch.int32)


def test_binding_checks_tensors():
    p = torch.zeros(2, 4, 8)
    t = i32(0, 1, -1)
    with pytest.raises(TypeError, match="device tensors"):
        gb.gdn_pool_copy(p, i32(0), i32(1))
    with pytest.raises(TypeError, match="device tensors"):
        gb.gdn_pool_fork(p, t, i32(0), i32(2))
    with pytest.raises(TypeError, match="device tensors"):
        gb.gdn_pool_compact(p, t)
    for bad in (torch.zeros(4, 8), torch.zeros(2, 4, 16)[:, :, ::2], torch.zeros(2, 8, 4).transpose(1, 2),
                torch.zeros(2, 8, 8)[:, ::2], torch.zeros(2, 0, 8), torch.zeros(2, 4, 0)):
        with pytest.raises(ValueError):
            gb.gdn_pool_copy(bad, i32(0), i32(1))
    with pytest.raises(ValueError, match="same number of rows"):
        gb.gdn_pool_copy((p, torch.zeros(2, 5, 8)), i32(0), i32(1))
    with pytest.raises(ValueError):
        gb.gdn_pool_copy([], i32(0), i32(1))
    with pytest.raises(ValueError):
        gb.gdn_pool_copy(p, i32(0), i32(1, 2))
    with pytest.raises(TypeError):
        gb.gdn_pool_copy(p, i32(0).long(), i32(1))
    with pytest.raises(ValueError, match="src_pools"):
        gb.gdn_pool_copy(p, i32(0), i32(1), src_pools=torch.zeros(2, 4, 16))
    with pytest.raises(ValueError):
        gb.gdn_pool_fork(p, t, i32(0), i32(2, 1))
    with pytest.raises(ValueError, match="n_rows"):
        gb.gdn_pool_fork(p, t, i32(0), i32(2), n_rows=5)
    with pytest.raises(ValueError, match="table_out"):
        gb.gdn_pool_fork(p, t, i32(0), i32(2), table_out=i32(0))
    with pytest.raises(ValueError, match="count"):
        gb.gdn_pool_compact(p, t, count=i32(0, 0))
    with pytest.raises(ValueError, match="at most"):
        gb.gdn_pool_compact(p, torch.zeros(8193, dtype=torch.int32))


def test_layers_may_be_apart():
    whole = torch.zeros(4, 6, 8)
    s, _ = gb._pool_structs(whole[::2])
    assert (s[0].row_bytes, s[0].layer_bytes, s[0].n_layers, s[0].n_slots) == (32, 2 * 6 * 32, 2, 6)
    s, _ = gb._pool_structs(whole[:, :3])
    assert (s[0].row_bytes, s[0].layer_bytes, s[0].n_layers, s[0].n_slots) == (32, 6 * 32, 4, 3)


@pytest.mark.parametrize("call", [copy, fork, compact])
def test_pools_larger_than_any_memory_are_refused(call):
    for p in (pool(row=1 << 40, slots=1 << 30, layers=1), pool(row=1 << 20, slots=8, layers=1 << 30, layer=1 << 46)):
        assert call(pools(p)) == E["GDN_ERR_SHAPE"]
