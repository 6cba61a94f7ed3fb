"""The row-pool entry points on the GPU against row-by-row copies on the host: contents and tables exactly."""
import numpy as np
import pytest
import torch

from gated_deltanet_recurrence_gdn_amd import binding as gb
from helpers import DEV, say

pytestmark = pytest.mark.gpu
SLOT = gb.CODES["GDN_ERR_SLOT"]


def ints(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device=DEV)


def make_pools(seed, layers, slots, h=2, d=32, channels=24):
    """Recurrent states (fp32) and convolution histories (bf16), and a guard row around each."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [torch.randn(layers, slots, h, d, d, generator=g, device=DEV),
            torch.randn(layers, slots, 3, channels, generator=g, device=DEV).to(torch.bfloat16)]


def host(pools):
    return [p.float().cpu() for p in pools]


def same(pools, want):
    for p, w in zip(pools, want):
        assert torch.equal(p.float().cpu(), w)


def status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def ref_copy(dst, src, s, d, within):
    old = [x.clone() for x in src]
    bad = False
    for i, (a, b) in enumerate(zip(s, d)):
        clash = any(j != i and (d[j] == b or (within and s[j] == b)) for j in range(len(s)))
        if a < -1 or a >= src[0].shape[1] or b < -1 or b >= dst[0].shape[1] or (b >= 0 and clash):
            bad = True
        elif b >= 0:
            for x, o in zip(dst, old):
                x[:, b] = 0 if a < 0 else o[:, a]
    return bad


def ref_fork(pools, table, parent, child, released, n_rows):
    old, m, slots, bad = [p.clone() for p in pools], len(table), pools[0].shape[1], False
    free = [r for r in range(n_rows) if r not in table]
    out = list(table)
    for s in released:
        if 0 <= s < m:
            out[s] = -1
        else:
            bad = True
    bad |= any(r < -1 or r >= slots for r in table)
    seen = set()
    for i, (p, c) in enumerate(zip(parent, child)):
        ok = i < len(free) and 0 <= c < m and -1 <= p < m and c not in seen
        if 0 <= c < m:
            seen.add(c)
        ok = ok and (table[c] == -1 or c in released)
        row = table[p] if ok and p >= 0 else -1
        ok = ok and (p < 0 or 0 <= row < slots)
        if not ok:
            bad = True
            continue
        out[c] = free[i]
        for x, o in zip(pools, old):
            x[:, free[i]] = 0 if p < 0 else o[:, row]
    return out, bad


def ref_compact(pools, table, released, n_rows):
    old, slots = [p.clone() for p in pools], pools[0].shape[1]
    bad = any(not 0 <= s < len(table) for s in released) or any(r < -1 or r >= slots for r in table)
    out = [-1 if i in released else r for i, r in enumerate(table)]
    live = sorted({r for r in out if 0 <= r < n_rows})
    n = len(live)
    to = dict(zip([r for r in live if r >= n], [r for r in range(n) if r not in live]))
    for a, b in to.items():
        for x, o in zip(pools, old):
            x[:, b] = o[:, a]
    return [to.get(r, r) for r in out], n, bad


@pytest.mark.parametrize("layers,slots,s,d", [
    (1, 4, [2], [0]),
    (3, 9, [1, 1, 1, 8], [0, 4, 7, 2]),            # one source many times
    (2, 9, [-1, 3, 5], [6, -1, 5]),                # a fresh row, a pair passed over, a row onto itself
    (2, 9, [0, 1, 2, 3], [4, 4, 5, 6]),            # two pairs with one destination: neither is copied
    (2, 9, [0, 4, 2], [4, 5, 6]),                  # a destination that another pair reads: not copied
    (2, 9, [0, 9, -2, 2], [1, 3, 4, 9]),           # rows outside the pool
    (1, 700, list(range(300)), list(range(399, 699))),
])
def test_copy(layers, slots, s, d):
    say("pool copy", layers, slots, len(s))
    pools, st = make_pools(1, layers, slots), status()
    want = host(pools)
    bad = ref_copy(want, want, s, d, True)
    gb.gdn_pool_copy(pools, ints(s), ints(d), status=st)
    same(pools, want)
    assert int(st.item()) == (SLOT if bad else 0)


def test_copy_between_pools_and_rows_of_odd_sizes():
    # row sizes from one 16-byte piece to several tiles and a rest
    shapes = [(1, 5, 4), (3, 5, 2, 8192), (2, 5, 3, 8200), (4, 5, 20484), (0, 5, 4)]
    g = torch.Generator(device=DEV).manual_seed(3)
    dst = [torch.randn(*s, generator=g, device=DEV) for s in shapes]
    src = [torch.randn(s[0], 7, *s[2:], generator=g, device=DEV) for s in shapes]
    want, frm = host(dst), host(src)
    s, d = [6, 6, 0, -1], [4, 0, 2, 1]
    assert not ref_copy(want, frm, s, d, False)
    st = status()
    gb.gdn_pool_copy(dst, ints(s), ints(d), src_pools=src, status=st)
    same(dst, want)
    same(src, frm)
    # a destination named twice, also between pools
    assert ref_copy(want, frm, [1, 2, 3], [0, 0, 4], False)
    gb.gdn_pool_copy(dst, ints([1, 2, 3]), ints([0, 0, 4]), src_pools=src, status=st)
    same(dst, want)
    assert int(st.item()) == SLOT


def test_copy_in_pools_with_layers_apart():
    whole = torch.randn(6, 8, 2, 16, device=DEV)
    want = whole.cpu().clone()
    want[1:5:2, 3] = want[1:5:2, 0]
    gb.gdn_pool_copy(whole[1:5:2], ints([0]), ints([3]))
    assert torch.equal(whole.cpu(), want)
    want[:, 1] = want[:, 4]
    gb.gdn_pool_copy(whole[:, :5], ints([4]), ints([1]))
    assert torch.equal(whole.cpu(), want)


def test_copy_past_four_gigabytes():
    """Rows whose offsets pass 32 bits."""
    p = torch.zeros(2, 700, 1 << 20, device=DEV)  # 5.9 GB, the second layer beyond 2^31 bytes
    p[:, 699] = torch.arange(1 << 20, device=DEV, dtype=torch.float32)
    gb.gdn_pool_copy(p, ints([699]), ints([650]))
    assert torch.equal(p[:, 650], p[:, 699]) and not bool(p[:, 649].any()) and not bool(p[:, 651].any())


FORKS = [
    ([0, 3, -1, -1], [1, 1], [2, 3], [], 8, 8),
    ([5, 2, -1, -1, -1], [0, -1, 1], [4, 2, 3], [0], 8, 8),        # a released parent, a fresh child
    ([5, 2, 7], [0, 0], [1, 2], [1, 2], 8, 8),                      # children in released places
    ([5, 2, 7], [0], [1], [], 8, 8),                                # the child holds a row: nothing
    ([0, 1, -1, -1, -1], [0, 0, 1], [2, 2, 3], [], 8, 8),           # a child named twice: the first
    ([0, 1, -1, -1], [2, -2, 4, 1], [3, 3, 3, 2], [], 8, 8),        # parents without a row or outside
    ([0, 1, -1, -1, -1], [0, 0, 0], [2, 3, 4], [], 4, 8),           # two free rows for three children
    ([0, 9, 2, -1], [1, 0], [3, 2], [2, 7, -1], 6, 10),             # a parent beyond n_rows; releases outside
    ([0, 12, -5, -1, -1], [0, 1], [3, 4], [], 8, 10),               # table entries outside the pool
    ([4, 4, 4, -1], [2], [3], [0, 1], 8, 8),                        # a shared row
    ([1, 2], [], [], [1], 4, 4),                                    # only a release
    ([-1], [-1], [0], [], 1, 1),
]


@pytest.mark.parametrize("table,parent,child,released,n_rows,slots", FORKS)
@pytest.mark.parametrize("in_place", [False, True])
def test_fork(table, parent, child, released, n_rows, slots, in_place):
    say("pool fork", table, parent, child, released, n_rows, slots)
    pools, st = make_pools(2, 2, slots), status()
    want = host(pools)
    want_table, bad = ref_fork(want, table, parent, child, released, n_rows)
    t = ints(table)
    out = t if in_place else torch.full_like(t, 77)
    gb.gdn_pool_fork(pools, t, ints(parent), ints(child), released=ints(released), n_rows=n_rows,
                     table_out=None if in_place else out, status=st)
    same(pools, want)
    assert out.tolist() == want_table
    assert int(st.item()) == (SLOT if bad else 0)
    if not in_place:
        assert t.tolist() == table


COMPACTS = [
    ([0, 1, 2], [], 8, 8),
    ([7, 1, 5, -1], [], 8, 8),
    ([7, 1, 5, 0, 6], [3, 1], 8, 8),
    ([7, 7, 2, 7, 2], [0], 8, 8),                    # shared rows
    ([9, 3, 8], [1], 6, 10),                         # rows beyond n_rows stay
    ([-1, -1], [0], 4, 4),
    ([3, 12, -7], [5], 8, 10),                       # entries and releases outside
    ([], [], 5, 5),
    ([0], [], 1, 1),
]


@pytest.mark.parametrize("table,released,n_rows,slots", COMPACTS)
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(table, released, n_rows, slots, in_place):
    say("pool compact", table, released, n_rows, slots)
    pools, st = make_pools(3, 2, slots), status()
    want = host(pools)
    want_table, live, bad = ref_compact(want, table, released, n_rows)
    t, count = ints(table), torch.full((1,), -3, dtype=torch.int32, device=DEV)
    out = t if in_place else torch.full_like(t, 77)
    gb.gdn_pool_compact(pools, t, released=ints(released), n_rows=n_rows, table_out=None if in_place else out,
                        count=count, status=st)
    same(pools, want)
    assert out.tolist() == want_table and int(count.item()) == live
    assert int(st.item()) == (SLOT if bad else 0)


@pytest.mark.parametrize("rows,seqs", [(31, 20), (32, 32), (33, 17), (1000, 700), (65536, 8192)])
def test_large_tables(rows, seqs):
    r = np.random.RandomState(rows)
    say("large tables", rows, seqs)
    pools = [torch.arange(rows * 4, device=DEV, dtype=torch.float32).reshape(1, rows, 4)]
    table = r.permutation(rows)[:seqs].tolist()
    released = r.permutation(seqs)[:seqs // 3].tolist()
    want = host(pools)
    t = ints(table)
    want_table, live, _ = ref_compact(want, table, set(released), rows)
    count = torch.zeros(1, dtype=torch.int32, device=DEV)
    gb.gdn_pool_compact(pools, t, released=ints(released), count=count)
    same(pools, want)
    assert t.tolist() == want_table and int(count.item()) == live
    # the released places filled again, each from a running sequence or fresh, in one call
    n = min(len(released), rows - live)
    keep = [i for i in range(seqs) if want_table[i] >= 0]
    parent = [int(p) for p in r.choice(keep + [-1], n)]
    more, bad = ref_fork_fast(want, want_table, parent, released[:n], rows)
    st = status()
    gb.gdn_pool_fork(pools, t, ints(parent), ints(released[:n]), status=st)
    same(pools, want)
    assert t.tolist() == more and int(st.item()) == 0 and not bad


def ref_fork_fast(pools, table, parent, child, n_rows):
    used = set(table)
    free = [r for r in range(n_rows) if r not in used]
    out = list(table)
    old = pools[0].clone()
    for i, (p, c) in enumerate(zip(parent, child)):
        out[c] = free[i]
        pools[0][:, free[i]] = 0 if p < 0 else old[:, table[p]]
    return out, False


def test_fork_and_compact_on_another_stream_and_in_a_graph():
    pools = make_pools(5, 2, 12)
    table = [4, 9, -1, -1, 11]
    want = host(pools)
    side = torch.cuda.Stream()
    t = ints(table)
    parent, child, released = ints([0, -1]), ints([2, 3]), ints([1])
    torch.cuda.synchronize()
    w1, _ = ref_fork(want, table, [0, -1], [2, 3], [1], 12)
    gb.gdn_pool_fork(pools, t, parent, child, released=released, stream=side)
    w2, live, _ = ref_compact(want, w1, [], 12)
    gb.gdn_pool_compact(pools, t, stream=side)
    side.synchronize()
    same(pools, want)
    assert t.tolist() == w2
    # captured: table -> table_out, so every replay does the same; eager work in between
    t0, t1, t2 = ints(table), ints(table), ints(table)
    pools = make_pools(6, 2, 12)
    start = [p.clone() for p in pools]
    count = torch.zeros(1, dtype=torch.int32, device=DEV)

    def step():
        gb.gdn_pool_fork(pools, t0, parent, child, released=released, table_out=t1)
        gb.gdn_pool_compact(pools, t1, table_out=t2, count=count)
        gb.gdn_pool_copy(pools, ints_src, ints_dst)

    ints_src, ints_dst = ints([0]), ints([11])
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    with torch.cuda.graph(graph):
        step()
    eager = None
    for _ in range(4):
        for p, o in zip(pools, start):
            p.copy_(o)
        step()
        torch.cuda.synchronize()
        eager = host(pools), t1.tolist(), t2.tolist()
        for p, o in zip(pools, start):
            p.copy_(o)
        t1.fill_(5)
        t2.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        same(pools, eager[0])
        assert (t1.tolist(), t2.tolist()) == eager[1:]


def test_prepared_calls():
    pools = make_pools(8, 1, 6)
    want = host(pools)
    call = gb.gdn_pool_copy(pools, ints([0]), ints([3]), prepare=True)
    fork = gb.gdn_pool_fork(pools, ints([0, -1]), ints([0]), ints([1]), prepare=True)
    torch.cuda.synchronize()
    same(pools, want)
    call()
    fork()
    for w in want:
        w[:, 3] = w[:, 0]
        w[:, 1] = w[:, 0]
    same(pools, want)
