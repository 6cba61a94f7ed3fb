"""Nothing beside what the row-pool calls are given is written: pools, tables and counts lie in larger buffers of known
values, which are compared after every call; rows end inside a copy's 32 KiB tiles, before, at and behind their ends."""
import pytest
import torch

from gated_deltanet_recurrence_gdn_amd import binding as gb
from helpers import DEV, say
from test_gpu_pool import host, ints, ref_compact, ref_copy, ref_fork, same

pytestmark = pytest.mark.gpu
PAD = 16384  # elements on either side: two tiles of float32


class Guarded:
    """Tensors with guards on either side."""

    def __init__(self):
        self.all = []

    def put(self, t, pad=PAD):
        fill = 77 if t.dtype == torch.int32 else -3.5
        whole = torch.full((t.numel() + 2 * pad,), fill, dtype=t.dtype, device=DEV)
        self.all.append((whole, pad, fill))
        inner = whole[pad:pad + t.numel()].view(t.shape)
        inner.copy_(t)
        return inner

    def check(self):
        for whole, pad, fill in self.all:
            assert bool((whole[:pad] == fill).all()) and bool((whole[-pad:] == fill).all())


TILE = 32768 // 4
ROWS = [4, TILE - 4, TILE, TILE + 4, 2 * TILE, 2 * TILE + 1020, 3 * TILE - 4]


@pytest.mark.parametrize("row", ROWS)
@pytest.mark.parametrize("layers", [1, 3])
def test_first_and_last_rows(row, layers):
    say("guards", row, layers)
    slots, g = 5, Guarded()
    pools = [g.put(torch.randn(layers, slots, row, device=DEV)), g.put(torch.randn(layers, slots, 8 * 9, device=DEV).to(torch.bfloat16))]
    other = [g.put(torch.randn_like(p)) for p in pools]
    st = g.put(ints([0]), 64)
    want, frm = host(pools), host(other)
    ref_copy(want, want, [1, -1], [4, 0], True)
    gb.gdn_pool_copy(pools, ints([1, -1]), ints([4, 0]), status=st)
    same(pools, want)
    ref_copy(want, frm, [0, 4, 2], [4, 0, 2], False)
    gb.gdn_pool_copy(pools, ints([0, 4, 2]), ints([4, 0, 2]), src_pools=other, status=st)
    same(pools, want)
    same(other, frm)
    # the last free row is the pool's last: row 4
    table = [0, 1, 3, -1, -1]
    t, out = g.put(ints(table), 64), g.put(ints([9] * 5), 64)
    more, _ = ref_fork(want, table, [1, -1], [3, 4], [], slots)
    gb.gdn_pool_fork(pools, t, ints([1, -1]), ints([3, 4]), table_out=out, status=st)
    same(pools, want)
    assert out.tolist() == more and t.tolist() == table
    count = g.put(ints([0]), 64)
    last, live, _ = ref_compact(want, more, [0, 2], slots)
    gb.gdn_pool_compact(pools, out, released=ints([0, 2]), count=count, status=st)
    same(pools, want)
    assert out.tolist() == last and count.tolist() == [live] and st.tolist() == [0]
    g.check()


@pytest.mark.parametrize("seqs,rows", [(1, 1), (63, 64), (1025, 2000), (8192, 65536)])
def test_tables_of_all_sizes(seqs, rows):
    g = Guarded()
    pool = g.put(torch.arange(rows * 4, device=DEV, dtype=torch.float32).view(1, rows, 4))
    t, count, st = g.put(ints([rows - 1 - i for i in range(seqs)]), 64), g.put(ints([0]), 64), g.put(ints([0]), 64)
    workspace = g.put(torch.full(((16 + 8 * rows) // 4,), 5, dtype=torch.int32, device=DEV), 64)
    gb.gdn_pool_compact(pool, t, count=count, workspace=workspace, status=st)
    # the m-th row in use at or above the count goes to the m-th free row below it
    want = sorted(range(rows - seqs, rows))
    free = [r for r in range(seqs) if r < rows - seqs]
    to = dict(zip([r for r in want if r >= seqs], free))
    assert t.tolist() == [to.get(rows - 1 - i, rows - 1 - i) for i in range(seqs)] and count.tolist() == [seqs] and st.tolist() == [0]
    for a, b in list(to.items())[::max(1, len(to) // 50)]:
        assert pool[0, b].tolist() == [4 * a, 4 * a + 1, 4 * a + 2, 4 * a + 3]
    g.check()
    if seqs < rows:
        n = min(seqs, rows - seqs)
        fork_ws = g.put(torch.full((2 * n,), 5, dtype=torch.int32, device=DEV), 64)
        gb.gdn_pool_fork(pool, t, ints([0] * n), ints(list(range(n))), released=ints(list(range(n))), workspace=fork_ws, status=st)
        assert t.tolist()[:n] == list(range(seqs, seqs + n)) and st.tolist() == [0]
        g.check()
