"""Pools whose layers lie between one another's (a model's states and convolution histories kept layer by layer in one
allocation, the two halves of every layer's rows): they share no byte and are taken; pools that do are refused."""
import random

import pytest
import torch

from gated_deltanet_recurrence_gdn_amd import binding as gb
from test_gpu_pool import host, ints, ref_compact, ref_copy, ref_fork, same, status
from test_pool_host import E, FAKE, compact, copy, fork, pool, pools


def ranges(p):
    return [(p.data + l * p.layer_bytes, p.data + l * p.layer_bytes + p.n_slots * p.row_bytes) for l in range(p.n_layers)]


def shares_a_byte(p, q):
    return any(a < d and c < b for a, b in ranges(p) for c, d in ranges(q))


def accepted(p, src=None):
    """What the checks say, of calls that have nothing to do."""
    none = dict(m=0, n_rel=0, table=None, rel=None, out=None)
    r = {copy(p, src=src, n=0, s=None, d=None)}
    if src is None:
        r |= {fork(p, n=0, parent=None, child=None, rows=1, ws=None, ws_bytes=0, **none)}
        no_workspace = compact(p, rows=1, ws=None, ws_bytes=0, **none)  # refused next, where the pools stand
        r |= {0 if no_workspace == E["GDN_ERR_WORKSPACE"] else no_workspace}
    assert len(r) == 1
    return r.pop() == 0


def test_layers_between_layers():
    state, history = pool(row=64, slots=4, layers=3, layer=512), pool(data=FAKE + 256, row=48, slots=4, layers=3, layer=512)
    assert accepted(pools(state, history)) and accepted(pools(history, state))
    assert accepted(pools(state), src=pools(pool(data=FAKE + 256, row=64, slots=4, layers=3, layer=512)))
    for shift in (-16, 16):  # one piece into the layer before it, or into the next one
        assert not accepted(pools(state, pool(data=FAKE + 256 + shift, row=64, slots=4, layers=3, layer=512)))
    # one layer inside a gap, before, behind and across
    for at, ok in ((256, True), (512 + 256, True), (-64, True), (1024 + 256, True), (1024 + 240, False), (-48, False), (255 + 1 - 16, False)):
        assert accepted(pools(state, pool(data=FAKE + at, row=16, slots=4, layers=1))) == ok, at


def test_random_layouts():
    r, seen = random.Random(4), [0, 0]
    for _ in range(4000):
        slots = r.randint(1, 4)

        def one():
            row = 16 * r.randint(1, 4)
            return pool(data=FAKE + 16 * r.randint(0, 80), row=row, slots=slots, layers=r.randint(0, 5),
                        layer=row * slots + 16 * r.choice([0, 1, 8, 20, 33]))

        p, q = one(), one()
        want = not shares_a_byte(p, q)
        assert accepted(pools(p, q)) == want, (ranges(p), ranges(q))
        q.row_bytes, q.n_layers = p.row_bytes, p.n_layers
        q.layer_bytes = max(q.layer_bytes, q.row_bytes * slots)
        want2 = not shares_a_byte(p, q)
        assert accepted(pools(p), src=pools(q)) == want2
        seen[want] += 1
    assert min(seen) > 500


def one_allocation(seed, layers=3, slots=8, h=2, d=32, channels=24):
    """States and histories of one layer after the other in one buffer, and the buffer."""
    a, b = slots * h * d * d, slots * 3 * channels
    g = torch.Generator(device="cuda:0").manual_seed(seed)
    whole = torch.randn(layers, a + b + 8, generator=g, device="cuda:0")
    return whole, [whole[:, :a].unflatten(1, (slots, h, d, d)), whole[:, a:a + b].unflatten(1, (slots, 3, channels))]


@pytest.mark.gpu
def test_states_and_histories_of_one_allocation():
    whole, p = one_allocation(7)
    rest = whole[:, -8:].clone()
    want, st = host(p), status()
    ref_copy(want, want, [2, -1], [5, 0], True)
    gb.gdn_pool_copy(p, ints([2, -1]), ints([5, 0]), status=st)
    same(p, want)
    table = [5, 2, 7, -1, -1]
    t = ints(table)
    more, _ = ref_fork(want, table, [0, 2], [3, 4], [1], 8)
    gb.gdn_pool_fork(p, t, ints([0, 2]), ints([3, 4]), released=ints([1]), status=st)
    same(p, want)
    assert t.tolist() == more
    last, live, _ = ref_compact(want, more, [0], 8)
    gb.gdn_pool_compact(p, t, released=ints([0]), status=st)
    same(p, want)
    assert t.tolist() == last and int(st.item()) == 0 and torch.equal(whole[:, -8:], rest)


@pytest.mark.gpu
def test_from_one_half_of_every_layer_to_the_other():
    whole = torch.randn(4, 10, 2, 16, device="cuda:0")
    want = whole.cpu().clone()
    want[:, 5 + 3] = want[:, 1]
    want[:, 5] = 0
    st = status()
    gb.gdn_pool_copy(whole[:, 5:], ints([1, -1]), ints([3, 0]), src_pools=whole[:, :5], status=st)
    assert torch.equal(whole.cpu(), want) and int(st.item()) == 0
