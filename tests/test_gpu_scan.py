"""The training scan (gdn_scan_forward, gdn_scan_backward) against the rule token by token in float64.

Tolerance.  An output is the end of at most 6 chained products in fp32, each a sum of at most 256 terms whose rounding
errors (half a step, 2^-24 relative) are independent: 6 sqrt(256) 2^-24 = 5.7e-6 of the output's 2-norm, doubled for the
triangular inverse, whose norm is below 2 for normalised keys and beta <= 1.  An output in bf16 or fp16 adds half a step
of its type for every element.
"""
import numpy as np
import pytest
import torch

from gated_deltanet_recurrence_gdn_amd import binding as gb
from helpers import DEV, say
from scan_reference import reference, rule

pytestmark = pytest.mark.gpu
TOL = 2 * 6 * 16 * 2.0 ** -24
GUARD = 64


def tol(dtype):
    return TOL + (0.0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2)


def guarded(shape, dtype, fill=float("nan")):
    """An output with guard values behind it, and those."""
    n = int(np.prod(shape))
    flat = torch.full((n + GUARD,), fill, dtype=dtype, device=DEV)
    flat[n:] = 7.0
    return flat[:n].view(shape), flat[n:]


def inputs(seed, lens, hq, hv, dk, dv, dtype=torch.float32, alpha="mixed", beta="mixed"):
    g = torch.Generator(device=DEV).manual_seed(seed)
    total = sum(lens)

    def n(*s):
        return torch.randn(*s, generator=g, device=DEV)

    unit = lambda t: t / t.square().sum(-1, keepdim=True).sqrt().clamp(min=1e-6)  # noqa: E731
    x = {"q": unit(n(total, hq, dk)).to(dtype), "k": unit(n(total, hq, dk)).to(dtype), "v": n(total, hv, dv).to(dtype)}
    slow = torch.linspace(-5.0, 1.0, hv, device=DEV)
    x["alpha"] = torch.exp(-torch.nn.functional.softplus(slow + n(total, hv)))
    if alpha == "one":
        x["alpha"].fill_(1.0)
    elif alpha == "zeros":  # resets, several within one chunk, and gates far below fp32's resolution
        x["alpha"][torch.rand(total, hv, generator=g, device=DEV) < 0.1] = 0.0
        x["alpha"][torch.rand(total, hv, generator=g, device=DEV) < 0.1] = 1e-12
    elif alpha == "strong":
        x["alpha"] *= 0.05
    x["beta"] = torch.sigmoid(n(total, hv))
    if beta == "ends":  # exactly 0 and 1
        x["beta"][:, ::2] = (x["beta"][:, ::2] > 0.5).float()
    x["state"] = 0.1 * n(len(lens), hv, dv, dk)
    return x, n(total, hv, dv), 0.1 * n(len(lens), hv, dv, dk)


def offsets(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def forward(x, lens, out_dtype=torch.float32, scale=1.0, tape=True, final=True, state=True, **kw):
    cu = offsets(lens)
    out, og = guarded(x["v"].shape, out_dtype)
    fin, fg = guarded(x["state"].shape, torch.float32)
    tp = torch.full((gb.gdn_scan_tape_bytes(cu, x["q"], x["v"]),), 0xff, dtype=torch.uint8, device=DEV) if tape else None
    gb.gdn_scan_forward(cu, x["q"], x["k"], x["v"], x["alpha"], x["beta"], out, tape=tp,
                        state=x["state"] if state is True else state, final_state=fin if final else None, scale=scale, **kw)
    assert bool((og == 7).all()) and bool((fg == 7).all())
    return out, fin, tp


def backward(x, lens, tape, dout, dfinal, scale=1.0, dstate=True, **kw):
    grads, guards = {}, []
    for n in ("q", "k", "v", "alpha", "beta", "state"):
        grads["d" + n], gd = guarded(x[n].shape, x[n].dtype)
        guards.append(gd)
    gb.gdn_scan_backward(offsets(lens), x["q"], x["k"], x["v"], x["alpha"], x["beta"], tape, dout, grads["dq"], grads["dk"],
                         grads["dv"], grads["dalpha"], grads["dbeta"], dfinal=dfinal,
                         dstate=grads["dstate"] if dstate else None, scale=scale, **kw)
    assert all(bool((gd == 7).all()) for gd in guards)
    return grads


def off(a, b):
    """Relative 2-norm of the difference; the gradient of a gate is compared at its own scale."""
    a, b = a.double().cpu(), b.double()
    assert bool(torch.isfinite(a).all())
    return float((a - b).norm() / b.norm()) if float(b.norm()) > 0 else float(a.norm())


def check(x, lens, scale=1.0, out_dtype=torch.float32, dout=None, dfinal=None, state=True):
    ref_x = dict(x) if state else dict(x, state=torch.zeros_like(x["state"]))
    do = dout.to(out_dtype)
    ref = reference(ref_x, lens, scale, do, dfinal)
    out, fin, tape = forward(x, lens, out_dtype, scale, state=True if state else None)
    got = backward(x, lens, tape, do, dfinal, scale)
    got.update(out=out, final=fin)
    worst = {n: off(got[n], ref[n]) for n in got}
    say({n: f"{e:.1e}" for n, e in worst.items()})
    for n, e in worst.items():
        assert e <= tol(got[n].dtype), (n, e)
    return got


SHAPES = [
    # lens, hq, hv, dk, dv
    ([1], 1, 1, 32, 16),
    ([2, 0, 1], 1, 2, 32, 32),
    ([63, 64, 65], 2, 4, 64, 32),
    ([0, 0], 1, 1, 64, 16),
    ([130, 1, 0, 61], 3, 3, 64, 48),
    ([200], 1, 3, 128, 128),
    ([129, 5], 2, 4, 128, 80),
    ([70], 1, 5, 32, 256),
    ([97, 31], 4, 4, 128, 256),
]


@pytest.mark.parametrize("lens,hq,hv,dk,dv", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_matches_the_rule(lens, hq, hv, dk, dv, dtype):
    say("scan", lens, hq, hv, dk, dv, dtype)
    x, dout, dfinal = inputs(11, lens, hq, hv, dk, dv, dtype)
    check(x, lens, dk ** -0.5, dtype, dout, dfinal)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_output_types_without_states(dtype, out_dtype):
    lens = [77, 3]
    x, dout, _ = inputs(12, lens, 2, 4, 64, 64, dtype)
    check(x, lens, 1.0, out_dtype, dout, None, state=False)


@pytest.mark.parametrize("alpha,beta", [("one", "mixed"), ("zeros", "mixed"), ("strong", "mixed"), ("mixed", "ends"), ("zeros", "ends")])
def test_gates_at_their_ends(alpha, beta):
    lens = [150, 40]
    say("gates", alpha, beta)
    x, dout, dfinal = inputs(13, lens, 1, 4, 64, 64, alpha=alpha, beta=beta)
    got = check(x, lens, 1.0, torch.float32, dout, dfinal)
    if alpha == "zeros":  # the gates that are zero have gradients of their own, accurate by themselves
        ref = reference(x, lens, 1.0, dout, dfinal)["dalpha"]
        at = (x["alpha"] < 1e-9).cpu()
        assert off(got["dalpha"].cpu()[at], ref[at]) <= TOL


def test_long_sequence():
    lens = [1500]
    x, dout, dfinal = inputs(14, lens, 1, 2, 64, 32)
    check(x, lens, 0.125, torch.float32, dout, dfinal)


def test_many_sequences():
    """More sequences than one launch's tables hold, empty ones among them."""
    r = np.random.RandomState(3)
    lens = [int(n) for n in r.choice([0, 1, 2, 9, 64, 66], 150)]
    x, dout, dfinal = inputs(15, lens, 1, 2, 32, 16)
    check(x, lens, 1.0, torch.float32, dout, dfinal)


def test_large_values():
    """Values far outside the f16 range: everything scales."""
    lens = [90]
    x, dout, dfinal = inputs(16, lens, 1, 2, 64, 32)
    x["v"] *= 3e7
    x["state"] *= 3e7
    x["q"] *= 1e6
    check(x, lens, 1.0, torch.float32, dout * 1e-9, dfinal * 1e-9)


def test_gradient_against_differences():
    lens, scale, h = [70, 20], 0.5, 1e-4
    x, dout, dfinal = inputs(17, lens, 1, 2, 32, 32)
    _, _, tape = forward(x, lens, scale=scale)
    got = backward(x, lens, tape, dout, dfinal, scale)
    x64 = {n: t.double().cpu() for n, t in x.items()}
    g = torch.Generator().manual_seed(1)

    def loss(y):
        out, final = rule(y["q"], y["k"], y["v"], y["alpha"], y["beta"], y["state"], lens, scale)
        return float((out * dout.double().cpu()).sum() + (final * dfinal.double().cpu()).sum())

    for n in x64:
        d = torch.randn(x64[n].shape, generator=g, dtype=torch.float64)
        slope = (loss({**x64, n: x64[n] + h * d}) - loss({**x64, n: x64[n] - h * d})) / (2 * h)
        grad = got["d" + n].double().cpu()
        # the kernel's error is TOL of |grad|, in a random direction of |d| = sqrt(size); the difference's own error
        # is of second order in h, about h^2 of the third derivative: 1e-6 of the slope's scale covers it
        assert abs(float((grad * d).sum()) - slope) <= (TOL + 1e-6) * float(grad.norm()) * float(d.norm()), n


def test_state_slots():
    lens = [30, 70, 0, 5]
    x, dout, dfinal = inputs(18, lens, 1, 2, 32, 32)
    pool = torch.randn(6, 2, 32, 32, device=DEV)
    slot = torch.tensor([4, 1, 0, 4], dtype=torch.int32, device=DEV)
    out, fin, tape = forward(x, lens, state=pool, state_slot=slot)
    y = dict(x, state=pool[slot.long()])
    out2, fin2, tape2 = forward(y, lens)
    assert torch.equal(out, out2) and torch.equal(fin, fin2)
    # slots outside the pool: those sequences are left alone, forward and backward
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    bad = torch.tensor([4, 6, -1, 4], dtype=torch.int32, device=DEV)
    out3, fin3, tape3 = forward(x, lens, state=pool, state_slot=bad, status=status)
    assert int(status.item()) == gb.CODES["GDN_ERR_SLOT"]
    keep = torch.ones(105, dtype=torch.bool)
    keep[30:100] = False
    keep = keep.to(DEV)
    assert torch.equal(out3[keep], out[keep]) and bool(out3[~keep].isnan().all())
    assert torch.equal(fin3[[0, 3]], fin[[0, 3]]) and bool(fin3[[1, 2]].isnan().all())
    a, b = backward(x, lens, tape2, dout, dfinal), backward(x, lens, tape3, dout, dfinal)
    for n in ("dq", "dk", "dv", "dalpha", "dbeta"):
        assert torch.equal(a[n][keep], b[n][keep]) and bool(b[n][~keep].isnan().all()), n
    assert torch.equal(a["dstate"][[0, 3]], b["dstate"][[0, 3]]) and bool(b["dstate"][[1, 2]].isnan().all())


def test_results_repeat_and_the_tape_is_only_read():
    lens = [140, 66]
    x, dout, dfinal = inputs(19, lens, 2, 6, 128, 64, torch.bfloat16)
    do = dout.to(torch.bfloat16)
    out, fin, tape = forward(x, lens, torch.bfloat16)
    again = tape.clone()
    a = backward(x, lens, tape, do, dfinal)
    b = backward(x, lens, tape, do, dfinal)
    assert torch.equal(tape, again)
    out2, fin2, _ = forward(x, lens, torch.bfloat16, tape=False)
    assert torch.equal(out, out2) and torch.equal(fin, fin2)
    for n in a:
        assert torch.equal(a[n], b[n]), n
    # no gradient of the initial states asked for, no final states asked for: the rest is the same
    c = backward(x, lens, tape, do, dfinal, dstate=False)
    assert all(torch.equal(a[n], c[n]) for n in a if n != "dstate")
    assert torch.equal(forward(x, lens, torch.bfloat16, final=False)[0], out)


def test_in_place_final_state_and_a_sequence_in_two_calls():
    x, _, _ = inputs(20, [200], 1, 2, 64, 32)
    whole, fin, _ = forward(x, [200])
    parts, state = [], x["state"].clone()
    for a, b in ((0, 71), (71, 200)):
        y = {n: x[n][a:b].contiguous() for n in ("q", "k", "v", "alpha", "beta")}
        out = torch.empty(b - a, 2, 32, device=DEV)
        gb.gdn_scan_forward([0, b - a], y["q"], y["k"], y["v"], y["alpha"], y["beta"], out, state=state, final_state=state)
        parts.append(out)
    assert off(torch.cat(parts), whole.cpu()) <= 2 * TOL and off(state, fin.cpu()) <= 2 * TOL


def test_other_streams_two_at_once():
    """Two training steps at once on two streams, each with its own tape and workspaces."""
    lens = [300, 20]
    sets = [inputs(21 + i, lens, 2, 4, 64, 64) for i in range(2)]
    want = []
    for x, dout, dfinal in sets:
        out, fin, tape = forward(x, lens)
        want.append((out, fin, backward(x, lens, tape, dout, dfinal)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for st, (x, dout, dfinal) in zip(streams, sets):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            out, fin, tape = forward(x, lens)
            got.append((out, fin, backward(x, lens, tape, dout, dfinal)))
    torch.cuda.synchronize()
    for (o, f, g), (o2, f2, g2) in zip(want, got):
        assert torch.equal(o, o2) and torch.equal(f, f2) and all(torch.equal(g[n], g2[n]) for n in g)


def test_captured_training_step():
    lens = [100, 33]
    x, dout, dfinal = inputs(23, lens, 1, 3, 64, 32)
    cu = offsets(lens)
    out, fin = torch.empty_like(x["v"]), torch.empty_like(x["state"])
    tape = torch.empty(gb.gdn_scan_tape_bytes(cu, x["q"], x["v"]), dtype=torch.uint8, device=DEV)
    g = {n: torch.empty_like(t) for n, t in x.items()}

    def step():
        gb.gdn_scan_forward(cu, x["q"], x["k"], x["v"], x["alpha"], x["beta"], out, tape=tape, state=x["state"], final_state=fin)
        gb.gdn_scan_backward(cu, x["q"], x["k"], x["v"], x["alpha"], x["beta"], tape, dout, g["q"], g["k"], g["v"], g["alpha"],
                             g["beta"], dfinal=dfinal, dstate=g["state"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        other, d2, f2 = inputs(30 + i, lens, 1, 3, 64, 32)
        for n in x:
            x[n].copy_(other[n])
        dout.copy_(d2)
        dfinal.copy_(f2)
        step()
        torch.cuda.synchronize()
        eager = [out.clone(), fin.clone()] + [t.clone() for t in g.values()]
        for t in [out, fin] + list(g.values()):
            t.fill_(float("nan"))
        tape.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, [out, fin] + list(g.values())):
            assert torch.equal(a, b)


def test_agrees_with_the_prefill():
    """The serving path on the same inputs, at its own bar."""
    lens = [200, 64]
    x, _, _ = inputs(24, lens, 2, 4, 128, 128, torch.bfloat16)
    out, fin, _ = forward(x, lens)
    st = x["state"].clone()
    pre = torch.empty_like(out)
    gb.gdn_prefill_varlen(offsets(lens), x["q"], x["k"], x["v"], x["alpha"], x["beta"], st, pre)
    assert float((pre - out).abs().max() / out.abs().max()) <= 2e-3
    assert float((st - fin).abs().max() / fin.abs().max()) <= 2e-3


def test_sequences_forked_scanned_and_compacted():
    """Rows, scans and the serving calls together: a prompt's state kept in a row, forked twice, the forks continued
    through the index table, the pool closed up, and the continuation verified from where the rows went."""
    hq, hv, d, T, N = 1, 2, 64, 90, 6
    x, _, _ = inputs(25, [T + 2 * N + 2 * N], hq, hv, d, d, torch.bfloat16)
    cut = lambda a, b: {n: x[n][a:b].contiguous() for n in ("q", "k", "v", "alpha", "beta")}  # noqa: E731
    ref_in = {n: t.double().cpu() for n, t in x.items()}

    def ref(path):
        i = torch.cat([torch.arange(a, b) for a, b in path])
        y = {n: ref_in[n][i] for n in ("q", "k", "v", "alpha", "beta")}
        return rule(y["q"], y["k"], y["v"], y["alpha"], y["beta"], torch.zeros(1, hv, d, d, dtype=torch.float64), [len(i)], 1.0)

    pool = torch.full((1, 8, hv, d, d), float("nan"), device=DEV)
    table = torch.tensor([5, -1, -1], dtype=torch.int32, device=DEV)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    status = ints(0)
    # the prompt, from a fresh state, into row 5
    y, kept = cut(0, T), torch.empty(1, 1, hv, d, d, device=DEV)
    out = torch.empty(T, hv, d, device=DEV)
    gb.gdn_scan_forward([0, T], y["q"], y["k"], y["v"], y["alpha"], y["beta"], out, final_state=kept[0])
    gb.gdn_pool_copy(pool, ints(0), ints(5), src_pools=kept, status=status)
    # two continuations, the prompt's own sequence ends
    gb.gdn_pool_fork(pool, table, ints(0, 0), ints(1, 2), released=ints(0), status=status)
    assert table.tolist() == [-1, 0, 1]
    y = cut(T, T + 2 * N)
    out = torch.empty(2 * N, hv, d, device=DEV)
    fin = torch.empty(2, hv, d, d, device=DEV)
    gb.gdn_scan_forward([0, N, 2 * N], y["q"], y["k"], y["v"], y["alpha"], y["beta"], out, state=pool[0],
                        state_slot=table[1:].contiguous(), final_state=fin, status=status)
    for i in range(2):
        o, s = ref([(0, T), (T + i * N, T + (i + 1) * N)])
        assert off(out[i * N:(i + 1) * N], o[T:]) <= 2 * TOL and off(fin[i:i + 1], s) <= 2 * TOL
    gb.gdn_pool_copy(pool, ints(0, 1), ints(6, 3), src_pools=fin[None].contiguous(), status=status)
    table.copy_(ints(-1, 6, 3))
    count = ints(0)
    gb.gdn_pool_compact(pool, table, count=count, status=status)
    assert int(count.item()) == 2 and sorted(table.tolist()) == [-1, 0, 1]
    # the next block of each, verified through the table
    y = {n: t.view(2, N, *t.shape[1:]) for n, t in cut(T + 2 * N, T + 4 * N).items()}
    out = torch.empty(2, N, hv, d, device=DEV)
    gb.gdn_verify_chain(y["q"], y["k"], y["v"], y["alpha"], y["beta"], pool[0], out=out,
                        state_slot=table[1:].contiguous(), status=status)
    for i in range(2):
        o, _ = ref([(0, T), (T + i * N, T + (i + 1) * N), (T + (2 + i) * N, T + (3 + i) * N)])
        assert off(out[i], o[T + N:]) <= 2 * TOL
    assert int(status.item()) == 0


# ---------------------------------------------------------------------------
# so many sequences, heads and value tiles that a workgroup walks two value tiles
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("hq,hv,dk,dv", [(1, 3, 32, 48), (2, 4, 64, 80), (1, 2, 128, 112), (4, 8, 128, 128)])
@pytest.mark.parametrize("dtype,out_dtype", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16),
                                             (torch.float32, torch.float16), (torch.bfloat16, torch.float32)])
def test_two_value_tiles_a_workgroup(hq, hv, dk, dv, dtype, out_dtype):
    r = np.random.RandomState(dk + dv)
    lens = [int(n) for n in r.choice([0, 1, 5, 63, 64, 65, 130], 60)]
    say("two tiles", hq, hv, dk, dv, dtype, out_dtype, sum(lens))
    assert len(lens) * hv * (dv // 16) > 2 * 256
    x, dout, dfinal = inputs(41, lens, hq, hv, dk, dv, dtype)
    check(x, lens, dk ** -0.5, out_dtype, dout, dfinal)


def test_the_number_of_sequences_does_not_change_a_sequence():
    """The tiles a workgroup walks follow from the call's size; the arithmetic of a sequence does not."""
    lens = [100, 30, 64, 7] * 16
    x, dout, dfinal = inputs(42, lens, 1, 4, 64, 80, torch.bfloat16)
    out, fin, tape = forward(x, lens)
    grads = backward(x, lens, tape, dout, dfinal)
    n, B = sum(lens[:4]), 4
    y = {m: (t[:B] if m == "state" else t[:n]).contiguous() for m, t in x.items()}
    out2, fin2, tape2 = forward(y, lens[:4])
    few = backward(y, lens[:4], tape2, dout[:n].contiguous(), dfinal[:B].contiguous())
    assert torch.equal(out[:n], out2) and torch.equal(fin[:B], fin2)
    for m in few:
        assert torch.equal(few[m], grads[m][:few[m].shape[0]]), m


@pytest.mark.parametrize("where", ["v", "alpha", "beta", "dout"])
def test_a_nan_stays_in_its_sequence_and_head(where):
    lens = [70, 200, 1, 33]
    x, dout, dfinal = inputs(43, lens, 2, 4, 64, 48)
    _, _, tape = first = forward(x, lens)
    grads = backward(x, lens, tape, dout, dfinal)
    x, dout = {n: t.clone() for n, t in x.items()}, dout.clone()
    (dout if where == "dout" else x[where])[70 + 100, 1] = float("nan")
    out, fin, tape = forward(x, lens)
    bad = backward(x, lens, tape, dout, dfinal)
    # value head 1 of sequence 1 from its chunk on (forward) and up to its chunk (backward) may be NaN; q/k head 0 sums it
    token = torch.ones(sum(lens), dtype=torch.bool, device=DEV)
    token[70:270] = False
    heads = [0, 2, 3]
    assert torch.equal(out[:, heads], first[0][:, heads]) and torch.equal(fin[:, heads], first[1][:, heads])
    assert torch.equal(out[token], first[0][token]) and torch.equal(fin[[0, 2, 3]], first[1][[0, 2, 3]])
    assert torch.equal(out[70:70 + 64], first[0][70:70 + 64])
    for n in ("dv", "dalpha", "dbeta"):
        assert torch.equal(bad[n][:, heads], grads[n][:, heads]), n
    for n in ("dq", "dk"):
        assert torch.equal(bad[n][:, 1], grads[n][:, 1]), n
    for n in ("dq", "dk", "dv", "dalpha", "dbeta"):
        assert torch.equal(bad[n][token], grads[n][token]), n
    assert torch.equal(bad["dstate"][[0, 2, 3]], grads["dstate"][[0, 2, 3]])
    if where != "dout":  # not hidden where it is an input of the rule
        assert bool(out[70 + 100, 1].isnan().any()) and bool(fin[1, 1].isnan().any())
    if where == "v":  # the rule is affine in the state: no value stands in the state's gradient
        assert torch.equal(bad["dstate"], grads["dstate"])
    else:
        assert bool(bad["dstate"][1, 1].isnan().any())


def test_gradient_of_the_state_in_place():
    lens = [70, 0, 130]
    x, dout, dfinal = inputs(44, lens, 1, 2, 64, 48)
    _, _, tape = forward(x, lens)
    want = backward(x, lens, tape, dout, dfinal)
    d, g = dfinal.clone(), {n: torch.empty_like(x[n]) for n in ("q", "k", "v", "alpha", "beta")}
    gb.gdn_scan_backward(offsets(lens), x["q"], x["k"], x["v"], x["alpha"], x["beta"], tape, dout, g["q"], g["k"], g["v"],
                         g["alpha"], g["beta"], dfinal=d, dstate=d)
    assert torch.equal(d, want["dstate"]) and all(torch.equal(g[n], want["d" + n]) for n in g)


# ---------------------------------------------------------------------------
# long sequences on few heads: the walks are cut into segments
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("lens,hq,hv,dk,dv,dtype", [
    ([1537], 1, 1, 32, 16, torch.float32),
    ([1500, 70, 0, 1100, 449, 1], 1, 2, 64, 48, torch.bfloat16),
    ([2500], 2, 2, 128, 32, torch.float32),
    ([1664, 1665], 1, 3, 128, 64, torch.bfloat16),
])
def test_segments(lens, hq, hv, dk, dv, dtype):
    say("segments", lens, hq, hv, dk, dv, dtype)
    x, dout, dfinal = inputs(45, lens, hq, hv, dk, dv, dtype)
    check(x, lens, dk ** -0.5, dtype, dout, dfinal)


def test_segments_with_slots_and_in_place():
    lens = [1600, 1700, 64, 1601]
    x, dout, dfinal = inputs(46, lens, 1, 2, 64, 32)
    want, fin, tape = forward(x, lens)
    grads = backward(x, lens, tape, dout, dfinal)
    slot = torch.tensor([2, 9, 0, 1], dtype=torch.int32, device=DEV)  # the second is outside the pool
    pool = torch.zeros(3, 2, 32, 64, device=DEV)
    for b in (0, 2, 3):
        pool[slot[b].long()] = x["state"][b]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, fin2, tape2 = forward(x, lens, state=pool, state_slot=slot, status=status)
    assert int(status.item()) == gb.CODES["GDN_ERR_SLOT"]
    keep = torch.ones(sum(lens), dtype=torch.bool, device=DEV)
    keep[1600:3300] = False
    assert torch.equal(out[keep], want[keep]) and bool(out[~keep].isnan().all())
    assert torch.equal(fin2[[0, 2, 3]], fin[[0, 2, 3]]) and bool(fin2[1].isnan().all())
    g2 = backward(x, lens, tape2, dout, dfinal)
    for n in ("dq", "dk", "dv", "dalpha", "dbeta"):
        assert torch.equal(g2[n][keep], grads[n][keep]) and bool(g2[n][~keep].isnan().all()), n
    assert torch.equal(g2["dstate"][[0, 2, 3]], grads["dstate"][[0, 2, 3]])
    state = x["state"].clone()
    out = torch.empty_like(want)
    gb.gdn_scan_forward(offsets(lens), x["q"], x["k"], x["v"], x["alpha"], x["beta"], out, state=state, final_state=state)
    assert torch.equal(out, want) and torch.equal(state, fin)


def test_segments_with_gates_at_their_ends():
    lens = [1700]
    for alpha, beta in (("zeros", "ends"), ("one", "mixed")):
        x, dout, dfinal = inputs(47, lens, 1, 2, 64, 32, alpha=alpha, beta=beta)
        check(x, lens, 0.125, torch.float32, dout, dfinal)


def test_a_nan_passes_from_segment_to_segment():
    lens = [1600, 1200]
    x, dout, dfinal = inputs(48, lens, 1, 2, 64, 32)
    want, fin, _ = forward(x, lens)
    x["v"][500, 1, 3] = float("nan")
    out, fin2, tape = forward(x, lens)
    chunk = 500 // 64 * 64
    assert torch.equal(out[:chunk], want[:chunk]) and torch.equal(out[1600:], want[1600:])
    assert torch.equal(out[:, 0], want[:, 0]) and torch.equal(fin2[1], fin[1])
    assert bool(out[500:1600, 1, 3].isnan().all()) and bool(fin2[0, 1, 3].isnan().all())
