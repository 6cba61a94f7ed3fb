"""The operators of a layer together, as they are used: a draft block through norm, projections, verify, gated norm and
output projection, its states kept and restored in 8 bits; and a training step through norms and scan."""
import numpy as np
import pytest
import torch

import layer_reference as ref
import scan_reference
from gated_deltanet_recurrence_gdn_amd import binding as gb
from helpers import DEV
from test_gpu_norm import codes_for, normal

pytestmark = pytest.mark.gpu

B, N, HQK, HV, D, WIDTH = 2, 16, 2, 6, 64, 640
QK, V = HQK * D, HV * D


def weights(seed, columns, inner):
    """8-bit weights with fp32 scales of 128 x 128 blocks, as a checkpoint has them."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    w = torch.randn(columns, inner, generator=g, device=DEV) * inner ** -0.5
    G, C = ref.cut(inner), ref.cut(columns)
    blocks = torch.nn.functional.pad(w, (0, G * 128 - inner, 0, C * 128 - columns)).reshape(C, 128, G, 128)
    scale = blocks.abs().amax((1, 3)) / 448
    return (blocks / scale[:, None, :, None]).reshape(C * 128, G * 128)[:columns, :inner].contiguous().to(torch.float8_e4m3fn), scale


class Layer:
    def __init__(self):
        self.norm, self.head = 1 + 0.1 * normal(1, WIDTH), 1 + 0.1 * normal(2, D)
        self.w_in, self.s_in = weights(3, 2 * QK + 2 * V, WIDTH)
        self.w_out, self.s_out = weights(4, WIDTH, V)
        M = B * N
        bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
        self.residual, (self.codes, self.scales) = bf(M, WIDTH), codes_for(M, WIDTH)
        self.q, self.k, self.v, self.z = bf(M, HQK, D), bf(M, HQK, D), bf(M, HV, D), bf(M, HV, D)
        self.out = torch.zeros(B, N, HV, D, device=DEV)
        self.persist = torch.zeros(B, N, HV, D, D, dtype=torch.float16, device=DEV)
        self.hcodes, self.hscales = codes_for(M, V)
        self.y = bf(M, WIDTH)

    def step(self, x, residual, alpha, beta, state):
        """One draft block of 16 tokens of two sequences."""
        gb.gdn_norm_forward(x, self.norm, codes=self.codes, scales=self.scales, residual=residual, residual_out=self.residual)
        gb.gdn_project(self.codes, self.scales, self.w_in, self.s_in, [self.q, self.k, self.v, self.z])
        heads = lambda t: t.view(B, N, *t.shape[1:])  # noqa: E731
        gb.gdn_verify_chain(heads(self.q), heads(self.k), heads(self.v), alpha, beta, state, out=self.out, persist=self.persist,
                            scale=D ** -0.5)
        gb.gdn_gated_norm_forward(self.out, heads(self.z), self.head, codes=self.hcodes, scales=self.hscales)
        gb.gdn_project(self.hcodes, self.hscales, self.w_out, self.s_out, self.y)


def inputs(seed):
    alpha = torch.sigmoid(normal(seed, B, N, HV) + 2)
    # keys of a few tenths keep the rule stable without normalising them
    return (normal(seed + 1, B * N, WIDTH, dtype=torch.bfloat16), normal(seed + 2, B * N, WIDTH, dtype=torch.bfloat16), alpha,
            0.05 * torch.sigmoid(normal(seed + 3, B, N, HV)), 0.1 * normal(seed + 4, B, HV, D, D))


def check_layer(s, x, residual, alpha, beta, state):
    """Each operator against its formula on what the one before it left."""
    assert torch.equal(s.residual, (x.float() + residual.float()).bfloat16())
    y, _ = ref.norm(s.residual, s.norm, 1e-6)
    ref.check_codes(y, s.codes, s.scales, ref.NORM)
    y, lost = ref.project(s.codes, s.scales, s.w_in, s.s_in)
    ref.near(torch.cat([t.reshape(B * N, -1) for t in (s.q, s.k, s.v, s.z)], 1), y, lost)
    q, k, v = (t.double().cpu().view(B, N, -1, D) for t in (s.q, s.k, s.v))
    group = HV // HQK
    S, out = state.double().cpu().clone(), torch.zeros(B, N, HV, D, dtype=torch.float64)
    for n in range(N):
        kh, qh = (t[:, n].repeat_interleave(group, 1) for t in (k, q))
        a, b = alpha[:, n].double().cpu()[..., None], beta[:, n].double().cpu()[..., None]
        e = v[:, n] - a * (S @ kh[..., None])[..., 0]
        S = a[..., None] * S + (b * e)[..., None] * kh[..., None, :]
        out[:, n] = D ** -0.5 * (S @ qh[..., None])[..., 0]
    got = s.out.double().cpu()
    assert float((got - out).abs().max() / out.abs().max()) <= 2e-3  # the verify's bar
    y, _ = ref.gated(s.out.view(B * N, HV, D), s.z, s.head, 1e-6)
    ref.check_codes(y.reshape(B * N, -1), s.hcodes, s.hscales, ref.GATED)
    y, lost = ref.project(s.hcodes, s.hscales, s.w_out, s.s_out)
    ref.near(s.y, y, lost)


def test_a_draft_block():
    s, given = Layer(), inputs(10)
    s.step(*given)
    check_layer(s, *given)


def test_a_draft_block_captured():
    """The whole block in one graph, replayed over other inputs, with the program's own work between."""
    s, given = Layer(), inputs(10)
    s.step(*given)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.step(*given)
    for seed in (20, 30, 40):
        for t, o in zip(given, inputs(seed)):
            t.copy_(o)
        graph.replay()
        torch.cuda.synchronize()
        check_layer(s, *given)


def test_two_streams_at_once():
    """Two layers' blocks on two streams: nothing is shared between calls."""
    a, b, x, y = Layer(), Layer(), inputs(10), inputs(50)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, given, st in ((a, x, streams[0]), (b, y, streams[1])):
            with torch.cuda.stream(st):
                s.step(*given)
    torch.cuda.synchronize()
    check_layer(a, *x)
    check_layer(b, *y)


def test_accepted_states_kept_in_8_bits():
    """The accepted nodes' persisted states to packed rows, and back into the pool that the next block starts from."""
    s, given = Layer(), inputs(10)
    s.step(*given)
    accepted = torch.tensor([5, 15], dtype=torch.int32, device=DEV)
    nodes = s.persist.flatten(0, 1)[None]  # a pool of one layer, a row for each node
    codes = torch.zeros(1, 4, HV, D, D, dtype=torch.int8, device=DEV)
    scales = torch.zeros(1, 4, HV, D, device=DEV)
    src = accepted + torch.tensor([0, N], dtype=torch.int32, device=DEV)
    rows = torch.tensor([3, 1], dtype=torch.int32, device=DEV)
    gb.gdn_pool_pack(nodes, codes, scales, src, rows)
    pool = torch.zeros(1, 5, HV, D, D, device=DEV)
    slots = torch.tensor([4, 0], dtype=torch.int32, device=DEV)
    gb.gdn_pool_unpack(codes, scales, pool, rows, slots)
    for b in range(B):
        kept = s.persist[b, accepted[b]].double()
        half = kept.abs().amax(-1, keepdim=True) / 254
        # half a step, and the roundings of the scale and of the product
        assert torch.all((pool[0, slots[b]].double() - kept).abs() <= half * (1 + 4 * ref.U) + 127 * 2 * half * 2 * ref.U)
    x, residual, alpha, beta, _ = inputs(60)
    gb.gdn_verify_chain(s.q.view(B, N, HQK, D), s.k.view(B, N, HQK, D), s.v.view(B, N, HV, D), alpha, beta, pool[0], state_slot=slots,
                        out=s.out, scale=D ** -0.5)
    torch.cuda.synchronize()
    assert s.out.isfinite().all()


def test_a_training_step():
    """norm -> scan -> gated norm, forward and backward through the library's calls, against automatic differentiation in
    float64 of the same formulas."""
    total, cu = 70, np.array([0, 33, 70], np.int32)
    x, residual, weight, head = normal(1, total, V), normal(2, total, V), 1 + 0.1 * normal(3, V), 1 + 0.1 * normal(4, D)
    q, k = (torch.nn.functional.normalize(normal(s, total, HQK, D), dim=-1) for s in (5, 6))
    alpha, beta = torch.sigmoid(normal(7, total, HV) + 2), torch.sigmoid(normal(8, total, HV))
    z, dy = normal(9, total, HV, D), normal(11, total, HV, D)
    r, v, out, y = torch.empty_like(x), torch.empty_like(x), torch.empty_like(z), torch.empty_like(z)
    gb.gdn_norm_forward(x, weight, residual=residual, residual_out=r, out=v)
    vh = v.view(total, HV, D)
    tape = torch.empty(gb.gdn_scan_tape_bytes(cu, q, vh), dtype=torch.uint8, device=DEV)
    gb.gdn_scan_forward(cu, q, k, vh, alpha, beta, out, tape=tape, scale=D ** -0.5)
    gb.gdn_gated_norm_forward(out, z, head, out=y)
    dout, dz, dhead = torch.empty_like(out), torch.empty_like(z), torch.empty_like(head)
    gb.gdn_gated_norm_backward(dy, out, z, head, dout, dz, dhead)
    grads = [torch.empty_like(t) for t in (q, k, vh, alpha, beta)]
    gb.gdn_scan_backward(cu, q, k, vh, alpha, beta, tape, dout, *grads, scale=D ** -0.5)
    dx, dweight = torch.empty_like(x), torch.empty_like(weight)
    gb.gdn_norm_backward(grads[2].view(total, V), r, weight, dx, dweight)
    # the same in float64
    leaves = [t.double().cpu().requires_grad_() for t in (x, residual, weight, head, q, k, alpha, beta, z)]
    x6, r6, w6, h6, q6, k6, a6, b6, z6 = leaves
    s6 = x6 + r6
    v6 = (s6 * (s6.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w6).view(total, HV, D)
    o6, _ = scan_reference.rule(q6, k6, v6, a6, b6, torch.zeros(2, HV, D, D, dtype=torch.float64), np.diff(cu), D ** -0.5)
    y6 = o6 * (o6.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * h6 * z6 * torch.sigmoid(z6)
    want = torch.autograd.grad(y6, leaves, dy.double().cpu())
    norm = torch.linalg.vector_norm
    # each call is off by some 1e-6 of the 2-norm; the norms' divisions by small heads amplify by less than 20
    close = lambda got, ref6: norm(got.double().cpu() - ref6) <= 2e-5 * norm(ref6)  # noqa: E731
    assert close(y, y6.detach())
    for got, ref6 in zip((dx, dx, dweight, dhead, grads[0], grads[1], grads[3], grads[4], dz), want):
        assert close(got, ref6)


def segment_stream(t):
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("no such segment")


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", ["norm", "gated"])
def test_workspaces_are_the_launching_streams(name, handle):
    side = torch.cuda.Stream()
    x, w = normal(1, 40, 4, 64), normal(2, 64)
    stream = side.cuda_stream if handle else side
    if name == "norm":
        call = gb.gdn_norm_backward(x, x, w, None, torch.empty_like(w), stream=stream, prepare=True)
    else:
        call = gb.gdn_gated_norm_backward(x, x, x, w, None, None, torch.empty_like(w), stream=stream, prepare=True)
    workspace = [t for t in call._keep if isinstance(t, torch.Tensor) and t.dtype == torch.uint8][-1]
    assert segment_stream(workspace) == side.cuda_stream
    side.wait_stream(torch.cuda.current_stream())
    call()
    torch.cuda.synchronize()


def test_prepared_calls_repeat():
    """A prepared call launches again what it was given, on the inputs as they are then."""
    s, given = Layer(), inputs(10)
    s.step(*given)
    x, residual = given[:2]
    calls = [gb.gdn_norm_forward(x, s.norm, codes=s.codes, scales=s.scales, residual=residual, residual_out=s.residual, prepare=True),
             gb.gdn_project(s.codes, s.scales, s.w_in, s.s_in, [s.q, s.k, s.v, s.z], prepare=True),
             gb.gdn_gated_norm_forward(s.out, s.z.view(B, N, HV, D), s.head, codes=s.hcodes, scales=s.hscales, prepare=True),
             gb.gdn_project(s.hcodes, s.hscales, s.w_out, s.s_out, s.y, prepare=True)]
    x.copy_(inputs(70)[0])
    for c in calls:
        c()
    torch.cuda.synchronize()
    y, _ = ref.norm(s.residual, s.norm, 1e-6)
    ref.check_codes(y, s.codes, s.scales, ref.NORM)
    y, lost = ref.project(s.hcodes, s.hscales, s.w_out, s.s_out)
    ref.near(s.y, y, lost)


def test_a_stream_of_another_device_is_refused():
    class Stream:
        cuda_stream, device_index = 0x1230, torch.cuda.current_device() + 1

    x, w = normal(1, 4, 64), normal(2, 64)
    with pytest.raises(ValueError, match="the current device is"):
        gb.gdn_norm_forward(x, w, out=torch.empty_like(x), stream=Stream())
