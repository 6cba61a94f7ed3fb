"""The training scan and the row-pool operators, as a user's program calls them, beside their plain forms.

Five operators in two groups:

- the gated delta rule over packed sequences at fp32 accuracy, forward (``forward`` cases) and forward with the
  backward pass (``train`` cases: one training step of the layer's recurrence, gradients returned);
- the pool of state rows that sequences live in: rows copied between pools (``copy``), sequences forked into rows of
  their own while finished ones are released (``fork``), live rows moved together (``compact``).

``run`` computes the plain form in torch, or calls the library where ``own`` is set.  ``exact`` evaluates the
definitions in 64 bits, token by token and row by row.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
CHUNK = 64
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------
def _scan_case(kind, dtype, lens, h_qk, h_v, d_k, d_v, state):
    return {"kind": kind, "dtype": dtype, "lens": lens, "h_qk": h_qk, "h_v": h_v, "d_k": d_k, "d_v": d_v, "state": state}


def _pool_case(kind, layers, rows, h_v, d, channels, seqs, n):
    return {"kind": kind, "layers": layers, "rows": rows, "h_v": h_v, "d": d, "channels": channels, "seqs": seqs, "n": n}


def listed():
    cases = [
        # one token through a small fp32 layer: what a call costs when there is nothing to do
        ("forward one token f32", _scan_case("forward", "f32", "1", 1, 2, 32, 32, True)),
        # a packed evaluation batch in fp32 with odd lengths, an empty sequence and fresh states
        ("forward packed f32", _scan_case("forward", "f32", "700,1,0,65,333", 4, 8, 64, 96, False)),
        # the 4096-token prompt of one full layer (16 / 48 heads, d = 128)
        ("forward 4096 bf16", _scan_case("forward", "bf16", "4096", 16, 48, 128, 128, True)),
        # a unit-test sized training step
        ("train small f32", _scan_case("train", "f32", "17,64,100", 2, 4, 32, 32, True)),
        # a training micro-batch of one full layer: documents of different lengths packed into 4096 tokens
        ("train packed 4096 bf16", _scan_case("train", "bf16", "2048,1023,517,300,208", 16, 48, 128, 128, False)),
        # one rank's share of the heads (16 / 48 over 8 ranks) of a long document
        ("train 16384 of 6 heads bf16", _scan_case("train", "bf16", "16384", 2, 6, 128, 128, True)),
        # one sequence's row of one small layer
        ("copy one row", _pool_case("copy", 1, 4, 2, 32, 128, 2, 1)),
        # cached prefixes restored for 8 requests, recurrent state and convolution history of 48 full layers
        ("copy 8 rows of 48 layers", _pool_case("copy", 48, 20, 48, 128, 10240, 10, 8)),
        # one request sampled four ways in a small model
        ("fork 4 rows", _pool_case("fork", 4, 16, 4, 64, 512, 8, 4)),
        # a scheduler step that forks 12 continuations over 48 full layers and drops finished requests
        ("fork 12 rows of 48 layers", _pool_case("fork", 48, 40, 48, 128, 10240, 24, 12)),
        # a small pool closed up after a few requests ended
        ("compact 64 small rows", _pool_case("compact", 2, 64, 2, 32, 128, 64, 20)),
        # the pool of 24 full layers closed up to the rows in use
        ("compact 48 rows of 24 layers", _pool_case("compact", 24, 48, 48, 128, 10240, 40, 16)),
    ]
    return [dict(c, name=n) for n, c in cases]


def _log_int(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    kind = rng.choice(["forward", "train", "forward", "train", "copy", "fork", "compact"])
    if kind in ("forward", "train"):
        h_qk = rng.choice([1, 2, 3, 4, 8, 16])
        h_v = h_qk * rng.choice([1, 2, 3, 4])
        d_k, d_v = rng.choice([32, 64, 128]), rng.choice([32, 64, 96, 128, 256])
        most = min(8192, 4096 * 48 * 128 * 128 // (h_v * d_k * d_v))
        total, count = _log_int(rng, 1, most), _log_int(rng, 1, 9)
        cuts = sorted(rng.randint(0, total) for _ in range(count - 1))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        return _scan_case(kind, rng.choice(["f32", "bf16"]), ",".join(map(str, lens)), h_qk, h_v, d_k, d_v, rng.random() < 0.5)
    h_v, d = rng.choice([2, 6, 16, 48]), rng.choice([32, 64, 128])
    layers = _log_int(rng, 1, 48)
    most = max(6, min(200, 48 * 20 * 48 * 128 * 128 // (layers * h_v * d * d)))
    rows = _log_int(rng, 6, most)
    seqs = rng.randint(2, max(2, rows // 2))
    n = rng.randint(1, max(1, min(seqs, rows - seqs)))
    return _pool_case(kind, layers, rows, h_v, d, 8 * rng.randint(1, 1280), seqs, n)


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------
def _scan_inputs(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    lens = [int(x) for x in case["lens"].split(",")]
    total, Hq, Hv, dk, dv, t = sum(lens), case["h_qk"], case["h_v"], case["d_k"], case["d_v"], DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    # queries and keys are normalised per head, gates per head range from long memory (0.98) to short (0.3)
    unit = lambda x: x / x.square().sum(-1, keepdim=True).sqrt()  # noqa: E731
    s = {"case": case, "lens": lens, "cu": np.concatenate([[0], np.cumsum(lens)]).astype(np.int32), "scale": dk ** -0.5}
    s["q"], s["k"] = unit(normal(total, Hq, dk)).to(t), unit(normal(total, Hq, dk)).to(t)
    s["v"] = normal(total, Hv, dv).to(t)
    slow = torch.linspace(-4.0, 0.5, Hv, device=DEV)
    s["alpha"] = torch.exp(-torch.log1p(torch.exp(slow + normal(total, Hv))))
    s["beta"] = 1 / (1 + torch.exp(-normal(total, Hv)))
    s["state"] = 0.1 * normal(len(lens), Hv, dv, dk) if case["state"] else None
    if case["kind"] == "train":
        s["dout"] = normal(total, Hv, dv).to(t)
        s["dfinal"] = 0.1 * normal(len(lens), Hv, dv, dk) if case["state"] else None
    return s


def _pool_inputs(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = np.random.RandomState(seed % (1 << 32))
    L, R, H, d, C, m, n = (case[x] for x in ("layers", "rows", "h_v", "d", "channels", "seqs", "n"))

    def ints(x):
        return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(DEV)

    if m > R or n > (m if case["kind"] == "compact" else R - m):
        raise ValueError("the pool has too few rows for this case")
    # the recurrent states in fp32 and the convolution's last three input rows in bf16
    s = {"case": case}
    s["pools"] = [torch.randn(L, R, H, d, d, generator=g, device=DEV),
                  torch.randn(L, R, 3, C, generator=g, device=DEV).to(torch.bfloat16)]
    place = r.permutation(R)
    if case["kind"] == "copy":
        # the first rows of the permutation are sources (some named more than once), the others destinations
        s["src"], s["dst"] = ints(r.choice(place[:m], n)), ints(place[m:m + n])
        return s
    table = place[:m]
    if case["kind"] == "fork":
        # n new sequences beside the m running ones, each from a running sequence or (one in eight) fresh;
        # every fourth running sequence ends
        s["table"] = ints(np.concatenate([table, np.full(n, -1)]))
        s["parent"] = ints(np.where(r.rand(n) < 0.125, -1, r.randint(0, m, n)))
        s["child"] = ints(m + r.permutation(n))
        s["released"] = ints(r.permutation(m)[:m // 4])
    else:
        s["table"] = ints(table)
        s["released"] = ints(r.permutation(m)[:n])
    return s


def prepare(case, seed):
    return (_scan_inputs if case["kind"] in ("forward", "train") else _pool_inputs)(case, seed)


# ---------------------------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------------------------
def _plain_scan(s, q, k, v, alpha, beta, state):
    """The rule in chunks of 64 tokens: within a chunk (I + A) E = V - gamma K S^T with A strictly lower triangular,
    between chunks the state.  The gates' running sums and the inverse of I + A are in 64 bits, the rest in 32."""
    lens, scale = s["lens"], s["scale"]
    B, total, Hv, dv, dk = len(lens), q.shape[0], v.shape[1], v.shape[2], q.shape[2]
    n = max(1, -(-max(lens) // CHUNK))
    t = torch.arange(n * CHUNK, device=DEV)
    lens_d = torch.tensor(lens, device=DEV)[:, None]
    start = torch.tensor(s["cu"][:-1].astype(np.int64), device=DEV)[:, None]
    at = torch.where(t < lens_d, start + t, total)  # [B][T]; tokens past a sequence's end read the padding row

    def chunks(x, fill):  # [total][H][...] -> [B][H][chunks][64][...]
        x = torch.cat([x, torch.full_like(x[:1], fill) if total else x.new_full((1, *x.shape[1:]), fill)])[at]
        return x.reshape(B, n, CHUNK, *x.shape[2:]).movedim(3, 1)

    q, k = (chunks(x, 0.0).repeat_interleave(Hv // q.shape[1], 1) for x in (q, k))
    v, beta = chunks(v, 0.0), chunks(beta, 0.0)
    b = torch.log(chunks(alpha.double(), 1.0)).cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=DEV).tril()
    D = torch.exp(torch.where(low, b[..., :, None] - b[..., None, :], -math.inf)).float()
    gamma, rest, whole = torch.exp(b).float()[..., None], torch.exp(b[..., -1:] - b).float()[..., None], torch.exp(b[..., -1]).float()
    A = ((k @ k.transpose(-1, -2)) * D * beta[..., None, :]).tril(-1).double()
    eye = torch.eye(CHUNK, dtype=torch.float64, device=DEV)
    inverse, power = eye - A, A @ A
    for _ in range(5):  # (I + A)^-1 = (I - A)(I + A^2)(I + A^4)...: A^64 = 0
        inverse, power = inverse + inverse @ power, power @ power
    inverse = inverse.float()
    P = (q @ k.transpose(-1, -2)) * D
    W, E0 = inverse @ (gamma * k), inverse @ v
    S = torch.zeros(B, Hv, dv, dk, device=DEV) if state is None else state
    outs = []
    for c in range(n):  # the state goes from chunk to chunk
        E = E0[:, :, c] - W[:, :, c] @ S.transpose(-1, -2)
        U = beta[:, :, c, :, None] * E
        outs.append(scale * (gamma[:, :, c] * (q[:, :, c] @ S.transpose(-1, -2)) + P[:, :, c] @ U))
        S = whole[:, :, c, None, None] * S + (rest[:, :, c] * U).transpose(-1, -2) @ k[:, :, c]
    out = torch.stack(outs, 1).movedim(2, 3).reshape(B * n * CHUNK, Hv, dv)
    return out[(t < lens_d).reshape(-1).nonzero()[:, 0]], S


def _run_plain_scan(s):
    t = s["q"].dtype
    names = ["q", "k", "v", "alpha", "beta"] + (["state"] if s["state"] is not None else [])
    x = {n: s[n].float() for n in names}
    if s["case"]["kind"] == "forward":
        out, S = _plain_scan(s, *(x.get(n) for n in ("q", "k", "v", "alpha", "beta", "state")))
        return {"out": out.to(t), "final": S}
    with torch.enable_grad():
        x = {n: y.detach().clone().requires_grad_() for n, y in x.items()}
        out, S = _plain_scan(s, *(x.get(n) for n in ("q", "k", "v", "alpha", "beta", "state")))
        to, by = [out], [s["dout"].float()]
        if s["dfinal"] is not None:
            to, by = to + [S], by + [s["dfinal"]]
        grads = torch.autograd.grad(to, [x[n] for n in names], by)
    r = {"out": out.detach().to(t), "final": S.detach()}
    r.update({"d" + n: g.to(t) if n in ("q", "k", "v") else g for n, g in zip(names, grads)})
    return r


def _run_plain_pool(s):
    kind, pools = s["case"]["kind"], s["pools"]
    R = pools[0].shape[1]
    if kind == "copy":
        src, dst = s["src"].long(), s["dst"].long()
        for p in pools:
            p[:, dst] = p[:, src]
        return {"pools": pools}
    table, row = s["table"].long(), torch.arange(R, device=DEV)
    if kind == "fork":
        used = torch.zeros(R + 1, dtype=torch.bool, device=DEV)
        used[torch.where(table >= 0, table, R)] = True
        new = torch.where(used[:R], R, row).sort().values[:s["child"].numel()]  # the lowest free rows
        parent = s["parent"].long()
        src = torch.where(parent >= 0, table[parent.clamp(min=0)], 0)
        for p in pools:
            fresh = (parent < 0).reshape(-1, *[1] * (p.dim() - 2))
            p[:, new] = torch.where(fresh, torch.zeros((), dtype=p.dtype, device=DEV), p[:, src])
        table = table.clone()
        table[s["released"].long()] = -1
        table[s["child"].long()] = new
        return {"pools": pools, "table": table.to(torch.int32)}
    table = table.clone()
    table[s["released"].long()] = -1
    used = torch.zeros(R + 1, dtype=torch.bool, device=DEV)
    used[torch.where(table >= 0, table, R)] = True
    used = used[:R]
    count = used.sum()
    src, dst = (used & (row >= count)).nonzero()[:, 0], (~used & (row < count)).nonzero()[:, 0]
    for p in pools:
        p[:, dst] = p[:, src]
    to = row.clone()
    to[src] = dst
    table = torch.where(table >= 0, to[table.clamp(min=0)], -1)
    return {"pools": pools, "table": table.to(torch.int32), "count": count.to(torch.int32).reshape(1)}


# ---------------------------------------------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------------------------------------------
def _run_own_scan(s):
    from gated_deltanet_recurrence_gdn_amd import binding as gdn

    cu, q, k, v, alpha, beta, state = (s[n] for n in ("cu", "q", "k", "v", "alpha", "beta", "state"))
    r = {"out": torch.empty_like(v), "final": torch.empty(len(s["lens"]), v.shape[1], v.shape[2], q.shape[2], device=DEV)}
    if s["case"]["kind"] == "forward":
        gdn.gdn_scan_forward(cu, q, k, v, alpha, beta, r["out"], state=state, final_state=r["final"], scale=s["scale"])
        return r
    tape = torch.empty(gdn.gdn_scan_tape_bytes(cu, q, v), dtype=torch.uint8, device=DEV)
    gdn.gdn_scan_forward(cu, q, k, v, alpha, beta, r["out"], tape=tape, state=state, final_state=r["final"], scale=s["scale"])
    for n in ("q", "k", "v", "alpha", "beta") + (("state",) if state is not None else ()):
        r["d" + n] = torch.empty_like(s[n])
    gdn.gdn_scan_backward(cu, q, k, v, alpha, beta, tape, s["dout"], r["dq"], r["dk"], r["dv"], r["dalpha"], r["dbeta"],
                          dfinal=s["dfinal"], dstate=r.get("dstate"), scale=s["scale"])
    return r


def _run_own_pool(s):
    from gated_deltanet_recurrence_gdn_amd import binding as gdn

    kind, pools = s["case"]["kind"], s["pools"]
    if kind == "copy":
        gdn.gdn_pool_copy(pools, s["src"], s["dst"])
        return {"pools": pools}
    table = torch.empty_like(s["table"])
    if kind == "fork":
        gdn.gdn_pool_fork(pools, s["table"], s["parent"], s["child"], released=s["released"], table_out=table)
        return {"pools": pools, "table": table}
    count = torch.empty(1, dtype=torch.int32, device=DEV)
    gdn.gdn_pool_compact(pools, s["table"], released=s["released"], table_out=table, count=count)
    return {"pools": pools, "table": table, "count": count}


def run(state):
    if state["case"]["kind"] in ("forward", "train"):
        return _run_own_scan(state) if own else _run_plain_scan(state)
    return _run_own_pool(state) if own else _run_plain_pool(state)


# ---------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def _exact_scan(case, seed):
    s = _scan_inputs(case, seed)
    train = case["kind"] == "train"
    q, k, v, alpha, beta = (s[n].double() for n in ("q", "k", "v", "alpha", "beta"))
    total, Hq, dk = q.shape
    Hv, dv = v.shape[1:]
    group, scale, cu = Hv // Hq, s["scale"], s["cu"]
    qh, kh = q.repeat_interleave(group, 1), k.repeat_interleave(group, 1)
    out, e = torch.empty_like(v), torch.empty_like(v)
    S = torch.zeros(len(s["lens"]), Hv, dv, dk, dtype=torch.float64, device=DEV)
    if s["state"] is not None:
        S.copy_(s["state"])
    before = torch.empty(total if train else 0, Hv, dv, dk, dtype=torch.float64, device=DEV)
    for b in range(len(s["lens"])):
        X = S[b]
        for t in range(cu[b], cu[b + 1]):
            if train:
                before[t] = X
            a = alpha[t, :, None, None]
            e[t] = v[t] - alpha[t, :, None] * (X @ kh[t, :, :, None])[..., 0]
            X = a * X + (beta[t, :, None] * e[t])[:, :, None] * kh[t, :, None, :]
            out[t] = scale * (X @ qh[t, :, :, None])[..., 0]
        S[b] = X
    if not train:
        return {"out": out, "final": S}
    dq, dk_, dv_ = torch.empty_like(qh), torch.empty_like(kh), torch.empty_like(v)
    dalpha, dbeta = torch.empty_like(alpha), torch.empty_like(beta)
    G = torch.zeros_like(S) if s["dfinal"] is None else s["dfinal"].double()
    do = scale * s["dout"].double()
    for b in range(len(s["lens"])):
        X = G[b]
        after = S[b]
        for t in range(cu[b + 1] - 1, cu[b] - 1, -1):
            be = beta[t, :, None]
            prev = before[t]
            X = X + do[t, :, :, None] * qh[t, :, None, :]
            dq[t] = (do[t, :, None, :] @ after)[:, 0]
            du = (X @ kh[t, :, :, None])[..., 0]
            dk_[t] = ((be * e[t])[:, None, :] @ X)[:, 0] - be * alpha[t, :, None] * (du[:, None, :] @ prev)[:, 0]
            dv_[t] = be * du
            dbeta[t] = (du * e[t]).sum(-1)
            X = X - (be * du)[:, :, None] * kh[t, :, None, :]
            dalpha[t] = (X * prev).sum((-1, -2))
            X = alpha[t, :, None, None] * X
            after = prev
        G[b] = X
    r = {"out": out, "final": S, "dq": dq.reshape(total, Hq, group, dk).sum(2), "dk": dk_.reshape(total, Hq, group, dk).sum(2),
         "dv": dv_, "dalpha": dalpha, "dbeta": dbeta}
    if s["state"] is not None:
        r["dstate"] = G
    return r


def _exact_pool(case, seed):
    s = _pool_inputs(case, seed)
    pools, kind = s["pools"], case["kind"]
    old = [p.clone() for p in pools]
    if kind == "copy":
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            for p, o in zip(pools, old):
                p[:, b] = o[:, a]
        return {"pools": pools}
    table, released = s["table"].tolist(), s["released"].tolist()
    if kind == "fork":
        free = [i for i in range(case["rows"]) if i not in table]
        to = [-1 if i in released else x for i, x in enumerate(table)]
        for i, (a, c) in enumerate(zip(s["parent"].tolist(), s["child"].tolist())):
            to[c] = free[i]
            for p, o in zip(pools, old):
                p[:, free[i]] = 0 if a < 0 else o[:, table[a]]
        return {"pools": pools, "table": None}
    live = sorted({x for i, x in enumerate(table) if i not in released})
    holes = [i for i in range(len(live)) if i not in live]
    for a, b in zip([x for x in live if x >= len(live)], holes):
        for p, o in zip(pools, old):
            p[:, b] = o[:, a]
    return {"pools": pools, "table": None, "count": None}


def exact(case, seed):
    return (_exact_scan if case["kind"] in ("forward", "train") else _exact_pool)(case, seed)


# ---------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------
def work(case):
    """Each input read once and each output written once; the scan's products are those of the rule itself (forward:
    S k, the update and S q; backward: G k, G^T u, S^T du, S^T do, the two updates of G and <G, S>)."""
    if case["kind"] in ("forward", "train"):
        lens = [int(x) for x in case["lens"].split(",")]
        T, e = sum(lens), 4 if case["dtype"] == "f32" else 2
        Hq, Hv, dk, dv = case["h_qk"], case["h_v"], case["d_k"], case["d_v"]
        states = len(lens) * Hv * dv * dk * 4
        inputs, out = T * (2 * Hq * dk * e + Hv * dv * e + 8 * Hv), T * Hv * dv * e
        if case["kind"] == "forward":
            return {"bytes": inputs + out + states * (2 if case["state"] else 1), "flops": 6 * T * Hv * dk * dv}
        # q, k, v and the gates in, out; dout in, their gradients out; states and their gradients where there are any
        return {"bytes": 2 * inputs + 2 * out + states * (4 if case["state"] else 1), "flops": (6 + 14) * T * Hv * dk * dv}
    row = case["layers"] * (case["h_v"] * case["d"] ** 2 * 4 + 3 * case["channels"] * 2)
    if case["kind"] == "compact":  # about as many rows move as holes lie below the live rows' count
        live = case["seqs"] - case["n"]
        moved = max(1, round(live * (1 - live / case["rows"])))
        return {"bytes": 2 * moved * row + 8 * case["seqs"] + 4 * case["n"], "flops": 0}
    return {"bytes": 2 * case["n"] * row + 8 * case["n"] + (8 * case["seqs"] if case["kind"] == "fork" else 0), "flops": 0}
