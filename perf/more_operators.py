"""What surrounds the gated delta rule in a layer, and its cache in 8 bits, as a user's program calls them, beside
their plain forms.

Four operators:

- the layer's input norm: root mean square norm with the residual's addition, output in 8 bits with scales (``norm``)
  or in the activations' type, and its gradients (``norm_train``);
- the gated norm of the rule's outputs, head by head (``gated``, ``gated_train``);
- the projections: the product of 8-bit operands with a scale for each block of 128, its columns cut into the tensors
  that the rule takes (``project``);
- state rows kept in 8 bits: written (and read back, so that what they stand for is returned: ``pack``) and restored
  (``unpack``).

8-bit activations are e4m3 with one power of two (e8m0) for each 128 channels of a row; 8-bit weights are e4m3 with one
scale for each 128 x 128 block, fp32 or a power of two; 8-bit states are integers with one fp32 scale for each value
channel.  ``run`` computes the plain form in torch, or calls the library where ``own`` is set.  ``exact`` evaluates the
definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
GROUP = 128  # channels that share a scale
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------
def _norm_case(kind, rows, width, dtype, residual, offset, out):
    return {"kind": kind, "rows": rows, "width": width, "dtype": dtype, "residual": residual, "offset": offset, "out": out}


def _gated_case(kind, rows, heads, d, x, z, out):
    return {"kind": kind, "rows": rows, "heads": heads, "d": d, "x": x, "z": z, "out": out}


def _project_case(tokens, columns, inner, scales, out):
    return {"kind": "project", "tokens": tokens, "columns": columns, "inner": inner, "scales": scales, "out": out}


def _pool_case(kind, layers, rows, h_v, d, n, dtype):
    return {"kind": kind, "layers": layers, "rows": rows, "h_v": h_v, "d": d, "n": n, "dtype": dtype}


def listed():
    cases = [
        # one decoded token's input norm: what a call costs when there is nothing to do
        ("norm one token e4m3", _norm_case("norm", 1, 5120, "bf16", "bf16", 1.0, "e4m3")),
        # the input norm of a 4096-token prompt, the residual kept in bf16
        ("norm 4096 tokens e4m3", _norm_case("norm", 4096, 5120, "bf16", "bf16", 1.0, "e4m3")),
        # a training step's norm over an odd number of packed tokens, the residual kept in fp32
        ("norm train 2999 tokens bf16", _norm_case("norm_train", 2999, 2560, "bf16", "f32", 0.0, "plain")),
        # a 16-token draft block's outputs of one layer (48 heads of 128, fp32 as the verify writes them by default)
        ("gated verify block e4m3", _gated_case("gated", 16, 48, 128, "f32", "bf16", "e4m3")),
        # a 4096-token prompt's outputs in f16
        ("gated 4096 tokens e4m3", _gated_case("gated", 4096, 48, 128, "f16", "bf16", "e4m3")),
        # the gated norm of a training micro-batch, forward and backward
        ("gated train 4096 tokens bf16", _gated_case("gated_train", 4096, 48, 128, "bf16", "bf16", "plain")),
        # one token's projections to q, k, v and the gate of a layer with 16 / 48 heads of 128
        ("project one token", _project_case(1, "2048,2048,6144,6144", 5120, "f32", "bf16")),
        # a 22-node tree's output projection, weights with powers of two as scales
        ("project tree e8m0", _project_case(22, "5120", 6144, "e8m0", "bf16")),
        # odd sizes: a ragged group along the inner length, columns that share no tile's border, gates of 6 heads
        ("project odd f16", _project_case(333, "777,6,6,250", 1936, "f32", "f16")),
        # a 4096-token prompt's projections of the full layer
        ("project 4096 tokens", _project_case(4096, "2048,2048,6144,6144", 5120, "f32", "bf16")),
        # the states of 48 full layers kept for 8 prefixes, and read back
        ("pack 8 rows of 48 layers", _pool_case("pack", 48, 12, 48, 128, 8, "f32")),
        # a cached prefix restored for each of 8 requests
        ("unpack 8 rows of 48 layers", _pool_case("unpack", 48, 12, 48, 128, 8, "f32")),
    ]
    return [dict(c, name=n) for n, c in cases]


def _log_int(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    kind = rng.choice(["norm", "norm_train", "gated", "gated_train", "project", "project", "project", "pack", "unpack"])
    if kind in ("norm", "norm_train"):
        width = 8 * _log_int(rng, 4, 1024)
        rows = _log_int(rng, 1, min(65536, 4096 * 5120 // width))
        out = rng.choice(["e4m3", "plain"]) if kind == "norm" else "plain"
        return _norm_case(kind, rows, width, rng.choice(["bf16", "bf16", "f16", "f32"]), rng.choice(["none", "bf16", "f32"]),
                          rng.choice([0.0, 1.0]), out)
    if kind in ("gated", "gated_train"):
        heads, d = rng.choice([1, 2, 3, 6, 16, 32, 48, 64]), rng.choice([16, 32, 48, 64, 96, 128, 128, 256])
        rows = _log_int(rng, 1, min(65536, 4096 * 48 * 128 // (heads * d)))
        out = rng.choice(["e4m3", "plain"]) if kind == "gated" else "plain"
        return _gated_case(kind, rows, heads, d, rng.choice(["f32", "bf16", "f16"]), rng.choice(["bf16", "bf16", "f32", "f16"]), out)
    if kind == "project":
        inner, total = 16 * _log_int(rng, 4, 512), _log_int(rng, 8, 16384)
        tokens = _log_int(rng, 1, 4096)
        cuts = sorted(rng.sample(range(1, total), min(rng.choice([0, 0, 1, 3]), total - 1)))
        columns = ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [total]))
        return _project_case(tokens, columns, inner, rng.choice(["f32", "e8m0"]), rng.choice(["bf16", "bf16", "f16"]))
    h_v, d = rng.choice([2, 6, 16, 48]), rng.choice([32, 64, 128])
    layers = _log_int(rng, 1, 48)
    rows = _log_int(rng, 2, max(2, min(64, 48 * 12 * 48 * 128 * 128 // (layers * h_v * d * d))))
    n = rng.randint(1, max(1, min(rows, 48 * 8 * 48 * 128 * 128 // (layers * h_v * d * d))))
    return _pool_case(kind, layers, rows, h_v, d, n, rng.choice(["f32", "f32", "f16", "bf16"]))


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------
def _cut(n):
    return -(-n // GROUP)


def _scale_bytes(rows, width):
    """Where the scales of activations go: rows of one byte a group, padded to four."""
    return torch.empty(rows, -(-_cut(width) // 4) * 4, dtype=torch.uint8, device=DEV).view(torch.float8_e8m0fnu)


def _power(top):
    """The smallest power of two that brings a group's largest magnitude to 448 at most, as its exponent."""
    m, e = torch.frexp(top)  # top = m 2^e, m in [0.5, 1): 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    return torch.where(top > 0, e, -126).clamp(-126, 127)


def _norm_inputs(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rows, width, t = case["rows"], case["width"], DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    s = {"case": case}
    # a residual stream has a few channels far larger than the rest
    loud = 1 + 30 * (torch.rand(width, generator=g, device=DEV) < 0.005).float()
    s["x"] = normal(rows, width).to(t)
    r = None if case["residual"] == "none" else DTYPES[case["residual"]]
    s["residual"] = None if r is None else (3 * loud * normal(rows, width)).to(r)
    s["weight"] = (1 - case["offset"] + 0.2 * normal(width)).to(torch.bfloat16)
    stored = t if r is None else r
    if case["kind"] == "norm_train":
        s["dout"] = normal(rows, width).to(t)
        s["dresidual"] = None if r is None else normal(rows, width).to(stored)
        s["dx"], s["dweight"] = torch.empty(rows, width, dtype=stored, device=DEV), torch.empty(width, device=DEV)
    s["stored"] = None if r is None else torch.empty(rows, width, dtype=r, device=DEV)
    if case["out"] == "plain":
        s["out"] = torch.empty(rows, width, dtype=t, device=DEV)
    else:
        s["codes"], s["scales"] = torch.empty(rows, width, dtype=torch.float8_e4m3fn, device=DEV), _scale_bytes(rows, width)
    return s


def _gated_inputs(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rows, H, d = case["rows"], case["heads"], case["d"]
    tx, tz = DTYPES[case["x"]], DTYPES[case["z"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    s = {"case": case}
    # the rule's outputs differ in size from head to head
    s["x"] = (torch.exp(normal(H, 1)) * 0.1 * normal(rows, H, d)).to(tx)
    s["z"] = (2 * normal(rows, H, d)).to(tz)
    s["weight"] = 1 + 0.2 * normal(d)
    if case["kind"] == "gated_train":
        s["dout"] = normal(rows, H, d).to(tz)
        s["dx"], s["dz"], s["dweight"] = torch.empty_like(s["x"]), torch.empty_like(s["z"]), torch.empty(d, device=DEV)
    if case["out"] == "plain":
        s["out"] = torch.empty(rows, H, d, dtype=tz, device=DEV)
    else:
        s["codes"], s["scales"] = torch.empty(rows, H * d, dtype=torch.float8_e4m3fn, device=DEV), _scale_bytes(rows, H * d)
    return s


def _project_inputs(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    M, K = case["tokens"], case["inner"]
    parts = [int(x) for x in case["columns"].split(",")]
    N, G = sum(parts), _cut(K)
    s = {"case": case, "parts": parts}
    # normed activations, some channels louder, quantised by groups of 128
    x = torch.randn(M, K, generator=g, device=DEV) * (1 + 10 * (torch.rand(K, generator=g, device=DEV) < 0.01).float())
    e = _power(torch.nn.functional.pad(x, (0, G * GROUP - K)).reshape(M, G, GROUP).abs().amax(-1))
    s["a"] = (x * torch.exp2(-e.float()).repeat_interleave(GROUP, 1)[:, :K]).to(torch.float8_e4m3fn)
    s["a_scales"] = _scale_bytes(M, K)
    s["a_scales"].view(torch.uint8)[:, :G] = (e + 127).to(torch.uint8)
    # weights of a linear layer, quantised by blocks of 128 x 128
    w = torch.randn(N, K, generator=g, device=DEV) * K ** -0.5
    w = torch.nn.functional.pad(w, (0, G * GROUP - K, 0, _cut(N) * GROUP - N)).reshape(_cut(N), GROUP, G, GROUP)
    top = w.abs().amax((1, 3))
    if case["scales"] == "f32":
        scale = top / 448
        s["w_scales"] = scale
    else:
        e = _power(top)
        scale = torch.exp2(e.float())
        s["w_scales"] = torch.full((_cut(N), -(-G // 4) * 4), 127, dtype=torch.uint8, device=DEV)
        s["w_scales"][:, :G] = (e + 127).to(torch.uint8)
        s["w_scales"] = s["w_scales"].view(torch.float8_e8m0fnu)
    w = (w / scale[:, None, :, None]).reshape(_cut(N) * GROUP, G * GROUP)[:N, :K]
    s["w"] = w.to(torch.float8_e4m3fn).contiguous()
    s["outs"] = [torch.empty(M, n, dtype=DTYPES[case["out"]], device=DEV) for n in parts]
    return s


def _pool_inputs(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = np.random.RandomState(seed % (1 << 32))
    L, R, H, d, n, t = case["layers"], case["rows"], case["h_v"], case["d"], case["n"], DTYPES[case["dtype"]]

    def ints(x):
        return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(DEV)

    s = {"case": case, "pool": torch.empty(L, R, H, d, d, dtype=t, device=DEV)}
    # value channels of a state differ in size
    s["pool"].copy_(0.1 * torch.randn(L, R, H, d, d, generator=g, device=DEV) * torch.exp(0.5 * torch.randn(L, 1, H, d, 1, generator=g, device=DEV)))
    s["src"], s["dst"] = ints(r.permutation(R)[:n]), ints(r.permutation(R)[:n])
    if case["kind"] == "unpack":  # what an earlier pack left
        s["codes"], s["scales"] = torch.empty(L, R, H, d, d, dtype=torch.int8, device=DEV), torch.empty(L, R, H, d, device=DEV)
        for layer in range(L):
            x = s["pool"][layer].float()
            s["scales"][layer] = (x.abs().amax(-1) / 127).clamp(min=2.0 ** -126)
            s["codes"][layer] = torch.round(x / s["scales"][layer][..., None]).to(torch.int8)
    else:
        s["codes"], s["scales"] = torch.zeros(L, R, H, d, d, dtype=torch.int8, device=DEV), torch.zeros(L, R, H, d, device=DEV)
        s["back"] = torch.zeros_like(s["pool"])
    return s


def prepare(case, seed):
    kind = case["kind"]
    return (_norm_inputs if kind in ("norm", "norm_train") else _gated_inputs if kind in ("gated", "gated_train")
            else _project_inputs if kind == "project" else _pool_inputs)(case, seed)


# ---------------------------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------------------------
def _plain_codes(y):
    """y [rows][width] in e4m3 with a power of two for each group of 128 channels."""
    rows, width = y.shape
    full = _cut(width) * GROUP
    y = torch.cat([y, y.new_zeros(rows, full - width)], 1) if full != width else y
    y = y.reshape(rows, full // GROUP, GROUP)
    e = _power(y.abs().amax(-1))
    codes = (y * torch.exp2(-e.float())[..., None]).reshape(rows, full)[:, :width].to(torch.float8_e4m3fn)
    return {"codes": codes, "scales": (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)}


def _run_plain_norm(s):
    case, x = s["case"], s["x"]
    r = x if s["residual"] is None else (x.float() + s["residual"].float()).to(s["residual"].dtype)
    v, w = r.float(), s["weight"].float() + case["offset"]
    rs = 1 / torch.sqrt(v.square().mean(-1, keepdim=True) + EPS)
    y = v * rs * w
    res = {} if s["residual"] is None else {"residual": r}
    res.update({"out": y.to(x.dtype)} if case["out"] == "plain" else _plain_codes(y))
    if case["kind"] == "norm_train":
        dy = s["dout"].float()
        g, n = dy * w, v * rs
        dx = rs * (g - n * (g * n).mean(-1, keepdim=True))
        if s["dresidual"] is not None:
            dx = dx + s["dresidual"].float()
        res.update({"dx": dx.to(r.dtype), "dweight": (dy * n).sum(0)})
    return res


def _run_plain_gated(s):
    case, x, z, w = s["case"], s["x"].float(), s["z"].float(), s["weight"]
    rs = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
    n, sig = x * rs, 1 / (1 + torch.exp(-z))
    gate = z * sig
    y = n * w * gate
    res = {"out": y.to(s["z"].dtype)} if case["out"] == "plain" else _plain_codes(y.reshape(x.shape[0], -1))
    if case["kind"] == "gated_train":
        dy = s["dout"].float()
        g = dy * gate * w
        res["dx"] = (rs * (g - n * (g * n).mean(-1, keepdim=True))).to(s["x"].dtype)
        res["dz"] = (dy * n * w * sig * (1 + z * (1 - sig))).to(s["z"].dtype)
        res["dweight"] = (dy * n * gate).sum((0, 1))
    return res


def _values(codes, scales, rows):
    """The values of 8-bit codes whose scales hold for `rows` rows and 128 columns each."""
    s = scales.float()
    s = s.repeat_interleave(rows, 0)[:codes.shape[0]] if rows > 1 else s
    return codes.float() * s.repeat_interleave(GROUP, 1)[:, :codes.shape[1]]


def _run_plain_project(s):
    y = _values(s["a"], s["a_scales"], 1) @ _values(s["w"], s["w_scales"], GROUP).T
    return [part.to(s["outs"][0].dtype).contiguous() for part in y.split(s["parts"], 1)]


def _run_plain_pool(s):
    src, dst = s["src"].long(), s["dst"].long()
    if s["case"]["kind"] == "unpack":
        s["pool"][:, dst] = (s["codes"][:, src].float() * s["scales"][:, src][..., None]).to(s["pool"].dtype)
        return s["pool"]
    x = s["pool"][:, src].float()
    # in 64 bits: the scale is the nearest to amax / 127, and quotients near a half go to the right side
    scale = (x.abs().amax(-1).double() / 127).float().clamp(min=2.0 ** -126)
    codes = torch.round(x.double() / scale.double()[..., None])
    s["codes"][:, dst], s["scales"][:, dst] = codes.to(torch.int8), scale
    s["back"][:, src] = (s["codes"][:, dst].float() * s["scales"][:, dst][..., None]).to(s["back"].dtype)
    return s["back"]


# ---------------------------------------------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------------------------------------------
def _run_own_norm(s):
    from gated_deltanet_recurrence_gdn_amd import binding as gdn

    case, x, r = s["case"], s["x"], s["stored"]
    res = {} if r is None else {"residual": r}
    if case["out"] == "plain":
        gdn.gdn_norm_forward(x, s["weight"], out=s["out"], residual=s["residual"], residual_out=r, eps=EPS,
                             weight_offset=case["offset"])
        res["out"] = s["out"]
    else:
        gdn.gdn_norm_forward(x, s["weight"], codes=s["codes"], scales=s["scales"], residual=s["residual"], residual_out=r,
                             eps=EPS, weight_offset=case["offset"])
        res.update(codes=s["codes"], scales=s["scales"][:, :_cut(case["width"])])
    if case["kind"] == "norm_train":
        gdn.gdn_norm_backward(s["dout"], x if r is None else r, s["weight"], s["dx"], s["dweight"], dresidual=s["dresidual"],
                              eps=EPS, weight_offset=case["offset"])
        res.update(dx=s["dx"], dweight=s["dweight"])
    return res


def _run_own_gated(s):
    from gated_deltanet_recurrence_gdn_amd import binding as gdn

    case = s["case"]
    if case["out"] == "plain":
        gdn.gdn_gated_norm_forward(s["x"], s["z"], s["weight"], out=s["out"], eps=EPS)
        res = {"out": s["out"]}
    else:
        gdn.gdn_gated_norm_forward(s["x"], s["z"], s["weight"], codes=s["codes"], scales=s["scales"], eps=EPS)
        res = {"codes": s["codes"], "scales": s["scales"][:, :_cut(case["heads"] * case["d"])]}
    if case["kind"] == "gated_train":
        gdn.gdn_gated_norm_backward(s["dout"], s["x"], s["z"], s["weight"], s["dx"], s["dz"], s["dweight"], eps=EPS)
        res.update(dx=s["dx"], dz=s["dz"], dweight=s["dweight"])
    return res


def _run_own_project(s):
    from gated_deltanet_recurrence_gdn_amd import binding as gdn

    gdn.gdn_project(s["a"], s["a_scales"], s["w"], s["w_scales"], s["outs"])
    return s["outs"]


def _run_own_pool(s):
    from gated_deltanet_recurrence_gdn_amd import binding as gdn

    if s["case"]["kind"] == "unpack":
        gdn.gdn_pool_unpack(s["codes"], s["scales"], s["pool"], s["src"], s["dst"])
        return s["pool"]
    gdn.gdn_pool_pack(s["pool"], s["codes"], s["scales"], s["src"], s["dst"])
    gdn.gdn_pool_unpack(s["codes"], s["scales"], s["back"], s["dst"], s["src"])
    return s["back"]


def run(state):
    kind = state["case"]["kind"]
    if kind in ("norm", "norm_train"):
        return _run_own_norm(state) if own else _run_plain_norm(state)
    if kind in ("gated", "gated_train"):
        return _run_own_gated(state) if own else _run_plain_gated(state)
    if kind == "project":
        return _run_own_project(state) if own else _run_plain_project(state)
    return _run_own_pool(state) if own else _run_plain_pool(state)


# ---------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def _exact_codes(y):
    """e4m3 by its definition: three bits after the leading one, steps of 2^-9 below 2^-6, ties to even."""
    rows, width = y.shape
    codes, scales = torch.empty_like(y), y.new_empty(rows, _cut(width))
    for g in range(_cut(width)):
        v = y[:, g * GROUP:(g + 1) * GROUP]
        top = v.abs().amax(1, keepdim=True)
        e = torch.ceil(torch.log2(top / 448))
        e = torch.where(top <= 448 * torch.exp2(e - 1), e - 1, torch.where(top > 448 * torch.exp2(e), e + 1, e))
        p = torch.exp2(torch.where(top > 0, e, -126).clamp(-126, 127))
        v = v / p
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        codes[:, g * GROUP:(g + 1) * GROUP], scales[:, g:g + 1] = torch.round(v / step) * step, p
    return {"codes": codes, "scales": scales}


def _exact_norm(case, seed):
    s = _norm_inputs(case, seed)
    r = s["x"] if s["residual"] is None else (s["x"].double() + s["residual"].double()).to(s["residual"].dtype)
    train = case["kind"] == "norm_train"
    v, w = r.double().requires_grad_(train), (s["weight"].double() + case["offset"]).requires_grad_(train)
    with torch.enable_grad():
        y = w * v * (v.pow(2).sum(-1, keepdim=True) / case["width"] + EPS).rsqrt()
    res = {} if s["residual"] is None else {"residual": r.double()}
    res.update({"out": y.detach()} if case["out"] == "plain" else _exact_codes(y.detach()))
    if train:
        dv, dw = torch.autograd.grad(y, [v, w], s["dout"].double())
        res.update(dx=dv if s["dresidual"] is None else dv + s["dresidual"].double(), dweight=dw)
    return res


def _exact_gated(case, seed):
    s = _gated_inputs(case, seed)
    train = case["kind"] == "gated_train"
    x, z, w = (s[n].double().requires_grad_(train) for n in ("x", "z", "weight"))
    with torch.enable_grad():
        y = w * x * (x.pow(2).sum(-1, keepdim=True) / case["d"] + EPS).rsqrt() * (z * torch.sigmoid(z))
    d = y.detach()
    res = {"out": d} if case["out"] == "plain" else _exact_codes(d.reshape(case["rows"], -1))
    if train:
        dx, dz, dw = torch.autograd.grad(y, [x, z, w], s["dout"].double())
        res.update(dx=dx, dz=dz, dweight=dw)
    return res


def _exact_project(case, seed):
    s = _project_inputs(case, seed)
    y = torch.zeros(case["tokens"], sum(s["parts"]), dtype=torch.float64, device=DEV)
    for g in range(_cut(case["inner"])):
        a, w = (s[n][:, g * GROUP:(g + 1) * GROUP].double() for n in ("a", "w"))
        by = s["w_scales"][:, g].double().repeat_interleave(GROUP)[:w.shape[0]]
        y += s["a_scales"][:, g].double()[:, None] * (a @ w.T.contiguous()) * by
    return list(y.split(s["parts"], 1))


def _exact_pool(case, seed):
    s = _pool_inputs(case, seed)
    keep = s["pool"] if case["kind"] == "unpack" else s["back"]
    res = torch.zeros(keep.shape, dtype=torch.float64, device=DEV)
    for layer in range(case["layers"]):
        res[layer] = keep[layer]
    for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
        for layer in range(case["layers"]):
            if case["kind"] == "unpack":
                res[layer, b] = s["codes"][layer, a].double() * s["scales"][layer, a].double()[..., None]
            else:
                x = s["pool"][layer, a].double()
                scale = (x.abs().amax(-1, keepdim=True) / 127).float().double()  # the scale is kept in 32 bits
                res[layer, a] = torch.round(x / scale) * scale
    return res


def exact(case, seed):
    kind = case["kind"]
    return (_exact_norm if kind in ("norm", "norm_train") else _exact_gated if kind in ("gated", "gated_train")
            else _exact_project if kind == "project" else _exact_pool)(case, seed)


# ---------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------
def work(case):
    """Each input read once and each output written once; a product's operations, a norm's few an element."""
    kind, size = case["kind"], {"f32": 4, "bf16": 2, "f16": 2, "none": 0}
    if kind in ("norm", "norm_train"):
        n, x, r = case["rows"] * case["width"], size[case["dtype"]], size[case["residual"]]
        bytes_ = n * (x + 2 * r) + 2 * case["width"] + (n * x if case["out"] == "plain" else n + case["rows"] * _cut(case["width"]))
        if kind == "norm_train":  # dout and dresidual in, dx and the weight's gradient out
            bytes_ += n * (x + r + (r or x)) + 4 * case["width"]
        return {"bytes": bytes_, "flops": n * (6 if kind == "norm" else 16)}
    if kind in ("gated", "gated_train"):
        n, x, z = case["rows"] * case["heads"] * case["d"], size[case["x"]], size[case["z"]]
        bytes_ = n * (x + z) + 4 * case["d"] + (n * z if case["out"] == "plain" else n + case["rows"] * _cut(case["heads"] * case["d"]))
        if kind == "gated_train":
            bytes_ += n * (2 * z + x) + 4 * case["d"]
        return {"bytes": bytes_, "flops": n * (10 if kind == "gated" else 30)}
    if kind == "project":
        M, K, N = case["tokens"], case["inner"], sum(int(x) for x in case["columns"].split(","))
        scales = M * _cut(K) + _cut(N) * _cut(K) * (4 if case["scales"] == "f32" else 1)
        return {"bytes": M * K + N * K + scales + 2 * M * N, "flops": 2 * M * N * K}
    row = case["layers"] * case["h_v"] * case["d"] ** 2
    packed, state = row * (1 + 4 / case["d"]), row * size[case["dtype"]]
    n = case["n"]
    return {"bytes": n * (packed + state) * (2 if kind == "pack" else 1) + 8 * n, "flops": 3 * n * row}
