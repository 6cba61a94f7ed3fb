"""The norms, the 8-bit formats, the projections and the 8-bit state rows in float64, from their definitions, and
bounds of what fp32 arithmetic may lose.  U is half a step of fp32: one rounding is off by at most U of the value."""
import torch

U = 2.0 ** -24
GROUP = 128
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -24}  # steps of subnormals


def cut(n):
    return -(-n // GROUP)


def groups(y):
    """[rows][width] -> [rows][groups][128], zeros behind the last channel."""
    rows, width = y.shape
    return torch.nn.functional.pad(y, (0, cut(width) * GROUP - width)).reshape(rows, cut(width), GROUP)


def exponent(top):
    """The smallest e >= -126 with top 2^-e <= 448."""
    m, e = torch.frexp(top.double())  # top = m 2^e, m in [0.5, 1)
    e = torch.where(m > 0.875, e - 8, e - 9)
    return torch.where(top > 0, e, -126).clamp(min=-126)


def e4m3(x):
    """The nearest e4m3 value, ties to even (|x| <= 448)."""
    a = x.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(x) * torch.round(a / step) * step


def check_codes(y, codes, scales, loss):
    """codes and scales are those of some y' with |y' - y| <= loss |y|: each between those of the ends."""
    rows, width = y.shape
    got = codes.float().double()
    byte = scales.view(torch.uint8)[:, :cut(width)].long()
    top = groups(y).abs().amax(-1)
    assert torch.all(byte >= exponent(top * (1 - loss)) + 127) and torch.all(byte <= exponent(top * (1 + loss)) + 127)
    down = torch.exp2(127 - byte.double()).repeat_interleave(GROUP, 1)[:, :width]
    low, high = e4m3(y.abs() * (1 - loss) * down), e4m3((y.abs() * (1 + loss) * down).clamp(max=448))
    assert torch.all((got.abs() >= low) & (got.abs() <= high))
    assert torch.all((got == 0) | (torch.sign(got) == torch.sign(y)))


def values(codes, scales, rows=1):
    """What codes stand for; a scale holds for `rows` rows and 128 columns."""
    s = scales.float().double().repeat_interleave(rows, 0)[:codes.shape[0]]
    return codes.float().double() * s.repeat_interleave(GROUP, 1)[:, :codes.shape[1]]


def near(got, want, slack):
    """|got - want| <= slack (tensor or number) plus the rounding to got's type, element by element."""
    w = want.double()
    off = (got.double() - w).abs()
    t = got.dtype
    most = slack + HALF[t] * (w.abs() + slack) + TINY[t]
    bad = ~(off <= most)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {float((off / most).nan_to_num(9e9).max()):.3g} of the bound"


# --- norm -------------------------------------------------------------------------------------------------------
# The sum of squares goes through at most 8 multiply-adds a vector, 4 vectors, 6 steps in a wave and 16 waves (35
# roundings, all terms positive); 1 / sqrt halves that and adds its own: division, sum, square root, division. 22 U.
RS = 22 * U
NORM = RS + 4 * U   # the product with s, w + w0, the product with it


def norm(r, w, eps):
    r, w = r.double(), w.double()
    rs = 1 / torch.sqrt(r.square().mean(-1, keepdim=True) + eps)
    return r * rs * w, rs


def norm_gradients(dout, r, w, eps, dresidual=None):
    """dx, dw and what fp32 may lose of them."""
    d, r, w = dout.double(), r.double(), w.double()
    y, rs = norm(r, w, eps)
    g, n = d * w, r * rs
    m = (g * n).mean(-1, keepdim=True)
    dx = rs * (g - n * m)
    # s twice in the second term, its mean's sum as the squares' (35 U of the magnitudes), five products
    lost = rs * (g.abs() * (RS + 5 * U) + n.abs() * (g * n).abs().mean(-1, keepdim=True) * (3 * RS + 45 * U))
    if dresidual is not None:
        dx = dx + dresidual.double()
        lost = lost + U * (dx.abs() + lost)
    dn = (d * n).flatten(0, -2)
    rows = dn.shape[0]
    return dx, lost, dn.sum(0), dn.abs().sum(0) * (RS + (2 + rows + 64) * U)


# --- gated norm -------------------------------------------------------------------------------------------------
# a head has at most 32 lanes: 8 + 5 (or 32) roundings, then as above; the gate: exponential and reciprocal 6 U
HEAD = 22 * U
GATE = 8 * U
GATED = HEAD + GATE + 4 * U


def gated(x, z, w, eps):
    x, z, w = x.double(), z.double(), w.double()
    rs = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    return x * rs * w * (z * torch.sigmoid(z)), rs


def gated_gradients(dout, x, z, w, eps):
    d, x, z, w = dout.double(), x.double(), z.double(), w.double()
    _, rs = gated(x, z, w, eps)
    a = torch.sigmoid(z)
    n, gate = x * rs, z * a
    g = d * gate * w
    m = (g * n).mean(-1, keepdim=True)
    dx = rs * (g - n * m)
    dx_lost = rs * (g.abs() * (HEAD + GATE + 6 * U) + n.abs() * (g * n).abs().mean(-1, keepdim=True) * (3 * HEAD + GATE + 45 * U))
    dz = d * n * w * a * (1 + z * (1 - a))
    dz_lost = (d * n * w).abs() * a * ((1 + z.abs() * (1 - a)) * (HEAD + GATE + 8 * U) + z.abs() * a * GATE)
    dn = d * n * gate
    terms = dn.shape.numel() // dn.shape[-1]
    return dx, dx_lost, dz, dz_lost, dn.flatten(0, -2).sum(0), dn.abs().flatten(0, -2).sum(0) * (HEAD + GATE + (4 + min(terms, 64) + terms / 1024 + 160) * U)


# --- projections ------------------------------------------------------------------------------------------------
def project(a, a_scales, w, w_scales):
    """y, and what the matrix instruction may lose of it: products within a group are aligned to the largest and cut
    16 bits below it at the latest, which takes at most 2^-16 of the largest from each of the 128."""
    x, v = values(a, a_scales), values(w, w_scales, GROUP)
    lost = groups(x).abs().amax(-1) @ groups(v).abs().amax(-1).T * (GROUP * 2.0 ** -16)
    y = x @ v.T
    return y, lost + U * cut(a.shape[1]) * (x.abs() @ v.abs().T)


# --- state rows in 8 bits ---------------------------------------------------------------------------------------
def pack(states):
    x = states.double()
    top = x.abs().amax(-1)
    bad = ~torch.isfinite(x).all(-1)
    scale = (top / 127).float().clamp(min=2.0 ** -126)  # of 24 bits by one rounding: 53 bits are more than 2 * 24 + 2
    codes = torch.round(x / scale.double()[..., None])
    return torch.where(bad[..., None], 0, codes).to(torch.int8), torch.where(bad, float("nan"), scale)
