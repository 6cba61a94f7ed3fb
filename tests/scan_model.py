"""The training scan's chunk algebra in float64 on the host, with its matrix products taken apart as the kernels take
them: each operand in up to three bf16 parts, six of the nine partial products.  It says what a lost partial product does
to each result; everything else in it is exact, or (rounded) carries the roundings of the kernels' sums.
"""
import torch

CHUNK = 64
# the partial products that are formed, by the parts of either side
KEPT = [(2, 0), (0, 2), (1, 1), (1, 0), (0, 1), (0, 0)]


def parts(x):
    """The three bf16 parts of fp32 values, each the rest of the one before rounded to nearest even; exact together."""
    x, r = x.float(), []
    for _ in range(3):
        r.append(x.to(torch.bfloat16).float())
        x = x - r[-1]
    return [p.double() for p in r]


class Model:
    """lost: the product and the partial product (parts of its left and right side) that is left out, or None.
    rounded: sums are rounded to fp32 as the matrix instructions' accumulators are, and what is formed from them too."""

    def __init__(self, lost=None, rounded=False):
        self.lost, self.rounded, self.seen = lost, rounded, {}

    def f(self, x):
        return x.float().double() if self.rounded else x

    def mul(self, name, a, b):
        """a @ b, both rounded to fp32 first, as the kernels hold them; 32 of the inner index at a time, small partial
        products first."""
        pa, pb = parts(a), parts(b)
        formed = [(i, j) for i, j in KEPT if bool(pa[i].any()) and bool(pb[j].any())]
        self.seen[name] = self.seen.get(name, set()) | set(formed)
        s = torch.zeros(a.shape[0], b.shape[1], dtype=torch.float64)
        for k in range(0, a.shape[1], 32):
            for i, j in formed:
                if (name, i, j) != self.lost:
                    s = self.f(s + pa[i][:, k:k + 32] @ pb[j][k:k + 32])
        return s

    def scan(self, x, scale, dout, dfinal):
        """Results of one sequence with one q/k head and one value head (q [T][d_k], ..., state [d_v][d_k])."""
        x = {n: t.double() for n, t in x.items()}
        T, mul, f, tri = x["q"].shape[0], self.mul, self.f, torch.tril
        assert T % CHUNK == 0
        S, tape, outs = x["state"], [], []
        for t in range(0, T, CHUNK):
            q, k, v, al, be = (x[n][t:t + CHUNK] for n in ("q", "k", "v", "alpha", "beta"))
            b = al.log().cumsum(0)
            D = f(torch.exp((b[:, None] - b[None, :]).clamp(max=0)).tril())
            eb, er = f(b.exp()[:, None]), f((b[-1] - b).exp()[:, None])
            kk, qk = mul("KK", k, k.T), mul("QK", q, k.T)
            N, P = f(tri(D * kk, -1)), f(tri(D * qk))
            eye = torch.eye(CHUNK, dtype=torch.float64)
            Y = f(N @ torch.linalg.inv(eye + be[:, None] * N))
            E = f(v - mul("YV", Y * be, v))
            W = f(eb * k - mul("YK", Y * (be[:, None] * eb).T, k))
            E = f(E - mul("WS", W, S.T))
            U = be[:, None] * E
            outs.append(f(scale * (f(eb * mul("QS", q, S.T)) + mul("PE", P * be, E))))
            tape.append((t, S, E, Y, D, eb, er, b, kk, qk, P))
            S = f(f(b[-1].exp()) * S + mul("KU", (er * U).T, k))
        r = {"out": torch.cat(outs), "final": S}
        G, grads = dfinal.double(), {n: torch.zeros_like(x[n]) for n in ("q", "k", "v", "alpha", "beta")}
        for t, S, E, Y, D, eb, er, b, kk, qk, P in reversed(tape):
            q, k, v, al, be = (x[n][t:t + CHUNK] for n in ("q", "k", "v", "alpha", "beta"))
            bc, do = be[:, None], scale * dout.double()[t:t + CHUNK]
            Z = f(P - P @ (bc * Y))
            dR = f(scale * mul("ZO", Z.T, dout[t:t + CHUNK].double()))
            Wb = f(er * k - mul("YbK", (bc * er * Y).T, k))
            dR = f(dR + mul("WbG", Wb, G.T))
            os = mul("OS", dout[t:t + CHUNK].double(), S)
            rs, eg = mul("RS", dR, S), mul("EG", E, G)
            dp, da = mul("OE", dout[t:t + CHUNK].double(), E.T), mul("RE", dR, E.T)
            X = f(tri(-bc * D * be * da, -1))
            Ps = f(tri(scale * D * be * dp))
            oq, xk, ek = f(scale * eb * os), f(bc * eb * rs), f(er * bc * eg)
            grads["q"][t:t + CHUNK] = f(oq + mul("PK", Ps, k))
            grads["k"][t:t + CHUNK] = f(f(ek - xk + mul("XK", X + X.T, k)) + mul("PQ", Ps.T, q))
            grads["v"][t:t + CHUNK] = f(bc * dR)
            grads["beta"][t:t + CHUNK] = da.diagonal()
            M = f(tri(f(X * kk) + Ps * qk, -1))
            y, z = (q * oq - k * xk).sum(1), (k * ek).sum(1)
            c = torch.zeros(CHUNK + 1, CHUNK + 1, dtype=torch.float64)
            c[1:, 1:] = M.cumsum(0).cumsum(1)
            i = torch.arange(CHUNK)
            spans = c[CHUNK, i] - c[i, i]  # rows i >= t, columns j < t
            after = y.flip(0).cumsum(0).flip(0) + (z.cumsum(0) - z)
            grads["alpha"][t:t + CHUNK] = (spans + after + b[-1].exp() * (G * S).sum()) / al
            G = f(f(b[-1].exp()) * G + f(mul("QO", (eb * do).T, q) - mul("KR", (bc * eb * dR).T, k)))
        r.update({"d" + n: g for n, g in grads.items()}, dstate=G)
        return r


def off(a, b):
    return float((a - b).norm() / b.norm())


def errors(got, want):
    return {n: off(got[n], want[n]) for n in want}


# A result is the end of at most 6 chained products.  A product's sum is rounded once per 32 inner indices and partial
# product, 24 times at d_k = 128, each by at most half a step and on average by 2^-24 / sqrt(3) of it, at random: 2^-23 of
# its 2-norm.  `Model(rounded=True)` gives 0.7e-7 to 2.3e-7 for the results of `case`.
BAR = 6 * 2.0 ** -23


def typed_bar(dtype):
    """For a result rounded to `dtype` against the exact one rounded to it, relative to its 2-norm: where the result before
    rounding is off by d, the rounded one is off by a whole step u with probability d / u, so the squares' sum is
    sum u d <= eps |x| |d| <= eps BAR |x|^2 on average (u <= eps x).  Twice its root covers the spread."""
    return BAR if dtype == torch.float32 else 2 * (torch.finfo(dtype).eps * BAR) ** 0.5


def case(dtype, seed=0, T=128, d_k=64, d_v=32):
    """Inputs of one sequence and head in which every product weighs: keys and queries with a common direction (a full
    triangular matrix), states and their gradients of the values' size, memory over more than a chunk."""
    g = torch.Generator().manual_seed(seed)

    def n(*s):
        return torch.randn(*s, generator=g)

    common = n(1, d_k)
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)  # noqa: E731
    x = {"q": unit(n(T, d_k) + common).to(dtype).float(), "k": unit(n(T, d_k) + common).to(dtype).float(),
         "v": n(T, d_v).to(dtype).float(), "alpha": torch.exp(-torch.nn.functional.softplus(-4 + n(T))),
         "beta": torch.sigmoid(1 + n(T)), "state": 2 * n(d_v, d_k)}
    return x, n(T, d_v).to(dtype).float(), 2 * n(d_v, d_k)


SCALE = 0.5


def exact(x, dout, dfinal):
    """The rule's results for `case`, token by token."""
    from scan_reference import reference

    full = {n: t[None, None] if n == "state" else t[:, None] for n, t in x.items()}
    r = reference(full, [x["q"].shape[0]], SCALE, dout[:, None], dfinal[None, None])
    return {n: t[0, 0] if n in ("final", "dstate") else t[:, 0] for n, t in r.items()}
