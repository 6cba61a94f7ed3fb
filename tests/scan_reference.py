"""The training scan in float64 on the host: the rule token by token, gradients by automatic differentiation of it."""
import torch


def rule(q, k, v, alpha, beta, state, lens, scale):
    """out [total][h_v][d_v] and final states [B][h_v][d_v][d_k] of packed sequences (all float64)."""
    group = v.shape[1] // q.shape[1]
    q, k = q.repeat_interleave(group, 1), k.repeat_interleave(group, 1)
    outs, finals, t = [], [], 0
    for b, n in enumerate(lens):
        S = state[b]
        for i in range(t, t + n):
            a, be = alpha[i, :, None, None], beta[i, :, None]
            e = v[i] - alpha[i, :, None] * (S * k[i, :, None, :]).sum(-1)
            S = a * S + (be * e)[:, :, None] * k[i, :, None, :]
            outs.append(scale * (S * q[i, :, None, :]).sum(-1))
        finals.append(S)
        t += n
    return (torch.stack(outs) if outs else v.new_zeros(0, *v.shape[1:])), torch.stack(finals)


def reference(x, lens, scale, dout=None, dfinal=None):
    """out and final of the inputs in `x` (a dict of tensors), and the gradients where dout is given."""
    y = {n: t.detach().double().cpu().clone().requires_grad_(dout is not None) for n, t in x.items()}
    out, final = rule(y["q"], y["k"], y["v"], y["alpha"], y["beta"], y["state"], lens, scale)
    r = {"out": out.detach(), "final": final.detach()}
    if dout is not None:
        loss = (out * dout.double().cpu()).sum()
        if dfinal is not None:
            loss = loss + (final * dfinal.double().cpu()).sum()
        if not loss.requires_grad:
            grads = [torch.zeros_like(t) for t in y.values()]
        else:
            grads = torch.autograd.grad(loss, list(y.values()), allow_unused=True)
            grads = [torch.zeros_like(t) if g is None else g for g, t in zip(grads, y.values())]
        r.update({"d" + n: g for n, g in zip(y, grads)})
    return r
