"""Plain 64-bit reference of linear attention with a decay for each head, written from its
definition: loops over sequences and tokens, torch on the CPU."""
import torch


def wide(t):
    return None if t is None else t.detach().cpu().double()


def _of_heads(t, heads):
    return t.repeat_interleave(heads // t.shape[1], 1)


def attention(q, k, v, g, beta, D, scale, cu, start, keep=None):
    """(out, last states): out has NaN outside the sequences.  start (nseq, heads, dk, dv).  keep: a
    list that takes (token, state before it, state after it)."""
    h = v.shape[1]
    q, k = _of_heads(q, h), _of_heads(k, h)
    g = g.expand(v.shape[0], h)
    out, last = torch.full_like(v, float("nan")), start.clone()
    for s in range(len(cu) - 1):
        S = start[s].clone()
        for t in range(cu[s], cu[s + 1]):
            w = k[t] if beta is None else beta[t][:, None] * k[t]
            before, S = S, torch.exp(g[t])[:, None, None] * S + w[:, :, None] * v[t][:, None]
            out[t] = scale * (q[t][:, :, None] * S).sum(1) + (0.0 if D is None else D[:, None] * v[t])
            if keep is not None:
                keep.append((t, before, S))
        last[s] = S
    return out, last


def gradients(q, k, v, g, beta, D, scale, cu, start, dout, dfinal, telescoped=False):
    """Gradients of sum(dout out) + sum(dfinal last), by the adjoint; zero outside the sequences.
    telescoped: dlog_decay as the sum of absolute terms that the kernels form it from (for error
    bounds, on absolute values)."""
    h, rq, rk = v.shape[1], v.shape[1] // q.shape[1], v.shape[1] // k.shape[1]
    keep = []
    _, last = attention(q, k, v, g, beta, D, scale, cu, start, keep)
    states = {t: (b, a) for t, b, a in keep}
    qh, kh = _of_heads(q, h), _of_heads(k, h)
    ge = g.expand(v.shape[0], h)
    dq, dk, dv = torch.zeros_like(qh), torch.zeros_like(kh), torch.zeros_like(v)
    dg, db, dD, d0 = torch.zeros_like(ge), torch.zeros_like(ge), torch.zeros(h).double(), dfinal.clone()
    for s in range(len(cu) - 1):
        R = dfinal[s].clone()  # the gradient of the state after token t, from the tokens behind it
        edge = (R * last[s]).sum((1, 2))
        for t in range(cu[s + 1] - 1, cu[s] - 1, -1):
            before, after = states[t]
            R = R + scale * qh[t][:, :, None] * dout[t][:, None]
            b = torch.ones(h).double() if beta is None else beta[t]
            dq[t] = scale * (after * dout[t][:, None]).sum(2)
            Rv = (R * v[t][:, None]).sum(2)
            dk[t] = b[:, None] * Rv
            dv[t] = b[:, None] * (R * kh[t][:, :, None]).sum(1)
            if D is not None:
                dv[t] += D[:, None] * dout[t]
                dD += (dout[t] * v[t]).sum(1)
            db[t] = (kh[t] * Rv).sum(1)
            edge = edge + (qh[t] * dq[t]).sum(1) + b * db[t]
            dg[t] = edge if telescoped else torch.exp(ge[t]) * (R * before).sum((1, 2))
            R = torch.exp(ge[t])[:, None, None] * R
        d0[s] = R
    group = lambda x, r: x.unflatten(1, (-1, r)).sum(2)
    res = {"dq": group(dq, rq), "dk": group(dk, rk), "dv": dv, "dlog_decay": dg.sum(0) if g.ndim == 1 else dg,
           "dinitial_state": d0}
    if beta is not None:
        res["dbeta"] = db
    if D is not None:
        res["dD"] = dD
    return res
