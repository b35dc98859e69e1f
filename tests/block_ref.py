"""Plain 64-bit references of the operators around the scan, written from their definitions:
loops over sequences, rows and steps, numpy on the CPU."""
import numpy as np


def bf16_bits(a):
    """float32 array -> the bf16 bits nearest to it (ties to even), as uint16."""
    u = np.ascontiguousarray(a, dtype=np.float32).view(np.uint32).astype(np.uint64)
    return (((u + 0x7FFF + ((u >> 16) & 1)) >> 16) & 0xFFFF).astype(np.uint16)


def widen(a):
    """float64 values of a float32 array or of bf16 bits (uint16)."""
    if a is None:
        return None
    if a.dtype == np.uint16:
        return (a.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    return a.astype(np.float64)


def silu(v):
    return v / (1.0 + np.exp(-v))


def softplus(v):
    return np.maximum(v, 0.0) + np.log1p(np.exp(-np.abs(v)))


def slots_of(nseq, slots, idx):
    """The slot of each sequence; None where its index is none."""
    idx = list(range(nseq)) if idx is None else [int(i) for i in idx]
    return [i if 0 <= i < slots else None for i in idx]


def packed_conv(x, w, b, cu, state, idx, initial, act):
    """(out, new state, |terms|): out has NaN outside the sequences; |terms| is the sum of the
    absolute values that each output adds up, for error bounds."""
    x, w, b = widen(x), widen(w), widen(b)
    t, d = x.shape
    width = w.shape[1]
    st = None if state is None else widen(state)
    out, mag = np.full((t, d), np.nan), np.zeros((t, d))
    where = slots_of(len(cu) - 1, 0 if st is None else len(st), idx)
    for s in range(len(cu) - 1):
        x_s = x[cu[s]:cu[s + 1]]
        if len(x_s) == 0:
            continue
        past = np.zeros((width - 1, d))
        if where[s] is not None and initial is not None and initial[s]:
            past = st[where[s]].copy()
        line = np.concatenate([past, x_s])
        for i in range(len(x_s)):
            terms = w.T * line[i:i + width]
            v = terms.sum(0) + (b if b is not None else 0.0)
            out[cu[s] + i] = silu(v) if act else v
            mag[cu[s] + i] = np.abs(terms).sum(0) + (np.abs(b) if b is not None else 0.0)
        if where[s] is not None:
            st[where[s]] = line[len(x_s):]
    return out, st, mag


def conv_forward(x, w, b, act):
    """Dense (batch, seqlen, dim) forward."""
    bt, length, d = x.shape
    width = w.shape[1]
    line = np.concatenate([np.zeros((bt, width - 1, d)), x], 1)
    v = np.zeros_like(x) + (b if b is not None else 0.0)
    for k in range(width):
        v = v + w[:, k] * line[:, k:k + length]
    return silu(v) if act else v


def conv_backward(x, w, b, dout, act):
    """(dx, dweight, dbias) by the formulas; with the sums of absolute terms of each."""
    bt, length, d = x.shape
    width = w.shape[1]
    line = np.concatenate([np.zeros((bt, width - 1, d)), x], 1)
    dv = dout.copy()
    if act:
        v = np.zeros_like(x) + (b if b is not None else 0.0)
        for k in range(width):
            v = v + w[:, k] * line[:, k:k + length]
        s = 1.0 / (1.0 + np.exp(-v))
        dv = dout * s * (1.0 + v * (1.0 - s))
    dx, dx_mag = np.zeros_like(x), np.zeros_like(x)
    dw, dw_mag = np.zeros((d, width)), np.zeros((d, width))
    for k in range(width):
        back = width - 1 - k  # out[t] reads x[t - back] with w[:, k]
        n = length - back
        if n > 0:
            dx[:, :n] += w[:, k] * dv[:, back:]
            dx_mag[:, :n] += np.abs(w[:, k] * dv[:, back:])
        dw[:, k] = (dv * line[:, k:k + length]).sum((0, 1))
        dw_mag[:, k] = np.abs(dv * line[:, k:k + length]).sum((0, 1))
    return (dx, dw, dv.sum((0, 1))), (dx_mag, dw_mag, np.abs(dv).sum((0, 1)))


def packed_scan(x, delta, A, B, C, D, z, cu, state, idx, initial, bias, soft):
    """(y, new state); y has NaN outside the sequences."""
    x, delta, A, B, C, D, z, bias = (widen(v) for v in (x, delta, A, B, C, D, z, bias))
    t, d = x.shape
    st = None if state is None else widen(state)
    y = np.full((t, d), np.nan)
    where = slots_of(len(cu) - 1, 0 if st is None else len(st), idx)
    step = delta + (bias if bias is not None else 0.0)
    if soft:
        step = softplus(step)
    for s in range(len(cu) - 1):
        if cu[s + 1] == cu[s]:
            continue
        h = np.zeros(A.shape)
        if where[s] is not None and initial is not None and initial[s]:
            h = st[where[s]].copy()
        for i in range(cu[s], cu[s + 1]):
            with np.errstate(invalid="ignore"):
                a = np.exp(np.where(step[i][:, None] == 0, 0.0, step[i][:, None] * A))
            h = a * h + (step[i] * x[i])[:, None] * B[i]
            y[i] = h @ C[i] + (D * x[i] if D is not None else 0.0)
            if z is not None:
                y[i] *= silu(z[i])
        if where[s] is not None:
            st[where[s]] = h
    return y, st


def grouped(v, group):
    return v.reshape(v.shape[0], -1, group)


def rstd_of(v, group, eps):
    """(rows, groups) factors (mean(v^2) + eps)^-1/2."""
    return 1.0 / np.sqrt((grouped(v, group) ** 2).mean(-1) + eps)


def spread(r, group):
    return np.repeat(r, group, axis=1)


def gated_norm(x, w, z, group, eps, norm_first):
    """(out, rstd)."""
    gate = silu(z) if z is not None else np.ones_like(x)
    u = x if norm_first else x * gate
    r = rstd_of(u, group, eps)
    out = u * spread(r, group) * w
    return (out * gate if norm_first else out), r


def gated_norm_grad(dout, x, w, z, rstd, group, norm_first):
    """{name: (gradient, sum of absolute terms)} from the forward's factors."""
    mean = lambda v: spread(grouped(v, group).mean(-1), group)
    r = spread(rstd, group)
    gate = silu(z) if z is not None else np.ones_like(x)
    hat = x * r * (1.0 if norm_first else gate)
    dn = dout * (gate if norm_first else 1.0)
    g = dn * w
    du = r * (g - hat * mean(g * hat))
    du_mag = r * (np.abs(g) + np.abs(hat) * mean(np.abs(g * hat)))
    res = {"dx": (du, du_mag) if norm_first else (du * gate, du_mag * np.abs(gate)),
           "dweight": ((dn * hat).sum(0), np.abs(dn * hat).sum(0))}
    if z is not None:
        s = 1.0 / (1.0 + np.exp(-z))
        slope = s * (1.0 + z * (1.0 - s))
        dgate, mag = (dout * hat * w, np.abs(dout * hat * w)) if norm_first else (du * x, du_mag * np.abs(x))
        # the slope's own terms, s and s z (1 - s), cancel near its zero
        res["dz"] = (dgate * slope, mag * s * (1.0 + np.abs(z)))
    return res


def residual_norm(x, w, h, wp, scale, alpha, eps):
    """(out, residual_out, rstd, rstd_post, sum of absolute terms of residual_out)."""
    v, rp = x, None
    if wp is not None:
        rp = rstd_of(x, x.shape[1], eps)
        v = x * rp * wp
    v = v * alpha * (scale if scale is not None else 1.0)
    new = v if h is None else h + v
    r = rstd_of(new, x.shape[1], eps)
    return new * r * w, new, r, rp, np.abs(v) + (np.abs(h) if h is not None else 0.0)


def residual_norm_grad(dout, dnew, x, w, new, rstd, wp, scale, rstd_post, alpha):
    """{name: (gradient, sum of absolute terms)} from the forward's results."""
    mean = lambda v: v.mean(-1, keepdims=True)
    hat = new * rstd
    g = dout * w
    dh = rstd * (g - hat * mean(g * hat))
    mag = rstd * (np.abs(g) + np.abs(hat) * mean(np.abs(g * hat)))
    if dnew is not None:
        dh, mag = dh + dnew, mag + np.abs(dnew)
    s = alpha * (scale if scale is not None else 1.0)
    dv, dv_mag = dh * s, mag * np.abs(s)
    res = {"dresidual": (dh, mag), "dweight": ((dout * hat).sum(0), np.abs(dout * hat).sum(0))}
    xh = x * rstd_post if wp is not None else x
    if scale is not None:
        p = xh * (wp if wp is not None else 1.0)
        res["dscale"] = ((alpha * dh * p).sum(0), np.abs(alpha * mag * p).sum(0))
    if wp is None:
        res["dx"] = (dv, dv_mag)
        return res
    res["dpost_weight"] = ((dv * xh).sum(0), (dv_mag * np.abs(xh)).sum(0))
    g, g_mag = dv * wp, dv_mag * np.abs(wp)
    res["dx"] = (rstd_post * (g - xh * mean(g * xh)), rstd_post * (g_mag + np.abs(xh) * mean(g_mag * np.abs(xh))))
    return res
