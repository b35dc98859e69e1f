"""The cases on which the operators around the selective scan are measured: the short causal
convolution and the scan over packed prompts and single tokens with their state caches, the
convolution's gradients, and the norms after the scan (gated) and between blocks (residual).

`run` computes a case with elementary torch operations (`own` false) or with this library's
kernels (`own` true); `exact` computes the same outputs from the definitions in 64 bits.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one generated token for each of four chats: the conv step of a d_inner 5120 layer, all latency
        dict(name="conv step 4", op="conv", form="step", tokens=4, seqs=4, dim=5120, width=4, dtype="bf16"),
        # a prefill batch of ragged prompts through the conv, half of them continuing a cached history
        dict(name="conv prompts 16384", op="conv", form="prompts", tokens=16384, seqs=24, dim=5120, width=4,
             dtype="bf16"),
        # the conv's gradients in a training step of the same layer (x is half of the projection's rows)
        dict(name="conv gradients 2x8192x5120", op="conv_grad", batch=2, tokens=8192, dim=5120, width=4, dtype="bf16",
             silu=True),
        # the same for a small odd layer in fp32: nothing divides evenly
        dict(name="conv gradients 3x1001x777", op="conv_grad", batch=3, tokens=1001, dim=777, width=3, dtype="fp32",
             silu=False),
        # one token for each of three chats through the scan's state, fp32
        dict(name="scan step 3", op="scan", form="step", tokens=3, seqs=3, dim=2048, dstate=16, dtype="fp32"),
        # a full decode batch: 256 requests of a d_inner 5120 layer, bound by moving their states
        dict(name="scan step 256", op="scan", form="step", tokens=256, seqs=256, dim=5120, dstate=16,
             dtype="bf16"),
        # a ragged prefill batch of a d_inner 2048 layer, odd token count
        dict(name="scan prompts 9001", op="scan", form="prompts", tokens=9001, seqs=40, dim=2048, dstate=16,
             dtype="bf16"),
        # few long documents: parallelism has to come from the time axis
        dict(name="scan prompts 32768", op="scan", form="prompts", tokens=32768, seqs=3, dim=5120, dstate=16,
             dtype="bf16"),
        # the gated norm of a decode batch, groups of 640 channels, norm before the gate
        dict(name="gated norm 256", op="gated_norm", train=False, rows=256, dim=5120, groups=8, norm_first=True,
             dtype="bf16"),
        # the gated norm of a training step: fp32 scan output, gate first, forward and gradients
        dict(name="gated norm training 16384", op="gated_norm", train=True, rows=16384, dim=5120, groups=1,
             norm_first=False, dtype="bf16"),
        # residual add and the next block's norm for a decode batch of an odd size
        dict(name="residual norm 37", op="residual_norm", train=False, rows=37, dim=2560, post=False,
             dtype="bf16"),
        # norms on both sides of the block with a learned residual scale, forward and gradients
        dict(name="residual norm training 16384", op="residual_norm", train=True, rows=16384, dim=2560, post=True,
             dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    n = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n + 1 if n in (1536, 3072) and n < hi else n


def draw(rng):
    """One more case: sizes over the listed ranges, half of them with no even divisor."""
    op = rng.choice(["conv_step", "conv_prompts", "conv_grad", "scan_step", "scan_prompts", "gated_norm",
                     "residual_norm"])
    dim = _log_int(rng, 64, 8192)
    if rng.random() < 0.5:
        dim = dim // 128 * 128 + 64
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "conv_step":
        n = _log_int(rng, 1, 1024)
        return dict(op="conv", form="step", tokens=n, seqs=n, dim=dim, width=rng.randint(2, 5), dtype=dtype)
    if op == "conv_prompts":
        t = _log_int(rng, 16, min(32768, 80_000_000 // dim))
        return dict(op="conv", form="prompts", tokens=t, seqs=_log_int(rng, 1, max(1, t // 16)), dim=dim,
                    width=rng.randint(2, 5), dtype=dtype)
    if op == "conv_grad":
        b = rng.randint(1, 5)
        return dict(op="conv_grad", batch=b, tokens=_log_int(rng, 1, min(16384, 80_000_000 // dim // b)), dim=dim,
                    width=rng.randint(2, 5), dtype=dtype, silu=rng.random() < 0.7)
    if op == "scan_step":
        n = _log_int(rng, 1, 512)
        return dict(op="scan", form="step", tokens=n, seqs=n, dim=dim, dstate=rng.choice([8, 16, 16, 32]), dtype=dtype)
    if op == "scan_prompts":
        ns = rng.choice([8, 16, 16, 32])
        t = _log_int(rng, 16, min(32768, 1_300_000_000 // (dim * ns)))
        return dict(op="scan", form="prompts", tokens=t, seqs=_log_int(rng, 1, max(1, t // 16)), dim=dim, dstate=ns,
                    dtype=dtype)
    rows = _log_int(rng, 1, min(32768, 80_000_000 // dim))
    train = rng.random() < 0.5
    if op == "gated_norm":
        groups = rng.choice([1, 1, 2, 8])
        per_group = dim // groups
        dim = groups * (per_group + 1 if per_group * groups in (1536, 3072) else per_group)
        return dict(op="gated_norm", train=train, rows=rows, dim=dim, groups=groups, norm_first=rng.random() < 0.5,
                    dtype=dtype)
    return dict(op="residual_norm", train=train, rows=rows, dim=dim, post=rng.random() < 0.5, dtype=dtype)


# ------------------------------------------------------------------------------ the inputs
def _randn(gen, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, device="cuda", generator=gen) * scale).to(dtype)


def _packing(case, s, seed):
    """Where the packed sequences start, the cache slot of each (the last of a padded decode
    batch has none), which of them continue what their slot holds, and which leave it something."""
    rng = np.random.default_rng(seed)
    n, t = case["seqs"], case["tokens"]
    if case["form"] == "step":
        cu = np.arange(n + 1)
    else:  # ragged, empty ones among them
        cu = np.concatenate([[0], np.sort(rng.integers(0, t + 1, n - 1)), [t]])
    slots = n + 3
    idx = rng.permutation(slots)[:n].astype(np.int32)
    if n >= 8:
        idx[-1] = -1
    dev = lambda a: torch.from_numpy(a).to("cuda")
    s.update(cu=dev(cu.astype(np.int32)), idx=dev(idx), longest=int(np.max(np.diff(cu))), slots=slots,
             initial=dev(np.arange(n) % 2 == 0), kept=dev(np.flatnonzero((np.diff(cu) > 0) & (idx >= 0))))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    op, dim = case["op"], case["dim"]
    if op == "conv":
        _packing(case, s, seed)
        w = case["width"]
        # the input projection's rows hold x and the gate side by side
        s.update(x=_randn(gen, case["tokens"], 2 * dim, dtype=dt)[:, :dim], w=_randn(gen, dim, w, scale=w ** -0.5),
                 b=_randn(gen, dim, scale=0.1), state=_randn(gen, s["slots"], w - 1, dim, dtype=dt))
    elif op == "conv_grad":
        w, b, t = case["width"], case["batch"], case["tokens"]
        s.update(x=_randn(gen, b, t, 2 * dim, dtype=dt)[:, :, :dim], w=_randn(gen, dim, w, scale=w ** -0.5),
                 b=_randn(gen, dim, scale=0.1), dout=_randn(gen, b, t, dim, dtype=dt))
    elif op == "scan":
        _packing(case, s, seed)
        n, t = case["dstate"], case["tokens"]
        rank = max(4, dim // 32)
        # step sizes: softplus(delta + bias) between about 1e-3 and 1e-1
        step = torch.exp(torch.rand(dim, device="cuda", generator=gen) * math.log(100.0) + math.log(1e-3))
        bc = _randn(gen, t, rank + 2 * n, dtype=dt)  # the second projection's rows: rank, B, C
        s.update(x=_randn(gen, t, dim, dtype=dt), z=_randn(gen, t, 2 * dim, dtype=dt)[:, dim:],
                 delta=_randn(gen, t, dim, dtype=dt, scale=0.5), bias=step + torch.log(-torch.expm1(-step)),
                 A=-torch.exp(torch.rand(dim, n, device="cuda", generator=gen) * math.log(16.0)),
                 B=bc[:, rank:rank + n], C=bc[:, rank + n:], D=_randn(gen, dim),
                 state=_randn(gen, s["slots"], dim, n, scale=0.1))
    elif op == "gated_norm":
        r = case["rows"]
        s.update(x=_randn(gen, r, dim), z=_randn(gen, r, 2 * dim, dtype=dt)[:, dim:],
                 w=1.0 + _randn(gen, dim, scale=0.1))
        if case["train"]:
            s["dout"] = _randn(gen, r, dim, dtype=dt)
    else:
        r = case["rows"]
        s.update(x=_randn(gen, r, dim, dtype=dt), h=_randn(gen, r, dim, scale=2.0), w=1.0 + _randn(gen, dim, scale=0.1))
        if case["post"]:
            s.update(wp=1.0 + _randn(gen, dim, scale=0.1), scale=_randn(gen, dim, scale=0.3))
        if case["train"]:
            s.update(dout=_randn(gen, r, dim, dtype=dt), dh=_randn(gen, r, dim))
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        return {"conv": _own_conv, "conv_grad": _own_conv_grad, "scan": _own_scan, "gated_norm": _own_gated,
                "residual_norm": _own_residual}[op](s)
    return {"conv": _plain_conv, "conv_grad": _plain_conv_grad, "scan": _plain_scan, "gated_norm": _plain_gated,
            "residual_norm": _plain_residual}[op](s)


# ------------------------------------------------------------------- the library's kernels
def _own_conv(s):
    import selective_state_space_20_amd as sss
    if s["case"]["form"] == "step":
        out = sss.causal_conv1d_update(s["x"], s["w"], s["b"], conv_state=s["state"], state_indices=s["idx"], silu=True)
    else:
        out = sss.causal_conv1d_packed_fwd(s["x"], s["w"], s["b"], cu_seqlens=s["cu"], conv_state=s["state"],
                                           state_indices=s["idx"], has_initial=s["initial"], silu=True)
    return {"out": out, "state": s["state"]}


def _own_conv_grad(s):
    import selective_state_space_20_amd as sss
    return sss.causal_conv1d_bwd(s["x"], s["w"], s["b"], dout=s["dout"], silu=s["case"]["silu"])


def _own_scan(s):
    import selective_state_space_20_amd as sss
    y = torch.empty_like(s["x"])
    if s["case"]["form"] == "step":
        sss.selective_state_update_slots(s["x"], s["delta"], s["A"], s["B"], s["C"], s["D"], s["z"], state=s["state"],
                                         state_indices=s["idx"], delta_bias=s["bias"], delta_softplus=True, out=y)
    else:
        sss.selective_scan_packed_fwd(s["x"], s["delta"], s["A"], s["B"], s["C"], s["D"], s["z"], cu_seqlens=s["cu"],
                                      state=s["state"], state_indices=s["idx"], has_initial=s["initial"],
                                      delta_bias=s["bias"], delta_softplus=True, out=y)
    return {"y": y, "state": s["state"]}


def _own_gated(s):
    import selective_state_space_20_amd as sss
    c = s["case"]
    opt = dict(eps=EPS, group_size=c["dim"] // c["groups"], norm_before_gate=c["norm_first"])
    if not c["train"]:
        return {"out": sss.rms_norm_gated_fwd(s["x"], s["w"], s["z"], **opt)}
    out, rstd = sss.rms_norm_gated_fwd(s["x"], s["w"], s["z"], return_rstd=True, **opt)
    opt.pop("eps")
    return {"out": out, **sss.rms_norm_gated_bwd(s["dout"], s["x"], s["w"], s["z"], rstd=rstd, **opt)}


def _own_residual(s):
    import selective_state_space_20_amd as sss
    c = s["case"]
    opt = dict(post_weight=s.get("wp"), scale=s.get("scale"))
    if not c["train"]:
        out, h = sss.rms_norm_residual_fwd(s["x"], s["w"], s["h"], eps=EPS, **opt)
        return {"out": out, "h": h}
    out, h, rstd, rstd_post = sss.rms_norm_residual_fwd(s["x"], s["w"], s["h"], eps=EPS, return_rstd=True, **opt)
    g = sss.rms_norm_residual_bwd(s["dout"], s["dh"], x=s["x"], residual_out=h, weight=s["w"], rstd=rstd,
                                  rstd_post=rstd_post, **opt)
    return {"out": out, "h": h, **g}


# -------------------------------------------------------------------------- the plain forms
def _sequence_of(s, tokens):
    """Of each token: its sequence, and its position in it."""
    t = torch.arange(tokens, device="cuda")
    cu = s["cu"].long()
    seq = torch.searchsorted(cu, t, right=True) - 1
    return seq, t - cu[seq]


def _started(s):
    """Which sequences start from what their slot holds: every one of a decode step, the marked
    ones of a prefill batch, none without a slot."""
    kept = s["idx"] >= 0
    return kept if s["case"]["form"] == "step" else kept & s["initial"]


def _plain_conv(s):
    c = s["case"]
    w, t = c["width"], c["tokens"]
    dt, cu, idx = s["x"].dtype, s["cu"].long(), s["idx"].long()
    slot = idx.clamp(min=0)
    past = s["state"][slot].float() * _started(s)[:, None, None]  # (seqs, w - 1, dim), zero where none is kept
    kept = s["kept"]  # the sequences that have tokens and a slot
    if c["form"] == "step":
        line = torch.cat([past, s["x"].float()[:, None]], 1)
        v = (line * s["w"].t()).sum(1) + s["b"]
        s["state"][slot[kept]] = line[kept, 1:].to(dt)
        return {"out": (v * torch.sigmoid(v)).to(dt), "state": s["state"]}
    seq, pos = _sequence_of(s, t)
    # every sequence's history rows in front of the packed tokens: one row number for each tap
    rows = torch.cat([past.reshape(-1, c["dim"]), s["x"].float()])
    tap = pos[:, None] + torch.arange(w, device="cuda")  # w - 1 and above: a token of the sequence
    row = torch.where(tap >= w - 1, len(past) * (w - 1) + cu[seq][:, None] + tap - (w - 1), seq[:, None] * (w - 1) + tap)
    v = (rows[row] * s["w"].t()).sum(1) + s["b"]
    out = (v * torch.sigmoid(v)).to(dt)
    # the last w - 1 of (history, tokens)
    tap = (cu[1:] - cu[:-1])[kept][:, None] + torch.arange(w - 1, device="cuda")
    row = torch.where(tap >= w - 1, len(past) * (w - 1) + cu[kept][:, None] + tap - (w - 1),
                      kept[:, None] * (w - 1) + tap)
    s["state"][slot[kept]] = rows[row].to(dt)
    return {"out": out, "state": s["state"]}


def _plain_conv_grad(s):
    w = s["case"]["width"]
    x, dout = s["x"].float(), s["dout"].float()
    win = torch.nn.functional.pad(x, (0, 0, w - 1, 0)).unfold(1, w, 1)  # (batch, tokens, dim, width)
    dv = dout
    if s["case"]["silu"]:
        v = (win * s["w"]).sum(-1) + s["b"]
        sg = torch.sigmoid(v)
        dv = dout * sg * (1 + v * (1 - sg))
    ahead = torch.nn.functional.pad(dv, (0, 0, 0, w - 1)).unfold(1, w, 1)
    return {"dx": (ahead * s["w"].flip(1)).sum(-1).to(s["x"].dtype), "dweight": (win * dv[..., None]).sum((0, 1)),
            "dbias": dv.sum((0, 1))}


def _plain_scan(s):
    c = s["case"]
    cu, slot, kept = s["cu"].long(), s["idx"].long().clamp(min=0), s["kept"]
    x, z = s["x"].float(), s["z"].float()
    v = s["delta"].float() + s["bias"]
    step = torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))
    a = torch.exp(step[..., None] * s["A"])
    b = (step * x)[..., None] * s["B"].float()[:, None, :]
    # a sequence's first step starts from its cached state (or zero) and from nothing before it
    past = s["state"][slot] * _started(s)[:, None, None]
    if c["form"] == "step":
        b += a * past
    else:
        tokens = cu[1:] > cu[:-1]
        first = cu[:-1][tokens]
        b[first] += a[first] * past[tokens]
        a[first] = 0
    # each step's (decay, input) pair joined with those before it, twice as many in every round
    span = 1
    while span < s["longest"]:
        more = a[span:] * b[:-span]
        b[span:] += more
        a[span:] = a[span:] * a[:-span]
        span *= 2
    y = (b * s["C"].float()[:, None, :]).sum(-1) + s["D"] * x
    y = (y * z * torch.sigmoid(z)).to(s["x"].dtype)
    s["state"][slot[kept]] = b[cu[1:][kept] - 1]
    return {"y": y, "state": s["state"]}


def _plain_gated(s):
    c = s["case"]
    n, dim, dt = c["groups"], c["dim"], s["z"].dtype
    grouped = lambda v: v.reshape(v.shape[0], n, dim // n)
    x, z = s["x"], s["z"].float()
    sg = torch.sigmoid(z)
    gate = z * sg
    u = grouped(x if c["norm_first"] else x * gate)
    rstd = torch.rsqrt(u.square().mean(-1, keepdim=True) + EPS)
    hat = (u * rstd).reshape(x.shape)
    normed = hat * s["w"]
    out = normed * gate if c["norm_first"] else normed
    if not c["train"]:
        return {"out": out.to(dt)}
    dout = s["dout"].float()
    dnormed = dout * gate if c["norm_first"] else dout
    g = grouped(dnormed * s["w"])
    du = (rstd * (g - grouped(hat) * (g * grouped(hat)).mean(-1, keepdim=True))).reshape(x.shape)
    dgate = dout * normed if c["norm_first"] else du * x
    return {"out": out.to(dt), "dx": du if c["norm_first"] else du * gate,
            "dz": (dgate * sg * (1 + z * (1 - sg))).to(dt), "dweight": (dnormed * hat).sum(0)}


def _plain_residual(s):
    c = s["case"]
    dt = s["x"].dtype
    x = s["x"].float()
    if c["post"]:
        rp = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        v = x * rp * s["wp"]
        h = s["h"] + s["scale"] * v
    else:
        h = s["h"] + x
    rstd = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    hat = h * rstd
    res = {"out": (hat * s["w"]).to(dt), "h": h}
    if not c["train"]:
        return res
    dout = s["dout"].float()
    g = dout * s["w"]
    dh = s["dh"] + rstd * (g - hat * (g * hat).mean(-1, keepdim=True))
    res.update(dresidual=dh, dweight=(dout * hat).sum(0))
    if not c["post"]:
        return {**res, "dx": dh.to(dt)}
    dv = dh * s["scale"]
    g = dv * s["wp"]
    xh = x * rp
    return {**res, "dx": (rp * (g - xh * (g * xh).mean(-1, keepdim=True))).to(dt), "dpost_weight": (dv * xh).sum(0),
            "dscale": (dh * v).sum(0)}


# --------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "conv":
        return _exact_conv(s)
    if case["op"] == "scan":
        return _exact_scan(s)
    return {"conv_grad": _exact_conv_grad, "gated_norm": _exact_gated, "residual_norm": _exact_residual}[case["op"]](s)


def _silu64(v):
    return v / (1 + torch.exp(-v))


def _exact_conv(s):
    """Sequence by sequence: the history and the tokens in one row of time, then the taps."""
    c = s["case"]
    w = c["width"]
    cu, idx, started = s["cu"].tolist(), s["idx"].tolist(), _started(s).tolist()
    x, state, out = s["x"].double(), s["state"].double(), torch.empty(c["tokens"], c["dim"], dtype=torch.float64,
                                                                     device="cuda")
    wt, b = s["w"].double(), s["b"].double()
    for i in range(c["seqs"]):
        if cu[i + 1] == cu[i]:
            continue
        past = state[idx[i]] if started[i] else torch.zeros(w - 1, c["dim"], dtype=torch.float64, device="cuda")
        line = torch.cat([past, x[cu[i]:cu[i + 1]]])
        n = cu[i + 1] - cu[i]
        v = b + sum(wt[:, k] * line[k:k + n] for k in range(w))
        out[cu[i]:cu[i + 1]] = _silu64(v)
        if idx[i] >= 0:
            state[idx[i]] = line[n:]
    return {"out": out, "state": state}


def _exact_conv_grad(s):
    c = s["case"]
    w = c["width"]
    x, wt, b = (t.double().requires_grad_(True) for t in (s["x"], s["w"], s["b"]))
    line = torch.cat([torch.zeros(c["batch"], w - 1, c["dim"], dtype=torch.float64, device="cuda"), x], 1)
    v = b + sum(wt[:, k] * line[:, k:k + c["tokens"]] for k in range(w))
    out = _silu64(v) if c["silu"] else v
    dx, dw, db = torch.autograd.grad(out, (x, wt, b), s["dout"].double())
    return {"dx": dx, "dweight": dw, "dbias": db}


def _exact_scan(s):
    """The recurrence, one step of every sequence at a time."""
    c = s["case"]
    cu, idx = s["cu"].long(), s["idx"].long()
    x, z, A, B, C, D = (s[k].double() for k in ("x", "z", "A", "B", "C", "D"))
    step = torch.nn.functional.softplus(s["delta"].double() + s["bias"].double(), threshold=1e9)
    state = s["state"].double()
    slot = idx.clamp(min=0)
    h = state[slot] * _started(s)[:, None, None]
    y = torch.zeros(c["tokens"] + 1, c["dim"], dtype=torch.float64, device="cuda")  # one row for what has ended
    for i in range(s["longest"]):
        at = cu[:-1] + i
        live = at < cu[1:]
        row = torch.where(live, at, 0)
        d = step[row] * live[:, None]  # no step where the sequence has ended: the state stays
        h = torch.exp(d[..., None] * A) * h + (d * x[row])[..., None] * B[row][:, None, :]
        y[torch.where(live, at, c["tokens"])] = torch.matmul(h, C[row][..., None])[..., 0] + D * x[row]
    keep = (cu[1:] > cu[:-1]) & (idx >= 0)
    state[slot[keep]] = h[keep]
    return {"y": y[:-1] * _silu64(z), "state": state}


def _rms64(v):
    return v / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)


def _exact_gated(s):
    c = s["case"]
    x, z, w = (s[k].double().requires_grad_(c["train"]) for k in ("x", "z", "w"))
    split = lambda v: v.unflatten(-1, (c["groups"], -1))
    if c["norm_first"]:
        out = _rms64(split(x)).flatten(-2) * w * _silu64(z)
    else:
        out = _rms64(split(x * _silu64(z))).flatten(-2) * w
    if not c["train"]:
        return {"out": out}
    dx, dz, dw = torch.autograd.grad(out, (x, z, w), s["dout"].double())
    return {"out": out.detach(), "dx": dx, "dz": dz, "dweight": dw}


def _exact_residual(s):
    c = s["case"]
    x, h, w = (s[k].double().requires_grad_(c["train"]) for k in ("x", "h", "w"))
    if c["post"]:
        wp, scale = (s[k].double().requires_grad_(c["train"]) for k in ("wp", "scale"))
        new = h + scale * (_rms64(x) * wp)
    else:
        new = h + x
    out = _rms64(new) * w
    res = {"out": out.detach(), "h": new.detach()}
    if not c["train"]:
        return res
    of = (x, h, w) + ((wp, scale) if c["post"] else ())
    g = torch.autograd.grad((out, new), of, (s["dout"].double(), s["dh"].double()))
    return {**res, **dict(zip(("dx", "dresidual", "dweight", "dpost_weight", "dscale"), g))}


# --------------------------------------------------------------------------------- the work
def work(case):
    """Bytes (inputs once, outputs once) and operations of one pass."""
    e = 2 if case["dtype"] == "bf16" else 4
    op, dim = case["op"], case["dim"]
    if op == "conv":
        t, n, w = case["tokens"], case["seqs"], case["width"]
        reads = n if case["form"] == "step" else (n + 1) // 2
        return {"bytes": 2 * t * dim * e + (reads + n) * (w - 1) * dim * e + dim * (w + 1) * 4 + 4 * n,
                "flops": t * dim * (2 * w + 5)}
    if op == "conv_grad":
        m, w = case["batch"] * case["tokens"] * dim, case["width"]
        return {"bytes": 3 * m * e + 2 * dim * (w + 1) * 4, "flops": m * (6 * w + 10)}
    if op == "scan":
        t, n, ns = case["tokens"], case["seqs"], case["dstate"]
        reads = n if case["form"] == "step" else (n + 1) // 2
        return {"bytes": 4 * t * dim * e + 2 * t * ns * e + dim * (ns + 2) * 4 + (reads + n) * dim * ns * 4 + 4 * n,
                "flops": t * dim * (7 * ns + 15)}
    # norms: (activation type, fp32) tensors of rows x dim, and vectors; a training pass has the
    # forward's inputs once, beside the incoming gradients, and both directions' outputs
    m, train = case["rows"] * dim, case["train"]
    if op == "gated_norm":
        acts, wide, vectors = (4, 2, 2) if train else (2, 1, 1)  # z, out (dout, dz); x (dx); w (dw)
    else:
        acts, wide = (4, 4) if train else (2, 2)  # x, out (dout, dx); h in and out (dh in and out)
        vectors = (3 if case["post"] else 1) * (2 if train else 1)
    return {"bytes": m * (acts * e + wide * 4) + vectors * dim * 4, "flops": m * (40 if train else 10)}
