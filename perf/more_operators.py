"""The cases on which the operators of linear attention with a decay for each head, and the layer
norms, are measured: attention over packed prompts and single tokens with its states in cache
slots, its gradients, and the layer norm over rows or groups of channels, alone or after the
residual addition, forward and gradients.

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
CHUNK = 64  # of the plain form


# ------------------------------------------------------------------------------ the cases
# kind: "ssm"   the state-space form: one query and key (C and B) for all heads or groups of them,
#               decay dt A, input weight dt, skip D
#       "gate"  linear attention with a decay for each token and head (a forget gate)
#       "fixed" linear attention with one decay for each head
def listed():
    return [
        # one generated token for each of three chats, a small fp32 layer: all latency
        dict(name="attention step 3", op="attention", form="step", tokens=3, seqs=3, heads=16, qk_heads=16, dk=64, dv=64,
             kind="gate", dtype="fp32"),
        # a full decode batch of a d_inner 5120 layer: 80 heads of 64, 128 states; bound by its states
        dict(name="attention step 256", op="attention", form="step", tokens=256, seqs=256, heads=80, qk_heads=1, dk=128,
             dv=64, kind="ssm", dtype="bf16"),
        # a few short prompts through a layer of odd sizes, in fp32: nothing divides evenly
        dict(name="attention prompts 301", op="attention", form="prompts", tokens=301, seqs=5, heads=5, qk_heads=5, dk=48,
             dv=77, kind="gate", dtype="fp32"),
        # a ragged prefill batch of the d_inner 5120 layer, half of the prompts continuing a cached state
        dict(name="attention prompts 16384", op="attention", form="prompts", tokens=16384, seqs=24, heads=80, qk_heads=1,
             dk=128, dv=64, kind="ssm", dtype="bf16"),
        # few long documents: parallelism has to come from the time axis; one decay for each head
        dict(name="attention prompts 32768", op="attention", form="prompts", tokens=32768, seqs=3, heads=16, qk_heads=16,
             dk=128, dv=128, kind="fixed", dtype="bf16"),
        # the gradients of a training step of a model of width 2048, two packed documents
        dict(name="attention gradients 8192", op="attention_grad", tokens=8192, seqs=2, heads=16, qk_heads=16, dk=128,
             dv=128, kind="gate", carried=False, dtype="bf16"),
        # the same for a small odd layer in fp32, keys shared by three heads each, through carried states
        dict(name="attention gradients 1001", op="attention_grad", tokens=1001, seqs=3, heads=6, qk_heads=2, dk=64, dv=50,
             kind="ssm", carried=True, dtype="fp32"),
        # the norm before a block for a decode batch of an odd size, residual added
        dict(name="layer norm 37", op="layer_norm", train=False, rows=37, dim=2560, groups=1, residual=True,
             dtype="bf16"),
        # the heads' norm of a prefill batch: 80 groups of 64 channels
        dict(name="layer norm of heads 16384", op="layer_norm", train=False, rows=16384, dim=5120, groups=80, residual=False,
             dtype="bf16"),
        # the norm before a block in a training step, forward and gradients, fp32 residual stream
        dict(name="layer norm training 16384", op="layer_norm", train=True, rows=16384, dim=2560, groups=1, residual=True,
             dtype="bf16"),
        # a small fp32 layer of odd width, forward and gradients
        dict(name="layer norm training 1003", op="layer_norm", train=True, rows=1003, dim=777, groups=1, residual=False,
             dtype="fp32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: sizes over the listed ranges, half of them with no even divisor."""
    op = rng.choice(["step", "prompts", "prompts", "gradients", "gradients", "layer_norm", "layer_norm"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "layer_norm":
        groups = rng.choice([1, 1, 1, 8, 40])
        dim = groups * (_log_int(rng, 64, 8192) if groups == 1 else _log_int(rng, 32, 160))
        return dict(op="layer_norm", train=rng.random() < 0.6, rows=_log_int(rng, 1, min(32768, 45_000_000 // dim)), dim=dim,
                    groups=groups, residual=rng.random() < 0.5, dtype=dtype)
    kind = rng.choice(["ssm", "gate", "fixed"])
    heads = _log_int(rng, 2, 80)
    qk = rng.choice([h for h in range(1, heads + 1) if heads % h == 0]) if kind == "ssm" else heads
    dk, dv = (rng.choice([64, 128]) if rng.random() < 0.5 else _log_int(rng, 16, 160) for _ in range(2))
    c = dict(heads=heads, qk_heads=qk, dk=dk, dv=dv, kind=kind, dtype=dtype)
    most = 8_000_000_000 // (heads * dk * dv) // (2 if dtype == "fp32" else 1)  # tokens
    if op == "step":
        n = _log_int(rng, 1, max(1, min(512, most // 128)))
        return dict(op="attention", form="step", tokens=n, seqs=n, **c)
    if op == "prompts":
        t = _log_int(rng, 16, min(32768, most))
        return dict(op="attention", form="prompts", tokens=t, seqs=_log_int(rng, 1, max(1, min(t // 16, 256))), **c)
    t = _log_int(rng, 16, min(16384, most // 4))
    return dict(op="attention_grad", tokens=t, seqs=_log_int(rng, 1, max(1, min(t // 16, 16))), carried=rng.random() < 0.5, **c)


# ------------------------------------------------------------------------------ the inputs
def _randn(gen, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, device="cuda", generator=gen) * scale).to(dtype)


def _packing(case, s, seed):
    """Where the packed sequences start, the cache slot of each (the last of a padded decode
    batch has none), and which of them continue what their slot holds."""
    rng = np.random.default_rng(seed)
    n, t = case["seqs"], case["tokens"]
    if case.get("form") == "step":
        cu = np.arange(n + 1)
    else:  # ragged, empty ones among them
        cu = np.concatenate([[0], np.sort(rng.integers(0, t + 1, n - 1)), [t]])
    slots = n + 3
    idx = rng.permutation(slots)[:n].astype(np.int32)
    if n >= 8:
        idx[-1] = -1
    dev = lambda a: torch.from_numpy(a).to("cuda")
    s.update(cu=dev(cu.astype(np.int32)), lens=np.diff(cu), idx=dev(idx), slots=slots, initial=dev(np.arange(n) % 2 == 0),
             kept=dev(np.flatnonzero((np.diff(cu) > 0) & (idx >= 0))))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "layer_norm":
        r, dim = case["rows"], case["dim"]
        s.update(x=_randn(gen, r, dim, dtype=dt) + 0.5, w=1.0 + _randn(gen, dim, scale=0.1), b=_randn(gen, dim, scale=0.1))
        s["x"] = s["x"].to(dt)
        if case["residual"]:
            s["h"] = _randn(gen, r, dim, scale=2.0)
        if case["train"]:
            s["dout"] = _randn(gen, r, dim, dtype=dt)
            if case["residual"]:
                s["dh"] = _randn(gen, r, dim)
        return s
    _packing(case, s, seed)
    t, h, g, dk, dv = (case[k] for k in ("tokens", "heads", "qk_heads", "dk", "dv"))
    # value, key and query side by side in a projection's rows
    rows = _randn(gen, t, h * dv + 2 * g * dk, dtype=dt)
    s.update(v=rows[:, :h * dv].unflatten(1, (h, dv)), k=rows[:, h * dv:h * dv + g * dk].unflatten(1, (g, dk)),
             q=rows[:, h * dv + g * dk:].unflatten(1, (g, dk)), scale=dk ** -0.5, beta=None, D=None)
    if case["kind"] == "ssm":
        # steps between about 1e-3 and 1e-1, decay rates between 1 and 16
        step = torch.exp(torch.rand(t, h, device="cuda", generator=gen) * math.log(100.0) + math.log(1e-3))
        s.update(beta=step, g=step * -torch.exp(torch.rand(h, device="cuda", generator=gen) * math.log(16.0)), scale=1.0,
                 D=_randn(gen, h))
    elif case["kind"] == "gate":
        s["g"] = torch.nn.functional.logsigmoid(_randn(gen, t, h) + 3.0)
    else:
        s["g"] = torch.log1p(-torch.exp2(-5.0 - 7.0 * torch.arange(h, device="cuda") / h))
    if case["op"] == "attention":
        s["state"] = _randn(gen, s["slots"], h, dk, dv)
    else:
        s["dout"] = _randn(gen, t, h, dv, dtype=dt)
        if case["carried"]:
            s.update(state=_randn(gen, case["seqs"], h, dk, dv), dstate=_randn(gen, case["seqs"], h, dk, dv, scale=0.1))
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        return {"attention": _own_attention, "attention_grad": _own_attention_grad, "layer_norm": _own_norm}[op](s)
    return {"attention": _plain_attention, "attention_grad": _plain_attention_grad, "layer_norm": _plain_norm}[op](s)


# ------------------------------------------------------------------- the library's kernels
def _own_attention(s):
    import selective_state_space_20_amd as sss
    opt = dict(beta=s["beta"], D=s["D"], scale=s["scale"], state=s["state"], state_indices=s["idx"])
    if s["case"]["form"] == "step":
        out = sss.linear_attention_update_slots(s["q"], s["k"], s["v"], s["g"], **opt)
    else:
        out = sss.linear_attention_packed_fwd(s["q"], s["k"], s["v"], s["g"], cu_seqlens=s["cu"], has_initial=s["initial"],
                                              **opt)
    return {"out": out, "state": s["state"]}


def _own_attention_grad(s):
    import selective_state_space_20_amd as sss
    return sss.linear_attention_packed_bwd(s["q"], s["k"], s["v"], s["g"], dout=s["dout"], cu_seqlens=s["cu"], beta=s["beta"],
                                           D=s["D"], scale=s["scale"], initial_state=s.get("state"),
                                           dfinal_state=s.get("dstate"))


def _own_norm(s):
    import selective_state_space_20_amd as sss
    c = s["case"]
    group = c["dim"] // c["groups"]
    got = sss.layer_norm_fwd(s["x"], s["w"], s["b"], s.get("h"), group_size=group, eps=EPS, return_stats=c["train"])
    if not c["train"]:
        return {"out": got[0], "h": got[1]} if c["residual"] else {"out": got}
    out, h, mean, rstd = got if c["residual"] else (got[0], None, *got[1:])
    grads = sss.layer_norm_bwd(s["dout"], s["x"] if h is None else h, s["w"], mean=mean, rstd=rstd, bias=True,
                               dresidual_out=s.get("dh"), group_size=group)
    return {"out": out, **({} if h is None else {"h": h}), **grads}


# -------------------------------------------------------------------------- the plain forms
def _cut(s):
    """The packed tokens in chunks of one sequence each: the token of each place (the one behind the
    last where there is none), each chunk's sequence, and of each sequence its first chunk."""
    lens = s["lens"]
    n = -(-lens // CHUNK)
    seq = np.repeat(np.arange(len(lens)), n)
    first = np.cumsum(n) - n
    start = (np.cumsum(lens) - lens)[seq] + (np.arange(len(seq)) - first[seq]) * CHUNK
    at = start[:, None] + np.arange(CHUNK)
    at = np.where(at < np.cumsum(lens)[seq][:, None], at, s["case"]["tokens"])
    dev = lambda a: torch.from_numpy(a).to("cuda")
    return dev(at), dev(seq)


def _chunked(q, k, v, g, beta, D, scale, start, at, seq, wide):
    """Attention in chunks: each by its own tokens and the state that the chunks before leave.
    q, k (tokens, qk heads, dk), v (tokens, heads, dv), g (tokens, heads) in 64 bits, start (sequences,
    heads, dk, dv); sums of decays in 64 bits, all else in the inputs' type.  Returns the outputs and the last states."""
    t, h = v.shape[0], v.shape[1]
    rep = h // q.shape[1]
    place = lambda x: torch.cat([x, x.new_zeros(1, *x.shape[1:])])[at].transpose(1, 2)  # (chunks, heads, CHUNK, ..)
    qc, kc, vc, gc = place(q), place(k), place(v), place(g)
    run_g = gc.cumsum(-1)
    total = run_g[..., -1]  # (chunks, heads)
    causal = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device="cuda").tril()
    decay = torch.exp((run_g[..., :, None] - run_g[..., None, :]).masked_fill(~causal, -math.inf)).to(wide)
    weight = torch.exp(total[..., None] - run_g).to(wide)
    if beta is not None:
        bc = place(beta)
        decay = decay * bc[..., None, :]
        weight = weight * bc
    scores = (qc @ kc.transpose(-1, -2)).repeat_interleave(rep, 1) * decay
    o = scores @ vc
    kw = kc.repeat_interleave(rep, 1)
    adds = kw.transpose(-1, -2) @ (weight[..., None] * vc)  # (chunks, heads, dk, dv): each chunk's part of the state
    # states between chunks, each a sum over the sequence's chunks before it and its first state
    upto = torch.cat([total.new_zeros(1, h), total.cumsum(0)])  # (chunks + 1, heads)
    same = (seq[:, None] == seq) & torch.ones(len(seq), len(seq), dtype=torch.bool, device="cuda").tril(-1)
    mix = torch.exp((upto[:-1, None] - upto[None, 1:]).masked_fill(~same[..., None], -math.inf)).to(wide)
    enter = mix.permute(2, 0, 1) @ adds.flatten(2).transpose(0, 1)  # (heads, chunks, dk dv)
    where = torch.arange(len(seq), device="cuda")
    seqs = torch.arange(start.shape[0], device="cuda")
    first = torch.searchsorted(seq, seqs)  # of each sequence
    enter = enter.transpose(0, 1).reshape(adds.shape) + (
        torch.exp(upto[:-1] - upto[first[seq]]).to(wide)[..., None, None] * start[seq])
    o = o + torch.exp(run_g).to(wide)[..., None] * (qc.repeat_interleave(rep, 1) @ enter)
    last = torch.exp(total).to(wide)[..., None, None] * enter + adds
    ends = torch.searchsorted(seq, seqs, right=True) - 1
    final = torch.where((ends >= first)[:, None, None, None], last[ends.clamp(min=0)], start)
    inside = at < t
    back = torch.empty(t, dtype=torch.long, device="cuda")
    back[at[inside]] = (where[:, None] * CHUNK + torch.arange(CHUNK, device="cuda"))[inside]
    o = o.transpose(1, 2).flatten(0, 1)[back] * scale
    return (o if D is None else o + D[:, None] * v), final


def _plain_attention(s):
    c = s["case"]
    idx, kept = s["idx"].long(), s["kept"]
    slot = idx.clamp(min=0)
    q, k, v = (s[n].float() for n in "qkv")
    if c["form"] == "step":
        rep = c["heads"] // c["qk_heads"]
        past = s["state"][slot] * (idx >= 0)[:, None, None, None]
        key = k.repeat_interleave(rep, 1)
        if s["beta"] is not None:
            key = key * s["beta"][..., None]
        now = torch.exp(s["g"]).expand(c["tokens"], -1)[..., None, None] * past + key[..., None] * v[:, :, None]
        o = (q.repeat_interleave(rep, 1)[..., None] * now).sum(2) * s["scale"]
        if s["D"] is not None:
            o = o + s["D"][:, None] * v
    else:
        past = s["state"][slot] * ((idx >= 0) & s["initial"])[:, None, None, None]
        g = s["g"].double().expand(c["tokens"], -1)
        o, now = _chunked(q, k, v, g, s["beta"], s["D"], s["scale"], past, *_cut(s), torch.float32)
    s["state"][slot[kept]] = now[kept]
    return {"out": o.to(s["v"].dtype), "state": s["state"]}


def _plain_attention_grad(s):
    # the decays' gradients are long sums of products that cancel: in 64 bits
    c = s["case"]
    wide = lambda x: None if x is None else x.double().requires_grad_()
    q, k, v, g, beta, D = (wide(s[n]) for n in ("q", "k", "v", "g", "beta", "D"))
    start = wide(s["state"]) if c["carried"] else torch.zeros(c["seqs"], c["heads"], c["dk"], c["dv"], device="cuda",
                                                             dtype=torch.float64)
    o, final = _chunked(q, k, v, g.expand(c["tokens"], -1), beta, D, s["scale"], start, *_cut(s), torch.float64)
    of = {"dq": q, "dk": k, "dv": v, "dlog_decay": g, "dbeta": beta, "dD": D,
          "dinitial_state": start if c["carried"] else None}
    of = {n: x for n, x in of.items() if x is not None}
    up = [s["dout"].double()] + ([s["dstate"].double()] if c["carried"] else [])
    grads = torch.autograd.grad([o, final][:len(up)], list(of.values()), up)
    return {n: d.to(s["v"].dtype if n in ("dq", "dk", "dv") else torch.float32) for n, d in zip(of, grads)}


def _plain_norm(s):
    c = s["case"]
    groups = lambda x: x.reshape(c["rows"], c["groups"], -1)
    h = s["x"].float() + s["h"] if c["residual"] else s["x"].float()
    dev = groups(h) - groups(h).mean(-1, keepdim=True)
    rstd = torch.rsqrt(dev.square().mean(-1, keepdim=True) + EPS)
    hat = dev * rstd
    dt = s["x"].dtype
    res = {"out": (hat.reshape(h.shape) * s["w"] + s["b"]).to(dt)}
    if c["residual"]:
        res["h"] = h
    if not c["train"]:
        return res
    dout = s["dout"].float()
    d = groups(dout * s["w"])
    dh = (rstd * (d - d.mean(-1, keepdim=True) - hat * (d * hat).mean(-1, keepdim=True))).reshape(h.shape)
    if c["residual"]:
        dh = dh + s["dh"]
        res["dresidual"] = dh
    return {**res, "dx": dh.to(dt), "dweight": (dout * hat.reshape(h.shape)).sum(0), "dbias": dout.sum(0)}


# ------------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"attention": _exact_attention, "attention_grad": _exact_attention_grad, "layer_norm": _exact_norm}[case["op"]](s)


def _by_length(s):
    """The sequences, longest first, and how many of them have a token at each position."""
    order = np.argsort(-s["lens"], kind="stable")
    lens = s["lens"][order]
    start = (np.cumsum(s["lens"]) - s["lens"])[order]
    live = (lens[:, None] > np.arange(lens[0] if len(lens) else 0)).sum(0)
    return order, torch.from_numpy(start).to("cuda"), live


def _operands64(s):
    c = s["case"]
    rep = c["heads"] // c["qk_heads"]
    q, k = (s[n].double().repeat_interleave(rep, 1) for n in "qk")
    one = torch.ones(c["tokens"], c["heads"], device="cuda", dtype=torch.float64)
    return (q * s["scale"], k, s["v"].double(), torch.exp(s["g"].double()) * one, one if s["beta"] is None else s["beta"].double(),
            torch.zeros(c["heads"], device="cuda").double() if s["D"] is None else s["D"].double())


def _exact_attention(s):
    c = s["case"]
    q, k, v, a, beta, D = _operands64(s)
    order, start, live = _by_length(s)
    idx = s["idx"].long()
    use = (idx >= 0) & (s["initial"] if c["form"] == "prompts" else True)
    S = (s["state"][idx.clamp(min=0)].double() * use[:, None, None, None])[order]
    o = torch.zeros_like(v)
    for t, n in enumerate(live):
        at = start[:n] + t
        S[:n] = a[at][..., None, None] * S[:n] + (beta[at][..., None] * k[at])[..., None] * v[at][:, :, None]
        o[at] = (q[at][:, :, None] @ S[:n])[:, :, 0]
    state = s["state"].double()
    final = torch.empty_like(S)
    final[order] = S
    state[idx[s["kept"]]] = final[s["kept"]]
    return {"out": o + D[:, None] * v, "state": state}


def _exact_attention_grad(s):
    c = s["case"]
    q, k, v, a, beta, D = _operands64(s)
    do = s["dout"].double()
    order, start, live = _by_length(s)
    zero = torch.zeros(c["seqs"], c["heads"], c["dk"], c["dv"], device="cuda", dtype=torch.float64)
    S = s["state"].double()[order] if c["carried"] else zero.clone()
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), D[:, None] * do
    db, dg = torch.zeros_like(a), torch.zeros_like(a)
    for t, n in enumerate(live):
        at = start[:n] + t
        S[:n] = a[at][..., None, None] * S[:n] + (beta[at][..., None] * k[at])[..., None] * v[at][:, :, None]
        dq[at] = (S[:n] @ do[at][..., None])[..., 0]
    # the adjoint R of the state; <R_t, a_t S_(t-1)> = q_t dq_t - beta_t dbeta_t + the next token's
    R = s["dstate"].double()[order] if c["carried"] else zero
    G = (R * S).sum((-1, -2))
    for t in range(len(live) - 1, -1, -1):
        n = live[t]
        at = start[:n] + t
        R[:n] += q[at][..., None] * do[at][:, :, None]
        Rv = (R[:n] @ v[at][..., None])[..., 0]
        dk[at] = beta[at][..., None] * Rv
        dv[at] += beta[at][..., None] * (k[at][:, :, None] @ R[:n])[:, :, 0]
        db[at] = (k[at] * Rv).sum(-1)
        G[:n] += (q[at] * dq[at]).sum(-1) - beta[at] * db[at]
        dg[at] = G[:n]
        R[:n] *= a[at][..., None, None]
    group = lambda x: x.unflatten(1, (c["qk_heads"], -1)).sum(2)
    res = {"dq": group(dq) * s["scale"], "dk": group(dk), "dv": dv, "dlog_decay": dg.sum(0) if s["g"].ndim == 1 else dg}
    if s["beta"] is not None:
        res["dbeta"] = db
    if s["D"] is not None:
        res["dD"] = (do * v).sum((0, 2))
    if c["carried"]:
        res["dinitial_state"] = torch.empty_like(R)
        res["dinitial_state"][order] = R
    return res


def _exact_norm(s):
    c = s["case"]
    x, w, b = (s[n].double().requires_grad_(c["train"]) for n in ("x", "w", "b"))
    h = x + s["h"].double() if c["residual"] else x
    if c["train"]:
        h.retain_grad()
    u = h.reshape(c["rows"], c["groups"], -1)
    hat = (u - u.mean(-1, keepdim=True)) / torch.sqrt(u.var(-1, unbiased=False, keepdim=True) + EPS)
    out = hat.reshape(h.shape) * w + b
    res = {"out": out.detach()}
    if c["residual"]:
        res["h"] = h.detach()
    if not c["train"]:
        return res
    roots, up = [out], [s["dout"].double()]
    if c["residual"]:
        roots, up = [out, h], up + [s["dh"].double()]
    dx, dw, db = torch.autograd.grad(roots, (x, w, b), up)
    return {**res, "dx": dx, "dweight": dw, "dbias": db, **({"dresidual": dx} if c["residual"] else {})}


# --------------------------------------------------------------------------------- the work
def work(case):
    """Bytes (inputs once, outputs once) and operations of one pass."""
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "layer_norm":
        m, train, dim = case["rows"] * case["dim"], case["train"], case["dim"]
        acts = 4 if train else 2                                     # x, out, dout, dx
        wide = (4 if train else 2) if case["residual"] else 0        # the stream in and out, its gradient in and out
        return {"bytes": m * (acts * e + wide * 4) + (4 if train else 2) * dim * 4, "flops": m * (25 if train else 10)}
    t, n, h, g, dk, dv = (case[k] for k in ("tokens", "seqs", "heads", "qk_heads", "dk", "dv"))
    decays = h if case["kind"] == "fixed" else t * h * (2 if case["kind"] == "ssm" else 1)
    if case["op"] == "attention":
        reads = n if case["form"] == "step" else (n + 1) // 2
        return {"bytes": t * (2 * g * dk + 2 * h * dv) * e + decays * 4 + (reads + n) * h * dk * dv * 4,
                "flops": 4 * t * h * dk * dv}
    return {"bytes": t * (4 * g * dk + 3 * h * dv) * e + 2 * decays * 4 + (3 * n * h * dk * dv * 4 if case["carried"] else 0),
            "flops": 10 * t * h * dk * dv}
