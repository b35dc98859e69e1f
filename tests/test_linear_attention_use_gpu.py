"""Linear attention and the layer norm as they are used: operands as they lie in a projection's rows, prompts in pieces
and then token by token, captured into graphs, on other streams, far into large memory, with boundaries of any
contents.  Results are compared with those of plain calls on copies of the same values, bit by bit where the same
kernels run on the same tiles."""
import pytest

from . import linear_ref as ref
from .test_linear_attention_gpu import DEV, close, i32, make, of_ref, ops, opt, roundings

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24


def operands(c):
    return dict(zip(("q", "k", "v", "log_decay"), ops(c)))


def grads(c, cu, **kw):
    import selective_state_space_20_amd as sss
    a = dict(operands(c), dout=c["dout"].to(DEV), cu_seqlens=i32(cu), **opt(c))
    a.update(kw)
    return sss.linear_attention_packed_bwd(a.pop("q"), a.pop("k"), a.pop("v"), a.pop("log_decay"), **a)


def fwd(c, cu, **kw):
    import selective_state_space_20_amd as sss
    a = dict(operands(c), cu_seqlens=i32(cu), **opt(c))
    a.update(kw)
    return sss.linear_attention_packed_fwd(a.pop("q"), a.pop("k"), a.pop("v"), a.pop("log_decay"), **a)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("dk, dv", [(64, 64), (24, 40), (33, 7), (128, 128)])
def test_layouts(bf16, dk, dv):
    """Slices of one row at any element, heads before tokens, one head expanded to all, strided decays."""
    import torch
    cu, h = [0, 70, 150], 4
    c = make(1, 150, 2, h, 2, 1, dk, dv, bf16, "ssm", cu)
    plain, plain_g = fwd(c, cu), grads(c, cu)
    dev = {n: c[n].to(DEV) for n in ("q", "k", "v", "g", "beta")}
    rows = torch.full((150, h * dv + 3 * dk + 5), float("nan"), dtype=c["v"].dtype, device=DEV)
    place = {"v": (1, h, dv), "q": (2 + h * dv, 2, dk), "k": (3 + h * dv + 2 * dk, 1, dk)}
    sliced = {}
    for n, (at, heads, d) in place.items():
        sliced[n] = rows[:, at:at + heads * d].unflatten(1, (heads, d))
        sliced[n].copy_(dev[n])
    wide = torch.full((150, 2 * h + 1), float("nan"), device=DEV)
    wide[:, :h], wide[:, h:2 * h] = dev["g"], dev["beta"]
    sliced.update(log_decay=wide[:, :h], beta=wide[:, h:2 * h])
    first = {n: dev[n].transpose(0, 1).contiguous().transpose(0, 1) for n in ("q", "k", "v")}
    spread = {"k": dev["k"].expand(150, h, dk), "q": dev["q"].repeat_interleave(2, 1)}
    for other in (sliced, first):
        assert torch.equal(fwd(c, cu, **other), plain)
        got = grads(c, cu, **other)
        assert all(torch.equal(got[n], plain_g[n]) for n in plain_g)
    assert torch.equal(fwd(c, cu, **spread), plain)
    got = grads(c, cu, **spread)  # of each head apart; their sums, rounded once more in bf16, those of the shared ones
    assert torch.equal(got["dv"], plain_g["dv"]) and torch.equal(got["dlog_decay"], plain_g["dlog_decay"])
    for n, r in (("dq", 2), ("dk", 4)):
        apart = got[n].float().unflatten(1, (-1, r))
        err = (apart.sum(2) - plain_g[n].float()).abs()
        assert bool((err <= (2.0 ** -8 if bf16 else 8 * EPS) * (apart.abs().sum(2) + plain_g[n].float().abs())).all()), n


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("kind", ["ssm", "gate", "fixed"])
def test_pieces_then_tokens(kind, bf16):
    """Prompts in two pieces and then token by token on the same slots: the whole sequences' outputs and states."""
    import torch
    import selective_state_space_20_amd as sss
    lens, new = [90, 3, 64, 1], 5
    n = len(lens)
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x + new)
    c = make(2, cu[-1], n, 3, 3, 1, 40, 48, bf16, kind, cu)
    c["start"] = torch.zeros_like(c["start"])
    dev, slots = operands(c), i32([2, 0, 3, 1])
    state = torch.full((5, 3, 40, 48), 9.0, device=DEV)
    got = [[] for _ in lens]
    initial = torch.zeros(n, dtype=torch.bool, device=DEV)
    cut = lambda name, parts: torch.cat([dev[name][a:b] for a, b in parts])
    beta = opt(c)["beta"]

    def part(parts, initial):
        lo = [0]
        for a, b in parts:
            lo.append(lo[-1] + b - a)
        g = dev["log_decay"] if kind == "fixed" else cut("log_decay", parts)
        o = dict(opt(c), beta=None if beta is None else torch.cat([beta[a:b] for a, b in parts]))
        return sss.linear_attention_packed_fwd(*(cut(x, parts) for x in "qkv"), g, cu_seqlens=i32(lo), state=state,
                                               state_indices=slots, has_initial=initial, **o).split([b - a for a, b in parts])

    half = [max(1, x // 2) for x in lens]
    for i, t in enumerate(part([(cu[i], cu[i] + half[i]) for i in range(n)], initial)):
        got[i].append(t)
    for i, t in enumerate(part([(cu[i] + half[i], cu[i] + lens[i]) for i in range(n)], ~initial)):
        got[i].append(t)
    for k in range(new):
        rows = [cu[i] + lens[i] + k for i in range(n)]
        g = dev["log_decay"] if kind == "fixed" else dev["log_decay"][rows]
        o = dict(opt(c), beta=None if beta is None else beta[rows])
        out = sss.linear_attention_update_slots(*(dev[x][rows] for x in "qkv"), g, state=state, state_indices=slots, **o)
        for i in range(n):
            got[i].append(out[i:i + 1])
    want, last = ref.attention(*of_ref(c), cu, ref.wide(c["start"]))
    mag, mag_last = ref.attention(*of_ref(c, True), cu, ref.wide(c["start"]))
    fp = (roundings(c, cu) + 40) * EPS
    close(torch.cat([torch.cat(t) for t in got]), want, fp * mag + (2 * 2.0 ** -8 * mag + 2.0 ** -8 * want.abs() if bf16 else 0),
          "out")
    for i, s in enumerate([2, 0, 3, 1]):
        close(state[s], last[i], ((2.0 ** -16 if bf16 else 0) + fp) * mag_last[i], "state")
    assert bool((state[4] == 9.0).all())


@pytest.mark.parametrize("bf16", [False, True])
def test_captured_calls(bf16):
    """A captured forward, step and gradients replay with other values and other lengths, and eager work between."""
    import torch
    import selective_state_space_20_amd as sss
    t, n = 300, 3
    c = make(3, t, n, 2, 1, 1, 64, 48, bf16, "ssm", [0, 100, 200, t])
    dev, o = operands(c), opt(c)
    cu, dout = i32([0, 100, 200, t]), c["dout"].to(DEV)
    start = c["start"].to(DEV)
    state = start.clone()
    norm_w = torch.rand(96, device=DEV)
    ws = torch.empty(sss.linear_attention_packed_fwd_workspace_size(t, 2, 64, 48), dtype=torch.uint8, device=DEV)

    def work():
        state.copy_(start)
        out = sss.linear_attention_packed_fwd(*dev.values(), cu_seqlens=cu, state=state, workspace=ws,
                                              has_initial=torch.ones(n, dtype=torch.bool, device=DEV), **o)
        kept = state.clone()
        one = sss.linear_attention_update_slots(*(x[:n] for x in dev.values()), state=state,
                                                **dict(o, beta=o["beta"][:n]))
        g = sss.linear_attention_packed_bwd(*dev.values(), dout=dout, cu_seqlens=cu, initial_state=start, **o)
        y, mean, rstd = sss.layer_norm_fwd(out.flatten(1), norm_w, norm_w, group_size=48, return_stats=True)
        d = sss.layer_norm_bwd(y, out.flatten(1), norm_w, mean=mean, rstd=rstd, bias=True, group_size=48)
        return {"out": out, "state": kept, "step": one, "stepped": state.clone(), **g, "y": y, "dx": d["dx"]}

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = work()
    for k, cuts in enumerate(([0, 100, 200, t], [0, 1, 1, t], [7, 130, 280, 290], [0, 0, 0, 64])):
        cu.copy_(i32(cuts))
        dev["v"].copy_(torch.randn(dev["v"].shape, generator=torch.Generator().manual_seed(k)).to(dev["v"].dtype))
        graph.replay()
        torch.cuda.synchronize()
        got = {n: x.clone() for n, x in kept.items()}
        want = work()
        torch.cuda.synchronize()
        rows = slice(cuts[0], cuts[-1])  # the forward leaves the others as they are
        for name, x in want.items():
            a, b = (got[name][rows], x[rows]) if name in ("out", "y", "dx") else (got[name], x)
            assert torch.equal(a, b), (k, name)


def test_given_stream():
    import torch
    import selective_state_space_20_amd as sss
    cu = [0, 120, 300]
    c = make(4, 300, 2, 2, 1, 2, 64, 64, True, "gate", cu)
    dev, dout = operands(c), c["dout"].to(DEV)
    x, w = torch.randn(300, 256, device=DEV), torch.randn(256, device=DEV)

    def every(**kw):
        st = torch.zeros(2, 2, 64, 64, device=DEV)
        bounds = i32(cu)
        torch.cuda.synchronize()
        o = [sss.linear_attention_packed_fwd(*dev.values(), cu_seqlens=bounds, state=st, **kw),
             sss.linear_attention_update_slots(*(t[:2] for t in dev.values()), state=st, **kw),
             *sss.linear_attention_packed_bwd(*dev.values(), dout=dout, cu_seqlens=bounds, **kw).values()]
        y, h, mean, rstd = sss.layer_norm_fwd(x, w, w, x, return_stats=True, **kw)
        o += [y, h, *sss.layer_norm_bwd(x, h, w, mean=mean, rstd=rstd, bias=True, dresidual_out=x, **kw).values()]
        torch.cuda.synchronize()
        return [*o, st]

    side = torch.cuda.Stream()
    for a, b in zip(every(), every(stream=side.cuda_stream)):
        assert torch.equal(a, b)
    with torch.cuda.stream(side):
        for a, b in zip(every(), every(stream=torch.cuda.default_stream().cuda_stream)):
            assert torch.equal(a, b)


def test_the_same_bits_every_time():
    import torch
    cu = [0, 33, 500]
    c = make(5, 500, 2, 4, 1, 2, 128, 64, True, "ssm", cu)
    runs = [[fwd(c, cu), *grads(c, cu, initial_state=c["start"].to(DEV), dfinal_state=c["dfinal"].to(DEV)).values()] for _ in range(3)]
    for other in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], other))


def test_nothing_to_do():
    import torch
    import selective_state_space_20_amd as sss
    e = lambda *s: torch.empty(*s, device=DEV)
    out = sss.linear_attention_packed_fwd(e(0, 2, 8), e(0, 2, 8), e(0, 2, 8), e(0, 2), cu_seqlens=i32([0]))
    assert out.shape == (0, 2, 8)
    df = torch.randn(3, 2, 8, 8, device=DEV)
    for tokens, cu in ((0, [0, 0, 0, 0]), (5, [2, 2, 2, 2])):
        r = lambda *s: torch.randn(*s, device=DEV)
        g = sss.linear_attention_packed_bwd(r(tokens, 2, 8), r(tokens, 2, 8), r(tokens, 2, 8), -torch.rand(2, device=DEV), D=r(2),
                                            dout=r(tokens, 2, 8), cu_seqlens=i32(cu), initial_state=r(3, 2, 8, 8),
                                            dfinal_state=df)
        assert torch.equal(g["dinitial_state"], df)
        assert all(bool((g[n] == 0).all()) for n in ("dq", "dk", "dv", "dlog_decay", "dD"))
    g = sss.linear_attention_packed_bwd(r(5, 2, 8), r(5, 2, 8), r(5, 2, 8), -torch.rand(5, 2, device=DEV), dout=r(5, 2, 8),
                                        cu_seqlens=i32([0]))
    assert all(bool((t == 0).all()) for t in g.values())


@pytest.mark.parametrize("cu", [[-5, 100], [-1, 4, 9, 100], [0, 50, -3, 100], [-2 ** 31, 2 ** 31 - 1], [70, 30, 120, -1, 100]])
@pytest.mark.parametrize("segments", [None, 4])
def test_malformed_boundaries(cu, segments, monkeypatch):
    """Nothing outside the outputs is read or written, whatever the boundaries hold."""
    import torch
    import selective_state_space_20_amd as sss
    if segments:
        monkeypatch.setenv("SSS_FORCE_SEGMENTS", str(segments))
    t, n = 100, len(cu) - 1
    c = make(6, t, n, 2, 2, 2, 32, 32, True, "gate", [0, t])
    out = torch.full((t + 4, 2, 32), 7.0, dtype=torch.bfloat16, device=DEV)
    state = torch.full((n + 2, 2, 32, 32), 7.0, device=DEV)
    fwd(c, cu, out=out[2:-2], state=state[1:-1])
    grads(c, cu, initial_state=state[1:-1].contiguous(), dfinal_state=state[1:-1].contiguous())
    torch.cuda.synchronize()
    for a in (out[:2], out[-2:], state[0], state[-1]):
        assert bool((a == 7.0).all())


def test_from_a_negative_boundary():
    import torch
    c = make(7, 100, 1, 2, 2, 2, 32, 32, True, "gate", [0, 100])
    assert torch.equal(fwd(c, [-5, 100]), fwd(c, [0, 100]))


def test_offsets_past_32_bits():
    """A cache of 17 GiB, token rows 10 GiB apart from end to end, and heads before tokens."""
    import torch
    import selective_state_space_20_amd as sss
    cu = [0, 130, 300]
    c = make(8, 300, 2, 2, 2, 2, 64, 64, True, "gate", cu)
    plain_state = torch.zeros(2, 2, 64, 64, device=DEV)
    plain = fwd(c, cu, state=plain_state)
    plain_g = grads(c, cu)
    slots = 560_000  # of 32 KiB
    state = torch.empty(slots, 2, 64, 64, device=DEV)
    far = [slots - 1, slots - 7]
    state[far] = 0
    assert torch.equal(fwd(c, cu, state=state, state_indices=i32(far)), plain)
    assert torch.equal(state[far], plain_state)
    rows = [x[:2] for x in operands(c).values()]
    a = sss.linear_attention_update_slots(*rows, state=plain_state, **opt(c))
    assert torch.equal(sss.linear_attention_update_slots(*rows, state=state, state_indices=i32(far), **opt(c)), a)
    assert torch.equal(state[far], plain_state)
    del state
    step = (1 << 24) - 512
    big = torch.empty(300 * step, dtype=torch.bfloat16, device=DEV)  # 10 GB
    other = {}
    for i, n in enumerate("qkv"):
        other[n] = big.as_strided((300, 2, 64), (step, 64, 1), 128 * i)
        other[n].copy_(c[n].to(DEV))
    assert torch.equal(fwd(c, cu, **other), plain)
    got = grads(c, cu, **other)
    assert all(torch.equal(got[n], plain_g[n]) for n in plain_g)
    del other, big
    x = torch.zeros(440_000, 2560, device=DEV)  # 4.5 GB
    x[-3:] = torch.randn(3, 2560, device=DEV)
    w = torch.randn(2560, device=DEV)
    out, mean, rstd = sss.layer_norm_fwd(x, w, return_stats=True)
    last, m3, r3 = sss.layer_norm_fwd(x[-3:].clone(), w, return_stats=True)
    assert torch.equal(out[-3:], last) and torch.equal(mean[-3:], m3)
    g = sss.layer_norm_bwd(x, x, w, mean=mean, rstd=rstd)
    g3 = sss.layer_norm_bwd(x[-3:].clone(), x[-3:].clone(), w, mean=m3, rstd=r3)
    assert torch.equal(g["dx"][-3:], g3["dx"])


@pytest.mark.parametrize("sequences", [62, 63, 64, 65, 130])
@pytest.mark.parametrize("segments", [None, 7])
def test_many_sequences(sequences, segments, monkeypatch):
    """As many boundaries and slots as a wave has lanes, fewer and more."""
    from . import test_linear_attention_gpu as base
    monkeypatch.setitem(base.LENGTHS, "many", [(5 * i) % 9 for i in range(sequences)])
    for bf16 in (False, True):
        base.check_prompts((2, 1, 1, 48, 36), bf16, segments, "many", "gate", monkeypatch)
        base.check_gradients((2, 1, 1, 48, 36), bf16, segments, "many", "gate", True, monkeypatch)
