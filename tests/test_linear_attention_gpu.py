"""Linear attention with a decay for each head on the GPU: packed prompts, the single-token step and
the gradients, against a plain 64-bit reference of the same inputs (tests/linear_ref.py).

Error bounds, fixed beforehand, per element, from the sum of the absolute values of the terms that it
adds up (the reference run on absolute values).  fp32 results of fp32 inputs: eps = 2^-24 of that sum
for each rounding on the way, at most those of the inner axes (dk + dv), of a tile (64), of the
tiles' chain (two per tile) and 64 for weights, exponents and joins; a decay e^d, d the sum of log
decays, has a relative error of up to |d| eps as well, but |d| e^d is below one.  bf16 results:
half a step, 2^-8, of the result, and 2^-8 of the terms for each of the two operands that are rounded
once (scores, states).  fp32 results of bf16 inputs: states are sums of two parts of 8 bits (2^-16
of the terms) in the outputs' walk, and of three (2^-24) where gradients of decays and input weights come from."""
import pytest

from . import linear_ref as ref

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24
DEV = "cuda:0"

LENGTHS = {
    "one token": [1],
    "one long": [333],
    "ragged": [3, 0, 70, 1, 1, 133, 0, 64, 129, 2],
    "all single": [1] * 33,
    "edges": [64, 65, 63, 128, 32, 31, 33],
}


def cumulative(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def make(seed, tokens, nseq, heads, qh, kh, dk, dv, bf16, kind, cu):
    """Inputs on the CPU; q, k, v in their type."""
    import torch
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    dt = torch.bfloat16 if bf16 else torch.float32
    c = {"q": r(tokens, qh, dk).to(dt), "k": r(tokens, kh, dk).to(dt), "v": r(tokens, heads, dv).to(dt),
         "beta": None, "D": None, "scale": dk ** -0.5}
    if kind == "ssm":
        step = torch.exp(torch.rand(tokens, heads, generator=gen) * 4.6 - 6.9)
        c.update(beta=step, g=-step * torch.exp(torch.rand(heads, generator=gen) * 2.77), D=r(heads), scale=1.0)
    elif kind == "gate":
        c["g"] = torch.nn.functional.logsigmoid(r(tokens, heads) * 2 + 1)
    else:
        c["g"] = torch.log1p(-torch.exp2(-1.0 - torch.arange(heads)))
    c["start"] = r(nseq, heads, dk, dv)
    c["dout"] = r(tokens, heads, dv).to(dt)
    c["dfinal"] = r(nseq, heads, dk, dv)
    return c


def ops(c, names=("q", "k", "v", "g")):
    return [c[n].to(DEV) for n in names]


def opt(c):
    dev = lambda t: None if t is None else t.to(DEV)
    return dict(beta=dev(c["beta"]), D=dev(c["D"]), scale=c["scale"])


def of_ref(c, absolute=False):
    w = [ref.wide(c[n]) for n in ("q", "k", "v", "g", "beta", "D")]
    if absolute:
        w = [x if x is None or i == 3 else x.abs() for i, x in enumerate(w)]
    return (*w, abs(c["scale"]) if absolute else c["scale"])


def roundings(c, cu):
    longest = max([b - a for a, b in zip(cu, cu[1:])] + [1])
    return c["q"].shape[2] + c["v"].shape[2] + 128 + 2 * (longest // 32 + 1)


def close(got, want, bound, what):
    import torch
    got = got.detach().cpu().double()
    bad = ~((got - want).abs() <= bound)
    assert not bool(bad.any()), (what, int(bad.sum()), float((got - want).abs().max()), float(want.abs().max()))


def i32(v):
    import torch
    return torch.tensor(v, dtype=torch.int32, device=DEV)


SHAPES = [  # heads, q heads, k heads, dk, dv
    (1, 1, 1, 16, 16), (3, 3, 3, 64, 64), (4, 1, 1, 128, 64), (2, 2, 1, 64, 128), (2, 1, 2, 128, 128), (2, 2, 2, 77, 51),
    (1, 1, 1, 256, 33), (1, 1, 1, 40, 200), (2, 2, 2, 160, 256), (1, 1, 1, 130, 120), (2, 1, 1, 1, 1),
]


@pytest.mark.parametrize("segments", [None, 1, 5])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_prompts(shape, bf16, segments, monkeypatch):
    check_prompts(shape, bf16, segments, "ragged", "gate", monkeypatch)


@pytest.mark.parametrize("segments", [None, 1, 4, 50])
@pytest.mark.parametrize("kind", ["ssm", "gate", "fixed"])
@pytest.mark.parametrize("lengths", LENGTHS)
def test_lengths(lengths, kind, segments, monkeypatch):
    for bf16 in (False, True):
        check_prompts((2, 1, 1, 48, 36), bf16, segments, lengths, kind, monkeypatch)


def check_prompts(shape, bf16, segments, lengths, kind, monkeypatch):
    import torch
    import selective_state_space_20_amd as sss
    if segments:
        monkeypatch.setenv("SSS_FORCE_SEGMENTS", str(segments))
    lens = LENGTHS[lengths]
    before, behind = 5, 3  # rows outside every sequence
    cu = [before + c for c in cumulative(lens)]
    n, tokens = len(lens), cu[-1] + behind
    heads, qh, kh, dk, dv = shape
    c = make(1, tokens, n, heads, qh, kh, dk, dv, bf16, kind, cu)
    slots = n + 2
    idx = [(3 * i + 1) % slots if slots % 3 else (i + 1) % slots for i in range(n)]
    if n > 2:
        idx[1] = -1
    initial = [i % 2 == 0 for i in range(n)]
    cache = torch.randn(slots, heads, dk, dv, generator=torch.Generator().manual_seed(7))
    start = torch.stack([cache[idx[i]] if initial[i] and idx[i] >= 0 else torch.zeros(heads, dk, dv) for i in range(n)])
    out = torch.full((tokens, heads, dv), 7.0, dtype=c["v"].dtype, device=DEV)
    state = cache.to(DEV)
    sss.linear_attention_packed_fwd(*ops(c), cu_seqlens=i32(cu), state=state, state_indices=i32(idx),
                                    has_initial=torch.tensor(initial, device=DEV), out=out, **opt(c))
    want, last = ref.attention(*of_ref(c), cu, ref.wide(start))
    mag, mag_last = ref.attention(*of_ref(c, True), cu, ref.wide(start).abs())
    fp = roundings(c, cu) * EPS
    rows = slice(cu[0], cu[-1])
    bound = fp * mag + (2 * 2.0 ** -8 * mag + 2.0 ** -8 * want.abs() if bf16 else 0)
    close(out[rows], want[rows], bound[rows], "out")
    assert bool((out[:cu[0]] == 7.0).all()) and bool((out[cu[-1]:] == 7.0).all())
    touched = set()
    for i in range(n):
        if idx[i] >= 0 and lens[i] > 0:
            close(state[idx[i]], last[i], ((2.0 ** -16 if bf16 else 0) + fp) * mag_last[i], "state")
            touched.add(idx[i])
    rest = [i for i in range(slots) if i not in touched]
    assert torch.equal(state[rest].cpu(), cache[rest])


@pytest.mark.parametrize("rows", [1, 2, 9])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_step(shape, bf16, rows):
    import torch
    import selective_state_space_20_amd as sss
    heads, qh, kh, dk, dv = shape
    for kind in ("ssm", "gate", "fixed"):
        cu = list(range(rows + 1))
        c = make(2, rows, rows, heads, qh, kh, dk, dv, bf16, kind, cu)
        idx = [(2 * i + 1) % (rows + 1) if (rows + 1) % 2 else i for i in range(rows)]
        if rows > 2:
            idx[1] = -1
        cache = torch.randn(rows + 1, heads, dk, dv, generator=torch.Generator().manual_seed(7))
        start = torch.stack([cache[i] if i >= 0 else torch.zeros(heads, dk, dv) for i in idx])
        state = cache.to(DEV)
        out = sss.linear_attention_update_slots(*ops(c), state=state, state_indices=i32(idx), **opt(c))
        want, last = ref.attention(*of_ref(c), cu, ref.wide(start))
        mag, mag_last = ref.attention(*of_ref(c, True), cu, ref.wide(start).abs())
        fp = roundings(c, cu) * EPS
        close(out, want, fp * mag + (2.0 ** -8 * want.abs() if bf16 else 0), "out")
        for i, s in enumerate(idx):
            if s >= 0:
                close(state[s], last[i], 8 * EPS * mag_last[i], "state")
        rest = [s for s in range(rows + 1) if s not in idx]
        assert torch.equal(state[rest].cpu(), cache[rest])


@pytest.mark.parametrize("segments", [None, 1, 5])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradients(shape, bf16, segments, monkeypatch):
    check_gradients(shape, bf16, segments, "ragged", "gate", True, monkeypatch)


@pytest.mark.parametrize("segments", [None, 1, 4, 50])
@pytest.mark.parametrize("kind", ["ssm", "gate", "fixed"])
@pytest.mark.parametrize("lengths", LENGTHS)
def test_gradients_of_lengths(lengths, kind, segments, monkeypatch):
    for bf16 in (False, True):
        check_gradients((2, 1, 1, 48, 36), bf16, segments, lengths, kind, lengths != "edges", monkeypatch)


def check_gradients(shape, bf16, segments, lengths, kind, carried, monkeypatch):
    import torch
    import selective_state_space_20_amd as sss
    if segments:
        monkeypatch.setenv("SSS_FORCE_SEGMENTS", str(segments))
    lens = LENGTHS[lengths]
    cu = [5 + x for x in cumulative(lens)]
    n, tokens = len(lens), cu[-1] + 3
    heads, qh, kh, dk, dv = shape
    c = make(3, tokens, n, heads, qh, kh, dk, dv, bf16, kind, cu)
    if not carried:
        c["start"], c["dfinal"] = (torch.zeros_like(c[x]) for x in ("start", "dfinal"))
    got = sss.linear_attention_packed_bwd(*ops(c), dout=c["dout"].to(DEV), cu_seqlens=i32(cu),
                                          initial_state=c["start"].to(DEV) if carried else None,
                                          dfinal_state=c["dfinal"].to(DEV) if carried else None, **opt(c))
    w = [ref.wide(c[x]) for x in ("start", "dout", "dfinal")]
    want = ref.gradients(*of_ref(c), cu, *w)
    mag = ref.gradients(*of_ref(c, True), cu, *(x.abs() for x in w), telescoped=True)
    if not carried:
        want.pop("dinitial_state")
    assert set(got) == set(want)
    fp = roundings(c, cu) * EPS
    for name, x in want.items():
        bound = fp * mag[name]
        if bf16 and name in ("dq", "dk", "dv"):
            bound = bound + 2 * 2.0 ** -8 * mag[name] + 2.0 ** -8 * x.abs()
        close(got[name], x, bound, name)
        # and as a whole, near what roundings of either sign leave
        rel = float((got[name].cpu().double() - x).norm() / x.norm().clamp(min=1e-30))
        assert rel <= (5e-3 if bf16 and name in ("dq", "dk", "dv") else 1e-5), (name, rel)


# ------------------------------------------------------------------------------ what is not finite
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dv", [4, 40])
def test_later_tokens_do_not_reach_earlier_ones(value, bf16, dv):
    """A value that is not finite, in q, k, v, beta or the decays of one token, changes nothing before it (but the
    order of the sums in its tile: both results are within the bound)."""
    import torch
    import selective_state_space_20_amd as sss
    cu, at = [0, 100, 170], 41
    c = make(4, 170, 2, 2, 2, 2, 24, dv, bf16, "ssm", cu)
    clean = sss.linear_attention_packed_fwd(*ops(c), cu_seqlens=i32(cu), **opt(c))
    mag, _ = ref.attention(*of_ref(c, True), cu, torch.zeros(2, 2, 24, dv).double())
    slack = 2 * roundings(c, cu) * EPS * mag + (2.0 ** -7 * mag if bf16 else 0)
    for name in ("q", "k", "v", "beta", "g"):
        d = dict(c)
        d[name] = c[name].clone()
        d[name][at, 1] = value
        out = sss.linear_attention_packed_fwd(*ops(d), cu_seqlens=i32(cu), **opt(d))
        same = torch.ones_like(out, dtype=torch.bool)
        same[at:100, 1] = False  # the token's head, from it on to the end of its sequence
        close(out[:at], clean[:at].cpu().double(), slack[:at], name)
        same[:at, 1] = False
        assert torch.equal(out[same], clean[same]), name
        if name == "q":
            assert torch.equal(out[at + 1:], clean[at + 1:])
        if name == "g" and value < 0:  # everything forgotten: as if the sequence began there
            assert bool(out.isfinite().all())
        elif not (name == "g" and value > 0):
            assert not bool(out[at, 1].isfinite().any()), name
        if name in ("v", "k") or value != value and name != "q":
            assert not bool(out[at:100, 1].isfinite().any()), name


@pytest.mark.parametrize("bf16", [False, True])
def test_gradients_apart(bf16):
    """Sequences have nothing to do with each other, nor do heads; and a token's value that is not finite reaches, in
    dv, only the tokens that it adds to."""
    import torch
    import selective_state_space_20_amd as sss
    cu, at = [0, 60, 130], 80
    c = make(5, 130, 2, 2, 2, 2, 24, 40, bf16, "gate", cu)
    grads = lambda x: sss.linear_attention_packed_bwd(*ops(x), dout=x["dout"].to(DEV), cu_seqlens=i32(cu), **opt(x))
    clean = grads(c)
    zero = torch.zeros(2, 2, 24, 40).double()
    mag = ref.gradients(*of_ref(c, True), cu, zero, ref.wide(c["dout"]).abs(), zero)
    near = lambda got, n, rows: close(got[n][rows], clean[n][rows].cpu().double(), (
        2 * roundings(c, cu) * EPS * mag[n] + (2.0 ** -7 * mag[n] if bf16 else 0))[rows], n)
    for name in ("q", "k", "v", "dout"):
        d = dict(c)
        d[name] = c[name].clone()
        d[name][at, 1] = float("nan")
        got = grads(d)
        for n, t in got.items():
            assert torch.equal(t[:60], clean[n][:60]) and torch.equal(t[:, 0], clean[n][:, 0]), (name, n)
        if name in ("q", "dout"):  # later tokens' dk and dv have no part of it
            near(got, "dv", slice(at + 1, None))
            near(got, "dk", slice(at + 1, None))
        else:  # nor have earlier tokens' dq
            near(got, "dq", slice(None, at))


def test_strong_decays_and_forgetting():
    """Log decays of zero, far below zero and -inf, beside each other, against the definition."""
    import torch
    import selective_state_space_20_amd as sss
    for bf16 in (False, True):
        cu = [0, 150]
        c = make(6, 150, 1, 2, 1, 1, 32, 32, bf16, "gate", cu)
        c["g"][::7], c["g"][3::11], c["g"][5::29], c["g"][20:40] = 0.0, -30.0, -float("inf"), -1e-4
        c["g"][77] = -3e38
        out = sss.linear_attention_packed_fwd(*ops(c), cu_seqlens=i32(cu), **opt(c))
        zero = torch.zeros(1, 2, 32, 32).double()
        want, _ = ref.attention(*of_ref(c), cu, zero)
        mag, _ = ref.attention(*of_ref(c, True), cu, zero)
        fp = (roundings(c, cu) + 64) * EPS  # exponents up to 30 log2(e) beside the decay's own rounding
        close(out, want, fp * mag + (2 * 2.0 ** -8 * mag + 2.0 ** -8 * want.abs() if bf16 else 0), "out")
