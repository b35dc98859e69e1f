"""How many bits the results of linear attention hold, on the GPU: against a plain 64-bit reference of the same inputs
(tests/linear_ref.py).

Error bounds, fixed beforehand, eps = 2^-24.  A bf16 result is the nearest bf16 to a value in fp32 precision: half a
step, 2^-8 of the result, and of the sum of the absolute values of its terms 2^-16 for each operand that the products take
as the sum of two bf16 parts (scores, states, weighted rows: a part leaves half a step of it, 2^-8, the second 2^-8 of
that) and the fp32 roundings on the way (`roundings`).  As a whole, its error is no more than that of a uniform rounding
of values at the lower end of their binade, 2^-8 / sqrt(3) of their norm.  fp32 results, of bf16 inputs as well: up to n
roundings in turn, of either sign and each uniform, leave sqrt(n / 3) eps of the norm, n the tokens of the longest
sequence, each a product that is added to a state, and 500 for inner axes, tiles, weights and joins; twice that for
the gradients of decays and weights, which two such sums make.  (333 tokens: 17 eps, 4500: 41 eps.)  The gradient of a head's one decay is a sum over all tokens whose parts cancel: its error is no more
than the sum of theirs, sqrt(tokens) times the norm of these (Cauchy-Schwarz), of which each of them has its share.
One part of the scores or of the states as operands of bf16 results, two where fp32 results come of them, fail."""
import pytest

from . import linear_ref as ref
from .test_linear_attention_gpu import DEV, close, cumulative, i32, make, of_ref, ops, opt, roundings

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24

SHAPES = [  # heads, q heads, k heads, dk, dv
    (2, 1, 1, 128, 64), (1, 1, 1, 64, 64), (2, 2, 1, 77, 51), (1, 1, 1, 128, 128), (1, 1, 1, 200, 40), (1, 1, 1, 48, 256),
    (1, 1, 1, 20, 5),
]


def whole(got, want, most, what, size=None):
    rel = float((got.detach().cpu().double() - want).norm() / (want.norm() if size is None else size).clamp(min=1e-30))
    assert rel <= most, (what, rel)


def check(c, cu, bf16):
    """Outputs, last states and gradients through carried states."""
    import selective_state_space_20_amd as sss
    import torch
    state = c["start"].to(DEV)
    n = len(cu) - 1
    out = sss.linear_attention_packed_fwd(*ops(c), cu_seqlens=i32(cu), state=state,
                                          has_initial=torch.ones(n, dtype=torch.bool, device=DEV), **opt(c))
    got = sss.linear_attention_packed_bwd(*ops(c), dout=c["dout"].to(DEV), cu_seqlens=i32(cu), initial_state=c["start"].to(DEV),
                                          dfinal_state=c["dfinal"].to(DEV), **opt(c))
    w = [ref.wide(c[x]) for x in ("start", "dout", "dfinal")]
    a = [x.abs() for x in w]
    want, mag = ref.gradients(*of_ref(c), cu, *w), ref.gradients(*of_ref(c, True), cu, *a, telescoped=True)
    want["out"], want["state"] = ref.attention(*of_ref(c), cu, w[0])
    mag["out"], _ = ref.attention(*of_ref(c, True), cu, a[0])
    got.update(out=out, state=state)
    assert set(got) == set(want)
    fp = roundings(c, cu) * EPS
    longest = max(b - a for a, b in zip(cu, cu[1:]))
    wide = ((500 + longest) / 3) ** 0.5 * EPS
    size = None
    if c["g"].ndim == 1:  # the norm of the tokens' parts
        every = ref.gradients(*of_ref(dict(c, g=c["g"].expand(cu[-1], -1))), cu, *w)
        size = cu[-1] ** 0.5 * every["dlog_decay"].norm()
    for name, x in want.items():
        if bf16 and name in ("out", "dq", "dk", "dv"):
            close(got[name], x, 2.0 ** -8 * x.abs() + (1 + 2.0 ** -8) * (3 * 2.0 ** -16 + fp) * mag[name], name)
            whole(got[name], x, 2.0 ** -8 / 3 ** 0.5, name)
        else:
            whole(got[name], x, wide * (2 if name in ("dlog_decay", "dbeta") else 1), name, size if name == "dlog_decay" else None)


@pytest.mark.parametrize("kind", ["ssm", "gate", "fixed"])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_bits(shape, bf16, kind):
    cu = cumulative([150, 1, 333, 64])
    check(make(11, cu[-1], 4, *shape, bf16, kind, cu), cu, bf16)


@pytest.mark.parametrize("segments", [None, 1, 3])
@pytest.mark.parametrize("bf16", [True, False])
def test_long_chain(bf16, segments, monkeypatch):
    """Sequences of thousands of tokens whose states last: decays of 1/32 to 1/4096 a token."""
    import torch
    if segments:
        monkeypatch.setenv("SSS_FORCE_SEGMENTS", str(segments))
    cu = cumulative([37, 4500])
    c = make(12, cu[-1], 2, 2, 1, 2, 24, 40, bf16, "gate", cu)
    c["g"] = torch.log1p(-torch.exp2(-5.0 - 7.0 * torch.arange(2)))
    check(c, cu, bf16)
