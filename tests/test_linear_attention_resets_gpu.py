"""Linear attention on the GPU where log decays of -1e4 or less cut a sequence: nothing passes them, in outputs, states or
gradients, so that the results are those of the pieces as sequences of their own (64-bit reference,
tests/linear_ref.py), however large the values on the other side; and no gradient goes to such a decay.

Error bounds, fixed beforehand: as in test_linear_attention_gpu.py, each from the absolute values of its own piece
alone."""
import pytest

from . import linear_ref as ref
from .test_linear_attention_gpu import DEV, EPS, close, i32, make, of_ref, ops, opt, roundings

pytestmark = pytest.mark.gpu

LENS = [403, 70]
# first and last tokens, tiles' edges (64 and 32 tokens), inside a tile, two in a row, segments' edges
CUTS = [0, 32, 64, 77, 128, 200, 201, 319, 320, 321, 402, 403 + 5, 403 + 69]


@pytest.mark.parametrize("segments", [None, 1, 4, 40])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("kind", ["ssm", "gate"])
@pytest.mark.parametrize("value", [-1e4, -3e38, -float("inf")])
def test_resets(value, kind, bf16, segments, monkeypatch):
    import torch
    import selective_state_space_20_amd as sss
    if segments:
        monkeypatch.setenv("SSS_FORCE_SEGMENTS", str(segments))
    cu, t = [0, 403, 473], 473
    c = make(21, t, 2, 2, 1, 2, 40, 48, bf16, kind, cu)
    c["g"][CUTS] = value
    c["g"][150], c["g"][260] = -30.0, -200.0  # strong, but no cut
    edges = sorted(set(CUTS + cu))
    for n, at in enumerate(edges[:-1]):  # every other piece a hundred times as large
        if n % 2:
            for name in ("q", "k", "v", "dout"):
                c[name][at:edges[n + 1]] *= 100
    state = c["start"].to(DEV)
    out = sss.linear_attention_packed_fwd(*ops(c), cu_seqlens=i32(cu), state=state,
                                          has_initial=torch.ones(2, dtype=torch.bool, device=DEV), **opt(c))
    got = sss.linear_attention_packed_bwd(*ops(c), dout=c["dout"].to(DEV), cu_seqlens=i32(cu), initial_state=c["start"].to(DEV),
                                          dfinal_state=c["dfinal"].to(DEV), **opt(c))
    # the pieces as sequences of their own: the first of each sequence starts from its state, the last ends in it
    start, dfinal = (torch.zeros(len(edges) - 1, 2, 40, 48).double() for _ in range(2))
    first, last = [edges.index(x) for x in cu[:-1]], [edges.index(x) - 1 for x in cu[1:]]
    start[first], dfinal[last] = ref.wide(c["start"]), ref.wide(c["dfinal"])
    start[0] = 0  # cut off by its first token
    dout = ref.wide(c["dout"])
    want = ref.gradients(*of_ref(c), edges, start, dout, dfinal)
    mag = ref.gradients(*of_ref(c, True), edges, start.abs(), dout.abs(), dfinal.abs(), telescoped=True)
    want["out"], want_state = ref.attention(*of_ref(c), edges, start)
    mag["out"], mag_state = ref.attention(*of_ref(c, True), edges, start.abs())
    want["state"], mag["state"] = want_state[last], mag_state[last]
    want["dinitial_state"], mag["dinitial_state"] = want["dinitial_state"][first], mag["dinitial_state"][first]
    got.update(out=out, state=state)
    assert set(got) == set(want)
    fp = (roundings(c, cu) + 512) * EPS  # exponents up to 200 log2(e)
    for name, x in want.items():
        bound = fp * mag[name]
        if bf16 and name in ("out", "dq", "dk", "dv"):
            bound = bound + 2 * 2.0 ** -8 * mag[name] + 2.0 ** -8 * x.abs()
        close(got[name], x, bound, name)
    assert bool((got["dlog_decay"][CUTS] == 0).all())
    assert bool((got["dinitial_state"][0] == 0).all())


@pytest.mark.parametrize("bf16", [False, True])
def test_a_head_that_keeps_nothing(bf16):
    """One decay for each head, one of them a cut: each token alone, no gradient of it."""
    import torch
    import selective_state_space_20_amd as sss
    c = make(22, 150, 1, 2, 2, 2, 24, 24, bf16, "fixed", [0, 150])
    c["g"] = torch.tensor([-float("inf"), -0.1])
    got = sss.linear_attention_packed_bwd(*ops(c), dout=c["dout"].to(DEV), cu_seqlens=i32([0, 150]), **opt(c))
    assert float(got["dlog_decay"][0]) == 0 and bool(got["dlog_decay"].isfinite().all())
    assert float(got["dlog_decay"][1]) != 0
