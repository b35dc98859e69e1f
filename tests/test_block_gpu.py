"""The packed convolution and scan, their single-token steps and the convolution's gradients on
the GPU, against plain 64-bit references of the same inputs (tests/block_ref.py).

Error bounds, fixed beforehand.  Convolution, per element: the taps add W + 1 terms in fp32
(eps = 2^-24 of the sum of their absolute values for each), silu has a slope below 1.1 and adds
an exp, an add, a reciprocal and a multiply, each within 2 ulp and the exponent's own rounding
(|v| eps): 2 (W + 6) eps of the terms, plus half a bf16 ulp (at most 2^-8) of the result where it is
rounded to bf16.  Gradients: the same per term, and eps times sqrt-free linear growth for the sums over
batch and time, which are formed in pieces of at most a few hundred terms: 600 eps of the sum of
absolute terms.  Scan: the library's rule, 1e-4 of the largest value for fp32 inputs and 2e-3 for
bf16 ones (whose values the reference shares, so that fp32's holds as well: 1e-4 is used), plus
2^-8 of each value where y is bf16."""
import numpy as np
import pytest

from . import block_ref as ref
from .gpu_util import to_dev

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24


def dev_of(a, dtype=None):
    return to_dev(a, "cuda:0")


def host(t):
    import torch
    return t.to(torch.float32).cpu().numpy().astype(np.float64)


def strided(a):
    """The device tensor of a, as the first half of rows twice as wide (NaN in the rest)."""
    import torch
    t = dev_of(a)
    wide = torch.full((*t.shape[:-1], 2 * t.shape[-1] + 3), float("nan"), dtype=t.dtype, device=t.device)
    wide[..., 1:1 + t.shape[-1]] = t
    return wide[..., 1:1 + t.shape[-1]]


def close(got, want, bound, what):
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (what, int(bad.sum()), float(np.nanmax(np.abs(got - want) - bound)))


def rand(rng, shape, bf16=False, scale=1.0):
    a = (rng.standard_normal(shape) * scale).astype(np.float32)
    return ref.bf16_bits(a) if bf16 else a


LENGTHS = {
    "one token": [1],
    "one long": [257],
    "ragged": [3, 0, 70, 1, 1, 33, 0, 0, 129, 2],
    "all single": [1] * 70,
    "many empty": [0] * 130 + [5] + [0] * 70 + [40],
    "block edges": [32, 32, 64, 31, 33, 1, 96],
}


def packing(lens, slots_extra=3, seed=0):
    rng = np.random.default_rng(seed)
    n = len(lens)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    idx = rng.permutation(n + slots_extra)[:n].astype(np.int32)
    if n > 2:
        idx[1] = -1
        idx[-1] = n + slots_extra  # out of range: no slot either
    initial = rng.integers(0, 2, n).astype(np.uint8)
    return cu, idx, initial, n + slots_extra


@pytest.fixture
def chunks(monkeypatch, request):
    if getattr(request, "param", None):
        monkeypatch.setenv("SSS_FORCE_SEGMENTS", str(request.param))
    return getattr(request, "param", None)


# ------------------------------------------------------------------------- convolution
@pytest.mark.parametrize("chunks", [None, 5, 40], indirect=True)
@pytest.mark.parametrize("lens", list(LENGTHS))
@pytest.mark.parametrize("dim,width,bf16", [(5, 4, True), (64, 4, True), (257, 4, True), (1030, 3, True), (3, 2, True),
                                            (130, 8, True), (65, 4, False), (1, 3, False), (300, 1, True),
                                            (514, 5, False)])
def test_packed_conv(lens, dim, width, bf16, chunks):
    import torch
    import selective_state_space_20_amd as sss
    cu, idx, initial, slots = packing(LENGTHS[lens])
    t = int(cu[-1])
    rng = np.random.default_rng(dim * width)
    x, w, b = rand(rng, (t, dim), bf16), rand(rng, (dim, width), scale=0.5), rand(rng, (dim,))
    state = rand(rng, (slots, width - 1, dim), bf16)
    used = {int(i) for s, i in enumerate(idx) if 0 <= i < slots and initial[s]}
    for s in range(slots):  # a slot that nothing continues may hold anything
        if s not in used and state.size:
            state[s] = 0x7FC0 if bf16 else np.nan
    want, want_state, mag = ref.packed_conv(x, w, b, cu, state, idx, initial, True)
    st = dev_of(state)
    before = st.clone()
    out = sss.causal_conv1d_packed_fwd(strided(x), dev_of(w), dev_of(b), cu_seqlens=dev_of(cu), conv_state=st,
                                       state_indices=dev_of(idx), has_initial=dev_of(initial), silu=True)
    got = host(out)
    close(got, want, 2 * (width + 6) * EPS * mag + (2.0 ** -8 * np.abs(want) if bf16 else 0) + 1e-37, "out")
    # copies of inputs: exact, and every slot that no sequence with tokens has is untouched
    np.testing.assert_array_equal(host(st), want_state)
    touched = {int(i) for s, i in enumerate(idx) if 0 <= i < slots and cu[s + 1] > cu[s]}
    for s in set(range(slots)) - touched:
        assert torch.equal(st[s].view(torch.int16 if bf16 else torch.int32),
                           before[s].view(torch.int16 if bf16 else torch.int32))


@pytest.mark.parametrize("dim,width,bf16", [(5120, 4, True), (4099, 3, True), (2560, 5, False), (2561, 8, False)])
def test_packed_conv_wide(dim, width, bf16):
    """Sizes past those where a lane takes 16 bytes of a row: sampled columns against the reference,
    the whole against the same sequences in two smaller calls."""
    import torch
    import selective_state_space_20_amd as sss
    rng = np.random.default_rng(dim)
    t = 8192 if bf16 else 7000
    cu = np.array([0, 3, 1500, 1500, 1507, 4000, t], np.int32)
    idx, initial = np.array([5, 3, 1, -1, 0, 2], np.int32), np.array([1, 1, 1, 1, 0, 1], np.uint8)
    x, w, b = rand(rng, (t, dim), bf16), rand(rng, (dim, width), scale=0.5), rand(rng, (dim,))
    state = rand(rng, (6, width - 1, dim), bf16)
    st, st2 = dev_of(state), dev_of(state)
    d = [dev_of(v) for v in (x, w, b, idx, initial)]
    out = sss.causal_conv1d_packed_fwd(d[0], d[1], d[2], cu_seqlens=dev_of(cu), conv_state=st, state_indices=d[3],
                                       has_initial=d[4], silu=True)
    parts = [sss.causal_conv1d_packed_fwd(d[0][lo:hi], d[1], d[2], cu_seqlens=dev_of(c), conv_state=st2,
                                          state_indices=d[3][s], has_initial=d[4][s], silu=True)
             for lo, hi, s, c in ((0, 1507, slice(0, 4), cu[:5]), (1507, t, slice(4, 6), cu[4:] - 1507))]
    assert torch.equal(torch.cat(parts), out) and torch.equal(st, st2)
    cols = np.unique(np.concatenate([np.arange(9), np.arange(dim - 9, dim), rng.integers(0, dim, 30)]))
    want, want_state, mag = ref.packed_conv(x[:, cols], w[cols], b[cols], cu, state[:, :, cols], idx, initial, True)
    close(host(out)[:, cols], want, 2 * (width + 6) * EPS * mag + (2.0 ** -8 * np.abs(want) if bf16 else 0) + 1e-37, "out")
    np.testing.assert_array_equal(host(st)[:, :, cols], want_state)


def test_packed_conv_without_cache_and_rows_outside():
    import torch
    import selective_state_space_20_amd as sss
    rng = np.random.default_rng(5)
    x, w = rand(rng, (50, 40)), rand(rng, (40, 4))
    cu = np.array([3, 10, 44], np.int32)
    out = torch.full((50, 40), 7.0, device="cuda:0")
    x[:3] = x[44:] = np.nan
    sss.causal_conv1d_packed_fwd(dev_of(x), dev_of(w), cu_seqlens=dev_of(cu), out=out)
    want, _, mag = ref.packed_conv(x, w, None, cu, None, None, None, False)
    got = host(out)
    assert (got[:3] == 7).all() and (got[44:] == 7).all()
    close(got[3:44], want[3:44], 2 * 10 * EPS * mag[3:44] + 1e-37, "out")


@pytest.mark.parametrize("rows,dim,width,bf16", [(1, 5120, 4, True), (3, 5121, 4, True), (70, 37, 3, True),
                                                 (5, 2, 2, True), (1, 1, 4, False), (9, 1001, 8, False),
                                                 (4, 64, 1, True), (300, 130, 5, True)])
def test_conv_update(rows, dim, width, bf16):
    import selective_state_space_20_amd as sss
    cu, idx, _, slots = packing([1] * rows)
    rng = np.random.default_rng(rows)
    x, w, b = rand(rng, (rows, dim), bf16), rand(rng, (dim, width), scale=0.5), rand(rng, (dim,))
    state = rand(rng, (slots, width - 1, dim), bf16)
    want, want_state, mag = ref.packed_conv(x, w, b, cu, state, idx, np.ones(rows), True)
    st = dev_of(state)
    out = sss.causal_conv1d_update(strided(x), dev_of(w), dev_of(b), conv_state=st, state_indices=dev_of(idx), silu=True)
    close(host(out), want, 2 * (width + 6) * EPS * mag + (2.0 ** -8 * np.abs(want) if bf16 else 0) + 1e-37, "out")
    np.testing.assert_array_equal(host(st), want_state)


def test_conv_prompt_then_steps_is_the_whole_prompt():
    """A prompt cut in two calls and then token by token, against the dense call on all of it."""
    import torch
    import selective_state_space_20_amd as sss
    rng = np.random.default_rng(6)
    x, w, b = dev_of(rand(rng, (90, 384), True)), dev_of(rand(rng, (384, 4))), dev_of(rand(rng, (384,)))
    whole = sss.causal_conv1d_fwd(x[None], w, b, silu=True)[0]
    st = torch.full((2, 3, 384), float("nan"), dtype=torch.bfloat16, device="cuda:0")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda:0")
    parts = [sss.causal_conv1d_packed_fwd(x[:41], w, b, cu_seqlens=i32(0, 41), conv_state=st, state_indices=i32(1), silu=True),
             sss.causal_conv1d_packed_fwd(x[41:43], w, b, cu_seqlens=i32(0, 2), conv_state=st, state_indices=i32(1),
                                          has_initial=torch.ones(1, dtype=torch.bool, device="cuda:0"), silu=True)]
    parts += [sss.causal_conv1d_update(x[i:i + 1], w, b, conv_state=st, state_indices=i32(1), silu=True) for i in range(43, 90)]
    assert torch.equal(torch.cat(parts), whole)
    assert torch.equal(st[1], x[87:])


@pytest.mark.parametrize("chunks", [None, 7], indirect=True)
@pytest.mark.parametrize("act", [True, False])
@pytest.mark.parametrize("batch,length,dim,width,bf16,grad32", [
    (2, 300, 64, 4, True, False), (1, 1, 5, 4, True, False), (3, 2, 257, 4, True, True), (2, 77, 1001, 3, False, False),
    (1, 500, 2, 8, False, False), (1, 64, 1, 2, True, False), (2, 129, 130, 1, True, False), (1, 1000, 12, 5, True, True)])
def test_conv_backward(batch, length, dim, width, bf16, grad32, act, chunks):
    import torch
    import selective_state_space_20_amd as sss
    rng = np.random.default_rng(length + dim)
    x, w, b = rand(rng, (batch, length, dim), bf16), rand(rng, (dim, width), scale=0.5), rand(rng, (dim,))
    dout = rand(rng, (batch, length, dim), bf16 and not grad32)
    (dx, dw, db), (mx, mw, mb) = ref.conv_backward(*(ref.widen(v) for v in (x, w, b, dout)), act)
    kw = {}
    if grad32:  # into the first half of wider fp32 rows
        wide = torch.full((batch, length, 2 * dim), -3.0, device="cuda:0")
        kw["dx"] = wide[:, :, :dim]
    g = sss.causal_conv1d_bwd(strided(x), dev_of(w), dev_of(b), dout=dev_of(dout), silu=act, **kw)
    out_bf16 = bf16 and not grad32
    # each dv carries the silu slope's own error: a few ulp of |dout| times a slope below 1.1
    c = 2 * (width + 12) * EPS
    close(host(g["dx"]), dx, c * (mx + np.abs(w).sum(1) * 4) + (2.0 ** -8 * np.abs(dx) if out_bf16 else 0) + 1e-30, "dx")
    close(host(g["dweight"]), dw, (600 + 4 * c / EPS) * EPS * (mw + 1e-6), "dweight")
    close(host(g["dbias"]), db, (600 + 4 * c / EPS) * EPS * (mb + 1e-6), "dbias")
    if grad32:
        assert bool((wide[:, :, dim:] == -3).all())
    again = sss.causal_conv1d_bwd(strided(x), dev_of(w), dev_of(b), dout=dev_of(dout), silu=act)
    assert torch.equal(again["dweight"], g["dweight"]) and torch.equal(again["dbias"], g["dbias"])


def test_conv_backward_against_differences():
    """The GPU's gradients against central differences of the 64-bit forward."""
    import selective_state_space_20_amd as sss
    rng = np.random.default_rng(8)
    x, w, b, dout = rand(rng, (2, 9, 6)), rand(rng, (6, 4)), rand(rng, (6,)), rand(rng, (2, 9, 6))
    g = sss.causal_conv1d_bwd(dev_of(x), dev_of(w), dev_of(b), dout=dev_of(dout), silu=True)
    x, w, b, dout = (v.astype(np.float64) for v in (x, w, b, dout))
    loss = lambda: float((dout * ref.conv_forward(x, w, b, True)).sum())
    for arr, got in ((x, host(g["dx"])), (w, host(g["dweight"])), (b, host(g["dbias"]))):
        for i in list(np.ndindex(arr.shape))[::5]:
            keep = arr[i]
            arr[i] = keep + 1e-5
            up = loss()
            arr[i] = keep - 1e-5
            down = loss()
            arr[i] = keep
            assert abs((up - down) / 2e-5 - got[i]) <= 1e-5 * (1 + abs(got[i]))


# -------------------------------------------------------------------------------- scan
def scan_inputs(rng, t, dim, n, bf16, bc16):
    A = -np.exp(rng.random((dim, n)) * np.log(16.0)).astype(np.float32)
    return dict(x=rand(rng, (t, dim), bf16), delta=rand(rng, (t, dim), bf16), A=A, B=rand(rng, (t, n), bc16),
                C=rand(rng, (t, n), bc16), D=rand(rng, (dim,)), z=rand(rng, (t, dim), bf16),
                bias=(rng.standard_normal(dim) - 3).astype(np.float32))


def scan_close(got, want, y16, what):
    tol = 1e-4 * np.nanmax(np.abs(want)) if want.size else 0.0
    close(got, want, tol + (2.0 ** -8 * np.abs(want) if y16 else 0), what)


@pytest.mark.parametrize("chunks", [None, 3, 30], indirect=True)
@pytest.mark.parametrize("lens", list(LENGTHS))
@pytest.mark.parametrize("dim,n,bf16,bc16,y16", [
    (5, 16, True, True, True), (64, 16, True, False, False), (130, 16, False, False, False), (129, 8, True, True, True),
    (70, 1, True, True, False), (66, 2, False, False, False), (65, 4, True, True, True), (96, 32, True, True, True),
    (33, 64, True, False, False), (200, 64, False, False, False)])
def test_packed_scan(lens, dim, n, bf16, bc16, y16, chunks):
    import torch
    import selective_state_space_20_amd as sss
    cu, idx, initial, slots = packing(LENGTHS[lens])
    t = int(cu[-1])
    rng = np.random.default_rng(dim * n)
    v = scan_inputs(rng, t, dim, n, bf16, bc16)
    state = rand(rng, (slots, dim, n))
    used = {int(i) for s, i in enumerate(idx) if 0 <= i < slots and initial[s]}
    for s in set(range(slots)) - used:
        state[s] = np.nan
    want, want_state = ref.packed_scan(v["x"], v["delta"], v["A"], v["B"], v["C"], v["D"], v["z"], cu, state, idx,
                                       initial, v["bias"], True)
    st = dev_of(state)
    y = torch.full((t, dim), float("nan"), dtype=torch.bfloat16 if y16 else torch.float32, device="cuda:0")
    sss.selective_scan_packed_fwd(strided(v["x"]), strided(v["delta"]), dev_of(v["A"]), strided(v["B"]), strided(v["C"]),
                                  dev_of(v["D"]), strided(v["z"]), cu_seqlens=dev_of(cu), state=st,
                                  state_indices=dev_of(idx), has_initial=dev_of(initial), delta_bias=dev_of(v["bias"]),
                                  delta_softplus=True, out=y)
    scan_close(host(y), want, y16, "y")
    got = host(st)
    touched = {int(i) for s, i in enumerate(idx) if 0 <= i < slots and cu[s + 1] > cu[s]}
    for s in range(slots):
        if s in touched:
            scan_close(got[s], want_state[s], False, f"slot {s}")
        else:
            np.testing.assert_array_equal(got[s], want_state[s])


@pytest.mark.parametrize("options", ["plain", "bias", "softplus", "no z", "no D", "no cache"])
def test_packed_scan_options(options):
    import selective_state_space_20_amd as sss
    cu = np.array([2, 40, 40, 141], np.int32)  # rows 0, 1 and 141.. belong to nobody
    rng = np.random.default_rng(11)
    v = scan_inputs(rng, 150, 70, 16, True, True)
    v["delta"] = ref.bf16_bits(np.abs(ref.widen(v["delta"])) * 0.1)
    v["bias"] = np.abs(v["bias"]) * 0.02
    D = None if options == "no D" else v["D"]
    z = None if options == "no z" else v["z"]
    bias = v["bias"] if options == "bias" else None
    state = None if options == "no cache" else rand(rng, (3, 70, 16))
    initial = None if state is None else np.array([1, 1, 0], np.uint8)
    want, want_state = ref.packed_scan(v["x"], v["delta"], v["A"], v["B"], v["C"], D, z, cu, state, None, initial, bias,
                                       options == "softplus")
    import torch
    y = torch.full((150, 70), 7.0, device="cuda:0")
    st = dev_of(state)
    sss.selective_scan_packed_fwd(dev_of(v["x"]), dev_of(v["delta"]), dev_of(v["A"]), dev_of(v["B"]), dev_of(v["C"]),
                                  dev_of(D), dev_of(z), cu_seqlens=dev_of(cu), state=st, has_initial=dev_of(initial),
                                  delta_bias=dev_of(bias), delta_softplus=options == "softplus", out=y)
    got = host(y)
    assert (got[:2] == 7).all() and (got[141:] == 7).all()
    scan_close(got[2:141], want[2:141], False, "y")
    if state is not None:
        scan_close(host(st), want_state, False, "state")


def test_packed_scan_decay_extremes():
    """A = 0 keeps the state for ever, A = -inf forgets it at once, zero steps change nothing."""
    import selective_state_space_20_amd as sss
    rng = np.random.default_rng(12)
    cu = np.array([0, 90, 200], np.int32)
    v = scan_inputs(rng, 200, 64, 16, False, False)
    v["delta"] = np.abs(v["delta"]) * 0.1
    v["delta"][50:70] = 0.0
    v["A"][:, 0], v["A"][:, 1] = 0.0, -np.inf
    state = rand(rng, (2, 64, 16))
    want, want_state = ref.packed_scan(v["x"], v["delta"], v["A"], v["B"], v["C"], v["D"], v["z"], cu, state, None,
                                       [1, 1], None, False)
    st = dev_of(state)
    y = sss.selective_scan_packed_fwd(*(dev_of(v[k]) for k in ("x", "delta", "A", "B", "C", "D", "z")),
                                      cu_seqlens=dev_of(cu), state=st, has_initial=dev_of(np.ones(2, np.uint8)))
    scan_close(host(y), want, False, "y")
    scan_close(host(st), want_state, False, "state")


@pytest.mark.parametrize("rows,dim,n,bf16,bc16,y16", [(1, 64, 16, True, True, True), (5, 37, 16, False, False, False),
                                                      (70, 130, 8, True, False, True), (3, 33, 1, True, True, False),
                                                      (2, 5, 2, False, False, False), (9, 100, 4, True, True, True),
                                                      (6, 70, 32, True, True, True), (33, 50, 64, True, True, False)])
def test_slot_update(rows, dim, n, bf16, bc16, y16):
    import torch
    import selective_state_space_20_amd as sss
    cu, idx, _, slots = packing([1] * rows)
    rng = np.random.default_rng(rows * n)
    v = scan_inputs(rng, rows, dim, n, bf16, bc16)
    state = rand(rng, (slots, dim, n))
    state[[s for s in range(slots) if s not in set(idx.tolist())]] = np.nan
    want, want_state = ref.packed_scan(v["x"], v["delta"], v["A"], v["B"], v["C"], v["D"], v["z"], cu, state, idx,
                                       np.ones(rows), v["bias"], True)
    st = dev_of(state)
    y = torch.full((rows, dim), float("nan"), dtype=torch.bfloat16 if y16 else torch.float32, device="cuda:0")
    sss.selective_state_update_slots(strided(v["x"]), strided(v["delta"]), dev_of(v["A"]), strided(v["B"]),
                                     strided(v["C"]), dev_of(v["D"]), strided(v["z"]), state=st,
                                     state_indices=dev_of(idx), delta_bias=dev_of(v["bias"]), delta_softplus=True, out=y)
    scan_close(host(y), want, y16, "y")
    got = host(st)
    touched = {int(i) for i in idx if 0 <= i < slots}
    for s in range(slots):
        if s in touched:
            scan_close(got[s], want_state[s], False, f"slot {s}")
        else:
            np.testing.assert_array_equal(got[s], want_state[s])


def test_slot_update_is_the_dense_update():
    """Identity slots, no front end: selective_state_update's results."""
    import torch
    import selective_state_space_20_amd as sss
    rng = np.random.default_rng(13)
    v = scan_inputs(rng, 7, 200, 16, True, False)
    v["delta"] = ref.bf16_bits(np.abs(ref.widen(v["delta"])) * 0.1)
    t = {k: dev_of(a) for k, a in v.items()}
    a, b = dev_of(rand(rng, (7, 200, 16))), None
    b = a.clone()
    ya = sss.selective_state_update(t["x"], t["delta"], t["A"], t["B"], t["C"], t["D"], t["z"], state=a)
    yb = sss.selective_state_update_slots(t["x"], t["delta"], t["A"], t["B"], t["C"], t["D"], t["z"], state=b)
    assert torch.allclose(ya, yb, rtol=1e-6, atol=1e-6) and torch.allclose(a, b, rtol=1e-6, atol=1e-6)


def test_scan_prompt_then_steps_is_the_whole_prompt():
    import torch
    import selective_state_space_20_amd as sss
    rng = np.random.default_rng(14)
    v = scan_inputs(rng, 300, 128, 16, True, True)
    t = {k: dev_of(a) for k, a in v.items()}
    i32 = lambda *s: torch.tensor(s, dtype=torch.int32, device="cuda:0")
    run = lambda fn, lo, hi, **kw: fn(t["x"][lo:hi], t["delta"][lo:hi], t["A"], t["B"][lo:hi], t["C"][lo:hi], t["D"],
                                      t["z"][lo:hi], delta_bias=t["bias"], delta_softplus=True, **kw)
    sw = torch.zeros(1, 128, 16, device="cuda:0")
    whole = run(sss.selective_scan_packed_fwd, 0, 300, cu_seqlens=i32(0, 300), state=sw)
    st = torch.full((3, 128, 16), float("nan"), device="cuda:0")
    parts = [run(sss.selective_scan_packed_fwd, 0, 190, cu_seqlens=i32(0, 190), state=st, state_indices=i32(2)),
             run(sss.selective_scan_packed_fwd, 190, 280, cu_seqlens=i32(0, 90), state=st, state_indices=i32(2),
                 has_initial=torch.ones(1, dtype=torch.uint8, device="cuda:0"))]
    parts += [run(sss.selective_state_update_slots, i, i + 1, state=st, state_indices=i32(2)) for i in range(280, 300)]
    got, want = host(torch.cat(parts)), host(whole)
    close(got, want, 1e-5 * np.abs(want).max(), "y")
    close(host(st[2]), host(sw[0]), 1e-5 * np.abs(host(sw)).max(), "state")


def test_sequences_larger_than_the_search_step():
    """More sequences than one and than two 64-way search steps hold."""
    import selective_state_space_20_amd as sss
    rng = np.random.default_rng(15)
    for n in (65, 4100):
        lens = rng.integers(0, 4, n)
        cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        t = int(cu[-1])
        x, w = rand(rng, (t, 8)), rand(rng, (8, 4))
        out = sss.causal_conv1d_packed_fwd(dev_of(x), dev_of(w), cu_seqlens=dev_of(cu))
        want, _, mag = ref.packed_conv(x, w, None, cu, None, None, None, False)
        close(host(out), want, 2 * 10 * EPS * mag + 1e-37, n)
        v = scan_inputs(rng, t, 4, 4, False, False)
        st = dev_of(np.zeros((n, 4, 4), np.float32))
        y = sss.selective_scan_packed_fwd(*(dev_of(v[k]) for k in ("x", "delta", "A", "B", "C", "D", "z")),
                                          cu_seqlens=dev_of(cu), state=st, delta_softplus=True)
        want, want_state = ref.packed_scan(*(v[k] for k in ("x", "delta", "A", "B", "C", "D", "z")), cu,
                                           np.zeros((n, 4, 4)), None, None, None, True)
        scan_close(host(y), want, False, n)
        scan_close(host(st), want_state, False, n)


def test_calls_run_on_the_current_stream_and_in_a_graph():
    """A decode step captured into a graph and replayed, with eager work in between."""
    import torch
    import selective_state_space_20_amd as sss
    rng = np.random.default_rng(16)
    v = scan_inputs(rng, 4, 64, 16, True, True)
    t = {k: dev_of(a) for k, a in v.items()}
    w = dev_of(rand(rng, (64, 4)))
    cst, st = torch.zeros(4, 3, 64, dtype=torch.bfloat16, device="cuda:0"), torch.zeros(4, 64, 16, device="cuda:0")
    y = torch.empty(4, 64, device="cuda:0")

    def step(cst, st, y):
        c = sss.causal_conv1d_update(t["x"], w, conv_state=cst, silu=True)
        sss.selective_state_update_slots(c, t["delta"], t["A"], t["B"], t["C"], t["D"], t["z"], state=st,
                                         delta_bias=t["bias"], delta_softplus=True, out=y)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ecst, est, ey = cst.clone(), st.clone(), y.clone()
    with torch.cuda.stream(side):
        step(cst.clone(), st.clone(), y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cst, st, y)
    for _ in range(5):
        graph.replay()
        step(ecst, est, ey)
        torch.cuda.synchronize()
        assert torch.equal(y, ey) and torch.equal(st, est) and torch.equal(cst, ecst)
