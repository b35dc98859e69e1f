"""The norms around the block on the GPU, forward and gradients, against plain 64-bit references.

Error bounds, fixed beforehand, in units of eps = 2^-24: a row's sum of squares is formed in
chains of at most 32 terms per lane and a tree of ten, so that its factor is within about 30 eps;
silu and its slope add less than 20 eps of their terms for |z| < 6, the products a few each:
128 eps of the absolute terms for a forward result and 400 eps for a gradient, which also holds
a mean over the row.  Parameter gradients are summed over at most a few hundred rows per
partial and as many partials: 1000 eps of their absolute terms.  Where a result is rounded to
bf16, half an ulp more: 2^-8 of its value."""
import numpy as np
import pytest

from . import block_ref as ref
from .gpu_util import to_dev
from .test_block_gpu import EPS, close, host, rand, strided

pytestmark = pytest.mark.gpu


def dev_of(a):
    return to_dev(a, "cuda:0")


def rounding(bf16, v):
    return 2.0 ** -8 * np.abs(v) if bf16 else 0.0


@pytest.mark.parametrize("norm_first", [False, True])
@pytest.mark.parametrize("rows,dim,groups,x16,z16", [
    (3, 5120, 1, False, True), (37, 5120, 8, False, True), (2, 1, 1, False, False), (5, 7, 1, True, True),
    (70, 8, 1, True, True), (9, 18, 2, False, True), (1, 511, 1, True, True), (4, 1026, 2, False, False),
    (3, 1032, 1, True, False), (2, 2057, 1, False, True), (5, 6150, 1, True, True), (2, 8191, 1, False, True),
    (2, 12289, 1, True, True), (1, 16384, 1, False, False), (2, 32768, 1, True, True), (1100, 24, 3, False, True),
    (6, 768, 6, True, None), (3, 4100, 1, False, None), (37, 129, 1, False, True), (9, 400, 2, True, True),
    (33, 640, 10, False, True), (5, 300, 20, False, False), (40, 16, 8, True, True)])
def test_gated_norm(rows, dim, groups, x16, z16, norm_first):
    import torch
    import selective_state_space_20_amd as sss
    rng = np.random.default_rng(rows * dim)
    group, out16 = dim // groups, x16 if z16 is None else z16
    x, w = rand(rng, (rows, dim), x16), rand(rng, (dim,))
    z = None if z16 is None else rand(rng, (rows, dim), z16)
    dout = rand(rng, (rows, dim), out16)
    wide = [ref.widen(v) for v in (x, w, z, dout)]
    opt = dict(group_size=group, norm_before_gate=norm_first)
    dz_ = strided(z) if z is not None else None
    out, rstd = sss.rms_norm_gated_fwd(strided(x), dev_of(w), dz_, eps=1e-5, return_rstd=True, **opt)
    want, r = ref.gated_norm(*wide[:3], group, 1e-5, norm_first)
    close(host(out), want, 128 * EPS * np.abs(want) + rounding(out16, want) + 1e-37, "out")
    close(host(rstd), r, 64 * EPS * r, "rstd")
    kw = {}
    if z is not None:
        big = torch.full((rows, 2 * dim), -3.0, dtype=dz_.dtype, device="cuda:0")
        kw["dz"] = big[:, dim:]
    g = sss.rms_norm_gated_bwd(dev_of(dout), strided(x), dev_of(w), dz_, rstd=rstd, **opt, **kw)
    grads = ref.gated_norm_grad(wide[3], *wide[:3], host(rstd), group, norm_first)
    assert set(g) == set(grads)
    for k, bf16 in (("dx", x16), ("dz", z16)):
        if k in grads:
            close(host(g[k]), grads[k][0], 400 * EPS * grads[k][1] + rounding(bf16, grads[k][0]) + 1e-37, k)
    close(host(g["dweight"]), grads["dweight"][0], 1000 * EPS * grads["dweight"][1] + 1e-37, "dweight")
    if z is not None:
        assert bool((big[:, :dim] == -3).all())
    again = sss.rms_norm_gated_bwd(dev_of(dout), strided(x), dev_of(w), dz_, rstd=rstd, **opt)
    assert torch.equal(again["dweight"], g["dweight"])


@pytest.mark.parametrize("post,scaled,first", [(True, True, False), (False, False, False), (True, False, False),
                                               (False, True, False), (False, False, True)])
@pytest.mark.parametrize("rows,dim,x16,h16", [
    (3, 2560, True, False), (1, 1, False, False), (5, 7, True, True), (70, 8, True, False), (2, 65, False, False),
    (9, 600, True, True), (1, 1025, True, False), (300, 40, False, False), (3, 2051, True, False),
    (2, 5120, False, True), (2, 8192, True, False), (2, 8200, True, False), (1, 16000, False, False),
    (2, 32768, True, True), (35, 100, True, False), (17, 250, False, True), (3, 9, True, False)])
def test_residual_norm(rows, dim, x16, h16, post, scaled, first):
    import torch
    import selective_state_space_20_amd as sss
    rng = np.random.default_rng(rows + dim)
    x, w, dout = rand(rng, (rows, dim), x16), rand(rng, (dim,)), rand(rng, (rows, dim), x16)
    h = None if first else rand(rng, (rows, dim), h16)
    dnew = rand(rng, (rows, dim), h16 and not first)
    wp, scale = rand(rng, (dim,)) if post else None, rand(rng, (dim,)) if scaled else None
    h16 = h16 and not first  # the stream starts in fp32
    xw, ww, hw, dw, nw, pw, sw = (ref.widen(v) for v in (x, w, h, dout, dnew, wp, scale))
    opt = dict(post_weight=dev_of(wp), scale=dev_of(scale), alpha=0.75)
    out, new, rstd, rstd_post = sss.rms_norm_residual_fwd(strided(x), dev_of(w), None if first else strided(h), eps=1e-5,
                                                          return_rstd=True, **opt)
    want, want_new, r, rp, mag = ref.residual_norm(xw, ww, hw, pw, sw, 0.75, 1e-5)
    close(host(new), want_new, 128 * EPS * mag + rounding(h16, want_new) + 1e-37, "residual_out")
    # the sum's cancellation carries over into its norm, through the factor too
    carry = 128 * EPS * (mag + np.abs(want_new) * np.sqrt((mag ** 2).mean(-1, keepdims=True)) * r) * r * np.abs(ww)
    close(host(out), want, 128 * EPS * np.abs(want) + carry + rounding(x16, want) + 1e-37, "out")
    assert (rstd_post is None) == (not post)
    # in place
    if not first:
        hh = dev_of(h)
        o2, n2 = sss.rms_norm_residual_fwd(dev_of(x), dev_of(w), hh, eps=1e-5, residual_out=hh, **opt)
        assert n2 is hh and torch.equal(n2, new) and torch.equal(o2, out)
    need_x = post or scaled
    g = sss.rms_norm_residual_bwd(dev_of(dout), dev_of(dnew), residual_out=new, weight=dev_of(w), rstd=rstd,
                                  x=strided(x) if need_x else None, rstd_post=rstd_post, **opt)
    grads = ref.residual_norm_grad(dw, nw, xw, ww, host(new), host(rstd)[:, None], pw, sw,
                                   host(rstd_post)[:, None] if post else None, 0.75)
    assert set(g) == set(grads)
    for k, bf16 in (("dx", x16), ("dresidual", h16)):
        close(host(g[k]), grads[k][0], 400 * EPS * grads[k][1] + rounding(bf16, grads[k][0]) + 1e-37, k)
    for k in ("dweight", "dpost_weight", "dscale"):
        if k in grads:
            close(host(g[k]), grads[k][0], 1000 * EPS * grads[k][1] + 1e-37, k)
    g2 = sss.rms_norm_residual_bwd(dev_of(dout), residual_out=new, weight=dev_of(w), rstd=rstd,
                                   x=strided(x) if need_x else None, rstd_post=rstd_post, want_dresidual=False, **opt)
    grads = ref.residual_norm_grad(dw, None, xw, ww, host(new), host(rstd)[:, None], pw, sw,
                                   host(rstd_post)[:, None] if post else None, 0.75)
    assert "dresidual" not in g2
    close(host(g2["dx"]), grads["dx"][0], 400 * EPS * grads["dx"][1] + rounding(x16, grads["dx"][0]) + 1e-37, "dx alone")


def test_norms_against_differences():
    """The GPU's gradients against central differences of the 64-bit forward."""
    import selective_state_space_20_amd as sss
    rng = np.random.default_rng(21)
    x, z, w, dout = (rand(rng, s) for s in ((4, 12), (4, 12), (12,), (4, 12)))
    for first in (False, True):
        out, rstd = sss.rms_norm_gated_fwd(dev_of(x), dev_of(w), dev_of(z), eps=0.01, group_size=4,
                                           norm_before_gate=first, return_rstd=True)
        g = sss.rms_norm_gated_bwd(dev_of(dout), dev_of(x), dev_of(w), dev_of(z), rstd=rstd, group_size=4,
                                   norm_before_gate=first)
        a = [v.astype(np.float64) for v in (x, w, z, dout)]
        loss = lambda: float((a[3] * ref.gated_norm(a[0], a[1], a[2], 4, 0.01, first)[0]).sum())
        for arr, got in zip(a, (g["dx"], g["dweight"], g["dz"])):
            got = host(got)
            for i in list(np.ndindex(arr.shape))[::3]:
                keep = arr[i]
                arr[i] = keep + 1e-5
                up = loss()
                arr[i] = keep - 1e-5
                down = loss()
                arr[i] = keep
                assert abs((up - down) / 2e-5 - got[i]) <= 2e-5 * (1 + abs(got[i]))


def test_zero_rows_and_zero_values():
    import torch
    import selective_state_space_20_amd as sss
    w = torch.ones(64, device="cuda:0")
    e = torch.empty(0, 64, device="cuda:0")
    out, rstd = sss.rms_norm_gated_fwd(e, w, e, return_rstd=True)
    assert out.shape == (0, 64)
    g = sss.rms_norm_gated_bwd(e, e, w, e, rstd=rstd)
    assert bool((g["dweight"] == 0).all()) and g["dx"].shape == (0, 64)
    out, h = sss.rms_norm_residual_fwd(e, w, e)
    g = sss.rms_norm_residual_bwd(e, residual_out=e, weight=w, rstd=torch.empty(0, device="cuda:0"))
    assert bool((g["dweight"] == 0).all())
    z = torch.zeros(3, 64, device="cuda:0")  # a row of zeros: out 0, no NaN
    out, h = sss.rms_norm_residual_fwd(z, w, z)
    assert bool((out == 0).all()) and bool((h == 0).all())
    x = torch.full((2, 64), 3.0, device="cuda:0")
    x[0, 5] = float("nan")  # stays in its row
    out = sss.rms_norm_gated_fwd(x, w, x)
    assert bool(out[0].isnan().all()) and bool(out[1].isfinite().all())


# rows on 512 lanes, in two to four pieces of each width, just below and above the widths' ends
@pytest.mark.parametrize("norm_first", [False, True])
@pytest.mark.parametrize("rows,dim,groups,x16,z16", [
    (1100, 3333, 1, False, True), (3, 4096, 1, True, False), (2, 8202, 2, False, False), (4, 6143, 1, False, True),
    (3, 6145, 1, False, True), (700, 5120, 1, False, True), (2, 9001, 1, True, True), (3, 13000, 1, False, None)])
def test_gated_norm_on_512_lanes(rows, dim, groups, x16, z16, norm_first):
    test_gated_norm(rows, dim, groups, x16, z16, norm_first)


@pytest.mark.parametrize("post,scaled,first", [(True, True, False), (False, False, True)])
@pytest.mark.parametrize("rows,dim,x16,h16", [
    (1100, 3333, True, False), (3, 4096, False, True), (2, 4097, False, False), (5, 6144, True, False),
    (3, 6145, True, False), (2, 6200, True, True), (600, 8192, True, True)])
def test_residual_norm_on_512_lanes(rows, dim, x16, h16, post, scaled, first):
    test_residual_norm(rows, dim, x16, h16, post, scaled, first)
