"""The layer norm's gradients as its forward call leaves off, on the GPU, with a bf16 residual stream: residual_out is
rounded, mean and rstd are of the sum before that.  Against the formula in 64 bits of what is handed over, and against the
gradient of the norm without the stream's rounding.

Error bounds, fixed beforehand, eps = 2^-24: hat = (h - mean) rstd of given numbers is within e = 4 eps (|h| + |mean|) rstd,
a sum over a row within 64 eps of its absolute terms, one over rows within 600 eps, as in test_layer_norm_gpu.py.  A
stream rounded to bf16 is off by half a step, 2^-8 of its value, and so hat by that times rstd.  bf16 results: half a
step, 2^-8 of the value."""
import pytest

from .test_layer_norm_gpu import DEV, EPS, rnd

pytestmark = pytest.mark.gpu


def gradients(h, mean, rstd, w, dout, dres, groups, off):
    """dx, dweight, dbias of the formula, each with its bound; off: how far h may be from what the kernel reads."""
    rows, dim = h.shape
    u = h.reshape(rows, groups, -1)
    m, r = mean[..., None], rstd[..., None]
    hat = (u - m) * r
    e = 4 * EPS * (u.abs() + m.abs()) * r + off.reshape(u.shape) * r
    g = (dout * w).reshape(u.shape)
    over = lambda t: t.mean(-1, keepdim=True)
    dh = r * (g - over(g) - hat * over(g * hat)) + dres.reshape(u.shape)
    slack = r * (64 * EPS * (g.abs() + over(g.abs()) + hat.abs() * over((g * hat).abs())) + e * over((g * hat).abs())
                 + (hat.abs() + e) * over(g.abs() * e)) + 4 * EPS * (dh.abs() + dres.reshape(u.shape).abs())
    flat = lambda t: t.reshape(h.shape)
    a = (dout * flat(hat)).abs()
    return {"dx": (flat(dh), flat(slack)), "dresidual": (flat(dh), flat(slack)),
            "dweight": ((dout * flat(hat)).sum(0), 600 * EPS * a.sum(0) + (dout.abs() * flat(e)).sum(0)),
            "dbias": (dout.sum(0), 600 * EPS * dout.abs().sum(0))}


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("rows, group, groups", [(70, 64, 3), (33, 250, 2), (9, 2560, 1), (5, 5001, 1), (1, 7, 1)])
@pytest.mark.parametrize("shift", [0.0, 30.0])
def test_gradients_of_what_the_forward_call_leaves(rows, group, groups, bf16, shift):
    import torch
    import selective_state_space_20_amd as sss
    dim, dt = group * groups, torch.bfloat16 if bf16 else torch.float32
    x, res = rnd(1, rows, dim, dtype=dt), rnd(2, rows, dim, dtype=torch.bfloat16, scale=2.0, shift=shift)
    w, b = rnd(3, dim, scale=0.3, shift=1.0), rnd(4, dim)
    dout, dres = rnd(5, rows, dim, dtype=dt), rnd(6, rows, dim, dtype=torch.bfloat16)
    _, h, mean, rstd = sss.layer_norm_fwd(x.to(DEV), w.to(DEV), b.to(DEV), res.to(DEV), group_size=group, eps=1e-3, return_stats=True)
    got = sss.layer_norm_bwd(dout.to(DEV), h, w.to(DEV), mean=mean, rstd=rstd, bias=True, dresidual_out=dres.to(DEV),
                             group_size=group)
    wide = lambda t: t.detach().cpu().double()
    exact = wide(x) + wide(res)
    u = exact.reshape(rows, groups, -1)
    # the statistics are of the sum before it is rounded
    d = 64 * EPS * u.abs().amax(-1)
    true_mean = u.mean(-1)
    true_rstd = 1 / torch.sqrt((u - true_mean[..., None]).square().mean(-1) + 1e-3)
    assert bool(((wide(mean) - true_mean).abs() <= d).all())
    assert bool(((wide(rstd) - true_rstd).abs() <= true_rstd * (true_rstd * d + 64 * EPS)).all())
    args = (wide(mean), wide(rstd), wide(w), wide(dout), wide(dres), groups)
    for h0, off in ((wide(h), 0 * exact), (exact, 2.0 ** -8 * exact.abs())):
        for name, (want, bound) in gradients(h0, *args, off).items():
            if got[name].dtype == torch.bfloat16:
                bound = bound + 2.0 ** -8 * (want.abs() + bound)
            err = (wide(got[name]) - want).abs()
            assert bool((err <= bound).all()), (name, float((err - bound).max()))
