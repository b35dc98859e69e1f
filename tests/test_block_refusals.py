"""What the operators around the scan refuse, before any device work (CPU only): the C calls on
fake addresses, and the binding on CPU tensors."""
import pytest
import torch

import selective_state_space_20_amd as sss
from selective_state_space_20_amd import load

NULL_ARG, BAD_DIM, UNSUPPORTED, WORKSPACE, ALIAS, HIP = -1, -2, -3, -4, -5, -6
P = 1 << 24  # fake addresses, far apart; never dereferenced


def call(fn, defaults, kw):
    a = dict(defaults)
    assert set(kw) <= set(a), set(kw) - set(a)
    a.update(kw)
    return getattr(load(), fn)(*a.values())


def conv(**kw):
    return call("causal_conv1d_packed_fwd", dict(
        x=P, x_stride=8, weight=2 * P, bias=0, conv_state=3 * P, cu=4 * P, idx=0, initial=0, out=5 * P, tokens=6,
        nseq=2, slots=2, dim=8, width=4, io_dtype=0, silu=1, stream=0), kw)


def conv_step(**kw):
    return call("causal_conv1d_update", dict(
        x=P, x_stride=8, weight=2 * P, bias=0, conv_state=3 * P, idx=0, out=5 * P, batch=2, slots=2, dim=8, width=4,
        io_dtype=0, silu=1, stream=0), kw)


def conv_bwd(**kw):
    return call("causal_conv1d_bwd", dict(
        x=P, xb=80, x_stride=8, weight=2 * P, bias=3 * P, dout=4 * P, dx=5 * P, dxb=80, dx_stride=8, dweight=6 * P,
        dbias=7 * P, batch=2, seqlen=10, dim=8, width=4, io_dtype=1, dout_dtype=1, dx_dtype=1, silu=1, workspace=8 * P,
        workspace_bytes=1 << 20, stream=0), kw)


def scan(**kw):
    return call("selective_scan_packed_fwd", dict(
        x=P, sx=8, delta=2 * P, sd=8, A=3 * P, B=4 * P, sb=16, C=5 * P, sc=16, D=0, z=6 * P, sz=8, bias=0, flags=0,
        state=7 * P, cu=8 * P, idx=0, initial=0, y=9 * P, tokens=6, nseq=2, slots=2, dim=8, dstate=16, io_dtype=1,
        bc_dtype=1, y_dtype=0, workspace=0, workspace_bytes=0, stream=0), kw)


def step(**kw):
    return call("selective_state_update_slots", dict(
        x=P, sx=8, delta=2 * P, sd=8, A=3 * P, B=4 * P, sb=16, C=5 * P, sc=16, D=0, z=6 * P, sz=8, bias=0, flags=0,
        state=7 * P, idx=0, y=9 * P, batch=2, slots=2, dim=8, dstate=16, io_dtype=1, bc_dtype=1, y_dtype=0, stream=0),
        kw)


def test_conv_rejections():
    for k in ("x", "weight", "cu", "out"):
        assert conv(**{k: 0}) == NULL_ARG, k
    assert conv(dim=0) == BAD_DIM and conv(tokens=-1) == BAD_DIM and conv(nseq=-1) == BAD_DIM
    assert conv(tokens=(1 << 30) + 1) == BAD_DIM and conv(slots=0) == BAD_DIM
    assert conv(slots=1) == BAD_DIM                      # two sequences, one slot, no indices
    assert conv(x_stride=7) == BAD_DIM and conv(x_stride=(1 << 24) + 1) == BAD_DIM
    assert conv(width=0) == UNSUPPORTED and conv(width=9) == UNSUPPORTED and conv(io_dtype=2) == UNSUPPORTED
    assert conv(x=P + 2) == UNSUPPORTED                  # fp32 at a 2-byte address
    assert conv(cu=4 * P + 2) == UNSUPPORTED
    assert conv(out=P) == ALIAS and conv(out=3 * P) == ALIAS and conv(conv_state=4 * P) == ALIAS
    assert conv(x_stride=20, out=P + 32) == ALIAS        # inside the span of strided rows
    assert conv(tokens=0) == 0 and conv(nseq=0) == 0     # nothing to do


def test_conv_step_rejections():
    for k in ("x", "weight", "conv_state", "out"):
        assert conv_step(**{k: 0}) == NULL_ARG, k
    assert conv_step(slots=1) == BAD_DIM and conv_step(batch=-1) == BAD_DIM
    assert conv_step(batch=1 << 30, idx=6 * P) == BAD_DIM   # more threads than a grid holds
    assert conv_step(io_dtype=1, x=P + 1) == UNSUPPORTED
    assert conv_step(out=3 * P) == ALIAS
    assert conv_step(batch=0) == 0


def test_conv_gradient_rejections():
    for k in ("x", "weight", "dout", "dx", "dweight", "dbias"):
        assert conv_bwd(**{k: 0}) == NULL_ARG, k
    assert conv_bwd(batch=0) == BAD_DIM and conv_bwd(seqlen=0) == BAD_DIM and conv_bwd(dim=0, width=9) == BAD_DIM
    assert conv_bwd(width=9) == UNSUPPORTED and conv_bwd(io_dtype=3) == UNSUPPORTED
    assert conv_bwd(io_dtype=0, dout_dtype=1, dx_dtype=0) == UNSUPPORTED  # bf16 gradients of fp32 inputs
    assert conv_bwd(x_stride=4) == BAD_DIM and conv_bwd(dxb=79) == BAD_DIM and conv_bwd(xb=-1) == BAD_DIM
    assert conv_bwd(workspace=8 * P + 4) == UNSUPPORTED
    assert conv_bwd(dx=P) == ALIAS and conv_bwd(dweight=2 * P) == ALIAS and conv_bwd(dbias=6 * P) == ALIAS


def test_scan_rejections():
    for k in ("x", "delta", "A", "B", "C", "cu", "y"):
        assert scan(**{k: 0}) == NULL_ARG, k
    assert scan(dstate=3) == UNSUPPORTED and scan(dstate=128) == UNSUPPORTED and scan(dim=0) == BAD_DIM
    assert scan(dstate=64, sb=64, sc=64, dim=(1 << 24) + 1, sx=1 << 24) == BAD_DIM
    assert scan(sb=15) == BAD_DIM and scan(sz=1) == BAD_DIM and scan(slots=1) == BAD_DIM
    assert scan(flags=1) == UNSUPPORTED and scan(flags=4) == UNSUPPORTED
    for k in ("io_dtype", "bc_dtype", "y_dtype"):
        assert scan(**{k: 2}) == UNSUPPORTED, k
    assert scan(A=3 * P + 2) == UNSUPPORTED and scan(workspace=4) == UNSUPPORTED
    assert scan(y=P) == ALIAS and scan(state=3 * P) == ALIAS and scan(y=7 * P) == ALIAS
    assert scan(tokens=0) == 0 and scan(nseq=0) == 0


def test_step_rejections():
    for k in ("x", "delta", "A", "B", "C", "state", "y"):
        assert step(**{k: 0}) == NULL_ARG, k
    assert step(slots=1) == BAD_DIM and step(dstate=5) == UNSUPPORTED and step(y=7 * P) == ALIAS
    assert step(batch=0) == 0


def test_workspace_queries():
    assert sss.selective_scan_packed_fwd_workspace_size(0, 64, 16) == 0
    assert sss.selective_scan_packed_fwd_workspace_size(100, 64, 3) == 0
    assert sss.selective_scan_packed_fwd_workspace_size(16384, 5120, 16) > 0
    assert sss.causal_conv1d_bwd_workspace_size(0, 5, 5, 4) == 0
    assert sss.causal_conv1d_bwd_workspace_size(2, 100, 64, 4) >= 2 * 5 * 64 * 4


# ------------------------------------------------------------------------------ binding
def t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def test_binding_rejects_host_tensors_types_and_shapes():
    cu = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="must be on a GPU"):
        sss.causal_conv1d_packed_fwd(t(4, 8), t(8, 4), cu_seqlens=cu)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        sss.causal_conv1d_packed_fwd(t(4, 8, dtype=torch.float16), t(8, 4), cu_seqlens=cu)
    with pytest.raises(ValueError, match="2-D"):
        sss.causal_conv1d_update(t(2, 4, 8), t(8, 4), conv_state=t(2, 3, 8))
    with pytest.raises(ValueError, match="must be on a GPU"):
        sss.causal_conv1d_bwd(t(2, 4, 8), t(8, 4), dout=t(2, 4, 8))
    with pytest.raises(ValueError, match="dout must be"):
        sss.causal_conv1d_bwd(t(2, 4, 8), t(8, 4), dout=t(2, 4, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        sss.selective_scan_packed_fwd(t(4, 8), t(4, 8), t(8, 16), t(4, 16, dtype=torch.float64), t(4, 16), cu_seqlens=cu)
    with pytest.raises(ValueError, match="must be on a GPU"):
        sss.selective_state_update_slots(t(4, 8), t(4, 8), t(8, 16), t(4, 16), t(4, 16), state=t(4, 8, 16))


def gated(**kw):
    return call("rms_norm_gated_fwd", dict(x=P, sx=8, weight=2 * P, z=3 * P, sz=8, out=4 * P, rstd=5 * P, rows=3, dim=8,
                                           group=4, eps=1e-5, flags=0, x_dtype=0, out_dtype=1, stream=0), kw)


def gated_bwd(**kw):
    return call("rms_norm_gated_bwd", dict(
        dout=P, x=2 * P, sx=8, weight=3 * P, z=4 * P, sz=8, rstd=5 * P, dx=6 * P, dz=7 * P, sdz=8, dweight=8 * P, rows=3,
        dim=8, group=4, flags=0, x_dtype=0, out_dtype=1, workspace=9 * P, workspace_bytes=1 << 20, stream=0), kw)


def residual(**kw):
    return call("rms_norm_residual_fwd", dict(
        x=P, sx=8, residual=2 * P, sr=8, post=3 * P, scale=4 * P, weight=5 * P, out=6 * P, residual_out=7 * P,
        rstd_post=8 * P, rstd=9 * P, rows=3, dim=8, alpha=1.0, eps=1e-5, io_dtype=1, residual_dtype=0, stream=0), kw)


def residual_bwd(**kw):
    return call("rms_norm_residual_bwd", dict(
        dout=P, dres_out=2 * P, x=3 * P, sx=8, residual_out=4 * P, post=5 * P, scale=6 * P, weight=7 * P, rstd_post=8 * P,
        rstd=9 * P, dx=10 * P, dres=11 * P, dweight=12 * P, dpost=13 * P, dscale=14 * P, rows=3, dim=8, alpha=1.0,
        io_dtype=1, residual_dtype=0, workspace=15 * P, workspace_bytes=1 << 20, stream=0), kw)


def test_gated_norm_rejections():
    for k in ("x", "weight", "out"):
        assert gated(**{k: 0}) == NULL_ARG, k
    for k in ("dout", "x", "weight", "rstd", "dx", "dz", "dweight"):
        assert gated_bwd(**{k: 0}) == NULL_ARG, k
    for fn in (gated, gated_bwd):
        assert fn(rows=-1) == BAD_DIM and fn(dim=0) == BAD_DIM and fn(group=3) == BAD_DIM and fn(sx=7) == BAD_DIM
        assert fn(dim=65536, group=65536, sx=65536, sz=65536) == UNSUPPORTED
        assert fn(rows=1 << 28) == BAD_DIM
        assert fn(flags=2) == UNSUPPORTED and fn(x_dtype=2) == UNSUPPORTED and fn(out_dtype=-1) == UNSUPPORTED
        assert fn(x=2 * P + 2) == UNSUPPORTED
    assert gated(out=P) == ALIAS and gated(out=3 * P) == ALIAS and gated(rstd=4 * P) == ALIAS
    assert gated_bwd(dx=2 * P) == ALIAS and gated_bwd(dz=6 * P) == ALIAS and gated_bwd(dweight=3 * P) == ALIAS
    assert gated_bwd(sdz=4) == BAD_DIM and gated_bwd(workspace=9 * P + 8) == UNSUPPORTED
    assert gated(rows=0) == 0


def test_residual_norm_rejections():
    for k in ("x", "weight", "out", "residual_out"):
        assert residual(**{k: 0}) == NULL_ARG, k
    for k in ("dout", "x", "residual_out", "weight", "rstd_post", "rstd", "dx", "dweight", "dpost", "dscale"):
        assert residual_bwd(**{k: 0}) == NULL_ARG, k
    for fn in (residual, residual_bwd):
        assert fn(rows=-1) == BAD_DIM and fn(dim=0) == BAD_DIM and fn(sx=7) == BAD_DIM
        assert fn(dim=32769, sx=32769) == UNSUPPORTED and fn(io_dtype=2) == UNSUPPORTED
        assert fn(residual_dtype=5) == UNSUPPORTED
    assert residual(out=P) == ALIAS and residual(residual_out=P) == ALIAS
    assert residual(residual=7 * P, sr=9) == ALIAS      # in place needs the same rows
    assert residual(residual=7 * P + 32) == ALIAS
    assert residual_bwd(dx=P) == ALIAS and residual_bwd(dscale=13 * P) == ALIAS
    assert residual(rows=0) == 0


def test_norm_binding_rejections():
    with pytest.raises(ValueError, match="must divide"):
        sss.rms_norm_gated_fwd(t(2, 8), t(8), group_size=3)
    with pytest.raises(ValueError, match="must be on a GPU"):
        sss.rms_norm_gated_fwd(t(2, 8), t(8))
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        sss.rms_norm_residual_fwd(t(2, 8, dtype=torch.float16), t(8))
    with pytest.raises(ValueError, match="x is needed"):
        sss.rms_norm_residual_bwd(t(2, 8), residual_out=t(2, 8), weight=t(8), rstd=t(2), scale=t(8))
    with pytest.raises(ValueError, match="rstd_post is needed"):
        sss.rms_norm_residual_bwd(t(2, 8), residual_out=t(2, 8), weight=t(8), rstd=t(2), x=t(2, 8), post_weight=t(8))
