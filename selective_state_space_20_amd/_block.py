"""Binding of the operators around the scan: the convolution and the scan over packed prompts
and their single-token steps on cache slots, the convolution's gradients, and the norms around
the block.

As in ``_lib``, only argument checks, output allocation and the C call: every step of the
computation runs in the library's HIP kernels.

``stream`` is the handle of the HIP stream that a call's work is queued on (None: the current one).
For another one than the current, the caller has it wait for what makes the operands, keeps the
operands until the work is done, and has the current stream wait before it uses the results.
"""
from __future__ import annotations

from . import _lib
from ._lib import SSS_BF16, SSS_DELTA_SOFTPLUS, SSS_F32, SSS_NORM_BEFORE_GATE, SSSError, load


_torch = _current_gpu = None


def torch_():
    """torch, imported with the first call (as the library is), not with the package."""
    global _torch, _current_gpu
    if _torch is None:
        load()
        import torch
        _current_gpu = torch._C._cuda_getDevice
        _torch = torch
    return _torch


# The checks below take one combined condition where all is well, since a decode step on small
# batches is as long as its call; what is wrong is found out afterwards.
def _refuse(t, name, dtype, shape, index):
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda or t.get_device() != index:
        raise ValueError(f"{name} must be on a GPU ({f'cuda:{index}' if index >= 0 else 'that of x'}), got {t.device}")


def _rows(t, name, dtype, rows, dim, index):
    """Checks a (rows, dim) tensor whose rows may be strided; returns (pointer, row stride)."""
    if t.dtype is dtype and t.shape == (rows, dim) and t.get_device() == index >= 0:
        s0, s1 = t.stride()
        if s1 == 1 and s0 >= dim and rows > 1:
            return t.data_ptr(), s0
        if rows <= 1 and (s1 == 1 or dim == 1):  # one row: its stride has no meaning, and may be any
            return t.data_ptr(), dim
        if dim == 1 and s0 >= 1:
            return t.data_ptr(), s0
        raise ValueError(f"{name}: rows must be {dim} adjacent elements and not overlap, got strides {(s0, s1)}")
    _refuse(t, name, dtype, (rows, dim), index)


def _dense(t, name, dtype, shape, index):
    """Checks a contiguous tensor on the call's GPU; returns its pointer (0 for None)."""
    if t is None:
        return 0
    if t.dtype is dtype and t.shape == shape and t.get_device() == index >= 0 and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, name, dtype, shape, index)
    raise ValueError(f"{name} must be contiguous")


def _new(like, shape, dtype, stream):
    """A tensor on like's GPU for the call's work, in memory of the stream that the work runs on."""
    if stream is None or stream == _torch._C._cuda_getCurrentRawStream(like.get_device()):
        return like.new_empty(shape, dtype=dtype)
    return _lib._empty(shape, dtype, like.device, stream)


def _out(out, name, like, dtype, shape, index, stream):
    """The given output, checked, or a new one on like's GPU; returns (tensor, pointer)."""
    if out is None:
        out = like.new_empty(shape, dtype=dtype) if stream is None else _new(like, shape, dtype, stream)
        return out, out.data_ptr()
    return out, _dense(out, name, dtype, shape, index)


def _scratch(workspace, nbytes, like, stream):
    """The given workspace, checked, or a new one; returns (tensor to keep, pointer, bytes)."""
    if workspace is None:
        if nbytes == 0:
            return None, 0, 0
        workspace = _new(like, (nbytes,), _torch.uint8, stream)
        return workspace, workspace.data_ptr(), nbytes
    return (workspace, *_lib._workspace(workspace, like.device))


def _keep(stream, index, *tensors):
    """Memory of the caller's that work on a given other stream writes: not handed out again before
    that work is done."""
    if stream != _torch._C._cuda_getCurrentRawStream(index):
        s = _lib._stream_of(stream, index)
        for t in tensors:
            if t is not None:
                t.record_stream(s)


def _code(dtype, name):
    torch = torch_()
    if dtype is torch.bfloat16:
        return SSS_BF16
    if dtype is torch.float32:
        return SSS_F32
    raise ValueError(f"{name} must be float32 or bfloat16, got {dtype}")


def _two_d(t, name):
    if t.ndim != 2:
        raise ValueError(f"{name} must be 2-D, got shape {tuple(t.shape)}")
    return t.shape


def _stream(stream, index):
    """The given stream, or the current one of the call's GPU (its handle without a Stream object)."""
    return stream if stream is not None else _torch._C._cuda_getCurrentRawStream(index)


class _Elsewhere:
    """The library with a GPU that is not the current one made current for each call."""

    def __init__(self, index):
        self.index = index

    def __getattr__(self, name):
        def call(*args):
            with _torch.cuda.device(self.index):
                return getattr(_lib._lib, name)(*args)
        return call


def _library(index):
    """The library, for operands on GPU `index`: its kernels run on the current GPU where the stream is
    the default one, whose handle is the same on all of them."""
    return _lib._lib if index == _current_gpu() else _Elsewhere(index)


def _cache(state, name, dtype, tail, index):
    """A (slots, *tail) cache; returns (pointer, slots)."""
    if state is None:
        return 0, 0
    if state.ndim != 1 + len(tail) or state.shape[0] < 1:
        raise ValueError(f"{name} must have shape (slots, {', '.join(map(str, tail))}), got {tuple(state.shape)}")
    slots = state.shape[0]
    return _dense(state, name, dtype, (slots, *tail), index), slots


def _sequences(cu_seqlens, state_indices, has_initial, state, slots, index):
    """Checks what describes a packed batch; returns (nseq, cu, indices, initial) with pointers."""
    torch = torch_()
    if cu_seqlens.ndim != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError(f"cu_seqlens must be 1-D with one entry more than sequences, got {tuple(cu_seqlens.shape)}")
    nseq = cu_seqlens.shape[0] - 1
    cu = _dense(cu_seqlens, "cu_seqlens", torch.int32, (nseq + 1,), index)
    idx = _dense(state_indices, "state_indices", torch.int32, (nseq,), index)
    if state is not None and state_indices is None and nseq > slots:
        raise ValueError(f"{nseq} sequences need as many slots or state_indices, the cache has {slots}")
    if state is None and has_initial is not None:
        raise ValueError("has_initial needs a cache to start from")
    ini = 0
    if has_initial is not None:
        if has_initial.dtype not in (torch.bool, torch.uint8):
            raise ValueError(f"has_initial must be bool or uint8, got {has_initial.dtype}")
        ini = _dense(has_initial, "has_initial", has_initial.dtype, (nseq,), index)
    return nseq, cu, idx, ini


def causal_conv1d_packed_fwd(x, weight, bias=None, *, cu_seqlens, conv_state=None, state_indices=None,
                             has_initial=None, silu=False, out=None, stream=None):
    """Causal depthwise convolution over packed prompts: out (tokens, dim) in x's dtype.

    x (tokens, dim) float32 or bfloat16, rows may be strided; weight (dim, width), bias (dim)
    float32; cu_seqlens (nseq + 1) int32.  conv_state (slots, width-1, dim) in x's dtype keeps
    each sequence's last width-1 inputs (updated in place) in slot state_indices[s] (int32; None:
    slot s; -1: none); has_initial (nseq) bool marks the sequences that continue their slot.
    Rows outside every sequence are left as they are in ``out``."""
    torch = torch_()
    gpu = x.get_device()
    tokens, dim = _two_d(x, "x")
    code = _code(x.dtype, "x")
    xp, xs = _rows(x, "x", x.dtype, tokens, dim, gpu)
    width = _two_d(weight, "weight")[1]
    wp = _dense(weight, "weight", torch.float32, (dim, width), gpu)
    bp = _dense(bias, "bias", torch.float32, (dim,), gpu)
    sp, slots = _cache(conv_state, "conv_state", x.dtype, (width - 1, dim), gpu)
    nseq, cu, idx, ini = _sequences(cu_seqlens, state_indices, has_initial, conv_state, slots, gpu)
    o, op = _out(out, "out", x, x.dtype, (tokens, dim), gpu, stream)
    if tokens == 0:
        return o
    rc = _library(gpu).causal_conv1d_packed_fwd(xp, xs, wp, bp, sp, cu, idx, ini, op, tokens, nseq, slots if sp else 0, dim,
                                         width, code, int(bool(silu)), _stream(stream, gpu))
    if rc != 0:
        raise SSSError(rc, "causal_conv1d_packed_fwd")
    if stream is not None:
        _keep(stream, gpu, o)
    return o


def causal_conv1d_update(x, weight, bias=None, *, conv_state, state_indices=None, silu=False, out=None, stream=None):
    """One token of each row through the convolution: out (batch, dim) in x's dtype.

    x (batch, dim), rows may be strided; conv_state (slots, width-1, dim) in x's dtype, updated
    in place, row b's in slot state_indices[b] (int32; None: slot b; -1: none, the row starts
    from zeros and keeps nothing)."""
    torch = torch_()
    gpu = x.get_device()
    batch, dim = _two_d(x, "x")
    code = _code(x.dtype, "x")
    xp, xs = _rows(x, "x", x.dtype, batch, dim, gpu)
    width = _two_d(weight, "weight")[1]
    wp = _dense(weight, "weight", torch.float32, (dim, width), gpu)
    bp = _dense(bias, "bias", torch.float32, (dim,), gpu)
    sp, slots = _cache(conv_state, "conv_state", x.dtype, (width - 1, dim), gpu)
    idx = _dense(state_indices, "state_indices", torch.int32, (batch,), gpu)
    if state_indices is None and batch > slots:
        raise ValueError(f"{batch} rows need as many slots or state_indices, the cache has {slots}")
    o, op = _out(out, "out", x, x.dtype, (batch, dim), gpu, stream)
    if batch == 0:
        return o
    rc = _library(gpu).causal_conv1d_update(xp, xs, wp, bp, sp, idx, op, batch, slots, dim, width, code, int(bool(silu)),
                                     _stream(stream, gpu))
    if rc != 0:
        raise SSSError(rc, "causal_conv1d_update")
    if stream is not None:
        _keep(stream, gpu, o)
    return o


def causal_conv1d_bwd_workspace_size(batch, seqlen, dim, width, io_dtype=SSS_BF16, device=0) -> int:
    return int(load().causal_conv1d_bwd_workspace_size(batch, seqlen, dim, width, io_dtype, device))


def _blocks(t, name, dtype, shape, index):
    """Checks a (batch, rows, dim) tensor whose rows and batch entries may be strided; returns
    (pointer, batch stride, row stride)."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or index < 0:
        _refuse(t, name, dtype, shape, index)
    batch, rows, dim = shape
    s0, s1, s2 = t.stride()
    if (s2 != 1 and dim != 1) or (rows > 1 and s1 < dim):
        raise ValueError(f"{name}: rows must be {dim} adjacent elements, got strides {(s0, s1, s2)}")
    if rows <= 1:  # sizes of one: strides without a meaning, which may be any
        s1 = dim
    return t.data_ptr(), s0 if batch > 1 else rows * s1, s1


def causal_conv1d_bwd(x, weight, bias=None, *, dout, silu=False, dx=None, workspace=None, stream=None):
    """Gradients of sum(dout * causal_conv1d_fwd(x, weight, bias, silu=silu)).

    x (batch, seqlen, dim) float32 or bfloat16, dense or strided in batch and time; dout (batch,
    seqlen, dim) float32 or x's dtype, contiguous.  Returns a dict of dx (x's dtype, or that of
    the given ``dx`` tensor: float32 or x's dtype, strided or not), dweight (dim, width) and,
    with a bias, dbias (dim), both float32."""
    torch = torch_()
    gpu = x.get_device()
    if x.ndim != 3:
        raise ValueError(f"x must be (batch, seqlen, dim), got shape {tuple(x.shape)}")
    batch, seqlen, dim = x.shape
    code = _code(x.dtype, "x")
    width = _two_d(weight, "weight")[1]
    if dout.dtype not in (torch.float32, x.dtype):
        raise ValueError(f"dout must be float32 or {x.dtype}, got {dout.dtype}")
    xp, xb, xr = _blocks(x, "x", x.dtype, (batch, seqlen, dim), gpu)
    wp = _dense(weight, "weight", torch.float32, (dim, width), gpu)
    bp = _dense(bias, "bias", torch.float32, (dim,), gpu)
    dp = _dense(dout, "dout", dout.dtype, (batch, seqlen, dim), gpu)
    if dx is None:
        dx = _new(x, (batch, seqlen, dim), x.dtype, stream)
        gp, gb, gr = dx.data_ptr(), seqlen * dim, dim
    else:
        if dx.dtype not in (torch.float32, x.dtype):
            raise ValueError(f"dx must be float32 or {x.dtype}, got {dx.dtype}")
        gp, gb, gr = _blocks(dx, "dx", dx.dtype, (batch, seqlen, dim), gpu)
    g = {"dx": dx, "dweight": _new(x, (dim, width), torch.float32, stream)}
    if bias is not None:
        g["dbias"] = _new(x, (dim,), torch.float32, stream)
    need = causal_conv1d_bwd_workspace_size(batch, seqlen, dim, width, code, gpu) if workspace is None else 0
    workspace, wsp, wsn = _scratch(workspace, need, x, stream)
    rc = _library(gpu).causal_conv1d_bwd(xp, xb, xr, wp, bp, dp, gp, gb, gr, g["dweight"].data_ptr(),
                                  g["dbias"].data_ptr() if bias is not None else 0, batch, seqlen, dim, width, code,
                                  _code(dout.dtype, "dout"), _code(dx.dtype, "dx"), int(bool(silu)), wsp, wsn,
                                  _stream(stream, gpu))
    if rc != 0:
        raise SSSError(rc, "causal_conv1d_bwd")
    if stream is not None:
        _keep(stream, gpu, workspace, *g.values())
    return g


def _scan_operands(x, delta, A, B, C, D, z, delta_bias):
    """The scan's operands, checked, as the leading arguments of the C calls."""
    torch = torch_()
    gpu = x.get_device()
    rows, dim = _two_d(x, "x")
    code = _code(x.dtype, "x")
    n = _two_d(A, "A")[1]
    bc = _code(B.dtype, "B")
    xp, xs = _rows(x, "x", x.dtype, rows, dim, gpu)
    dp, ds = _rows(delta, "delta", x.dtype, rows, dim, gpu)
    Ap = _dense(A, "A", torch.float32, (dim, n), gpu)
    Bp, bs = _rows(B, "B", B.dtype, rows, n, gpu)
    Cp, cs = _rows(C, "C", B.dtype, rows, n, gpu)
    zp, zs = _rows(z, "z", x.dtype, rows, dim, gpu) if z is not None else (0, 0)
    Dp = _dense(D, "D", torch.float32, (dim,), gpu)
    bp = _dense(delta_bias, "delta_bias", torch.float32, (dim,), gpu)
    return (xp, xs, dp, ds, Ap, Bp, bs, Cp, cs, Dp, zp, zs, bp), rows, dim, n, code, bc, gpu


def selective_scan_packed_fwd_workspace_size(tokens, dim, dstate, device=0) -> int:
    return int(load().selective_scan_packed_fwd_workspace_size(tokens, dim, dstate, device))


def selective_scan_packed_fwd(x, delta, A, B, C, D=None, z=None, *, cu_seqlens, state=None, state_indices=None,
                              has_initial=None, delta_bias=None, delta_softplus=False, out=None, workspace=None,
                              stream=None):
    """The selective scan over packed prompts: y (tokens, dim), float32 or ``out``'s dtype.

    x, delta, z (tokens, dim) float32 or bfloat16 (one dtype), B, C (tokens, dstate) float32 or
    bfloat16 (one dtype), rows may be strided; A (dim, dstate), D, delta_bias (dim) float32;
    cu_seqlens (nseq + 1) int32.  state (slots, dim, dstate) float32 keeps each sequence's last
    state (updated in place) in slot state_indices[s] (int32; None: slot s; -1: none);
    has_initial (nseq) bool marks the sequences that continue their slot.  Rows outside every
    sequence are left as they are in ``out``."""
    torch = torch_()
    ops, tokens, dim, n, code, bc, gpu = _scan_operands(x, delta, A, B, C, D, z, delta_bias)
    sp, slots = _cache(state, "state", torch.float32, (dim, n), gpu)
    nseq, cu, idx, ini = _sequences(cu_seqlens, state_indices, has_initial, state, slots, gpu)
    yd = torch.float32 if out is None else out.dtype
    yc = _code(yd, "out")
    y, yp = _out(out, "out", x, yd, (tokens, dim), gpu, stream)
    if tokens == 0:
        return y
    need = selective_scan_packed_fwd_workspace_size(tokens, dim, n, gpu) if workspace is None else 0
    workspace, wsp, wsn = _scratch(workspace, need, x, stream)
    rc = _library(gpu).selective_scan_packed_fwd(*ops, SSS_DELTA_SOFTPLUS if delta_softplus else 0, sp, cu, idx, ini, yp,
                                          tokens, nseq, slots, dim, n, code, bc, yc, wsp, wsn, _stream(stream, gpu))
    if rc != 0:
        raise SSSError(rc, "selective_scan_packed_fwd")
    if stream is not None:
        _keep(stream, gpu, workspace, y)
    return y


def selective_state_update_slots(x, delta, A, B, C, D=None, z=None, *, state, state_indices=None, delta_bias=None,
                                 delta_softplus=False, out=None, stream=None):
    """One decode step on cache slots: y (batch, dim), float32 or ``out``'s dtype.

    Operands as selective_scan_packed_fwd with one row per request; state (slots, dim, dstate)
    float32 updated in place, row b's in slot state_indices[b] (int32; None: slot b; -1: none, the
    row starts from zero and keeps nothing)."""
    torch = torch_()
    ops, batch, dim, n, code, bc, gpu = _scan_operands(x, delta, A, B, C, D, z, delta_bias)
    sp, slots = _cache(state, "state", torch.float32, (dim, n), gpu)
    idx = _dense(state_indices, "state_indices", torch.int32, (batch,), gpu)
    if state_indices is None and batch > slots:
        raise ValueError(f"{batch} rows need as many slots or state_indices, the cache has {slots}")
    yd = torch.float32 if out is None else out.dtype
    yc = _code(yd, "out")
    y, yp = _out(out, "out", x, yd, (batch, dim), gpu, stream)
    if batch == 0:
        return y
    rc = _library(gpu).selective_state_update_slots(*ops, SSS_DELTA_SOFTPLUS if delta_softplus else 0, sp, idx, yp, batch,
                                             slots, dim, n, code, bc, yc, _stream(stream, gpu))
    if rc != 0:
        raise SSSError(rc, "selective_state_update_slots")
    if stream is not None:
        _keep(stream, gpu, y)
    return y


def _group(dim, group_size):
    g = dim if group_size is None else int(group_size)
    if g < 1 or dim % g != 0:
        raise ValueError(f"group_size must divide {dim}, got {group_size}")
    return g


def rms_norm_gated_fwd(x, weight, z=None, *, eps=1e-5, group_size=None, norm_before_gate=False, out=None,
                       return_rstd=False, stream=None):
    """Norm after the scan, fused with the gate: rmsnorm(x * silu(z)) * weight, or
    rmsnorm(x) * weight * silu(z) with norm_before_gate; over groups of group_size channels.

    x (rows, dim) float32 or bfloat16 (the scan's output), z (rows, dim) float32 or bfloat16, rows
    may be strided; weight (dim) float32.  Returns out (rows, dim) in z's dtype (x's without z),
    and with return_rstd the (rows, groups) float32 factors that rms_norm_gated_bwd takes."""
    torch = torch_()
    gpu = x.get_device()
    rows, dim = _two_d(x, "x")
    xc = _code(x.dtype, "x")
    g = _group(dim, group_size)
    xp, xs = _rows(x, "x", x.dtype, rows, dim, gpu)
    od = z.dtype if z is not None else x.dtype
    oc = _code(od, "z")
    zp, zs = _rows(z, "z", od, rows, dim, gpu) if z is not None else (0, 0)
    wp = _dense(weight, "weight", torch.float32, (dim,), gpu)
    o, op = _out(out, "out", x, od, (rows, dim), gpu, stream)
    rstd = _new(x, (rows, dim // g), torch.float32, stream) if return_rstd else None
    if rows > 0:
        rc = _library(gpu).rms_norm_gated_fwd(xp, xs, wp, zp, zs, op, rstd.data_ptr() if return_rstd else 0, rows, dim, g,
                                       float(eps), SSS_NORM_BEFORE_GATE if norm_before_gate else 0, xc, oc,
                                       _stream(stream, gpu))
        if rc != 0:
            raise SSSError(rc, "rms_norm_gated_fwd")
        if stream is not None:
            _keep(stream, gpu, o, rstd)
    return (o, rstd) if return_rstd else o


def rms_norm_gated_bwd_workspace_size(rows, dim, group_size=None, device=0) -> int:
    return int(load().rms_norm_gated_bwd_workspace_size(rows, dim, _group(dim, group_size), device))


def rms_norm_gated_bwd(dout, x, weight, z=None, *, rstd, group_size=None, norm_before_gate=False, dz=None,
                       workspace=None, stream=None):
    """Gradients of sum(dout * rms_norm_gated_fwd(...)): a dict of dx (x's dtype), dz (z's dtype,
    with z; into the given ``dz``, strided or not) and dweight float32.  dout (rows, dim) in the
    forward output's dtype, contiguous; rstd as the forward returned it."""
    torch = torch_()
    gpu = x.get_device()
    rows, dim = _two_d(x, "x")
    xc = _code(x.dtype, "x")
    g = _group(dim, group_size)
    od = z.dtype if z is not None else x.dtype
    oc = _code(od, "z")
    dp = _dense(dout, "dout", od, (rows, dim), gpu)
    xp, xs = _rows(x, "x", x.dtype, rows, dim, gpu)
    zp, zs = _rows(z, "z", od, rows, dim, gpu) if z is not None else (0, 0)
    wp = _dense(weight, "weight", torch.float32, (dim,), gpu)
    rp = _dense(rstd, "rstd", torch.float32, (rows, dim // g), gpu)
    res = {"dx": _new(x, (rows, dim), x.dtype, stream), "dweight": _new(x, (dim,), torch.float32, stream)}
    gp, gs = 0, 0
    if z is not None:
        if dz is None:
            res["dz"] = _new(x, (rows, dim), od, stream)
            gp, gs = res["dz"].data_ptr(), dim
        else:
            res["dz"] = dz
            gp, gs = _rows(dz, "dz", od, rows, dim, gpu)
    need = rms_norm_gated_bwd_workspace_size(rows, dim, g, gpu) if workspace is None else 0
    workspace, wsp, wsn = _scratch(workspace, need, x, stream)
    rc = _library(gpu).rms_norm_gated_bwd(dp, xp, xs, wp, zp, zs, rp, res["dx"].data_ptr(), gp, gs, res["dweight"].data_ptr(),
                                   rows, dim, g, SSS_NORM_BEFORE_GATE if norm_before_gate else 0, xc, oc, wsp, wsn,
                                   _stream(stream, gpu))
    if rc != 0:
        raise SSSError(rc, "rms_norm_gated_bwd")
    if stream is not None:
        _keep(stream, gpu, workspace, *res.values())
    return res


def rms_norm_residual_fwd(x, weight, residual=None, *, post_weight=None, scale=None, alpha=1.0, eps=1e-5, out=None,
                          residual_out=None, return_rstd=False, stream=None):
    """Between two blocks: residual_out = residual + alpha * scale * v with v = x, or
    rmsnorm(x) * post_weight, and out = rmsnorm(residual_out) * weight.

    x (rows, dim) float32 or bfloat16, residual (rows, dim) float32 or bfloat16, rows may be
    strided; weight, post_weight, scale (dim) float32.  Returns (out in x's dtype, residual_out in
    the residual's dtype, float32 without one), and with return_rstd also the (rows,) float32
    factors rstd and rstd_post (None without post_weight).  residual_out may be the residual."""
    torch = torch_()
    gpu = x.get_device()
    rows, dim = _two_d(x, "x")
    xc = _code(x.dtype, "x")
    hd = (residual.dtype if residual is not None else residual_out.dtype if residual_out is not None
          else torch.float32)
    hc = _code(hd, "residual")
    xp, xs = _rows(x, "x", x.dtype, rows, dim, gpu)
    hp, hs = _rows(residual, "residual", hd, rows, dim, gpu) if residual is not None else (0, 0)
    wp = _dense(weight, "weight", torch.float32, (dim,), gpu)
    pp = _dense(post_weight, "post_weight", torch.float32, (dim,), gpu)
    sp = _dense(scale, "scale", torch.float32, (dim,), gpu)
    o, op = _out(out, "out", x, x.dtype, (rows, dim), gpu, stream)
    h, ho = _out(residual_out, "residual_out", x, hd, (rows, dim), gpu, stream)
    rstd = rstd_post = None
    if return_rstd:
        rstd = _new(x, (rows,), torch.float32, stream)
        rstd_post = _new(x, (rows,), torch.float32, stream) if post_weight is not None else None
    if rows > 0:
        rc = _library(gpu).rms_norm_residual_fwd(xp, xs, hp, hs, pp, sp, wp, op, ho,
                                          0 if rstd_post is None else rstd_post.data_ptr(),
                                          0 if rstd is None else rstd.data_ptr(), rows, dim, float(alpha), float(eps),
                                          xc, hc, _stream(stream, gpu))
        if rc != 0:
            raise SSSError(rc, "rms_norm_residual_fwd")
        if stream is not None:
            _keep(stream, gpu, o, h, rstd, rstd_post)
    return (o, h, rstd, rstd_post) if return_rstd else (o, h)


def rms_norm_residual_bwd_workspace_size(rows, dim, device=0) -> int:
    return int(load().rms_norm_residual_bwd_workspace_size(rows, dim, device))


def rms_norm_residual_bwd(dout, dresidual_out=None, *, residual_out, weight, rstd, x=None, post_weight=None, scale=None,
                          rstd_post=None, alpha=1.0, want_dresidual=True, workspace=None, stream=None):
    """Gradients of sum(dout * out) + sum(dresidual_out * residual_out) of rms_norm_residual_fwd.

    dout (rows, dim) in x's dtype and dresidual_out (or None) and residual_out in the residual's,
    contiguous; rstd, rstd_post as the forward returned them; x is needed with post_weight or
    scale.  Returns a dict of dx (x's dtype), dresidual (the residual's, unless not wanted),
    dweight, and dpost_weight / dscale with post_weight / scale, float32."""
    torch = torch_()
    gpu = dout.get_device()
    rows, dim = _two_d(dout, "dout")
    xd, hd = dout.dtype, residual_out.dtype
    xc, hc = _code(xd, "dout"), _code(hd, "residual_out")
    if x is None and (post_weight is not None or scale is not None):
        raise ValueError("x is needed for the gradients through post_weight or scale")
    if post_weight is not None and rstd_post is None:
        raise ValueError("rstd_post is needed with post_weight")
    dp = _dense(dout, "dout", xd, (rows, dim), gpu)
    ep = _dense(dresidual_out, "dresidual_out", hd, (rows, dim), gpu)
    hp = _dense(residual_out, "residual_out", hd, (rows, dim), gpu)
    xp, xs = _rows(x, "x", xd, rows, dim, gpu) if x is not None else (0, 0)
    wp = _dense(weight, "weight", torch.float32, (dim,), gpu)
    pp = _dense(post_weight, "post_weight", torch.float32, (dim,), gpu)
    sp = _dense(scale, "scale", torch.float32, (dim,), gpu)
    rp = _dense(rstd, "rstd", torch.float32, (rows,), gpu)
    rpp = _dense(rstd_post, "rstd_post", torch.float32, (rows,), gpu) if post_weight is not None else 0
    vec = lambda: _new(dout, (dim,), torch.float32, stream)
    res = {"dx": _new(dout, (rows, dim), dout.dtype, stream), "dweight": vec()}
    if want_dresidual:
        res["dresidual"] = _new(dout, (rows, dim), hd, stream)
    if post_weight is not None:
        res["dpost_weight"] = vec()
    if scale is not None:
        res["dscale"] = vec()
    ptr = lambda k: res[k].data_ptr() if k in res else 0
    need = rms_norm_residual_bwd_workspace_size(rows, dim, gpu) if workspace is None else 0
    workspace, wsp, wsn = _scratch(workspace, need, dout, stream)
    rc = _library(gpu).rms_norm_residual_bwd(dp, ep, xp, xs, hp, pp, sp, wp, rpp, rp, ptr("dx"), ptr("dresidual"),
                                      ptr("dweight"), ptr("dpost_weight"), ptr("dscale"), rows, dim, float(alpha), xc,
                                      hc, wsp, wsn, _stream(stream, gpu))
    if rc != 0:
        raise SSSError(rc, "rms_norm_residual_bwd")
    if stream is not None:
        _keep(stream, gpu, workspace, *res.values())
    return res
