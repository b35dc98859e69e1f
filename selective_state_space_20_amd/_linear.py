"""Binding of linear attention with a decay for each head: packed prompts, single tokens on cache
slots, and gradients.  As in ``_block``, only argument checks, output allocation and the C call.

``stream`` is the handle of the HIP stream that a call's work is queued on, as in ``_block``."""
from __future__ import annotations

from ._block import _cache, _code, _dense, _keep, _library, _new, _out, _refuse, _rows, _scratch, _sequences, _stream, torch_
from ._lib import SSSError, load


def _three_d(t, name):
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must be (tokens, heads, head size), got shape {tuple(shape)}")
    return shape


# Each attribute of a tensor is asked for once: the step on small batches is as long as its call.
def _heads(t, name, shape, dtype, rows, heads, dim, index):
    """Checks a (rows, heads, dim) tensor, tokens and heads of any stride; returns (pointer, strides, heads)."""
    r, n, d = shape
    if n < 1 or heads % n != 0:
        raise ValueError(f"{name}: its {n} heads must divide the call's {heads}")
    if r != rows or d != dim or t.dtype is not dtype or t.get_device() != index or index < 0:
        _refuse(t, name, dtype, (rows, n, dim), index)
    st, sh, s1 = t.stride()
    if s1 != 1 and dim != 1:
        raise ValueError(f"{name}: a head must be {dim} adjacent elements, got strides {(st, sh, s1)}")
    # sizes of one: strides without a meaning, which may be any
    return t.data_ptr(), st if rows > 1 else 0, sh if n > 1 else 0, n


def _operands(q, k, v, log_decay, beta, D, scale):
    """The checked operands as the leading arguments of the C calls, and the sizes."""
    torch = torch_()
    f32, gpu, dtype = torch.float32, v.get_device(), v.dtype
    of_v = _three_d(v, "v")
    rows, heads, dv = of_v
    code = _code(dtype, "v")
    if heads < 1 or dv < 1:
        raise ValueError(f"v must have heads and elements, got shape {tuple(of_v)}")
    of_q = _three_d(q, "q")
    dk = of_q[2]
    qp = _heads(q, "q", of_q, dtype, rows, heads, dk, gpu)
    kp = _heads(k, "k", _three_d(k, "k"), dtype, rows, heads, dk, gpu)
    vp = _heads(v, "v", of_v, dtype, rows, heads, dv, gpu)[:3]
    if log_decay.ndim == 1:  # one for each head
        gp, gs = _dense(log_decay, "log_decay", f32, (heads,), gpu), 0
    else:
        gp, gs = _rows(log_decay, "log_decay", f32, rows, heads, gpu)
    bp, bs = _rows(beta, "beta", f32, rows, heads, gpu) if beta is not None else (0, 0)
    Dp = _dense(D, "D", f32, (heads,), gpu)
    return (*qp, *kp, *vp, gp, gs, bp, bs, Dp, float(scale)), rows, heads, qp[3], kp[3], dk, dv, code, gpu


def linear_attention_packed_fwd_workspace_size(tokens, heads, dk, dv, device=0) -> int:
    return int(load().linear_attention_packed_fwd_workspace_size(tokens, heads, dk, dv, device))


def linear_attention_packed_fwd(q, k, v, log_decay, *, cu_seqlens, beta=None, D=None, scale=1.0, state=None,
                                state_indices=None, has_initial=None, out=None, workspace=None, stream=None):
    """Linear attention over packed prompts: out (tokens, heads, dv) in v's dtype, with
    S_t = exp(log_decay_t) S_(t-1) + beta_t k_t v_t^T and out_t = scale q_t S_t + D v_t.

    q, k (tokens, heads or a divisor of them, dk) and v (tokens, heads, dv) float32 or bfloat16 (one
    dtype), tokens and heads may be strided; log_decay (tokens, heads), rows may be strided, or (heads)
    float32; beta (tokens, heads), D (heads) float32; dk, dv up to 256; cu_seqlens (nseq + 1) int32.
    state (slots, heads, dk, dv) float32 keeps each sequence's last state (updated in place) in slot
    state_indices[s] (int32; None: slot s; -1: none); has_initial (nseq) bool marks the sequences that
    continue their slot.  Rows outside every sequence are left as they are in ``out``."""
    torch = torch_()
    ops, tokens, heads, _, _, dk, dv, code, gpu = _operands(q, k, v, log_decay, beta, D, scale)
    sp, slots = _cache(state, "state", torch.float32, (heads, dk, dv), gpu)
    nseq, cu, idx, ini = _sequences(cu_seqlens, state_indices, has_initial, state, slots, gpu)
    o, op = _out(out, "out", v, v.dtype, (tokens, heads, dv), gpu, stream)
    if tokens == 0:
        return o
    need = linear_attention_packed_fwd_workspace_size(tokens, heads, dk, dv, gpu) if workspace is None else 0
    workspace, wsp, wsn = _scratch(workspace, need, v, stream)
    rc = _library(gpu).linear_attention_packed_fwd(*ops, sp, cu, idx, ini, op, tokens, nseq, slots, heads, dk, dv, code, wsp,
                                                   wsn, _stream(stream, gpu))
    if rc != 0:
        raise SSSError(rc, "linear_attention_packed_fwd")
    if stream is not None:
        _keep(stream, gpu, workspace, o)
    return o


def linear_attention_update_slots(q, k, v, log_decay, *, state, beta=None, D=None, scale=1.0, state_indices=None, out=None,
                                  stream=None):
    """One token of each row on cache slots: out (batch, heads, dv) in v's dtype.

    Operands as linear_attention_packed_fwd with one row per request; state (slots, heads, dk, dv)
    float32 updated in place, row b's in slot state_indices[b] (int32; None: slot b; -1: none, the
    row starts from zero and keeps nothing)."""
    torch = torch_()
    ops, batch, heads, _, _, dk, dv, code, gpu = _operands(q, k, v, log_decay, beta, D, scale)
    sp, slots = _cache(state, "state", torch.float32, (heads, dk, dv), gpu)
    idx = _dense(state_indices, "state_indices", torch.int32, (batch,), gpu)
    if state_indices is None and batch > slots:
        raise ValueError(f"{batch} rows need as many slots or state_indices, the cache has {slots}")
    o, op = _out(out, "out", v, v.dtype, (batch, heads, dv), gpu, stream)
    if batch == 0:
        return o
    rc = _library(gpu).linear_attention_update_slots(*ops, sp, idx, op, batch, slots, heads, dk, dv, code,
                                                     _stream(stream, gpu))
    if rc != 0:
        raise SSSError(rc, "linear_attention_update_slots")
    if stream is not None:
        _keep(stream, gpu, o)
    return o


def linear_attention_packed_bwd_workspace_size(tokens, nseq, heads, q_heads, k_heads, dk, dv, device=0) -> int:
    return int(load().linear_attention_packed_bwd_workspace_size(tokens, nseq, heads, q_heads, k_heads, dk, dv, device))


def linear_attention_packed_bwd(q, k, v, log_decay, *, dout, cu_seqlens, beta=None, D=None, scale=1.0, initial_state=None,
                                dfinal_state=None, want_dinitial=None, workspace=None, stream=None):
    """Gradients of sum(dout * out) + sum(dfinal_state * last states) of linear_attention_packed_fwd, each
    sequence starting from initial_state[s] (nseq, heads, dk, dv) float32 (None: zero).

    dout (tokens, heads, dv) in v's dtype, contiguous; dfinal_state like initial_state, or None.  Returns a
    dict of dq, dk, dv (in their dtype), dlog_decay (log_decay's shape), dbeta with beta, dD with D, and
    dinitial_state (with initial_state, unless want_dinitial says otherwise), float32.  Tokens outside
    every sequence get zero."""
    torch = torch_()
    ops, tokens, heads, qh, kh, dk, dv, code, gpu = _operands(q, k, v, log_decay, beta, D, scale)
    nseq, cu, _, _ = _sequences(cu_seqlens, None, None, None, 0, gpu)
    op = _dense(dout, "dout", v.dtype, (tokens, heads, dv), gpu)
    shape = (nseq, heads, dk, dv)
    ip = _dense(initial_state, "initial_state", torch.float32, shape, gpu)
    fp = _dense(dfinal_state, "dfinal_state", torch.float32, shape, gpu)
    f32 = torch.float32
    g = {"dq": _new(v, (tokens, qh, dk), v.dtype, stream), "dk": _new(v, (tokens, kh, dk), v.dtype, stream),
         "dv": _new(v, (tokens, heads, dv), v.dtype, stream), "dlog_decay": _new(v, log_decay.shape, f32, stream)}
    if beta is not None:
        g["dbeta"] = _new(v, (tokens, heads), f32, stream)
    if D is not None:
        g["dD"] = _new(v, (heads,), f32, stream)
    if want_dinitial if want_dinitial is not None else initial_state is not None:
        g["dinitial_state"] = _new(v, shape, f32, stream)
    ptr = lambda n: g[n].data_ptr() if n in g else 0
    need = (linear_attention_packed_bwd_workspace_size(tokens, nseq, heads, qh, kh, dk, dv, gpu) if workspace is None else 0)
    workspace, wsp, wsn = _scratch(workspace, need, v, stream)
    rc = _library(gpu).linear_attention_packed_bwd(*ops, op, cu, ip, fp, ptr("dq"), ptr("dk"), ptr("dv"), ptr("dlog_decay"),
                                                   ptr("dbeta"), ptr("dD"), ptr("dinitial_state"), tokens, nseq, heads, dk, dv,
                                                   code, wsp, wsn, _stream(stream, gpu))
    if rc != 0:
        raise SSSError(rc, "linear_attention_packed_bwd")
    if stream is not None:
        _keep(stream, gpu, workspace, *g.values())
    return g
