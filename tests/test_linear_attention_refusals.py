"""What linear attention and the layer norm refuse, before any device work (CPU only): the C calls on fake addresses,
and the binding on CPU tensors; where the binding's memory comes from and on what stream and GPU the calls run."""
import pytest
import torch

import selective_state_space_20_amd as sss
from selective_state_space_20_amd import _linear, load

from . import test_stream_memory as sm
from .test_stream_memory import gpu  # noqa: F401

NULL_ARG, BAD_DIM, UNSUPPORTED, WORKSPACE, ALIAS, HIP = -1, -2, -3, -4, -5, -6
P = 1 << 40  # fake addresses, far apart; never dereferenced


def call(fn, defaults, kw):
    a = dict(defaults)
    assert set(kw) <= set(a), set(kw) - set(a)
    a.update(kw)
    return getattr(load(), fn)(*a.values())


HEADS = dict(q=P, qs=64, qh=16, q_heads=4, k=2 * P, ks=32, kh=16, k_heads=2, v=3 * P, vs=128, vh=32, g=4 * P, gs=4, beta=5 * P,
             bs=4, D=6 * P, scale=1.0)
SIZES = dict(heads=4, dk=16, dv=32, io_dtype=1)


def attention(**kw):
    return call("linear_attention_packed_fwd", dict(
        HEADS, state=7 * P, cu=8 * P, idx=0, initial=0, out=9 * P, tokens=100, nseq=2, slots=2, **SIZES, workspace=10 * P,
        workspace_bytes=1 << 30, stream=0), kw)


def step(**kw):
    return call("linear_attention_update_slots", dict(HEADS, state=7 * P, idx=0, out=9 * P, batch=2, slots=2, **SIZES, stream=0), kw)


def grads(**kw):
    return call("linear_attention_packed_bwd", dict(
        HEADS, dout=7 * P, cu=8 * P, initial=9 * P, dfinal=10 * P, dq=11 * P, dk_out=12 * P, dv_out=13 * P, dg=14 * P, dbeta=15 * P,
        dD=16 * P, dinitial=17 * P, tokens=100, nseq=2, **SIZES, workspace=18 * P, workspace_bytes=1 << 30, stream=0), kw)


@pytest.mark.parametrize("fn, extra", [(attention, ("cu", "out")), (step, ("state", "out")),
                                       (grads, ("dout", "cu", "dq", "dk_out", "dv_out", "dg", "dbeta", "dD"))])
def test_operands(fn, extra):
    for k in ("q", "k", "v", "g", *extra):
        assert fn(**{k: 0}) == NULL_ARG, k
    rows = "batch" if fn is step else "tokens"
    for kw in ({rows: -1}, {rows: (1 << 30) + 1}, {"heads": 0}, {"heads": 1 << 17, "q_heads": 1, "k_heads": 1}, {"q_heads": 3},
               {"k_heads": 0}, {"dk": 0}, {"dv": 0}, {"qs": -1}, {"kh": -1}, {"vs": (1 << 24) + 1}, {"qh": (1 << 40) + 1},
               {"gs": 3}, {"bs": 3}, {"bs": 0}):
        assert fn(**kw) == BAD_DIM, kw
    assert fn(dk=257) == UNSUPPORTED and fn(dv=257) == UNSUPPORTED and fn(io_dtype=2) == UNSUPPORTED
    for k in ("q", "v"):
        assert fn(**{k: HEADS[k] + 1}) == UNSUPPORTED, k  # bf16 at an odd address
    for k in ("g", "beta", "D"):
        assert fn(**{k: HEADS[k] + 2}) == UNSUPPORTED, k


def test_attention():
    assert attention(state=8 * P) == ALIAS and attention(out=P) == ALIAS and attention(out=7 * P) == ALIAS
    assert attention(out=3 * P + 64) == ALIAS and attention(out=4 * P) == ALIAS
    assert attention(nseq=3) == BAD_DIM and attention(slots=0) == BAD_DIM and attention(nseq=-1) == BAD_DIM
    assert attention(workspace=10 * P + 8) == UNSUPPORTED
    assert attention(tokens=0) == 0 and attention(nseq=0) == 0


def test_step():
    assert step(out=7 * P) == ALIAS and step(state=P) == ALIAS
    assert step(slots=1) == BAD_DIM and step(batch=3) == BAD_DIM
    assert step(batch=1 << 29, slots=1 << 29, idx=11 * P) in (BAD_DIM, ALIAS)  # more threads than a launch has
    assert step(batch=0) == 0


def test_gradients():
    for a, b in (("dq", 11), ("dk_out", 12), ("dv_out", 13), ("dg", 14), ("dbeta", 15), ("dD", 16), ("dinitial", 17)):
        for other in (1, 4, 7, 9, 10, 18 if a == "dq" else 3):
            if other == 18:
                continue
            assert grads(**{a: other * P}) == ALIAS, (a, other)
    assert grads(dq=12 * P) == ALIAS
    assert grads(workspace=18 * P + 4) == UNSUPPORTED


def test_workspace_sizes():
    assert sss.linear_attention_packed_fwd_workspace_size(10, 4, 300, 16) == 0
    assert sss.linear_attention_packed_bwd_workspace_size(10, 1, 4, 3, 4, 16, 16) == 0
    shared = sss.linear_attention_packed_bwd_workspace_size(1000, 1, 8, 1, 8, 64, 64)
    apart = sss.linear_attention_packed_bwd_workspace_size(1000, 1, 8, 8, 8, 64, 64)
    assert shared - apart == 1000 * 8 * 64 * 4  # one row of fp32 parts for each head


def norm(**kw):
    return call("layer_norm_fwd", dict(x=P, xs=8, res=2 * P, rs=8, w=3 * P, b=4 * P, out=5 * P, res_out=6 * P, mean=7 * P, rstd=8 * P,
                                       rows=4, dim=8, group=8, eps=1e-5, io=1, rd=0, stream=0), kw)


def norm_grads(**kw):
    return call("layer_norm_bwd", dict(dout=P, dres_out=2 * P, x=3 * P, xs=8, w=4 * P, mean=5 * P, rstd=6 * P, dx=7 * P, dres=8 * P,
                                       dw=9 * P, db=10 * P, rows=4, dim=8, group=8, io=1, xd=0, ws=11 * P, wsn=1 << 20, stream=0), kw)


def test_layer_norm():
    assert norm(x=0) == NULL_ARG and norm(out=0) == NULL_ARG
    assert norm(dim=0) == BAD_DIM and norm(group=3) == BAD_DIM and norm(rows=-1) == BAD_DIM and norm(xs=7) == BAD_DIM
    assert norm(rs=7) == BAD_DIM and norm(io=2) == UNSUPPORTED and norm(rd=3) == UNSUPPORTED
    assert norm(dim=40000, group=40000, xs=40000, rs=40000) == UNSUPPORTED
    assert norm(x=P + 1) == UNSUPPORTED and norm(res=2 * P + 2) == UNSUPPORTED
    assert norm(out=P) == ALIAS and norm(res_out=P) == ALIAS and norm(mean=8 * P) == ALIAS and norm(out=2 * P) == ALIAS
    assert norm(res=6 * P, rs=9) == ALIAS      # in place, but not the same rows
    assert norm(rows=0) == 0 and norm(rows=0, res=0, res_out=0, w=0, b=0, mean=0, rstd=0, rd=9) == 0


def test_layer_norm_gradients():
    for k in ("dout", "x", "mean", "rstd", "dx", "dw"):
        assert norm_grads(**{k: 0}) == NULL_ARG, k
    assert norm_grads(group=5) == BAD_DIM and norm_grads(xs=7) == BAD_DIM
    assert norm_grads(io=7) == UNSUPPORTED and norm_grads(ws=11 * P + 4) == UNSUPPORTED
    assert norm_grads(dx=P) == ALIAS and norm_grads(dres=2 * P) == ALIAS and norm_grads(dw=10 * P) == ALIAS


def test_binding_on_cpu_tensors():
    t = lambda *s: torch.zeros(*s)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        sss.linear_attention_packed_fwd(t(4, 2, 8), t(4, 2, 8), t(4, 2, 8), t(4, 2), cu_seqlens=cu)
    with pytest.raises(ValueError, match="GPU"):
        sss.layer_norm_fwd(t(4, 8), t(8))
    with pytest.raises(ValueError, match="heads"):
        sss.linear_attention_packed_fwd(t(4, 3, 8), t(4, 2, 8), t(4, 2, 8), t(4, 2), cu_seqlens=cu)
    with pytest.raises(ValueError, match="v must be"):
        sss.linear_attention_packed_fwd(t(4, 2, 8), t(4, 2, 8), t(4, 16), t(4, 2), cu_seqlens=cu)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        sss.linear_attention_packed_fwd(t(4, 2, 8), t(4, 2, 8), t(4, 2, 8).half(), t(4, 2), cu_seqlens=cu)
    with pytest.raises(ValueError, match="divide"):
        sss.layer_norm_fwd(t(4, 8), t(8), group_size=3)


def calls(t):
    x, w, cu = t((6, 8)), t((8,)), t((3,), sm.I32)
    q, v, g, state = t((6, 2, 4)), t((6, 2, 8)), t((6, 2)), t((6, 2, 4, 8))
    start = t((2, 2, 4, 8))
    return {
        "attention": lambda **k: sss.linear_attention_packed_fwd(q, q, v, g, cu_seqlens=cu, beta=g, state=state, **k),
        "attention step": lambda **k: sss.linear_attention_update_slots(q, q, v, g, state=state, **k),
        "attention gradients": lambda **k: sss.linear_attention_packed_bwd(
            q, q, v, g, dout=v, cu_seqlens=cu, beta=g, D=t((2,)), initial_state=start, dfinal_state=start, **k),
        "layer norm": lambda **k: sss.layer_norm_fwd(x, w, w, x, return_stats=True, **k),
        "layer norm gradients": lambda **k: sss.layer_norm_bwd(x, x, w, mean=t((6, 1)), rstd=t((6, 1)), bias=True, dresidual_out=x,
                                                               **k),
    }


MADE = {"attention": 2, "attention step": 1, "attention gradients": 8, "layer norm": 4, "layer norm gradients": 5}


@pytest.fixture
def stand_in(gpu, monkeypatch):  # noqa: F811
    def make(*a):
        g, lib = gpu(*a)
        monkeypatch.setattr(_linear, "load", lambda: lib)
        monkeypatch.setattr(_linear, "torch_", lambda: sm._block._torch)
        return g, lib
    return make


@pytest.mark.parametrize("name", list(MADE))
@pytest.mark.parametrize("current, given", [(0, 7), (5, 7), (5, 0), (0, None), (5, None), (5, 5)])
def test_memory_of_the_stream(stand_in, name, current, given):
    g, lib = stand_in(current)
    res = calls(g.tensor)[name](stream=given)
    runs_on = current if given is None else given
    assert lib.streams == [runs_on] and len(g.made) == MADE[name] and [t.stream for t in g.made] == [runs_on] * len(g.made)
    if runs_on != current:
        for t in res.values() if isinstance(res, dict) else res if isinstance(res, tuple) else [res]:
            assert current in t.recorded
    assert g.now == [current]


@pytest.mark.parametrize("name", list(MADE))
def test_the_operands_gpu_is_current(stand_in, name):
    g, lib = stand_in(0, 1, 0)
    calls(g.tensor)[name]()
    assert lib.devices == [1] and g.devices == [0]
