"""Linear attention's gradients over as many tokens as memory holds: no size that the header allows is refused, and
elements past 2^30 and 2^32 are where they belong."""
import pytest

from .test_linear_attention_gpu import DEV, i32
from .test_linear_attention_refusals import P, WORKSPACE, grads

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shared", [False, True])
def test_no_size_is_refused(shared):
    """Fake addresses, never met: the sizes are looked at before the workspace, which is not given."""
    heads, dk, dv = 32, 128, 128
    qk = 1 if shared else heads
    row = dict(qs=qk * dk, qh=dk, q_heads=qk, ks=qk * dk, kh=dk, k_heads=qk, vs=heads * dv, vh=dv, gs=heads, bs=heads, heads=heads,
               dk=dk, dv=dv, workspace=0, workspace_bytes=0)
    assert grads(tokens=1 << 20, **row) == WORKSPACE  # 2^32 elements of q for each head
    assert grads(tokens=1 << 22, **row) == WORKSPACE
    assert grads(tokens=1 << 10, nseq=1 << 24, **dict(row, heads=1, q_heads=1, k_heads=1, dk=1, dv=1)) == WORKSPACE


def test_sums_over_shared_heads_past_32_bits():
    import torch
    import selective_state_space_20_amd as sss
    heads, qh, dk, tokens, n = 64, 32, 256, (1 << 18) + 77, 150  # dq 2^31 elements, of each head 2^32
    gen = torch.Generator(device=DEV).manual_seed(1)
    r = lambda *s: torch.randn(*s, device=DEV, generator=gen)
    few = {"q": r(n, qh, dk).bfloat16(), "k": r(n, 1, dk).bfloat16(), "v": r(n, heads, 1).bfloat16(), "log_decay": -r(n, heads).abs() * 0.1}
    dout = r(n, heads, 1).bfloat16()
    alone = sss.linear_attention_packed_bwd(*few.values(), dout=dout, cu_seqlens=i32([0, n]))
    at = tokens - n  # the same tokens at the end of many that no sequence has
    many = {}
    for name, x in few.items():
        many[name] = torch.zeros(tokens, *x.shape[1:], dtype=x.dtype, device=DEV)
        many[name][at:] = x
    wide = torch.zeros(tokens, heads, 1, dtype=torch.bfloat16, device=DEV)
    wide[at:] = dout
    got = sss.linear_attention_packed_bwd(*many.values(), dout=wide, cu_seqlens=i32([at, tokens]))
    for name, x in alone.items():
        # two roundings of the same value (in other segments), each within half a step of it
        rel = float((got[name][at:].double() - x.double()).norm() / x.double().norm())
        assert rel <= 2 * 2.0 ** -8 / 3 ** 0.5, (name, rel)
        assert not bool(got[name][:at].any()), name


def test_more_sequences_than_a_launch_has_workgroups():
    """The gradients of states of sequences without tokens are those of the last states."""
    import torch
    import selective_state_space_20_amd as sss
    nseq, t = (1 << 23) + 5, 40
    r = lambda *s: torch.randn(*s, device=DEV)
    cu = torch.full((nseq + 1,), t, dtype=torch.int32, device=DEV)
    cu[0] = 0
    dfinal = r(nseq, 1, 2, 3)
    got = sss.linear_attention_packed_bwd(r(t, 1, 2), r(t, 1, 2), r(t, 1, 3), -r(t, 1).abs(), dout=r(t, 1, 3), cu_seqlens=cu,
                                          dfinal_state=dfinal, want_dinitial=True)
    assert torch.equal(got["dinitial_state"][1:], dfinal[1:])
    assert bool(got["dinitial_state"][0].isfinite().all()) and not torch.equal(got["dinitial_state"][0], dfinal[0])
