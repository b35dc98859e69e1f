"""How large the calls of linear attention may be: sizes whose bytes pass 64 bits are refused before any device work (CPU: fake
addresses, never met), and the step's launch is counted in the threads that it has."""
import pytest

from .test_linear_attention_refusals import BAD_DIM, P, attention, grads, step


def test_a_step_of_too_many_workgroups_is_refused():
    for batch, heads in ((1 << 24, 1), (1 << 18, 64)):  # 2^32 threads
        assert step(batch=batch, heads=heads, q_heads=1, k_heads=1, slots=1, idx=6 * P + (P >> 1), dk=1, dv=1, gs=heads, bs=heads,
                    vs=heads) == BAD_DIM


HUGE = dict(heads=1 << 16, q_heads=1, k_heads=1, gs=1 << 16, bs=1 << 16, vs=1 << 24, dk=256, dv=256, vh=256)


@pytest.mark.parametrize("call, count", [(attention, "slots"), (step, "slots"), (grads, "nseq")])
def test_states_of_more_bytes_than_64_bits_count(call, count):
    for n in (1 << 28, 1 << 29, 1 << 30):  # 2^62, 2^63 and 2^64 bytes
        assert call(**HUGE, **{count: n}) == BAD_DIM, n


@pytest.mark.gpu
def test_a_step_below_the_bound():
    """A batch of which nearly all rows are padding: between 2^31 and 2^32 threads."""
    import torch
    import selective_state_space_20_amd as sss
    batch, heads, dk, dv = 1 << 17, 80, 4, 4
    gen = torch.Generator(device="cuda:0").manual_seed(1)
    r = lambda *s: torch.randn(*s, device="cuda:0", generator=gen)
    q, k, v, g = r(batch, 1, dk), r(batch, 1, dk), r(batch, heads, dv), -r(batch, heads).abs()
    state = r(2, heads, dk, dv)
    idx = torch.full((batch,), -1, dtype=torch.int32, device="cuda:0")
    idx[0], idx[-1] = 0, 1
    few, kept = [0, batch // 2, batch - 1], state.clone()
    want = sss.linear_attention_update_slots(q[few], k[few], v[few], g[few], state=kept, state_indices=idx[few])
    out = sss.linear_attention_update_slots(q, k, v, g, state=state, state_indices=idx)
    assert torch.equal(out[few], want) and torch.equal(state, kept)
