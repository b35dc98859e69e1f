"""Strides of sizes of one have no meaning and may be any: one token of a long buffer's rows, one batch
entry.  On the CPU with stand-ins for the tensors and the library (the strides that reach it); on the GPU
the results."""
import pytest

import selective_state_space_20_amd as sss

from .test_stream_memory import F32, I32, gpu  # noqa: F401  (fixture)

FAR = 1 << 40  # no row stride that the library takes


def with_strides(t, strides):
    t.stride = lambda: strides
    return t


@pytest.mark.parametrize("far", [FAR, 0, 3])
def test_one_row_of_a_long_buffer(gpu, far):  # noqa: F811
    g, lib = gpu(0)
    t = g.tensor
    row = lambda n: with_strides(t((1, n)), (far, 1))
    A, m, v = t((8, 2)), lambda: row(2), t((8,))
    state = t((3, 8, 2))
    sss.causal_conv1d_update(row(8), t((8, 4)), conv_state=t((3, 3, 8)))
    sss.causal_conv1d_packed_fwd(row(8), t((8, 4)), cu_seqlens=t((2,), I32))
    sss.selective_state_update_slots(row(8), row(8), A, m(), m(), z=row(8), state=state)
    sss.selective_scan_packed_fwd(row(8), row(8), A, m(), m(), z=row(8), cu_seqlens=t((2,), I32))
    sss.rms_norm_gated_fwd(row(8), v, row(8))
    sss.rms_norm_gated_bwd(row(8), row(8), v, row(8), rstd=t((1, 1)), dz=row(8))
    sss.rms_norm_residual_fwd(row(8), v, row(8))
    sss.rms_norm_residual_bwd(row(8), residual_out=row(8), weight=v, rstd=t((1,)), x=row(8), scale=v)
    x = with_strides(t((2, 1, 8)), (8, far, 1))
    sss.causal_conv1d_bwd(x, t((8, 4)), dout=t((2, 1, 8)), dx=with_strides(t((2, 1, 8)), (8, far, 1)))
    x = with_strides(t((1, 5, 8)), (far, 16, 1))
    sss.causal_conv1d_bwd(x, t((8, 4)), dout=t((1, 5, 8)), dx=with_strides(t((1, 5, 8)), (far, 16, 1)))
    at = {"causal_conv1d_update": [1], "causal_conv1d_packed_fwd": [1], "selective_state_update_slots": [1, 3, 6, 8, 11],
          "selective_scan_packed_fwd": [1, 3, 6, 8, 11], "rms_norm_gated_fwd": [1, 4], "rms_norm_gated_bwd": [2, 5, 9],
          "rms_norm_residual_fwd": [1, 3], "rms_norm_residual_bwd": [3]}
    for name, a in lib.calls:
        if name == "causal_conv1d_bwd":
            continue
        got = [a[i] for i in at[name]]
        assert all(s in (2, 8) for s in got), (name, got)
    (_, one_row), (_, one_batch) = [c for c in lib.calls if c[0] == "causal_conv1d_bwd"]
    assert one_row[1:3] == (8, 8) and one_row[7:9] == (8, 8)
    assert one_batch[2] == 16 and one_batch[8] == 16 and max(one_batch[1], one_batch[7]) <= 5 * 16


def test_rows_that_overlap_are_refused(gpu):  # noqa: F811
    g, _ = gpu(0)
    for strides in ((7, 1), (0, 1), (8, 2), (1, 8)):
        with pytest.raises(ValueError, match="adjacent"):
            sss.rms_norm_gated_fwd(with_strides(g.tensor((2, 8)), strides), g.tensor((8,)))
    for strides in ((8, 2), (2, 8)):
        with pytest.raises(ValueError, match="adjacent"):
            sss.rms_norm_gated_fwd(with_strides(g.tensor((1, 8)), strides), g.tensor((8,)))


@pytest.mark.gpu
def test_last_token_of_a_long_buffer():
    """Batch 1, 5000 tokens x 4096: the last token's row is a view with a stride past 2^24."""
    import torch
    g = torch.Generator(device="cuda:0").manual_seed(9)
    r = lambda *s: torch.randn(*s, device="cuda:0", generator=g)
    x, w, z = r(1, 5000, 4096), torch.rand(4096, device="cuda:0"), r(1, 5000, 4096)
    assert x[:, -1].stride(0) > 1 << 24
    assert torch.equal(sss.rms_norm_gated_fwd(x[:, -1], w, z[:, -1]),
                       sss.rms_norm_gated_fwd(x[:, -1].clone(), w, z[:, -1].clone()))
    cw, cache = r(4096, 4), r(2, 3, 4096)
    other = cache.clone()
    assert torch.equal(sss.causal_conv1d_update(x[:, -1], cw, conv_state=cache),
                       sss.causal_conv1d_update(x[:, -1].clone(), cw, conv_state=other))
    assert torch.equal(cache, other)
