"""Rates A that are no ordinary numbers: a NaN reaches every result of its channel and no other, -inf
forgets the state in a step and keeps it in one of size zero."""
import pytest

pytestmark = pytest.mark.gpu


def operands(rows, dim, n, bf16):
    import torch
    g = torch.Generator(device="cuda:0").manual_seed(7)
    r = lambda *s: torch.randn(*s, device="cuda:0", generator=g)
    t = torch.bfloat16 if bf16 else torch.float32
    return dict(x=r(rows, dim).to(t), delta=(0.1 + r(rows, dim).abs()).to(t), A=-r(dim, n).abs() - 0.1, B=r(rows, n).to(t),
                C=r(rows, n).to(t), D=r(dim), z=r(rows, dim).to(t))


def packed(v, chunks, **kw):
    import torch
    import selective_state_space_20_amd as sss
    cu = torch.tensor([0, 3, 50, 200], dtype=torch.int32, device="cuda:0")
    st = torch.zeros(3, *v["A"].shape, device="cuda:0")
    return sss.selective_scan_packed_fwd(**v, cu_seqlens=cu, state=st, **kw), st


def slots(v, chunks, **kw):
    import torch
    import selective_state_space_20_amd as sss
    st = torch.ones(v["x"].shape[0], *v["A"].shape, device="cuda:0")
    return sss.selective_state_update_slots(**v, state=st, **kw), st


def chunked(fn, chunks, monkeypatch):
    if chunks:
        monkeypatch.setenv("SSS_FORCE_SEGMENTS", str(chunks))
    return fn


CALLS = [(packed, None), (packed, 7), (slots, None)]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("n", [1, 2, 16, 64])
@pytest.mark.parametrize("fn, chunks", CALLS)
def test_nan_reaches_its_channel(fn, chunks, n, bf16, monkeypatch):
    chunked(fn, chunks, monkeypatch)
    v = operands(200, 70, n, bf16)
    want, want_state = fn(v, chunks)
    v["A"] = v["A"].clone()
    v["A"][5, n // 2] = v["A"][69, n - 1] = float("nan")
    y, st = fn(v, chunks)
    hit = [5, 69]
    rest = [d for d in range(70) if d not in hit]
    assert bool(y[:, hit].isnan().all()) and bool(st[:, 5, n // 2].isnan().all()) and bool(st[:, 69, n - 1].isnan().all())
    assert bool((y[:, rest] == want[:, rest]).all()) and bool((st[:, rest] == want_state[:, rest]).all())


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("fn, chunks", CALLS)
def test_minus_infinity_forgets(fn, chunks, bf16, monkeypatch):
    chunked(fn, chunks, monkeypatch)
    v = operands(200, 70, 16, bf16)
    v["A"] = v["A"].clone()
    v["A"][3] = float("-inf")
    y, st = fn(v, chunks)
    f = {k: t.double() for k, t in v.items()}
    h = f["delta"][:, 3, None] * f["B"] * f["x"][:, 3, None]  # nothing of the state before
    want = ((h * f["C"]).sum(1) + f["D"][3] * f["x"][:, 3]) * f["z"][:, 3] / (1 + (-f["z"][:, 3]).exp())
    assert bool(((y[:, 3].double() - want).abs() <= 1e-4 * want.abs().max()).all())
    v["delta"] = v["delta"].clone()
    v["delta"][:, 3] = 0.0
    _, st = fn(v, chunks)
    assert bool((st[:, 3] == (1.0 if fn is slots else 0.0)).all())
