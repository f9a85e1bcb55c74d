"""What the header says of linear attention's calls and of pools of states beyond their values."""
import pytest

import linear_ref as ref
from test_gpu_linear import inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("where", ["v", "k"])
def test_inf_is_confined(where, dt):
    """An Inf (with bf16 inputs it may arrive as NaN) reaches its chunk of 32 tokens and what follows, of its batch row and its
    group's heads; of v, only its own column of the state."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    v, g, k, q = inputs(ref.make(2, 200, 4, 64, 64, 2, dt, False, seed=950))
    y0, f0 = ssd.linear_forward(v, g, k, q)
    (v if where == "v" else k)[0, 130, 1, 5] = float("inf")
    y1, f1 = ssd.linear_forward(v, g, k, q)
    assert torch.equal(y0[1], y1[1]) and torch.equal(f0[1], f1[1])
    assert torch.equal(y0[0, :, :2], y1[0, :, :2]) and torch.equal(f0[0, :2], f1[0, :2])
    assert torch.equal(y0[0, :128], y1[0, :128])
    if where == "v":
        assert not y1[0, 130:, 2:, 5].isfinite().any() and not f1[0, 2:, 5].isfinite().any()
        rest = torch.arange(64, device="cuda") != 5
        assert torch.equal(y0[..., rest], y1[..., rest]) and torch.equal(f0[:, :, rest], f1[:, :, rest])
    else:
        assert not y1[0, 130:, 2:].isfinite().any() and not f1[0, 2:, :, 5].isfinite().any()


def test_a_pool_too_large_to_move_in_place():
    """More than 2048 slots are refused in place and move through a buffer, in two calls: what the header says."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    n, H, P, N = 4000, 2, 16, 16
    gen = torch.Generator(device="cuda").manual_seed(3)
    pool = torch.randn((2, n, H, P, N), generator=gen, device="cuda")
    old = pool.clone()
    table = lambda t: torch.tensor(t, dtype=torch.int32, device="cuda")      # noqa: E731
    with pytest.raises(ssd.SSDError):
        ssd.state_move(pool, torch.arange(n, dtype=torch.int32, device="cuda"))
    into, take = [3990, 17, 5, 2500, 6], [17, 3990, 3999, 17, 17]             # two change places, one moves down, two forks
    buffer = torch.empty((2, len(take), H, P, N), device="cuda")
    ssd.state_move(buffer, table(take), source=pool)
    src = torch.full((n,), -2, dtype=torch.int32, device="cuda")
    src[into], src[3999] = table(range(len(take))), -1
    ssd.state_move(pool, src, source=buffer)
    want = old.clone()
    want[:, into], want[:, 3999] = old[:, take], 0
    assert torch.equal(pool, want)
