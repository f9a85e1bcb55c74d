"""Packed batches of linear attention with very long rows, whose segments follow each other over many turns."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def packed(lens, H, P, N, dtype, seed):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T = sum(lens)
    v, k, q = (torch.randn((T, H, w), generator=gen, device="cuda", dtype=dtype) for w in (P, N, N))
    g = -torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    return v, g, k, q, cu


def milliseconds(call, calls=3):
    import torch
    call()
    times = []
    for _ in range(calls):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    return min(times)


def test_a_long_packed_row_costs_what_it_costs_in_a_batch():
    """2^19 tokens of 300 heads are 512 turns of a chain.  Finding a segment's place must not grow with its turn: tried one
    after another it made the packed row take 3.3 times the batch's."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    v, g, k, q, cu = packed([1 << 19], 300, 16, 16, torch.bfloat16, 1)
    one = milliseconds(lambda: ssd.linear_forward_varlen(v, g, k, q, cu))
    batch = milliseconds(lambda: ssd.linear_forward(v[None], g, k[None], q[None]))
    assert one <= 2 * batch, (one, batch)


@pytest.mark.parametrize("lens,H", [([150000, 5, 0, 70001, 1024 * 40, 2048], 64), ([1] * 100 + [40000] + [3000] * 100 + [1025] * 55, 2)],
                         ids=["few", "256rows"])
def test_rows_of_many_turns(lens, H):
    """Rows with up to 147 segments beside short and empty ones, against each row by itself."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    P = N = 16
    v, g, k, q, cu = packed(lens, H, P, N, torch.float32, 2)
    y, fin = ssd.linear_forward_varlen(v, g, k, q, cu)
    ends = np.cumsum([0] + lens)
    for i in sorted({0, 1, 2, 3, len(lens) // 2, len(lens) - 3, len(lens) - 2, len(lens) - 1, int(np.argmax(lens))}):
        at = slice(ends[i], ends[i + 1])
        a, b = ssd.linear_forward(v[None, at], g, k[None, at], q[None, at])
        # fp32 on both sides: 33 roundings of 2^-24 a chunk, of random signs, and twice that for two sides
        limit = 2 * 2.0 ** -24 * (33 * (-(-lens[i] // 32) + 1)) ** 0.5
        assert (y[at] - a[0]).norm() <= limit * a.norm() and (fin[i] - b[0]).norm() <= limit * b.norm()
