"""Calls of the gated delta rule that its documentation allows: offsets that change between a graph's replays, one tensor in
two places, a workspace kept by the caller, padding tokens, and the views it refuses."""
import numpy as np
import pytest

import delta_ref as ref
from test_gpu_delta import check, dev, inputs

pytestmark = pytest.mark.gpu


def test_varlen_replayed_with_other_offsets():
    """Offsets are read on the device: a captured packed batch runs whatever lengths it holds at the replay."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    H, P, N, G, T = 4, 64, 128, 2, 260
    d = ref.make(1, T, H, P, N, G, "bf16", False, seed=60)
    x = [t[0] for t in inputs(d)]
    h = dev(0.3 * np.random.default_rng(61).standard_normal((4, H, P, N)))
    cu = torch.tensor([0, 65, 130, 195, T], dtype=torch.int32, device="cuda")
    ssd.delta_forward_varlen(*x, cu, h)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, fin = ssd.delta_forward_varlen(*x, cu, h)
    for offsets in ([0, 1, 2, 3, T], [0, 0, 200, 200, T], [0, 33, 97, 259, T], [0, 65, 130, 195, T]):
        cu.copy_(torch.tensor(offsets, dtype=torch.int32))
        want = [t.clone() for t in ssd.delta_forward_varlen(*x, cu, h)]
        torch.cuda.synchronize()
        print(offsets, flush=True)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(fin, want[1])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_one_tensor_in_two_places(dt):
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    d = ref.make(2, 70, 4, 32, 64, 2, dt, True, seed=62)
    v, g, beta, k, _ = inputs(d)
    h = dev(d["init"])
    a = ssd.delta_forward(v, g, beta, k, k, h)
    b = ssd.delta_forward(v, g, beta, k, k.clone(), h)
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    a = ssd.delta_backward(v, g, beta, k, k, v, h, h)
    b = ssd.delta_backward(v, g, beta, k, k.clone(), v.clone(), h, h.clone())
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_workspace_of_the_callers():
    """Kept between calls of different sizes, larger than needed; one that is too small is refused."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    lib = ssd.load_library()
    ws = torch.empty(lib.ssd_delta_forward_workspace_bytes(2, 300, 4, 64, 128, 2, ssd.SSD_BF16) + 4096, dtype=torch.uint8,
                     device="cuda")
    for L in (300, 1, 77, 300):
        d = ref.make(2, L, 4, 64, 128, 2, "bf16", True, seed=63 + L)
        x, h = inputs(d), dev(d["init"])
        a, b = ssd.delta_forward(*x, h, workspace=ws), ssd.delta_forward(*x, h)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    need = lib.ssd_delta_forward_workspace_bytes(2, 300, 4, 64, 128, 2, ssd.SSD_BF16)
    with pytest.raises(ssd.SSDError):
        ssd.delta_forward(*x, h, workspace=ws[:need - 1])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_padding_leaves_the_state(dt):
    """Rows of one batch with tokens behind their end that hold zeros: their final states are those of their own length."""
    import mamba_ssd_sequence_chunked_amd as ssd
    d = ref.make(3, 90, 4, 32, 48, 2, dt, True, seed=64)
    ends = (90, 41, 0)
    for row, n in enumerate(ends):
        for t in ("v", "g", "beta", "k", "q"):
            d[t][row, n:] = 0.0
    y, fin = ssd.delta_forward(*inputs(d), dev(d["init"]))
    for row, n in enumerate(ends):
        want = ref.forward(*(d[t][row:row + 1, :n] for t in ("v", "g", "beta", "k", "q")), d["init"][row:row + 1])
        check(y[row:row + 1, :n], fin[row:row + 1], want, dt, 48)
        assert not y[row, n:].any()


def test_views_that_are_refused():
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    d = ref.make(2, 40, 4, 32, 64, 2, "f32", True, seed=65)
    v, g, beta, k, q = inputs(d)
    with pytest.raises(ValueError):                          # strided: every second token
        ssd.delta_forward(v[:, ::2], g[:, ::2], beta[:, ::2], k[:, ::2], q[:, ::2])
    flat = torch.empty(v.numel() + 1, device="cuda")
    off = flat[1:].view(v.shape)                             # 4 bytes off
    off.copy_(v)
    with pytest.raises(ssd.SSDError):
        ssd.delta_forward(off, g, beta, k, q)
    with pytest.raises(ValueError):
        ssd.delta_backward(v, g, beta, k, q, v[:, :39].contiguous())
