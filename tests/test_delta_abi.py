"""Host-side checks of the gated delta rule's entry points (no GPU): every refused call returns its status before
anything is enqueued, so the pointers here are never dereferenced; the binding refuses CPU tensors and wrong shapes."""
import ctypes

import pytest
import torch

import mamba_ssd_sequence_chunked_amd as ssd

OK, ERR_NULL, ERR_SHAPE, ERR_DTYPE, ERR_WS, ERR_ALIAS = 0, -1, -2, -3, -4, -6
P = ctypes.c_void_p


def fake(i):
    return P(0x10000000 + 0x1000000 * i)


SIZES = [
    (dict(P=48), ERR_SHAPE), (dict(P=256), ERR_SHAPE), (dict(N=8), ERR_SHAPE), (dict(N=40), ERR_SHAPE),
    (dict(N=272), ERR_SHAPE), (dict(G=3), ERR_SHAPE), (dict(G=0), ERR_SHAPE), (dict(H=0), ERR_SHAPE),
    (dict(H=65536), ERR_SHAPE), (dict(dtype=2), ERR_DTYPE), (dict(dtype=-1), ERR_DTYPE),
]


def forward(**kw):
    a = dict(v=fake(1), g=fake(2), beta=fake(3), k=fake(4), q=fake(5), init=None, y=fake(6), fin=fake(7), b=2, L=100,
             H=4, P=16, N=16, G=1, dtype=0, ws=fake(9), ws_bytes=1 << 30)
    a.update(kw)
    return ssd.load_library().ssd_delta_forward(
        a["v"], a["g"], a["beta"], a["k"], a["q"], a["init"], a["y"], a["fin"], a["b"], a["L"], a["H"], a["P"],
        a["N"], a["G"], a["dtype"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(L=-1), ERR_SHAPE), (dict(b=-1), ERR_SHAPE), (dict(b=65536), ERR_SHAPE),
    (dict(b=2, L=1 << 30), ERR_SHAPE),                    # 2^31 tokens
    (dict(b=1, L=1 << 27), ERR_SHAPE),                    # 2^24 blocks of 32 tokens x heads
    (dict(b=60000, L=(1 << 62)), ERR_SHAPE),              # the product would overflow
    (dict(b=65535, L=1, H=129, P=64), ERR_SHAPE),         # 2^29 rows x heads x columns of v
    (dict(v=None), ERR_NULL), (dict(g=None), ERR_NULL), (dict(fin=None), ERR_NULL), (dict(ws=None), ERR_NULL),
    (dict(ws_bytes=8), ERR_WS),
    (dict(y=fake(1)), ERR_ALIAS), (dict(fin=fake(6)), ERR_ALIAS), (dict(init=fake(7)), ERR_ALIAS),
    (dict(k=P(0x10000008)), ERR_SHAPE),                   # misaligned
    (dict(b=0), OK),
])
def test_forward_refuses(kw, code):
    assert forward(**kw) == code


def varlen(**kw):
    a = dict(v=fake(1), g=fake(2), beta=fake(3), k=fake(4), q=fake(5), cu=fake(10), nseq=3, init=None, y=fake(6),
             fin=fake(7), T=300, H=4, P=16, N=16, G=1, dtype=0, ws=fake(9), ws_bytes=1 << 30)
    a.update(kw)
    return ssd.load_library().ssd_delta_forward_varlen(
        a["v"], a["g"], a["beta"], a["k"], a["q"], a["cu"], a["nseq"], a["init"], a["y"], a["fin"], a["T"], a["H"],
        a["P"], a["N"], a["G"], a["dtype"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(T=-1), ERR_SHAPE), (dict(nseq=-1), ERR_SHAPE), (dict(nseq=(1 << 24) + 1), ERR_SHAPE),
    (dict(nseq=0), ERR_SHAPE), (dict(nseq=0, T=0), OK), (dict(cu=None), ERR_NULL), (dict(fin=None), ERR_NULL),
    (dict(ws_bytes=8), ERR_WS), (dict(fin=fake(10)), ERR_ALIAS), (dict(y=fake(10)), ERR_ALIAS),
])
def test_varlen_refuses(kw, code):
    assert varlen(**kw) == code


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(L=-1), ERR_SHAPE), (dict(b=65536), ERR_SHAPE), (dict(v=None), ERR_NULL), (dict(dy=None), ERR_NULL),
    (dict(dk=None), ERR_NULL), (dict(dinit=None), ERR_NULL), (dict(ws=None), ERR_NULL), (dict(ws_bytes=300), ERR_WS),
    (dict(dk=fake(4)), ERR_ALIAS), (dict(dq=fake(11)), ERR_ALIAS), (dict(dinit=fake(14)), ERR_ALIAS),
    (dict(dfinal=fake(13)), ERR_ALIAS), (dict(dv=P(0x10000008)), ERR_SHAPE), (dict(b=0), OK),
])
def test_backward_refuses(kw, code):
    a = dict(v=fake(1), g=fake(2), beta=fake(3), k=fake(4), q=fake(5), init=None, dy=fake(6), dfinal=None, dv=fake(8),
             dg=fake(9), dbeta=fake(10), dk=fake(11), dq=fake(12), dinit=fake(13), b=2, L=100, H=4, P=16, N=16, G=1,
             dtype=0, ws=fake(14), ws_bytes=1 << 30)
    a.update(kw)
    assert ssd.load_library().ssd_delta_backward(
        a["v"], a["g"], a["beta"], a["k"], a["q"], a["init"], a["dy"], a["dfinal"], a["dv"], a["dg"], a["dbeta"],
        a["dk"], a["dq"], a["dinit"], a["b"], a["L"], a["H"], a["P"], a["N"], a["G"], a["dtype"], a["ws"],
        a["ws_bytes"], None) == code


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(b=-1), ERR_SHAPE), (dict(b=65535, H=257), ERR_SHAPE), (dict(state=None), ERR_NULL), (dict(q=None), ERR_NULL), (dict(y=fake(2)), ERR_ALIAS),
    (dict(y=fake(1)), ERR_ALIAS), (dict(state=P(0x10000004)), ERR_SHAPE), (dict(b=0), OK),
])
def test_step_refuses(kw, code):
    a = dict(state=fake(1), v=fake(2), g=fake(3), beta=fake(4), k=fake(5), q=fake(6), y=fake(7), b=2, H=4, P=16, N=16,
             G=1, dtype=1)
    a.update(kw)
    assert ssd.load_library().ssd_delta_step(a["state"], a["v"], a["g"], a["beta"], a["k"], a["q"], a["y"], a["b"],
                                             a["H"], a["P"], a["N"], a["G"], a["dtype"], None) == code


def test_workspace_sizes():
    lib = ssd.load_library()
    assert lib.ssd_delta_forward_workspace_bytes(2, 100, 4, 16, 16, 1, 0) > 0
    assert lib.ssd_delta_forward_workspace_bytes(0, 0, 4, 16, 16, 1, 1) > 0
    assert lib.ssd_delta_forward_workspace_bytes(2, 100, 4, 48, 16, 1, 0) == 0
    assert lib.ssd_delta_forward_workspace_bytes(2, 100, 4, 16, 16, 1, 3) == 0
    assert lib.ssd_delta_forward_varlen_workspace_bytes(300, 3, 4, 16, 16, 1, 0) > 0
    assert lib.ssd_delta_forward_varlen_workspace_bytes(300, -3, 4, 16, 16, 1, 0) == 0


def test_binding_refuses():
    v, g, k = torch.zeros(1, 8, 2, 16), torch.zeros(1, 8, 2), torch.zeros(1, 8, 1, 16)
    with pytest.raises(ValueError, match="GPU"):
        ssd.delta_forward(v, g, g, k, k)
    with pytest.raises(ValueError):
        ssd.delta_forward(v, g[:, :4], g, k, k)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        ssd.delta_forward(v.half(), g, g, k.half(), k.half())
    with pytest.raises(ValueError):
        ssd.delta_forward(v[0], g, g, k, k)
    with pytest.raises(ValueError):
        ssd.delta_step(torch.zeros(1, 2, 16, 16), v[:, 0], g[:, 0], g[:, 0], k[:, 0], k[:, 0])
    with pytest.raises(ValueError):
        ssd.delta_forward_varlen(v[0], g[0], g[0], k[0], k[0], torch.zeros(2, dtype=torch.int32))
