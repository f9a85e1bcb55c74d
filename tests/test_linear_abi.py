"""Host-side checks of linear attention's entry points and of state_move (no GPU): every refused call returns its
status before anything is enqueued, so the pointers here are never dereferenced; the binding refuses CPU tensors and
wrong shapes."""
import ctypes

import pytest
import torch

import mamba_ssd_sequence_chunked_amd as ssd

OK, ERR_NULL, ERR_SHAPE, ERR_DTYPE, ERR_WS, ERR_ALIAS = 0, -1, -2, -3, -4, -6
P = ctypes.c_void_p


def fake(i):
    return P(0x10000000 + 0x1000000 * i)


SIZES = [
    (dict(P=40), ERR_SHAPE), (dict(P=272), ERR_SHAPE), (dict(P=0), ERR_SHAPE), (dict(N=8), ERR_SHAPE),
    (dict(N=40), ERR_SHAPE), (dict(N=272), ERR_SHAPE), (dict(G=3), ERR_SHAPE), (dict(G=0), ERR_SHAPE),
    (dict(H=0), ERR_SHAPE), (dict(H=65536), ERR_SHAPE), (dict(H=8192, P=256), ERR_SHAPE), (dict(H=8192, N=144), ERR_SHAPE),
    (dict(dtype=2), ERR_DTYPE), (dict(dtype=-1), ERR_DTYPE),
]


def forward(**kw):
    a = dict(v=fake(1), g=fake(2), k=fake(4), q=fake(5), init=None, y=fake(6), fin=fake(7), b=2, L=100, H=4, P=16, N=16,
             G=2, dtype=0, ws=fake(9), ws_bytes=1 << 20)
    a.update(kw)
    return ssd.load_library().ssd_linear_forward(
        a["v"], a["g"], a["k"], a["q"], a["init"], a["y"], a["fin"], a["b"], a["L"], a["H"], a["P"], a["N"], a["G"],
        a["dtype"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(L=-1), ERR_SHAPE), (dict(b=-1), ERR_SHAPE), (dict(b=65536), ERR_SHAPE),
    (dict(b=2, L=1 << 30), ERR_SHAPE),                    # 2^31 tokens
    (dict(b=60000, L=(1 << 62)), ERR_SHAPE),              # the product would overflow
    (dict(b=65535, L=1, H=258), ERR_SHAPE),               # 2^24 workgroups
    (dict(b=65535, L=1, H=16, P=128, N=256), ERR_SHAPE),  # 2^34 elements of state
    (dict(v=None), ERR_NULL), (dict(g=None), ERR_NULL), (dict(fin=None), ERR_NULL), (dict(ws=None), ERR_NULL),
    (dict(ws_bytes=8), ERR_WS),
    (dict(y=fake(1)), ERR_ALIAS), (dict(fin=fake(6)), ERR_ALIAS), (dict(init=fake(7)), ERR_ALIAS),
    (dict(y=fake(2)), ERR_ALIAS), (dict(ws=fake(5)), ERR_ALIAS),
    (dict(k=P(0x14000008)), ERR_SHAPE), (dict(v=P(0x11000002)), ERR_SHAPE),       # misaligned
    (dict(b=0), OK),
])
def test_forward_refuses(kw, code):
    assert forward(**kw) == code


def varlen(**kw):
    a = dict(v=fake(1), g=fake(2), k=fake(4), q=fake(5), cu=fake(10), nseq=3, init=None, y=fake(6), fin=fake(7), T=300,
             H=4, P=16, N=16, G=2, dtype=0, ws=fake(9), ws_bytes=1 << 20)
    a.update(kw)
    return ssd.load_library().ssd_linear_forward_varlen(
        a["v"], a["g"], a["k"], a["q"], a["cu"], a["nseq"], a["init"], a["y"], a["fin"], a["T"], a["H"], a["P"], a["N"],
        a["G"], a["dtype"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(T=-1), ERR_SHAPE), (dict(nseq=-1), ERR_SHAPE), (dict(nseq=(1 << 24) + 1), ERR_SHAPE), (dict(T=1 << 31), ERR_SHAPE),
    (dict(nseq=0), ERR_SHAPE), (dict(nseq=0, T=0), OK), (dict(cu=None), ERR_NULL), (dict(fin=None), ERR_NULL),
    (dict(ws_bytes=8), ERR_WS), (dict(fin=fake(10)), ERR_ALIAS), (dict(y=fake(10)), ERR_ALIAS),
])
def test_varlen_refuses(kw, code):
    assert varlen(**kw) == code


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(L=-1), ERR_SHAPE), (dict(b=65536), ERR_SHAPE), (dict(v=None), ERR_NULL), (dict(dy=None), ERR_NULL),
    (dict(dk=None), ERR_NULL), (dict(dinit=None), ERR_NULL), (dict(dg=None), ERR_NULL), (dict(ws=None), ERR_NULL),
    (dict(ws_bytes=300), ERR_WS), (dict(dk=fake(4)), ERR_ALIAS), (dict(dq=fake(11)), ERR_ALIAS),
    (dict(dinit=fake(14)), ERR_ALIAS), (dict(dfinal=fake(13)), ERR_ALIAS), (dict(dg=fake(2)), ERR_ALIAS),
    (dict(dv=P(0x18000008)), ERR_SHAPE), (dict(b=0, g=None), ERR_NULL),
])
def test_backward_refuses(kw, code):
    a = dict(v=fake(1), g=fake(2), k=fake(4), q=fake(5), init=None, dy=fake(6), dfinal=None, dv=fake(8), dg=fake(9),
             dk=fake(11), dq=fake(12), dinit=fake(13), b=2, L=100, H=4, P=16, N=16, G=2, dtype=0, ws=fake(14),
             ws_bytes=1 << 20)
    a.update(kw)
    assert ssd.load_library().ssd_linear_backward(
        a["v"], a["g"], a["k"], a["q"], a["init"], a["dy"], a["dfinal"], a["dv"], a["dg"], a["dk"], a["dq"],
        a["dinit"], a["b"], a["L"], a["H"], a["P"], a["N"], a["G"], a["dtype"], a["ws"], a["ws_bytes"], None) == code


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(b=-1), ERR_SHAPE), (dict(b=65536), ERR_SHAPE), (dict(b=65535, H=258), ERR_SHAPE), (dict(n=-1), ERR_SHAPE),
    (dict(slots=None, n=3), ERR_SHAPE), (dict(n=(1 << 24) + 1), ERR_SHAPE),
    (dict(state=None), ERR_NULL), (dict(q=None), ERR_NULL), (dict(y=None), ERR_NULL),
    (dict(y=fake(2)), ERR_ALIAS), (dict(y=fake(1)), ERR_ALIAS), (dict(slots=fake(7)), ERR_ALIAS), (dict(g=fake(1)), ERR_ALIAS),
    (dict(state=P(0x11000004)), ERR_SHAPE), (dict(q=P(0x16000004)), ERR_SHAPE), (dict(b=0), OK),
])
def test_step_refuses(kw, code):
    a = dict(state=fake(1), slots=fake(8), n=2, v=fake(2), g=fake(3), k=fake(5), q=fake(6), y=fake(7), b=2, H=4, P=16,
             N=16, G=2, dtype=1)
    a.update(kw)
    assert ssd.load_library().ssd_linear_step(a["state"], a["slots"], a["n"], a["v"], a["g"], a["k"], a["q"], a["y"],
                                              a["b"], a["H"], a["P"], a["N"], a["G"], a["dtype"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(layers=-1), ERR_SHAPE), (dict(layers=65536), ERR_SHAPE), (dict(n=-1, m=-1), ERR_SHAPE), (dict(n=2049, m=2049), ERR_SHAPE),
    (dict(n=65536, source=fake(3)), ERR_SHAPE), (dict(m=5), ERR_SHAPE), (dict(size=6), ERR_SHAPE), (dict(size=0), ERR_SHAPE),
    (dict(size=(1 << 32) + 4), ERR_SHAPE), (dict(states=None), ERR_NULL), (dict(src=None), ERR_NULL),
    (dict(source=fake(1)), ERR_ALIAS), (dict(src=fake(1)), ERR_ALIAS), (dict(states=P(0x11000004)), ERR_SHAPE),
    (dict(source=P(0x13000008)), ERR_SHAPE), (dict(n=0, m=0), OK), (dict(layers=0), OK),
])
def test_move_refuses(kw, code):
    a = dict(states=fake(1), source=None, src=fake(2), layers=2, n=8, m=8, size=256)
    a.update(kw)
    assert ssd.load_library().ssd_state_move(a["states"], a["source"], a["src"], a["layers"], a["n"], a["m"], a["size"],
                                             None) == code


def test_workspace_sizes():
    lib = ssd.load_library()
    assert lib.ssd_linear_forward_workspace_bytes(2, 100, 4, 16, 16, 2, 0) > 0
    assert lib.ssd_linear_forward_workspace_bytes(0, 0, 4, 16, 16, 1, 1) > 0
    assert lib.ssd_linear_forward_workspace_bytes(2, 100, 4, 40, 16, 1, 0) == 0
    assert lib.ssd_linear_forward_workspace_bytes(2, 100, 4, 16, 16, 1, 3) == 0
    assert lib.ssd_linear_forward_varlen_workspace_bytes(300, 3, 4, 16, 16, 1, 0) > 0
    assert lib.ssd_linear_forward_varlen_workspace_bytes(300, -3, 4, 16, 16, 1, 0) == 0
    # an fp32 copy of every head's dk and dv where they are shared
    own, shared = (lib.ssd_linear_backward_workspace_bytes(2, 4096, 256, 64, 128, G, 1) for G in (256, 64))
    assert shared - own >= 2 * 4096 * 256 * (64 + 128) * 4


def test_binding_refuses():
    v, g, k, q = torch.zeros(1, 8, 1, 16), torch.zeros(2), torch.zeros(1, 8, 1, 16), torch.zeros(1, 8, 2, 16)
    with pytest.raises(ValueError, match="GPU"):
        ssd.linear_forward(v, g, k, q)
    with pytest.raises(ValueError):
        ssd.linear_forward(v, g[:1], k, q)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        ssd.linear_forward(v.half(), g, k.half(), q.half())
    with pytest.raises(ValueError):
        ssd.linear_forward(v[0], g, k, q)
    with pytest.raises(ValueError, match="GPU"):
        ssd.linear_backward(v, g, k, q, torch.zeros(1, 8, 2, 16))
    with pytest.raises(ValueError, match="GPU"):
        ssd.linear_step(torch.zeros(1, 2, 16, 16), v[:, 0], g, k[:, 0], q[:, 0])
    with pytest.raises(ValueError):                       # three states, one row, no slots
        ssd.linear_step(torch.zeros(3, 2, 16, 16), v[:, 0], g, k[:, 0], q[:, 0])
    with pytest.raises(ValueError):
        ssd.linear_forward_varlen(v[0], g, k[0], q[0], torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="GPU"):
        ssd.state_move(torch.zeros(4, 2, 16, 16), torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):
        ssd.state_move(torch.zeros(4, 16), torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):
        ssd.state_move(torch.zeros(4, 2, 16, 16), torch.zeros(4, dtype=torch.int32), source=torch.zeros(2, 4, 2, 16, 16))
