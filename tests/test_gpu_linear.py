"""Linear attention with a decay for each head and the moves of its states, against the float64 recurrence (linear_ref).

Tolerances, fixed before the first run.  A rounding moves a value by at most half a step, ROUND relative to it; all results
are sums in which every term enters linearly, so each is held, element by element, to its magnitude (the same sum over
absolute values) times the roundings a term can meet on its way:

 * fp32 work: a term is one of at most L + N + P summands of sums in fp32, each off by half a step of a partial sum;
   weights are powers exp(g n) whose exponent, at most 104 where the power is not zero, is rounded (104 half steps), of which
   a term meets at most two, and their products.
 * bf16 inputs, fp32 results: the weighted values that enter a state are pairs of bf16 values (ROUND^2); what dg sums
   reads the states as pairs too.
 * bf16 results: one bf16 operand on the way (a term comes through the scores or through a state), and the result's own
   rounding.
"""
import numpy as np
import pytest

import linear_ref as ref

pytestmark = pytest.mark.gpu

ROUND = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def fp32_unit(L, N, P):
    return (L + N + P + 400) * ROUND["f32"]


def state_unit(dtype, L, N, P):
    return fp32_unit(L, N, P) + (ROUND["bf16"] ** 2 if dtype == "bf16" else 0.0)


def y_unit(dtype, L, N, P):
    return state_unit(dtype, L, N, P) + 2 * ROUND[dtype] + 2 * ROUND[dtype] ** 2


def dg_unit(dtype, L, N, P):
    return 2 * state_unit(dtype, L, N, P)


def dev(a, dtype="f32"):
    import torch
    if a is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(a)).to("cuda")
    return t.to(torch.bfloat16 if dtype == "bf16" else torch.float32)


def inputs(d):
    t = d["dtype"]
    return [dev(d["v"], t), dev(d["g"]), dev(d["k"], t), dev(d["q"], t)]


def f64(t):
    return t.detach().cpu().double().numpy()


def hold(name, got, want, size, unit):
    got = f64(got)
    assert got.shape == want.shape and np.isfinite(got).all(), name
    over = np.abs(got - want) / (unit * size + 2.0 ** -120)
    assert over.size == 0 or over.max() <= 1, (name, over.max())


def check(y, fin, want, dt, L, N, P):
    (yr, Sr), (ym, Sm) = want
    hold("y", y, yr, ym, y_unit(dt, L, N, P))
    hold("final", fin, Sr, Sm, state_unit(dt, L, N, P))


def rel2(got, want):
    return np.linalg.norm(f64(got) - want) / np.linalg.norm(want)


# (batch, seqlen, nheads, headdim, dstate, ngroups, dtype, init, kind)
CASES = [
    (1, 1, 1, 16, 16, 1, "f32", False, "ladder"),
    (2, 1, 2, 64, 128, 1, "bf16", True, "ladder"),
    (1, 2, 3, 32, 16, 3, "bf16", False, "ladder"),
    (2, 31, 4, 16, 32, 2, "f32", True, "ladder"),
    (2, 32, 4, 64, 128, 4, "bf16", False, "ladder"),
    (1, 33, 2, 128, 64, 1, "bf16", True, "ladder"),
    (3, 63, 5, 80, 48, 5, "bf16", True, "ladder"),
    (1, 64, 6, 32, 256, 2, "f32", True, "ladder"),
    (2, 65, 3, 256, 256, 1, "bf16", True, "ladder"),
    (1, 65, 2, 256, 144, 2, "f32", True, "ladder"),
    (1, 130, 2, 112, 256, 2, "f32", False, "ladder"),
    (2, 257, 4, 64, 128, 2, "bf16", True, "ladder"),
    (1, 300, 7, 16, 240, 7, "bf16", False, "ladder"),
    (2, 95, 2, 64, 80, 1, "f32", True, "strong"),
    (2, 160, 4, 64, 128, 4, "bf16", True, "strong"),
    (2, 130, 5, 32, 64, 5, "f32", True, "edges"),
    (2, 130, 10, 48, 96, 5, "bf16", True, "edges"),
    (1, 200, 4, 32, 32, 4, "f32", True, "long"),
    (1, 200, 4, 64, 128, 4, "bf16", True, "long"),
    # few rows: cut into segments
    (1, 900, 3, 64, 128, 3, "bf16", True, "ladder"),
    (2, 601, 2, 32, 64, 1, "f32", False, "ladder"),
    (1, 1100, 2, 192, 32, 2, "bf16", True, "edges"),
]


def ident(c):
    return "b{}_L{}_H{}_P{}_N{}_G{}_{}_{}_{}".format(*c)


@pytest.mark.parametrize("c", CASES, ids=ident)
def test_forward(c):
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    b, L, H, P, N, G, dt, init, kind = c
    d = ref.make(b, L, H, P, N, G, dt, init, seed=100 + CASES.index(c), kind=kind)
    y, fin = ssd.linear_forward(*inputs(d), dev(d["init"]))
    torch.cuda.synchronize()
    check(y, fin, ref.forward(d["v"], d["g"], d["k"], d["q"], d["init"]), dt, L, N, P)


@pytest.mark.parametrize("c", CASES, ids=ident)
def test_backward(c):
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    b, L, H, P, N, G, dt, init, kind = c
    d = ref.make(b, L, H, P, N, G, dt, init, seed=200 + CASES.index(c), kind=kind)
    got = ssd.linear_backward(*inputs(d), dev(d["dy"], dt), dev(d["init"]), dev(d["dfinal"]))
    torch.cuda.synchronize()
    want, size = ref.backward(d["v"], d["g"], d["k"], d["q"], d["dy"], d["init"], d["dfinal"])
    for n in ("dv", "dk", "dq"):
        hold(n, got[n], want[n], size[n], y_unit(dt, L, N, P))
    hold("dinit", got["dinit"], want["dinit"], size["dinit"], state_unit(dt, L, N, P))
    hold("dg", got["dg"], want["dg"], size["dg"], dg_unit(dt, L, N, P) + b * ROUND["f32"])


def test_accuracy_as_stated():
    """The header's statements, in the 2-norm."""
    import mamba_ssd_sequence_chunked_amd as ssd
    d = ref.make(2, 700, 8, 64, 128, 4, "bf16", True, seed=5)
    y, fin = ssd.linear_forward(*inputs(d), dev(d["init"]))
    (yr, S), _ = ref.forward(d["v"], d["g"], d["k"], d["q"], d["init"])
    assert rel2(fin, S) <= 5e-7 and rel2(y, yr) <= 2.6e-3
    got = ssd.linear_backward(*inputs(d), dev(d["dy"], "bf16"), dev(d["init"]), dev(d["dfinal"]))
    want, size = ref.backward(d["v"], d["g"], d["k"], d["q"], d["dy"], d["init"], d["dfinal"])
    assert rel2(got["dinit"], want["dinit"]) <= 5e-7 and rel2(got["dg"], want["dg"]) <= 4e-6
    assert all(rel2(got[n], want[n]) <= 2.6e-3 for n in ("dv", "dk", "dq"))
    d = ref.make(2, 700, 8, 64, 128, 4, "f32", True, seed=6)
    y, fin = ssd.linear_forward(*inputs(d), dev(d["init"]))
    (yr, S), _ = ref.forward(d["v"], d["g"], d["k"], d["q"], d["init"])
    assert rel2(fin, S) <= 1e-6 and rel2(y, yr) <= 1e-6


def test_gradient_of_the_decay_against_differences():
    """(loss(g + h) - loss(g - h)) / 2h of the library's own forward.  The loss is summed in 64 bits from fp32 outputs, each
    off by at most fp32_unit of its magnitude; h^2 of the third derivative is at most (h L)^2 of the terms' size."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    b, L, H, P, N = 1, 40, 2, 16, 32
    d = ref.make(b, L, H, P, N, H, "f32", True, seed=7)
    v, g, k, q = inputs(d)
    init, dy, dfinal = dev(d["init"]), dev(d["dy"]), dev(d["dfinal"])
    got = ssd.linear_backward(v, g, k, q, dy, init, dfinal)["dg"]
    h = 2.0 ** -9
    _, (ym, Sm) = ref.forward(d["v"], d["g"], d["k"], d["q"], d["init"])
    size = ref.backward(d["v"], d["g"], d["k"], d["q"], d["dy"], d["init"], d["dfinal"])[1]["dg"]
    for i in range(H):
        loss = []
        for s in (h, -h):
            gs = g.clone()
            gs[i] += s
            y, fin = ssd.linear_forward(v, gs, k, q, init)
            loss.append(float((y.double() * dy.double()).sum() + (fin.double() * dfinal.double()).sum()))
        step = float((g[i] + h).double() - (g[i] - h).double())
        magnitude = float((ym * np.abs(d["dy"])).sum() + (Sm * np.abs(d["dfinal"])).sum())
        room = 2 * fp32_unit(L, N, P) * magnitude / step + (h * L) ** 2 * size[i]
        assert abs((loss[0] - loss[1]) / step - float(got[i])) <= room


def test_empty_and_no_batch():
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    d = ref.make(2, 0, 4, 32, 64, 2, "bf16", True, seed=8)
    y, fin = ssd.linear_forward(*inputs(d), dev(d["init"]))
    assert y.shape == (2, 0, 4, 32) and torch.equal(fin, dev(d["init"]))
    assert torch.count_nonzero(ssd.linear_forward(*inputs(d))[1]) == 0
    out = ssd.linear_backward(*inputs(d), dev(d["dy"], "bf16"), dev(d["init"]), dev(d["dfinal"]))
    assert torch.equal(out["dinit"], dev(d["dfinal"])) and not out["dg"].any() and out["dk"].numel() == 0
    d = ref.make(0, 5, 4, 32, 64, 2, "f32", seed=8)
    y, fin = ssd.linear_forward(*inputs(d))
    assert y.numel() == 0 and fin.shape == (0, 4, 32, 64)
    assert not ssd.linear_backward(*inputs(d), dev(d["dy"]))["dg"].any()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_split_and_resumed(dt):
    """Running a sequence in pieces, each from the last one's final state, gives the whole run."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    d = ref.make(2, 150, 4, 64, 96, 2, dt, True, seed=9)
    v, g, k, q = inputs(d)
    S, ys = dev(d["init"]), []
    for a, z in ((0, 1), (1, 40), (40, 104), (104, 150)):
        y, S = ssd.linear_forward(*(t if t is g else t[:, a:z].contiguous() for t in (v, g, k, q)), S)
        ys.append(y)
    check(torch.cat(ys, 1), S, ref.forward(d["v"], d["g"], d["k"], d["q"], d["init"]), dt, 150, 96, 64)


def test_nan_is_confined():
    """A NaN in k reaches its own 64-token chunk and what follows, of its batch row and its group's heads only; with decay
    and all it never reaches back further."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    d = ref.make(2, 200, 4, 64, 64, 2, "bf16", False, seed=10)
    v, g, k, q = inputs(d)
    y0, f0 = ssd.linear_forward(v, g, k, q)
    k[0, 130, 1, 5] = float("nan")
    y1, f1 = ssd.linear_forward(v, g, k, q)
    assert torch.equal(y0[1], y1[1]) and torch.equal(f0[1], f1[1])
    assert torch.equal(y0[0, :, :2], y1[0, :, :2]) and torch.equal(f0[0, :2], f1[0, :2])
    assert torch.equal(y0[0, :128], y1[0, :128])
    assert torch.isnan(y1[0, 130:, 2:]).all() and torch.isnan(f1[0, 2:]).any()


# ---- packed sequences -----------------------------------------------------------------------------------

VARLEN = [
    ([5, 0, 64, 1, 33, 200], 4, 64, 128, 2, "bf16", True),
    ([0, 0, 7], 3, 16, 48, 3, "f32", True),
    ([1] * 70, 2, 32, 32, 1, "bf16", False),
    ([700, 3, 1200, 0, 65], 2, 64, 64, 2, "bf16", True),
    ([1500], 2, 32, 16, 2, "f32", False),
    ([300, 600], 2, 256, 160, 1, "bf16", True),
]


@pytest.mark.parametrize("c", VARLEN, ids=lambda c: "n{}_T{}_{}".format(len(c[0]), sum(c[0]), c[5]))
def test_varlen(c):
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    lens, H, P, N, G, dt, init = c
    T, n = sum(lens), len(lens)
    d = ref.make(1, T, H, P, N, G, dt, False, seed=300 + VARLEN.index(c))
    h = np.random.default_rng(12).standard_normal((n, H, P, N)).astype(np.float32) if init else None
    cu = np.concatenate([[0], np.cumsum(lens)])
    v, g, k, q = inputs(d)
    y, fin = ssd.linear_forward_varlen(v[0], g, k[0], q[0], dev(cu).int(), dev(h))
    torch.cuda.synchronize()
    for i in range(n):
        s = np.s_[:, cu[i]:cu[i + 1]]
        want = ref.forward(d["v"][s], d["g"], d["k"][s], d["q"][s], None if h is None else h[i:i + 1])
        check(y[None, cu[i]:cu[i + 1]], fin[i:i + 1], want, dt, lens[i], N, P)


def test_varlen_of_thousands():
    """More sequences than one step of the search looks at, twice over; equal to the batch they are."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    n, L, H, P, N = 4500, 2, 1, 16, 16
    d = ref.make(n, L, H, P, N, 1, "bf16", True, seed=13)
    v, g, k, q = inputs(d)
    cu = torch.arange(0, 2 * n + 1, 2, dtype=torch.int32, device="cuda")
    flat = [t.reshape(n * L, *t.shape[2:]) for t in (v, k, q)]
    y, fin = ssd.linear_forward_varlen(flat[0], g, flat[1], flat[2], cu, dev(d["init"]))
    yr, fr = ssd.linear_forward(v, g, k, q, dev(d["init"]))
    assert torch.equal(y.view_as(yr), yr) and torch.equal(fin, fr)


@pytest.mark.parametrize("cu", [[5, 2, 90, -7, 1000], [0, 0, 0, 0, 0], [90, 60, 30, 0, -1],
                                [-2 ** 31, 2 ** 31 - 1, 0, 40, 90]], ids=["jumps", "zeros", "falling", "extreme"])
@pytest.mark.parametrize("T", [90, 1400])
def test_varlen_bad_offsets_stay_inside(cu, T):
    """Offsets are not checked: with any others the values are unspecified, the accesses are not; what no offset names
    stays as it was."""
    import torch
    from test_gpu_guard import Guarded, _lib, _p, _stream
    H, P, N, G = 3, 32, 48, 3
    d = ref.make(1, T, H, P, N, G, "bf16", False, seed=14)
    v, g, k, q = (t[0] if t.dim() > 1 else t for t in inputs(d))
    offsets = torch.tensor(cu, dtype=torch.int32, device="cuda")
    y, fin = Guarded((T, H, P), torch.bfloat16), Guarded((4, H, P, N), torch.float32)
    ws = Guarded((_lib().ssd_linear_forward_varlen_workspace_bytes(T, 4, H, P, N, G, 1),), torch.uint8)
    rc = _lib().ssd_linear_forward_varlen(_p(v), _p(g), _p(k), _p(q), _p(offsets), 4, None, _p(y.t), _p(fin.t), T, H, P, N,
                                          G, 1, _p(ws.t), ws.n, _stream())
    assert rc == 0
    torch.cuda.synchronize()
    assert y.intact() and fin.intact() and ws.intact()


def test_varlen_leaves_what_lies_behind():
    """Tokens behind the last sequence: y stays as it was."""
    import torch
    from test_gpu_guard import _lib, _p, _stream
    T, H, P, N, G = 150, 2, 64, 64, 2
    d = ref.make(1, T, H, P, N, G, "bf16", False, seed=15)
    v, g, k, q = (t[0] if t.dim() > 1 else t for t in inputs(d))
    cu = torch.tensor([0, 30, 97], dtype=torch.int32, device="cuda")
    y = torch.full((T, H, P), 3.0, dtype=torch.bfloat16, device="cuda")
    fin = torch.empty((2, H, P, N), device="cuda")
    n = _lib().ssd_linear_forward_varlen_workspace_bytes(T, 2, H, P, N, G, 1)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert _lib().ssd_linear_forward_varlen(_p(v), _p(g), _p(k), _p(q), _p(cu), 2, None, _p(y), _p(fin), T, H, P, N, G, 1,
                                            _p(ws), n, _stream()) == 0
    torch.cuda.synchronize()
    assert (y[97:] == 3.0).all()
    s = np.s_[:, 30:97]
    check(y[None, 30:97], fin[1:], ref.forward(d["v"][s], d["g"], d["k"][s], d["q"][s]), "bf16", 67, N, P)


# ---- one token ------------------------------------------------------------------------------------------

STEPS = [
    (1, 1, 16, 16, 1, "f32"), (3, 4, 64, 128, 2, "bf16"), (2, 6, 32, 48, 3, "f32"), (5, 2, 256, 256, 1, "bf16"),
    (2, 3, 112, 240, 3, "bf16"), (4, 5, 256, 16, 5, "f32"), (130, 2, 16, 64, 2, "bf16"),
]


@pytest.mark.parametrize("c", STEPS, ids=lambda c: "b{}_H{}_P{}_N{}_G{}_{}".format(*c))
@pytest.mark.parametrize("kind", ["ladder", "edges"])
def test_step(c, kind):
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    b, H, P, N, G, dt = c
    d = ref.make(b, 1, H, P, N, G, dt, True, seed=400 + STEPS.index(c), kind=kind)
    v, g, k, q = (t[:, 0].contiguous() if t.dim() > 1 else t for t in inputs(d))
    want = ref.forward(d["v"], d["g"], d["k"], d["q"], d["init"])
    S = dev(d["init"])
    y = ssd.linear_step(S, v, g, k, q)
    check(y[:, None], S, want, "f32" if dt == "f32" else dt, 1, N, P)
    # in a pool, the rows in any order
    pool = torch.randn((b + 3, H, P, N), device="cuda")
    slots = torch.randperm(b + 3, generator=torch.Generator().manual_seed(1))[:b].int().cuda()
    pool[slots.long()] = dev(d["init"])
    old = pool.clone()
    out = torch.empty_like(y)
    assert ssd.linear_step(pool, v, g, k, q, slots=slots, y=out) is out
    assert torch.equal(out, y) and torch.equal(pool[slots.long()], S)
    rest = torch.ones(b + 3, dtype=torch.bool)
    rest[slots.long().cpu()] = False
    assert torch.equal(pool[rest.cuda()], old[rest.cuda()])


def test_step_padding_and_repeated_slots():
    """A slot out of range touches nothing and answers zero; of rows with one slot the first has it."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    b, H, P, N, G = 9, 3, 32, 64, 3
    d = ref.make(b, 1, H, P, N, G, "bf16", False, seed=16)
    v, g, k, q = (t[:, 0].contiguous() if t.dim() > 1 else t for t in inputs(d))
    pool = torch.randn((6, H, P, N), device="cuda")
    slots = torch.tensor([4, -1, 0, 4, 6, 2 ** 31 - 1, -2 ** 31, 0, 5], dtype=torch.int32, device="cuda")
    rows, at = [0, 2, 8], [4, 0, 5]
    S = pool[at].clone()
    want = ssd.linear_step(S, v[rows], g, k[rows], q[rows])
    old = pool.clone()
    y = ssd.linear_step(pool, v, g, k, q, slots=slots)
    assert torch.equal(y[rows], want) and torch.equal(pool[at], S)
    assert not y[[1, 3, 4, 5, 6, 7]].any()
    assert torch.equal(pool[[1, 2, 3]], old[[1, 2, 3]])
    # an empty pool has no slot at all
    none = torch.empty((0, H, P, N), device="cuda")
    assert not ssd.linear_step(none, v, g, k, q, slots=slots).any()


def test_step_padding_with_infinite_inputs():
    """Rows of padding answer zero whatever their inputs hold."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    d = ref.make(2, 1, 2, 16, 16, 2, "bf16", False, seed=17)
    v, g, k, q = (t[:, 0].contiguous() if t.dim() > 1 else t for t in inputs(d))
    q[1], v[1] = float("inf"), float("nan")
    pool = torch.randn((2, 2, 16, 16), device="cuda")
    y = ssd.linear_step(pool, v, g, k, q, slots=torch.tensor([1, -1], dtype=torch.int32, device="cuda"))
    assert not y[1].any() and torch.isfinite(pool).all()


# ---- moves ----------------------------------------------------------------------------------------------

def moved(states, src, source=None):
    """The map in numpy, on the bits."""
    new = states.copy()
    frm = states if source is None else source
    for i, s in enumerate(src):
        if 0 <= s < frm.shape[-4]:
            new[..., i, :, :, :] = frm[..., s, :, :, :]
        elif s == -1:
            new[..., i, :, :, :] = 0
    return new


# (layers or None, slots, heads, headdim, dstate, share of slots that move)
MOVES = [
    (None, 1, 1, 16, 16, 1.0), (None, 7, 3, 16, 16, 1.0), (3, 16, 2, 32, 48, 0.5), (None, 127, 1, 16, 16, 1.0),
    (2, 129, 1, 16, 16, 1.0), (None, 300, 1, 16, 32, 0.9), (None, 700, 1, 16, 16, 1.0), (None, 2048, 1, 16, 16, 1.0),
    (4, 33, 5, 16, 80, 0.1), (None, 6, 24, 64, 128, 0.7), (None, 40, 7, 16, 16, 0.0),
]


@pytest.mark.parametrize("c", MOVES, ids=lambda c: "l{}_n{}_H{}_P{}_N{}_{}".format(*c))
@pytest.mark.parametrize("kind", ["any", "permutation", "one"])
def test_move_in_place(c, kind):
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    layers, n, H, P, N, share = c
    rng = np.random.default_rng([MOVES.index(c), len(kind)])
    shape = (n, H, P, N) if layers is None else (layers, n, H, P, N)
    x = rng.integers(0, 2 ** 32, shape, dtype=np.uint32)             # any bits, NaN among them
    if kind == "permutation":
        src = rng.permutation(n)
    elif kind == "one":
        src = np.full(n, n // 2)
    else:
        src = np.where(rng.random(n) < share, rng.integers(-3, n + 3, n), np.arange(n))
    t = torch.from_numpy(x.view(np.float32).copy()).cuda()
    out = ssd.state_move(t, torch.from_numpy(src.astype(np.int32)).cuda())
    assert out is t
    assert np.array_equal(t.cpu().numpy().view(np.uint32), moved(x, src))


@pytest.mark.parametrize("n,m,layers", [(5, 3, None), (2500, 40, None), (4500, 4100, None), (9, 200, 3)])
def test_move_between_pools(n, m, layers):
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    rng = np.random.default_rng(n)
    lead = () if layers is None else (layers,)
    x, s = (rng.integers(0, 2 ** 32, (*lead, z, 1, 16, 16), dtype=np.uint32) for z in (n, m))
    src = rng.integers(-3, m + 3, n)
    t, f = (torch.from_numpy(z.view(np.float32).copy()).cuda() for z in (x, s))
    ssd.state_move(t, torch.from_numpy(src.astype(np.int32)).cuda(), source=f)
    assert np.array_equal(t.cpu().numpy().view(np.uint32), moved(x, src, s))
    assert np.array_equal(f.cpu().numpy().view(np.uint32), s)


def test_move_extreme_indices():
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    t = torch.randn((5, 2, 16, 16), device="cuda")
    old = t.clone()
    ssd.state_move(t, torch.tensor([-2 ** 31, 2 ** 31 - 1, 5, -2, 4], dtype=torch.int32, device="cuda"))
    assert torch.equal(t, old)
    assert ssd.state_move(torch.empty((0, 2, 16, 16), device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")).numel() == 0


# ---- together -------------------------------------------------------------------------------------------

def test_prefill_fork_decode_compact():
    """Prompts prefilled as a packed batch, put into slots, one forked, beams reordered, decoded in the pool, compacted:
    every sequence's outputs are those of its whole token sequence run at once."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    H, P, N, G, dt = 4, 64, 128, 2, "bf16"
    lens, steps = [40, 130, 9], 6
    T = sum(lens)
    d = ref.make(1, T, H, P, N, G, dt, False, seed=18)
    v, g, k, q = inputs(d)
    cu = np.concatenate([[0], np.cumsum(lens)])
    _, fin = ssd.linear_forward_varlen(v[0], g, k[0], q[0], dev(cu).int())
    pool = torch.full((6, H, P, N), float("nan"), device="cuda")
    table = lambda *s: torch.tensor(s, dtype=torch.int32, device="cuda")       # noqa: E731
    ssd.state_move(pool, table(2, -1, 0, -2, 1, -1), source=fin)     # sequence 2 in slot 0, 0 in 2, 1 in 4
    ssd.state_move(pool, table(0, 4, 2, 4, 4, 5))                    # slots 1 and 3 continue sequence 1 too
    ssd.state_move(pool, table(2, 1, 0, 3, 4, 5))                    # slots 0 and 2 change places
    owner = [0, 1, 2, 1, 1]                                          # of slots 0 to 4 now
    more = ref.make(5, steps, H, P, N, G, dt, False, seed=19)
    mv, _, mk, mq = inputs(more)
    slots, ys = table(3, 0, -1, 4, 1, 2), []
    rows = [3, 0, 0, 4, 1, 2]                                        # which of the 5 streams a row decodes
    for t in range(steps):
        if t == 3:                                                   # slot 1 ends; slot 4 moves down into its place
            ssd.state_move(pool, table(0, 4, 2, 3, -1, 5))
            slots = table(3, 0, -1, 1, -1, 2)
        ys.append(ssd.linear_step(pool, mv[rows, t], g, mk[rows, t], mq[rows, t], slots=slots))
    torch.cuda.synchronize()
    y = f64(torch.stack(ys, 1))
    assert not y[2].any() and not y[4, 3:].any() and not pool[4].any()
    for row, stream, last in ((0, 3, steps), (1, 0, steps), (3, 4, steps), (4, 1, 3), (5, 2, steps)):
        s = np.s_[:, cu[owner[stream]]:cu[owner[stream] + 1]]
        whole = [np.concatenate([d[n][s], more[n][stream:stream + 1, :last]], 1) for n in ("v", "k", "q")]
        (yr, _), (ym, _) = ref.forward(whole[0], d["g"], whole[1], whole[2])
        n = whole[0].shape[1]
        over = np.abs(y[row, :last] - yr[0, -last:]) / (y_unit(dt, n, N, P) * ym[0, -last:])
        assert over.max() <= 1


# ---- sizes at which rows are cut -------------------------------------------------------------------------

# (batch, seqlen, nheads, headdim, dstate, ngroups, dtype): more walks than CUs, so that segments follow each other, with
# one and several slices of columns, shared keys, both types; fewer, so that they walk at once
CUT = [
    (5, 2051, 56, 16, 32, 56, "bf16"), (2, 2100, 140, 32, 16, 70, "f32"), (1, 2049, 150, 144, 32, 150, "bf16"),
    (300, 2048, 1, 16, 16, 1, "bf16"), (6, 2500, 100, 16, 16, 100, "bf16"), (2, 1500, 8, 32, 48, 4, "bf16"),
]


@pytest.mark.parametrize("c", CUT, ids=lambda c: "b{}_L{}_H{}_P{}_N{}_G{}_{}".format(*c))
def test_cut_rows(c):
    """Rows that are cut give what their heads give alone (one row and head, against the float64 recurrence, and every
    head against a call with fewer, which is cut otherwise)."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    b, L, H, P, N, G, dt = c
    gen = torch.Generator(device="cuda").manual_seed(500 + CUT.index(c))
    T = torch.bfloat16 if dt == "bf16" else torch.float32
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")        # noqa: E731
    v, k, q, dy = rand(b, L, G, P).to(T), rand(b, L, G, N).to(T), (rand(b, L, H, N) / N ** 0.5).to(T), rand(b, L, H, P).to(T)
    g = -torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H)
    init, dfinal = rand(b, H, P, N), rand(b, H, P, N)
    y, fin = ssd.linear_forward(v, g, k, q, init)
    out = ssd.linear_backward(v, g, k, q, dy, init, dfinal)
    again = ssd.linear_backward(v, g, k, q, dy, init, dfinal)
    assert all(torch.equal(out[n], again[n]) for n in out)
    m = H // G
    norm = lambda x, z: float((x.double() - z.double()).norm() / z.double().norm())        # noqa: E731
    near, last = (5.2e-3 if dt == "bf16" else 2e-6), 6e-6        # twice what the header states of each
    for i, j in ((0, 0), (b - 1, G - 1), (b // 2, G // 2)):
        hs = slice(j * m, (j + 1) * m)
        one = [t[i:i + 1, :, j:j + 1].contiguous() for t in (v, k)]
        qs, ds = (t[i:i + 1, :, hs].contiguous() for t in (q, dy))
        s0, s1 = (t[i:i + 1, hs].contiguous() for t in (init, dfinal))
        yr, fr = ssd.linear_forward(one[0], g[hs].contiguous(), one[1], qs, s0)
        assert norm(y[i:i + 1, :, hs], yr) <= near and norm(fin[i:i + 1, hs], fr) <= last
        r = ssd.linear_backward(one[0], g[hs].contiguous(), one[1], qs, ds, s0, s1)
        assert norm(out["dq"][i:i + 1, :, hs], r["dq"]) <= near and norm(out["dinit"][i:i + 1, hs], r["dinit"]) <= last
        assert norm(out["dk"][i:i + 1, :, j:j + 1], r["dk"]) <= near and norm(out["dv"][i:i + 1, :, j:j + 1], r["dv"]) <= near
    i, j = b - 1, G // 2
    (yr, Sr), (ym, Sm) = ref.forward(*(f64(t.float())[i:i + 1, :, j:j + 1] if t is not g else f64(g)[j * m:j * m + 1]
                                       for t in (v, g, k)), f64(q.float())[i:i + 1, :, j * m:j * m + 1],
                                     f64(init)[i:i + 1, j * m:j * m + 1])
    hold("y", y[i:i + 1, :, j * m:j * m + 1], yr, ym, y_unit(dt, L, N, P))
    hold("final", fin[i:i + 1, j * m:j * m + 1], Sr, Sm, state_unit(dt, L, N, P))


@pytest.mark.parametrize("lens", [[2500, 0, 1, 1024, 1025, 900, 30], [4000], [1024] * 9, [5] * 250 + [1500]],
                         ids=["mixed", "one", "whole", "many"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_varlen_in_chains(lens, dt):
    """Packed rows whose segments follow each other: each as alone, and the same as in any other cut."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    n, T = len(lens), sum(lens)
    H = -(-512 // n)
    P, N = 16, 32
    gen = torch.Generator(device="cuda").manual_seed(n)
    D = torch.bfloat16 if dt == "bf16" else torch.float32
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")        # noqa: E731
    v, k, q = rand(T, H, P).to(D), rand(T, H, N).to(D), (rand(T, H, N) / N ** 0.5).to(D)
    g = -torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H)
    h = rand(n, H, P, N)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    y, fin = ssd.linear_forward_varlen(v, g, k, q, cu, h)
    for i in sorted({0, 1, n // 2, n - 1} & set(range(n))):
        a, z = int(cu[i]), int(cu[i + 1])
        yr, fr = ssd.linear_forward(v[None, a:z], g, k[None, a:z], q[None, a:z], h[i:i + 1])
        assert float((fin[i] - fr[0]).norm()) <= 6e-6 * float(fr.norm())
        assert z == a or float((y[a:z].float() - yr[0].float()).norm()) <= (5.2e-3 if dt == "bf16" else 2e-6) * float(yr.float().norm())


@pytest.mark.parametrize("cu", [[5, 2, 90, -7, 100000], [0, 3000, 0, 3000, 0], [2900, 60, 30, 0, -1]],
                         ids=["jumps", "again", "falling"])
def test_chain_with_bad_offsets_ends(cu):
    """Offsets that overlap name more segments than there is room for: the call ends, inside its buffers."""
    import torch
    from test_gpu_guard import Guarded, _lib, _p, _stream
    T, H, P, N = 3000, 128, 16, 16
    d = ref.make(1, T, H, P, N, H, "bf16", False, seed=21)
    v, g, k, q = (t[0] if t.dim() > 1 else t for t in inputs(d))
    offsets = torch.tensor(cu, dtype=torch.int32, device="cuda")
    y, fin = Guarded((T, H, P), torch.bfloat16), Guarded((4, H, P, N), torch.float32)
    ws = Guarded((_lib().ssd_linear_forward_varlen_workspace_bytes(T, 4, H, P, N, H, 1),), torch.uint8)
    assert _lib().ssd_linear_forward_varlen(_p(v), _p(g), _p(k), _p(q), _p(offsets), 4, None, _p(y.t), _p(fin.t), T, H, P, N,
                                            H, 1, _p(ws.t), ws.n, _stream()) == 0
    torch.cuda.synchronize()
    assert y.intact() and fin.intact() and ws.intact()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_strong_decays_in_segments(dt):
    """Rows cut at once with decays that leave nothing of most of a segment, next to ones that leave all of it; and values
    so large that what little is left counts."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    L, P, N = 1400, 32, 32
    g = np.array([0.0, -0.1, -0.2, -0.5, -3.0, -90.0, -np.inf, -1e-3], np.float32)
    H = len(g)
    d = ref.make(1, L, H, P, N, H, dt, True, seed=22)
    d["g"] = g
    for at in (100, 600, 1000):
        d["v"][0, at] *= 2.0 ** 60                           # powers of two: exact in either type
    args = (d["v"], d["g"], d["k"], d["q"])
    still = (d["v"], np.zeros(H), d["k"], d["q"])
    y, fin = ssd.linear_forward(*inputs(d), dev(d["init"]))
    # a power of the decay below 2^-126 is taken as 0: a term is off by 2^-126 of what it were without decay at most
    want, (ys, Ss) = ref.forward(*args, d["init"]), ref.forward(*still, d["init"])[1]
    hold("y", y, want[0][0], want[1][0] + 2.0 ** -126 / y_unit(dt, L, N, P) * ys, y_unit(dt, L, N, P))
    hold("final", fin, want[0][1], want[1][1] + 2.0 ** -126 / state_unit(dt, L, N, P) * Ss, state_unit(dt, L, N, P))
    got = ssd.linear_backward(*inputs(d), dev(d["dy"], dt), dev(d["init"]), dev(d["dfinal"]))
    want, size = ref.backward(*args, d["dy"], d["init"], d["dfinal"])
    most = ref.backward(*still, d["dy"], d["init"], d["dfinal"])[1]
    for n, unit in (("dv", y_unit), ("dk", y_unit), ("dq", y_unit), ("dinit", state_unit), ("dg", dg_unit)):
        u = unit(dt, L, N, P)
        hold(n, got[n], want[n], size[n] + 2.0 ** -126 / u * most[n], u)


@pytest.mark.parametrize("cut", [False, True])
def test_slow_decay_does_not_drift(cut):
    """A decay next to 1 over many chunks: its power, rounded alike every time, would be off by up to 2^-25 a chunk, 6e-6 here.
    A chunk rounds the state once where it decays and, in fp32, once for each of its 32 tokens, which a matrix product adds to
    the accumulator one by one: 33 roundings of 2^-24 at most in each of 188 chunks, which in the 2-norm, their signs being
    random, are 2^-24 sqrt(6204) = 4.7e-6 at most."""
    import mamba_ssd_sequence_chunked_amd as ssd
    L, P, N = 6000, 16, 16
    H = 300 if not cut else 3
    d = ref.make(1, L, 3, P, N, 3, "f32", True, seed=23)
    d["g"] = np.array([-1e-5, -3.3e-6, -7e-5], np.float32)
    d["init"] *= 300                                          # what is carried from the start counts most
    if not cut:
        for n in ("v", "k", "q"):
            d[n] = np.tile(d[n], (1, 1, H // 3, 1))
        d["g"], d["init"] = np.tile(d["g"], H // 3), np.tile(d["init"], (1, H // 3, 1, 1))
    _, fin = ssd.linear_forward(*inputs(d), dev(d["init"]))
    (_, S), _ = ref.forward(d["v"][:, :, :3], d["g"][:3], d["k"][:, :, :3], d["q"][:, :, :3], d["init"][:, :3])
    for h in range(3):
        assert rel2(fin[:, h::3], np.tile(S[:, h:h + 1], (1, H // 3, 1, 1))) <= 2.0 ** -24 * 6204 ** 0.5
