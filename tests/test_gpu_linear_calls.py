"""Calls of linear attention and of state_move that their documentation allows: guard bands around every output and the
workspace, captured and replayed calls, two streams at once, one tensor in two places, a workspace kept by the caller,
offsets past 32 bits, and the views that are refused."""
import numpy as np
import pytest

import linear_ref as ref
from test_gpu_delta_guard import call, typed
from test_gpu_guard import Guarded, _code, _lib, _p, _stream
from test_gpu_linear import ROUND, check, dev, dg_unit, hold, inputs, state_unit, y_unit

pytestmark = pytest.mark.gpu

# (batch, seqlen, nheads, headdim, dstate, ngroups, dtype, init): odd sizes, cut rows, shared keys, wide rows
SHAPES = [
    (2, 77, 6, 64, 128, 2, "bf16", True), (1, 33, 5, 16, 48, 1, "f32", False), (3, 129, 3, 80, 80, 3, "bf16", False),
    (1, 95, 2, 256, 256, 1, "f32", True), (1, 700, 2, 144, 240, 2, "bf16", True), (1, 31, 270, 64, 128, 5, "bf16", False),
    (2, 2049, 150, 16, 16, 150, "bf16", True), (1, 300, 3, 32, 16, 3, "f32", True),
]
IDS = ["b{}_L{}_H{}_P{}_N{}_G{}_{}_i{}".format(*c) for c in SHAPES]


def make(c, seed):
    b, L, H, P, N, G, dt, init = c
    return ref.make(b, L, H, P, N, G, dt, init, seed=seed + SHAPES.index(c))


@pytest.mark.parametrize("c", SHAPES, ids=IDS)
def test_forward_and_varlen_guards(c):
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    b, L, H, P, N, G, dt, init = c
    d = make(c, 700)
    (v, g, k, q), h, lib, code = inputs(d), dev(d["init"]), _lib(), _code(dt)
    y, fin = Guarded((b, L, H, P), typed(dt)), Guarded((b, H, P, N), torch.float32)
    ws = Guarded((lib.ssd_linear_forward_workspace_bytes(b, L, H, P, N, G, code),), torch.uint8)
    call("ssd_linear_forward", [v, g, k, q, h], [y, fin], ws, [b, L, H, P, N, G, code])
    yr, fr = ssd.linear_forward(v, g, k, q, h)
    assert torch.equal(y.t, yr) and torch.equal(fin.t, fr)

    # one long sequence, an empty one and the rest
    cut = L // 2 + 1
    cu = torch.tensor([0, cut, cut, b * L], dtype=torch.int32, device="cuda")
    vf, kf, qf = (t.reshape(b * L, *t.shape[2:]) for t in (v, k, q))
    y, fin = Guarded((b * L, H, P), typed(dt)), Guarded((3, H, P, N), torch.float32)
    ws = Guarded((lib.ssd_linear_forward_varlen_workspace_bytes(b * L, 3, H, P, N, G, code),), torch.uint8)
    call("ssd_linear_forward_varlen", [vf, g, kf, qf, cu, 3, None], [y, fin], ws, [b * L, H, P, N, G, code])
    yr, fr = ssd.linear_forward_varlen(vf, g, kf, qf, cu)
    assert torch.equal(y.t, yr) and torch.equal(fin.t, fr)


@pytest.mark.parametrize("c", SHAPES, ids=IDS)
def test_backward_guards(c):
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    b, L, H, P, N, G, dt, init = c
    d = make(c, 720)
    (v, g, k, q), h, dy, df, T = inputs(d), dev(d["init"]), dev(d["dy"], dt), dev(d["dfinal"]), typed(dt)
    outs = dict(dv=Guarded(v.shape, T), dg=Guarded((H,), torch.float32), dk=Guarded(k.shape, T), dq=Guarded(q.shape, T),
                dinit=Guarded((b, H, P, N), torch.float32))
    ws = Guarded((_lib().ssd_linear_backward_workspace_bytes(b, L, H, P, N, G, _code(dt)),), torch.uint8)
    call("ssd_linear_backward", [v, g, k, q, h, dy, df], list(outs.values()), ws, [b, L, H, P, N, G, _code(dt)])
    want = ssd.linear_backward(v, g, k, q, dy, h, df)
    assert all(torch.equal(outs[n].t, want[n]) for n in want)


@pytest.mark.parametrize("b,H,P,N,G,dt", [(3, 5, 48, 80, 5, "bf16"), (1, 2, 256, 256, 1, "f32"), (9, 3, 16, 16, 3, "bf16")])
def test_step_and_move_guards(b, H, P, N, G, dt):
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    d = ref.make(b, 1, H, P, N, G, dt, True, seed=740)
    v, g, k, q = (t[:, 0].contiguous() if t.dim() > 1 else t for t in inputs(d))
    n = b + 2
    pool, y = Guarded((n, H, P, N), torch.float32), Guarded((b, H, P), typed(dt))
    start = torch.randn((n, H, P, N), device="cuda")
    pool.t.copy_(start)
    slots = torch.tensor([(i * 2) % n if i != 1 else -1 for i in range(b)], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    assert _lib().ssd_linear_step(_p(pool.t), _p(slots), n, _p(v), _p(g), _p(k), _p(q), _p(y.t), b, H, P, N, G, _code(dt),
                                  _stream()) == 0
    torch.cuda.synchronize()
    assert pool.intact() and y.intact()
    other = start.clone()
    assert torch.equal(ssd.linear_step(other, v, g, k, q, slots=slots), y.t) and torch.equal(other, pool.t)
    src = torch.arange(n - 1, -1, -1, dtype=torch.int32, device="cuda")
    src[0] = -1
    assert _lib().ssd_state_move(_p(pool.t), None, _p(src), 1, n, n, H * P * N, _stream()) == 0
    torch.cuda.synchronize()
    assert pool.intact() and torch.equal(pool.t[1:], other.flip(0)[1:]) and not pool.t[0].any()


def test_captured_and_replayed():
    """A forward whose rows are a chain, one that is cut at once, a packed batch with other offsets, and decoding with
    reordering, in one graph; replayed on new inputs with eager work between."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    P, N = 16, 32
    shapes = [(2, 2050, 150), (1, 1400, 4)]
    data = [[t for t in inputs(ref.make(b, L, H, P, N, H, "bf16", False, seed=760))] for b, L, H in shapes]
    T, H = 260, 4
    vl = [t[0] if t.dim() > 1 else t for t in inputs(ref.make(1, T, H, P, N, H, "bf16", False, seed=761))]
    cu = torch.tensor([0, 65, 130, 195, T], dtype=torch.int32, device="cuda")
    pool = torch.zeros((6, H, P, N), device="cuda")
    into = torch.tensor([0, 1, 2, 3, -1, -1], dtype=torch.int32, device="cuda")
    src = torch.tensor([1, 0, 2, 2, 3, -1], dtype=torch.int32, device="cuda")
    slots = torch.tensor([0, 3, 4, -1], dtype=torch.int32, device="cuda")
    tok = [t[:4].contiguous() if t.dim() > 1 else t for t in vl]

    def run():
        out = [ssd.linear_forward(*x) for x in data]
        back = ssd.linear_backward(*data[0], data[0][0])
        y, fin = ssd.linear_forward_varlen(vl[0], vl[1], vl[2], vl[3], cu)
        ssd.state_move(pool, into, source=fin)
        ssd.state_move(pool, src)
        return [t for o in out for t in o] + list(back.values()) + [y, fin, ssd.linear_step(pool, *tok, slots=slots), pool]

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for n, offsets in enumerate(([0, 1, 2, 3, T], [0, 0, 200, 200, T], [0, 33, 97, 259, T])):
        for x in data:
            x[0].copy_(torch.randn(x[0].shape, device="cuda"))
        cu.copy_(torch.tensor(offsets, dtype=torch.int32))
        want = [t.clone() for t in run()]
        torch.cuda.synchronize()
        print("replay", n, flush=True)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_streams_at_once():
    """Chains on two streams: each has its own workspace and counters."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    P, N, H = 16, 32, 160
    xs = [inputs(ref.make(2, 2048 + 7 * s, H, P, N, H, "bf16", False, seed=770 + s)) for s in range(2)]
    want = [ssd.linear_forward(*x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(ssd.linear_forward(*xs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for g in got[i] for a, b in zip(g, want[i]))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_one_tensor_in_two_places(dt):
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    d = ref.make(2, 70, 4, 64, 64, 4, dt, True, seed=780)
    v, g, k, _ = inputs(d)
    h = dev(d["init"])
    a, b = ssd.linear_forward(k, g, k, k, h), ssd.linear_forward(k, g, k.clone(), k.clone(), h)
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    a = ssd.linear_backward(v, g, k, k, v, h, h)
    b = ssd.linear_backward(v, g, k, k.clone(), v.clone(), h, h.clone())
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_workspace_of_the_callers():
    """Kept between calls of different sizes and cuts, with whatever the last call left in it; one too small is refused."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    lib = ssd.load_library()
    sizes = [(2, 2050, 150), (1, 1500, 4), (2, 2050, 150), (300, 10, 1)]
    need = [lib.ssd_linear_forward_workspace_bytes(b, L, H, 16, 32, H, ssd.SSD_BF16) for b, L, H in sizes]
    ws = torch.full((max(need),), 0xa5, dtype=torch.uint8, device="cuda")
    for b, L, H in sizes:
        x = inputs(ref.make(b, L, H, 16, 32, H, "bf16", False, seed=790))
        r, s = ssd.linear_forward(*x, workspace=ws), ssd.linear_forward(*x)
        assert torch.equal(r[0], s[0]) and torch.equal(r[1], s[1])
    x = inputs(ref.make(*sizes[0], 16, 32, sizes[0][2], "bf16", False, seed=790))
    with pytest.raises(ssd.SSDError):
        ssd.linear_forward(*x, workspace=ws[:need[0] - 1])


def test_padding_leaves_the_rest():
    """Rows of one batch with tokens behind their end that hold zeros: their outputs up to there are those of their own
    length, and their final states decay on."""
    import mamba_ssd_sequence_chunked_amd as ssd
    d = ref.make(3, 90, 4, 32, 48, 2, "bf16", True, seed=795)
    ends = (90, 41, 0)
    for row, n in enumerate(ends):
        for t in ("v", "k", "q"):
            d[t][row, n:] = 0.0
    y, fin = ssd.linear_forward(*inputs(d), dev(d["init"]))
    check(y, fin, ref.forward(d["v"], d["g"], d["k"], d["q"], d["init"]), "bf16", 90, 48, 32)
    assert not y[2].any()


def test_offsets_past_32_bits():
    """More than 2^32 bytes of q, y and a pool: the last tokens and slots are those of a call on them alone."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    b, L, H, P, N = 1, 41000, 256, 16, 256
    gen = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn((b, L, H, N), generator=gen, device="cuda", dtype=torch.bfloat16)
    k, v = (torch.randn((b, L, 1, w), generator=gen, device="cuda", dtype=torch.bfloat16) for w in (N, P))
    assert q.numel() * 2 > 2 ** 32
    g = torch.full((H,), -7.0, device="cuda")                # 200 tokens back nothing is left
    y, fin = ssd.linear_forward(v, g, k, q)
    yt, ft = ssd.linear_forward(*(t if t is g else t[:, -256:].contiguous() for t in (v, g, k, q)))
    assert torch.equal(y[:, -128:], yt[:, -128:]) or (y[:, -128:].float() - yt[:, -128:].float()).norm() <= 5.2e-3 * yt[:, -128:].float().norm()
    assert (fin - ft).norm() <= 1e-6 * ft.norm()
    del q, y, k, v
    pool = torch.zeros((34000, 8, 64, 64), device="cuda")    # 4.5 GB
    assert pool.numel() * 4 > 2 ** 32
    src = torch.full((34000,), -2, dtype=torch.int32, device="cuda")
    one = torch.randn((2, 8, 64, 64), generator=gen, device="cuda")
    src[33999], src[0], src[16500] = 1, 0, 1
    ssd.state_move(pool, src, source=one)
    assert torch.equal(pool[33999], one[1]) and torch.equal(pool[0], one[0]) and torch.equal(pool[16500], one[1])
    assert not pool[1:16500].any() and not pool[16501:33999].any()
    v, k = torch.randn((1, 8, 64), device="cuda"), torch.randn((1, 8, 64), device="cuda")
    state = one[1:2].clone()
    want = ssd.linear_step(state, v, g[:8].contiguous(), k, k)
    got = ssd.linear_step(pool, v, g[:8].contiguous(), k, k, slots=torch.tensor([33999], dtype=torch.int32, device="cuda"))
    assert torch.equal(got, want) and torch.equal(pool[33999], state[0])


def test_views_that_are_refused():
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    d = ref.make(2, 40, 4, 32, 64, 2, "f32", True, seed=798)
    v, g, k, q = inputs(d)
    with pytest.raises(ValueError):                          # strided: every second token
        ssd.linear_forward(v[:, ::2], g, k[:, ::2], q[:, ::2])
    flat = torch.empty(v.numel() + 1, device="cuda")
    off = flat[1:].view(v.shape)                             # 4 bytes off
    off.copy_(v)
    with pytest.raises(ssd.SSDError):
        ssd.linear_forward(off, g, k, q)
    pool = torch.zeros((4, 4, 32, 64), device="cuda")
    rows = [t[:, 0].contiguous() for t in (v, k, q)]
    with pytest.raises(ValueError):                          # slots in 64 bits
        ssd.linear_step(pool, rows[0], g, rows[1], rows[2], slots=torch.tensor([0, 1], device="cuda"))
    with pytest.raises(ValueError):                          # a view of every second slot
        ssd.state_move(torch.zeros((8, 4, 32, 64), device="cuda")[::2], torch.zeros(4, dtype=torch.int32, device="cuda"))
    with pytest.raises(ssd.SSDError):                        # a pool moved into itself by name
        ssd.state_move(pool, torch.zeros(4, dtype=torch.int32, device="cuda"), source=pool)
    with pytest.raises(ssd.SSDError):                        # y in the states
        ssd.linear_step(pool, rows[0], g, rows[1], rows[2], slots=torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                        y=pool.view(-1)[:256].view(2, 4, 32))


def packed(lens, H, P, N, dt, seed):
    """Inputs of a packed batch, and its offsets."""
    import torch
    v, g, k, q = inputs(ref.make(1, sum(lens), H, P, N, H, dt, False, seed=seed))
    return v[0], g, k[0], q[0], torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("lens,H", [([1700] * 30 + [1] * 95 + [0] * 5 + [1650] * 30 + [40] * 95, 2), ([33] * 40, 16), ([400, 370] * 5, 30),
                                    ([2000, 40, 1100], 3), ([700, 300], 3), ([31] * 300, 4)],
                         ids=["chain255", "short", "chain", "cut", "whole", "many"])
def test_packed_rows_alone(lens, H):
    """Rows of a packed batch, run whole, cut at once and in chains, against each row by itself."""
    import mamba_ssd_sequence_chunked_amd as ssd
    P = N = 16
    v, g, k, q, cu = packed(lens, H, P, N, "f32", 800)
    y, fin = ssd.linear_forward_varlen(v, g, k, q, cu)
    ends = np.cumsum([0] + lens)
    for i in sorted(set(range(0, len(lens), max(1, len(lens) // 12))) | {len(lens) - 1}):
        at = slice(ends[i], ends[i + 1])
        a, b = ssd.linear_forward(v[None, at].contiguous(), g, k[None, at].contiguous(), q[None, at].contiguous())
        # fp32 on both sides: 33 roundings of 2^-24 a chunk, in at most 54 chunks, of random signs
        limit = 2 * 2.0 ** -24 * (33 * 54) ** 0.5
        assert (y[at] - a[0]).norm() <= limit * a.norm() and (fin[i] - b[0]).norm() <= limit * b.norm()


@pytest.mark.parametrize("H,T", [(60, 5000), (3, 2600), (150, 700)])
def test_captured_packed_with_other_offsets(H, T):
    """A chain, rows cut at once, and whole ones, captured with one set of offsets and replayed with others."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    v, g, k, q, cu = packed([T // 5] * 5, H, 16, 32, "bf16", 810)
    ssd.linear_forward_varlen(v, g, k, q, cu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ssd.linear_forward_varlen(v, g, k, q, cu)
    for offsets in ([0, T, T, T, T, T], [0, 1, 2, 3, 4, T], [0, 0, 0, T // 2, T, T], [0, T // 3, T // 3, T // 2, T - 1, T]):
        cu.copy_(torch.tensor(offsets, dtype=torch.int32))
        q.normal_()
        want = ssd.linear_forward_varlen(v, g, k, q, cu)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("b,L,H,G,dt", [(1, 40, 9, 3, "bf16"), (1, 2100, 3, 3, "bf16"), (1, 300, 5, 1, "f32"), (2, 2048, 75, 75, "bf16")])
@pytest.mark.parametrize("P,N", [(16, 32), (32, 48), (64, 16), (48, 112), (128, 64), (112, 128), (16, 144)])
def test_backward_of_each_width(b, L, H, G, P, N, dt):
    """Every pairing of the widths that the backward's walks are made for: whole rows, rows cut at once and chains.  The
    last group's heads against the formulas, and the call again."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    d = ref.make(b, L, H, P, N, G, dt, True, seed=820)
    (v, g, k, q), h, dy, df = inputs(d), dev(d["init"]), dev(d["dy"], dt), dev(d["dfinal"])
    got = ssd.linear_backward(v, g, k, q, dy, h, df)
    again = ssd.linear_backward(v, g, k, q, dy, h, df)
    assert all(torch.equal(got[n], again[n]) for n in got)
    m = H // G
    want, size = ref.backward(d["v"][:, :, -1:], d["g"][-m:], d["k"][:, :, -1:], d["q"][:, :, -m:], d["dy"][:, :, -m:],
                              d["init"][:, -m:], d["dfinal"][:, -m:])
    hold("dv", got["dv"][:, :, -1:], want["dv"], size["dv"], y_unit(dt, L, N, P))
    hold("dk", got["dk"][:, :, -1:], want["dk"], size["dk"], y_unit(dt, L, N, P))
    hold("dq", got["dq"][:, :, -m:], want["dq"], size["dq"], y_unit(dt, L, N, P))
    hold("dinit", got["dinit"][:, -m:], want["dinit"], size["dinit"], state_unit(dt, L, N, P))
    hold("dg", got["dg"][-m:], want["dg"], size["dg"], dg_unit(dt, L, N, P) + b * ROUND["f32"])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("L", [40, 3000])
def test_nan_decay_shows_in_its_head(L, dt):
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    H, P, N, G = 4, 32, 48, 2
    v, g, k, q = inputs(ref.make(1, L, H, P, N, G, dt, False, seed=830))
    bad = g.clone()
    bad[1] = float("nan")                                    # of heads 0 and 1, which share a key
    rest = torch.tensor([0, 2, 3], device="cuda")
    (y, fin), (yr, fr) = ssd.linear_forward(v, bad, k, q), ssd.linear_forward(v, g, k, q)
    assert y[:, :, 1].isnan().all() and fin[:, 1].isnan().all()
    assert torch.equal(y[:, :, rest], yr[:, :, rest]) and torch.equal(fin[:, rest], fr[:, rest])
    b, br = ssd.linear_backward(v, bad, k, q, yr), ssd.linear_backward(v, g, k, q, yr)
    assert b["dg"][1].isnan() and b["dinit"][:, 1].isnan().all() and b["dq"][:, :, 1].isnan().all()
    assert b["dk"][:, :, 0].isnan().all() and b["dv"][:, :, 0].isnan().all()
    assert all(torch.equal(b[n][:, :, 1], br[n][:, :, 1]) for n in ("dk", "dv")) and torch.equal(b["dg"][rest], br["dg"][rest])
    one = [t[:, 0].contiguous() for t in (v, k, q)]
    s, sr = torch.ones((1, H, P, N), device="cuda"), torch.ones((1, H, P, N), device="cuda")
    y, yr = ssd.linear_step(s, one[0], bad, one[1], one[2]), ssd.linear_step(sr, one[0], g, one[1], one[2])
    assert y[:, 1].isnan().all() and s[:, 1].isnan().all()
    assert torch.equal(y[:, rest], yr[:, rest]) and torch.equal(s[:, rest], sr[:, rest])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_widest_rows(dt):
    """A token's row of 2^20 elements, the most that is taken: each head as by itself."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    H, P, N, L, T = 4096, 256, 256, 37, typed(dt)
    gen = torch.Generator(device="cuda").manual_seed(7)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda", dtype=T)          # noqa: E731
    v, k, q, dy = rand(1, L, H // 2, P), rand(1, L, H // 2, N), rand(1, L, H, N), rand(1, L, H, P)
    g = -torch.rand(H, generator=gen, device="cuda")
    y, fin = ssd.linear_forward(v, g, k, q)
    for h in (0, 4095, 2047):
        pick = lambda t, i: t[:, :, i:i + 1].contiguous()                            # noqa: E731
        a, b = ssd.linear_forward(pick(v, h // 2), g[h:h + 1].contiguous(), pick(k, h // 2), pick(q, h))
        assert torch.equal(y[:, :, h:h + 1], a) and torch.equal(fin[:, h:h + 1], b)
    del y, fin
    got = ssd.linear_backward(v, g, k, q, dy)
    for h in (0, 4094):
        pair = lambda t: t[:, :, h:h + 2].contiguous()                               # noqa: E731
        one = ssd.linear_backward(pick(v, h // 2), g[h:h + 2].contiguous(), pick(k, h // 2), pair(q), pair(dy))
        assert torch.equal(got["dq"][:, :, h:h + 2], one["dq"]) and torch.equal(got["dinit"][:, h:h + 2], one["dinit"])
        assert torch.equal(got["dk"][:, :, h // 2:h // 2 + 1], one["dk"]) and torch.equal(got["dv"][:, :, h // 2:h // 2 + 1], one["dv"])
        assert torch.equal(got["dg"][h:h + 2], one["dg"])
    with pytest.raises(ssd.SSDError):                        # 2^20 + 256
        ssd.linear_forward(*(torch.empty(s, dtype=T, device="cuda") if len(s) > 1 else torch.zeros(s, device="cuda")
                             for s in ((1, 1, 1, P), (H + 1,), (1, 1, 1, N), (1, 1, H + 1, N))))


def test_most_rows_of_one_token():
    """65535 rows of a token, each from its state: what a step does, forwards and back."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    b, H, P, N = 65535, 2, 16, 16
    gen = torch.Generator(device="cuda").manual_seed(8)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")                   # noqa: E731
    v, k, q, h, dy, g = rand(b, 1, 1, P), rand(b, 1, 1, N), rand(b, 1, H, N), rand(b, H, P, N), rand(b, 1, H, P), -rand(H).abs()
    y, fin = ssd.linear_forward(v, g, k, q, h)
    state = h.clone()
    ys = ssd.linear_step(state, v[:, 0], g, k[:, 0], q[:, 0])
    # the same few fp32 sums in another order: 16 terms of a token's output, each rounded twice, 2 of a state's element
    assert (y[:, 0] - ys).norm() <= 2.0 ** -24 * 33 ** 0.5 * 2 * ys.norm() and (fin - state).norm() <= 2.0 ** -22 * state.norm()
    got = ssd.linear_backward(v, g, k, q, dy, h)
    D = dy[:, 0, :, :, None].double() * q[:, 0, :, None, :].double()
    a = g.double().exp()[:, None, None]
    want = dict(dinit=a * D, dv=(D * k[:, 0, :, None, :]).sum((1, 3))[:, None, None], dk=(D * v[:, 0, :, :, None]).sum((1, 2))[:, None, None],
                dq=(dy[:, 0, :, :, None].double() * state).sum(2)[:, None], dg=(D * a * h).sum((0, 2, 3)))
    for n, w in want.items():
        # dg: a row's 256 terms, rounded 3 times each and added in fp32 in chains of 16 and a tree of 64 lanes: fewer than 64
        # roundings of at most the terms' 2-norm, their signs being random, doubled; rows are added in 64 bits
        size, count = ((D * a * h).square().sum((0, 2, 3)).sqrt().norm(), 64) if n == "dg" else (w.norm(), 33)
        assert (got[n].double() - w).norm() <= 2.0 ** -24 * count ** 0.5 * 2 * size, n


@pytest.mark.parametrize("b,L,H,P,N,G", [(1, 22, 1, 64, 240, 1), (5, 32, 8, 16, 128, 4), (7, 1, 14, 48, 160, 14), (4, 393, 10, 64, 32, 2),
                                         (1, 151, 3, 64, 16, 3), (2, 2048, 150, 16, 48, 150)])
def test_gradient_of_the_decay_as_in_fp32(b, L, H, P, N, G):
    """bf16 inputs: what leads to dg keeps 2^-24 of every operand (three bf16 values), so it is off by fp32's roundings, and
    by as much again for what the three values leave."""
    import mamba_ssd_sequence_chunked_amd as ssd
    d = ref.make(b, L, H, P, N, G, "bf16", True, seed=840)
    got = ssd.linear_backward(*inputs(d), dev(d["dy"], "bf16"), dev(d["init"]), dev(d["dfinal"]))
    m = H // G
    want, size = ref.backward(d["v"][:, :, -1:], d["g"][-m:], d["k"][:, :, -1:], d["q"][:, :, -m:], d["dy"][:, :, -m:],
                              d["init"][:, -m:], d["dfinal"][:, -m:])
    hold("dg", got["dg"][-m:], want["dg"], size["dg"], 2 * dg_unit("f32", L, N, P) + b * ROUND["f32"])
