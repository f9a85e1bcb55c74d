"""Guard bands around every output and workspace of the gated delta rule's entry points, and the sizes at which the
walk shares a workgroup among heads (more than 256 workgroups of 64 columns of v).

As in test_gpu_guard: each output and the workspace is a view into a larger allocation with a canary pattern on both
sides; after the call the canaries and the inputs are unchanged and the outputs equal those of a plain call bit for
bit."""
import numpy as np
import pytest

import delta_ref as ref
from test_gpu_delta import check, dev, f64, grads, inputs, rel2, ROUND, state_unit
from test_gpu_guard import Guarded, _code, _lib, _p, _stream

pytestmark = pytest.mark.gpu

T = {"f32": "float32", "bf16": "bfloat16"}


def typed(dt):
    import torch
    return getattr(torch, T[dt])


def call(name, args, outs, ws, more):
    """Runs an entry point, then looks at the bands and the inputs."""
    import torch
    before = [None if t is None else t.clone() for t in args if isinstance(t, torch.Tensor) or t is None]
    kept = [t for t in args if isinstance(t, torch.Tensor) or t is None]
    rc = getattr(_lib(), name)(*[_p(a) if isinstance(a, torch.Tensor) or a is None else a for a in args],
                               *[_p(o.t) for o in outs], *more, *([_p(ws.t), ws.n] if ws else []), _stream())
    assert rc == 0, name
    torch.cuda.synchronize()
    assert all(o.intact() for o in outs) and (ws is None or ws.intact()), name
    for a, b in zip(kept, before):
        assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))


SHAPES = [
    # (batch, seqlen, nheads, headdim, dstate, ngroups, dtype, init)
    (2, 77, 6, 64, 128, 2, "bf16", True),
    (1, 33, 5, 16, 48, 1, "f32", False),
    (3, 129, 3, 32, 80, 3, "bf16", False),
    (1, 95, 2, 128, 256, 1, "f32", True),
    (1, 130, 18, 128, 240, 2, "bf16", True),
    (1, 31, 270, 64, 128, 5, "bf16", False),
    (3, 40, 50, 128, 64, 1, "bf16", True),
]
IDS = ["b{}_L{}_H{}_P{}_N{}_G{}_{}_i{}".format(*c) for c in SHAPES]


@pytest.mark.parametrize("c", SHAPES, ids=IDS)
def test_forward_and_varlen_guards(c):
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    b, L, H, P, N, G, dt, init = c
    d = ref.make(b, L, H, P, N, G, dt, init, seed=700 + SHAPES.index(c))
    x, h, lib, code = inputs(d), dev(d["init"]), _lib(), _code(dt)
    y, fin = Guarded((b, L, H, P), typed(dt)), Guarded((b, H, P, N), torch.float32)
    ws = Guarded((lib.ssd_delta_forward_workspace_bytes(b, L, H, P, N, G, code),), torch.uint8)
    call("ssd_delta_forward", [*x, h], [y, fin], ws, [b, L, H, P, N, G, code])
    yr, fr = ssd.delta_forward(*x, h)
    assert torch.equal(y.t, yr) and torch.equal(fin.t, fr)

    # one long sequence, an empty one and the rest
    cut = L // 2 + 1
    cu = torch.tensor([0, cut, cut, b * L], dtype=torch.int32, device="cuda")
    xf = [t.reshape(b * L, *t.shape[2:]) for t in x]
    y, fin = Guarded((b * L, H, P), typed(dt)), Guarded((3, H, P, N), torch.float32)
    ws = Guarded((lib.ssd_delta_forward_varlen_workspace_bytes(b * L, 3, H, P, N, G, code),), torch.uint8)
    call("ssd_delta_forward_varlen", [*xf, cu, 3, None], [y, fin], ws, [b * L, H, P, N, G, code])
    yr, fr = ssd.delta_forward_varlen(*xf, cu)
    assert torch.equal(y.t, yr) and torch.equal(fin.t, fr)


@pytest.mark.parametrize("cu", [[5, 2, 90, -7, 1000], [0, 0, 0, 0, 0], [90, 60, 30, 0, -1], [-2 ** 31, 2 ** 31 - 1, 0, 40, 90]],
                         ids=["jumps", "zeros", "falling", "extreme"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_varlen_bad_offsets_stay_inside(cu, dt):
    """Offsets are not checked: with any others the values are unspecified, the accesses are not."""
    import torch
    d = ref.make(1, 90, 4, 32, 64, 2, dt, False, seed=41)
    x, lib, code = [t[0] for t in inputs(d)], _lib(), _code(dt)
    offs = torch.tensor(cu, dtype=torch.int32, device="cuda")
    h = dev(0.1 * np.ones((4, 4, 32, 64)))
    y, fin = Guarded((90, 4, 32), typed(dt)), Guarded((4, 4, 32, 64), torch.float32)
    ws = Guarded((lib.ssd_delta_forward_varlen_workspace_bytes(90, 4, 4, 32, 64, 2, code),), torch.uint8)
    call("ssd_delta_forward_varlen", [*x, offs, 4, h], [y, fin], ws, [90, 4, 32, 64, 2, code])


@pytest.mark.parametrize("c", SHAPES, ids=IDS)
def test_backward_guards(c):
    import torch
    b, L, H, P, N, G, dt, init = c
    d = ref.make(b, L, H, P, N, G, dt, init, seed=800 + SHAPES.index(c))
    lib, code = _lib(), _code(dt)
    f, t = torch.float32, typed(dt)
    outs = dict(dv=Guarded((b, L, H, P), t), dg=Guarded((b, L, H), f), dbeta=Guarded((b, L, H), f),
                dk=Guarded((b, L, G, N), t), dq=Guarded((b, L, G, N), t), dinit=Guarded((b, H, P, N), f))
    ws = Guarded((lib.ssd_delta_backward_workspace_bytes(b, L, H, P, N, G, code),), torch.uint8)
    call("ssd_delta_backward", [*inputs(d), dev(d["init"]), dev(d["dy"], dt), dev(d["dfinal"])], list(outs.values()), ws,
         [b, L, H, P, N, G, code])
    want = grads(d)
    assert all(torch.equal(o.t, want[n]) for n, o in outs.items())


@pytest.mark.parametrize("c", [(3, 5, 16, 48, 5, "f32"), (5, 6, 64, 128, 2, "bf16"), (2, 3, 128, 240, 1, "bf16")],
                         ids=["f32", "bf16", "wide"])
def test_step_guards(c):
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    b, H, P, N, G, dt = c
    d = ref.make(b, 1, H, P, N, G, dt, True, seed=43)
    x, h = [t[:, 0].contiguous() for t in inputs(d)], dev(d["init"])
    S, y = Guarded((b, H, P, N), torch.float32), Guarded((b, H, P), typed(dt))
    S.t.copy_(h)
    before = [t.clone() for t in x]
    rc = _lib().ssd_delta_step(_p(S.t), *[_p(t) for t in x], _p(y.t), b, H, P, N, G, _code(dt), _stream())
    assert rc == 0
    torch.cuda.synchronize()
    assert S.intact() and y.intact() and all(torch.equal(a, z) for a, z in zip(x, before))
    yr = ssd.delta_step(h, *x)
    assert torch.equal(y.t, yr) and torch.equal(S.t, h)


MANY = [
    # more than 256 workgroups of 64 columns: pairs of heads, one head of 128 columns, and groups of an odd number of heads
    (3, 70, 100, 64, 80, 2, "bf16", True, "layer"),
    (2, 65, 70, 128, 48, 1, "bf16", False, "layer"),
    (1, 40, 265, 64, 32, 5, "bf16", True, "layer"),
    (2, 33, 130, 64, 128, 1, "bf16", True, "resets"),
]


@pytest.mark.parametrize("c", MANY, ids=["b{}_L{}_H{}_P{}_N{}_G{}_{}_{}_{}".format(*c) for c in MANY])
def test_many_heads(c):
    import mamba_ssd_sequence_chunked_amd as ssd
    b, L, H, P, N, G, dt, init, kind = c
    d = ref.make(b, L, H, P, N, G, dt, init, seed=900 + MANY.index(c), kind=kind)
    want = ref.forward(d["v"], d["g"], d["beta"], d["k"], d["q"], d["init"])
    check(*ssd.delta_forward(*inputs(d), dev(d["init"])), want, dt, N)


def test_many_heads_backward():
    """Tolerances as in test_gpu_delta.test_backward."""
    d = ref.make(1, 97, 260, 64, 48, 2, "bf16", True, seed=910)
    got = grads(d)
    want = ref.backward(d["v"], d["g"], d["beta"], d["k"], d["q"], d["dy"], d["init"], d["dfinal"])
    for n in ("dg", "dbeta", "dinit"):
        assert rel2(f64(got[n]), want[n]) <= 4 * state_unit("bf16", 48), n
    for n in ("dv", "dk", "dq"):
        assert rel2(f64(got[n]), want[n]) <= 4 * ROUND["bf16"], n


def test_offsets_past_32_bits():
    """More than 2^32 elements of v: the sequence in two parts, cut at a chunk's end, gives the same bits.

    Not so the second part's dbeta and dg: the state it starts from is the forward's, which sums three of the four
    products of two pairs, while the whole backward goes on from its own walk's, which sums all four. Each is within
    four of the state's units of the exact gradient (as in test_gpu_delta.test_backward), so they are within eight of
    each other; an offset that wrapped would be off by their whole size."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    H, P, N, L, cut = 128, 128, 16, (1 << 18) + 197, 1 << 17
    gen = torch.Generator(device="cuda").manual_seed(5)
    bf = lambda *s: torch.empty(1, L, *s, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)   # noqa: E731
    v, dy, k, q = bf(H, P), bf(H, P), bf(1, N), bf(1, N)
    assert v.numel() > 1 << 32
    k = torch.nn.functional.normalize(k.float(), dim=-1).bfloat16()
    q = torch.nn.functional.normalize(q.float(), dim=-1).bfloat16()
    g = -0.1 * torch.rand(1, L, H, device="cuda", generator=gen)
    beta = torch.rand(1, L, H, device="cuda", generator=gen)
    x = (v, g, beta, k, q)
    a, z = [t[:, :cut] for t in x], [t[:, cut:] for t in x]

    y, fin = ssd.delta_forward(*x)
    ya, mid = ssd.delta_forward(*a)
    yz, end = ssd.delta_forward(*z, mid)
    assert torch.isfinite(fin).all() and torch.equal(fin, end)
    assert torch.equal(y[:, :cut], ya) and torch.equal(y[:, cut:], yz)
    del y, ya, yz

    whole = ssd.delta_backward(*x, dy)
    back = ssd.delta_backward(*z, dy[:, cut:], mid)
    assert torch.equal(whole["dv"][:, cut:], back["dv"])
    for n in ("dbeta", "dg"):
        assert (whole[n][:, cut:] - back[n]).norm() <= 8 * state_unit("bf16", N) * back[n].norm(), n
    front = ssd.delta_backward(*a, dy[:, :cut], None, back["dinit"])
    assert torch.equal(whole["dinit"], front["dinit"])
    for n in ("dv", "dbeta", "dg"):
        assert torch.equal(whole[n][:, :cut], front[n]), n
    for n in ("dk", "dq"):               # summed over other slices of the heads: fp32 sums, rounded to bf16
        for w, p in ((whole[n][:, cut:], back[n]), (whole[n][:, :cut], front[n])):
            assert (w.float() - p.float()).norm() <= 2 * ROUND["bf16"] * p.float().norm(), n


def test_two_streams_at_once():
    """Calls that overlap in time, each on its own workspace."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    d = [ref.make(2, 700, 6, 64, 128, 2, "bf16", True, seed=50 + i) for i in range(2)]
    x = [inputs(e) for e in d]
    h = [dev(e["init"]) for e in d]
    dy = [dev(e["dy"], "bf16") for e in d]
    want = [(ssd.delta_forward(*x[i], h[i]), ssd.delta_backward(*x[i], dy[i], h[i])) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append((ssd.delta_forward(*x[i], h[i]), ssd.delta_backward(*x[i], dy[i], h[i])))
    torch.cuda.synchronize()
    for i in range(2):
        for (y, f), b in got[i]:
            assert torch.equal(y, want[i][0][0]) and torch.equal(f, want[i][0][1])
            assert all(torch.equal(b[n], want[i][1][n]) for n in b)
