"""The gated delta rule's entry points against the float64 recurrence (delta_ref).

Tolerances, fixed before the first run.  A rounding moves a value by at most half a step, ROUND relative to it;
fp32 sums of n terms by at most n half steps of their magnitudes.

 * the state (final states, and what y reads): for fp32 inputs every product sums at most N + 32 terms and there
   are fewer than 32 further roundings per token; for bf16 inputs four operands on the way into the state (the
   state and the solved values of a block, the block's triangular inverse, the update) are pairs of bf16 values,
   each off by at most ROUND[bf16]^2.  Each token may add that much of drift.
 * y: three bf16 operands (state, scores, update) and y's own rounding; for fp32 inputs as many fp32 roundings.
"""
import numpy as np
import pytest

import delta_ref as ref

pytestmark = pytest.mark.gpu

ROUND = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def state_unit(dtype, N):
    sums = (N + 64) * ROUND["f32"]
    return sums + (4 * ROUND["bf16"] ** 2 if dtype == "bf16" else 0.0)


def y_unit(dtype, N):
    return 4 * ROUND[dtype] + (N + 64) * ROUND["f32"]


def dev(a, dtype="f32"):
    import torch
    if a is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(a)).to("cuda")
    return t.to(torch.bfloat16 if dtype == "bf16" else torch.float32)


def inputs(d):
    t = d["dtype"]
    return [dev(d["v"], t), dev(d["g"]), dev(d["beta"]), dev(d["k"], t), dev(d["q"], t)]


def f64(t):
    return t.detach().cpu().double().numpy()


def check(y, fin, want, dtype, N, qn=None):
    yr, Sr, sy, drift = want
    y, fin = f64(y), f64(fin)
    assert np.isfinite(y).all() and np.isfinite(fin).all()
    su = state_unit(dtype, N)
    over = np.abs(fin - Sr) / (su * drift[..., None] + 2.0 ** -120)
    assert over.size == 0 or over.max() <= 1, ("final", over.max())
    # y also carries the state's error, at most su drift |q| (drift up to the last token bounds none of the
    # earlier ones, so the largest sum over a row is used)
    room = y_unit(dtype, N) * sy + su * sy.max(axis=1, keepdims=True, initial=0) * y.shape[1] + 2.0 ** -120
    over = np.abs(y - yr) / room
    assert over.size == 0 or over.max() <= 1, ("y", over.max())


# (batch, seqlen, nheads, headdim, dstate, ngroups, dtype, init, kind)
CASES = [
    (1, 1, 1, 16, 16, 1, "f32", False, "layer"),
    (2, 1, 2, 64, 128, 1, "bf16", True, "layer"),
    (1, 2, 3, 32, 16, 3, "bf16", False, "layer"),
    (2, 31, 4, 16, 32, 2, "f32", True, "layer"),
    (2, 32, 4, 64, 128, 1, "bf16", False, "layer"),
    (1, 33, 2, 128, 64, 1, "bf16", True, "layer"),
    (3, 63, 5, 64, 48, 5, "bf16", True, "layer"),
    (1, 64, 6, 32, 256, 2, "f32", True, "layer"),
    (2, 65, 3, 128, 256, 1, "bf16", True, "layer"),
    (1, 130, 2, 128, 256, 2, "f32", False, "layer"),
    (2, 257, 4, 64, 128, 2, "bf16", True, "layer"),
    (1, 300, 7, 16, 240, 7, "bf16", False, "layer"),
    (2, 95, 2, 64, 80, 1, "f32", True, "strong"),
    (2, 160, 4, 64, 128, 1, "bf16", True, "strong"),
    (2, 130, 2, 32, 64, 1, "f32", True, "resets"),
    (2, 130, 6, 64, 128, 3, "bf16", True, "resets"),
    (1, 100, 2, 32, 64, 1, "f32", True, "repeat"),
    (1, 100, 2, 64, 128, 1, "bf16", True, "repeat"),
    (1, 1000, 3, 64, 128, 1, "bf16", True, "layer"),
]


def ident(c):
    return "b{}_L{}_H{}_P{}_N{}_G{}_{}_{}_{}".format(*c)


@pytest.mark.parametrize("c", CASES, ids=ident)
def test_forward(c):
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    b, L, H, P, N, G, dt, init, kind = c
    d = ref.make(b, L, H, P, N, G, dt, init, seed=100 + CASES.index(c), kind=kind)
    y, fin = ssd.delta_forward(*inputs(d), dev(d["init"]))
    torch.cuda.synchronize()
    check(y, fin, ref.forward(d["v"], d["g"], d["beta"], d["k"], d["q"], d["init"]), dt, N)


def test_forward_keeps_fp32_accuracy_for_bf16_inputs():
    """The header's statement on the final states, in the 2-norm."""
    import mamba_ssd_sequence_chunked_amd as ssd
    d = ref.make(2, 700, 4, 64, 128, 2, "bf16", True, seed=5)
    _, fin = ssd.delta_forward(*inputs(d), dev(d["init"]))
    S = ref.forward(d["v"], d["g"], d["beta"], d["k"], d["q"], d["init"])[1]
    assert np.linalg.norm(f64(fin) - S) <= 1e-5 * np.linalg.norm(S)


def test_forward_empty_and_no_batch():
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    d = ref.make(2, 0, 4, 32, 64, 2, "bf16", True, seed=6)
    y, fin = ssd.delta_forward(*inputs(d), dev(d["init"]))
    assert y.shape == (2, 0, 4, 32) and torch.equal(fin, dev(d["init"]))
    assert torch.count_nonzero(ssd.delta_forward(*inputs(d))[1]) == 0
    d = ref.make(0, 5, 4, 32, 64, 2, "f32", seed=6)
    y, fin = ssd.delta_forward(*inputs(d))
    assert y.numel() == 0 and fin.shape == (0, 4, 32, 64)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_forward_split_and_resumed(dt):
    """Running a sequence in pieces, each from the last one's final state, gives the whole run."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    d = ref.make(2, 150, 4, 64, 96, 2, dt, True, seed=8)
    x = inputs(d)
    S, ys = dev(d["init"]), []
    for a, z in ((0, 1), (1, 40), (40, 104), (104, 150)):
        y, S = ssd.delta_forward(*(t[:, a:z].contiguous() for t in x), S)
        ys.append(y)
    check(torch.cat(ys, 1), S, ref.forward(d["v"], d["g"], d["beta"], d["k"], d["q"], d["init"]), dt, 96)


def test_forward_is_causal_by_blocks_and_confined():
    """A NaN reaches at most its own 32-token block and what follows, in its head's group only."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    d = ref.make(2, 100, 4, 64, 64, 2, "bf16", False, seed=9)
    x = inputs(d)
    y0, f0 = ssd.delta_forward(*x)
    x[3][1, 70, 1] = float("nan")                # a key of row 1, group 1 (heads 2, 3)
    y1, f1 = ssd.delta_forward(*x)
    assert torch.equal(y1[0], y0[0]) and torch.equal(f1[0], f0[0])
    assert torch.equal(y1[1, :, :2], y0[1, :, :2]) and torch.equal(f1[1, :2], f0[1, :2])
    assert torch.equal(y1[1, :64], y0[1, :64])
    assert torch.isnan(y1[1, 96:, 2:]).all() and torch.isnan(f1[1, 2:]).all()


def test_forward_repeats_bit_for_bit():
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    d = ref.make(2, 333, 6, 64, 128, 2, "bf16", True, seed=10)
    x, h = inputs(d), dev(d["init"])
    a = ssd.delta_forward(*x, h)
    for _ in range(3):
        b = ssd.delta_forward(*x, h)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ---- packed sequences -------------------------------------------------------------------------------

VARLEN = [
    # (lengths, nheads, headdim, dstate, ngroups, dtype, init)
    ([1], 2, 16, 16, 1, "f32", True),
    ([0, 5, 0, 0, 33, 1, 0], 3, 32, 48, 3, "bf16", True),
    ([32, 64, 31, 33, 96], 4, 64, 128, 2, "bf16", False),
    ([1] * 40, 2, 64, 64, 1, "f32", False),
    ([7, 200, 3, 77], 2, 128, 256, 1, "bf16", True),
    ([0, 0], 2, 16, 32, 1, "bf16", True),
    ([150, 1, 2, 64], 5, 16, 96, 5, "f32", True),
]


@pytest.mark.parametrize("c", VARLEN, ids=lambda c: "n{}_T{}_H{}_P{}_N{}_G{}_{}_{}".format(len(c[0]), sum(c[0]), *c[1:]))
def test_varlen(c):
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    lens, H, P, N, G, dt, init = c
    T = sum(lens)
    d = ref.make(1, T, H, P, N, G, dt, False, seed=300 + VARLEN.index(c))
    r = np.random.default_rng(3)
    h0 = (0.3 * r.standard_normal((len(lens), H, P, N))).astype(np.float32).astype(np.float64) if init else None
    cu = np.concatenate([[0], np.cumsum(lens)])
    y, fin = ssd.delta_forward_varlen(*(t[0] for t in inputs(d)), torch.tensor(cu, dtype=torch.int32, device="cuda"),
                                      dev(h0))
    torch.cuda.synchronize()
    assert y.shape == (T, H, P) and fin.shape == (len(lens), H, P, N)
    for i, n in enumerate(lens):
        part = [d[x][:, cu[i]:cu[i + 1]] for x in ("v", "g", "beta", "k", "q")]
        want = ref.forward(*part, None if h0 is None else h0[i:i + 1])
        check(y[None, cu[i]:cu[i + 1]], fin[i:i + 1], want, dt, N)


def test_varlen_of_equal_lengths_is_the_batch():
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    d = ref.make(3, 70, 4, 64, 128, 2, "bf16", True, seed=12)
    x, h = inputs(d), dev(d["init"])
    y, fin = ssd.delta_forward(*x, h)
    cu = torch.arange(4, dtype=torch.int32, device="cuda") * 70
    yv, fv = ssd.delta_forward_varlen(*(t.reshape(210, *t.shape[2:]) for t in x), cu, h)
    assert torch.equal(yv.reshape(y.shape), y) and torch.equal(fv, fin)


# ---- one token --------------------------------------------------------------------------------------

STEPS = [
    (1, 1, 16, 16, 1, "f32"),
    (3, 4, 32, 48, 2, "bf16"),
    (5, 3, 64, 128, 3, "bf16"),
    (2, 8, 128, 256, 2, "f32"),
    (7, 2, 64, 240, 1, "bf16"),
    (4, 5, 16, 64, 5, "f32"),
]


@pytest.mark.parametrize("c", STEPS, ids=["b{}_H{}_P{}_N{}_G{}_{}".format(*c) for c in STEPS])
def test_steps(c):
    """Twelve tokens, the state carried: fp32 arithmetic for both input types."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    b, H, P, N, G, dt = c
    d = ref.make(b, 12, H, P, N, G, dt, True, seed=500 + STEPS.index(c), kind="resets")
    x, S = inputs(d), dev(d["init"])
    ys = [ssd.delta_step(S, *(t[:, i].contiguous() for t in x)) for i in range(12)]
    torch.cuda.synchronize()
    yr, Sr, sy, drift = ref.forward(d["v"], d["g"], d["beta"], d["k"], d["q"], d["init"])
    su = state_unit("f32", N)
    assert (np.abs(f64(S) - Sr) <= su * drift[..., None]).all()
    room = (ROUND[dt] + su) * sy + 12 * su * sy.max(axis=1, keepdims=True)
    assert (np.abs(f64(torch.stack(ys, 1)) - yr) <= room).all()


def test_prefill_then_decode():
    """A prefill's final state is where decoding goes on: the run as a server makes it."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    d = ref.make(2, 75, 4, 64, 128, 1, "bf16", False, seed=14)
    x = inputs(d)
    y, S = ssd.delta_forward(*(t[:, :60].contiguous() for t in x))
    ys = [y] + [ssd.delta_step(S, *(t[:, i].contiguous() for t in x))[:, None] for i in range(60, 75)]
    check(torch.cat(ys, 1), S, ref.forward(d["v"], d["g"], d["beta"], d["k"], d["q"]), "bf16", 128)


# ---- gradients --------------------------------------------------------------------------------------

# (batch, seqlen, nheads, headdim, dstate, ngroups, dtype, init, kind)
GRADS = [
    (1, 1, 1, 16, 16, 1, "f32", False, "layer"),
    (2, 1, 2, 64, 128, 1, "bf16", True, "layer"),
    (2, 2, 3, 32, 16, 3, "bf16", False, "layer"),
    (2, 33, 4, 16, 48, 2, "f32", True, "layer"),
    (1, 64, 6, 64, 128, 1, "bf16", False, "layer"),
    (2, 65, 2, 128, 64, 1, "bf16", True, "layer"),
    (1, 97, 5, 64, 80, 5, "f32", False, "layer"),
    (2, 129, 4, 64, 128, 2, "bf16", True, "layer"),
    (1, 200, 3, 128, 256, 1, "bf16", True, "layer"),
    (1, 130, 2, 128, 256, 2, "f32", True, "layer"),
    (3, 260, 8, 32, 240, 1, "bf16", False, "layer"),
    (1, 128, 20, 16, 32, 1, "f32", True, "layer"),
    (2, 140, 4, 64, 128, 1, "bf16", True, "strong"),
    (2, 140, 4, 32, 64, 2, "f32", True, "resets"),
    (2, 140, 6, 64, 128, 2, "bf16", True, "resets"),
    (1, 70, 2, 32, 64, 1, "f32", True, "repeat"),
    (1, 700, 4, 64, 128, 1, "bf16", True, "layer"),
]


def grads(d):
    import mamba_ssd_sequence_chunked_amd as ssd
    return ssd.delta_backward(*inputs(d), dev(d["dy"], d["dtype"]), dev(d["init"]), dev(d["dfinal"]))


def rel2(a, b):
    return np.linalg.norm(a - b) / max(np.linalg.norm(b), 1e-300) if a.size else 0.0


@pytest.mark.parametrize("c", GRADS, ids=ident)
def test_backward(c):
    """In the 2-norm: fp32 gradients to four of the state's units, the others to their three operands' and their own
    rounding."""
    import torch
    b, L, H, P, N, G, dt, init, kind = c
    d = ref.make(b, L, H, P, N, G, dt, init, seed=700 + GRADS.index(c), kind=kind)
    got = grads(d)
    torch.cuda.synchronize()
    want = ref.backward(d["v"], d["g"], d["beta"], d["k"], d["q"], d["dy"], d["init"], d["dfinal"])
    for n, w in want.items():
        a = f64(got[n])
        assert a.shape == w.shape and np.isfinite(a).all(), n
        tol = 4 * state_unit(dt, N) + (4 * ROUND["bf16"] if dt == "bf16" and n in ("dv", "dk", "dq") else 0.0)
        e = rel2(a, w)
        print(f"{n} {e:.2e}", flush=True)
        assert (a == 0).all() if not w.any() else e <= tol, (n, e, tol)


def test_backward_keeps_fp32_accuracy_for_bf16_inputs():
    d = ref.make(2, 600, 4, 64, 128, 2, "bf16", True, seed=31)
    got = grads(d)
    want = ref.backward(d["v"], d["g"], d["beta"], d["k"], d["q"], d["dy"], d["init"], d["dfinal"])
    for n in ("dg", "dbeta", "dinit"):
        assert rel2(f64(got[n]), want[n]) <= 1e-5, n


def test_backward_against_differences():
    """The gradients of the GPU's forward, by the GPU's backward: a step along a random direction."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    d = ref.make(2, 45, 4, 16, 32, 2, "f32", True, seed=32)
    got = {n: f64(t) for n, t in grads(d).items()}

    def loss(x):
        y, S = ssd.delta_forward(*inputs(x), dev(x["init"]))
        return (f64(y) * d["dy"]).sum() + (f64(S) * d["dfinal"]).sum()

    r = np.random.default_rng(1)
    for n in ("v", "g", "beta", "k", "q", "init"):
        step = 1e-2 * r.standard_normal(d[n].shape)
        up, dn = dict(d), dict(d)
        up[n], dn[n] = d[n] + step, d[n] - step
        slope = (got["d" + n] * step).sum()
        # the third-order term is about step^2 of the slope's terms; fp32 losses of about 30 differ by 1e-5
        assert abs((loss(up) - loss(dn)) / 2 - slope) <= 2e-3 * np.linalg.norm(got["d" + n]) * np.linalg.norm(step) + 1e-4, n


def test_backward_empty():
    import torch
    d = ref.make(2, 0, 4, 32, 64, 2, "bf16", True, seed=33)
    got = grads(d)
    assert torch.equal(got["dinit"], dev(d["dfinal"])) and got["dk"].shape == (2, 0, 2, 64)
    assert grads(ref.make(0, 9, 4, 32, 64, 2, "f32", seed=33))["dinit"].numel() == 0


def test_backward_repeats_bit_for_bit():
    import torch
    d = ref.make(2, 150, 8, 64, 128, 1, "bf16", True, seed=34)
    a, b = grads(d), grads(d)
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_training_step_captured_and_replayed():
    """Forward and backward of one step in a graph, replayed on new inputs with eager work between."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    shape = (2, 130, 4, 64, 64, 1, "bf16", True)

    def hand(seed):
        d = ref.make(*shape, seed=seed)
        return inputs(d) + [dev(d["dy"], "bf16"), dev(d["init"]), dev(d["dfinal"])]

    x = hand(40)

    def run():
        return list(ssd.delta_forward(*x[:5], x[6])) + list(ssd.delta_backward(*x).values())

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for k in range(3):
        for t, n in zip(x, hand(41 + k)):
            t.copy_(n)
        want = [t.clone() for t in run()]
        torch.cuda.synchronize()
        print(f"replay {k}", flush=True)
        graph.replay()
        torch.cuda.synchronize()
        for a, w in zip(out, want):
            assert torch.equal(a, w), k


# ---- streams and graphs -----------------------------------------------------------------------------

def test_on_another_stream():
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    d = ref.make(2, 200, 4, 64, 128, 1, "bf16", True, seed=15)
    x, h = inputs(d), dev(d["init"])
    y0, f0 = ssd.delta_forward(*x, h)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y1, f1 = ssd.delta_forward(*x, h)
    s.synchronize()
    assert torch.equal(y0, y1) and torch.equal(f0, f1)


def test_captured_and_replayed():
    """A prefill and four decoding steps in one graph, replayed on new inputs with eager work between."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    shape = (2, 90, 4, 64, 128, 2, "bf16", True)
    x = inputs(ref.make(*shape, seed=20))
    h = dev(ref.make(*shape, seed=20)["init"])

    def run():
        y, S = ssd.delta_forward(*(t[:, :86].contiguous() for t in x), h)
        return [y, S] + [ssd.delta_step(S, *(t[:, i].contiguous() for t in x)) for i in range(86, 90)]

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for k in range(3):
        d = ref.make(*shape, seed=21 + k)
        for t, n in zip(x, inputs(d)):
            t.copy_(n)
        h.copy_(dev(d["init"]))
        want = [t.clone() for t in run()]
        torch.cuda.synchronize()
        print(f"replay {k}", flush=True)
        graph.replay()
        torch.cuda.synchronize()
        for a, w in zip(out, want):
            assert torch.equal(a, w), k
