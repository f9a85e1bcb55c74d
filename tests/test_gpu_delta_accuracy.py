"""How near the gated delta rule's outputs are to the float64 recurrence (delta_ref), each head for itself.

Tolerances, fixed before the first run:

 * dg: a token's value is reached by a sum of at most 64 terms of the gradient's own size from the nearer end of its chunk,
   so that errors of one term add up at random to at most 8 of them.  For bf16 inputs the term's operands are pairs of
   bf16 values, off by at most 2^-18 each, two to a product: 2^-17.  For fp32 inputs a term sums products over N and
   64 more values, whose half steps of 2^-24 add up at random: sqrt(N + 64) of them.
 * A rounding's error is spread evenly over its half step: 1 / sqrt(3) of it in the mean.  Roundings of different values
   add up at random, so a sum's error is counted in the root of its terms' squares.
 * y: for bf16 inputs its own rounding, the state's and the scores' to bf16 (each rounded once where it leads to y);
   for both types 4 times the fp32 unit: the products' sums, and those of the state that they are made from.  A score q . k
   is a sum of N products itself: rounded to bf16 it is off by half a step of its value, but as an fp32 sum by half steps
   of its terms (with |q . k| = 0.004 of unit vectors, fp32's half step of the terms' 1 / sqrt(N) is 2e-6 of the value), so
   the fp32 unit counts a score's terms and not its value.
 * dv: its own rounding; dk, dq: four, their own and those of a product's two operands in two products.
 * final states, dbeta, dg, dinit for bf16 inputs: the header's 1e-5 of the norm.  Where all keys of a row are alike and
   beta is 1, a block's 32 updates are differences of values, sqrt(2) as large as the values, and add up to one of
   them, so what is left of their 32 roundings (2^-18, of pairs) is sqrt(32) sqrt(2) = 8 of them; dk and dq then sum 64 such
   updates rounded to bf16: sqrt(64) sqrt(2) roundings.
"""
import numpy as np
import pytest

import delta_ref as ref
from test_gpu_delta import CASES, GRADS, ROUND, VARLEN, dev, f64, grads, ident, inputs, rel2
from test_gpu_delta_guard import MANY

pytestmark = pytest.mark.gpu


def dg_unit(dtype, N):
    return 8 * (2.0 ** -17 if dtype == "bf16" else np.sqrt(N + 64) * 2.0 ** -24)


def per_head(got, want):
    """The 2-norm of the difference over that of the reference, the largest of all rows and heads; (b, L, H, ...)."""
    d, w = (np.moveaxis(a, 2, 1).reshape(a.shape[0], a.shape[2], -1) for a in (got - want, want))
    d, w = np.linalg.norm(d, axis=-1), np.linalg.norm(w, axis=-1)
    assert (d[w == 0] == 0).all()
    return (d / np.where(w > 0, w, 1)).max(initial=0)


# (batch, seqlen, nheads, headdim, dstate, ngroups, dtype, states)
SHAPES = [
    (1, 256, 6, 64, 64, 2, "f32", False),
    (2, 150, 4, 64, 128, 2, "bf16", True),
    (1, 256, 5, 128, 64, 5, "bf16", False),
    (1, 97, 4, 32, 48, 1, "f32", True),
    (2, 40, 4, 16, 32, 4, "bf16", True),
    (1, 65, 3, 64, 256, 1, "bf16", True),
]


@pytest.mark.parametrize("decay", [-0.01, -0.5, -2.0, -4.0, -8.0, -15.0, -40.0])
@pytest.mark.parametrize("c", SHAPES, ids=["b{}_L{}_H{}_P{}_N{}_G{}_{}_{}".format(*c) for c in SHAPES])
def test_log_decay_gradient_of_a_steady_decay(c, decay):
    """The gradient shrinks with the decay; its error has to shrink with it."""
    b, L, H, P, N, G, dt, init = c
    d = ref.make(b, L, H, P, N, G, dt, init, seed=1200 + SHAPES.index(c))
    d["g"][:] = np.float32(decay) * np.float32(1 + 0.1 * np.random.default_rng(3).random(d["g"].shape)).astype(np.float64)
    got = f64(grads(d)["dg"])
    want = ref.backward(d["v"], d["g"], d["beta"], d["k"], d["q"], d["dy"], d["init"], d["dfinal"])["dg"]
    e = per_head(got, want)
    print(f"dg {e:.2e}", flush=True)
    assert e <= dg_unit(dt, N)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_log_decay_gradient_of_mixed_heads(dt):
    """Heads that hardly decay beside heads that forget at once, and tokens of one head that do either."""
    d = ref.make(2, 200, 6, 64, 64, 1, dt, True, seed=1220)
    for h, g in enumerate((-0.001, -0.1, -1.0, -6.0, -20.0)):
        d["g"][:, :, h] = np.float32(g)
    d["g"][:, :, 5] = np.float32(-0.05)
    d["g"][:, ::7, 5] = np.float32(-9.0)
    got = f64(grads(d)["dg"])
    want = ref.backward(d["v"], d["g"], d["beta"], d["k"], d["q"], d["dy"], d["init"], d["dfinal"])["dg"]
    e = per_head(got, want)
    print(f"dg {e:.2e}", flush=True)
    assert e <= dg_unit(dt, 64)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("reset", [-np.inf, -2000.0, -150.0])
def test_log_decay_gradient_of_a_reset_is_zero(dt, reset):
    """Nothing passes a reset, so its log decay has no gradient: not a small one, none."""
    d = ref.make(2, 130, 4, 32, 64, 2, dt, True, seed=1230)
    at = np.random.default_rng(5).random(d["g"].shape) < 0.2
    at[:, 0, 0] = at[:, -1, 1] = at[:, 63:65, 2] = True
    d["g"][at] = reset
    got = f64(grads(d)["dg"])
    assert (got[at] == 0).all()
    want = ref.backward(d["v"], d["g"], d["beta"], d["k"], d["q"], d["dy"], d["init"], d["dfinal"])["dg"]
    assert per_head(got, want) <= dg_unit(dt, 64)


# ---- y, final states and the other gradients, in the 2-norm -----------------------------------------

def fp32_unit(N):
    return np.sqrt(N + 64) * 2.0 ** -24


def mean_rounding(dtype):
    return ROUND[dtype] / np.sqrt(3)


def y_size(v, g, beta, k, q, init=None):
    """The roots of the squares of y's terms, like y: the entering state's products with q, the block's scores' with its
    updates, and y itself; and the same with the products that a score is summed from in the score's place."""
    b, L, H, P = v.shape
    K, Q = ref.heads(k, H), ref.heads(q, H)
    S = np.zeros((b, H, P, k.shape[3])) if init is None else init.copy()
    out, fine = np.zeros_like(v), np.zeros_like(v)
    for t in range(L):
        if t % ref.BLOCK == 0:
            S0, us, ks = S, [], []
        a = np.exp(g[:, t])[:, :, None]
        S0 = a[..., None] * S0
        us = [a * u for u in us]
        Sp = a[..., None] * S
        kt, qt = K[:, t, :, None, :], Q[:, t, :, None, :]
        u = beta[:, t, :, None] * (v[:, t] - (Sp * kt).sum(-1))
        S = Sp + u[..., None] * kt
        us.append(u)
        ks.append(K[:, t])
        out[:, t] = ((S0 * qt) ** 2).sum(-1) + (S * qt).sum(-1) ** 2
        fine[:, t] = out[:, t]
        for uj, kj in zip(us, ks):
            out[:, t] += ((Q[:, t] * kj).sum(-1)[..., None] * uj) ** 2
            fine[:, t] += ((Q[:, t] * kj) ** 2).sum(-1)[..., None] * uj ** 2
    return np.sqrt(out), np.sqrt(fine)


def check_y(y, want, size, dtype, N):
    """Each row and head for itself."""
    err, room, fine = (np.linalg.norm(np.moveaxis(a, 2, 1).reshape(a.shape[0], a.shape[2], -1), axis=-1)
                       for a in (f64(y) - want, *size))
    tol = 4 * fp32_unit(N) * fine + (mean_rounding("bf16") * room if dtype == "bf16" else 0.0)
    print(f"y {(err / np.maximum(tol, 1e-300)).max(initial=0):.2f} of its tolerance", flush=True)
    assert (err <= tol).all()


def state_tolerance(dtype, N, kind):
    if dtype == "f32":
        return 8 * fp32_unit(N)
    return 8 * 2.0 ** -18 if kind == "repeat" else 1e-5


REPEATS = [
    (1, 300, 4, 64, 128, 2, "bf16", False, "repeat"),
    (2, 95, 3, 128, 64, 1, "bf16", True, "repeat"),
    (1, 160, 4, 16, 256, 4, "bf16", True, "repeat"),
]


@pytest.mark.parametrize("c", CASES + MANY + REPEATS, ids=ident)
def test_forward_accuracy(c):
    import mamba_ssd_sequence_chunked_amd as ssd
    b, L, H, P, N, G, dt, init, kind = c
    d = ref.make(b, L, H, P, N, G, dt, init, seed=1300 + L, kind=kind)
    x = [d[n] for n in ("v", "g", "beta", "k", "q", "init")]
    y, fin = ssd.delta_forward(*inputs(d), dev(d["init"]))
    want = ref.forward(*x)
    check_y(y, want[0], y_size(*x), dt, N)
    e = rel2(f64(fin), want[1])
    print(f"final {e:.2e}", flush=True)
    assert e <= state_tolerance(dt, N, kind)


@pytest.mark.parametrize("c", VARLEN, ids=lambda c: "n{}_T{}_H{}_P{}_N{}_G{}_{}_{}".format(len(c[0]), sum(c[0]), *c[1:]))
def test_varlen_accuracy(c):
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    lens, H, P, N, G, dt, init = c
    d = ref.make(1, sum(lens), H, P, N, G, dt, False, seed=1400 + sum(lens))
    h0 = 0.3 * np.random.default_rng(4).standard_normal((len(lens), H, P, N)) if init else None
    h0 = None if h0 is None else h0.astype(np.float32).astype(np.float64)
    cu = np.concatenate([[0], np.cumsum(lens)])
    y, fin = ssd.delta_forward_varlen(*(t[0] for t in inputs(d)), torch.tensor(cu, dtype=torch.int32, device="cuda"), dev(h0))
    for i in range(len(lens)):
        x = [d[n][:, cu[i]:cu[i + 1]] for n in ("v", "g", "beta", "k", "q")] + [None if h0 is None else h0[i:i + 1]]
        want = ref.forward(*x)
        check_y(y[None, cu[i]:cu[i + 1]], want[0], y_size(*x), dt, N)
        e = rel2(f64(fin[i:i + 1]), want[1])
        assert e <= state_tolerance(dt, N, "layer") if want[1].any() else not f64(fin[i]).any(), (i, e)


@pytest.mark.parametrize("c", GRADS + REPEATS[1:], ids=ident)
def test_backward_accuracy(c):
    b, L, H, P, N, G, dt, init, kind = c
    d = ref.make(b, L, H, P, N, G, dt, init, seed=1500 + L, kind=kind)
    got = grads(d)
    want = ref.backward(d["v"], d["g"], d["beta"], d["k"], d["q"], d["dy"], d["init"], d["dfinal"])
    for n, w in want.items():
        tol = state_tolerance(dt, N, kind)
        if dt == "bf16" and n in ("dv", "dk", "dq"):
            many = 1 if n == "dv" else 8 * np.sqrt(2) if kind == "repeat" else 2
            tol += many * mean_rounding("bf16")
        e = rel2(f64(got[n]), w)
        print(f"{n} {e:.2e} of {tol:.2e}", flush=True)
        assert e <= tol if w.any() else not f64(got[n]).any(), n


def test_backward_confines_what_is_not_finite():
    """A NaN in dy reaches the gradients before it and those of its chunk of 64 tokens, in its row and group only."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    d = ref.make(2, 200, 4, 64, 64, 2, "bf16", True, seed=1600)
    x, dy = inputs(d), dev(d["dy"], "bf16")
    a = ssd.delta_backward(*x, dy, dev(d["init"]), dev(d["dfinal"]))
    dy[1, 70, 3] = float("nan")                  # group 1: heads 2 and 3
    b = ssd.delta_backward(*x, dy, dev(d["init"]), dev(d["dfinal"]))
    for n in a:
        assert torch.equal(a[n][0], b[n][0]), n
        if n == "dinit":
            assert torch.equal(a[n][1, :3], b[n][1, :3]) and torch.isnan(b[n][1, 3]).all()
            continue
        own = slice(1, None) if n in ("dk", "dq") else slice(3, None)
        rest = slice(0, own.start)
        assert torch.equal(a[n][1, :, rest], b[n][1, :, rest]), n
        assert torch.equal(a[n][1, 128:], b[n][1, 128:]), n
    assert torch.isnan(b["dv"][1, :71, 3]).all()


@pytest.mark.parametrize("c", [c for c in GRADS if c[6] == "bf16" and c[1] > 1] + REPEATS, ids=ident)
def test_key_and_query_gradients_accuracy(c):
    """What a rounding to bf16 is off by in the mean, counted exactly: its half step is 2^-8 / m of a value of mantissa m,
    the mean of 1 / m^2 over evenly spread logarithms 0.541, so 2^-8 sqrt(0.541 / 3) = 1.66e-3.  dk and dq are made of
    two halves, what is left of the states and the chunk's own pairs of tokens: the first's two operands are rounded, the
    second's are not, and the sum is, so 1.66e-3 sqrt(1 + 2 / 2).  Where all keys are alike the two halves cancel in
    part: two roundings more."""
    b, L, H, P, N, G, dt, init, kind = c
    d = ref.make(b, L, H, P, N, G, dt, init, seed=1700 + L, kind=kind)
    got = grads(d)
    want = ref.backward(d["v"], d["g"], d["beta"], d["k"], d["q"], d["dy"], d["init"], d["dfinal"])
    tol = 2.0 ** -8 * np.sqrt(0.541 / 3) * np.sqrt(4 if kind == "repeat" else 2)
    for n in ("dk", "dq"):
        e = rel2(f64(got[n]), want[n])
        print(f"{n} {e:.2e} of {tol:.2e}", flush=True)
        assert e <= tol, n
