"""How near the gated delta rule's outputs are to the float64 recurrence (delta_ref), each head for itself.

Tolerances, fixed before the first run:

 * dg: a token's value is reached by a sum of at most 64 terms of the gradient's own size from the nearer end of its chunk,
   so that errors of one term add up at random to at most 8 of them.  For bf16 inputs the term's operands are pairs of
   bf16 values, off by at most 2^-18 each, two to a product: 2^-17.  For fp32 inputs a term sums products over N and
   64 more values, whose half steps of 2^-24 add up at random: sqrt(N + 64) of them.
"""
import numpy as np
import pytest

import delta_ref as ref
from test_gpu_delta import dev, f64, grads, inputs

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
