"""The delta tests' float64 reference against closed forms and differences (CPU)."""
import numpy as np
import pytest

import delta_ref as ref


def test_first_token_and_no_write():
    d = ref.make(2, 1, 4, 8, 16, 2, init=True, seed=1)
    y, S, _, _ = ref.forward(d["v"], d["g"], d["beta"], d["k"], d["q"], d["init"])
    for b in range(2):
        for h in range(4):
            k, q = d["k"][b, 0, h // 2], d["q"][b, 0, h // 2]
            want = np.exp(d["g"][b, 0, h]) * d["init"][b, h] @ (np.eye(16) - d["beta"][b, 0, h] * np.outer(k, k))
            want += d["beta"][b, 0, h] * np.outer(d["v"][b, 0, h], k)
            np.testing.assert_allclose(S[b, h], want, atol=1e-13)
            np.testing.assert_allclose(y[b, 0, h], want @ q, atol=1e-13)
    # beta 0 writes nothing: the state only decays
    y, S, _, _ = ref.forward(d["v"], d["g"], 0 * d["beta"], d["k"], d["q"], d["init"])
    np.testing.assert_allclose(S, np.exp(d["g"][:, 0])[:, :, None, None] * d["init"], atol=1e-14)


def test_orthonormal_keys_are_recalled():
    """No decay, beta 1, orthonormal keys: the state answers every key with its value; a key written again
    answers with its last value."""
    r = np.random.default_rng(3)
    N = 16
    Qm, _ = np.linalg.qr(r.standard_normal((N, N)))
    ks = np.concatenate([Qm, Qm[:5]])[None, :, None, :]
    v = r.standard_normal((1, N + 5, 1, 4))
    z = np.zeros((1, N + 5, 1))
    y, S, _, _ = ref.forward(v, z, z + 1, ks, ks, None)
    np.testing.assert_allclose(y, v, atol=1e-12)
    np.testing.assert_allclose(S[0, 0] @ Qm[:5].T, v[0, N:, 0].T, atol=1e-12)
    np.testing.assert_allclose(S[0, 0] @ Qm[5:].T, v[0, 5:N, 0].T, atol=1e-12)


def test_chunked_form():
    """The triangular form of a chunk equals the recurrence."""
    d = ref.make(1, 24, 1, 6, 16, 1, init=True, seed=5)
    y, S, _, _ = ref.forward(d["v"], d["g"], d["beta"], d["k"], d["q"], d["init"])
    K, Q, V, S0 = d["k"][0, :, 0], d["q"][0, :, 0], d["v"][0, :, 0], d["init"][0, 0]
    cs, be = np.cumsum(d["g"][0, :, 0]), d["beta"][0, :, 0]
    G = np.exp(np.minimum(cs[:, None] - cs[None, :], 0))
    X = np.tril(G * (K @ K.T), -1)
    e = np.linalg.solve(np.eye(24) + X * be[None, :], V - np.exp(cs)[:, None] * (K @ S0.T))
    U = be[:, None] * e
    np.testing.assert_allclose(np.exp(cs)[:, None] * (Q @ S0.T) + np.tril(G * (Q @ K.T)) @ U, y[0, :, 0], atol=1e-12)
    np.testing.assert_allclose(np.exp(cs[-1]) * S0 + (np.exp(cs[-1] - cs)[:, None] * U).T @ K, S[0, 0], atol=1e-12)


@pytest.mark.parametrize("kind", ["layer", "strong"])
def test_gradients_against_differences(kind):
    d = ref.make(2, 7, 4, 3, 16, 2, init=True, seed=7, kind=kind)
    names = ("v", "g", "beta", "k", "q", "init")
    grads = ref.backward(d["v"], d["g"], d["beta"], d["k"], d["q"], d["dy"], d["init"], d["dfinal"])

    def loss(x):
        y, S, _, _ = ref.forward(*(x[n] for n in names))
        return (y * d["dy"]).sum() + (S * d["dfinal"]).sum()

    r = np.random.default_rng(11)
    for n in names:
        step = 1e-5 * r.standard_normal(d[n].shape)
        up, dn = dict(d), dict(d)
        up[n], dn[n] = d[n] + step, d[n] - step
        want = (loss(up) - loss(dn)) / 2
        got = (grads["d" + n] * step).sum()
        assert abs(got - want) <= 1e-8 * max(1.0, abs(want)) * 1e-2 + 1e-10, (n, got, want)


def test_log_decay_gradient_telescopes():
    """dg_t = dg_{t+1} + dy_t . y_t - dv_t . v_t, and after the last token <dfinal, final>."""
    d = ref.make(2, 40, 4, 8, 16, 2, init=True, seed=9)
    y, S, _, _ = ref.forward(d["v"], d["g"], d["beta"], d["k"], d["q"], d["init"])
    gr = ref.backward(d["v"], d["g"], d["beta"], d["k"], d["q"], d["dy"], d["init"], d["dfinal"])
    local = (d["dy"] * y).sum(-1) - (gr["dv"] * d["v"]).sum(-1)
    tail = (d["dfinal"] * S).sum((-1, -2))[:, None]
    np.testing.assert_allclose(local[:, ::-1].cumsum(1)[:, ::-1] + tail, gr["dg"], atol=1e-10)
