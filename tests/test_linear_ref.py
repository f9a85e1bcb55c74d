"""The float64 reference of linear attention against other forms of the same sums, and its gradients against
differences (no GPU)."""
import numpy as np
import pytest

import linear_ref as ref


def args(d):
    return d["v"], d["g"], d["k"], d["q"]


def test_forward_is_the_dense_sum():
    """y = ((Q K^T) o a^(t - s)) V + a^(t + 1) Q S^T, written out as a matrix."""
    b, L, H, P, N, G = 2, 13, 4, 3, 5, 2
    d = ref.make(b, L, H, P, N, G, "f32", True, seed=1)
    (y, S), _ = ref.forward(*args(d), d["init"])
    t = np.arange(L)
    for i in range(b):
        for h in range(H):
            a, j = np.exp(float(d["g"][h])), h // (H // G)
            K, V, Q = (x.astype(np.float64) for x in (d["k"][i, :, j], d["v"][i, :, j], d["q"][i, :, h]))
            M = np.where(t[:, None] >= t[None, :], a ** np.maximum(t[:, None] - t[None, :], 0), 0.0) * (Q @ K.T)
            want = M @ V + a ** (t[:, None] + 1.0) * (Q @ d["init"][i, h].T.astype(np.float64))
            assert np.allclose(y[i, :, h], want, rtol=1e-12, atol=1e-12)
            want = (V * (a ** (L - 1.0 - t))[:, None]).T @ K + a ** L * d["init"][i, h]
            assert np.allclose(S[i, h], want, rtol=1e-12, atol=1e-12)


def test_decay_limits():
    """g = 0 is the plain sum, g = -inf leaves every token alone."""
    d = ref.make(1, 9, 2, 3, 4, 2, "f32", True, seed=2)
    d["g"] = np.array([0.0, -np.inf], np.float32)
    (y, S), _ = ref.forward(*args(d), d["init"])
    assert np.allclose(S[0, 0], d["init"][0, 0] + np.einsum("tp,tn->pn", d["v"][0, :, 0], d["k"][0, :, 0]), atol=1e-5)
    assert np.allclose(y[0, :, 1], (d["k"][0, :, 1] * d["q"][0, :, 1]).sum(-1)[:, None] * d["v"][0, :, 1], atol=1e-5)
    out, _ = ref.backward(*args(d), d["dy"], d["init"], d["dfinal"])
    assert out["dg"][1] == 0 and np.abs(out["dinit"][0, 1]).max() == 0


@pytest.mark.parametrize("G", [1, 2, 4])
def test_gradients_against_differences(G):
    b, L, H, P, N = 2, 7, 4, 3, 5
    d = ref.make(b, L, H, P, N, G, "f32", True, seed=3 + G)
    x = {n: d[n].astype(np.float64) for n in ("v", "g", "k", "q", "init")}

    def loss():
        (y, S), _ = ref.forward(x["v"], x["g"], x["k"], x["q"], x["init"])
        return (y * d["dy"]).sum() + (S * d["dfinal"]).sum()

    got, size = ref.backward(x["v"], x["g"], x["k"], x["q"], d["dy"], x["init"], d["dfinal"])
    rng = np.random.default_rng(4)
    for n, g in (("v", "dv"), ("g", "dg"), ("k", "dk"), ("q", "dq"), ("init", "dinit")):
        assert (np.abs(got[g]) <= size[g] * (1 + 1e-12)).all()
        for _ in range(12):
            i = tuple(rng.integers(0, s) for s in x[n].shape)
            old, h = x[n][i], 1e-5
            x[n][i] = old + h
            up = loss()
            x[n][i] = old - h
            down = loss()
            x[n][i] = old
            # the loss is at most of second order but in g; (1e-5)^2 of its size, and 1e-16 / h of it
            assert abs((up - down) / (2 * h) - got[g][i]) <= 1e-8 * max(1.0, size[g][i]) * L * L, (n, i)


def test_group_gradients_are_sums():
    d = ref.make(1, 6, 6, 2, 3, 2, "f32", True, seed=9)
    got, _ = ref.backward(*args(d), d["dy"], d["init"], d["dfinal"])
    rep = lambda t: np.repeat(t, 3, axis=2)        # noqa: E731
    own, _ = ref.backward(rep(d["v"]), d["g"], rep(d["k"]), d["q"], d["dy"], d["init"], d["dfinal"])
    assert np.allclose(got["dv"], own["dv"].reshape(1, 6, 2, 3, 2).sum(3)) and np.allclose(got["dq"], own["dq"])
