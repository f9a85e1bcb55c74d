"""The gated delta rule in float64 numpy, token by token: the reference of the delta tests.

    S' = exp(g) S;  e = v - S' k;  u = beta e;  S = S' + u k^T;  y = S q

Arrays as the library takes them: v (b, L, H, P), g and beta (b, L, H), k and q (b, L, G, N), states
(b, H, P, N).  ``forward`` also returns what rounding errors are counted in, row by row of the state (the rows
do not mix):

  scale_y[t]  |q| times the size of what y_t is summed from: the state entering the block of 32 tokens that t is
              in, decayed to t, and the block's own |u_j| |k_j| (Cauchy-Schwarz on every partial product).  An
              operand of y that is rounded by eps moves y by at most eps scale_y.
  drift       sum over tokens of (|S'| + |u| |k|), decayed to the end: a relative error eps made at each token in
              the state or its update moves the final state by at most eps drift, because what follows is a
              decay and a contraction (beta |k|^2 <= 2).
"""
import numpy as np

BLOCK = 32


def heads(t, H):
    return np.repeat(t, H // t.shape[2], axis=2)


def forward(v, g, beta, k, q, init=None, trace=False):
    """Returns y, final, scale_y, drift (and the per-token decayed states and errors e when trace)."""
    b, L, H, P = v.shape
    N = k.shape[3]
    K, Q = heads(k, H), heads(q, H)
    norm = lambda a: np.sqrt((a * a).sum(-1))        # noqa: E731
    S = np.zeros((b, H, P, N)) if init is None else init.astype(np.float64).copy()
    drift = np.zeros((b, H, P))
    y, sy = np.zeros((b, L, H, P)), np.zeros((b, L, H, P))
    kept = []
    for t in range(L):
        a = np.exp(g[:, t])[:, :, None]
        if t % BLOCK == 0:
            inside = norm(S)
        kt, qt = K[:, t, :, None, :], Q[:, t, :, None, :]
        Sp = a[..., None] * S
        e = v[:, t] - (Sp * kt).sum(-1)
        u = beta[:, t, :, None] * e
        S = Sp + u[..., None] * kt
        y[:, t] = (S * qt).sum(-1)
        wrote = np.abs(u) * norm(kt)
        inside = a * inside + wrote
        drift = a * drift + norm(Sp) + wrote
        # the state's own error reaches y too, but at a smaller unit: counted by the caller
        sy[:, t] = inside * norm(qt)
        if trace:
            kept.append((Sp, e))
    return (y, S, sy, drift) + ((kept,) if trace else ())


def step(state, v, g, beta, k, q):
    y, S, sy, drift = forward(v[:, None], g[:, None], beta[:, None], k[:, None], q[:, None], state)
    return y[:, 0], S, sy[:, 0], drift


def backward(v, g, beta, k, q, dy, init=None, dfinal=None):
    """Gradients of <y, dy> + <final, dfinal> by the recurrence's adjoint."""
    b, L, H, P = v.shape
    G, N = k.shape[2:]
    K, Q = heads(k, H), heads(q, H)
    _, _, _, _, kept = forward(v, g, beta, k, q, init, trace=True)
    D = np.zeros((b, H, P, N)) if dfinal is None else dfinal.astype(np.float64).copy()
    dv, dg, db = np.zeros_like(v), np.zeros_like(g), np.zeros_like(beta)
    dK, dQ = np.zeros_like(K), np.zeros_like(Q)
    for t in range(L - 1, -1, -1):
        Sp, e = kept[t]
        kt, qt, bt = K[:, t, :, None, :], Q[:, t, :, None, :], beta[:, t, :, None]
        St = Sp + (bt * e)[..., None] * kt
        dQ[:, t] = (St * dy[:, t][..., None]).sum(2)
        D = D + dy[:, t][..., None] * qt
        w = (D * kt).sum(-1)
        db[:, t] = (w * e).sum(-1)
        dv[:, t] = bt * w
        dK[:, t] = (D * (bt * e)[..., None]).sum(2) - (Sp * (bt * w)[..., None]).sum(2)
        D = D - (bt * w)[..., None] * kt
        dg[:, t] = (D * Sp).sum((-1, -2))
        D = D * np.exp(g[:, t])[:, :, None, None]
    return dict(dv=dv, dg=dg, dbeta=db, dk=dK.reshape(b, L, G, H // G, N).sum(3),
                dq=dQ.reshape(b, L, G, H // G, N).sum(3), dinit=D)


# ---- inputs ---------------------------------------------------------------------------------------

def bf16_round(a):
    """To the nearest bfloat16 (ties to even), as float64."""
    u = np.ascontiguousarray(a, dtype=np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32).astype(np.float64)


def make(b, L, H, P, N, G, dtype="f32", init=False, seed=0, kind="layer"):
    """Inputs as float64 arrays that hold values of their storage types.

    kind "layer": random unit keys, decays as a layer makes them; "repeat": every token of a row has the same
    key and beta 1 (the triangular system's hardest case); "resets": some log decays -inf, some betas 0;
    "strong": log decays down to -40."""
    r = np.random.default_rng(seed)
    store = bf16_round if dtype == "bf16" else (lambda a: a.astype(np.float32).astype(np.float64))
    f32 = lambda a: a.astype(np.float32).astype(np.float64)      # noqa: E731
    v, dy = r.standard_normal((2, b, L, H, P))
    k, q = r.standard_normal((2, b, L, G, N))
    k /= np.maximum(np.linalg.norm(k, axis=-1, keepdims=True), 1e-30)
    q /= np.maximum(np.linalg.norm(q, axis=-1, keepdims=True), 1e-30)
    g = -np.exp(r.uniform(0, np.log(16.0), H)) * np.logaddexp(0, r.standard_normal((b, L, H)) - 3.5)
    beta = 1 / (1 + np.exp(-r.standard_normal((b, L, H))))
    if kind == "repeat":
        k[:] = k[:, :1]
        beta[:] = 1.0
        g *= 0.01
    elif kind == "resets":
        g[r.random(g.shape) < 0.05] = -np.inf
        beta[r.random(g.shape) < 0.1] = 0.0
    elif kind == "strong":
        g = -40.0 * r.random(g.shape) ** 4
    h0 = r.standard_normal((2, b, H, P, N)) * 0.3
    return dict(v=store(v), g=f32(g), beta=f32(beta), k=store(k), q=store(q), dy=store(dy),
                init=f32(h0[0]) if init else None, dfinal=f32(h0[1]) if init else None, dtype=dtype)
