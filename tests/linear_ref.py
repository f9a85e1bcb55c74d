"""Linear attention with a decay for each head in float64 numpy, token by token: the reference of the linear tests.

    S_t = exp(g) S_{t-1} + v_t k_t^T;  y_t = S_t q_t

Arrays as the library takes them: v (b, L, G, P), g (H), k (b, L, G, N), q and dy (b, L, H, N or P), states
(b, H, P, N).  Every function also returns its results' magnitudes: the same sums over the absolute values of their
terms (all terms enter linearly), which is what rounding errors are counted in: an operand that is rounded by eps moves
a result by at most eps times its magnitude.
"""
import numpy as np


def heads(t, H):
    return np.repeat(t.astype(np.float64), H // t.shape[2], axis=2)


def decay(g):
    return np.exp(np.maximum(np.asarray(g, np.float64), -1000.0))[:, None, None]


def _walk(v, a, k, q, S):
    y = np.zeros((*q.shape[:3], v.shape[3]))
    for t in range(q.shape[1]):
        S = a * S + v[:, t, :, :, None] * k[:, t, :, None, :]
        y[:, t] = (S * q[:, t, :, None, :]).sum(-1)
    return y, S


def forward(v, g, k, q, init=None):
    """(y, final), (their magnitudes)."""
    b, L, H, N = q.shape
    P = v.shape[3]
    S = np.zeros((b, H, P, N)) if init is None else np.asarray(init, np.float64)
    v, k, q, a = heads(v, H), heads(k, H), q.astype(np.float64), decay(g)
    return _walk(v, a, k, q, S), _walk(np.abs(v), a, np.abs(k), np.abs(q), np.abs(S))


def _adjoint(v, a, k, q, dy, S, D):
    b, L, H, P = dy.shape
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    dS, dg = np.zeros_like(S), np.zeros(H)          # dS = dS_t/dg
    for t in range(L):
        dS = a * (dS + S)
        S = a * S + v[:, t, :, :, None] * k[:, t, :, None, :]
        dq[:, t] = (S * dy[:, t, :, :, None]).sum(-2)
        dg += (dy[:, t, :, :, None] * dS * q[:, t, :, None, :]).sum((0, 2, 3))
    dg += (D * dS).sum((0, 2, 3))
    for t in range(L - 1, -1, -1):
        D = D + dy[:, t, :, :, None] * q[:, t, :, None, :]
        dv[:, t] = (D * k[:, t, :, None, :]).sum(-1)
        dk[:, t] = (D * v[:, t, :, :, None]).sum(-2)
        D = a * D
    return dict(dv=dv, dg=dg, dk=dk, dq=dq, dinit=D)


def backward(v, g, k, q, dy, init=None, dfinal=None):
    """Gradients for dL/dy = dy and dL/d(final) = dfinal, and their magnitudes."""
    b, L, H, N = q.shape
    G, P = v.shape[2:]
    zero = np.zeros((b, H, P, N))
    S, D = (zero if x is None else np.asarray(x, np.float64) for x in (init, dfinal))
    v, k, q, dy, a = heads(v, H), heads(k, H), q.astype(np.float64), dy.astype(np.float64), decay(g)
    out = []
    for f in (lambda x: x, np.abs):
        r = _adjoint(f(v), a, f(k), f(q), f(dy), f(S), f(D))
        for n in ("dv", "dk"):
            r[n] = r[n].reshape(b, L, G, H // G, -1).sum(3)
        out.append(r)
    return out


# ---- inputs ---------------------------------------------------------------------------------------------

def round_bf16(a):
    u = np.ascontiguousarray(a, np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32)


def make(b, L, H, P, N, G, dtype, init=False, seed=0, kind="ladder"):
    """Seeded inputs, values exact in dtype.  Kinds of decay: rates from 1 down to 1/256 over the heads; strong ones up to
    40; none at all and all of it (0, -inf and what no power of fits fp32) among others; hardly any."""
    rng = np.random.default_rng([seed, b, L, H, P, N, G])
    T = round_bf16 if dtype == "bf16" else (lambda x: np.asarray(x, np.float32))
    d = dict(v=T(rng.standard_normal((b, L, G, P))), k=T(rng.standard_normal((b, L, G, N))),
             q=T(rng.standard_normal((b, L, H, N)) / np.sqrt(N)), dy=T(rng.standard_normal((b, L, H, P))), dtype=dtype)
    i = np.arange(1, H + 1)
    g = {"ladder": -np.exp2(-8.0 * i / H), "strong": -0.5 * 80.0 ** (i / H),
         "edges": np.resize([0.0, -np.inf, -0.3, -2000.0, -104.5], H), "long": -1e-5 * i}[kind]
    d["g"] = g.astype(np.float32)
    d["init"] = rng.standard_normal((b, H, P, N)).astype(np.float32) if init else None
    d["dfinal"] = rng.standard_normal((b, H, P, N)).astype(np.float32) if init else None
    return d
