"""The gated delta rule's calls as they are used, each beside its plain form in elementary torch operations.

Per head, with a state S of headdim x dstate:

    a_t = exp(g_t);  S' = a_t S_{t-1};  e_t = v_t - S' k_t;  S_t = S' + beta_t e_t k_t^T;  y_t = S_t q_t

``run`` makes one pass through an operator: the forward over whole sequences, the same over packed sequences
of different lengths, one token of decoding, or the backward.  With ``own`` false it is computed from the
chunked formulas below in 32 bits (prefix sums of the log decays in 64), with ``own`` true by the library.
``exact`` is the recurrence itself, token by token, in 64 bits.
"""
import math

import numpy as np
import torch

own = False

CHUNK = 64          # tokens per chunk of the plain form


# ----------------------------------------------------------------------------------------------
# cases

def _case(op, batch, seqlen, nheads, headdim, dstate, ngroups, dtype, init, name=None, nseq=0, lo=0, hi=0):
    c = dict(op=op, batch=batch, seqlen=seqlen, nheads=nheads, headdim=headdim, dstate=dstate, ngroups=ngroups,
             dtype=dtype, init=init, nseq=nseq, lo=lo, hi=hi)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # a training step's forward, or a large prefill, at the library's headline layer shape
        _case("forward", 4, 4096, 80, 64, 128, 1, "bf16", False, "forward_l2p7b"),
        # the small layer shape, continued from a state
        _case("forward", 8, 2048, 24, 64, 128, 1, "bf16", True, "forward_l130m"),
        # one long document: few independent rows, a long chain, a large state
        _case("forward", 1, 65536, 80, 64, 256, 8, "bf16", False, "forward_long64k"),
        # the smallest forward: fp32, where latency counts
        _case("forward", 1, 512, 4, 16, 16, 1, "f32", False, "forward_tiny_f32"),
        # a packed training batch of documents of very different lengths
        _case("varlen", 1, 16384, 80, 64, 128, 1, "bf16", False, "varlen_2p7b", lo=64, hi=4096),
        # a serving step's prefill: many short prompts, each continued from its own state, wide heads
        _case("varlen", 1, 0, 16, 128, 128, 4, "bf16", True, "varlen_short", nseq=37, lo=1, hi=150),
        # decoding a large batch at the headline layer shape
        _case("step", 256, 1, 80, 64, 128, 1, "bf16", True, "step_b256"),
        # decoding for a single user: latency
        _case("step", 1, 1, 24, 64, 128, 1, "bf16", True, "step_b1"),
        # decoding in fp32 with the largest heads and states, an odd batch
        _case("step", 13, 1, 20, 128, 256, 4, "f32", True, "step_f32_wide"),
        # a training step's backward at the headline layer shape
        _case("backward", 4, 4096, 80, 64, 128, 1, "bf16", False, "backward_l2p7b"),
        # the small layer shape's backward through a carried state
        _case("backward", 8, 2048, 24, 64, 128, 1, "bf16", True, "backward_l130m"),
        # a ragged fp32 backward with several groups
        _case("backward", 2, 501, 6, 32, 48, 3, "f32", True, "backward_ragged_f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["forward", "forward", "varlen", "step", "backward", "backward"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    headdim = rng.choice([16, 32, 64, 64, 128])
    dstate = 16 * _log_int(rng, 1, 16)
    ngroups = rng.choice([1, 1, 2, 4, 5])
    nheads = ngroups * _log_int(rng, 1, max(1, 80 // ngroups))
    init = rng.random() < 0.5
    if op == "step":
        return _case(op, _log_int(rng, 1, 256), 1, nheads, headdim, dstate, ngroups, dtype, True)
    # at most the tokens x heads x state of a quarter of the headline shape (fp32 an eighth of that)
    cap = 4096 * 80 * 64 * 128 // (8 if dtype == "f32" else 1)
    most = max(8, min(16384, cap // (nheads * headdim * dstate)))
    if op == "varlen":
        nseq = rng.randint(1, 40)
        hi = max(1, most // nseq)
        return _case(op, 1, 0, nheads, headdim, dstate, ngroups, dtype, init, nseq=nseq, lo=1, hi=_log_int(rng, 1, hi))
    tokens = _log_int(rng, 1, most)
    batch = min(tokens, _log_int(rng, 1, 8))
    return _case(op, batch, tokens // batch, nheads, headdim, dstate, ngroups, dtype, init)


def _lengths(case):
    """Sequence lengths of a packed batch: nseq of them, or as many as fill seqlen tokens."""
    rng = np.random.default_rng([case["nseq"], case["seqlen"], case["lo"], case["hi"]])
    if case["nseq"]:
        return [int(n) for n in rng.integers(case["lo"], case["hi"] + 1, case["nseq"])]
    out, left = [], case["seqlen"]
    while left > 0:
        out.append(min(left, int(rng.integers(case["lo"], case["hi"] + 1))))
        left -= out[-1]
    return out


# ----------------------------------------------------------------------------------------------
# inputs

def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    T = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    H, P, N, G = case["nheads"], case["headdim"], case["dstate"], case["ngroups"]
    op = case["op"]
    s = dict(op=op)
    if op == "varlen":
        lens = _lengths(case)
        lead, rows = (sum(lens),), len(lens)
        s["cu_seqlens"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=dev)
        s["lengths"] = lens
    elif op == "step":
        lead, rows = (case["batch"],), case["batch"]
    else:
        lead, rows = (case["batch"], case["seqlen"]), case["batch"]

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    s["v"] = randn(*lead, H, P).to(T)
    # log decays as a layer makes them: step sizes in [1e-3, 1e-1] through a softplus, a rate per head
    lo = torch.rand((*lead, H), generator=gen, device=dev) * (1e-1 - 1e-3) + 1e-3
    dt = torch.nn.functional.softplus(randn(*lead, H) + torch.log(torch.expm1(lo)))
    s["g"] = -dt * torch.exp(torch.rand(H, generator=gen, device=dev) * math.log(16.0))
    s["beta"] = torch.sigmoid(randn(*lead, H))
    # keys and queries of unit length, the queries scaled by the state width as in attention
    k, q = randn(*lead, G, N), randn(*lead, G, N)
    s["k"] = (k / k.norm(dim=-1, keepdim=True)).to(T)
    s["q"] = (q / q.norm(dim=-1, keepdim=True) / math.sqrt(N) * 4).to(T)
    s["init"] = 0.1 * randn(rows, H, P, N) if case["init"] else None
    if op == "backward":
        s["dy"] = randn(*lead, H, P).to(T)
        s["dfinal"] = 0.1 * randn(rows, H, P, N) if case["init"] else None
    return s


# ----------------------------------------------------------------------------------------------
# one pass

def run(state):
    s = state
    op = s["op"]
    if own:
        import mamba_ssd_sequence_chunked_amd as ssd
        if op == "forward":
            return ssd.delta_forward(s["v"], s["g"], s["beta"], s["k"], s["q"], s["init"])
        if op == "varlen":
            return ssd.delta_forward_varlen(s["v"], s["g"], s["beta"], s["k"], s["q"], s["cu_seqlens"], s["init"])
        if op == "step":
            return ssd.delta_step(s["init"], s["v"], s["g"], s["beta"], s["k"], s["q"]), s["init"]
        return ssd.delta_backward(s["v"], s["g"], s["beta"], s["k"], s["q"], s["dy"], s["init"], s["dfinal"])
    if op == "forward":
        return _forward(s["v"], s["g"], s["beta"], s["k"], s["q"], s["init"])
    if op == "varlen":
        return _varlen(s)
    if op == "step":
        return _step(s["init"], s["v"], s["g"], s["beta"], s["k"], s["q"])
    return _backward(s["v"], s["g"], s["beta"], s["k"], s["q"], s["dy"], s["init"], s["dfinal"])


# ----------------------------------------------------------------------------------------------
# the plain forms

def _heads(t, H):
    """(..., G, N) shared by groups -> (..., H, N)."""
    return t if t.shape[-2] == H else t.repeat_interleave(H // t.shape[-2], dim=-2)


def _chunks(t, nc):
    """(b, L, H, D) or (b, L, H) -> (b, H, nc, CHUNK, ...) with zeros behind the sequence."""
    b, L = t.shape[:2]
    pad = nc * CHUNK - L
    if pad:
        t = torch.cat([t, t.new_zeros((b, pad) + tuple(t.shape[2:]))], dim=1)
    t = t.reshape((b, nc, CHUNK) + tuple(t.shape[2:]))
    return t.movedim(3, 1).contiguous()


def _unit_lower_inverse(L):
    """(I + L)^-1 for strictly lower L, by halves: [[A, 0], [B, D]]^-1 = [[A', 0], [-D' B A', D']]."""
    n = L.shape[-1]
    i = torch.arange(n, device=L.device)
    X = torch.eye(n, device=L.device, dtype=L.dtype).expand(L.shape).contiguous()
    w = 1
    while w < n:
        corner = ((i[:, None] // (2 * w)) == (i[None, :] // (2 * w))) & ((i[:, None] // w) > (i[None, :] // w))
        X = X - X @ ((L * corner) @ X)
        w *= 2
    return X


def _tables(v, g, beta, k, q):
    """Everything of the chunked form that does not need the state."""
    b, L, H, P = v.shape
    nc = -(-L // CHUNK)
    K = _chunks(_heads(k.float(), H), nc)
    Q = _chunks(_heads(q.float(), H), nc)
    V = _chunks(v.float(), nc)
    be = _chunks(beta.float(), nc)
    cs = torch.cumsum(_chunks(g.double(), nc), dim=-1)
    i = torch.arange(CHUNK, device=v.device)
    low = i[:, None] >= i[None, :]
    Gm = torch.exp(torch.where(low, cs[..., :, None] - cs[..., None, :], -math.inf)).float()
    X = (K @ K.transpose(-1, -2)) * Gm * (i[:, None] > i[None, :])
    M = (Q @ K.transpose(-1, -2)) * Gm
    gam = torch.exp(cs).float()[..., None]
    dele = torch.exp(cs[..., -1:] - cs).float()[..., None]
    return K, Q, V, be[..., None], X, M, Gm, gam, dele


def _forward_chunks(v, g, beta, k, q, init):
    """The chunked forward in fp32: the tables, then per chunk the entering states, e and y; the final state."""
    b, L, H, P = v.shape
    N = k.shape[-1]
    t = _tables(v, g, beta, k, q)
    K, Q, V, be, X, M, Gm, gam, dele = t
    inv = _unit_lower_inverse(X * be.transpose(-1, -2))
    S = v.new_zeros((b, H, P, N), dtype=torch.float32) if init is None else init.float()
    nc = K.shape[2]
    Ss, es, ys = [S], [], []
    for c in range(nc):
        St = S.transpose(-1, -2)
        e = inv[:, :, c] @ (V[:, :, c] - gam[:, :, c] * (K[:, :, c] @ St))
        u = be[:, :, c] * e
        ys.append(gam[:, :, c] * (Q[:, :, c] @ St) + M[:, :, c] @ u)
        S = gam[:, :, c, -1:] * S + (dele[:, :, c] * u).transpose(-1, -2) @ K[:, :, c]
        Ss.append(S)
        es.append(e)
    y = torch.cat(ys, dim=2) if ys else v.new_zeros((b, H, 0, P), dtype=torch.float32)
    return t, Ss, es, y


def _forward(v, g, beta, k, q, init):
    L = v.shape[1]
    _, Ss, _, y = _forward_chunks(v, g, beta, k, q, init)
    return y[:, :, :L].movedim(1, 2).to(v.dtype).contiguous(), Ss[-1]


def _varlen(s):
    """Packed sequences: laid out as a padded batch (keys, values and log decays of zero behind an end leave the
    state as it is), the chunked form, and packed again.  Batches of sequences of like length, so that
    the padding stays small."""
    lens = s["lengths"]
    names = ("v", "g", "beta", "k", "q")
    y = torch.empty_like(s["v"])
    H, P, N = s["v"].shape[1], s["v"].shape[2], s["k"].shape[2]
    fin = s["v"].new_zeros((len(lens), H, P, N), dtype=torch.float32)
    order = sorted(range(len(lens)), key=lambda i: lens[i])
    starts = np.concatenate([[0], np.cumsum(lens)]).tolist()
    for a in range(0, len(order), 8):
        ids = order[a:a + 8]
        L = max(lens[i] for i in ids)
        if L == 0:
            if s["init"] is not None:
                fin[ids] = s["init"][ids]
            continue
        part = {n: s[n].new_zeros((len(ids), L) + tuple(s[n].shape[1:])) for n in names}
        for r, i in enumerate(ids):
            for n in names:
                part[n][r, :lens[i]] = s[n][starts[i]:starts[i] + lens[i]]
        yy, ff = _forward(*(part[n] for n in names), None if s["init"] is None else s["init"][ids])
        fin[ids] = ff
        for r, i in enumerate(ids):
            y[starts[i]:starts[i] + lens[i]] = yy[r, :lens[i]]
    return y, fin


def _step(S, v, g, beta, k, q):
    H = v.shape[1]
    K, Q = _heads(k.float(), H)[:, :, None, :], _heads(q.float(), H)[:, :, None, :]
    S1 = S * torch.exp(g)[:, :, None, None]
    u = beta[..., None] * (v.float() - (S1 * K).sum(-1))
    S1 = S1 + u[..., None] * K
    S.copy_(S1)
    return (S1 * Q).sum(-1).to(v.dtype), S


def _backward(v, g, beta, k, q, dy, init, dfinal):
    b, L, H, P = v.shape
    G, N = k.shape[-2:]
    (K, Q, V, be, X, M, Gm, gam, dele), Ss, es, y = _forward_chunks(v, g, beta, k, q, init)
    nc = K.shape[2]
    dY = _chunks(dy.float(), nc)
    invT = _unit_lower_inverse(be * X).transpose(-1, -2)
    Hs = v.new_zeros((b, H, P, N), dtype=torch.float32) if dfinal is None else dfinal.float()
    i = torch.arange(CHUNK, device=v.device)
    strict = i[:, None] > i[None, :]
    dVs, dbs, dKs, dQs, tails = [], [], [], [], []
    for c in range(nc - 1, -1, -1):
        S, e, d, ga, de, bc = Ss[c], es[c], dY[:, :, c], gam[:, :, c], dele[:, :, c], be[:, :, c]
        Kc, Qc, Gc = K[:, :, c], Q[:, :, c], Gm[:, :, c]
        u = bc * e
        w = invT[:, :, c] @ (M[:, :, c].transpose(-1, -2) @ d + de * (Kc @ Hs.transpose(-1, -2)))
        W = (d @ u.transpose(-1, -2)) * Gc
        Z = -(w @ u.transpose(-1, -2)) * Gc * bc * strict
        dVs.append(bc * w)
        dbs.append((w * e).sum(-1))
        dQs.append(ga * (d @ S) + W @ Kc)
        dKs.append(W.transpose(-1, -2) @ Qc + (Z + Z.transpose(-1, -2)) @ Kc + de * (u @ Hs) - bc * ga * (w @ S))
        # the log decay's gradient behind the chunk's last token
        tails.append((Hs.double() * Ss[c + 1].double()).sum((-1, -2)))
        Hs = ga[:, :, -1:] * Hs + (ga * d).transpose(-1, -2) @ Qc - (bc * ga * w).transpose(-1, -2) @ Kc

    def tokens(parts):                       # chunks, last first -> (b, L, H, ...)
        t = torch.cat(parts[::-1], dim=2)[:, :, :L]
        return t.movedim(1, 2).contiguous()

    dv32 = torch.cat(dVs[::-1], dim=2)
    # dg_t = dg_{t+1} + dy_t . y_t - dv_t . v_t
    local = (dY.reshape(b, H, -1, P).double() * y.double()).sum(-1) - (dv32.double() * V.reshape(b, H, -1, P).double()).sum(-1)
    local = local.reshape(b, H, nc, CHUNK)
    dg = local.flip(-1).cumsum(-1).flip(-1) + torch.stack(tails[::-1], dim=2)[..., None]
    dg = dg.reshape(b, H, -1)[:, :, :L].movedim(1, 2).float().contiguous()
    if init is None:
        dg[:, 0] = 0.0                       # nothing decays into the first token

    def groups(t):                           # sum over the heads that share a key
        return t.reshape(b, L, G, H // G, N).sum(3).to(k.dtype)

    return dict(dv=tokens(dVs).to(v.dtype), dg=dg, dbeta=tokens(dbs), dk=groups(tokens(dKs)), dq=groups(tokens(dQs)),
                dinit=Hs)


# ----------------------------------------------------------------------------------------------
# the definition in 64 bits

def _recurrence(v, g, beta, k, q, S, keep=None):
    """Token by token: y (b, L, H, P) and the final state, all float64; keep(t, S) sees the state before token t."""
    ys = []
    for t in range(v.shape[1]):
        if keep is not None:
            keep(t, S)
        Sp = S * torch.exp(g[:, t])[:, :, None, None]
        e = v[:, t] - torch.einsum("bhpn,bhn->bhp", Sp, k[:, t])
        S = Sp + (beta[:, t, :, None] * e)[..., None] * k[:, t, :, None, :]
        ys.append(torch.einsum("bhpn,bhn->bhp", S, q[:, t]))
    return (torch.stack(ys, 1) if ys else torch.zeros_like(v)), S


def exact(case, seed):
    s = prepare(case, seed)
    H, P, N = case["nheads"], case["headdim"], case["dstate"]
    op = case["op"]
    v, g, beta = s["v"].double(), s["g"].double(), s["beta"].double()
    k, q = _heads(s["k"].double(), H), _heads(s["q"].double(), H)

    def start(rows):
        return v.new_zeros((rows, H, P, N)) if s["init"] is None else s["init"].double()

    if op == "forward":
        return _recurrence(v, g, beta, k, q, start(case["batch"]))
    if op == "step":
        y, S = _recurrence(v[:, None], g[:, None], beta[:, None], k[:, None], q[:, None], start(case["batch"]))
        return y[:, 0], S
    if op == "varlen":
        S0 = start(len(s["lengths"]))
        ys, fins, at = [], [], 0
        for i, n in enumerate(s["lengths"]):
            y, f = _recurrence(*(t[None, at:at + n] for t in (v, g, beta, k, q)), S0[i:i + 1])
            ys.append(y[0])
            fins.append(f)
            at += n
        return torch.cat(ys), torch.cat(fins)
    return _exact_backward(s, v, g, beta, k, q, start(case["batch"]))


def _exact_backward(s, v, g, beta, k, q, S0):
    """The recurrence's adjoint, token by token from the end, the states recomputed from marks every 64 tokens."""
    b, L, H, P = v.shape
    G, N = s["k"].shape[-2:]
    dy = s["dy"].double()
    marks = {}
    _recurrence(v, g, beta, k, q, S0, keep=lambda t, S: marks.__setitem__(t, S) if t % 64 == 0 else None)
    D = torch.zeros_like(S0) if s["dfinal"] is None else s["dfinal"].double()
    dv, dk, dq, dg, db = (torch.zeros_like(t) for t in (v, k, q, g, beta))
    for a in range((L - 1) // 64 * 64, -1, -64):
        z = min(L, a + 64)
        before = {}
        _recurrence(*(t[:, a:z] for t in (v, g, beta, k, q)), marks.pop(a), keep=before.__setitem__)
        for t in range(z - 1, a - 1, -1):
            kt, qt, bt = k[:, t], q[:, t], beta[:, t, :, None]
            al = torch.exp(g[:, t])[:, :, None, None]
            Sp = before.pop(t - a) * al
            e = v[:, t] - torch.einsum("bhpn,bhn->bhp", Sp, kt)
            dq[:, t] = torch.einsum("bhpn,bhp->bhn", Sp, dy[:, t]) + (dy[:, t] * bt * e).sum(-1, keepdim=True) * kt
            D = D + dy[:, t, :, :, None] * qt[:, :, None, :]
            du = torch.einsum("bhpn,bhn->bhp", D, kt)
            db[:, t] = (du * e).sum(-1)
            dv[:, t] = bt * du
            dk[:, t] = torch.einsum("bhpn,bhp->bhn", D, bt * e) - torch.einsum("bhpn,bhp->bhn", Sp, bt * du)
            D = D - (bt * du)[..., None] * kt[:, :, None, :]
            dg[:, t] = (D * Sp).sum((-1, -2))
            D = D * al

    def groups(t):
        return t.reshape(b, L, G, H // G, N).sum(3)

    return dict(dv=dv, dg=dg, dbeta=db, dk=groups(dk), dq=groups(dq), dinit=D)


# ----------------------------------------------------------------------------------------------
# what one pass cannot do without

def work(case):
    H, P, N, G = case["nheads"], case["headdim"], case["dstate"], case["ngroups"]
    es = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op == "varlen":
        lens = _lengths(case)
        rows, tokens = len(lens), sum(lens)
    else:
        rows, tokens = case["batch"], case["batch"] * case["seqlen"]
    value, shared, scalar, state = tokens * H * P * es, tokens * G * N * es, tokens * H * 4, rows * H * P * N * 4
    if op == "backward":
        return {"bytes": 3 * value + 4 * shared + 4 * scalar + state * (3 if case["init"] else 1),
                "flops": 16.0 * tokens * H * P * N}
    return {"bytes": 2 * value + 2 * shared + 2 * scalar + state * (2 if case["init"] else 1),
            "flops": 6.0 * tokens * H * P * N}
