"""What linear attention's results keep, in the 2-norm and against float64: the statements of the header."""
import numpy as np
import pytest

import linear_ref as ref
from test_gpu_linear import dev, f64, inputs, rel2

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("L", [29, 32, 61])
def test_one_token_and_padding(L, dt):
    """A token, then zeros: its state is the token's product times a power of the decay, and errs by that power's error.  The
    power is off by an ulp of expf and a rounding (3 half steps), the weighted value, its product and the chunks' decays by
    one each: 7 half steps of 2^-24 are 4.2e-7.  Backwards the same for the state before the first token where only the
    last has a gradient.  With fp32 inputs a token's output adds a sum over N terms to that."""
    import torch
    import mamba_ssd_sequence_chunked_amd as ssd
    H, P, N = 24, 16, 16
    d = ref.make(1, L, H, P, N, H, dt, False, seed=900)
    d["g"] = np.linspace(-0.05, -60.0 / L, H).astype(np.float32)
    d["v"][:, 1:] = 0.0
    d["dy"][:, :-1] = 0.0
    y, fin = ssd.linear_forward(*inputs(d))
    (yr, S), (ym, _) = ref.forward(d["v"], d["g"], d["k"], d["q"])
    got = ssd.linear_backward(*inputs(d), dev(d["dy"], dt))
    want, _ = ref.backward(d["v"], d["g"], d["k"], d["q"], d["dy"], None, np.zeros((1, H, P, N)))
    torch.cuda.synchronize()
    for h in range(H):
        assert rel2(fin[:, h], S[:, h]) <= 5e-7, h
        assert rel2(got["dinit"][:, h], want["dinit"][:, h]) <= 5e-7, h
    if dt == "f32":
        assert (np.abs(f64(y) - yr) <= (8 + N) * 2.0 ** -24 * ym).all()


def drawn(b, L, H, P, N, G, dt, kind, seed):
    """Inputs on the GPU: v, g, k, q, dy, init, dfinal."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T = torch.bfloat16 if dt == "bf16" else torch.float32
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")        # noqa: E731
    i = torch.arange(1, H + 1, device="cuda")
    g = {"ladder": -torch.exp2(-8.0 * i / H), "slow": torch.full((H,), -1e-4, device="cuda"),
         "none": torch.zeros(H, device="cuda")}[kind].contiguous()
    return (rand(b, L, G, P).to(T), g, rand(b, L, G, N).to(T), (rand(b, L, H, N) / N ** 0.5).to(T), rand(b, L, H, P).to(T),
            rand(b, H, P, N), rand(b, H, P, N))


def exact(v, g, k, q, dy, init, dfinal, groups):
    """Results of the heads of some groups in float64, and the 2-norm of what each of their tokens adds to dg."""
    H, G = q.shape[2], k.shape[2]
    m = H // G
    hs = np.concatenate([np.arange(j * m, (j + 1) * m) for j in groups])
    v, k = (np.repeat(f64(t[:, :, groups].float()), m, 2) for t in (v, k))
    q, dy = (f64(t[:, :, hs].float()) for t in (q, dy))
    S, D, a = f64(init[:, hs]), f64(dfinal[:, hs]), np.exp(f64(g[hs]))[:, None, None]
    b, L = q.shape[:2]
    y, dq, dk, dv, dS, dg, terms = np.zeros_like(dy), np.zeros_like(q), np.zeros_like(k), np.zeros_like(v), np.zeros_like(S), 0.0, 0.0
    last = D
    for t in range(L):
        dS = a * (dS + S)
        S = a * S + v[:, t, :, :, None] * k[:, t, :, None, :]
        y[:, t] = (S * q[:, t, :, None, :]).sum(-1)
        dq[:, t] = (S * dy[:, t, :, :, None]).sum(-2)
        term = (dy[:, t] * (dS * q[:, t, :, None, :]).sum(-1)).sum(-1)
        dg, terms = dg + term.sum(0), terms + (term ** 2).sum(0)
    term = (last * dS).sum((2, 3))
    dg, terms = dg + term.sum(0), terms + (term ** 2).sum(0)
    for t in range(L - 1, -1, -1):
        D = D + dy[:, t, :, :, None] * q[:, t, :, None, :]
        dv[:, t], dk[:, t] = (D * k[:, t, :, None, :]).sum(-1), (D * v[:, t, :, :, None]).sum(-2)
        D = a * D
    group = lambda x: x.reshape(b, L, len(groups), m, -1).sum(3)          # noqa: E731
    return hs, dict(y=y, final=S, dq=dq, dk=group(dk), dv=group(dv), dinit=D, dg=dg), np.sqrt(terms.sum())


def run(v, g, k, q, dy, init, dfinal):
    import mamba_ssd_sequence_chunked_amd as ssd
    y, fin = ssd.linear_forward(v, g, k, q, init)
    return dict(ssd.linear_backward(v, g, k, q, dy, init, dfinal), y=y, final=fin)


def rounded(L, dt):
    """What a state's own roundings add up to over L tokens without decay.  It is rounded with every token (fp32) or three
    times a chunk of 32 (bf16, whose three values are three products).  A rounding's rms is half a step by the square root of
    3, and the state grows like the square root of its tokens, so n of them are 2^-24 sqrt(n / 6) of its norm."""
    return 2.0 ** -24 * ((L if dt == "f32" else 3 * L / 32) / 6) ** 0.5


# whole rows, rows cut at once, chains (300 heads from 2048 tokens on) with up to 256 rows of state on either side, shared
# keys, decays under which little, much and nearly all of a row is left
STATED = [
    (1, 22, 1, 64, 240, 1, "ladder"), (2, 700, 8, 64, 128, 4, "ladder"), (3, 1111, 20, 16, 224, 5, "slow"), (1, 2048, 4, 256, 256, 4, "slow"),
    (1, 2048, 300, 16, 144, 300, "ladder"), (1, 2048, 300, 144, 16, 300, "ladder"), (1, 2048, 300, 48, 32, 60, "slow"),
    (3, 1500, 6, 32, 48, 3, "none"),
]


@pytest.mark.parametrize("c", STATED, ids=lambda c: "b{}_L{}_H{}_P{}_N{}_G{}_{}".format(*c))
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_accuracy_over_2048_tokens(c, dt):
    """The header's statements for rows of up to 2048 tokens.  In fp32 a state that hardly decays is rounded with every token,
    which adds up (see rounded): 1.1e-6 over 2048 of them, and with bf16 inputs 3.4e-7, which 5e-7 holds."""
    b, L, H, P, N, G, kind = c
    x = drawn(b, L, H, P, N, G, dt, kind, seed=910 + STATED.index(c))
    got = run(*x)
    groups = sorted({0, G // 2, G - 1})
    hs, want, terms = exact(*x, groups)
    norm = lambda n, at: np.linalg.norm(f64(got[n].float())[at] - want[n]) / np.linalg.norm(want[n])           # noqa: E731
    adds = rounded(L, dt) if dt == "f32" else 0.0
    for n in ("final", "dinit"):
        assert norm(n, np.s_[:, hs]) <= 5e-7 + adds, n
    assert np.linalg.norm(f64(got["dg"])[hs] - want["dg"]) <= (1e-6 + 2 * adds) * terms
    outputs = 2.6e-3 if dt == "bf16" else 1e-6 + adds
    for n, at in (("y", hs), ("dq", hs), ("dk", groups), ("dv", groups)):
        assert norm(n, np.s_[:, :, at]) <= outputs, n


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("H", [300, 3])
def test_accuracy_of_long_rows_without_decay(dt, H):
    """A state's roundings add up on top of what short rows are off by; dg has one such sum in the state and one in its
    derivative."""
    L, P, N = 16384, 16, 16
    x = drawn(1, L, H, P, N, H, dt, "none", seed=930)
    got = run(*x)
    hs, want, terms = exact(*x, [0, H - 1])
    adds = rounded(L, dt)
    for n in ("final", "dinit"):
        assert np.linalg.norm(f64(got[n])[:, hs] - want[n]) <= (5e-7 + adds) * np.linalg.norm(want[n]), n
    assert np.linalg.norm(f64(got["dg"])[hs] - want["dg"]) <= (1e-6 + 2 * adds) * terms
