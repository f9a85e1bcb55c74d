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
