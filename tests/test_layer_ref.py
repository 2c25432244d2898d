"""CPU pins of the 64-bit references that the layer operators are checked against."""
import numpy as np
import pytest

import _layer_ref as R


def test_element_values_match_torch_float8():
    import torch

    c = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(c).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.element_values(c, R.MXFP8), want, equal_nan=True)
    assert R.element_values(np.arange(16, dtype=np.uint8), R.MXFP4)[:8].tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6]


@pytest.mark.parametrize("fmt", [R.MXFP4, R.MXFP8])
def test_quantizer_matches_the_oracle(orc, fmt):
    import synth

    X = synth.bf16_normal(5, synth.S_ACT, (37, 256), 1.0, 0.05, 30.0)
    X[3, :40] = 0
    X[4, 7] = 0x7F80           # Inf
    X[5, 100] = 0x7FC0         # NaN
    X[6, :32] = 0x0001         # subnormals
    x = (X.astype(np.uint32) << 16).view(np.float32)
    codes, scales = R.mx_quantize(x, fmt)
    want, ws = orc.act_quant_mxfp8(X) if fmt == R.MXFP8 else orc.act_quant(X)
    assert np.array_equal(scales, ws)
    assert np.array_equal(R.pack(codes, fmt), want)


def test_rotation_is_a_rotation():
    r = np.random.default_rng(0)
    x = r.standard_normal((5, 3, 64))
    t = r.uniform(0, 100, (5, 16))
    for layout in (0, 1):
        y = R.rotate(x, np.cos(t), np.sin(t), 32, layout)
        assert np.array_equal(y[..., 32:], x[..., 32:])
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
        assert np.allclose(R.rotate(y, np.cos(t), -np.sin(t), 32, layout), x)


def test_attention_against_a_loop():
    r = np.random.default_rng(1)
    q, k, v = r.standard_normal((3, 8)), r.standard_normal((5, 8)), r.standard_normal((5, 8))
    seen = np.array([[1, 1, 0, 1, 0], [0, 0, 0, 0, 0], [1, 1, 1, 1, 1]], bool)
    k[4], v[2] = k[4], v[2]
    out, lse, _, _ = R.attend(q, k, v, seen, 0.5)
    for i in range(3):
        at = np.flatnonzero(seen[i])
        if not len(at):
            assert not out[i].any() and lse[i] == -np.inf
            continue
        e = np.exp([0.5 * q[i] @ k[t] for t in at])
        assert np.allclose(out[i], (e[:, None] * v[at]).sum(0) / e.sum())
        assert np.isclose(lse[i], np.log(e.sum()))


def test_by_parts_frequencies_stay_between_the_two():
    w = R.rope_frequencies(128, 10000.0)
    s = R.rope_frequencies(128, 10000.0, 2, 4.0, 4096, 32.0, 1.0)
    assert np.all(s <= w) and np.all(s >= w / 4 * (1 - 1e-12))
    assert s[0] == w[0] and np.isclose(s[-1], w[-1] / 4)
