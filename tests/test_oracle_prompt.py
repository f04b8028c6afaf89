"""Pins of the prompt oracle: rotation against complex numbers and its group property, prompt
attention against the decode oracle row by row."""

import numpy as np
import pytest

import oracle
from oracle import prompt


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_is_a_complex_product(inter):
    rng = np.random.default_rng(3)
    x, pos, f = rng.normal(size=(5, 3, 64)), np.array([0, 1, 7, 4096, 10 ** 6]), \
        np.array([1.0, 0.37, 1e-4, 2.5e-6] * 4)
    y, mag = prompt.rope(x, pos, f, inter)
    lo = np.arange(0, 32, 2) if inter else np.arange(16)
    hi = lo + (1 if inter else 16)
    z = (x[..., lo] + 1j * x[..., hi]) * np.exp(1j * pos[:, None, None] * f)
    np.testing.assert_allclose(y[..., lo], z.real, atol=1e-12)
    np.testing.assert_allclose(y[..., hi], z.imag, atol=1e-12)
    np.testing.assert_array_equal(y[..., 32:], x[..., 32:])
    np.testing.assert_array_equal(y[0], x[0])
    assert (mag + 1e-12 >= np.abs(y)).all()


def test_prompt_rows_equal_the_decode_oracle():
    rng = np.random.default_rng(4)
    PS, Hkv, G, D = 16, 2, 2, 64
    new, past = (20, 0, 1), (0, 5, 33)
    lens = np.array([n + p for n, p in zip(new, past)])
    cu = np.concatenate([[0], np.cumsum(new)])
    table = np.arange(9).reshape(3, 3)
    K, V = rng.normal(size=(9, Hkv, PS, D)), rng.normal(size=(9, Hkv, PS, D))
    q = rng.normal(size=(cu[-1], Hkv * G, D))
    out, lse, mass, logit = prompt.prefill(q, K, V, table, lens, cu, PS, 0.125)
    seq, pos = prompt.row_places(cu, lens)
    for i, (b, t) in enumerate(zip(seq, pos)):
        o, s = oracle.attend(q[i:i + 1], K, V, table[b:b + 1], np.array([t + 1]), PS, 0.125)
        np.testing.assert_allclose(out[i], o[0], atol=1e-12)
        np.testing.assert_allclose(lse[i], s[0], atol=1e-12)
    assert (mass + 1e-12 >= np.abs(out)).all() and (logit > 0).all()
