"""Pins of the MXFP4 oracle: every code, hand-expanded blocks, rounding ties,
a brute-force quantiser, the clamps, and the scores on dequantised values."""
import numpy as np
import pytest

from oracle import dsa_oracle as O
from oracle import serving_oracle as S


def test_every_code():
    packed = np.arange(256, dtype=np.uint8).reshape(2, 128)[:, :64]
    v = S.mxfp4_dequantize(packed, np.full((2, 4), 127, np.uint8))
    grid = [0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6]
    for r in range(2):
        for i in range(64):
            assert v[r, 2 * i] == grid[packed[r, i] & 15] and v[r, 2 * i + 1] == grid[packed[r, i] >> 4]
    s = S.mxfp4_dequantize(np.full((1, 64), 0x22, np.uint8), np.array([[0, 1, 254, 255]], np.uint8))
    assert s[0, 0] == 2.0 ** -127 and s[0, 32] == 2.0 ** -126 and s[0, 64] == 2.0 ** 127 and np.isnan(s[0, 96])


def test_hand_block():
    """Largest magnitude 6.9: e = 2 - 2 = 0; ties go to the even code."""
    x = np.zeros(128)
    x[:16] = [6.9, -6.9, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.26, -0.74, 1.26, 1.74, 2.51, 3.49, 5.01]
    x[32] = 8.0                                    # the next binade: e = 1, 8 / 2 = 4
    x[33] = 0.5                                    # 0.25 of the grid's unit: a tie, to 0
    p, s = S.mxfp4_quantize(x[None])
    assert s.tolist() == [[127, 128, 127, 127]]
    v = S.mxfp4_dequantize(p, s)[0]
    assert v[:16].tolist() == [6, -6, 0, 1, 1, 2, 2, 4, 4, 0.5, -0.5, 1.5, 1.5, 3, 3, 6]
    assert v[32] == 8.0 and v[33] == 0.0 and not v[34:].any()
    assert p[0, 0] == 0xF7 and p[0, 16] == 0x06


def test_against_brute_force():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((40, 32)) * np.exp2(rng.integers(-20, 20, (40, 1)))
    p, s = S.mxfp4_quantize(x)
    v = S.mxfp4_dequantize(p, s)
    for b in range(40):
        unit = 2.0 ** (int(s[b, 0]) - 127)
        top = np.abs(x[b]).max()
        assert 4 * unit <= top < 8 * unit
        for a, q in zip(np.abs(x[b]), np.abs(v[b])):
            assert abs(a - q) == min(abs(a - unit * g) for g in S.E2M1_VALUES)


def test_zero_clamp_and_non_finite():
    x = np.zeros((1, 128))
    x[0, 32] = 2.0 ** -130                         # e clamps at -127: 2^-3 of the unit rounds to 0
    x[0, 64], x[0, 65] = np.inf, 1.0
    x[0, 96] = np.nan
    p, s = S.mxfp4_quantize(x)
    assert s.tolist() == [[127, 0, 255, 255]] and not p.any()
    x = np.full((1, 32), 2.0 ** -127)
    p, s = S.mxfp4_quantize(x)
    assert s[0, 0] == 0 and np.array_equal(S.mxfp4_dequantize(p, s), x)


def test_groups_are_independent():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((3, 128))
    p, s = S.mxfp4_quantize(x)
    for g in range(4):
        pg, sg = S.mxfp4_quantize(x[:, 32 * g:32 * g + 32])
        assert np.array_equal(pg, p[:, 16 * g:16 * g + 16]) and np.array_equal(sg[:, 0], s[:, g])


@pytest.mark.parametrize("T", [1, 3])
def test_scores_are_the_formula_on_dequantised_values(T):
    rng = np.random.default_rng(3)
    n = 70
    seqs = O.Seqs(np.array([n]), np.array([0, T]), np.array([[1, 0]]), 64)
    kI, sc = S.mxfp4_quantize(rng.standard_normal((128, 128)))
    q = rng.standard_normal((T, 64, 128)).astype(np.float32)
    bits = (q.view(np.uint32) >> 16).astype(np.uint16)
    w = rng.standard_normal((T, 64)).astype(np.float32)
    got = S.index_scores_mx4(seqs, bits, w, kI, sc)
    k = S.mxfp4_dequantize(kI, sc)
    for t in range(T):
        qv = S.mxfp4_dequantize(*S.mxfp4_quantize(O.bf16_to_f64(bits[t])))
        pos = n - T + t
        assert got[t].shape == (pos + 1,)
        for s in (0, 1, 63, 64, pos):
            row = (64 if s < 64 else 0) + s % 64
            want = sum(float(w[t, h]) * max(0.0, float(qv[h] @ k[row])) for h in range(64))
            assert abs(got[t][s] - want) < 1e-9
