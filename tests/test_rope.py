"""Rotary positions on the CPU: the frequency table against its formulas, the
fixed-point phase, the oracle's pins, and the binding's refusals."""
import math

import numpy as np
import pytest
import torch

import sparse_indexed_attention_b200 as dsa
from oracle import serving_oracle as S

CPU = torch.device("cpu")


def test_oracle_rotates_pairs():
    x = np.arange(1.0, 13.0).reshape(1, 1, 12)
    f = [math.pi / 2, math.pi]                    # a quarter turn and half a turn per position
    y = S.rope(x, [1], f, offset=4)[0, 0]
    assert np.allclose(y, [1, 2, 3, 4, -6, 5, -7, -8, 9, 10, 11, 12], atol=1e-14)
    y = S.rope(x, [1], f, offset=4, interleaved=False)[0, 0]
    assert np.allclose(y, [1, 2, 3, 4, -7, -6, 5, -8, 9, 10, 11, 12], atol=1e-14)
    back = S.rope(S.rope(x, [7], [0.3, 2e-3], 2, True, 1.5), [7], [0.3, 2e-3], 2, True, 1.5, transpose=True)
    assert np.allclose(back[..., 2:6], 2.25 * x[..., 2:6]) and np.array_equal(back[..., 6:], x[..., 6:])


def test_oracle_transpose_is_the_gradient():
    rng = np.random.default_rng(0)
    x, g = rng.standard_normal((2, 3, 2, 8))
    pos, f = [5, -2, 1000], [1.0, 0.1, 0.01]
    h = 1e-6
    dx = S.rope(g, pos, f, 1, False, 1.3, transpose=True)
    for i in np.ndindex(*x.shape):
        e = np.zeros_like(x)
        e[i] = h
        num = ((S.rope(x + e, pos, f, 1, False, 1.3) - S.rope(x - e, pos, f, 1, False, 1.3)) * g).sum() / (2 * h)
        assert abs(num - dx[i]) < 1e-7


def test_frequencies():
    F = dsa.RopeTable.frequencies
    assert np.allclose(F(8, 10000.0), [1, 0.1, 0.01, 0.001])
    assert np.allclose(F(8, 10000.0, scaling="linear", factor=4.0), [0.25, 0.025, 0.0025, 0.00025])
    n = F(8, 10000.0, scaling="ntk", factor=4.0)
    assert n[0] == 1.0 and math.isclose(n[3], 0.001 / 4.0, rel_tol=1e-12)
    y = F(64, 10000.0, scaling="yarn", factor=32.0, original_max=4096)
    base = F(64, 10000.0)
    low, high = 10, 23                             # 64 ln(4096 / (32 2pi)) / (2 ln 1e4) = 10.47, for 1 turn: 22.51
    for j in range(32):
        r = min(max((j - low) / (high - low), 0.0), 1.0)
        assert math.isclose(y[j], base[j] / 32 * r + base[j] * (1 - r), rel_tol=1e-12)


def test_phase_is_exact_far_out():
    """position * turns mod 2^64 is the phase, to well under fp32 resolution at position 2^24: the double's
    frequency is good to 2^-53, the table's unit is 2^-64."""
    t = dsa.RopeTable.build(64, 500000.0, device="cpu")
    f = dsa.RopeTable.frequencies(64, 500000.0)
    for p in (1, 131071, 2 ** 24 + 1, -77777):
        for j in (0, 1, 17, 31):
            got = (p * int(t.turns[j])) % 2 ** 64 / 2 ** 64
            want = S._phase(p, f[j]) / (2 * math.pi)
            assert abs((got - want + 0.5) % 1.0 - 0.5) < 2.0 ** -26


@pytest.mark.parametrize("kw", [dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=8, theta=1.0),
                                dict(rot_dim=8, scaling="dynamic"), dict(rot_dim=8, factor=2.0),
                                dict(rot_dim=8, scaling="linear", factor=0.5), dict(rot_dim=2, scaling="ntk", factor=2.0),
                                dict(rot_dim=8, scaling="yarn", factor=2.0, beta_fast=0.5),
                                dict(rot_dim=8, amplitude=math.nan)])
def test_table_refusals(kw):
    with pytest.raises(ValueError):
        dsa.RopeTable.build(device="cpu", **kw)


@pytest.fixture
def on_cpu(monkeypatch):
    """The binding's checks on CPU tensors; no call of these tests reaches a launch."""
    monkeypatch.setattr(dsa, "_cuda_device", lambda t, name: t.device)
    monkeypatch.setattr(dsa, "_stream", lambda dev: None)


def test_refusals(on_cpu):
    tab = dsa.RopeTable.build(8, device="cpu")
    x, pos = torch.zeros(4, 2, 16), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(TypeError, match="dtype"):
        dsa.dsa_rope(x.double(), pos, tab)
    with pytest.raises(TypeError, match="dtype"):
        dsa.dsa_rope(x, pos.float(), tab)
    with pytest.raises(ValueError, match="shape"):
        dsa.dsa_rope(x, pos[:3], tab)
    with pytest.raises(ValueError, match="shape"):
        dsa.dsa_rope(x[None], pos, tab)
    with pytest.raises(ValueError, match="last dim"):
        dsa.dsa_rope(x.transpose(1, 2), pos, tab)
    with pytest.raises(TypeError, match="RopeTable"):
        dsa.dsa_rope(x, pos, tab.turns)
    with pytest.raises(RuntimeError, match="gradient"):
        dsa.dsa_rope(x.clone().requires_grad_(), pos, tab)
    with pytest.raises(ValueError, match="shape"):
        dsa.dsa_rope(x, pos, tab, out=torch.zeros(4, 2, 8))
    for offset in (9, -1):
        with pytest.raises(dsa.DsaError, match="INVALID_ARG"):
            dsa.dsa_rope(x, pos, tab, offset=offset)
    big = dsa.RopeTable.build(1026, device="cpu")
    with pytest.raises(dsa.DsaError, match="UNSUPPORTED"):
        dsa.dsa_rope(torch.zeros(4, 1, 2048), pos, big)
    with pytest.raises(dsa.DsaError, match="INVALID_ARG"):      # every head in the same place
        dsa.dsa_rope(x, pos, tab, out=torch.zeros(4, 1, 16).expand(4, 2, 16))
    with pytest.raises(dsa.DsaError, match="INVALID_ARG"):
        dsa.dsa_rope(torch.zeros(1, 2, 16).expand(4, 2, 16), pos, tab, out=torch.zeros(1, 2, 16).expand(4, 2, 16))


def test_overlap_rule(on_cpu):
    tab = dsa.RopeTable.build(8, device="cpu")
    pos = torch.zeros(4, dtype=torch.int64)
    buf = torch.zeros(4 * 2 * 40)
    v = buf.view(4, 2, 40)

    def ok(x, out):
        T, H, D, xt, xh = dsa._rope_view(x, "x", CPU, x.dtype)
        return dsa._rope_disjoint(x, out, T, H, D, xt, xh, *dsa._rope_view(out, "out", CPU, x.dtype)[3:])

    def brute(x, out):
        at = lambda t: {t.storage_offset() + i * t.stride(0) + h * t.stride(1) + d for i in range(4)  # noqa: E731
                        for h in range(2) for d in range(t.shape[2])}
        same = x.data_ptr() == out.data_ptr() and x.stride() == out.stride()
        return same or not (at(x) & at(out))

    views = [v[..., a:a + 16] for a in range(0, 25, 4)] + [buf.view(2, 4, 40).transpose(0, 1)[..., 3:19],
                                                           buf[:128].view(4, 2, 16), buf[128:256].view(4, 2, 16)]
    for x in views:
        for out in views:
            assert not ok(x, out) or brute(x, out)             # never accepts an overlap
            if x.stride() == out.stride() and x.stride(1) == 40 and brute(x, out):
                assert ok(x, out)                              # slices of one buffer's rows are accepted
    with pytest.raises(ValueError, match="overlap"):
        dsa.dsa_rope(v[..., :16], pos, tab, out=v[..., 8:24])
