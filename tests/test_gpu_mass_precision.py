"""How exact the accumulated attention weight is, on inputs whose dot products leave
nothing to the tensor core's rounding, so that tight bounds follow by arithmetic.

exponent:  the dots are integers below 2^24, exact in any order.  The weight 2^(D c - L), c =
    scale log2(e), L = lse log2(e), is off by one fp32 rounding of the exponent r and one of its
    two parts' sum, 2^-23 |r| in all (c and L in two fp32 terms each are good to 2^-47), by 2^-22
    for 2^r, and the sum over half of the heads, at most H/8 + 2 additions deep, by 2^-24 for each.
tiles:  the dims 0..127 give 2^20, the dims 512..575 give -2^20, and the tiles between them
    multiples of 2^-4 below 2^9: within a tile every partial sum is exact in 24 bits, and only the
    additions of tiles 1, 2 and 3 to 2^20 round, each by 2^-4 at most.

Each half of the heads rounds its share to 2^-41.  Besides the kernel, each test holds the plain
arithmetic of the mistake it is there for against the same bound: one term for c or for L, and one
truncating chain over all dims."""
import dataclasses

import numpy as np
import pytest
import torch

from dsa_workloads import bits16, to_device
from oracle import dsa_oracle as O
from tests import parity as P
from tests.specs import SMALL, workload as make_workload

pytestmark = pytest.mark.gpu

UNIT, LOG2E, K = 2.0 ** -40, 1.0 / np.log(2.0), 300
BASE = SMALL["decode_small"].scaled(name="mass_precision", batch=4, ctx=(300, 900), topk=K, planted=0)


def _workload(heads, kv_fp8, q, kv, scale_bytes):
    """BASE with the query q [T, H, 576] and latent rows kv [R, 576] (before their tile scales)."""
    wl = make_workload(BASE.scaled(name=f"mass_precision_{heads}_{kv_fp8}", heads=heads, kv_fp8=kv_fp8))
    rng = np.random.default_rng(heads)
    q = torch.from_numpy(q(rng, wl.T, heads)).bfloat16()
    kv = kv(rng, wl.num_phys_pages * 64)
    if kv_fp8:
        codes = torch.from_numpy(kv).float().to(torch.float8_e4m3fn).view(torch.uint8)
        scales = torch.full((kv.shape[0], 8), 127, dtype=torch.uint8)
        scales[:, :5] = torch.tensor(scale_bytes, dtype=torch.uint8)
        return dataclasses.replace(wl, q=q, kv=codes, kv_scale=scales)
    kv = kv * 2.0 ** (np.repeat(np.array(scale_bytes) - 127, [128] * 4 + [64]))
    return dataclasses.replace(wl, q=q, kv=torch.from_numpy(kv).bfloat16(), kv_scale=None)


def _lists(wl):
    rng = np.random.default_rng(1)
    return np.stack([rng.choice(int(p) + 1, K, replace=int(p) + 1 < K) for p in wl.token_pos()]).astype(np.int32)


def _run(lib, wl, idx, lse, scale):
    d = to_device(wl)
    mass = torch.zeros((len(wl.ctx_len), wl.max_ctx), dtype=torch.int64, device="cuda")
    lib.dsa_attn_mass(d.seqs, d.q, d.kv, torch.from_numpy(idx).cuda(), torch.from_numpy(lse).cuda(), scale, mass,
                      kv_scale=d.kv_scale)
    return mass.cpu().numpy() * UNIT


def _tokens(wl, idx, scale):
    """Per token: its positions, the rows, the query in 64 bits, the dots and the fp32 lse."""
    seqs = P.oracle_seqs(wl)
    for t in range(wl.T):
        b, _ = seqs.token_seq_pos(t)
        s = np.unique(idx[t])
        kv = O.kv_rows(P.kv_host(wl), seqs.rows(b, s.astype(np.int64)))
        q = O.bf16_to_f64(bits16(wl.q[t]))
        dots = q @ kv.T
        x = scale * dots
        m = x.max(1, keepdims=True)
        lse = (m[:, 0] + np.log(np.exp(x - m).sum(1))).astype(np.float32)
        yield t, b, s, kv, q, dots, lse


def _dedup(wl, idx):
    """Each position once per list."""
    out = np.full_like(idx, -1)
    for t in range(len(idx)):
        s = np.unique(idx[t])
        out[t, :len(s)] = s
    return out


@pytest.mark.parametrize("kv_fp8", [False, True])
@pytest.mark.parametrize("heads", [16, 64, 128])
def test_large_logits(lib, heads, kv_fp8):
    base = np.random.default_rng(0).choice([-2.0, -1.0, 1.0, 2.0], 576)
    # one query for all heads: the errors of their lse do not cancel in the mean
    wl = _workload(heads, kv_fp8, lambda rng, T, H: (base * (rng.random((T, 1, 576)) > 0.1)).repeat(H, 1),
                   lambda rng, R: 3 * base + rng.integers(-1, 2, (R, 576)), [127] * 5)
    # of the scales near 1/20, one whose factor c is far from an fp32 number
    scales = np.float32(0.05) * (1 + np.arange(400, dtype=np.float32) * np.float32(2.0 ** -12))
    c = scales.astype(np.float64) * LOG2E
    scale = float(scales[np.argmax(np.abs(c - c.astype(np.float32)))])
    c, c32 = scale * LOG2E, float(np.float32(scale * LOG2E))
    idx = _dedup(wl, _lists(wl))
    lse = np.zeros((wl.T, heads), np.float32)
    shape = (len(wl.ctx_len), wl.max_ctx)
    ref, tol, one_c, one_l = (np.zeros(shape) for _ in range(4))
    for t, b, s, kv, q, dots, lse[t] in _tokens(wl, np.where(idx < 0, idx[:, :1], idx), scale):
        assert (np.abs(q) @ np.abs(kv).T).max() < 2 ** 24
        el = lse[t].astype(np.float64)[:, None] * LOG2E
        r = dots * c - el
        p = np.exp2(r)
        ref[b, s] += p.mean(0)
        off = p * (np.log(2) * (2.0 ** -23 * np.abs(r) + 2.0 ** -40) + 2.0 ** -22)
        tol[b, s] += off.mean(0) + p.mean(0) * (heads / 8 + 2) * 2.0 ** -24 + UNIT
        one_c[b, s] += np.exp2(dots * c32 - el).mean(0)
        one_l[b, s] += np.exp2(dots * c - el.astype(np.float32).astype(np.float64)).mean(0)
    got = _run(lib, wl, idx, lse, scale)
    err = np.abs(got - ref)
    assert (err <= tol).all(), float((err / np.maximum(tol, 1e-300)).max())
    seen = tol > 0
    assert (np.abs(one_c - ref) > tol)[seen].mean() > 0.9
    assert (np.abs(one_l - ref) > tol)[seen].mean() > 0.2          # a token's lse may happen to be near an fp32 number


@pytest.mark.parametrize("kv_fp8", [False, True])
@pytest.mark.parametrize("heads", [16, 64, 128])
def test_tiles_are_added_with_rounding(lib, heads, kv_fp8):
    def q(rng, T, H):
        x = rng.choice([-1.0, -0.5, 0.5, 1.0], (T, H, 576))
        x[..., :128] = x[..., 512:] = 1.0
        return x

    def kv(rng, R):
        x = rng.integers(-15, 16, (R, 576)) / 8.0
        x[:, :128], x[:, 512:] = 1.0, -1.0
        return x
    wl = _workload(heads, kv_fp8, q, kv, [140, 127, 127, 127, 141])       # 2^13 and -2^14
    scale = 0.125
    idx = _dedup(wl, _lists(wl))
    lse = np.zeros((wl.T, heads), np.float32)
    shape = (len(wl.ctx_len), wl.max_ctx)
    ref, tol, chain = (np.zeros(shape) for _ in range(3))
    for t, b, s, kv64, q64, dots, lse[t] in _tokens(wl, np.where(idx < 0, idx[:, :1], idx), scale):
        assert np.abs(q64[:, 128:512]).max() * np.abs(kv64[:, 128:512]).max() * 128 < 2 ** 9
        el = lse[t].astype(np.float64)[:, None] * LOG2E
        r = dots * scale * LOG2E - el
        p = np.exp2(r)
        ref[b, s] += p.mean(0)
        off = p * (np.expm1(scale * 3 * 2.0 ** -4) + np.log(2) * (2.0 ** -23 * np.abs(r) + 2.0 ** -40) + 2.0 ** -22)
        tol[b, s] += off.mean(0) + p.mean(0) * (heads / 8 + 2) * 2.0 ** -24 + UNIT
        acc = np.zeros_like(dots)                                          # 36 accumulations of 16 dims, each truncated
        for i in range(0, 576, 16):
            acc = acc + q64[:, i:i + 16] @ kv64[:, i:i + 16].T
            m, e = np.frexp(acc)
            acc = np.ldexp(np.trunc(np.ldexp(m, 24)), e - 24)
        chain[b, s] += np.exp2(acc * scale * LOG2E - el).mean(0)
    got = _run(lib, wl, idx, lse, scale)
    err = np.abs(got - ref)
    assert (err <= tol).all(), float((err / np.maximum(tol, 1e-300)).max())
    assert (np.abs(chain - ref) > tol)[tol > 0].mean() > 0.9
