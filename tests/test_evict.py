"""Eviction on the CPU: pins of the oracle and the host's refusals."""
import ctypes

import numpy as np
import pytest
import torch

import sparse_indexed_attention_b200 as dsa
from oracle import dsa_oracle as O
from oracle import serving_oracle as S


def test_select_by_hand():
    mass = np.array([[5, 1, 9, 1, 7, 1, 0, 3], [0] * 8, [8, 7, 6, 5, 4, 3, 2, 1]])
    keep, n = S.evict_select([8, 8, 3], mass, 4, recent=1, sink=1)
    assert keep.tolist() == [[0, 2, 4, 7], [0, 1, 2, 7], [0, 1, 2, -1]] and n.tolist() == [4, 4, 3]
    keep, _ = S.evict_select([8], mass[:1], 5)
    assert keep.tolist() == [[0, 1, 2, 4, 7]]              # 1, 3 and 5 tie: the lowest stays
    keep, _ = S.evict_select([4], [[2 ** 40 + 1, 2 ** 40, 2 ** 40 + 2, 2 ** 41]], 2)
    assert keep.tolist() == [[0, 3]]                       # equal in fp32


def test_mass_is_the_mean_probability():
    rng = np.random.default_rng(0)
    n, H = 70, 4
    seqs = O.Seqs(np.array([n]), np.array([0, 2]), np.array([[1, 0]]), 64)
    to16 = lambda x: (x.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)  # noqa: E731
    q, kv = to16(rng.standard_normal((2, H, 576))), to16(rng.standard_normal((128, 576)))
    idx = np.full((2, 80), -1)
    idx[0, :n - 1], idx[1, :n] = rng.permutation(n - 1), rng.permutation(n)
    _, lse = O.sparse_mla(seqs, q, kv, idx, 0.05)
    mass = S.attn_mass(seqs, q, kv, idx, 0.05, lse, 100)
    assert mass.shape == (1, 100) and abs(mass.sum() - 2.0) < 1e-12 and not mass[0, n:].any()
    rows = seqs.rows(0, np.arange(n))
    p = np.zeros(n)
    for t, m in ((0, n - 1), (1, n)):
        for h in range(H):
            e = np.exp(0.05 * (O.bf16_to_f64(kv[rows[:m]]) @ O.bf16_to_f64(q[t, h])))
            p[:m] += e / e.sum() / H
    assert np.allclose(mass[0, :n], p, rtol=1e-12)


P = ctypes.c_void_p
GOOD = P(0x10000)
BAD, WS, UNS = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_WORKSPACE, dsa.DSA_ERR_UNSUPPORTED


def _seqs(T=4, B=1, max_ctx=100, max_pages=2, phys=8):
    return ctypes.byref(dsa.DsaSeqsC(B, T, 64, max_pages, phys, max_ctx, 0x10000, 0x10000, 0x10000))


def test_mass_refusals():
    lib, f = dsa.raw(), ctypes.c_float(0.04)

    def call(kv_scale=None, kvd=dsa.DSA_KV_BF16, K=16, H=16, scale=f, lse=GOOD, mass=GOOD, ld=100, n=256, idx=GOOD):
        return lib.dsa_attn_mass(_seqs(), GOOD, GOOD, kv_scale, kvd, idx, K, H, scale, lse, mass, ld, GOOD, n, None)
    assert call(K=0) == UNS and call(K=2049) == UNS and call(H=48) == UNS
    assert call(lse=None) == BAD and call(mass=None) == BAD and call(ld=99) == BAD and call(idx=None) == BAD
    assert call(scale=ctypes.c_float(float("inf"))) == BAD and call(mass=P(0x10008)) == BAD
    assert call(kvd=dsa.DSA_KV_FP8_E4M3) == BAD and call(n=255) == WS


def test_select_refusals():
    lib = dsa.raw()

    def call(B=2, ctx=100, ld=100, budget=8, recent=2, sink=2, mass=GOOD, n=256):
        return lib.dsa_evict_select(GOOD, B, ctx, mass, ld, budget, recent, sink, GOOD, GOOD, GOOD, n, None)
    assert call(B=0) == BAD and call(ld=99) == BAD and call(budget=0) == BAD and call(mass=None) == BAD
    assert call(recent=7) == BAD and call(recent=9, sink=0) == BAD and call(recent=-1) == BAD and call(n=8) == WS
    assert call(sink=2 ** 31 - 1) == BAD and call(ctx=2 ** 30 + 1, ld=2 ** 31) == UNS


def test_compact_refusals():
    lib = dsa.raw()
    rows = 8 * 64

    def call(pools=((0x100000, 0x100000, 128),), budget=64, pages=2, new=8, mass=(None, 0, None, 0), n=1 << 20,
             max_ctx=100):
        cp = (dsa.DsaPoolC * 9)()
        for i, (s, d, r) in enumerate(pools):
            cp[i].src, cp[i].dst, cp[i].row_bytes = s, d, r
        return lib.dsa_evict_compact(_seqs(max_ctx=max_ctx), GOOD, GOOD, budget, GOOD, pages, new, cp, len(pools),
                                     *mass, GOOD, n, None)
    size = rows * 128
    apart = 0x100000 + size
    assert call(budget=0) == BAD and call(new=0) == BAD and call(pages=1, budget=65) == BAD
    assert call(pools=((0x100000, 0x100000, 6),)) == UNS and call(pools=((0x100000, 0x100000, 65540),)) == UNS
    assert call(pools=((0x100000, 0x100008, 128),)) == BAD                    # alignment
    assert call(pools=((0x100000, apart - 64, 128),)) == BAD                  # overlap without being the same
    assert call(pools=((0x100000, 0x100000, 128), (0x100000 + 64, 0x900000, 128))) == BAD   # another source inside it
    assert call(pools=((0x100000, 0x900000, 128), (0x200000, 0x900000, 128))) == BAD        # one destination twice
    assert call(pools=((0x100000, 0x100000, 128),) * 2) == BAD
    assert call(pools=((0x100000, 0x900000, 128),) * 9) == BAD
    assert call(mass=(GOOD, 100, None, 0)) == BAD and call(mass=(GOOD, 100, GOOD, 100)) == BAD
    assert call(mass=(GOOD, 99, P(0x900000), 100)) == BAD and call(mass=(GOOD, 100, P(0x900000), 63)) == BAD
    assert call(n=256) == WS
    s = dsa.DsaSeqsC(1, 1, 64, 1, 8, 1, None, None, None)
    assert lib.dsa_workspace_size(dsa.DSA_OP_EVICT_COMPACT, ctypes.byref(s), 1, 16) == 512
    assert lib.dsa_workspace_size(dsa.DSA_OP_ATTN_MASS, ctypes.byref(s), 1, 16) == 256
    assert lib.dsa_workspace_size(10, ctypes.byref(s), 1, 16) == 0


def test_binding_refusals(monkeypatch):
    monkeypatch.setattr(dsa, "_cuda_device", lambda t, name: t.device)
    seqs = dsa.Seqs(torch.tensor([0, 1], dtype=torch.int32), torch.tensor([5], dtype=torch.int32),
                    torch.zeros(1, 1, dtype=torch.int32), 1, 5, 1)
    q, kv = torch.zeros(1, 16, 576).bfloat16(), torch.zeros(64, 576).bfloat16()
    idx, lse, mass = torch.zeros(1, 8).int(), torch.zeros(1, 16), torch.zeros(1, 5).long()
    with pytest.raises(ValueError, match="max_ctx"):
        dsa.dsa_attn_mass(seqs, q, kv, idx, lse, 0.1, mass[:, :4].contiguous())
    with pytest.raises(TypeError, match="dtype"):
        dsa.dsa_attn_mass(seqs, q, kv, idx, lse, 0.1, mass.float())
    with pytest.raises(ValueError, match="shape"):
        dsa.dsa_attn_mass(seqs, q, kv, idx, lse[:, :8].contiguous(), 0.1, mass)
    with pytest.raises(TypeError, match="dtype"):
        dsa.dsa_attn_mass(seqs, q, kv, idx, lse, 0.1, mass, kv_scale=torch.zeros(64, 8).byte())
    ctx = torch.tensor([5], dtype=torch.int32)
    for kw in (dict(budget=0), dict(budget=4, recent=3, sink=2), dict(budget=4, sink=-1)):
        with pytest.raises(ValueError, match="budget"):
            dsa.dsa_evict_select(ctx, mass, **kw)
    with pytest.raises(ValueError, match="shape"):
        dsa.dsa_evict_select(ctx.repeat(2), mass, 4)
    keep, n, table = torch.zeros(1, 4).int(), torch.zeros(1).int(), torch.zeros(1, 1).int()
    with pytest.raises(ValueError, match="at least 64"):
        dsa.dsa_evict_compact(seqs, keep, n, table, [kv[:63]])
    with pytest.raises(TypeError, match="dtype"):
        dsa.dsa_evict_compact(seqs, keep, n, table, [(kv, kv.float())])
    with pytest.raises(ValueError, match="shape"):
        dsa.dsa_evict_compact(seqs, keep, n, table, [(kv, kv[:, :512].contiguous())])
    with pytest.raises(ValueError, match="contiguous"):
        dsa.dsa_evict_compact(seqs, keep, n, table, [torch.zeros(64, 8)[:, :4]])
    with pytest.raises(TypeError, match="tensor"):
        dsa.dsa_evict_compact(seqs, keep, n, table, [(kv, None)])
    with pytest.raises(TypeError, match="torch.Tensor"):
        dsa.dsa_evict_compact(seqs, keep, n, table, [kv], mass=mass)
    with pytest.raises(ValueError, match="at most 8"):
        dsa.dsa_evict_compact(seqs, keep, n, table, [kv] * 9)
