"""The MXFP4 index cache on the GPU: quantiser, writer and reader bit for bit
against the oracle, the indexer's scores, and the whole path.

Tolerance of a score: products of E2M1 values are exact; the 128 products of a
dot are added in fp32 (each addition off by at most 2^-23, tensor cores may
truncate), then 64 weighted terms, so it is off by at most 2^-23 (130 sum_h |w_h|
|q_h| . |k| + 70 sum_h |w_h| relu_h)."""
import numpy as np
import pytest
import torch

from dsa_workloads import bits16, to_device
from oracle import dsa_oracle as O
from oracle import serving_oracle as S
from tests import parity as P
from tests.specs import SMALL, workload as make_workload

pytestmark = pytest.mark.gpu

SPECS = {n: SMALL[n].scaled(name=n + "_mx4", ki_fp8=False)
         for n in ("decode_small", "prefill_fp8_700", "chunked_small")}
SPECS["one_token"] = SPECS["decode_small"].scaled(name="one_token_mx4", batch=3, ctx=(1, 2), planted=0)
SPECS["page_edges"] = SPECS["decode_small"].scaled(name="page_edges_mx4", batch=5, ctx=(63, 66), planted=0)
SPECS["many_items"] = SPECS["decode_small"].scaled(name="many_items_mx4", batch=40, ctx=(900, 1100), planted=4)


def _cache(wl):
    """The workload's bf16 index keys as an MXFP4 cache (oracle's quantiser)."""
    kI, sc = S.mxfp4_quantize(O.bf16_to_f64(bits16(wl.kI)))
    return kI, sc


_made = {}


def _workload(name):
    if name not in _made:
        wl = make_workload(SPECS[name])
        _made[name] = (wl, *_cache(wl))
    return _made[name]


def _fold(packed):
    """Codes with the sign of a zero dropped."""
    c = np.stack([packed & 15, packed >> 4], -1)
    return np.where(c == 8, 0, c)


def _rows_for_quantiser():
    rng = np.random.default_rng(5)
    T = 13
    x = rng.standard_normal((T, 64, 128)) * np.exp2(rng.integers(-60, 60, (T, 64, 4)).repeat(32, axis=2))
    x[0, 0] = 0.0
    x[0, 1, :32] = 0.0
    x[0, 1, 32:48] = [6, -6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0]
    x[0, 1, 48:64] = 0.0
    x[0, 2] = rng.standard_normal(128) * 2.0 ** -130      # bf16 subnormals: the exponent clamps
    x[0, 3] = rng.standard_normal(128) * 2.0 ** 126       # the top of the range
    x[1, 0, :32] = 2.0 ** np.arange(-16, 16)
    x[2, 0, 5], x[2, 0, 40], x[2, 0, 70] = np.nan, np.inf, -np.inf
    return torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)


def test_quantise_and_back(lib):
    qI = _rows_for_quantiser()
    codes, scales = lib.dsa_quantize_index_query_mx4(qI.cuda())
    ref_codes, ref_scales = S.mxfp4_quantize(O.bf16_to_f64(bits16(qI)))
    assert np.array_equal(scales.cpu().numpy(), ref_scales)
    assert np.array_equal(_fold(codes.cpu().numpy()), _fold(ref_codes))
    back = lib.dsa_dequantize_mx4(codes, scales).float().cpu().numpy()
    assert np.array_equal(back, S.mxfp4_dequantize(ref_codes, ref_scales).astype(np.float32), equal_nan=True)


def test_dequantise_every_code(lib):
    codes = torch.arange(256, dtype=torch.uint8).repeat(64).view(256, 64)
    scales = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 4)
    got = lib.dsa_dequantize_mx4(codes.cuda(), scales.cuda()).cpu()
    ref = torch.from_numpy(S.mxfp4_dequantize(codes.numpy(), scales.numpy())).to(torch.bfloat16)
    assert torch.equal(got.nan_to_num(nan=7.0), ref.nan_to_num(nan=7.0))


@pytest.mark.parametrize("name", list(SPECS))
def test_append_writes_its_rows_alone(lib, name):
    wl, _, _ = _workload(name)
    d = to_device(wl)
    R = wl.num_phys_pages * 64
    g = torch.Generator().manual_seed(1)
    k = torch.randn((wl.T, 128), generator=g).to(torch.bfloat16)
    kI0 = torch.randint(0, 256, (R, 64), generator=g, dtype=torch.uint8)
    sc0 = torch.randint(0, 256, (R, 4), generator=g, dtype=torch.uint8)
    kI, sc = kI0.cuda(), sc0.cuda()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    lib.dsa_append_index_keys_mx4(d.seqs, k.cuda(), kI, sc, ws=ws)
    assert lib.dsa_check_error(ws) == lib.DSA_OK
    seqs = P.oracle_seqs(wl)
    want, wsc = kI0.numpy().copy(), sc0.numpy().copy()
    codes, scales = S.mxfp4_quantize(O.bf16_to_f64(bits16(k)))
    touched = np.zeros(R, bool)
    for t in range(wl.T):
        b, pos = seqs.token_seq_pos(t)
        r = seqs.rows(b, [pos])[0]
        want[r], wsc[r], touched[r] = codes[t], scales[t], True
    assert np.array_equal(sc.cpu().numpy(), wsc)
    got = kI.cpu().numpy()
    assert np.array_equal(got[~touched], want[~touched])
    assert np.array_equal(_fold(got[touched]), _fold(want[touched]))


def test_append_skips_what_it_cannot_place(lib):
    wl, _, _ = _workload("chunked_small")
    d = to_device(wl)
    R = wl.num_phys_pages * 64
    k = torch.randn(wl.T, 128).bfloat16().cuda()
    kI, sc = torch.full((R, 64), 7, dtype=torch.uint8).cuda(), torch.full((R, 4), 9, dtype=torch.uint8).cuda()
    for bad in (-1, wl.num_phys_pages):
        pt = torch.full_like(d.seqs.page_table, bad)
        seqs = lib.Seqs(d.seqs.q_seq_start, d.seqs.ctx_len, pt, d.seqs.num_phys_pages, d.seqs.max_ctx, wl.T)
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        lib.dsa_append_index_keys_mx4(seqs, k, kI, sc, ws=ws)
        assert lib.dsa_check_error(ws) == lib.DSA_ERR_BAD_INDEX
    cl = d.seqs.ctx_len.clone()
    cl[:] = d.seqs.max_ctx + 1
    seqs = lib.Seqs(d.seqs.q_seq_start, cl, d.seqs.page_table, d.seqs.num_phys_pages, d.seqs.max_ctx, wl.T)
    lib.dsa_append_index_keys_mx4(seqs, k, kI, sc, ws=ws)
    assert lib.dsa_check_error(ws) == lib.DSA_ERR_BAD_INDEX
    assert (kI == 7).all() and (sc == 9).all()


def _score_tolerance(wl, kI, sc, t):
    seqs = P.oracle_seqs(wl)
    b, pos = seqs.token_seq_pos(int(t))
    k = S.mxfp4_dequantize(kI, sc)[seqs.rows(b, np.arange(pos + 1))]
    q = S.mxfp4_dequantize(*S.mxfp4_quantize(O.bf16_to_f64(bits16(wl.qI[int(t)]))))
    w = np.abs(wl.w.numpy()[int(t)].astype(np.float64))
    return 2.0 ** -23 * (130 * w @ (np.abs(q) @ np.abs(k).T) + 70 * w @ np.maximum(q @ k.T, 0))


@pytest.mark.parametrize("name", list(SPECS))
def test_scores(lib, name):
    wl, kI, sc = _workload(name)
    d = to_device(wl)
    ws = torch.zeros(lib.dsa_workspace_size(lib.DSA_OP_INDEX_SCORES, d.seqs), dtype=torch.uint8, device="cuda")
    filled = torch.full((wl.T, (wl.max_ctx + 3) // 4 * 4), 123.0, device="cuda")
    lib.dsa_index_scores(d.seqs, d.qI, d.w, torch.from_numpy(kI).cuda(), torch.from_numpy(sc).cuda(), scores=filled,
                         ws=ws)
    assert lib.dsa_check_error(ws) == lib.DSA_OK
    tokens = np.arange(wl.T) if wl.T <= 64 else P.sample_tokens(wl, 24)
    ref = S.index_scores_mx4(P.oracle_seqs(wl), bits16(wl.qI), wl.w.numpy(), kI, sc, tokens=tokens)
    got = filled.cpu().numpy()
    pos = wl.token_pos()
    for t, r in zip(tokens, ref):
        err = np.abs(got[t, :pos[t] + 1] - r)
        tol = _score_tolerance(wl, kI, sc, t)
        assert (err <= tol).all(), (t, float((err / tol).max()))
        assert (got[t, pos[t] + 1:] == 123.0).all()        # entries past the position stay


def test_scales_pick_their_group(lib):
    """Doubling one group's scale changes what that group contributes, in keys and in queries."""
    wl, kI, sc = _workload("decode_small")
    d = to_device(wl)
    for g in range(4):
        moved = sc.copy()
        moved[:, g] += 3
        got = lib.dsa_index_scores(d.seqs, d.qI, d.w, torch.from_numpy(kI).cuda(), torch.from_numpy(moved).cuda())
        ref = S.index_scores_mx4(P.oracle_seqs(wl), bits16(wl.qI), wl.w.numpy(), kI, moved)
        for t, r in enumerate(ref):
            assert (np.abs(got[t, :len(r)].cpu().numpy() - r) <= _score_tolerance(wl, kI, moved, t)).all()
        import dataclasses
        q = wl.qI.clone()
        q[..., 32 * g:32 * g + 32] *= 8
        wl2 = dataclasses.replace(wl, qI=q)
        got = lib.dsa_index_scores(d.seqs, q.cuda(), d.w, torch.from_numpy(kI).cuda(), torch.from_numpy(sc).cuda())
        ref = S.index_scores_mx4(P.oracle_seqs(wl2), bits16(q), wl.w.numpy(), kI, sc)
        for t, r in enumerate(ref):
            assert (np.abs(got[t, :len(r)].cpu().numpy() - r) <= _score_tolerance(wl2, kI, sc, t)).all()


@pytest.mark.parametrize("name", ["decode_small", "chunked_small", "page_edges"])
@pytest.mark.parametrize("select", [False, True])
def test_whole_path(lib, name, select):
    """Selection and attention through the one call, against the separate stages
    (bit for bit) and the oracle's selection."""
    wl, kI, sc = _workload(name)
    if select and wl.T != wl.spec.batch:
        pytest.skip("the selection inside the indexer serves decode batches")
    d = to_device(wl)
    K = wl.spec.topk
    kI_d, sc_d = torch.from_numpy(kI).cuda(), torch.from_numpy(sc).cuda()
    idx = torch.empty((wl.T, K), dtype=torch.int32, device="cuda")
    out, lse = lib.dsa_index_topk_attn(d.seqs, d.qI, d.w, kI_d, sc_d, d.q, d.kv, K, wl.scale, idx_out=idx,
                                       out_dtype=torch.float32, select_in_indexer=select)
    scores = lib.dsa_index_scores(d.seqs, d.qI, d.w, kI_d, sc_d)
    pos = torch.from_numpy(wl.token_pos() + 1).int().cuda()
    assert torch.equal(idx, lib.dsa_topk(scores, pos, K))
    out2, lse2 = lib.dsa_sparse_mla_fwd(d.seqs, d.q, d.kv, idx, wl.scale, out_dtype=torch.float32)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    tokens = np.arange(wl.T) if wl.T <= 64 else P.sample_tokens(wl, 16)
    ref = S.index_scores_mx4(P.oracle_seqs(wl), bits16(wl.qI), wl.w.numpy(), kI, sc, tokens=tokens)
    for t, r in zip(tokens, ref):
        assert not P.selection_violations(idx[t].cpu().numpy(), r, K)


@pytest.mark.parametrize("name", ["decode_small", "chunked_small"])
def test_a_nan_block_makes_its_scores_nan(lib, name):
    """A key or a query with an infinity or NaN: scale byte 255 in its block, NaN in the
    scores that block enters, and nowhere else."""
    import dataclasses
    wl, kI, sc = _workload(name)
    seqs, d = P.oracle_seqs(wl), to_device(wl)
    k = torch.randn(wl.T, 128, generator=torch.Generator().manual_seed(3)).bfloat16()
    k[0, 40], k[1, 100] = float("nan"), -float("inf")
    q = wl.qI.clone()
    q[2, 5, 17] = float("inf")
    wl = dataclasses.replace(wl, qI=q)
    kI_d, sc_d = torch.from_numpy(kI).cuda(), torch.from_numpy(sc).cuda()
    lib.dsa_append_index_keys_mx4(d.seqs, k.cuda(), kI_d, sc_d)
    kI, sc = kI_d.cpu().numpy(), sc_d.cpu().numpy()
    got = lib.dsa_index_scores(d.seqs, q.cuda(), d.w, kI_d, sc_d).cpu().numpy()
    tokens = np.arange(wl.T) if wl.T <= 64 else np.unique([0, 1, 2, 3, *P.sample_tokens(wl, 16)])
    seen = 0
    for t, r in zip(tokens, S.index_scores_mx4(seqs, bits16(q), wl.w.numpy(), kI, sc, tokens=tokens)):
        nan = np.isnan(r)
        assert np.array_equal(np.isnan(got[t, :len(r)]), nan), t
        tol = _score_tolerance(wl, kI, sc, t)
        assert (np.abs(got[t, :len(r)] - r)[~nan] <= tol[~nan]).all()
        seen += nan.any()
        assert nan.all() == (t == 2)
    assert seen >= 3
    # the selection takes such a position before every number
    K = min(32, wl.spec.topk)
    for select in (False, True) if wl.T == wl.spec.batch else (False,):
        idx = torch.empty((wl.T, K), dtype=torch.int32, device="cuda")
        lib.dsa_index_topk_attn(d.seqs, q.cuda(), d.w, kI_d, sc_d, d.q, d.kv, K, wl.scale, idx_out=idx,
                                select_in_indexer=select)
        for t in (0, 1):
            assert int(wl.token_pos()[t]) in idx[t].tolist()


@pytest.mark.parametrize("select", [False, True])
@pytest.mark.parametrize("name", ["decode_small", "chunked_small", "many_items"])
def test_short_wait_limit_winds_down(lib, name, select):
    """A wait limit of 1 ns: producers, issuers and epilogue give up by themselves and say
    so (or were fast enough); the next calls are clean and give the same bits as before."""
    wl, kI, sc = _workload(name)
    if select and wl.T != wl.spec.batch:
        pytest.skip("the selection inside the indexer serves decode batches")
    d, K = to_device(wl), wl.spec.topk
    kI_d, sc_d = torch.from_numpy(kI).cuda(), torch.from_numpy(sc).cuda()
    op = lib.DSA_OP_INDEX_TOPK_ATTN_FUSED if select else lib.DSA_OP_INDEX_TOPK_ATTN
    spaces = [torch.zeros(lib.dsa_workspace_size(o, d.seqs, K, wl.spec.heads), dtype=torch.uint8, device="cuda")
              for o in (lib.DSA_OP_INDEX_SCORES, op)]

    def scores():
        return lib.dsa_index_scores(d.seqs, d.qI, d.w, kI_d, sc_d, ws=spaces[0])

    def path():
        idx = torch.empty((wl.T, K), dtype=torch.int32, device="cuda")
        out, lse = lib.dsa_index_topk_attn(d.seqs, d.qI, d.w, kI_d, sc_d, d.q, d.kv, K, wl.scale, idx_out=idx, ws=spaces[1],
                                           select_in_indexer=select)
        return idx, out, lse
    want = scores(), *path()
    assert [lib.dsa_check_error(w) for w in spaces] == [lib.DSA_OK] * 2
    for _ in range(5):
        lib.dsa_set_wait_limit_ns(1)
        try:
            scores()
            path()
        finally:
            lib.dsa_set_wait_limit_ns(0)
        assert all(lib.dsa_check_error(w) in (lib.DSA_OK, lib.DSA_ERR_TIMEOUT) for w in spaces)
        assert all(torch.equal(a, b) for a, b in zip(want, (scores(), *path())))
        assert [lib.dsa_check_error(w) for w in spaces] == [lib.DSA_OK] * 2
