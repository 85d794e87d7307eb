"""Eviction on the GPU against the float64 oracle.

Tolerance of the mass: a logit's 576 exact products are added in fp32 (each
addition off by at most 2^-23 of what is added), its use in 2^x adds 2^-21 (1 +
|logit|) at most, and 2^x is good to 2^-22: p is off by p times the sum of those.
Each addition to the mass rounds to 2^-41."""
import numpy as np
import pytest
import torch

from dsa_workloads import bits16, to_device
from oracle import dsa_oracle as O
from oracle import serving_oracle as S
from tests import parity as P
from tests.specs import SMALL, workload as make_workload

pytestmark = pytest.mark.gpu

UNIT = 2.0 ** -40
MASS = {
    "decode_h128": SMALL["decode_small"],
    "decode_h16_fp8": SMALL["decode_small"].scaled(name="decode_h16_fp8", heads=16, topk=300, kv_fp8=True),
    "chunked_h64": SMALL["chunked_small"],
    "chunked_h32_fp8": SMALL["chunked_small"].scaled(name="chunked_h32_fp8", heads=32, topk=77, kv_fp8=True, batch=2,
                                                     chunk=(3, 40)),
    "prefill_h128_fp8": SMALL["prefill_fp8_700"].scaled(name="prefill_h128_fp8", heads=128, kv_fp8=True, ctx=(200, 200)),
    "one_token": SMALL["decode_small"].scaled(name="mass_one", batch=3, ctx=(1, 2), topk=1, planted=0),
    "full_list": SMALL["decode_small"].scaled(name="mass_2048", batch=2, ctx=(2100, 3000), topk=2048, heads=64),
}


def _lists(wl, seed=0):
    """Distinct causal positions in random order, unused slots scattered among them."""
    rng = np.random.default_rng(seed)
    idx = np.full((wl.T, wl.spec.topk), -1, np.int32)
    for t, pos in enumerate(wl.token_pos()):
        m = min(wl.spec.topk, int(pos) + 1)
        m = m if t % 3 else max(1, m // 2)
        idx[t, rng.choice(wl.spec.topk, m, replace=False)] = rng.choice(int(pos) + 1, m, replace=False)
    return idx


def _reference(wl, idx, lse):
    seqs = P.oracle_seqs(wl)
    mass, tol = np.zeros((len(wl.ctx_len), wl.max_ctx)), np.zeros((len(wl.ctx_len), wl.max_ctx))
    for t in range(wl.T):
        b, _ = seqs.token_seq_pos(t)
        s = idx[t][idx[t] >= 0].astype(np.int64)
        kv = O.kv_rows(P.kv_host(wl), seqs.rows(b, s))
        q = O.bf16_to_f64(bits16(wl.q[t]))
        x = wl.scale * (q @ kv.T)
        p = np.exp(x - lse[t].astype(np.float64)[:, None])
        off = wl.scale * 576 * 2.0 ** -23 * (np.abs(q) @ np.abs(kv).T) + 2.0 ** -21 * (1 + np.abs(x)) + 2.0 ** -22 \
            + 2.0 ** -23 * np.abs(lse[t].astype(np.float64))[:, None]
        mass[b, s] += p.mean(0)
        tol[b, s] += (p * off).mean(0) + UNIT
    return mass, tol


@pytest.mark.parametrize("name", list(MASS))
def test_mass(lib, name):
    wl = make_workload(MASS[name])
    d = to_device(wl)
    idx = _lists(wl)
    seqs = P.oracle_seqs(wl)
    _, lse = O.sparse_mla(seqs, bits16(wl.q), P.kv_host(wl), idx, wl.scale)
    lse = lse.astype(np.float32)
    ref, tol = _reference(wl, idx, lse)
    B, ld = wl.spec.batch, wl.max_ctx + 3
    mass = torch.full((B, ld), 5, dtype=torch.int64, device="cuda")
    idx_d, lse_d = torch.from_numpy(idx).cuda(), torch.from_numpy(lse).cuda()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    args = (d.seqs, d.q, d.kv, idx_d, lse_d, wl.scale)
    assert lib.dsa_attn_mass(*args, mass, kv_scale=d.kv_scale, ws=ws) is mass
    assert lib.dsa_check_error(ws) == lib.DSA_OK and lib.dsa_launches_in_last_call() == 1
    got = (mass.cpu().numpy() - 5) * UNIT
    assert not got[:, wl.max_ctx:].any()
    err = np.abs(got[:, :wl.max_ctx] - ref)
    assert (err <= tol).all(), float((err / np.maximum(tol, 1e-300)).max())
    # added to what is there, and the same bits in any order of additions
    again = mass.clone()
    lib.dsa_attn_mass(*args, again, kv_scale=d.kv_scale, ws=ws)
    assert torch.equal(again - mass, mass - 5)
    # the framework's own lse serves as well
    out, lse2 = lib.dsa_sparse_mla_fwd(d.seqs, d.q, d.kv, idx_d, wl.scale, kv_scale=d.kv_scale)
    own = torch.zeros((B, ld), dtype=torch.int64, device="cuda")
    lib.dsa_attn_mass(d.seqs, d.q, d.kv, idx_d, lse2, wl.scale, own, kv_scale=d.kv_scale, ws=ws)
    total = own.sum(1).cpu().numpy() * UNIT
    q_len = np.diff(wl.q_seq_start)
    assert np.abs(total - q_len).max() <= 2e-3 * q_len.max()      # each token's weights add up to one


def test_mass_rows_without_entries_and_odd_values(lib):
    wl = make_workload(MASS["decode_h128"])
    d = to_device(wl)
    idx = torch.full((wl.T, 130), -1, dtype=torch.int32, device="cuda")
    idx[0, 7] = 3
    lse = torch.zeros((wl.T, 128), device="cuda")
    kv = d.kv.clone()
    used = int(d.seqs.page_table[0, 0]) * 64 + 3
    other = torch.ones(kv.shape[0], dtype=torch.bool, device="cuda")
    other[used] = False
    kv[other] = float("nan")                      # rows that no list names
    q = d.q.clone()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def run(q=q, lse=lse, idx=idx, kv=kv):
        mass = torch.zeros((wl.spec.batch, wl.max_ctx), dtype=torch.int64, device="cuda")
        lib.dsa_attn_mass(d.seqs, q, kv, idx, lse, wl.scale, mass, ws=ws)
        return mass
    x = (q[0].double() @ kv[used].double()) * wl.scale
    m = run(lse=(x + 2.0).float().expand(wl.T, 128).contiguous())
    assert abs(int(m[0, 3]) * UNIT - np.exp(-2.0)) < 1e-4 and int((m != 0).sum()) == 1
    assert int(run(lse=torch.full_like(lse, float("inf"))).abs().sum()) == 0
    assert int(run(lse=torch.full_like(lse, float("nan"))).abs().sum()) == 0
    assert int(run(lse=torch.full_like(lse, -1e4))[0, 3]) == 2 ** 40          # limited to one
    assert int(run(lse=torch.full_like(lse, -float("inf")))[0, 3]) == 2 ** 40
    bad = kv.clone()
    bad[used] = float("nan")
    assert int(run(kv=bad).abs().sum()) == 0
    assert lib.dsa_check_error(ws) == lib.DSA_OK
    wrong = idx.clone()
    wrong[0, 8], wrong[1, 0] = int(wl.token_pos()[0]) + 1, -2
    assert torch.equal(run(idx=wrong) != 0, run() != 0)
    assert lib.dsa_check_error(ws) == lib.DSA_ERR_BAD_INDEX
    pt = d.seqs.page_table.clone()
    pt[0, 0] = wl.num_phys_pages
    seqs = lib.Seqs(d.seqs.q_seq_start, d.seqs.ctx_len, pt, d.seqs.num_phys_pages, d.seqs.max_ctx, wl.T)
    mass = torch.zeros((wl.spec.batch, wl.max_ctx), dtype=torch.int64, device="cuda")
    lib.dsa_attn_mass(seqs, q, kv, idx, lse, wl.scale, mass, ws=ws)
    assert lib.dsa_check_error(ws) == lib.DSA_ERR_BAD_INDEX and not mass.any()


def test_mass_one_position_from_many_tokens(lib):
    """Every token of a prompt attends to the same few positions: colliding additions."""
    wl = make_workload(MASS["chunked_h64"])
    d = to_device(wl)
    idx = torch.full((wl.T, 5), -1, dtype=torch.int32, device="cuda")
    idx[:, 0], idx[:, 3] = 0, 1
    _, lse = lib.dsa_sparse_mla_fwd(d.seqs, d.q, d.kv, idx[:, :4].contiguous(), wl.scale)
    runs = []
    for _ in range(3):
        mass = torch.zeros((wl.spec.batch, wl.max_ctx), dtype=torch.int64, device="cuda")
        lib.dsa_attn_mass(d.seqs, d.q, d.kv, idx, lse, wl.scale, mass)
        runs.append(mass)
    assert torch.equal(runs[0], runs[1]) and torch.equal(runs[0], runs[2])
    q_len = torch.from_numpy(np.diff(wl.q_seq_start)).double()
    got = runs[0].sum(1).cpu().double() * UNIT
    assert ((got - q_len).abs() <= 2e-3 * q_len).all()


@pytest.mark.parametrize("kv_fp8", [False, True])
@pytest.mark.parametrize("heads", [64, 128])
def test_mass_short_wait_limit_winds_down(lib, heads, kv_fp8):
    """A wait limit of 1 ns: the kernel gives up by itself and says so (or was
    fast enough); the next call is clean and right."""
    wl = make_workload(SMALL["decode_small"].scaled(name=f"limit_{heads}_{kv_fp8}", heads=heads, kv_fp8=kv_fp8))
    d = to_device(wl)
    idx = torch.from_numpy(_lists(wl)).cuda()
    _, lse = lib.dsa_sparse_mla_fwd(d.seqs, d.q, d.kv, idx, wl.scale, kv_scale=d.kv_scale)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def run():
        mass = torch.zeros((wl.spec.batch, wl.max_ctx), dtype=torch.int64, device="cuda")
        lib.dsa_attn_mass(d.seqs, d.q, d.kv, idx, lse, wl.scale, mass, kv_scale=d.kv_scale, ws=ws)
        return mass
    want = run()
    assert lib.dsa_check_error(ws) == lib.DSA_OK
    lib.dsa_set_wait_limit_ns(1)
    try:
        run()
    finally:
        lib.dsa_set_wait_limit_ns(0)
    assert lib.dsa_check_error(ws) in (lib.DSA_OK, lib.DSA_ERR_TIMEOUT)
    assert torch.equal(run(), want) and lib.dsa_check_error(ws) == lib.DSA_OK


def test_mass_negative_and_zero_scale(lib):
    wl = make_workload(MASS["decode_h16_fp8"])
    d = to_device(wl)
    idx = _lists(wl)
    for scale in (-0.03, 0.0):
        _, lse = O.sparse_mla(P.oracle_seqs(wl), bits16(wl.q), P.kv_host(wl), idx, scale)
        mass = torch.zeros((wl.spec.batch, wl.max_ctx), dtype=torch.int64, device="cuda")
        lib.dsa_attn_mass(d.seqs, d.q, d.kv, torch.from_numpy(idx).cuda(), torch.from_numpy(lse).float().cuda(), scale,
                          mass, kv_scale=d.kv_scale)
        ref = S.attn_mass(P.oracle_seqs(wl), bits16(wl.q), P.kv_host(wl), idx, scale, lse.astype(np.float32), wl.max_ctx)
        got = mass.cpu().numpy() * UNIT
        assert np.abs(got - ref).max() <= 2e-3 * ref.max() and np.array_equal(got > 0, ref > 0)


def test_mass_query_with_extreme_heads(lib):
    """FP8 cache: heads of zeros, of subnormals, of huge values, and values far below their head's largest."""
    wl = make_workload(MASS["decode_h16_fp8"])
    d = to_device(wl)
    q = wl.q.clone().double()
    q[:, 0] = 0.0
    q[:, 1] *= 2.0 ** -130
    q[:, 2] *= 2.0 ** -60
    q[:, 3, 10:] *= 2.0 ** -12
    q[:, 4, ::2] *= 2.0 ** -20
    q = q.to(torch.bfloat16)
    idx = _lists(wl)
    _, lse = O.sparse_mla(P.oracle_seqs(wl), bits16(q), P.kv_host(wl), idx, wl.scale)
    lse = lse.astype(np.float32)
    import dataclasses
    ref, tol = _reference(dataclasses.replace(wl, q=q), idx, lse)
    mass = torch.zeros((wl.spec.batch, wl.max_ctx), dtype=torch.int64, device="cuda")
    args = (d.seqs, q.cuda(), d.kv, torch.from_numpy(idx).cuda())
    lib.dsa_attn_mass(*args, torch.from_numpy(lse).cuda(), wl.scale, mass, kv_scale=d.kv_scale)
    # the query's two terms: off by 2^-22 of the head's largest value at most, per dim
    kv = np.abs(O.kv_rows(P.kv_host(wl), np.arange(wl.num_phys_pages * 64))).sum(1).max()
    top = float(q.abs().amax(-1).double().max())
    assert (np.abs(mass.cpu().numpy() * UNIT - ref) <= tol + ref * wl.scale * kv * top * 2.0 ** -22).all()
    inf = q.clone()
    inf[0, 5, 7] = float("inf")
    mass.zero_()
    lib.dsa_attn_mass(d.seqs, inf.cuda(), d.kv, args[3], torch.from_numpy(lse).cuda(), wl.scale, mass,
                      kv_scale=d.kv_scale)
    # the infinite head's half of the heads adds nothing for its token
    assert mass[0].sum() < 0.8 * 2 ** 40 and abs(int(mass[1].sum()) * UNIT - 1.0) < 2e-3


@pytest.mark.parametrize("kv_fp8", [False, True])
@pytest.mark.parametrize("heads", [16, 64, 128])
def test_mass_many_blocks_and_waves(lib, heads, kv_fp8):
    """Full lists for more tokens than SMs, again and again: every wait ends, and
    every run adds the same integers."""
    wl = make_workload(SMALL["chunked_small"].scaled(name=f"waves_{heads}_{kv_fp8}", heads=heads, kv_fp8=kv_fp8,
                                                     batch=2, prefix=(2100, 2200), chunk=(190, 200), topk=2048))
    d = to_device(wl)
    idx = torch.from_numpy(np.tile(np.arange(2048, dtype=np.int32), (wl.T, 1))).cuda()
    _, lse = lib.dsa_sparse_mla_fwd(d.seqs, d.q, d.kv, idx, wl.scale, kv_scale=d.kv_scale)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    first = None
    for _ in range(40):
        mass = torch.zeros((2, wl.max_ctx), dtype=torch.int64, device="cuda")
        lib.dsa_attn_mass(d.seqs, d.q, d.kv, idx, lse, wl.scale, mass, kv_scale=d.kv_scale, ws=ws)
        first = mass if first is None else first
        assert torch.equal(mass, first)
    assert lib.dsa_check_error(ws) == lib.DSA_OK
    q_len = torch.from_numpy(np.diff(wl.q_seq_start)).double()
    assert ((first.sum(1).cpu().double() * UNIT - q_len).abs() <= 2e-3 * q_len).all()


# ---------------------------------------------------------------------------


def _masses(B, n, kind, seed=0):
    g = torch.Generator().manual_seed(seed)
    if kind == "zero":
        return torch.zeros((B, n), dtype=torch.int64)
    if kind == "few":
        return torch.randint(0, 3, (B, n), generator=g)
    if kind == "ends":                             # the whole range of the type
        m = torch.randint(-2 ** 62, 2 ** 62, (B, n), generator=g)
        m[:, ::7] = 2 ** 63 - 1
        m[:, 1::11] = -2 ** 63
        return m
    return torch.exp(3 * torch.randn((B, n), generator=g)).mul(2.0 ** 28).long() * (torch.rand((B, n), generator=g) > 0.3)


@pytest.mark.parametrize("kind", ["zero", "few", "ends", "heavy"])
@pytest.mark.parametrize("n,budget,recent,sink", [
    (1, 1, 0, 0), (5, 5, 2, 2), (7, 3, 3, 0), (64, 63, 0, 4), (1000, 1, 0, 0), (4096, 2049, 64, 4),
    (4097, 100, 0, 0), (5003, 4999, 7, 3), (33000, 8192, 256, 4), (50021, 3, 1, 1)])
def test_select(lib, n, budget, recent, sink, kind):
    ctx = [n, max(0, n - 3), 0, min(n, budget), n // 2, min(n, budget + 1)]
    mass = _masses(len(ctx), n + 2, kind)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    keep, lens = lib.dsa_evict_select(torch.tensor(ctx, dtype=torch.int32).cuda(), mass.cuda(), budget, recent, sink,
                                      ws=ws)
    assert lib.dsa_check_error(ws) == lib.DSA_OK
    ref, ref_len = S.evict_select(ctx, mass.numpy(), budget, recent, sink)
    assert np.array_equal(lens.cpu().numpy(), ref_len)
    assert np.array_equal(keep.cpu().numpy(), ref)


@pytest.mark.parametrize("kind", ["few", "heavy"])
@pytest.mark.parametrize("B,n", [(3, 1024), (2, 1025), (5, 2049), (40, 3001), (75, 2500), (149, 1500), (300, 700),
                                 (19, 9000), (80, 45000)])
def test_select_batches(lib, B, n, kind):
    """Every size of cluster and block that batches of these sizes take."""
    budget, recent, sink = n // 3, 17, 3
    ctx = [n - 5 * b % (n - budget // 2) for b in range(B)]
    mass = _masses(B, n + 1, kind)
    keep, lens = lib.dsa_evict_select(torch.tensor(ctx, dtype=torch.int32).cuda(), mass.cuda(), budget, recent, sink)
    ref, ref_len = S.evict_select(ctx, mass.numpy(), budget, recent, sink)
    assert np.array_equal(lens.cpu().numpy(), ref_len)
    assert np.array_equal(keep.cpu().numpy(), ref)


@pytest.mark.parametrize("extra", [-3, 0, 1003])
def test_select_past_shared_memory(lib, extra):
    """A sequence whose keys do not fit the cluster's shared memory is read again instead."""
    n, budget = 8 * 40960 + extra, 100001
    mass = _masses(2, n, "heavy")
    ctx = torch.tensor([n, n - 77], dtype=torch.int32)
    keep, lens = lib.dsa_evict_select(ctx.cuda(), mass.cuda(), budget, recent=1000, sink=5)
    assert lens.tolist() == [budget, budget]
    for b in range(2):
        m = mass[b, :ctx[b]].float().numpy().astype(np.float64)
        m[:5] = m[int(ctx[b]) - 1000:] = np.inf
        want = np.sort(np.lexsort((np.arange(len(m)), -m))[:budget])
        assert np.array_equal(keep[b].cpu().numpy(), want)


def test_select_bad_lengths(lib):
    mass = _masses(3, 50, "heavy").cuda()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    keep, lens = lib.dsa_evict_select(torch.tensor([51, 20, -1], dtype=torch.int32).cuda(), mass, 8, ws=ws)
    assert lib.dsa_check_error(ws) == lib.DSA_ERR_BAD_INDEX
    assert lens.tolist() == [0, 8, 0] and (keep[0] == -1).all() and (keep[2] == -1).all() and (keep[1] >= 0).all()


# ---------------------------------------------------------------------------


def _cache(ctx, new_pages_each, seed=0):
    """Page tables of ragged sequences and spare pages for their new caches."""
    rng = np.random.default_rng(seed)
    pages = [(n + 63) // 64 for n in ctx]
    total = sum(pages) + len(ctx) * new_pages_each + 3
    perm = rng.permutation(total).astype(np.int32)
    table = np.full((len(ctx), max(max(pages), 1)), -1, np.int32)
    at = 0
    for b, p in enumerate(pages):
        table[b, :p] = perm[at:at + p]
        at += p
    return table, perm[at:at + len(ctx) * new_pages_each].reshape(len(ctx), -1), total


def _seqs(lib, ctx, table, total):
    B = len(ctx)
    return lib.Seqs(torch.arange(B + 1, dtype=torch.int32).cuda(), torch.tensor(ctx, dtype=torch.int32).cuda(),
                    torch.from_numpy(table).cuda(), total, max(max(ctx), 1), B)


def _rows(table, s):
    return table[s // 64].astype(np.int64) * 64 + s % 64


@pytest.mark.parametrize("inside", [True, False])
@pytest.mark.parametrize("ctx,budget", [([1, 2], 1), ([64, 65, 0, 300], 64), ([1000, 130, 999], 129), ([700], 2000)])
def test_compact(lib, ctx, budget, inside):
    new = (min(budget, max(ctx)) + 63) // 64
    table, new_table, total = _cache(ctx, new)
    g = torch.Generator().manual_seed(3)
    pools = [torch.randn((total * 64, 576), generator=g).bfloat16(),                      # 1152-byte rows
             torch.randint(0, 256, (total * 64, 64), generator=g, dtype=torch.uint8),
             torch.randint(0, 256, (total * 64, 8), generator=g, dtype=torch.uint8),
             torch.randint(0, 256, (total * 64, 4), generator=g, dtype=torch.uint8),
             torch.randn(total * 64, generator=g),                                        # one fp32 per row
             torch.randint(0, 256, (total * 64, 2, 10), generator=g, dtype=torch.uint8)]
    mass = _masses(len(ctx), max(ctx) + 1, "heavy")
    seqs = _seqs(lib, ctx, table, total)
    keep, lens = lib.dsa_evict_select(seqs.ctx_len, mass.cuda(), budget, recent=min(budget, 1))
    src = [p.cuda() for p in pools]
    dst = src if inside else [torch.full_like(p, 7) for p in src]
    new_mass = torch.full((len(ctx), new * 64), -1, dtype=torch.int64, device="cuda")
    ws = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    lib.dsa_evict_compact(seqs, keep, lens, torch.from_numpy(new_table).cuda(),
                          src if inside else list(zip(src, dst)), mass=mass.cuda(), new_mass=new_mass, ws=ws)
    assert lib.dsa_check_error(ws) == lib.DSA_OK and lib.dsa_launches_in_last_call() == 2
    want = [p.clone() if inside else torch.full_like(p, 7) for p in pools]
    want_mass = torch.full((len(ctx), new * 64), -1, dtype=torch.int64)
    for b, n in enumerate(lens.tolist()):
        k = keep[b, :n].cpu().numpy().astype(np.int64)
        to, frm = torch.from_numpy(_rows(new_table[b], np.arange(n))), torch.from_numpy(_rows(table[b], k))
        for w, p in zip(want, pools):
            w[to] = p[frm]
        want_mass[b, :n] = mass[b, torch.from_numpy(k)]
    for w, p in zip(want, dst):
        assert torch.equal(p.cpu(), w)
    assert torch.equal(new_mass.cpu(), want_mass)


def test_compact_refuses_pages_in_use(lib):
    ctx, budget = [300, 200], 100
    table, new_table, total = _cache(ctx, 2)
    pool0 = torch.randn((total * 64, 8))
    seqs = _seqs(lib, ctx, table, total)
    keep, lens = lib.dsa_evict_select(seqs.ctx_len, _masses(2, 300, "heavy").cuda(), budget)
    ws = torch.zeros(4096, dtype=torch.uint8, device="cuda")

    def run(nt, keep=keep, lens=lens, dst=None):
        pool = pool0.cuda()
        lib.dsa_evict_compact(seqs, keep, lens, torch.from_numpy(nt).cuda(), [pool if dst is None else (pool, dst)],
                              ws=ws)
        return pool.cpu() if dst is None else dst.cpu(), lib.dsa_check_error(ws)
    good, st = run(new_table)
    assert st == lib.DSA_OK
    read, twice, off = (new_table.copy() for _ in range(3))
    read[0, 1] = table[1, 0]                       # a page that sequence 1 still reads
    got, st = run(read)
    r = lambda page: slice(int(page) * 64, int(page) * 64 + 64)  # noqa: E731
    assert st == lib.DSA_ERR_BAD_INDEX and torch.equal(got[r(table[1, 0])], pool0[r(table[1, 0])])
    assert torch.equal(got[r(new_table[1, 0])], good[r(new_table[1, 0])])
    got, st = run(read, dst=torch.zeros_like(pool0).cuda())
    assert st == lib.DSA_OK                        # another array: its pages are free
    twice[1, 0] = new_table[0, 0]
    got, st = run(twice)
    assert st == lib.DSA_ERR_BAD_INDEX and torch.equal(got[r(new_table[0, 0])], pool0[r(new_table[0, 0])])
    off[0, 0], off[1, 0] = total, -1
    got, st = run(off)
    assert st == lib.DSA_ERR_BAD_INDEX and torch.equal(got[r(new_table[0, 1])][:36], good[r(new_table[0, 1])][:36])
    bad_keep = keep.clone()
    bad_keep[0, 3], bad_keep[1, 0] = 300, -1
    got, st = run(new_table, keep=bad_keep)
    assert st == lib.DSA_ERR_BAD_INDEX
    assert torch.equal(got[int(new_table[0, 0]) * 64 + 3], pool0[int(new_table[0, 0]) * 64 + 3])
    bad_len = lens.clone()
    bad_len[0] = 101
    got, st = run(new_table, lens=bad_len)
    assert st == lib.DSA_ERR_BAD_INDEX and torch.equal(got[r(new_table[0, 0])], pool0[r(new_table[0, 0])])
    assert run(new_table)[1] == lib.DSA_OK         # the same workspace, clean again


@pytest.mark.parametrize("inside", [True, False])
@pytest.mark.parametrize("row_bytes", [46508, 65528, 65532, 65536])
def test_compact_wide_rows(lib, row_bytes, inside):
    """Rows up to the largest, whole blocks of them and part of one."""
    ctx, budget = [70, 33, 5], 40
    table, new_table, total = _cache(ctx, 1)
    seqs = _seqs(lib, ctx, table, total)
    keep, lens = lib.dsa_evict_select(seqs.ctx_len, _masses(3, 70, "heavy").cuda(), budget)
    assert lens.tolist() == [40, 33, 5]
    src = torch.randint(0, 256, (total * 64, row_bytes), generator=torch.Generator("cuda").manual_seed(row_bytes),
                        dtype=torch.uint8, device="cuda")
    dst = src if inside else torch.full_like(src, 7)
    want = dst.clone()
    ws = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    for b, n in enumerate(lens.tolist()):
        to = torch.from_numpy(_rows(new_table[b], np.arange(n))).cuda()
        want[to] = src[torch.from_numpy(_rows(table[b], keep[b, :n].cpu().numpy().astype(np.int64))).cuda()]
    lib.dsa_evict_compact(seqs, keep, lens, torch.from_numpy(new_table).cuda(), [src if inside else (src, dst)], ws=ws)
    assert lib.dsa_check_error(ws) == lib.DSA_OK
    assert torch.equal(dst, want)


def test_default_workspace_tells_of_a_refused_page(lib):
    """The error flag of calls without a workspace is where the other operators have it,
    whatever the pools' sizes."""
    flag = lambda: lib.dsa_check_error(lib.workspace(0, "cuda", "evict_compact"))  # noqa: E731
    flag()                                         # what calls before this test have left
    for ctx in ([300, 200], [70], [30000, 5]):
        table, new_table, total = _cache(ctx, 1)
        seqs = _seqs(lib, ctx, table, total)
        keep, lens = lib.dsa_evict_select(seqs.ctx_len, _masses(len(ctx), max(ctx), "heavy").cuda(), 50)
        pool = torch.randn((total * 64, 8)).cuda()
        lib.dsa_evict_compact(seqs, keep, lens, torch.from_numpy(new_table).cuda(), [pool])
        assert flag() == lib.DSA_OK
        new_table[0, 0] = table[0, 0]
        lib.dsa_evict_compact(seqs, keep, lens, torch.from_numpy(new_table).cuda(), [pool])
        assert flag() == lib.DSA_ERR_BAD_INDEX and flag() == lib.DSA_OK
