"""Zigzag context parallelism over an MXFP4 index cache: two gloo ranks on CPU with the
oracle standing in for the GPU call, and 2 and 4 ranks one after the other on
one GPU.  Either must equal the single call exactly."""
import os
import sys

import numpy as np
import pytest
import torch
import torch.multiprocessing as mp

from sparse_indexed_attention_b200.cp import PAGE, ZigzagPlan, cp_prefill
from tests.test_cp import ROOT, _free_port, _shard


def _workload(ctx=512, **kw):
    from dsa_workloads import CONFIGS, make_workload
    return make_workload(CONFIGS["long_prefill_32k"].scaled(name=f"cp_mx4_{ctx}", ctx=(ctx, ctx), ki_mx4=True, **kw))


SMALL = dict(heads=16, topk=64)


def _attend(seqs, qI, w, kI, kI_scale, q, kv, K, scale):
    from dsa_workloads import bits16
    from oracle import dsa_oracle as O
    from oracle import serving_oracle as S
    s = O.Seqs(seqs.ctx_len.numpy().astype(np.int64), seqs.q_seq_start.numpy().astype(np.int64),
               seqs.page_table.numpy(), PAGE)
    idx = O.topk_rows(S.index_scores_mx4(s, bits16(qI), w.numpy(), kI.numpy(), kI_scale.numpy()), K)
    out, lse = O.sparse_mla(s, bits16(q), bits16(kv), idx, scale)
    return torch.from_numpy(out), torch.from_numpy(lse)


def _rank_main(rank, world, port, q):
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port), WORLD_SIZE=str(world), RANK=str(rank))
    sys.path.insert(0, ROOT)
    import torch.distributed as dist
    dist.init_process_group("gloo", rank=rank, world_size=world)
    try:
        wl = _workload(**SMALL)
        plan = ZigzagPlan.make(wl.T, world)
        qI, w, qq, kI, ks, kv, _ = _shard(wl, plan, rank)
        out, lse = cp_prefill(plan, None, qI, w, qq, kI, ks, kv, wl.spec.topk, wl.scale, attend=_attend)
        if rank == 0:
            q.put((out.numpy(), lse.numpy()))
    finally:
        dist.destroy_process_group()


@pytest.mark.timeout(600)
def test_two_gloo_ranks_equal_one():
    import queue
    import time

    from sparse_indexed_attention_b200 import Seqs
    ctx = mp.get_context("spawn")
    q = ctx.Queue()
    port = _free_port()
    procs = [ctx.Process(target=_rank_main, args=(r, 2, port, q)) for r in range(2)]
    for p in procs:
        p.start()
    got, deadline = None, time.time() + 500
    while got is None and time.time() < deadline:
        try:
            got = q.get(timeout=5)
        except queue.Empty:
            if any(p.exitcode not in (None, 0) for p in procs):
                break
    for p in procs:
        p.join(timeout=120)
    assert got is not None and all(p.exitcode == 0 for p in procs), [p.exitcode for p in procs]
    wl = _workload(**SMALL)
    assert wl.kI.shape[1] == 64 and wl.kI_scale.shape[1] == 4
    seqs = Seqs.from_host(wl.q_seq_start, wl.ctx_len, wl.page_table, wl.num_phys_pages, device="cpu")
    out, lse = _attend(seqs, wl.qI, wl.w, wl.kI, wl.kI_scale, wl.q, wl.kv, wl.spec.topk, wl.scale)
    assert np.array_equal(got[0], out.numpy()) and np.array_equal(got[1], lse.numpy())


@pytest.mark.gpu
@pytest.mark.parametrize("ranks", [2, 4])
def test_ranks_on_one_gpu_equal_one_call(lib, ranks):
    from dsa_workloads import to_device
    wl = _workload(2048, topk=512)
    d, K = to_device(wl), wl.spec.topk
    want = lib.dsa_index_topk_attn(d.seqs, d.qI, d.w, d.kI, d.kI_scale, d.q, d.kv, K, wl.scale, out_dtype=torch.float32)
    plan = ZigzagPlan.make(wl.T, ranks)
    shards = [[None if x is None else x.contiguous().cuda() for x in _shard(wl, plan, r)] for r in range(ranks)]
    pools = [torch.cat([s[i] for s in shards]) for i in (3, 4, 5)]
    got = []
    for r in range(ranks):
        qs, cl, pt = plan.rank_batch(r)
        seqs = lib.Seqs.from_host(qs, cl, pt, wl.T // PAGE, device="cuda")
        qI, w, q = shards[r][:3]
        got.append(lib.dsa_index_topk_attn(seqs, qI, w, pools[0], pools[1], q, pools[2], K, wl.scale,
                                           out_dtype=torch.float32))
    assert lib.dsa_check_error(lib.workspace(0, "cuda", "index_topk_attn")) == lib.DSA_OK
    for i, x in enumerate(want):
        assert torch.equal(plan.restore(torch.stack([g[i] for g in got])), x)
