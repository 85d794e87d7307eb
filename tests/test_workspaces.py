"""The workspaces of calls that are given none: one per stream, so that calls at the
same time do not write into each other's scratch."""
import threading

import numpy as np
import pytest
import torch

import sparse_indexed_attention_b200 as dsa


def test_one_buffer_per_device_and_key():
    mine = dsa.workspace(512, "cpu", "one_buffer")
    assert dsa.workspace(300, "cpu", "one_buffer") is mine and dsa.workspace(0, "cpu", "one_buffer") is mine
    assert dsa.workspace(512, "cpu", "another") is not mine


@pytest.mark.gpu
def test_streams_have_their_own():
    key = "streams_have_their_own"
    mine = dsa.workspace(512, "cuda", key)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert dsa.workspace(0, "cuda", key) is mine      # a look before the stream has one
        other = dsa.workspace(4096, "cuda", key)
        assert other.data_ptr() != mine.data_ptr()
        assert dsa.workspace(512, "cuda", key) is other and dsa.workspace(0, "cuda", key) is other
    assert dsa.workspace(512, "cuda", key) is mine and dsa.workspace(0, "cuda", key) is mine
    with torch.cuda.graph(torch.cuda.CUDAGraph()):        # the capturing stream has none: a large enough one
        assert dsa.workspace(2048, "cuda", key) is other
        torch.zeros(1, device="cuda")


class _Batch:
    """A batch's scores and its compaction inside a pool, without workspaces."""

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        ctx, budget = [1500 + 100 * seed, 700, 64], 300
        pages = [(n + 63) // 64 for n in ctx]
        spare = (budget + 63) // 64
        total = 100
        perm = torch.randperm(total, generator=g).int()
        table = torch.full((3, max(pages)), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(pages):
            table[b, :n] = perm[at:at + n]
            at += n
        self.new_table = perm[at:at + 3 * spare].view(3, spare).contiguous().cuda()
        # a table that names a page which is read: the compaction must leave that page alone
        self.bad_table = self.new_table.clone()
        self.bad_table[0, 0] = int(table[1, 0])
        self.seqs = dsa.Seqs.from_host(np.arange(4), np.array(ctx), table, total)
        R = total * 64
        self.kI = torch.randint(0, 256, (R, 64), generator=g, dtype=torch.uint8).cuda()
        self.sc = torch.randint(115, 130, (R, 4), generator=g, dtype=torch.uint8).cuda()
        self.qI, self.w = torch.randn((3, 64, 128), generator=g).bfloat16().cuda(), torch.randn((3, 64), generator=g).cuda()
        self.pool = torch.randint(0, 256, (R, 576), generator=g, dtype=torch.uint8).cuda()
        mass = torch.randint(0, 2 ** 40, (3, max(ctx)), generator=g).cuda()
        self.keep, self.lens = dsa.dsa_evict_select(self.seqs.ctx_len, mass, budget, recent=16, sink=4)

    def run(self, times=20):
        out = []
        for i in range(times):
            out.append(dsa.dsa_index_scores(self.seqs, self.qI, self.w, self.kI, self.sc))
            pool = self.pool.clone()
            dsa.dsa_evict_compact(self.seqs, self.keep, self.lens, self.bad_table if i % 2 else self.new_table, [pool])
            out.append(pool)
        return out


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["two streams", "two threads", "two threads on one stream"])
def test_two_at_once_without_workspaces(how):
    batches = [_Batch(s) for s in (1, 2)]
    want = [b.run(2) for b in batches]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in batches]
    if how == "two threads on one stream":
        streams[1] = streams[0]
    got, wrong = [[], []], []

    def work(i):
        try:
            with torch.cuda.stream(streams[i]):
                torch.cuda._sleep(2_000_000)              # the streams' work overlaps
                got[i] = batches[i].run(40)
        except BaseException as e:  # noqa: BLE001 (a thread's failure is the test's)
            wrong.append(e)
    if how == "two streams":
        for _ in range(20):
            for i, s in enumerate(streams):
                with torch.cuda.stream(s):
                    torch.cuda._sleep(50_000)
                    got[i] += batches[i].run(2)
    else:
        ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
        for t in ts:
            t.start()
        for t in ts:
            t.join()
    assert not wrong, wrong
    for s in streams[:1 if streams[0] is streams[1] else 2]:
        with torch.cuda.stream(s):
            assert dsa.dsa_check_error(dsa.workspace(0, "cuda", "index_scores")) == dsa.DSA_OK
            assert dsa.dsa_check_error(dsa.workspace(0, "cuda", "evict_compact")) == dsa.DSA_ERR_BAD_INDEX
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert len(b) == 80
        for i, x in enumerate(b):
            assert torch.equal(x, a[i % 4]), i


def test_a_larger_buffer_keeps_the_error_flag():
    small = dsa.workspace(512, "cpu", "keeps_the_flag")
    small[:8] = torch.tensor([2, 0, 0, 0, 9, 9, 9, 9], dtype=torch.uint8)
    large = dsa.workspace(4096, "cpu", "keeps_the_flag")
    assert large.numel() == 4096 and large[0] == 2 and not large[1:].any()


@pytest.mark.gpu
def test_an_error_outlives_a_larger_call():
    flag = lambda: dsa.dsa_check_error(dsa.workspace(0, "cuda", "topk"))  # noqa: E731
    with torch.cuda.stream(torch.cuda.Stream()):           # a stream without workspaces
        scores = torch.randn(2, 64, device="cuda")
        dsa.dsa_topk(scores, torch.tensor([65, 64], dtype=torch.int32, device="cuda"), 8)     # a row too long
        before = dsa.workspace(0, "cuda", "topk").numel()
        scores = torch.randn(2, 100_000, device="cuda")
        dsa.dsa_topk(scores, torch.full((2,), 100_000, dtype=torch.int32, device="cuda"), 8)
        assert dsa.workspace(0, "cuda", "topk").numel() > before
        assert flag() == dsa.DSA_ERR_BAD_INDEX and flag() == dsa.DSA_OK
