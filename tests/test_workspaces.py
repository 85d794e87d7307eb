"""The workspaces of calls that are given none: one per thread and stream, so that
calls at the same time do not write into each other's scratch."""
import threading

import numpy as np
import pytest
import torch

import sparse_indexed_attention_b200 as dsa


def _in_thread(fn):
    got = []
    t = threading.Thread(target=lambda: got.append(fn()))
    t.start()
    t.join()
    return got[0]


def test_threads_have_their_own():
    key = "threads_have_their_own"
    mine = dsa.workspace(512, "cpu", key)
    assert dsa.workspace(300, "cpu", key) is mine and dsa.workspace(0, "cpu", key) is mine
    other = _in_thread(lambda: dsa.workspace(512, "cpu", key))
    assert other.data_ptr() != mine.data_ptr() and not other.any()
    assert dsa.workspace(512, "cpu", key) is mine


def test_a_look_finds_the_newest_buffer():
    key = "found_by_a_look"
    other = _in_thread(lambda: dsa.workspace(512, "cpu", key))
    assert dsa.workspace(0, "cpu", key) is other          # nothing of this thread's yet
    mine = dsa.workspace(512, "cpu", key)
    assert mine is not other and dsa.workspace(0, "cpu", key) is mine


@pytest.mark.gpu
def test_streams_have_their_own():
    key = "streams_have_their_own"
    mine = dsa.workspace(512, "cuda", key)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert dsa.workspace(0, "cuda", key) is mine      # a look before the stream has one
        other = dsa.workspace(512, "cuda", key)
        assert other.data_ptr() != mine.data_ptr()
        assert dsa.workspace(512, "cuda", key) is other and dsa.workspace(0, "cuda", key) is other
    assert dsa.workspace(512, "cuda", key) is mine and dsa.workspace(0, "cuda", key) is mine


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
@pytest.mark.parametrize("threads", [False, True])
def test_two_at_once_without_workspaces(threads):
    batches = [_Batch(s) for s in (1, 2)]
    want = [b.run(2) for b in batches]
    torch.cuda.synchronize()
    got, wrong = [None, None], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                torch.cuda._sleep(2_000_000)              # the streams' work overlaps
                got[i] = batches[i].run()
                torch.cuda.current_stream().synchronize()
                assert dsa.dsa_check_error(dsa.workspace(0, "cuda", "index_scores")) == dsa.DSA_OK
                assert dsa.dsa_check_error(dsa.workspace(0, "cuda", "evict_compact")) == dsa.DSA_ERR_BAD_INDEX
        except BaseException as e:  # noqa: BLE001 (a thread's failure is the test's)
            wrong.append(e)
    if threads:
        ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
        for t in ts:
            t.start()
        for t in ts:
            t.join()
    else:
        streams = [torch.cuda.Stream() for _ in batches]
        got = [[], []]
        for _ in range(10):
            for i, s in enumerate(streams):
                with torch.cuda.stream(s):
                    torch.cuda._sleep(50_000)
                    got[i] += batches[i].run(2)
    torch.cuda.synchronize()
    assert not wrong, wrong
    for a, b in zip(want, got):
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
