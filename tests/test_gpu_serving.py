"""The operators around the path used together, as a serving loop uses them:
rotate, quantise and append, score, select, attend, accumulate weight, evict,
and go on with the smaller cache; and the same calls captured in a CUDA graph."""
import numpy as np
import pytest
import torch

from dsa_workloads import bits16
from oracle import dsa_oracle as O
from oracle import serving_oracle as S

pytestmark = pytest.mark.gpu

H, K, SCALE = 32, 256, 576 ** -0.5


class Model:
    """Three sequences, an MXFP4 index cache and a bf16 latent cache, every page in one pool."""

    def __init__(self, lib, ctx=(400, 131, 640), budget=128, seed=0):
        self.lib, self.ctx, self.budget = lib, list(ctx), budget
        g = torch.Generator().manual_seed(seed)
        self.B, self.steps = len(ctx), 8
        pages = [(n + self.steps + 63) // 64 for n in ctx]
        spare = (budget + self.steps + 63) // 64
        self.num_pages = sum(pages) + self.B * spare
        perm = torch.randperm(self.num_pages, generator=g).int()
        self.table = torch.full((self.B, max(pages)), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.new_table = perm[at:].view(self.B, spare).contiguous()
        R = self.num_pages * 64
        self.kI = torch.zeros((R, 64), dtype=torch.uint8, device="cuda")
        self.kI_scale = torch.full((R, 4), 127, dtype=torch.uint8, device="cuda")
        self.kv = torch.zeros((R, 576), dtype=torch.bfloat16, device="cuda")
        self.mass = torch.zeros((self.B, max(ctx) + self.steps), dtype=torch.int64, device="cuda")
        self.rope = lib.RopeTable.build(64, scaling="yarn", factor=8.0)
        self.gen = g

    def inputs(self, T):
        r = lambda *s: torch.randn(s, generator=self.gen)  # noqa: E731
        return {"qI": r(T, 64, 128).bfloat16().cuda(), "k": r(T, 128).bfloat16().cuda(), "w": (r(T, 64) / 8).cuda(),
                "q": r(T, H, 576).bfloat16().cuda(), "kv": r(T, 576).bfloat16().cuda()}

    def seqs(self, q_len, ctx, table):
        starts = np.concatenate([[0], np.cumsum(q_len)])
        return self.lib.Seqs.from_host(starts, np.array(ctx), table, self.num_pages)

    def step(self, seqs, x, pos, rows, out=None, lse=None, idx=None, ws=None):
        """One call of every operator on a batch; x is rotated in place."""
        lib, (wa, wp, wm) = self.lib, ws or (None, None, None)
        lib.dsa_rope(x["q"], pos, self.rope, offset=512, out=x["q"])
        lib.dsa_rope(x["kv"], pos, self.rope, offset=512, out=x["kv"])
        lib.dsa_rope(x["qI"], pos, self.rope, out=x["qI"])
        lib.dsa_rope(x["k"], pos, self.rope, out=x["k"])
        lib.dsa_append_index_keys_mx4(seqs, x["k"], self.kI, self.kI_scale, ws=wa)
        self.kv.index_copy_(0, rows, x["kv"])
        out, lse = lib.dsa_index_topk_attn(seqs, x["qI"], x["w"], self.kI, self.kI_scale, x["q"], self.kv, K, SCALE,
                                           out=out, lse=lse, idx_out=idx, out_dtype=torch.float32, ws=wp)
        lib.dsa_attn_mass(seqs, x["q"], self.kv, idx, lse, SCALE, self.mass, ws=wm)
        return out, lse


def _rows(table, b, s):
    return table[b, s // 64].long() * 64 + s % 64


def test_prefill_evict_decode(lib):
    m = Model(lib)
    q_len = m.ctx
    T = sum(q_len)
    seqs = m.seqs(q_len, m.ctx, m.table)
    pos = torch.cat([torch.arange(n) for n in q_len])
    seq = torch.arange(m.B).repeat_interleave(torch.tensor(q_len))
    x = m.inputs(T)
    raw = {k: v.clone() for k, v in x.items()}
    idx = torch.empty((T, K), dtype=torch.int32, device="cuda")
    out, lse = m.step(seqs, x, pos.cuda(), _rows(m.table, seq, pos).cuda(), idx=idx)
    # each part against the oracle on sampled tokens
    t = [0, 1, 399, 400, 530, 531, T - 1]
    f = lib.RopeTable.frequencies(64, scaling="yarn", factor=8.0)
    ref = S.rope(raw["q"][t].double().cpu().numpy(), pos[t].tolist(), f, 512, True, m.rope.amplitude)
    assert np.abs(x["q"][t].double().cpu().numpy() - ref).max() <= 2.0 ** -8 * np.abs(ref).max()
    oseqs = O.Seqs(np.array(m.ctx), np.concatenate([[0], np.cumsum(q_len)]), m.table.numpy(), 64)
    scores = S.index_scores_mx4(oseqs, bits16(x["qI"].cpu()), x["w"].cpu().numpy(), m.kI.cpu().numpy(),
                                m.kI_scale.cpu().numpy(), tokens=t)
    kv = bits16(m.kv.cpu())
    got = idx.cpu().numpy()
    for tok, row in zip(t, scores):
        want = set(O.topk_select(row, K)) - {-1}
        have = set(got[tok]) - {-1}
        tau = np.sort(row)[::-1][min(K, len(row)) - 1]
        assert len(have) == len(want) and all(abs(row[s] - tau) <= 1e-3 * abs(tau) for s in want ^ have)
    ref_out, ref_lse = O.sparse_mla(oseqs, bits16(x["q"].cpu()), kv, got, SCALE, tokens=t)
    assert np.abs(out[t].cpu().numpy() - ref_out).max() <= 1e-2 * np.sqrt((ref_out ** 2).mean())
    unit = 2.0 ** -lib.DSA_MASS_FRACTION_BITS
    assert np.abs(m.mass.sum(1).cpu().numpy() * unit - np.array(q_len)).max() <= 2e-3 * max(q_len)

    # cut every cache back to the budget, in the same pool
    keep, keep_len = lib.dsa_evict_select(seqs.ctx_len, m.mass, m.budget, recent=16, sink=4)
    assert keep_len.tolist() == [min(n, m.budget) for n in m.ctx]
    new_mass = torch.zeros((m.B, m.budget + m.steps), dtype=torch.int64, device="cuda")
    ws = torch.zeros(lib.dsa_workspace_size(lib.DSA_OP_EVICT_COMPACT, seqs), dtype=torch.uint8, device="cuda")
    lib.dsa_evict_compact(seqs, keep, keep_len, m.new_table.cuda(), [m.kI, m.kI_scale, m.kv], mass=m.mass,
                          new_mass=new_mass, ws=ws)
    assert lib.dsa_check_error(ws) == lib.DSA_OK
    kept = keep_len.tolist()
    for b in range(m.B):
        s = keep[b, :kept[b]].long().cpu()
        a, z = _rows(m.table, b, s).cuda(), _rows(m.new_table, torch.tensor(b), torch.arange(kept[b])).cuda()
        for pool in (m.kI, m.kI_scale, m.kv):
            assert torch.equal(pool[a], pool[z])
        assert torch.equal(new_mass[b, :kept[b]], m.mass[b, s.cuda()])

    # the next tokens: the small cache attends as the large one does over the kept positions
    m.mass = new_mass
    x = m.inputs(m.B)
    ctx = [n + 1 for n in kept]
    small = m.seqs([1] * m.B, ctx, m.new_table)
    at = torch.tensor(kept)
    idx = torch.empty((m.B, K), dtype=torch.int32, device="cuda")
    out, lse = m.step(small, x, torch.tensor(m.ctx).cuda(), _rows(m.new_table, torch.arange(m.B), at).cuda(), idx=idx)
    big_rows = _rows(m.table, torch.arange(m.B), torch.tensor(m.ctx)).cuda()
    m.kv.index_copy_(0, big_rows, x["kv"])
    old = torch.full((m.B, K), -1, dtype=torch.int32)
    for b in range(m.B):
        s = idx[b][idx[b] >= 0].long().cpu()
        full = torch.cat([keep[b, :kept[b]].cpu(), torch.tensor([m.ctx[b]], dtype=torch.int32)])
        old[b, :len(s)] = full[s]
        assert len(s) == min(K, ctx[b])
    big = m.seqs([1] * m.B, [n + 1 for n in m.ctx], m.table)
    out2, lse2 = lib.dsa_sparse_mla_fwd(big, x["q"], m.kv, old.cuda(), SCALE, out_dtype=torch.float32)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_decode_step_in_a_graph(lib):
    """Every operator captured once and replayed: the same bits as eager calls,
    also after the inputs change, with workspaces of the graph's own."""
    m = Model(lib)
    q_len = m.ctx
    pos = torch.cat([torch.arange(n) for n in q_len])
    seq = torch.arange(m.B).repeat_interleave(torch.tensor(q_len))
    idx0 = torch.empty((sum(q_len), K), dtype=torch.int32, device="cuda")
    m.step(m.seqs(q_len, m.ctx, m.table), m.inputs(sum(q_len)), pos.cuda(), _rows(m.table, seq, pos).cuda(), idx=idx0)
    seqs = m.seqs([1] * m.B, [n + 1 for n in m.ctx], m.table)
    at = torch.tensor(m.ctx)
    rows, pos = _rows(m.table, torch.arange(m.B), at).cuda(), at.cuda()
    need = lib.dsa_workspace_size(lib.DSA_OP_INDEX_TOPK_ATTN, seqs, K, H)
    spaces = [tuple(torch.zeros(n, dtype=torch.uint8, device="cuda") for n in (256, need, 256)) for _ in range(2)]
    fresh = m.inputs(m.B)
    x = {k: v.clone() for k, v in fresh.items()}
    out = torch.zeros((m.B, H, 512), device="cuda")
    lse = torch.zeros((m.B, H), device="cuda")
    idx = torch.zeros((m.B, K), dtype=torch.int32, device="cuda")
    keep = torch.zeros((m.B, 64), dtype=torch.int32, device="cuda")
    kept = torch.zeros(m.B, dtype=torch.int32, device="cuda")
    base = m.mass.clone()

    def step(ws):
        m.step(seqs, x, pos, rows, out=out, lse=lse, idx=idx, ws=ws)
        lib.dsa_evict_select(seqs.ctx_len, m.mass, 64, recent=8, sink=1, keep=keep, keep_len=kept)

    def state():
        return [t.clone() for t in (out, lse, idx, m.mass, keep, kept, m.kI, m.kI_scale, m.kv)]

    def reset(inputs):
        m.mass.copy_(base)
        for k, v in inputs.items():
            x[k].copy_(v)
        torch.cuda.synchronize()
    lib.dsa_evict_select(seqs.ctx_len, m.mass, 64, recent=8, sink=1)     # its cached workspace exists before the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(spaces[0])
    for inputs in (fresh, m.inputs(m.B)):
        reset(inputs)
        step(spaces[1])
        want = state()
        reset(inputs)
        for t in (out, lse, idx, keep, kept):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, state()):
            assert torch.equal(a, b)
    for ws in spaces[0]:
        assert lib.dsa_check_error(ws) == lib.DSA_OK


def test_two_streams_at_once(lib):
    """Two batches on two streams, each with its own workspaces."""
    models = [Model(lib, seed=s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in models]
    want, work = [], []
    for m in models:
        q_len = m.ctx
        pos = torch.cat([torch.arange(n) for n in q_len])
        seq = torch.arange(m.B).repeat_interleave(torch.tensor(q_len))
        seqs, T = m.seqs(q_len, m.ctx, m.table), sum(q_len)
        need = lib.dsa_workspace_size(lib.DSA_OP_INDEX_TOPK_ATTN, seqs, K, H)
        ws = tuple(torch.zeros(n, dtype=torch.uint8, device="cuda") for n in (256, need, 256))
        idx = torch.empty((T, K), dtype=torch.int32, device="cuda")
        x = m.inputs(T)
        work.append((m, seqs, x, {k: v.clone() for k, v in x.items()}, pos.cuda(), _rows(m.table, seq, pos).cuda(), idx, ws))
    for m, seqs, x, raw, pos, rows, idx, ws in work:
        out, lse = m.step(seqs, x, pos, rows, idx=idx, ws=ws)
        want.append([t.clone() for t in (out, lse, idx, m.mass)])
        m.mass.zero_()
        for k in x:
            x[k].copy_(raw[k])
        idx.zero_()
    torch.cuda.synchronize()
    got = []
    for stream, (m, seqs, x, raw, pos, rows, idx, ws) in zip(streams, work):
        with torch.cuda.stream(stream):
            out, lse = m.step(seqs, x, pos, rows, idx=idx, ws=ws)
            got.append((out, lse, idx, m.mass))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_a_workspace_made_during_capture_belongs_to_the_graph(lib):
    key = "made_during_capture"
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        inside = lib.workspace(512, "cuda", key)
    outside = lib.workspace(512, "cuda", key)
    assert outside.data_ptr() != inside.data_ptr() and not outside.any()
    assert lib.workspace(512, "cuda", key) is outside
