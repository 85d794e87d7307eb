"""Host paths of the operators around the path, without a GPU: each call runs its
checks and its dispatch and then fails at its first CUDA call (DSA_ERR_CUDA).
The buffers are host memory, so the test never runs where a GPU is present."""
import pytest
import torch

import sparse_indexed_attention_b200 as dsa
from tests.test_host_paths import _aligned

pytestmark = [pytest.mark.timeout(60),
              pytest.mark.skipif(torch.cuda.is_available(), reason="host buffers must not reach a GPU launch")]


@pytest.fixture
def host_binding(monkeypatch):
    monkeypatch.setattr(dsa, "_cuda_device", lambda t, name: t.device)
    monkeypatch.setattr(dsa, "_stream", lambda dev: None)
    monkeypatch.setattr(dsa, "workspace", lambda n, dev, key=None: _aligned(torch.zeros(max(n, 256), dtype=torch.uint8)))


@pytest.mark.parametrize("T,heads,kv_fp8", [(1, 16, False), (3, 128, False), (3, 128, True), (400, 64, True)])
def test_entry_points_return_without_a_gpu(host_binding, T, heads, kv_fp8):
    z = lambda *s, dt=torch.float32: _aligned(torch.zeros(s, dtype=dt))  # noqa: E731
    u8, bf, i32, i64 = torch.uint8, torch.bfloat16, torch.int32, torch.int64
    R, ctx = 16 * 64, 500
    starts = _aligned(torch.tensor([0, T], dtype=i32))
    seqs = dsa.Seqs(starts, _aligned(torch.tensor([ctx], dtype=i32)), z(1, 8, dt=i32), 16, ctx, T)
    kv = z(R, 576, dt=u8 if kv_fp8 else bf)
    kv_scale = z(R, 8, dt=u8) if kv_fp8 else None
    kI, kI_scale = z(R, 64, dt=u8), z(R, 4, dt=u8)
    mass, keep, kept = z(1, 512, dt=i64), z(1, 64, dt=i32), z(1, dt=i32)
    table = dsa.RopeTable.build(64, device="cpu")
    calls = [
        lambda: dsa.dsa_rope(z(T, heads, 576, dt=bf), z(T, dt=i64), table, offset=512),
        lambda: dsa.dsa_rope(z(T, 577), z(T, dt=i32), dsa.RopeTable.build(64, interleaved=False, device="cpu"), offset=1),
        lambda: dsa.dsa_quantize_index_query_mx4(z(T, 64, 128, dt=bf), z(T, 64, 64, dt=u8), z(T, 64, 4, dt=u8)),
        lambda: dsa.dsa_append_index_keys_mx4(seqs, z(T, 128, dt=bf), kI, kI_scale),
        lambda: dsa.dsa_dequantize_mx4(kI, kI_scale, out=z(R, 128, dt=bf)),
        lambda: dsa.dsa_index_scores(seqs, z(T, 64, 128, dt=bf), z(T, 64), kI, kI_scale, scores=z(T, 512)),
        lambda: dsa.dsa_index_topk_attn(seqs, z(T, 64, 128, dt=bf), z(T, 64), kI, kI_scale, z(T, heads, 576, dt=bf), kv,
                                        128, 0.04, out=z(T, heads, 512, dt=bf), kv_scale=kv_scale, want_lse=False),
        lambda: dsa.dsa_attn_mass(seqs, z(T, heads, 576, dt=bf), kv, z(T, 300, dt=i32), z(T, heads), 0.04, mass,
                                  kv_scale=kv_scale),
        lambda: dsa.dsa_evict_select(seqs.ctx_len, mass, 64, keep=keep, keep_len=kept),
        lambda: dsa.dsa_evict_select(seqs.ctx_len, z(1, 400000, dt=i64), 64, keep=keep, keep_len=kept),
        lambda: dsa.dsa_evict_compact(seqs, keep, kept, z(1, 1, dt=i32), [kI, kI_scale], mass=mass,
                                      new_mass=z(1, 64, dt=i64)),
    ]
    for call in calls:
        with pytest.raises(dsa.DsaError, match="DSA_ERR_CUDA"):
            call()


def test_default_workspaces_have_the_documented_keys(monkeypatch):
    """workspace(0, device, key) finds the buffer of a call that was given none."""
    used = []

    def workspace(n, dev, key=None):
        used.append(key)
        return _aligned(torch.zeros(max(n, 256), dtype=torch.uint8))
    monkeypatch.setattr(dsa, "_cuda_device", lambda t, name: t.device)
    documented = dsa.workspace.__doc__
    monkeypatch.setattr(dsa, "workspace", workspace)
    z = lambda *s, dt=torch.float32: _aligned(torch.zeros(s, dtype=dt))  # noqa: E731
    u8, bf, i32, i64 = torch.uint8, torch.bfloat16, torch.int32, torch.int64
    seqs = dsa.Seqs(_aligned(torch.tensor([0, 1], dtype=i32)), _aligned(torch.tensor([100], dtype=i32)),
                    z(1, 2, dt=i32), 8, 100, 1)
    R = 8 * 64
    kI, kI_scale, kv, mass, keep = z(R, 64, dt=u8), z(R, 4, dt=u8), z(R, 576, dt=bf), z(1, 128, dt=i64), z(1, 64, dt=i32)
    q, idx, lse = z(1, 16, 576, dt=bf), z(1, 64, dt=i32), z(1, 16)
    calls = {
        "append_index_keys": lambda: dsa.dsa_append_index_keys_mx4(seqs, z(1, 128, dt=bf), kI, kI_scale),
        "index_scores": lambda: dsa.dsa_index_scores(seqs, z(1, 64, 128, dt=bf), z(1, 64), kI, kI_scale, scores=z(1, 128)),
        "topk": lambda: dsa.dsa_topk(z(1, 128), z(1, dt=i32), 64, idx=idx),
        "sparse_mla": lambda: dsa.dsa_sparse_mla_fwd(seqs, q, kv, idx, 0.04, out=z(1, 16, 512, dt=bf), lse=lse),
        "index_topk_attn": lambda: dsa.dsa_index_topk_attn(seqs, z(1, 64, 128, dt=bf), z(1, 64), kI, kI_scale, q, kv, 64,
                                                           0.04, out=z(1, 16, 512, dt=bf), lse=lse),
        "attn_mass": lambda: dsa.dsa_attn_mass(seqs, q, kv, idx, lse, 0.04, mass),
        "evict_select": lambda: dsa.dsa_evict_select(seqs.ctx_len, mass, 64, keep=keep, keep_len=z(1, dt=i32)),
        "evict_compact": lambda: dsa.dsa_evict_compact(seqs, keep, z(1, dt=i32), z(1, 1, dt=i32), [kI, (kv, z(R, 576, dt=bf))]),
    }
    for key, call in calls.items():
        used.clear()
        with pytest.raises(dsa.DsaError, match="DSA_ERR_CUDA"):
            call()
        assert used == [key] and f'"{key}"' in documented
