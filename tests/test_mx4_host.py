"""Host checks of the MXFP4 index cache, without a GPU."""
import ctypes

import pytest
import torch

import sparse_indexed_attention_b200 as dsa

P = ctypes.c_void_p
GOOD = P(0x10000)


def _seqs(T=4, B=1):
    return dsa.DsaSeqsC(B, T, 64, 2, 8, 100, 0x10000, 0x10000, 0x10000)


def test_c_entry_points_refuse_before_launch():
    lib = dsa.raw()
    s = ctypes.byref(_seqs())
    BAD, WS = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_WORKSPACE
    assert lib.dsa_quantize_index_query_mx4(GOOD, 0, GOOD, GOOD, None) == BAD
    assert lib.dsa_quantize_index_query_mx4(GOOD, 4, GOOD, P(0x10002), None) == BAD
    assert lib.dsa_dequantize_mx4(GOOD, GOOD, 0, GOOD, None) == BAD
    assert lib.dsa_dequantize_mx4(GOOD, GOOD, 1 << 31, GOOD, None) == dsa.DSA_ERR_UNSUPPORTED
    assert lib.dsa_append_index_keys_mx4(s, GOOD, GOOD, None, GOOD, 256, None) == BAD
    assert lib.dsa_append_index_keys_mx4(s, GOOD, P(0x10040), GOOD, GOOD, 256, None) == BAD
    assert lib.dsa_append_index_keys_mx4(s, GOOD, GOOD, GOOD, GOOD, 255, None) == WS
    assert lib.dsa_index_scores(s, GOOD, GOOD, GOOD, None, dsa.DSA_KI_MXFP4, GOOD, 128, GOOD, 1 << 20, None) == BAD
    assert lib.dsa_workspace_size(dsa.DSA_OP_APPEND_INDEX_KEYS, s, 1, 16) == 256


def test_format_follows_the_row_size(monkeypatch):
    monkeypatch.setattr(dsa, "_cuda_device", lambda t, name: t.device)
    seqs = dsa.Seqs(torch.tensor([0, 1], dtype=torch.int32), torch.tensor([5], dtype=torch.int32),
                    torch.zeros(1, 1, dtype=torch.int32), 1, 5, 1)
    qI, w = torch.zeros(1, 64, 128, dtype=torch.bfloat16), torch.zeros(1, 64)
    sc = torch.full((64, 4), 127, dtype=torch.uint8)
    k4, k8 = torch.zeros(64, 64, dtype=torch.uint8), torch.zeros(64, 128, dtype=torch.uint8)
    assert dsa._ki_dtype(sc, k4) == dsa.DSA_KI_MXFP4 and dsa._ki_dtype(sc, k8) == dsa.DSA_KI_MXFP8
    dsa._need_index_inputs(seqs, qI, w, k4, sc)
    with pytest.raises(ValueError, match="at least 64"):
        dsa._need_index_inputs(seqs, qI, w, k4[:63], sc)
    with pytest.raises(TypeError, match="dtype"):
        dsa._need_index_inputs(seqs, qI, w, k4.view(torch.float8_e4m3fn), sc)
    with pytest.raises(ValueError, match="shape"):
        dsa._need_index_inputs(seqs, qI, w, k4, torch.ones(64))   # packed codes need E8M0 scales
    k = torch.zeros(1, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="shape"):
        dsa.dsa_append_index_keys_mx4(seqs, k, k8, sc)
    with pytest.raises(TypeError, match="dtype"):
        dsa.dsa_append_index_keys_mx4(seqs, k.float(), k4, sc)
    with pytest.raises(ValueError, match="shape"):
        dsa.dsa_append_index_keys_mx4(seqs, k.expand(2, 128), k4, sc)
    with pytest.raises(ValueError, match="shape"):
        dsa.dsa_dequantize_mx4(k4, sc[:63])
    with pytest.raises(ValueError, match="contiguous"):
        dsa.dsa_dequantize_mx4(torch.zeros(64, 128, dtype=torch.uint8)[:, :64], sc)
    with pytest.raises(ValueError, match="expected"):
        dsa.dsa_dequantize_mx4(k8, sc)


def test_workload_rows_are_mxfp4_encodings():
    import numpy as np

    from dsa_workloads import CONFIGS, make_workload, mx4_rows
    from oracle import serving_oracle as S
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((50, 128)) * np.exp2(rng.integers(-9, 9, (50, 1)))).astype(np.float32)
    x[0] = 0.0
    x[1, :8] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    x[1, 8:32] = 0.0
    codes, scales = mx4_rows(torch.from_numpy(x))
    ref_codes, ref_scales = S.mxfp4_quantize(x)
    assert np.array_equal(codes.numpy(), ref_codes) and np.array_equal(scales.numpy(), ref_scales)
    wl = make_workload(CONFIGS["decode_b64_8k_32k"].scaled(batch=2, ctx=(300, 700), ki_mx4=True, planted=8))
    assert wl.kI.shape == (wl.num_phys_pages * 64, 64) and wl.kI_scale.shape == (wl.num_phys_pages * 64, 4)


def test_bench_names_the_format():
    import bench
    from dsa_workloads import CONFIGS
    spec = CONFIGS["decode_b8_128k"].scaled(ki_mx4=True)
    assert (bench.index_cache(spec), bench.index_row_bytes(spec)) == ("mxfp4", 68)


def test_stream_of_a_device_without_an_index(monkeypatch):
    """\"cuda\" means the current device, as everywhere in torch."""
    seen = []
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: seen.append(i) or 0, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    dsa._stream(torch.device("cuda"))
    dsa._stream(torch.device("cuda", 1))
    assert seen == [3, 1]
