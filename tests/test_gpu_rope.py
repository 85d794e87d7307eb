"""Rotary positions on the GPU against the float64 oracle.

Tolerance of one output, in fp32 before its rounding: the phase is rounded to
2^-26 turn (1e-7 rad), sinpif / cospif are good to 1 ulp (6e-8), the amplitude
and the two products add 6e-8 each: below 4e-7 of (|a| + |b|) * amplitude.
Storing it in type t adds half a step, eps(t) / 2 of the value."""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as S

pytestmark = pytest.mark.gpu

CASES = [  # T, H, D, rot, offset, interleaved, scaling, factor
    (1, 1, 2, 2, 0, True, "none", 1.0),
    (1, 128, 64, 64, 0, True, "yarn", 32.0),
    (5, 3, 576, 64, 512, True, "none", 1.0),
    (130, 1, 64, 64, 0, False, "ntk", 8.0),
    (7, 64, 128, 64, 64, False, "linear", 4.0),
    (9, 2, 33, 18, 5, True, "none", 1.0),        # odd offset and size: single elements
    (9, 2, 33, 18, 5, False, "none", 1.0),
    (3, 2, 40, 12, 8, False, "none", 1.0),       # half of 6: no 16-byte vectors in the half layout
    (2, 1, 1024, 1024, 0, False, "yarn", 4.0),
]


def _table(lib, c):
    return lib.RopeTable.build(c[3], 10000.0, interleaved=c[5], scaling=c[6], factor=c[7])


def _freqs(lib, c):
    return lib.RopeTable.frequencies(c[3], 10000.0, scaling=c[6], factor=c[7])


def _check(lib, got, x, pos, c, tab, transpose=False):
    ref = S.rope(x.double().cpu().numpy(), pos.tolist(), _freqs(lib, c), c[4], c[5], tab.amplitude, transpose)
    xa = np.abs(x.double().cpu().numpy())
    part = xa.copy()                              # |a| + |b| of each value's pair
    n = c[3] // 2
    i0 = c[4] + (2 * np.arange(n) if c[5] else np.arange(n))
    i1 = i0 + (1 if c[5] else n)
    part[..., i0] = part[..., i1] = xa[..., i0] + xa[..., i1]
    tol = 4e-7 * part * abs(tab.amplitude) + (torch.finfo(x.dtype).eps / 2) * np.abs(ref) * 1.01 + 1e-30
    if x.dtype == torch.float16:
        tol += 2.0 ** -25                         # half a step among fp16's subnormals
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= tol).all(), float((err / tol).max())
    rest = np.ones(c[2], bool)
    rest[c[4]:c[4] + c[3]] = False
    assert np.array_equal(got.cpu().float().numpy()[..., rest], x.cpu().float().numpy()[..., rest])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("c", CASES, ids=str)
def test_rope(lib, c, dtype):
    g = torch.Generator().manual_seed(sum(c[:5]))
    x = torch.randn(c[0], c[1], c[2], generator=g).to(dtype).cuda()
    pos = torch.randint(-5, 2 ** 20, (c[0],), generator=g)
    pos[0] = 2 ** 31 - 1                          # far out
    tab = _table(lib, c)
    for transpose in (False, True):
        for p in (pos, pos.int()):
            got = lib.dsa_rope(x, p.cuda(), tab, offset=c[4], transpose=transpose)
            _check(lib, got, x, pos, c, tab, transpose)
    kept = x.clone()
    assert lib.dsa_rope(x, pos.cuda(), tab, offset=c[4], out=x) is x
    _check(lib, x, kept, pos, c, tab)


def test_views(lib):
    """Slices of wider rows, heads outside tokens, and rows without heads."""
    c = (6, 4, 64, 64, 0, True, "none", 1.0)
    tab = _table(lib, c)
    pos = torch.arange(100, 106)
    up = torch.randn(6, 4, 192).bfloat16().cuda()
    q = torch.zeros(6, 4, 576).bfloat16().cuda()
    lib.dsa_rope(up[..., 128:], pos.cuda(), tab, out=q[..., 512:])
    _check(lib, q[..., 512:], up[..., 128:], pos, c, tab)
    assert not q[..., :512].any()
    heads_first = torch.randn(4, 6, 64).cuda().transpose(0, 1)
    out = torch.zeros(4, 6, 64).cuda().transpose(0, 1)
    lib.dsa_rope(heads_first, pos.cuda(), tab, out=out)
    _check(lib, out, heads_first, pos, c, tab)
    odd = torch.randn(6 * 4 * 65 + 1).cuda()[1:].view(6, 4, 65)[..., :64]     # off the 16-byte grid
    _check(lib, lib.dsa_rope(odd, pos.cuda(), tab), odd, pos, c, tab)
    wide = torch.randn(6, 576).half().cuda()      # one latent row per token
    got = lib.dsa_rope(wide, pos.cuda(), tab, offset=512)
    _check(lib, got[:, None], wide[:, None], pos, (6, 1, 576, 64, 512, True, "none", 1.0), tab)
    same = torch.randn(1, 4, 64).cuda().expand(6, 4, 64)
    _check(lib, lib.dsa_rope(same, pos.cuda(), tab), same, pos, c, tab)
    assert lib.dsa_rope(up[:0], pos[:0].cuda(), tab).shape == (0, 4, 192)


def test_non_finite_values_stay_in_their_pair(lib):
    tab = lib.RopeTable.build(64)
    x = torch.randn(2, 1, 64)
    x[0, 0, 10], x[1, 0, 21] = float("nan"), float("inf")
    y = lib.dsa_rope(x.cuda(), torch.tensor([3, 4]).cuda(), tab).cpu()
    bad = torch.zeros(2, 64, dtype=torch.bool)
    bad[0, 10:12] = bad[1, 20:22] = True
    assert torch.equal(~torch.isfinite(y[:, 0]), bad)


def test_large_and_captured(lib):
    """Many blocks with a ragged end, on another stream and in a CUDA graph."""
    tab = lib.RopeTable.build(64, interleaved=False)
    x = torch.randn(5003, 33, 64).bfloat16().cuda()
    pos = torch.arange(5003).cuda()
    want = lib.dsa_rope(x, pos, tab)
    f = lib.RopeTable.frequencies(64)
    rows = [0, 1, 2500, 5001, 5002]
    ref = S.rope(x[rows].double().cpu().numpy(), rows, f, 0, False)
    assert np.abs(want[rows].double().cpu().numpy() - ref).max() <= 2.0 ** -8 * np.abs(ref).max()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = lib.dsa_rope(x, pos, tab)
    side.synchronize()
    assert torch.equal(other, want)
    out = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.dsa_rope(x, pos, tab, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and lib.dsa_launches_in_last_call() == 1


@pytest.mark.parametrize("T,H,D,rot,offset", [(4743, 67, 128, 64, 32), (1801, 37, 97, 66, 5)])
@pytest.mark.parametrize("interleaved", [True, False])
def test_the_largest_calls(lib, T, H, D, rot, offset, interleaved):
    """Ragged calls of more than 16 x 148 x 6 x 256 units, whose blocks take eight units per
    thread: the bits of calls on a few tokens each, and the oracle's values on some rows."""
    c = (T, H, D, rot, offset, interleaved, "linear", 4.0)
    units = (rot // 16 if D % 8 == 0 and not interleaved else rot // 8 if D % 8 == 0 else rot // 2) \
        + (D - rot) // (8 if D % 8 == 0 else 1)
    assert units * T * H >= 16 * 148 * 6 * 256
    g = torch.Generator("cuda").manual_seed(T + D)
    x = torch.randn((T, H, D), generator=g, device="cuda").bfloat16()
    pos = torch.randint(-5, 2 ** 20, (T,), generator=g, device="cuda")
    tab = _table(lib, c)
    got = lib.dsa_rope(x, pos, tab, offset=offset)
    for t in range(0, T, 97):
        assert torch.equal(got[t:t + 97], lib.dsa_rope(x[t:t + 97], pos[t:t + 97], tab, offset=offset))
    some = [0, 1, 2, T // 2, T - 3, T - 2, T - 1]
    _check(lib, got[some], x[some], pos[some].cpu(), c, tab)
    kept = x.clone()
    lib.dsa_rope(x, pos, tab, offset=offset, out=x)
    assert torch.equal(x, got)
    rest = torch.ones(D, dtype=torch.bool, device="cuda")
    rest[offset:offset + rot] = False
    assert torch.equal(got[..., rest], kept[..., rest])
