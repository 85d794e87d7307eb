"""Plain float64 restatement of the operators around the path: rotary
positions, the MXFP4 index cache, and eviction by accumulated attention
weight.  Test infrastructure, like ``dsa_oracle``, whose sequences, bf16
decoding and MX block size it uses; it shares no code with the CUDA side."""
from __future__ import annotations

import math

import numpy as np

from . import dsa_oracle as O

# ----------------------------------------------------------------------------
# Rotary positions
# ----------------------------------------------------------------------------


def rope(x, positions, freqs, offset=0, interleaved=True, amplitude=1.0, transpose=False):
    """x [T, H, D]: each pair of the dims offset .. offset + 2 len(freqs) - 1 as
    a complex number times amplitude * exp(+-i position * freq)."""
    y = np.array(x, dtype=np.float64)
    n = len(freqs)
    # the phase in integers: double frequencies are exact ratios, and position
    # * frequency is reduced mod 2 pi with 60 digits' worth of integer pi
    ang = np.array([[_phase(int(p), f) for f in freqs] for p in positions]).reshape(len(positions), n)
    turn = amplitude * np.exp((-1j if transpose else 1j) * ang)[:, None, :]
    if interleaved:
        i0, i1 = offset + 2 * np.arange(n), offset + 2 * np.arange(n) + 1
    else:
        i0, i1 = offset + np.arange(n), offset + n + np.arange(n)
    z = (y[..., i0] + 1j * y[..., i1]) * turn
    y[..., i0], y[..., i1] = z.real, z.imag
    return y


_PI_DIGITS = 3141592653589793238462643383279502884197169399375105820974944  # pi * 10^60


def _phase(p: int, f: float) -> float:
    num, den = float(f).as_integer_ratio()
    scaled = p * num * 10 ** 60 // den                     # angle * 10^60, rounded down
    return (scaled % (2 * _PI_DIGITS)) / 10 ** 60


# ----------------------------------------------------------------------------
# MXFP4: E2M1 elements, one E8M0 scale per 32
# ----------------------------------------------------------------------------

E2M1_VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E2M1_EMAX = 2          # exponent of E2M1's top binade: 6 = 1.5 * 2^2
E8M0_NAN = 255


def mxfp4_quantize(x):
    """Real values [..., n] -> (packed codes [..., n/2], element 2i in the low
    four bits, sign in bit 3; E8M0 scale codes [..., n/32]).  e = floor(log2
    max|block|) - 2 clamped to [-127, 127] (0 for a zero block); element =
    the grid value nearest to x / 2^e, ties to the even code, at most 6.  A
    block with an infinity or NaN has scale 255 (NaN) and codes 0."""
    x = np.asarray(x, dtype=np.float64)
    blocks = x.reshape(*x.shape[:-1], -1, O.MX_BLOCK)
    codes = np.zeros(blocks.shape, dtype=np.uint8)
    scales = np.zeros(blocks.shape[:-1], dtype=np.uint8)
    for i in np.ndindex(*scales.shape):
        b = blocks[i]
        if not np.isfinite(b).all():
            scales[i] = E8M0_NAN
            continue
        amax = np.abs(b).max()
        e = 0 if amax == 0 else min(127, max(-127, math.frexp(amax)[1] - 1 - E2M1_EMAX))
        scales[i] = e + O.E8M0_BIAS
        y = np.minimum(np.abs(b) / math.ldexp(1.0, e), 6.0)
        d = np.abs(y[:, None] - E2M1_VALUES)               # [32, 8]
        near = d == d.min(axis=1, keepdims=True)           # one value, or the two of a tie
        c = np.where(near[:, 0::2].any(1), 2 * near[:, 0::2].argmax(1), 2 * near[:, 1::2].argmax(1) + 1)
        codes[i] = c + 8 * (np.signbit(b) & (c > 0))
    flat = codes.reshape(x.shape)
    return flat[..., 0::2] | (flat[..., 1::2] << 4), scales


def mxfp4_dequantize(packed, scales) -> np.ndarray:
    p = np.asarray(packed, dtype=np.uint8)
    c = np.stack([p & 15, p >> 4], axis=-1).reshape(*p.shape[:-1], -1)
    v = np.where(c & 8, -1.0, 1.0) * E2M1_VALUES[c & 7]
    v = v.reshape(*v.shape[:-1], -1, O.MX_BLOCK) * O.e8m0_decode(scales)[..., None]
    return v.reshape(*p.shape[:-1], -1)


def index_scores_mx4(seqs: O.Seqs, qI_bits, w, kI, kI_scale, tokens=None):
    """Indexer scores over an MXFP4 cache (kI packed codes [R, 64], kI_scale
    [R, 4]): the formula on the dequantised keys and the query quantised alike."""
    out = []
    for t in range(seqs.num_tokens) if tokens is None else tokens:
        b, pos = seqs.token_seq_pos(int(t))
        rows = seqs.rows(b, np.arange(pos + 1))
        k = mxfp4_dequantize(np.asarray(kI)[rows], np.asarray(kI_scale)[rows])
        q = mxfp4_dequantize(*mxfp4_quantize(O.bf16_to_f64(np.asarray(qI_bits)[int(t)])))
        out.append(np.asarray(w, np.float64)[int(t)] @ np.maximum(q @ k.T, 0.0))
    return out


# ----------------------------------------------------------------------------
# Eviction by accumulated attention weight
# ----------------------------------------------------------------------------


def attn_mass(seqs: O.Seqs, q_bits, kv_bits, idx, scale, lse, max_ctx) -> np.ndarray:
    """mass[b, s] = sum over the query tokens of b of the weight that their
    heads give position s on average: mean_h exp(scale q[t,h] . KV[s] - lse[t,h])."""
    mass = np.zeros((len(seqs.ctx_len), max_ctx))
    for t in range(seqs.num_tokens):
        b, _ = seqs.token_seq_pos(t)
        s = np.asarray(idx[t])
        s = s[s >= 0].astype(np.int64)
        kv = O.kv_rows(kv_bits, seqs.rows(b, s))
        logits = scale * (O.bf16_to_f64(q_bits[t]) @ kv.T)
        np.add.at(mass[b], s, np.exp(logits - np.asarray(lse[t], np.float64)[:, None]).mean(0))
    return mass


def evict_select(ctx_len, mass, budget: int, recent: int = 0, sink: int = 0):
    """Per sequence: the positions kept, ascending, -1 behind them, and how
    many.  All of them if ctx_len <= budget; else the first `sink`, the last
    `recent` and, of the others, those of the largest mass (compared in fp32,
    ties to the lower position)."""
    B = len(ctx_len)
    keep, lens = np.full((B, budget), -1, np.int32), np.zeros(B, np.int32)
    for b, n in enumerate(int(x) for x in ctx_len):
        forced = [s for s in range(n) if s < sink or s >= n - recent]
        rest = [s for s in range(n) if sink <= s < n - recent]
        m = np.asarray(mass[b]).astype(np.float32)
        rest.sort(key=lambda s: (-m[s], s))
        chosen = sorted(range(n) if n <= budget else forced + rest[:budget - len(forced)])
        keep[b, :len(chosen)], lens[b] = chosen, len(chosen)
    return keep, lens
