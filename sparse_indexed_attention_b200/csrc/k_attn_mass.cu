// Accumulated attention weight of cached positions, what eviction ranks by:
//
//   mass[b, s] += (1 / H) sum_h exp(scale q[t,h] . KV[s] - lse[t,h])
//
// for every query token t of sequence b and every selected position s.  The
// probabilities are recomputed from the logits and the attention's lse; the
// value product is not needed, so this is the first half of sparse MLA.
//
// Layout.  A CTA takes one token and a slice of its index list, in blocks of
// 128 rows.  S^T = KV Q^T puts a cached row in each TMEM lane and the heads in
// the columns (M = 128 rows, N = H heads, K = 576), so the sum over heads stays
// inside one thread -- the transposed product of the attention kernel would
// need a reduction over lanes -- and a row is gathered once for all heads.
//   * four loader warps resolve the slice's rows (index list -> page table ->
//     pool row) and copy them, 128 rows x 64 dims (16 KB) at a time, into a ring of
//     128-byte-swizzled operand slots, each with its own barriers: the query
//     (H x 1152 bytes) fills most of shared memory, and the ring keeps loads in
//     flight across blocks;
//   * one thread issues the MMAs, four per slot, each slot's 64 dims into an
//     accumulator of its own (a ring of four);
//   * eight warps, two per lane quarter with half of the heads each, add the
//     nine partial logits in registers and take p = 2^(c S - L_h), summed over h.
// Precision.  The tensor core's fp32 additions truncate: one chain of 36
// accumulations per logit was off by 3e-6 of the mass (an fp32 product rounded to
// nearest: 6.5e-7), all one way.  Chains of four, added with rounding, are not.
// c = scale log2 e and L = lse log2 e are used as two fp32 terms each: one would
// be off by 2^-24 of the logit, 1e-6 of p at logits of 16.
//
// The sum over tokens is held in 64-bit fixed point (units of 2^-40 of one
// token's whole attention, 8.4 million tokens before it overflows): integer
// additions commute, so the result does not depend on the order of the atomics.
//
// What bounds it: a block's 147 KB of rows against 36 MMAs.  MEASURED
#include "kv8.cuh"
#include "sm100.cuh"
#include "tensor_map.cuh"

namespace dsa {

namespace {

using namespace sm100;

constexpr int kRows = 128;                   // rows per block (the MMA's M)
constexpr int kAtoms = kDQK / 64;            // 9 slices of 64 dims
constexpr int kSlotBytes = kRows * 128;
constexpr int kSumWarps = 8;                 // warps 0-7
constexpr int kLoaders = 128;                // warps 8-11
constexpr int kLoaderBarrier = 1, kSumBarrier = 2;
constexpr int kMmaWarp = 12;
constexpr int kThreads = 13 * 32;            // warp 12 issues MMAs and owns TMEM
constexpr int kMaxSlots = 8;
constexpr int kAccs = 4;                     // accumulators of up to 128 columns
constexpr int kTmemCols = 512;
constexpr int kPerLoader = kMaxK / kLoaders;
constexpr int kRowsPerLoader = kRows * 8 / kLoaders;  // a thread's 16-byte pieces of a slot
constexpr int kAhead = 3;                    // FP8 cache: slots whose codes are loaded ahead (a divisor of kAtoms)

struct MassArgs {
  SeqsDev s;
  const uint8_t* kv;         // bf16 rows, or E4M3 codes
  const uint8_t* kv_scale;   // FP8 cache: tile-scale bytes [rows, 8]
  const int32_t* idx;
  const float* lse;
  unsigned long long* mass;
  int64_t ld;
  int K, H, ks, splits, slots;
  float c_hi, c_lo;          // scale * log2(e) as two terms
  uint32_t* err;
  uint64_t wait_ns;
};

// Shared memory from a 1024-aligned base: query, ring, rows, lse, barriers.
struct Layout {
  int q_atom, ring, rows, lse, half, bars, total;
  __host__ __device__ Layout(int H, int slots) {
    q_atom = H * 128;
    ring = kAtoms * q_atom;
    rows = ring + slots * kSlotBytes;
    lse = rows + kMaxK * 4;
    half = lse + 128 * 8;                  // [2] the second heads' sums of a block's rows
    bars = half + 2 * kRows * 4;
    total = bars + (2 * kMaxSlots + 2 * kAccs + 4) * 8 + 16;
  }
};

// Two warpgroups meet at the block's sums: the second arrives with its half, the first waits.
__device__ __forceinline__ void sums_arrive() {
  asm volatile("barrier.cta.arrive %0, %1;" ::"n"(kSumBarrier), "n"(kSumWarps * 32) : "memory");
}
__device__ __forceinline__ void sums_wait() {
  asm volatile("barrier.cta.sync %0, %1;" ::"n"(kSumBarrier), "n"(kSumWarps * 32) : "memory");
}

// CH: chunks of 32 heads that a summing thread holds (two for H = 128).
template <bool kKv8, int CH>
__global__ void __launch_bounds__(kThreads, 1)
k_attn_mass(const __grid_constant__ CUtensorMap tq, const MassArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const Layout L(a.H, a.slots);
  int32_t* rows = reinterpret_cast<int32_t*>(smem + L.rows);       // pool row of each slot of the slice, -1 = none
  float2* lse = reinterpret_cast<float2*>(smem + L.lse);           // lse * log2(e) per head, two terms
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L.bars);
  uint64_t* full = bars;                       // [slots]
  uint64_t* empty = bars + kMaxSlots;          // [slots]
  uint64_t* s_full = bars + 2 * kMaxSlots;     // [kAccs]
  uint64_t* s_empty = s_full + kAccs;          // [kAccs]
  uint64_t* q_full = s_empty + kAccs;
  uint64_t* ready = q_full + 1;                // rows and lse are in shared memory
  uint64_t* mma_drain = ready + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x / a.splits, sp = blockIdx.x % a.splits;
  const int kbeg = sp * a.ks, kend = min(a.K, kbeg + a.ks);
  if (threadIdx.x == 0) {
    for (int i = 0; i < a.slots; ++i) {
      mbar_init(&full[i], kLoaders);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < kAccs; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], kSumWarps);
    }
    mbar_init(q_full, 1);
    mbar_init(ready, 1);
    mbar_init(mma_drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();
  const TokenPlace at = locate_token(a.s, t);
  if (at.pos < 0 && threadIdx.x == 0) raise_error(a.err, kErrBadIndex);
  const int nblk = at.pos >= 0 && kend > kbeg ? (kend - kbeg + kRows - 1) / kRows : 0;
  const int acc_cols = a.H < 64 ? 64 : a.H;

  if (threadIdx.x == kMmaWarp * 32 && nblk > 0) {
    mbar_arrive_expect_tx(q_full, (uint32_t)(kAtoms * L.q_atom));
    for (int i = 0; i < kAtoms; ++i) tma_load_2d(smem + i * L.q_atom, &tq, q_full, 64 * i, t * a.H);
  }
  if (warp >= kSumWarps && warp < kMmaWarp && nblk > 0) {
    // ---------------------------------------------------------------- loaders
    const int li = threadIdx.x - kSumWarps * 32;
    const int n = kend - kbeg;
    {
      int sidx[kPerLoader], page[kPerLoader];
      const int32_t* list = a.idx + (int64_t)t * a.K + kbeg;
      const int32_t* table = a.s.page_table + (int64_t)at.seq * a.s.max_pages;
#pragma unroll
      for (int i = 0; i < kPerLoader; ++i) {
        const int k = li + i * kLoaders;
        sidx[i] = k < n ? __ldg(list + k) : -1;
      }
#pragma unroll
      for (int i = 0; i < kPerLoader; ++i) {
        page[i] = -1;
        if (sidx[i] >= 0 && sidx[i] <= at.pos) page[i] = __ldg(table + (sidx[i] >> 6));
      }
#pragma unroll
      for (int i = 0; i < kPerLoader; ++i) {
        const int k = li + i * kLoaders;
        int row = -1;
        if (page[i] >= 0 && page[i] < a.s.num_phys_pages)
          row = page[i] * kPage + (sidx[i] & (kPage - 1));
        else if (sidx[i] != -1)
          raise_error(a.err, kErrBadIndex);
        if (k < nblk * kRows) rows[k] = row;
      }
      if (li < a.H) {
        const float v = __ldg(a.lse + (int64_t)t * a.H + li);
        constexpr float kLog2e = 1.4426950408889634f, kLog2eLo = 1.9259629911266175e-8f;
        const float hi = v * kLog2e;
        // an infinite lse keeps its sign; its low term would be NaN
        const float lo = isinf(v) ? 0.f : fmaf(v, kLog2eLo, fmaf(v, kLog2e, -hi));
        lse[li] = make_float2(hi, lo);
      }
    }
    bool ok = !bar_red_or(kLoaderBarrier, kLoaders, false);
    if (li == 0) mbar_arrive(ready);
    const int rsub = li >> 3, piece = li & 7;  // this thread's rows: rsub + 16 u, their 16-byte piece of each atom
    const uint32_t swz = (uint32_t)rsub * 128u + (((uint32_t)piece ^ ((uint32_t)rsub & 7u)) << 4);
    const uint32_t ring = smem_u32(smem + L.ring);
    // FP8 cache: codes pass through registers, loaded kAhead slots ahead of their conversion
    constexpr int kRaw = kKv8 ? kRowsPerLoader : 1;
    uint2 raw[kAhead][kRaw], scl[kRaw], scl_next[kRaw];
    auto load_codes = [&](int j, int i, uint2 (&to)[kRaw]) {
#pragma unroll
      for (int u = 0; u < kRaw; ++u) {
        const int row = rows[j * kRows + rsub + 16 * u];
        to[u] = row >= 0 ? ld_nc_v2(a.kv + (int64_t)row * kDQK + 64 * i + 8 * piece) : make_uint2(0u, 0u);
      }
    };
    auto load_scales = [&](int j, uint2 (&to)[kRaw]) {
#pragma unroll
      for (int u = 0; u < kRaw; ++u) {
        const int row = rows[j * kRows + rsub + 16 * u];
        to[u] = row >= 0 ? ld_nc_v2(a.kv_scale + (int64_t)row * 8) : make_uint2(0x7F7F7F7Fu, 0x7Fu);
      }
    };
    if constexpr (kKv8) {
      load_scales(0, scl);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) load_codes(0, i, raw[i]);
    }
    int slot = 0, phase = 0;
    for (int j = 0; j < nblk && ok; ++j) {
      int row[kRowsPerLoader];
#pragma unroll
      for (int u = 0; u < kRowsPerLoader; ++u) row[u] = rows[j * kRows + rsub + 16 * u];
#pragma unroll
      for (int i = 0; i < kAtoms; ++i) {
        ok = ok && !*abort_flag && mbar_wait(&empty[slot], phase ^ 1, a.err, a.wait_ns);
        if (ok) {
          if constexpr (kKv8) {
            uint8_t* dst = smem + L.ring + slot * kSlotBytes + swz;
            const int tile = i >> 1;
#pragma unroll
            for (int u = 0; u < kRaw; ++u) {
              const uint32_t byte = (tile < 4 ? (scl[u].x >> (8 * tile)) : scl[u].y) & 0xFFu;
              *reinterpret_cast<uint4*>(dst + u * 2048) = e4m3x8_to_bf16x8(raw[i % kAhead][u], tile_scale(byte));
            }
            fence_proxy_async_smem();  // the MMAs read these stores through the async proxy
            mbar_arrive(&full[slot]);
            if (i + kAhead < kAtoms) {
              load_codes(j, i + kAhead, raw[i % kAhead]);
            } else if (j + 1 < nblk) {
              if (i + kAhead == kAtoms) load_scales(j + 1, scl_next);
              load_codes(j + 1, i + kAhead - kAtoms, raw[i % kAhead]);
            }
          } else {
            const uint32_t dst = ring + slot * kSlotBytes + swz;
#pragma unroll
            for (int u = 0; u < kRowsPerLoader; ++u) {
              const bool live = row[u] >= 0;
              const uint8_t* src = a.kv + (live ? (int64_t)row[u] * (kDQK * 2) : 0) + 128 * i + 16 * piece;
              cp_async_16_zfill(dst + u * 2048, src, live ? 16u : 0u);
            }
            cp_async_mbar_arrive(&full[slot]);  // counts once this thread's copies land
          }
        }
        if (++slot == a.slots) {
          slot = 0;
          phase ^= 1;
        }
      }
      if constexpr (kKv8) {
#pragma unroll
        for (int u = 0; u < kRaw; ++u) scl[u] = scl_next[u];
      }
    }
    if (!ok) *abort_flag = 1;
    cp_async_wait_all();  // nothing this thread copies is still in flight at exit
    __syncwarp();
  } else if (warp == kMmaWarp && nblk > 0) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      const uint32_t idesc = make_idesc(true, kRows, a.H);
      bool ok = mbar_wait(q_full, 0, a.err, a.wait_ns);
      int slot = 0, phase = 0, acc = 0, aphase = 0;
      for (int j = 0; j < nblk && ok; ++j) {
        for (int i = 0; i < kAtoms; ++i) {
          ok = !*abort_flag && mbar_wait(&full[slot], phase, a.err, a.wait_ns) &&
               mbar_wait(&s_empty[acc], aphase ^ 1, a.err, a.wait_ns);
          if (!ok) break;
          fence_proxy_async_smem();  // the rows were written by cp.async (generic proxy)
          tc_fence_after();
          const uint32_t ab = smem_u32(smem + L.ring + slot * kSlotBytes), bb = smem_u32(smem + i * L.q_atom);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ss<true>(tmem + acc * acc_cols, sw128_kmajor_desc(ab + kk * 32), sw128_kmajor_desc(bb + kk * 32), idesc,
                         kk != 0);
          mma_commit(&empty[slot]);
          mma_commit(&s_full[acc]);
          if (++slot == a.slots) {
            slot = 0;
            phase ^= 1;
          }
          if (++acc == kAccs) {
            acc = 0;
            aphase ^= 1;
          }
        }
      }
      if (!ok) *abort_flag = 1;
      // drain, also after a failed wait: the query's copy has landed and no MMA
      // still reads shared memory or writes TMEM
      mbar_wait(q_full, 0, a.err, kDrainLimitNs);
      mma_commit(mma_drain);
      mbar_wait(mma_drain, 0, a.err, kDrainLimitNs);
    }
    __syncwarp();
  } else if (warp < kSumWarps && nblk > 0) {
    // ---------------------------------------------------------------- sums
    const int wg = warp >> 2, r = threadIdx.x & 127;  // half of the heads, row of the block
    const int heads = a.H >> 1, h0 = wg * heads;
    const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16) + h0;
    const float inv_h = 1.f / (float)a.H;  // a power of two
    float* other = reinterpret_cast<float*>(smem + L.half);
    bool ok = __all_sync(0xffffffffu, mbar_wait(ready, 0, a.err, a.wait_ns));
    int acc = 0, aphase = 0;
    for (int j = 0; j < nblk; ++j) {
      const int k = j * kRows + r;
      const bool live = ok && rows[k] >= 0;
      const int s = live ? __ldg(a.idx + (int64_t)t * a.K + kbeg + k) : 0;
      float x[CH][32];
#pragma unroll
      for (int i = 0; i < kAtoms; ++i) {
        ok = ok && __all_sync(0xffffffffu, !*abort_flag && mbar_wait(&s_full[acc], aphase, a.err, a.wait_ns));
        if (ok) {
          tc_fence_after();
          uint32_t v[CH][32];  // fewer than 32 heads: the other columns are read and left out below
#pragma unroll
          for (int c = 0; c < CH; ++c) tmem_ld32(t_lane + acc * acc_cols + 32 * c, v[c]);
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            tmem_ld_wait_regs(v[c]);
#pragma unroll
            for (int e = 0; e < 32; ++e) x[c][e] = i == 0 ? __uint_as_float(v[c][e]) : x[c][e] + __uint_as_float(v[c][e]);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_empty[acc]);
        }
        if (++acc == kAccs) {
          acc = 0;
          aphase ^= 1;
        }
      }
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float2 lh = lse[h0 + 32 * c + e];
          const float p = ex2_ftz(fmaf(x[c][e], a.c_hi, -lh.x) + fmaf(x[c][e], a.c_lo, -lh.y));
          if (32 * c + e < heads) sum[e & 3] += p;
        }
      float w = (sum[0] + sum[1]) + (sum[2] + sum[3]);
      // the second half's sum goes through shared memory, two buffers: the ring of
      // accumulators lets no warp run a whole block ahead of another
      if (wg == 1) {
        other[(j & 1) * kRows + r] = w;
        sums_arrive();
        continue;
      }
      sums_wait();
      w = (w + other[(j & 1) * kRows + r]) * inv_h;
      // a NaN (from a NaN or an lse that does not belong to these logits) adds nothing
      const float lim = w > 0.f ? fminf(w, 1.f) : 0.f;
      if (ok && live && lim > 0.f)
        atomicAdd(a.mass + (int64_t)at.seq * a.ld + s, (unsigned long long)__float2ll_rn(lim * 0x1p40f));
    }
    if (!ok) *abort_flag = 1;
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Slices of a token's list: CTAs run one per SM, each with a start of about
// two and a half blocks' time (barriers, TMEM, row ids, query), so the cost of a
// split is its waves times (start + blocks).
int mass_splits(int T, int K) {
  const int blocks = (K + kRows - 1) / kRows;
  int best = 1;
  double least = 1e30;
  for (int sp = 1; sp <= blocks; ++sp) {
    const int per = (blocks + sp - 1) / sp;
    const int64_t ctas = (int64_t)T * ((blocks + per - 1) / per);
    const double cost = (double)((ctas + 147) / 148) * (2.5 + per);
    if (cost < least - 1e-9) {
      least = cost;
      best = sp;
    }
  }
  return best;
}

template <bool kKv8, int CH>
cudaError_t launch(const CUtensorMap& tq, const MassArgs& a, int64_t ctas, cudaStream_t st) {
  static thread_local int attr_dev = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (attr_dev != dev) {
    cudaError_t e = cudaFuncSetAttribute(k_attn_mass<kKv8, CH>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
    attr_dev = dev;
  }
  return launch_pdl("attn_mass", k_attn_mass<kKv8, CH>, dim3((unsigned)ctas), dim3(kThreads),
                    (size_t)(Layout(a.H, a.slots).total + 1024), st, tq, a);
}

}  // namespace

cudaError_t launch_attn_mass(const SeqsDev& s, const __nv_bfloat16* q, const void* kv, const uint8_t* kv8_scale,
                             const int32_t* idx, int K, int H, float scale, const float* lse, int64_t* mass,
                             int64_t ld, uint32_t* err, cudaStream_t st) {
  CUtensorMap tq;
  if (!make_bf16_rows_map(&tq, q, kDQK, (uint64_t)s.num_tokens * H, H)) return cudaErrorInvalidValue;
  const int blocks = (K + kRows - 1) / kRows;
  const int per = (blocks + mass_splits(s.num_tokens, K) - 1) / mass_splits(s.num_tokens, K);
  const int splits = (blocks + per - 1) / per;
  const double c = (double)scale * 1.4426950408889634;
  const float c_hi = (float)c;
  MassArgs a{s,  static_cast<const uint8_t*>(kv), kv8_scale, idx, lse, reinterpret_cast<unsigned long long*>(mass),
             ld, K, H, per * kRows, splits, H == 128 ? 4 : kMaxSlots, c_hi, (float)(c - c_hi), err, wait_limit_ns()};
  const int64_t ctas = (int64_t)s.num_tokens * splits;
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  cudaError_t e = H == 128 ? (kv8_scale ? launch<true, 2>(tq, a, ctas, st) : launch<false, 2>(tq, a, ctas, st))
                           : (kv8_scale ? launch<true, 1>(tq, a, ctas, st) : launch<false, 1>(tq, a, ctas, st));
  if (e != cudaSuccess) return e;
  return counted(cudaGetLastError());
}

}  // namespace dsa
