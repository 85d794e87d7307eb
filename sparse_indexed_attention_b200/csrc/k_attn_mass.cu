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
//   * eight loader warps resolve the slice's rows (index list -> page table ->
//     pool row) and copy them, 128 rows x 64 dims (16 KB) at a time, into a ring of
//     128-byte-swizzled operand slots, each with its own barriers: the query
//     (H x 1152 bytes) fills most of shared memory, and the ring keeps loads in
//     flight across blocks;
//   * one thread issues the MMAs, four per slot, into one of two accumulators;
//   * four warps read the other accumulator: p = 2^(c S - L_h), summed over h.
//     c = scale log2 e and L = lse log2 e are used as two fp32 terms each: one
//     would be off by 2^-24 of the logit, 1e-6 of p at logits of 16.
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
constexpr int kLoaders = 256;                // warps 4-11
constexpr int kLoaderBarrier = 1;
constexpr int kMmaWarp = 12;
constexpr int kThreads = 13 * 32;            // warps 0-3 sum, 4-11 load, 12 issues MMAs and owns TMEM
constexpr int kMaxSlots = 9;
constexpr int kTmemCols = 256;               // two accumulators of up to 128 columns
constexpr int kPerLoader = kMaxK / kLoaders;

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
  int q_atom, ring, rows, lse, bars, total;
  __host__ __device__ Layout(int H, int slots) {
    q_atom = H * 128;
    ring = kAtoms * q_atom;
    rows = ring + slots * kSlotBytes;
    lse = rows + kMaxK * 4;
    bars = lse + 128 * 8;
    total = bars + (2 * kMaxSlots + 8) * 8 + 16;
  }
};

template <bool kKv8>
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
  uint64_t* s_full = bars + 2 * kMaxSlots;     // [2]
  uint64_t* s_empty = s_full + 2;              // [2]
  uint64_t* q_full = s_empty + 2;
  uint64_t* ready = q_full + 1;                // rows and lse are in shared memory
  uint64_t* mma_drain = ready + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kMaxSlots + 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x / a.splits, sp = blockIdx.x % a.splits;
  const int kbeg = sp * a.ks, kend = min(a.K, kbeg + a.ks);
  if (threadIdx.x == 0) {
    for (int i = 0; i < a.slots; ++i) {
      mbar_init(&full[i], kLoaders);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 4);
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
  const int acc_cols = a.H < 32 ? 32 : a.H;

  if (threadIdx.x == kMmaWarp * 32 && nblk > 0) {
    mbar_arrive_expect_tx(q_full, (uint32_t)(kAtoms * L.q_atom));
    for (int i = 0; i < kAtoms; ++i) tma_load_2d(smem + i * L.q_atom, &tq, q_full, 64 * i, t * a.H);
  }
  if (warp >= 4 && warp < kMmaWarp && nblk > 0) {
    // ---------------------------------------------------------------- loaders
    const int li = threadIdx.x - 128;
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
    const int rsub = li >> 3, piece = li & 7;  // this thread's rows: rsub + 32 u, their 16-byte piece of each atom
    const uint32_t swz = (uint32_t)rsub * 128u + (((uint32_t)piece ^ ((uint32_t)rsub & 7u)) << 4);
    const uint32_t ring = smem_u32(smem + L.ring);
    // FP8 cache: a block's codes are loaded one block ahead of their conversion
    uint2 raw[4][kAtoms], scl[4];
    auto load_block = [&](int j) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int row = rows[j * kRows + rsub + 32 * u];
        const uint8_t* src = a.kv + (int64_t)(row < 0 ? 0 : row) * kDQK + 8 * piece;
#pragma unroll
        for (int i = 0; i < kAtoms; ++i) raw[u][i] = row >= 0 ? ld_nc_v2(src + 64 * i) : make_uint2(0u, 0u);
        scl[u] = row >= 0 ? ld_nc_v2(a.kv_scale + (int64_t)row * 8) : make_uint2(0x7F7F7F7Fu, 0x7Fu);
      }
    };
    if constexpr (kKv8) load_block(0);
    int slot = 0, phase = 0;
    for (int j = 0; j < nblk && ok; ++j) {
      int row[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) row[u] = rows[j * kRows + rsub + 32 * u];
#pragma unroll
      for (int i = 0; i < kAtoms; ++i) {
        ok = ok && !*abort_flag && mbar_wait(&empty[slot], phase ^ 1, a.err, a.wait_ns);
        if (ok) {
          if constexpr (kKv8) {
            uint8_t* dst = smem + L.ring + slot * kSlotBytes + swz;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int tile = i >> 1;
              const uint32_t byte = (tile < 4 ? (scl[u].x >> (8 * tile)) : scl[u].y) & 0xFFu;
              *reinterpret_cast<uint4*>(dst + u * 4096) = e4m3x8_to_bf16x8(raw[u][i], tile_scale(byte));
            }
            fence_proxy_async_smem();  // the MMAs read these stores through the async proxy
            mbar_arrive(&full[slot]);
          } else {
            const uint32_t dst = ring + slot * kSlotBytes + swz;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const bool live = row[u] >= 0;
              const uint8_t* src = a.kv + (live ? (int64_t)row[u] * (kDQK * 2) : 0) + 128 * i + 16 * piece;
              cp_async_16_zfill(dst + u * 4096, src, live ? 16u : 0u);
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
        if (ok && j + 1 < nblk) load_block(j + 1);
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
      int slot = 0, phase = 0;
      for (int j = 0; j < nblk && ok; ++j) {
        const int acc = j & 1;
        ok = !*abort_flag && mbar_wait(&s_empty[acc], ((j >> 1) & 1) ^ 1, a.err, a.wait_ns);
        tc_fence_after();
        for (int i = 0; i < kAtoms && ok; ++i) {
          ok = mbar_wait(&full[slot], phase, a.err, a.wait_ns);
          if (!ok) break;
          fence_proxy_async_smem();  // written by cp.async (generic proxy)
          tc_fence_after();
          const uint32_t ab = smem_u32(smem + L.ring + slot * kSlotBytes), bb = smem_u32(smem + i * L.q_atom);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ss<true>(tmem + acc * acc_cols, sw128_kmajor_desc(ab + kk * 32), sw128_kmajor_desc(bb + kk * 32), idesc,
                         (i | kk) != 0);
          mma_commit(&empty[slot]);
          if (++slot == a.slots) {
            slot = 0;
            phase ^= 1;
          }
        }
        if (ok) mma_commit(&s_full[acc]);
      }
      if (!ok) *abort_flag = 1;
      // drain, also after a failed wait: the query's copy has landed and no MMA
      // still reads shared memory or writes TMEM
      mbar_wait(q_full, 0, a.err, kDrainLimitNs);
      mma_commit(mma_drain);
      mbar_wait(mma_drain, 0, a.err, kDrainLimitNs);
    }
    __syncwarp();
  } else if (warp < 4 && nblk > 0) {
    // ---------------------------------------------------------------- sums
    const int r = threadIdx.x;
    const uint32_t t_lane = tmem + ((uint32_t)(warp * 32) << 16);
    const float inv_h = 1.f / (float)a.H;  // a power of two
    bool ok = __all_sync(0xffffffffu, mbar_wait(ready, 0, a.err, a.wait_ns));
    for (int j = 0; j < nblk && ok; ++j) {
      const int acc = j & 1, k = j * kRows + r;
      const bool live = rows[k] >= 0;
      const int s = live ? __ldg(a.idx + (int64_t)t * a.K + kbeg + k) : 0;
      ok = __all_sync(0xffffffffu, !*abort_flag && mbar_wait(&s_full[acc], (j >> 1) & 1, a.err, a.wait_ns));
      if (!ok) break;
      tc_fence_after();
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (int c = 0; c < a.H; c += 32) {
        uint32_t v[32];
        tmem_ld32(t_lane + acc * acc_cols + c, v);
        tmem_ld_wait_regs(v);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float2 lh = lse[c + i];
          const float x = __uint_as_float(v[i]);
          const float p = ex2_ftz(fmaf(x, a.c_hi, -lh.x) + fmaf(x, a.c_lo, -lh.y));
          if (c + i < a.H) sum[i & 3] += p;  // H = 16 fills half a chunk
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_empty[acc]);
      const float w = ((sum[0] + sum[1]) + (sum[2] + sum[3])) * inv_h;
      // a NaN (from a NaN or an lse that does not belong to these logits) adds nothing
      const float lim = w > 0.f ? fminf(w, 1.f) : 0.f;
      if (live && lim > 0.f)
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

template <bool kKv8>
cudaError_t launch(const CUtensorMap& tq, const MassArgs& a, int64_t ctas, cudaStream_t st) {
  static thread_local int attr_dev = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (attr_dev != dev) {
    cudaError_t e = cudaFuncSetAttribute(k_attn_mass<kKv8>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
    attr_dev = dev;
  }
  return launch_pdl("attn_mass", k_attn_mass<kKv8>, dim3((unsigned)ctas), dim3(kThreads),
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
  cudaError_t e = kv8_scale ? launch<true>(tq, a, ctas, st) : launch<false>(tq, a, ctas, st);
  if (e != cudaSuccess) return e;
  return counted(cudaGetLastError());
}

}  // namespace dsa
