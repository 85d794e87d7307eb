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
//     pool row) and copy them, 128 rows x 128 dims (a tile, 32 KB; the last of a
//     row's five is half of one) at a time, into a ring of 128-byte-swizzled operand
//     slots, each with its own barriers: the query (H x 1152 bytes) fills most of
//     shared memory, and the ring keeps loads in flight across blocks;
//   * two warps, taking tiles in turn, issue the MMAs, eight per tile, each
//     tile into an accumulator of its own (a ring of four): the waits, fence, issue and
//     commits are one serial chain per tile, and two of them overlap;
//   * eight warps, two per lane quarter with half of the heads each, add the
//     five partial logits in registers and take p = 2^(c S - L_h), summed over h.
// FP8 cache.  The tensor core multiplies its E4M3 codes as they are.  The tiles'
// scales, a power of two per row and tile, multiply the partial logits in the thread
// that owns the row.  The query becomes two E4M3 terms, q 2^s = t1 + 2^-5 t2 with the
// head's largest value in [2^7, 2^8): a bf16 has eight significant bits and each term
// holds four, so their sum is exact down to 2^-14 of that value and off by 2^-22 of it
// at most below.  They are 2 H columns of one product of twice the rate.
// (Converting the codes instead, to bf16 or fp16 for one product, took 2.7 and 1.6
// times as long: a tile then crosses shared memory four times.)
// Precision.  The tensor core's fp32 additions truncate: one chain of 36
// accumulations per logit was off by 3e-6 of the mass (an fp32 product rounded to
// nearest: 6.5e-7), all one way.  Chains of eight, added with rounding, are not.
// c = scale log2 e and L = lse log2 e are used as two fp32 terms each: one would
// be off by 2^-24 of the logit, 1e-6 of p at logits of 16.
//
// The sum over tokens is held in 64-bit fixed point (units of 2^-40 of one
// token's whole attention, 8.4 million tokens before it overflows): integer
// additions commute, so the result does not depend on the order of the atomics.
//
// What bounds it (warm, one B200): 400 tokens of 2048 of 2300 rows take 139 us with 128 heads
// (869 TFLOP/s, 53 % of the measured bf16 rate: MMAs of a tile against its issue, and
// three waves of CTAs for 2.7) and 96 us with 64 (the gather: 10 TB/s out of L2); over
// the FP8 cache 64 heads take 115 us and 128 heads 199 (the sums: two terms per head).  A
// decode step of 8 tokens takes 8 to 9 us (FP8 cache: 10 with 64 heads, 16 with 128): one
// block per CTA, the chain of its steps.
#include "kv8.cuh"
#include "sm100.cuh"
#include "tensor_map.cuh"

namespace dsa {

namespace {

using namespace sm100;

constexpr int kRows = 128;                   // rows per block (the MMA's M)
constexpr int kAtoms = kDQK / 64;            // 9 slices of 64 dims
constexpr int kAtomBytes = kRows * 128;
constexpr int kTiles = 5;                    // of a row: two atoms each, the last one
constexpr int kSumWarps = 8;                 // warps 0-7
constexpr int kIssuers = 2;                  // warps 8-9, an elected lane of each; warp 8 owns TMEM
constexpr int kLoaderBarrier = 1, kSumBarrier = 2;
constexpr int kMmaWarp = kSumWarps;
constexpr int kLoadWarp = kMmaWarp + kIssuers;
constexpr int kMaxSlots = 8;
constexpr int kMaxAccs = 4;
constexpr int kTmemCols = 512;

struct MassArgs {
  SeqsDev s;
  const __nv_bfloat16* q;
  const uint8_t* kv;         // bf16 rows, or E4M3 codes
  const uint8_t* kv_scale;   // FP8 cache: tile-scale bytes [rows, 8]
  const int32_t* idx;
  const float* lse;
  unsigned long long* mass;
  int64_t ld;
  int K, H, ks, splits;
  float c_hi, c_lo;          // scale * log2(e) as two terms
  uint32_t* err;
  uint64_t wait_ns;
};

// Shared memory from a 1024-aligned base: query, ring, rows, heads, barriers.
struct Layout {
  int ring, rows, head, bars, total;
  __host__ __device__ Layout(int H, int ring_bytes, int ks) {
    ring = kAtoms * H * 128;
    rows = ring + ring_bytes;
    head = rows + ks * 4;                  // and 32 entries more: chunks of heads are read whole
    bars = head + H * 16 + 512;
    total = bars + (2 * kMaxSlots + 2 * kMaxAccs + 5) * 8 + 16;
  }
};

__device__ __forceinline__ void tmem_ld(uint32_t at, uint32_t (&v)[32]) { tmem_ld32(at, v); }
__device__ __forceinline__ void tmem_ld(uint32_t at, uint32_t (&v)[16]) { tmem_ld16(at, v); }

// A barrier of the summing warps.
__device__ __forceinline__ void sums_sync() {
  asm volatile("barrier.cta.sync %0, %1;" ::"n"(kSumBarrier), "n"(kSumWarps * 32) : "memory");
}

// FP8 cache: the token's query as two E4M3 terms in shared memory, by the summing
// warps.  Tile i of the operand holds 2 H rows (the heads' first terms, then their
// second ones) of 128 dims in the 128-byte swizzle, the last tile 64 dims in the
// 64-byte swizzle.  256 / H neighbouring threads share a head; its factor becomes
// scale log2(e) / 2^s.  (Two passes over the query, the second from L2: 128 heads
// would not fit in registers.)
__device__ __forceinline__ void query_to_e4m3(const __nv_bfloat16* q, uint8_t* dst, int H, float c_hi, float c_lo,
                                              float4* head) {
  const int per = kSumWarps * 32 / H;            // threads per head: 2, 4, 8 or 16
  const int h = threadIdx.x / per, sub = threadIdx.x % per;
  constexpr int kChunks = kDQK / 8;              // 16-byte pieces of a head
  const uint4* src = reinterpret_cast<const uint4*>(q + (int64_t)h * kDQK);
  uint32_t m = 0;
#pragma unroll 18
  for (int k = sub; k < kChunks; k += per) {
    const uint4 v = __ldg(src + k);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
  }
  for (int o = 1; o < per; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  // largest value to [2^7, 2^8); a head with an infinity or NaN, which the terms
  // would lose, gets a factor of NaN
  const int s = min(126, m == 0u || m >= 0x7F80u ? 0 : 134 - (int)(m >> 7));
  const float up = __uint_as_float((uint32_t)(127 + s) << 23), down = __uint_as_float((uint32_t)(127 - s) << 23);
#pragma unroll 9
  for (int k = sub; k < kChunks; k += per) {
    const uint4 v = __ldg(src + k);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t t1[2] = {0u, 0u}, t2[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = make_float2(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xFFFF0000u) * up);
      const __nv_fp8x2_storage_t a = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
      const __half2_raw ar = __nv_cvt_fp8x2_to_halfraw2(a, __NV_E4M3);
      const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&ar));
      const __nv_fp8x2_storage_t b =
          __nv_cvt_float2_to_fp8x2(make_float2((f.x - g.x) * 32.f, (f.y - g.y) * 32.f), __NV_SATFINITE, __NV_E4M3);
      t1[i >> 1] |= (uint32_t)a << (16 * (i & 1));
      t2[i >> 1] |= (uint32_t)b << (16 * (i & 1));
    }
    const int tile = k >> 4, piece = (k & 15) >> 1;  // 16-byte piece of the row, this thread's half of it
    uint8_t* at = dst + tile * (2 * H * 128) + 8 * (k & 1);
    int second;
    if (tile < kTiles - 1) {
      at += h * 128 + ((piece ^ (h & 7)) << 4);
      second = H * 128;
    } else {
      at += h * 64 + ((piece ^ ((h >> 1) & 3)) << 4);
      second = H * 64;
    }
    *reinterpret_cast<uint2*>(at) = make_uint2(t1[0], t1[1]);
    *reinterpret_cast<uint2*>(at + second) = make_uint2(t2[0], t2[1]);  // H is a multiple of 16: the same swizzle
  }
  if (sub == 0) {
    head[h].z = m < 0x7F80u ? c_hi * down : __uint_as_float(0x7FC00000u);
    head[h].w = c_lo * down;
  }
}

constexpr int kLoaders = 128;
constexpr int kThreads = 32 * kLoadWarp + kLoaders;
constexpr int kPerLoader = kMaxK / kLoaders;  // list entries a loader resolves

// A barrier's parity tells its next phase from this one, not from the one after, so
// nobody may wait for a slot or an accumulator two uses ahead: the one loader group
// waits in order, and each slot and accumulator comes back to the same issuer.
template <bool kKv8, int CH>
struct Ring {
  static constexpr int slot_bytes = (kKv8 ? 1 : 2) * kAtomBytes;  // 128 dims of 128 rows
  static constexpr int slots = (CH == 2 ? 2 : 4) * (kKv8 ? 2 : 1);
  static constexpr int accs = kKv8 && CH == 2 ? 2 : 4;            // of 2 H (FP8) or H columns
  static_assert(slots % kIssuers == 0 && accs % kIssuers == 0 && slots <= kMaxSlots && accs <= kMaxAccs, "see above");
};

// CH: chunks of W heads that a summing thread holds (2 x 32 for H = 128, 32 for 64, 16
// for fewer).
template <bool kKv8, int CH, int W>
__global__ void __launch_bounds__(kThreads, 1)
k_attn_mass(const __grid_constant__ CUtensorMap tq, const MassArgs a) {
  using R = Ring<kKv8, CH>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const Layout L(a.H, R::slots * R::slot_bytes, a.ks);
  int32_t* rows = reinterpret_cast<int32_t*>(smem + L.rows);       // pool row of each slot of the slice, -1 = none
  float4* head = reinterpret_cast<float4*>(smem + L.head);          // per head: lse * log2(e), the logit's factor; two terms each
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L.bars);
  uint64_t* full = bars;                       // [slots]
  uint64_t* empty = bars + kMaxSlots;          // [slots]
  uint64_t* s_full = bars + 2 * kMaxSlots;     // [accs]
  uint64_t* s_empty = s_full + kMaxAccs;       // [accs]
  uint64_t* q_full = s_empty + kMaxAccs;       // the query's tile has landed, or (FP8 cache) its terms are written
  uint64_t* ready = q_full + 1;                // rows and lse are in shared memory
  uint64_t* mma_drain = ready + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x / a.splits, sp = blockIdx.x % a.splits;
  const int kbeg = sp * a.ks, kend = min(a.K, kbeg + a.ks);
  if (threadIdx.x == 0) {
    for (int i = 0; i < R::slots; ++i) {
      mbar_init(&full[i], kLoaders);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < R::accs; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], kSumWarps);
    }
    mbar_init(q_full, kKv8 ? kSumWarps : 1);
    mbar_init(ready, 1);
    mbar_init(mma_drain, kIssuers);
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
  const int cols = (kKv8 ? 2 : 1) * a.H, acc_cols = cols < 64 ? 64 : cols;

  if (!kKv8 && threadIdx.x == kMmaWarp * 32 && nblk > 0) {
    mbar_arrive_expect_tx(q_full, (uint32_t)(kAtoms * a.H * 128));
    for (int i = 0; i < kAtoms; ++i) tma_load_2d(smem + i * a.H * 128, &tq, q_full, 64 * i, t * a.H);
  }
  if (warp >= kLoadWarp && nblk > 0) {
    // ---------------------------------------------------------------- loaders
    const int li = threadIdx.x - kLoadWarp * 32;
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
        if constexpr (kKv8)  // the factors follow from the query's scale
          *reinterpret_cast<float2*>(head + li) = make_float2(hi, lo);
        else
          head[li] = make_float4(hi, lo, a.c_hi, a.c_lo);
      }
    }
    bool ok = !bar_red_or(kLoaderBarrier, kLoaders, false);
    if (li == 0) mbar_arrive(ready);
    const uint32_t ring = smem_u32(smem + L.ring);
    int slot = 0, phase = 0;
    // thread: rows rsub + 16 u, their 16-byte piece of each 128 bytes
    constexpr int kUnits = kRows * 8 / kLoaders, kStep = kLoaders / 8, kRowBytes = kKv8 ? kDQK : 2 * kDQK;
    const int rsub = li >> 3, piece = li & 7;
    const uint32_t swz = (uint32_t)rsub * 128u + (((uint32_t)piece ^ ((uint32_t)rsub & 7u)) << 4);
    for (int j = 0; j < nblk && ok; ++j) {
      int row[kUnits];
#pragma unroll
      for (int u = 0; u < kUnits; ++u) row[u] = rows[j * kRows + rsub + kStep * u];
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        ok = ok && !*abort_flag && mbar_wait(&empty[slot], phase ^ 1, a.err, a.wait_ns);
        if (ok) {
          const uint32_t dst = ring + slot * R::slot_bytes + swz;
          // the last tile: one atom of bf16, or the first 64 bytes of codes
          const int atoms = kKv8 || i == kTiles - 1 ? 1 : 2;
          if (!kKv8 || i < kTiles - 1 || piece < 4) {
#pragma unroll
            for (int h = 0; h < atoms; ++h)
#pragma unroll
              for (int u = 0; u < kUnits; ++u) {
                const bool live = row[u] >= 0;
                const uint8_t* src =
                    a.kv + (live ? (int64_t)row[u] * kRowBytes : 0) + i * R::slot_bytes / kRows + 128 * h + 16 * piece;
                cp_async_16_zfill(dst + h * kAtomBytes + u * kStep * 128, src, live ? 16u : 0u);
              }
          }
          cp_async_mbar_arrive(&full[slot]);  // counts once this thread's copies land
        }
        if (++slot == R::slots) {
          slot = 0;
          phase ^= 1;
        }
      }
    }
    if (!ok) *abort_flag = 1;
    cp_async_wait_all();  // nothing this thread copies is still in flight at exit
    __syncwarp();
  } else if (warp >= kMmaWarp && warp < kLoadWarp && nblk > 0) {
    // ---------------------------------------------------------------- MMA issuers
    // The whole warp runs the loop and one elected lane issues: control and operands
    // stay uniform, which the issue of an MMA wants (operands in uniform registers).
    {
      const uint32_t idesc = make_idesc(!kKv8, kRows, cols);  // bf16, or E4M3 (kind::f8f6f4)
      const int first = __shfl_sync(0xffffffffu, warp, 0) - kMmaWarp;
      bool ok = __all_sync(0xffffffffu, mbar_wait(q_full, 0, a.err, a.wait_ns));
      if constexpr (kKv8) fence_proxy_async_smem();  // the terms were written by the summing warps
      int i = first;  // tile of the block
      int slot = i, phase = 0, acc = i, aphase = 0;
      for (int it = first; it < nblk * kTiles; it += kIssuers) {
        ok = __all_sync(0xffffffffu, ok && !*abort_flag && mbar_wait(&s_empty[acc], aphase ^ 1, a.err, a.wait_ns) &&
                                         mbar_wait(&full[slot], phase, a.err, a.wait_ns));
        if (!ok) break;
        fence_proxy_async_smem();  // the rows were written by cp.async (generic proxy)
        tc_fence_after();
        // descriptors move by bytes / 16: 32 bytes inside the swizzled rows, or an atom
        const uint64_t ad = sw128_kmajor_desc(smem_u32(smem + L.ring + slot * R::slot_bytes));
        const bool last = i == kTiles - 1;
        if (elect_one()) {
        if constexpr (kKv8) {
          const uint32_t at = smem_u32(smem + i * cols * 128);
          const uint64_t bd = last ? sw64_kmajor_desc(at) : sw128_kmajor_desc(at);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)  // 32 dims each
            if (kk < 2 || !last)
              mma_ss<false>(tmem + acc * acc_cols, ad + 2 * kk, bd + 2 * kk, idesc, kk != 0);
        } else {
          const uint64_t bd = sw128_kmajor_desc(smem_u32(smem + 2 * i * a.H * 128));
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)  // 16 dims each
            if (kk < 4 || !last)
              mma_ss<true>(tmem + acc * acc_cols, ad + (kk >> 2) * (kAtomBytes / 16) + 2 * (kk & 3),
                           bd + (kk >> 2) * (a.H * 8) + 2 * (kk & 3), idesc, kk != 0);
        }
        mma_commit(&empty[slot]);
        mma_commit(&s_full[acc]);
        }
        __syncwarp();
        i = i + kIssuers < kTiles ? i + kIssuers : i + kIssuers - kTiles;
        slot += kIssuers;
        if (slot >= R::slots) {
          slot -= R::slots;
          phase ^= 1;
        }
        acc += kIssuers;
        if (acc >= R::accs) {
          acc -= R::accs;
          aphase ^= 1;
        }
      }
      if (!ok) *abort_flag = 1;
      // drain, also after a failed wait: the query's copy has landed and no MMA
      // still reads shared memory or writes TMEM
      if constexpr (!kKv8) mbar_wait(q_full, 0, a.err, kDrainLimitNs);
      if (elect_one()) mma_commit(mma_drain);
      __syncwarp();
      mbar_wait(mma_drain, 0, a.err, kDrainLimitNs);
    }
    __syncwarp();
  } else if (warp < kSumWarps && nblk > 0) {
    // ---------------------------------------------------------------- sums
    const int wg = warp >> 2, r = threadIdx.x & 127;  // half of the heads, row of the block
    const int heads = a.H >> 1, h0 = wg * heads;
    const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16) + h0;
    const float inv_h = 1.f / (float)a.H, most = (float)heads * inv_h;  // powers of two
    bool ok = __all_sync(0xffffffffu, mbar_wait(ready, 0, a.err, a.wait_ns));
    if constexpr (kKv8) {
      query_to_e4m3(a.q + (int64_t)t * a.H * kDQK, smem, a.H, a.c_hi, a.c_lo, head);
      fence_proxy_async_smem();  // the MMAs read the terms through the async proxy
      sums_sync();               // the factors that other threads wrote
      if (lane == 0) mbar_arrive(q_full);
    }
    // this thread's row of a block: pool row, position and (FP8 cache) tile scales
    int row_next = -1, s_next = 0;
    uint2 tiles_next = make_uint2(0u, 0u);
    auto row_of = [&](int j) {
      const int k = j * kRows + r;
      row_next = rows[k];
      if (row_next >= 0) {
        s_next = __ldg(a.idx + (int64_t)t * a.K + kbeg + k);
        if constexpr (kKv8) tiles_next = ld_nc_v2(a.kv_scale + (int64_t)row_next * 8);
      }
    };
    if (ok) row_of(0);
    int acc = 0, aphase = 0;
    for (int j = 0; j < nblk; ++j) {
      const bool live = ok && row_next >= 0;
      const int s = s_next;
      const uint2 tiles = tiles_next;
      if (ok && j + 1 < nblk) row_of(j + 1);  // its loads' latency overlaps this block (after a failed wait: no row ids)
      float x[CH][W];
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        ok = ok && __all_sync(0xffffffffu, !*abort_flag && mbar_wait(&s_full[acc], aphase, a.err, a.wait_ns));
        if (ok) {
          tc_fence_after();
          const uint32_t at = t_lane + acc * acc_cols;
          // fewer than W heads: the other columns are read and left out below
          if constexpr (kKv8) {
            const float s1 = tile_scale((i < kTiles - 1 ? tiles.x >> (8 * i) : tiles.y) & 0xFFu), s2 = s1 * 0x1p-5f;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
              uint32_t v1[W], v2[W];
              tmem_ld(at + W * c, v1);
              if constexpr (CH == 1) tmem_ld(at + a.H + W * c, v2);
              tmem_ld_wait_regs(v1);
#pragma unroll
              for (int e = 0; e < W; ++e)
                x[c][e] = i == 0 ? __uint_as_float(v1[e]) * s1 : fmaf(__uint_as_float(v1[e]), s1, x[c][e]);
              if constexpr (CH == 2) tmem_ld(at + a.H + W * c, v2);  // 64 logits leave registers for one term
              tmem_ld_wait_regs(v2);
#pragma unroll
              for (int e = 0; e < W; ++e) x[c][e] = fmaf(__uint_as_float(v2[e]), s2, x[c][e]);
            }
          } else {
            uint32_t v[CH][W];
#pragma unroll
            for (int c = 0; c < CH; ++c) tmem_ld(at + W * c, v[c]);
#pragma unroll
            for (int c = 0; c < CH; ++c) tmem_ld_wait_regs(v[c]);
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
              for (int e = 0; e < W; ++e) {
                const float y = __uint_as_float(v[c][e]);
                x[c][e] = i == 0 ? y : x[c][e] + y;
              }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_empty[acc]);
        }
        if (++acc == R::accs) {
          acc = 0;
          aphase ^= 1;
        }
      }
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int e = 0; e < W; ++e) {
          const float4 h = head[h0 + W * c + e];
          const float p = ex2_ftz(fmaf(x[c][e], h.z, -h.x) + fmaf(x[c][e], h.w, -h.y));
          if (W * c + e < heads) sum[e & 3] += p;
        }
      // this half's share of the mean over all heads
      const float w = ((sum[0] + sum[1]) + (sum[2] + sum[3])) * inv_h;
      // a NaN (from a NaN or an lse that does not belong to these logits) adds nothing
      const float lim = w > 0.f ? fminf(w, most) : 0.f;
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
// split is its waves times (start + blocks).  Measured: 8 tokens x 2048 rows take
// 9.0 us in 16 slices, 26.6 in 2, 47.9 in 1; 400 tokens 137 us in 1, 148 in 2.
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

template <bool kKv8, int CH, int W>
cudaError_t launch(const CUtensorMap& tq, MassArgs a, cudaStream_t st) {
  static thread_local int attr_dev = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (attr_dev != dev) {
    cudaError_t e =
        cudaFuncSetAttribute(k_attn_mass<kKv8, CH, W>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
    attr_dev = dev;
  }
  using R = Ring<kKv8, CH>;
  const int T = a.s.num_tokens, blocks = (a.K + kRows - 1) / kRows;
  const int sp = mass_splits(T, a.K), per = (blocks + sp - 1) / sp;
  a.ks = per * kRows;
  a.splits = (blocks + per - 1) / per;
  const int64_t ctas = (int64_t)T * a.splits;
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_pdl("attn_mass", k_attn_mass<kKv8, CH, W>, dim3((unsigned)ctas), dim3(kThreads),
                    (size_t)(Layout(a.H, R::slots * R::slot_bytes, a.ks).total + 1024), st, tq, a);
}

}  // namespace

cudaError_t launch_attn_mass(const SeqsDev& s, const __nv_bfloat16* q, const void* kv, const uint8_t* kv8_scale,
                             const int32_t* idx, int K, int H, float scale, const float* lse, int64_t* mass,
                             int64_t ld, uint32_t* err, cudaStream_t st) {
  CUtensorMap tq;
  if (!make_bf16_rows_map(&tq, q, kDQK, (uint64_t)s.num_tokens * H, H)) return cudaErrorInvalidValue;
  const double c = (double)scale * 1.4426950408889634;
  const float c_hi = (float)c;
  const MassArgs a{s, q, static_cast<const uint8_t*>(kv), kv8_scale, idx, lse, reinterpret_cast<unsigned long long*>(mass),
                   ld, K, H, 0, 0, c_hi, (float)(c - c_hi), err, wait_limit_ns()};
  cudaError_t e;
  if (kv8_scale)
    e = H == 128 ? launch<true, 2, 32>(tq, a, st) : H == 64 ? launch<true, 1, 32>(tq, a, st) : launch<true, 1, 16>(tq, a, st);
  else
    e = H == 128  ? launch<false, 2, 32>(tq, a, st)
        : H == 64 ? launch<false, 1, 32>(tq, a, st)
                  : launch<false, 1, 16>(tq, a, st);
  if (e != cudaSuccess) return e;
  return counted(cudaGetLastError());
}

}  // namespace dsa
