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
//   * two threads, taking tiles in turn, issue the MMAs, eight per tile, each
//     tile into an accumulator of its own (a ring of four): the waits, fence, issue and
//     commits are one serial chain per tile, and two of them overlap;
//   * eight warps, two per lane quarter with half of the heads each, add the
//     five partial logits in registers and take p = 2^(c S - L_h), summed over h.
// FP8 cache.  Its codes become fp16, one conversion instruction per pair and exact;
// their tiles' scales, powers of two per row, multiply the partial logits instead
// in the thread that owns the row.  The query becomes fp16 as
// well, each head times the power of two that brings its largest value to 2^14:
// values 2^-28 of that and less lose bits, 2^-39 of the largest at most.  (As bf16
// the codes cost five times the instructions, and that bounded the kernel: 106 us
// where the bf16 cache takes 47.)  A CTA takes 64 heads then, which leaves shared
// memory for the staged codes and registers for twice the loader warps.
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
// What bounds it: a block's 147 KB of rows against 36 MMAs.  MEASURED
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
constexpr int kSlotBytes = 2 * kAtomBytes;
constexpr int kSumWarps = 8;                 // warps 0-7
constexpr int kIssuers = 2;                  // warps 8-9, one thread each; warp 8 owns TMEM
constexpr int kLoaderBarrier = 1, kSumBarrier = 2;
constexpr int kMmaWarp = kSumWarps;
constexpr int kLoadWarp = kMmaWarp + kIssuers;
constexpr int kMaxSlots = 4;
constexpr int kAccs = 4;                     // accumulators of up to 128 columns
constexpr int kTmemCols = 512;

struct MassArgs {
  SeqsDev s;
  const uint8_t* kv;         // bf16 rows, or E4M3 codes
  const uint8_t* kv_scale;   // FP8 cache: tile-scale bytes [rows, 8]
  const int32_t* idx;
  const float* lse;
  unsigned long long* mass;
  int64_t ld;
  int K, H, hg, ks, splits, slots;  // hg heads per CTA
  float c_hi, c_lo;          // scale * log2(e) as two terms
  uint32_t* err;
  uint64_t wait_ns;
};

// Shared memory from a 1024-aligned base: query, ring, staged codes, rows, lse, barriers.
struct Layout {
  int q_atom, ring, stage, rows, head, bars, total;
  __host__ __device__ Layout(int H, int slots, int ahead, int ks) {
    q_atom = H * 128;
    ring = kAtoms * q_atom;
    stage = ring + slots * kSlotBytes;
    rows = stage + ahead * (kSlotBytes / 2);
    head = rows + ks * 4;                  // and 32 entries more: chunks of 32 heads are read whole
    bars = head + H * 16 + 512;
    total = bars + (2 * kMaxSlots + 2 * kAccs + 5) * 8 + 16;
  }
};

// A barrier of the summing warps.
__device__ __forceinline__ void sums_sync() {
  asm volatile("barrier.cta.sync %0, %1;" ::"n"(kSumBarrier), "n"(kSumWarps * 32) : "memory");
}

// FP8 cache: the query tile in shared memory from bf16 to fp16, in place, by the
// summing warps.  256 / heads neighbouring threads share a head; its factor becomes
// scale log2(e) / 2^s with s the power that was multiplied in.
__device__ __forceinline__ void query_to_f16(uint8_t* q, int q_atom, int heads, float c_hi, float c_lo, float4* head) {
  const int per = kSumWarps * 32 / heads;        // threads per head: 4, 8 or 16
  const int h = threadIdx.x / per, sub = threadIdx.x % per;
  const int chunks = kAtoms * 8;                 // 16-byte pieces of a head
  uint32_t m = 0;
  for (int k = sub; k < chunks; k += per) {
    const uint4 v = *reinterpret_cast<const uint4*>(q + (k >> 3) * q_atom + h * 128 + (k & 7) * 16);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
  }
  for (int o = 1; o < per; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  // largest value to [2^14, 2^15); zero, infinite and NaN heads keep their scale
  int s = m == 0u || m >= 0x7F80u ? 0 : 141 - (int)(m >> 7);
  s = min(s, 126);
  const float up = __uint_as_float((uint32_t)(127 + s) << 23), down = __uint_as_float((uint32_t)(127 - s) << 23);
  for (int k = sub; k < chunks; k += per) {
    uint4* at = reinterpret_cast<uint4*>(q + (k >> 3) * q_atom + h * 128 + (k & 7) * 16);
    uint4 v = *at;
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 r = __floats2half2_rn(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xFFFF0000u) * up);
      w[i] = *reinterpret_cast<const uint32_t*>(&r);
    }
    *at = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (sub == 0) {
    head[h].z = c_hi * down;
    head[h].w = c_lo * down;
  }
}

// Operand slots and staged FP8 codes (16 KB per tile) share what the query leaves.
template <bool kKv8, int CH>
struct Roles {
  static_assert(!kKv8 || CH == 1, "FP8 cache: up to 64 heads per CTA");
  static constexpr int groups = kKv8 ? 2 : 1;    // loader groups of 128 threads, taking tiles in turn
  static constexpr int loaders = 128 * groups;
  static constexpr int threads = 32 * kLoadWarp + loaders;
  // A barrier's parity tells its next phase from this one, not from the one after, so
  // nobody may wait for a slot or an accumulator two uses ahead: each comes back to
  // the same issuer and the same loader group, which waits in the order of its uses.
  static constexpr int slots = kKv8 || CH == 2 ? 2 : 4;
  static_assert(slots % groups == 0 && slots % kIssuers == 0 && kAccs % kIssuers == 0, "see above");
  static constexpr int ahead = kKv8 ? 2 : 0;     // tiles that a group stages ahead
};

// CH: chunks of 32 heads that a summing thread holds (two for H = 128).
template <bool kKv8, int CH>
__global__ void __launch_bounds__(Roles<kKv8, CH>::threads, 1)
k_attn_mass(const __grid_constant__ CUtensorMap tq, const MassArgs a) {
  constexpr int kLoaders = Roles<kKv8, CH>::loaders;
  constexpr int kPerLoader = (kMaxK + kLoaders - 1) / kLoaders;  // list entries a loader resolves
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const Layout L(a.hg, a.slots, Roles<kKv8, CH>::ahead * Roles<kKv8, CH>::groups, a.ks);
  int32_t* rows = reinterpret_cast<int32_t*>(smem + L.rows);       // pool row of each slot of the slice, -1 = none
  float4* head = reinterpret_cast<float4*>(smem + L.head);          // per head: lse * log2(e), the logit's factor; two terms each
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L.bars);
  uint64_t* full = bars;                       // [slots]
  uint64_t* empty = bars + kMaxSlots;          // [slots]
  uint64_t* s_full = bars + 2 * kMaxSlots;     // [kAccs]
  uint64_t* s_empty = s_full + kAccs;          // [kAccs]
  uint64_t* q_full = s_empty + kAccs;
  uint64_t* q_half = q_full + 1;               // FP8 cache: the query is fp16
  uint64_t* ready = q_half + 1;                // rows and lse are in shared memory
  uint64_t* mma_drain = ready + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = a.H / a.hg, unit = blockIdx.x / groups, head0 = (blockIdx.x % groups) * a.hg;
  const int t = unit / a.splits, sp = unit % a.splits;
  const int kbeg = sp * a.ks, kend = min(a.K, kbeg + a.ks);
  if (threadIdx.x == 0) {
    for (int i = 0; i < a.slots; ++i) {
      mbar_init(&full[i], kKv8 ? kLoaders / 32 / Roles<kKv8, CH>::groups : kLoaders);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < kAccs; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], kSumWarps);
    }
    mbar_init(q_full, 1);
    mbar_init(q_half, kSumWarps);
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
  const int acc_cols = a.hg < 64 ? 64 : a.hg;

  if (threadIdx.x == kMmaWarp * 32 && nblk > 0) {
    mbar_arrive_expect_tx(q_full, (uint32_t)(kAtoms * L.q_atom));
    for (int i = 0; i < kAtoms; ++i) tma_load_2d(smem + i * L.q_atom, &tq, q_full, 64 * i, t * a.H + head0);
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
      if (li < a.hg) {
        const float v = __ldg(a.lse + (int64_t)t * a.H + head0 + li);
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
    if constexpr (!kKv8) {
      // thread: rows rsub + kStep u, their 16-byte piece of each atom
      constexpr int kUnits = kRows * 8 / kLoaders, kStep = kLoaders / 8;
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
            const uint32_t dst = ring + slot * kSlotBytes + swz;
#pragma unroll
            for (int h = 0; h < (i < kTiles - 1 ? 2 : 1); ++h)
#pragma unroll
              for (int u = 0; u < kUnits; ++u) {
                const bool live = row[u] >= 0;
                const uint8_t* src = a.kv + (live ? (int64_t)row[u] * (kDQK * 2) : 0) + 256 * i + 128 * h + 16 * piece;
                cp_async_16_zfill(dst + h * kAtomBytes + u * kStep * 128, src, live ? 16u : 0u);
              }
            cp_async_mbar_arrive(&full[slot]);  // counts once this thread's copies land
          }
          if (++slot == a.slots) {
            slot = 0;
            phase ^= 1;
          }
        }
      }
    } else {
      // Group g of 128 threads takes tiles g, g + 2, ...: the waits, fence and barrier
      // of a tile cost each warp as much as its conversions.  Thread: rows rsub + 16 u, 16
      // codes each.  They come kAhead of the group's tiles early into a place of the
      // thread's own (no barrier), are converted and stored where the bf16 gather
      // would have put the values.  A row that is not live reads row 0 of the pool:
      // its logits, in a lane of their own, are not used.
      using R = Roles<kKv8, CH>;
      constexpr int kGroup = kLoaders / R::groups, kUnits = kRows * 8 / kGroup, kAhead = R::ahead;
      static_assert(kGroup == 128 && kUnits == 8, "16 rows per step");
      const int g = li / kGroup, lt = li % kGroup, rsub = lt >> 3, piece = lt & 7;
      uint8_t* stage = smem + L.stage + g * (kAhead * kSlotBytes / 2) + lt * 16;
      // 16 codes fill two 16-byte pieces; the second atom's lanes write theirs in
      // the other order, so that a row's eight lanes hit eight different bank groups
      const uint32_t base = (uint32_t)(piece >> 2) * kAtomBytes + (uint32_t)rsub * 128u;
      const uint32_t swz = base + (((uint32_t)(2 * (piece & 3) + (piece >> 2)) ^ ((uint32_t)rsub & 7u)) << 4);
      const bool second = piece >= 4;
      const int total = nblk * kTiles;
      int next = g, next_place = 0;  // the next tile to fetch and its place
      auto fetch = [&]() {
        if (next < total) {
          const int j = next / kTiles, i = next - j * kTiles;
          if (i < kTiles - 1 || !second) {
            const uint8_t* src = a.kv + 128 * i + 16 * piece;
            const int32_t* rj = rows + j * kRows + rsub;
#pragma unroll
            for (int u = 0; u < kUnits; ++u)
              cp_async_16(stage + (next_place * kUnits + u) * (kGroup * 16), src + (int64_t)max(rj[16 * u], 0) * kDQK);
          }
          next += R::groups;
          if (++next_place == kAhead) next_place = 0;
        }
        cp_async_commit();
      };
      for (int i = 0; i < kAhead; ++i) fetch();
      int place = 0, tile = g;
      slot = g;
      for (int it = g; it < total; it += R::groups) {
        cp_async_wait<kAhead - 1>();  // this thread's codes of the tile are in place
        uint4 c[kUnits];
#pragma unroll
        for (int u = 0; u < kUnits; ++u)
          c[u] = *reinterpret_cast<const uint4*>(stage + (place * kUnits + u) * (kGroup * 16));
        if (++place == kAhead) place = 0;
        fetch();
        ok = __all_sync(0xffffffffu, ok && !*abort_flag && mbar_wait(&empty[slot], phase ^ 1, a.err, a.wait_ns));
        if (!ok) break;
        if (tile < kTiles - 1 || !second) {
          uint8_t* dst = smem + L.ring + slot * kSlotBytes;
#pragma unroll
          for (int u = 0; u < kUnits; ++u) {
            const uint4 lo = e4m3x8_to_f16x8(make_uint2(c[u].x, c[u].y));
            const uint4 hi = e4m3x8_to_f16x8(make_uint2(c[u].z, c[u].w));
            *reinterpret_cast<uint4*>(dst + swz + u * 2048) = second ? hi : lo;
            *reinterpret_cast<uint4*>(dst + (swz ^ 16u) + u * 2048) = second ? lo : hi;
          }
        }
        fence_proxy_async_smem();  // the MMAs read these stores through the async proxy
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[slot]);
        tile = tile + R::groups < kTiles ? tile + R::groups : tile + R::groups - kTiles;
        slot += R::groups;
        if (slot >= a.slots) {
          slot -= a.slots;
          phase ^= 1;
        }
      }
    }
    if (!ok) *abort_flag = 1;
    cp_async_wait_all();  // nothing this thread copies is still in flight at exit
    __syncwarp();
  } else if (warp >= kMmaWarp && warp < kLoadWarp && nblk > 0) {
    // ---------------------------------------------------------------- MMA issuers
    if (lane == 0) {
      const uint32_t idesc = make_idesc(!kKv8, kRows, a.hg);  // bf16 or (FP8 cache) fp16 operands
      bool ok = mbar_wait(kKv8 ? q_half : q_full, 0, a.err, a.wait_ns);
      if constexpr (kKv8) fence_proxy_async_smem();  // the query was rewritten by the summing warps
      int i = warp - kMmaWarp;  // tile of the block
      int slot = i, phase = 0, acc = i, aphase = 0;
      for (int it = i; it < nblk * kTiles; it += kIssuers) {
        ok = ok && !*abort_flag && mbar_wait(&s_empty[acc], aphase ^ 1, a.err, a.wait_ns) &&
             mbar_wait(&full[slot], phase, a.err, a.wait_ns);
        if (!ok) break;
        fence_proxy_async_smem();  // the rows were written by cp.async (generic proxy)
        tc_fence_after();
        const uint64_t ad = sw128_kmajor_desc(smem_u32(smem + L.ring + slot * kSlotBytes));
        const uint64_t bd = sw128_kmajor_desc(smem_u32(smem + 2 * i * L.q_atom));
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // descriptors move by bytes / 16: an atom, or 32 bytes in the 128-byte rows
          if (h == 1 && i == kTiles - 1) break;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ss<true>(tmem + acc * acc_cols, ad + h * (kAtomBytes / 16) + 2 * kk, bd + h * (L.q_atom / 16) + 2 * kk,
                         idesc, (h | kk) != 0);
        }
        mma_commit(&empty[slot]);
        mma_commit(&s_full[acc]);
        i = i + kIssuers < kTiles ? i + kIssuers : i + kIssuers - kTiles;
        slot += kIssuers;
        if (slot >= a.slots) {
          slot -= a.slots;
          phase ^= 1;
        }
        acc += kIssuers;
        if (acc >= kAccs) {
          acc -= kAccs;
          aphase ^= 1;
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
    const int heads = a.hg >> 1, h0 = wg * heads;
    const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16) + h0;
    const float inv_h = 1.f / (float)a.H, most = (float)heads * inv_h;  // powers of two
    bool ok = __all_sync(0xffffffffu, mbar_wait(ready, 0, a.err, a.wait_ns));
    if constexpr (kKv8) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait(q_full, 0, a.err, a.wait_ns));
      if (ok) query_to_f16(smem, L.q_atom, a.hg, a.c_hi, a.c_lo, head);
      fence_proxy_async_smem();  // the MMAs read the query through the async proxy
      sums_sync();               // the factors that other threads wrote
      if (lane == 0) mbar_arrive(q_half);
    }
    int acc = 0, aphase = 0;
    for (int j = 0; j < nblk; ++j) {
      const int k = j * kRows + r;
      const bool live = ok && rows[k] >= 0;
      const int s = live ? __ldg(a.idx + (int64_t)t * a.K + kbeg + k) : 0;
      uint2 tiles = make_uint2(0u, 0u);  // FP8 cache: the row's tile scales
      if constexpr (kKv8) tiles = live ? ld_nc_v2(a.kv_scale + (int64_t)rows[k] * 8) : tiles;
      float x[CH][32];
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        ok = ok && __all_sync(0xffffffffu, !*abort_flag && mbar_wait(&s_full[acc], aphase, a.err, a.wait_ns));
        if (ok) {
          tc_fence_after();
          uint32_t v[CH][32];  // fewer than 32 heads: the other columns are read and left out below
#pragma unroll
          for (int c = 0; c < CH; ++c) tmem_ld32(t_lane + acc * acc_cols + 32 * c, v[c]);
#pragma unroll
          for (int c = 0; c < CH; ++c) tmem_ld_wait_regs(v[c]);
          const float sc = kKv8 ? tile_scale((i < kTiles - 1 ? tiles.x >> (8 * i) : tiles.y) & 0xFFu) : 1.f;
#pragma unroll
          for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float y = __uint_as_float(v[c][e]);
              if constexpr (kKv8)
                x[c][e] = i == 0 ? y * sc : fmaf(y, sc, x[c][e]);
              else
                x[c][e] = i == 0 ? y : x[c][e] + y;
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
          const float4 h = head[h0 + 32 * c + e];
          const float p = ex2_ftz(fmaf(x[c][e], h.z, -h.x) + fmaf(x[c][e], h.w, -h.y));
          if (32 * c + e < heads) sum[e & 3] += p;
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
cudaError_t launch(const CUtensorMap& tq, MassArgs a, cudaStream_t st) {
  using R = Roles<kKv8, CH>;
  static thread_local int attr_dev = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (attr_dev != dev) {
    cudaError_t e =
        cudaFuncSetAttribute(k_attn_mass<kKv8, CH>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
    attr_dev = dev;
  }
  a.hg = kKv8 && a.H > 64 ? 64 : a.H;
  const int T = a.s.num_tokens * (a.H / a.hg), blocks = (a.K + kRows - 1) / kRows;
  const int sp = mass_splits(T, a.K), per = (blocks + sp - 1) / sp;
  a.ks = per * kRows;
  a.splits = (blocks + per - 1) / per;
  a.slots = R::slots;
  const int64_t ctas = (int64_t)T * a.splits;
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_pdl("attn_mass", k_attn_mass<kKv8, CH>, dim3((unsigned)ctas), dim3(R::threads),
                    (size_t)(Layout(a.hg, a.slots, R::ahead * R::groups, a.ks).total + 1024), st, tq, a);
}

}  // namespace

cudaError_t launch_attn_mass(const SeqsDev& s, const __nv_bfloat16* q, const void* kv, const uint8_t* kv8_scale,
                             const int32_t* idx, int K, int H, float scale, const float* lse, int64_t* mass,
                             int64_t ld, uint32_t* err, cudaStream_t st) {
  CUtensorMap tq;
  if (!make_bf16_rows_map(&tq, q, kDQK, (uint64_t)s.num_tokens * H, kv8_scale && H > 64 ? 64 : H)) return cudaErrorInvalidValue;
  const double c = (double)scale * 1.4426950408889634;
  const float c_hi = (float)c;
  const MassArgs a{s, static_cast<const uint8_t*>(kv), kv8_scale, idx, lse, reinterpret_cast<unsigned long long*>(mass),
                   ld, K, H, 0, 0, 0, 0, c_hi, (float)(c - c_hi), err, wait_limit_ns()};
  cudaError_t e = kv8_scale ? launch<true, 1>(tq, a, st)
                            : (H == 128 ? launch<false, 2>(tq, a, st) : launch<false, 1>(tq, a, st));
  if (e != cudaSuccess) return e;
  return counted(cudaGetLastError());
}

}  // namespace dsa
