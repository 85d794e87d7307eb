// Eviction from the paged caches by accumulated attention weight: which
// positions of each sequence stay (select), and their rows, moved to new pages
// (mark + compact).
//
// select.  The budget's largest of a row of keys, ties to the lower position.  A
// key is the mass rounded to fp32, order-preserving in 32 bits (24 bits of a
// ranking statistic; 64-bit keys would double the digits of the radix select);
// the positions that always stay -- the first `sink`, the last `recent` --
// have the largest key.  One cluster of CTAs takes a sequence, each a run of
// its positions with the keys in shared memory, read from HBM once.  The
// cluster resolves the budget's key digit by digit (11, 11, 10 bits): every
// CTA counts its keys and adds its counts to the bins' owners through distributed
// shared memory, and each finds the same bin by a scan.  Counts before each CTA give
// the output offsets, so the positions come out ascending.  Latency bound: four
// cluster barriers and the passes over the keys: 8 x 32,768 positions 14 us, one
// sequence of 3001 9.9 us.
//
// mark.  A destination page must be no page that the call reads and no
// destination twice, or rows would be overwritten while others still read
// them.  One cluster checks this on bitmaps over the pool's pages, so that a bad
// table is an error and not a race.
//
// compact.  A block takes half a destination page of one sequence: 32 rows of
// every pool, 16 bytes per access where the row size allows.  HBM bound: each
// kept byte is read once and written once, as streaming data (35.5 -> 32.1 us): 8 x
// 8192 rows of 1228 bytes take 32 us with the check of the pages (6 us), 94 % of the
// measured copy rate in between.
#include <cooperative_groups.h>

#include "row_of.cuh"
#include "topk_select.cuh"

namespace dsa {

namespace {

namespace cg = cooperative_groups;
using topk::kD1Bins;
using topk::kD2Bins;
using topk::kD3Bins;

constexpr int kCluster = 8;                    // most CTAs per sequence (the portable cluster size)
constexpr int kSlotsMax = 40960;               // keys a CTA keeps in shared memory (160 KB)
constexpr uint32_t kForced = 0xFFFFFFFFu;      // above any key of a number

struct SelectArgs {
  const int32_t* ctx_len;
  const int64_t* mass;
  int64_t ld;
  int max_ctx, budget, recent, sink;
  int32_t* keep;
  int32_t* keep_len;
  uint32_t* err;
};

struct SelectSmem {
  uint32_t hist[kD1Bins];                      // this CTA's counts of the current digit
  uint32_t total[kD1Bins + kD2Bins + kD3Bins]; // the cluster's counts: this CTA's share of each digit's bins
  uint32_t buf[33];
  uint32_t bin, above, inside, gt, eq;
};

// kStaged: the CTA's keys fit in shared memory; otherwise each pass reads the
// masses again (from L2 in the main).
template <bool kStaged, int kSelThreads>
__global__ void __launch_bounds__(kSelThreads) k_evict_select(const SelectArgs a) {
  extern __shared__ uint32_t keys[];
  __shared__ SelectSmem sm;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int b = blockIdx.x / C, tid = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  const int n = __ldg(a.ctx_len + b);
  int32_t* keep = a.keep + (int64_t)b * a.budget;
  const bool bad = n < 0 || n > a.max_ctx;
  const int kept = bad ? 0 : min(n, a.budget);
  for (int i = kept + rank * kSelThreads + tid; i < a.budget; i += C * kSelThreads) keep[i] = -1;
  if (rank == 0 && tid == 0) {
    a.keep_len[b] = kept;
    if (bad) raise_error(a.err, kErrBadIndex);
  }
  if (kept == n || bad) {  // nothing to choose; the same for the whole cluster
    for (int i = rank * kSelThreads + tid; i < kept; i += C * kSelThreads) keep[i] = i;
    return;
  }
  const int per = ((n + C - 1) / C + 3) & ~3;
  const int s0 = min(n, rank * per), len = min(n, s0 + per) - s0;
  const int64_t* mass = a.mass + (int64_t)b * a.ld + s0;
  auto key_of = [&](int i) -> uint32_t {
    const int s = s0 + i;
    return s < a.sink || s >= n - a.recent ? kForced : order_key(__ll2float_rn(__ldg(mass + i)));
  };
  auto key_at = [&](int i) -> uint32_t { return kStaged ? keys[i] : key_of(i); };
  for (int i = tid; i < kD1Bins; i += kSelThreads) sm.hist[i] = 0u;
  for (int i = tid; i < kD1Bins + kD2Bins + kD3Bins; i += kSelThreads) sm.total[i] = 0u;
  __syncthreads();
  auto started = cluster.barrier_arrive();  // waited for before the first addition to another CTA's share
  uint32_t prefix = 0, need = (uint32_t)a.budget;
  for (int level = 0; level < 3; ++level) {
    const int off = level == 0 ? 0 : (level == 1 ? kD1Bins : kD1Bins + kD2Bins), bins = level < 2 ? kD1Bins : kD3Bins;
    if (level > 0) {
      for (int d = tid; d < bins; d += kSelThreads) sm.hist[d] = 0u;
      __syncthreads();
    }
    constexpr int kKeys = 4;  // loads of a batch are issued before its counts
    for (int i0 = 0; i0 < len; i0 += kKeys * kSelThreads) {
      uint32_t key[kKeys];
#pragma unroll
      for (int u = 0; u < kKeys; ++u) {
        const int i = i0 + u * kSelThreads + tid;
        key[u] = i >= len ? 0u : (level == 0 ? key_of(i) : key_at(i));
      }
#pragma unroll
      for (int u = 0; u < kKeys; ++u) {
        const int i = i0 + u * kSelThreads + tid;
        bool in = i < len;
        if (kStaged && level == 0 && in) keys[i] = key[u];
        uint32_t digit;
        if (level == 0) {
          digit = topk::digit1(key[u]);
        } else if (level == 1) {
          in = in && topk::digit1(key[u]) == prefix;
          digit = topk::digit2(key[u]);
        } else {
          in = in && (key[u] >> 10) == prefix;
          digit = topk::digit3(key[u]);
        }
        hist_add(sm.hist, digit, in);  // never-attended positions share one bin
      }
    }
    __syncthreads();
    // bins of the digit are summed in equal shares by the cluster's CTAs; adding
    // the few bins that hold keys to their owners moves less than every CTA
    // reading every table (8 CTAs: 8 us less per call)
    if (level == 0) cluster.barrier_wait(std::move(started));
    const int share = __ffs(bins / C) - 1, mask = bins / C - 1;  // (bins and C are powers of two)
    for (int d = tid; d < bins; d += kSelThreads) {
      const uint32_t v = sm.hist[d];
      if (v) atomicAdd(cluster.map_shared_rank(sm.total + off, d >> share) + (d & mask), v);
    }
    cluster.sync();
    // from the highest digit down, `pt` digits per thread; the thread in which
    // the running count reaches `need` holds the digit
    constexpr int kPer = kD1Bins / kSelThreads;
    const int pt = bins / kSelThreads, top = bins - 1 - tid * pt;
    uint32_t c[kPer], sum = 0;
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int d = top - u;
      c[u] = u < pt ? cluster.map_shared_rank(sm.total + off, d >> share)[d & mask] : 0u;
      sum += c[u];
    }
    uint32_t all;
    uint32_t above = topk::block_scan(sum, sm.buf, &all);
    if (above < need && need <= above + sum) {
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        if (above < need && need <= above + c[u]) {
          sm.bin = (uint32_t)(top - u);
          sm.above = above;
          sm.inside = c[u];
        }
        above += c[u];
      }
    }
    __syncthreads();
    prefix = (prefix << (level < 2 ? 11 : 10)) | sm.bin;
    need -= sm.above;
    if (need == sm.inside) {  // the whole bin stays: its lowest key is the border
      prefix <<= level == 0 ? 21 : (level == 1 ? 10 : 0);
      need = 0xFFFFFFFFu;
      break;
    }
    __syncthreads();
  }
  // Keys above tau stay, and the `need` lowest positions of those that equal it
  // (need = 2^32 - 1: all of them, and tau may be lower than any key of its bin).
  const bool whole = need == 0xFFFFFFFFu;
  const uint32_t tau = prefix;
  if (tid < 2) (tid == 0 ? sm.gt : sm.eq) = 0u;
  __syncthreads();
  uint32_t gt = 0, eq = 0;
  for (int i = tid; i < len; i += kSelThreads) {
    const uint32_t key = key_at(i);
    gt += key > tau ? 1u : 0u;
    eq += key == tau ? 1u : 0u;
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if ((tid & 31) == 0) {
    atomicAdd(&sm.gt, gt);
    atomicAdd(&sm.eq, eq);
  }
  cluster.sync();
  uint32_t gt_before = 0, eq_before = 0;
  for (int r = 0; r < rank; ++r) {
    gt_before += *cluster.map_shared_rank(&sm.gt, r);
    eq_before += *cluster.map_shared_rank(&sm.eq, r);
  }
  auto done = cluster.barrier_arrive();  // no CTA leaves while another reads its shared memory
  const uint32_t taken = min(eq_before, need), at = gt_before + taken, left = whole ? 0xFFFFFFFFu : need - taken;
  topk::emit_selected(
      len, tau, left, a.budget - (int)at, [&](int i) { return make_int2(s0 + i, (int)key_at(i)); }, keep + at,
      sm.buf);
  cluster.barrier_wait(std::move(done));
}

// ---------------------------------------------------------------- compaction

constexpr int kMoveThreads = 128;
constexpr int kMoveRows = 32;                  // per block: a part of one destination page

struct MoveArgs {
  SeqsDev s;
  const int32_t* keep;
  const int32_t* keep_len;
  int budget;
  const int32_t* new_table;
  int new_max_pages, new_pages;
  int npools;
  const uint8_t* src[DSA_MAX_POOLS];
  uint8_t* dst[DSA_MAX_POOLS];
  int row_bytes[DSA_MAX_POOLS], vec[DSA_MAX_POOLS];
  RowDivisor by[DSA_MAX_POOLS];  // a row's vectors (at most 16,384, and 32 rows a block)
  const int64_t* mass;
  int64_t* new_mass;
  int64_t ld, new_ld;
  bool in_place;           // some pool is its own destination: its pages must not be read
  uint32_t *read, *written, *twice;  // bitmaps over pages
  int words;               // of each bitmap
  uint32_t* err;
};

// Rows of sequence b that move: none when its lengths are impossible.
__device__ __forceinline__ int rows_to_move(const MoveArgs& a, int b) {
  const int n = __ldg(a.keep_len + b), ctx = __ldg(a.s.ctx_len + b);
  const bool ok = n >= 0 && n <= a.budget && n <= ctx && ctx <= a.s.max_ctx && (ctx + kPage - 1) / kPage <= a.s.max_pages;
  return ok ? n : -1;
}

__global__ void __launch_bounds__(1024) k_evict_mark(const MoveArgs a) {
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = (int)cluster.block_rank() * 1024 + threadIdx.x, step = (int)cluster.num_blocks() * 1024;
  pdl_wait();
  pdl_trigger();
  for (int i = tid; i < 3 * a.words; i += step) a.read[i] = 0u;  // the three bitmaps are one run
  __threadfence();
  cluster.sync();
  const int64_t from = a.in_place ? (int64_t)a.s.batch * a.s.max_pages : 0;
  const int64_t all = from + (int64_t)a.s.batch * a.new_max_pages;
  for (int64_t i = tid; i < all; i += step) {
    if (i < from) {
      const int b = (int)(i / a.s.max_pages), p = (int)(i % a.s.max_pages);
      const int ctx = __ldg(a.s.ctx_len + b);
      if (ctx <= a.s.max_ctx && p * kPage < ctx) {
        const int page = __ldg(a.s.page_table + i);
        if (page >= 0 && page < a.new_pages) atomicOr(a.read + (page >> 5), 1u << (page & 31));
      }
    } else {
      const int64_t j = i - from;
      const int b = (int)(j / a.new_max_pages), p = (int)(j % a.new_max_pages);
      if (p * kPage < rows_to_move(a, b)) {
        const int page = __ldg(a.new_table + j);
        if (page >= 0 && page < a.new_pages && (atomicOr(a.written + (page >> 5), 1u << (page & 31)) >> (page & 31) & 1u))
          atomicOr(a.twice + (page >> 5), 1u << (page & 31));
      }
    }
  }
}

// Rows of V vectors: element i of the block is vector i % nv of its row i / nv.
template <class V>
struct RowsOf {
  const uint8_t* src;
  uint8_t* dst;
  int row_bytes, total;
  RowDivisor by;
  __device__ __forceinline__ bool load(int i, const int* rows, V* v) const {
    if (i >= total) return false;
    const RowColumn at = row_of((uint32_t)i, by);
    const int row = rows[at.row];
    if (row < 0) return false;
    *v = __ldcs(reinterpret_cast<const V*>(src + (int64_t)row * row_bytes) + (int)at.column);  // read once, as it is written
    return true;
  }
  __device__ __forceinline__ void store(int i, const V& v) const { __stcs(reinterpret_cast<V*>(dst) + i, v); }
};

// A batch of loads is issued before its stores.
constexpr int kMoveBatch = 6;
template <class V>
__device__ __forceinline__ void move_rows(const RowsOf<V>& m, const int* rows) {
  for (int i0 = threadIdx.x; i0 < m.total; i0 += kMoveBatch * kMoveThreads) {
    V v[kMoveBatch];
    bool in[kMoveBatch];
#pragma unroll
    for (int u = 0; u < kMoveBatch; ++u) in[u] = m.load(i0 + u * kMoveThreads, rows, &v[u]);
#pragma unroll
    for (int u = 0; u < kMoveBatch; ++u)
      if (in[u]) m.store(i0 + u * kMoveThreads, v[u]);
  }
}

template <class V>
__device__ __forceinline__ void move_pool(const MoveArgs& a, int k, int64_t first_row, const int* rows, int n) {
  const int nv = a.row_bytes[k] / (int)sizeof(V);
  move_rows(RowsOf<V>{a.src[k], a.dst[k] + first_row * a.row_bytes[k], a.row_bytes[k], n * nv,
                      RowDivisor{(uint32_t)nv, a.by[k].magic, a.by[k].add}}, rows);
}

// One block: kMoveRows rows of sequence b's new cache, from row i0.  They are
// resolved before the wait for k_evict_mark: what they depend on was complete when
// that kernel let this one start (it waits for its predecessor first).
__global__ void __launch_bounds__(kMoveThreads) k_evict_compact(const MoveArgs a) {
  __shared__ int rows[kMoveRows];
  __shared__ int page;
  const int chunks = (a.budget + kMoveRows - 1) / kMoveRows, b = blockIdx.x / chunks, tid = threadIdx.x;
  const int i0 = (int)(blockIdx.x % chunks) * kMoveRows, p = i0 / kPage;
  const int kept = rows_to_move(a, b);
  const int n = min(kMoveRows, kept - i0);
  int s = -1, row = -1;
  if (tid < n) {
    s = __ldg(a.keep + (int64_t)b * a.budget + i0 + tid);
    if (s >= 0 && s < __ldg(a.s.ctx_len + b))
      row = (int)phys_row(a.s.page_table, a.s.max_pages, a.s.num_phys_pages, b, s, a.err);
    else
      raise_error(a.err, kErrBadIndex);
    rows[tid] = row;
  }
  int d = -1;
  if (tid == 0 && n > 0 && p < a.new_max_pages) d = __ldg(a.new_table + (int64_t)b * a.new_max_pages + p);
  pdl_wait();
  pdl_trigger();
  if (kept < 0 && i0 == 0 && tid == 0) raise_error(a.err, kErrBadIndex);
  if (n <= 0) return;
  if (tid == 0) {
    bool ok = d >= 0 && d < a.new_pages;
    if (ok) {
      const uint32_t bit = 1u << (d & 31);
      ok = !((__ldcg(a.read + (d >> 5)) | __ldcg(a.twice + (d >> 5))) & bit);
    }
    if (!ok) raise_error(a.err, kErrBadIndex);
    page = ok ? d : -1;
  }
  __syncthreads();
  if (page < 0) return;
  if (a.mass && row >= 0)
    a.new_mass[(int64_t)b * a.new_ld + i0 + tid] = __ldg(a.mass + (int64_t)b * a.ld + s);
  const int64_t first_row = (int64_t)page * kPage + i0 % kPage;
  for (int k = 0; k < a.npools; ++k) {
    if (a.vec[k] == 16)
      move_pool<uint4>(a, k, first_row, rows, n);
    else if (a.vec[k] == 8)
      move_pool<uint2>(a, k, first_row, rows, n);
    else
      move_pool<uint32_t>(a, k, first_row, rows, n);
  }
}

template <class... KArgs, class... Args>
cudaError_t launch_cluster(const char* name, void (*kernel)(KArgs...), int grid, int cluster, int threads, size_t smem,
                           cudaStream_t st, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
  if (e == cudaSuccess) timer_mark(name, st);
  return e == cudaSuccess ? counted(cudaGetLastError()) : e;
}

template <int kSelThreads>
cudaError_t launch_select(const SelectArgs& a, int B, int C, int64_t slots, cudaStream_t st) {
  if (slots > kSlotsMax)
    return launch_cluster("evict_select", k_evict_select<false, kSelThreads>, B * C, C, kSelThreads, 0, st, a);
  static thread_local int attr_dev = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (attr_dev != dev) {
    cudaError_t e = cudaFuncSetAttribute(k_evict_select<true, kSelThreads>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kSlotsMax * 4);
    if (e != cudaSuccess) return e;
    attr_dev = dev;
  }
  return launch_cluster("evict_select", k_evict_select<true, kSelThreads>, B * C, C, kSelThreads, (size_t)slots * 4, st, a);
}

}  // namespace

cudaError_t launch_evict_select(const int32_t* ctx_len, int B, int max_ctx, const int64_t* mass, int64_t ld, int budget,
                                int recent, int sink, int32_t* keep, int32_t* keep_len, uint32_t* err,
                                cudaStream_t st) {
  const SelectArgs a{ctx_len, mass, ld, max_ctx, budget, recent, sink, keep, keep_len, err};
  // A cluster's size: about 1024 positions per CTA (one sequence of 1000: 8.2 us alone,
  // 8.7 with two CTAs; 3001: 12.6 alone, 9.9 with four; 32,768: 56 and 15 with
  // eight), as far as all CTAs find an SM of their own (64 x 3001: 12.4 us with two, 29.6
  // with eight; 32 x 32,768: 24.4 with four, 44 with eight), and no smaller than
  // keeps the keys in shared memory.  512 threads while each takes at most four keys or
  // shares its SM (cheaper barriers; 3001 by four: 9.9 for 10.4 us), else 1024
  // (32,768 by eight: 15.0 for 16.6).
  auto slots = [&](int C) { return (((int64_t)max_ctx + C - 1) / C + 3) & ~(int64_t)3; };
  int C = 1;
  while (C < kCluster && slots(C) > 1024) C *= 2;
  while (C > 1 && (int64_t)B * C > 148) C /= 2;
  while (C < kCluster && slots(C) > kSlotsMax) C *= 2;
  const bool few = slots(C) <= 4 * 512 || (int64_t)B * C > 148;
  return few ? launch_select<512>(a, B, C, slots(C), st) : launch_select<1024>(a, B, C, slots(C), st);
}

size_t evict_bitmap_bytes(int pages) { return (size_t)3 * (((size_t)pages + 31) / 32) * 4; }

cudaError_t launch_evict_compact(const SeqsDev& s, const EvictMove& m, void* bitmaps, uint32_t* err, cudaStream_t st) {
  MoveArgs a{};
  a.s = s;
  a.keep = m.keep;
  a.keep_len = m.keep_len;
  a.budget = m.budget;
  a.new_table = m.new_table;
  a.new_max_pages = m.new_max_pages;
  a.new_pages = m.new_pages;
  a.npools = m.npools;
  for (int k = 0; k < m.npools; ++k) {
    const dsa_pool_t& p = m.pools[k];
    a.src[k] = static_cast<const uint8_t*>(p.src);
    a.dst[k] = static_cast<uint8_t*>(p.dst);
    a.row_bytes[k] = p.row_bytes;
    a.vec[k] = p.row_bytes % 16 == 0 ? 16 : (p.row_bytes % 8 == 0 ? 8 : 4);
    a.by[k] = row_divisor((uint32_t)(p.row_bytes / a.vec[k]));
    a.in_place = a.in_place || p.src == p.dst;
  }
  a.mass = m.mass;
  a.new_mass = m.new_mass;
  a.ld = m.ld;
  a.new_ld = m.new_ld;
  a.words = (m.new_pages + 31) / 32;
  a.read = static_cast<uint32_t*>(bitmaps);
  a.written = a.read + a.words;
  a.twice = a.written + a.words;
  a.err = err;
  cudaError_t e = launch_cluster("evict_mark", k_evict_mark, kCluster, kCluster, 1024, 0, st, a);
  if (e != cudaSuccess) return e;
  const int64_t grid = ((int64_t)m.budget + kMoveRows - 1) / kMoveRows * s.batch;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  e = launch_pdl("evict_compact", k_evict_compact, dim3((unsigned)grid), dim3(kMoveThreads), 0, st, a);
  if (e != cudaSuccess) return e;
  return counted(cudaGetLastError());
}

}  // namespace dsa
