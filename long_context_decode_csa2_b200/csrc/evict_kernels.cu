// Eviction from a cache by accumulated attention weight.
//
// Of the L entries of a sequence n = min(keep, L) stay: the first `first`,
// the last `last` (the recent ones), and of the others the best by (weight
// descending, position ascending).  The kept entries keep their order and
// move to the destination's positions 0 .. n-1, so a page pool gets its
// pages back; the window, visibility by prefix and appends go on as before.
//
// k_evict_select finds the kept positions, a cluster of C CTAs per sequence.
// Each CTA owns a run of positions, holds their rank keys in shared memory
// as far as it has room (the rest is read again, from L2 as a rule) and
// counts them by digits of 11, 11 and 10 bits; the cluster adds the
// histograms through distributed shared memory, and after three digits the
// key of the last kept entry and how many of its equals stay are known.  A
// last ordered pass writes the positions.  Most entries of a long cache were
// never selected and stand at exactly 0: a thread counts zeros in a register
// and leaves the histogram's atomics to the others.
//
// k_evict_move copies the rows: a CTA takes a run of destination rows, so its
// writes are contiguous and every CTA moves the same amount whatever the
// selection.  It is bound by HBM (a row is 272 + 68 + 4 bytes read and
// written).
#include <cooperative_groups.h>

#include <algorithm>

#include "device_common.cuh"
#include "sm100.cuh"

namespace cg = cooperative_groups;

namespace csa2 {

namespace {

constexpr int kEThreads = 1024;
constexpr int kEWarps = kEThreads / 32;
constexpr int kBins = 2048;
constexpr int kPer = 4;                       // consecutive positions of a thread in the ordered pass
constexpr int kTileE = kEThreads * kPer;
constexpr int kMaxCluster = 16;
constexpr uint32_t kZeroKey = 0x80000000u;    // rank key of an entry that was never selected

struct SelSmem {
  uint32_t hist[kBins];       // this CTA's counts of the current digit
  uint32_t total[kBins];      // the cluster's
  uint32_t scan[kEWarps];
  uint32_t bin, above;        // the threshold's bin, and how many keys lie in the bins above it
  uint32_t zeros;
  uint32_t counts[2];         // this CTA's keys above the threshold, and equal to it
};

// What stays of sequence b.
struct Plan {
  int64_t len;
  int n, first, last, need;   // need: how many of the entries between first and last stay
};

__device__ __forceinline__ Plan make_plan(const EvictArgs& a, int b, uint32_t* status) {
  Plan p;
  p.len = seg_len_checked(a.src, b, status);
  int64_t n = a.keep[b];
  if (n < 0) n = 0;
  if (n > p.len) n = p.len;
  if (n > a.max_keep) {
    set_status(status, CSA2_DEV_LENGTH);
    n = a.max_keep;
  }
  bool fits;
  if (a.dst_pages) {
    fits = n <= (int64_t(a.dst_max_pages) << a.dst_shift);
  } else {
    const int64_t off = a.dst_row_off[b];
    fits = off >= 0 && (off & 7) == 0 && off + n <= a.dst_rows;
  }
  if (!fits) {
    set_status(status, CSA2_DEV_ROW_LAYOUT);
    n = 0;
  }
  p.n = int(n);
  p.last = int(min(int64_t(a.last), n));
  p.first = int(min(int64_t(a.first), n - p.last));
  p.need = p.n - p.first - p.last;
  return p;
}

__device__ __forceinline__ uint32_t warp_incl(uint32_t v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

__global__ void __launch_bounds__(kEThreads) k_evict_select(EvictArgs a, int cap) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  SelSmem& sm = *reinterpret_cast<SelSmem*>(smem_raw);
  uint32_t* skeys = reinterpret_cast<uint32_t*>(smem_raw + sizeof(SelSmem));
  cg::cluster_group cl = cg::this_cluster();
  const int C = int(cl.num_blocks()), rank = int(cl.block_rank());
  const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  launch_dependents();
  grid_wait();
  const Plan p = make_plan(a, b, rank == 0 && tid == 0 ? a.status : nullptr);
  int32_t* kept = a.kept + int64_t(b) * a.max_keep;
  for (int64_t j = p.n + rank * kEThreads + tid; j < a.max_keep; j += int64_t(C) * kEThreads) kept[j] = -1;
  // this CTA's run of positions (whole tiles, so that runs differ by a tile at most)
  const int64_t tiles = (p.len + kTileE - 1) / kTileE;
  const int64_t lo = min(p.len, tiles * rank / C * kTileE), hi = min(p.len, tiles * (rank + 1) / C * kTileE);
  const int64_t mid0 = p.first, mid1 = p.len - p.last;  // the entries that compete
  const bool choose = p.need > 0 && p.need < mid1 - mid0;
  auto key_of = [&](int64_t pos) { return rank_key(__ldg(a.acc_src + seg_row(a.src, b, pos, a.status))); };
  uint32_t thr = 0, above = 0;  // need == all of them: every key is at or above the threshold 0
  int64_t take_eq = 0;          // of the keys equal to the threshold, how many stay
  if (choose) {
    for (int64_t pos = lo + tid; pos < min(hi, lo + cap); pos += kEThreads) skeys[pos - lo] = key_of(pos);
    __syncthreads();
    auto key = [&](int64_t pos) { return pos - lo < cap ? skeys[pos - lo] : key_of(pos); };
    const int64_t m0 = max(lo, mid0), m1 = min(hi, mid1);
    int64_t left = p.need;
    uint32_t mask = 0;
    for (int digit = 0; digit < 3; ++digit) {
      const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0;
      const uint32_t width = digit == 2 ? 1023u : 2047u;
      for (int i = tid; i < kBins; i += kEThreads) sm.hist[i] = 0;
      if (tid == 0) sm.zeros = 0;
      __syncthreads();
      uint32_t zeros = 0;
      for (int64_t pos = m0 + tid; pos < m1; pos += kEThreads) {
        const uint32_t u = key(pos);
        if (u == kZeroKey) ++zeros;
        else if ((u & mask) == thr) atomicAdd(&sm.hist[(u >> shift) & width], 1u);
      }
      zeros = __reduce_add_sync(0xffffffffu, zeros);
      if (lane == 0 && zeros) atomicAdd(&sm.zeros, zeros);
      __syncthreads();
      if (tid == 0 && (kZeroKey & mask) == thr) sm.hist[(kZeroKey >> shift) & width] += sm.zeros;
      cl.sync();
      // CTA r adds bins r * 2048 / C .. of every CTA and hands the sums to all
      const int per = kBins / C;
      for (int i = tid; i < per; i += kEThreads) {
        uint32_t s = 0;
        for (int c = 0; c < C; ++c) s += cl.map_shared_rank(sm.hist, c)[rank * per + i];
        for (int c = 0; c < C; ++c) cl.map_shared_rank(sm.total, c)[rank * per + i] = s;
      }
      cl.sync();
      // the bin that holds the left-th largest key: thread t owns bins 2047 - 2t and 2046 - 2t
      const uint32_t v0 = sm.total[kBins - 1 - 2 * tid], v1 = sm.total[kBins - 2 - 2 * tid];
      const uint32_t incl = warp_incl(v0 + v1, lane);
      if (lane == 31) sm.scan[warp] = incl;
      __syncthreads();
      uint32_t before = 0;
      for (int w = 0; w < warp; ++w) before += sm.scan[w];
      before += incl - v0 - v1;
      if (int64_t(before) < left && int64_t(before) + v0 + v1 >= left) {
        const bool second = int64_t(before) + v0 < left;
        sm.bin = uint32_t(kBins - 1 - 2 * tid - (second ? 1 : 0));
        sm.above = before + (second ? v0 : 0);
      }
      __syncthreads();
      thr |= sm.bin << shift;
      mask |= width << shift;
      left -= sm.above;
    }
    take_eq = left;
    // this CTA's keys above and at the threshold
    uint32_t gt = 0, eq = 0;
    for (int64_t pos = m0 + tid; pos < m1; pos += kEThreads) {
      const uint32_t u = key(pos);
      gt += u > thr;
      eq += u == thr;
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (tid < 2) sm.counts[tid] = 0;
    __syncthreads();
    if (lane == 0) {
      atomicAdd(&sm.counts[0], gt);
      atomicAdd(&sm.counts[1], eq);
    }
    cl.sync();
  }
  // ---- the ordered list ----
  // What precedes this CTA's run: protected entries, keys above the threshold
  // and equals.
  int64_t pre_gt = 0, pre_eq = 0;
  if (choose) {
    for (int c = 0; c < rank; ++c) {
      const uint32_t* o = cl.map_shared_rank(sm.counts, c);
      pre_gt += o[0];
      pre_eq += o[1];
    }
    pre_gt += min(lo, mid0) + max(int64_t(0), lo - mid1);
  } else if (p.need > 0) {
    pre_gt = lo;  // everything stays
  } else {
    pre_gt = min(lo, mid0) + max(int64_t(0), lo - mid1);
  }
  for (int64_t t0 = lo; t0 < hi; t0 += kTileE) {
    const int64_t pos0 = t0 + tid * kPer;
    uint32_t flag[kPer], cnt = 0;  // 1 = stays, 1 << 16 = equal to the threshold
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int64_t pos = pos0 + j;
      uint32_t f = 0;
      if (pos < hi) {
        if (pos < mid0 || pos >= mid1) {
          f = 1;
        } else if (choose) {
          const uint32_t u = pos - lo < cap ? skeys[pos - lo] : key_of(pos);
          f = u > thr ? 1u : u == thr ? 1u << 16 : 0u;
        } else {
          f = p.need > 0 ? 1u : 0u;
        }
      }
      flag[j] = f;
      cnt += f;
    }
    const uint32_t incl = warp_incl(cnt, lane);
    __syncthreads();  // the last tile's scan is read
    if (lane == 31) sm.scan[warp] = incl;
    __syncthreads();
    uint32_t before = 0, tile = 0;
    for (int w = 0; w < kEWarps; ++w) {
      if (w < warp) before += sm.scan[w];
      tile += sm.scan[w];
    }
    before += incl - cnt;
    int64_t g = pre_gt + (before & 0xFFFFu), e = pre_eq + (before >> 16);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const bool eq = flag[j] == 1u << 16;
      if (flag[j] == 1u || (eq && e < take_eq)) kept[g + min(e, take_eq)] = int32_t(pos0 + j);
      g += flag[j] == 1u;
      e += eq;
    }
    pre_gt += tile & 0xFFFFu;
    pre_eq += tile >> 16;
  }
  // No CTA leaves while another reads its shared memory, and every CTA has
  // read the length (seq_len_out may be seq_len itself).
  cl.sync();
  if (rank == 0 && tid == 0) a.seq_len_out[b] = p.n;
}

constexpr int kMThreads = 256;
constexpr int kMRows = 64;  // destination rows of a CTA

// 16-byte copy of chunk i of the rows' `per` chunks each.
template <int kPerRow>
__device__ __forceinline__ void move_plane(const uint8_t* src, uint8_t* dst, const int64_t (&srow)[kMRows],
                                           const int64_t (&drow)[kMRows], int tid) {
  constexpr int kN = (kMRows * kPerRow + kMThreads - 1) / kMThreads;
  uint4 v[kN];
#pragma unroll
  for (int m = 0; m < kN; ++m) {
    const int i = tid + m * kMThreads;
    const int r = i / kPerRow;
    if (r < kMRows && drow[r] >= 0) v[m] = __ldg(reinterpret_cast<const uint4*>(src) + srow[r] * kPerRow + i % kPerRow);
  }
#pragma unroll
  for (int m = 0; m < kN; ++m) {
    const int i = tid + m * kMThreads;
    const int r = i / kPerRow;
    if (r < kMRows && drow[r] >= 0) reinterpret_cast<uint4*>(dst)[drow[r] * kPerRow + i % kPerRow] = v[m];
  }
}

__global__ void __launch_bounds__(kMThreads) k_evict_move(EvictArgs a) {
  __shared__ int64_t srow[kMRows], drow[kMRows];
  const int b = blockIdx.y, tid = threadIdx.x;
  const int64_t r0 = int64_t(blockIdx.x) * kMRows;
  launch_dependents();
  grid_wait();
  if (tid < kMRows) {
    const int64_t r = r0 + tid;
    const int pos = r < a.max_keep ? __ldg(a.kept + int64_t(b) * a.max_keep + r) : -1;
    int64_t s = -1, d = -1;
    if (pos >= 0) {
      s = seg_row(a.src, b, pos, a.status);
      if (a.dst_pages) {
        // a row whose destination page lies outside the cache is not written
        const int64_t pg = __ldg(a.dst_pages + int64_t(b) * a.dst_max_pages + (r >> a.dst_shift));
        if (pg < 0 || ((pg + 1) << a.dst_shift) > a.dst_rows) set_status(a.status, CSA2_DEV_ROW_LAYOUT);
        else d = (pg << a.dst_shift) + (r & ((int64_t(1) << a.dst_shift) - 1));
      } else {
        d = a.dst_row_off[b] + r;
      }
    }
    srow[tid] = s;
    drow[tid] = d;
  }
  if (__syncthreads_and(tid >= kMRows || drow[tid] < 0)) return;
  move_plane<kMainCodeBytes / 16>(a.main_src.codes, a.main_dst.codes, srow, drow, tid);
  move_plane<kMainScaleBytes / 16>(a.main_src.scales, a.main_dst.scales, srow, drow, tid);
  if (a.idx_src.codes) {
    move_plane<kIdxCodeBytes / 16>(a.idx_src.codes, a.idx_dst.codes, srow, drow, tid);
    if (tid < kMRows && drow[tid] >= 0)
      reinterpret_cast<uint32_t*>(a.idx_dst.scales)[drow[tid]] =
          __ldg(reinterpret_cast<const uint32_t*>(a.idx_src.scales) + srow[tid]);
  }
  if (tid < kMRows && drow[tid] >= 0) a.acc_dst[drow[tid]] = __ldg(a.acc_src + srow[tid]);
}

}  // namespace

csa2_status launch_evict(const EvictArgs& a, cudaStream_t st) {
  // CTAs per sequence: a tile of positions each while all clusters fit on
  // the GPU at once
  int C = 1;
  while (C < kMaxCluster && 2 * C * int64_t(a.B) <= num_sms() && int64_t(C) * kTileE < a.src.max_len) C *= 2;
  const int64_t tiles = (a.src.max_len + kTileE - 1) / kTileE;
  const int64_t run = (tiles + C - 1) / C * kTileE;
  const size_t room = 200 * 1024 - sizeof(SelSmem);
  const int cap = int(std::min<int64_t>(run, int64_t(room / 4)));
  const size_t smem = sizeof(SelSmem) + size_t(cap) * 4;
  cudaFuncSetAttribute(k_evict_select, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  cudaFuncSetAttribute(k_evict_select, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  launch_k_cluster(k_evict_select, dim3(C, a.B), dim3(kEThreads), smem, st, C, a, cap);
  const csa2_status rc = check_launch("csa2_cache_evict");
  if (rc != CSA2_OK) return rc;
  if (a.max_keep > 0)
    launch_k(k_evict_move, dim3(unsigned((a.max_keep + kMRows - 1) / kMRows), a.B), dim3(kMThreads), 0, st, a);
  return check_launch("csa2_cache_evict");
}

}  // namespace csa2
