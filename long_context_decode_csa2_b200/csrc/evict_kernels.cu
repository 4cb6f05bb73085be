// Eviction from a cache by accumulated attention weight.
//
// Of the L entries of a sequence n = min(keep, L) stay: the first `first`,
// the last `last` (the recent ones), and of the others the best by (weight
// descending, position ascending).  The kept entries keep their order and
// move to the destination's positions 0 .. n-1, so a page pool gets its
// pages back; the window, visibility by prefix and appends go on as before.
//
// k_evict_select finds the kept positions, a cluster of C CTAs per sequence.
// Each CTA owns a run of positions and each of its warps a part of the run,
// whose rank keys it holds in shared memory as far as there is room (the rest
// is read again, from L2 as a rule).  Most entries of a long cache were never
// selected and stand at exactly 0, so the first pass only counts the entries
// above 0 and at 0: where that puts the threshold at 0 it is known, and so
// are every warp's counts above and at it.  Otherwise the cluster counts the
// keys of the threshold's sign by digits of 11, 10 and 10 bits and adds the
// histograms through distributed shared memory; once the threshold's bin
// holds at most 1024 keys, every CTA collects them and the one sought is
// found by counting.  Then each warp writes its kept positions in order.
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
constexpr int kStep = 128;                    // positions of a warp's step, 4 per lane
constexpr int kBatch = 4;                     // steps whose loads are in flight together
constexpr int kBins = 2048;
constexpr int kList = kEThreads;              // keys of the threshold's bin that are ranked one per thread
constexpr int kMaxCluster = 16;
constexpr int kRunKeys = 8192;                // positions per CTA that are worth a CTA
constexpr uint32_t kZeroKey = 0x80000000u;    // rank key of an entry that was never selected

struct __align__(16) SelSmem {
  uint32_t hist[kBins];       // this CTA's counts of the current digit
  uint32_t total[kBins];      // the cluster's
  uint32_t list[kList];       // this CTA's keys in the threshold's bin
  uint32_t all[kList];        // the cluster's
  uint32_t scan[kEWarps];
  uint32_t listed, gathered;
  uint32_t bin, above, thr, take;
  uint32_t warp_gt[kEWarps], warp_eq[kEWarps];  // every warp's keys above the threshold (first: 0) and at it
  uint32_t gt[2][kMaxCluster], eq[2][kMaxCluster];  // every CTA's: above and at 0, above and at the threshold
};

static_assert(sizeof(SelSmem) % 16 == 0, "the keys behind it are read as 16-byte words");

// What stays of sequence b.
struct Plan {
  int64_t len;
  int n, first, last, need;   // need: how many of the entries between first and last stay
};

__device__ __forceinline__ Plan make_plan(const EvictArgs& a, int b, uint32_t* status) {
  // (the loads first, so that they are in flight together)
  const int64_t keep = a.keep[b];
  const int64_t dst_off = a.dst_pages ? 0 : a.dst_row_off[b];
  Plan p;
  p.len = seg_len_checked(a.src, b, status);
  int64_t n = max(int64_t(0), min(keep, p.len));
  if (n > a.max_keep) {
    set_status(status, CSA2_DEV_LENGTH);
    n = a.max_keep;
  }
  const bool fits = a.dst_pages ? n <= (int64_t(a.dst_max_pages) << a.dst_shift)
                                : dst_off >= 0 && (dst_off & 7) == 0 && dst_off + n <= a.dst_rows;
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

// Rank keys of positions p .. p+3 (p a multiple of 4) of sequence b; 0 where a
// position does not compete (outside [m0, m1)).  Four positions never cross a
// page or the end of the accumulators, whose rows come in groups of 8.
__device__ __forceinline__ float4 load_acc(const EvictArgs& a, int b, int p, int m0, int m1, bool vec) {
  if (p + 4 <= m0 || p >= m1) return make_float4(0.f, 0.f, 0.f, 0.f);
  const float* src = a.acc_src + seg_row(a.src, b, p, a.status);
  if (vec) return __ldg(reinterpret_cast<const float4*>(src));
  return make_float4(__ldg(src), __ldg(src + 1), __ldg(src + 2), __ldg(src + 3));
}
__device__ __forceinline__ uint4 keys4(float4 f, int p, int m0, int m1) {
  uint4 k = make_uint4(rank_key(f.x), rank_key(f.y), rank_key(f.z), rank_key(f.w));
  if (p < m0 || p + 4 > m1) {
    if (p < m0 || p >= m1) k.x = 0;
    if (p + 1 < m0 || p + 1 >= m1) k.y = 0;
    if (p + 2 < m0 || p + 2 >= m1) k.z = 0;
    if (p + 3 < m0 || p + 3 >= m1) k.w = 0;
  }
  return k;
}

__global__ void __launch_bounds__(kEThreads) k_evict_select(EvictArgs a, int warp_cap) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  SelSmem& sm = *reinterpret_cast<SelSmem*>(smem_raw);
  cg::cluster_group cl = cg::this_cluster();
  const int C = int(cl.num_blocks()), rank = int(cl.block_rank());
  const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t* mine = reinterpret_cast<uint32_t*>(smem_raw + sizeof(SelSmem)) + warp * warp_cap;  // this warp's keys
  const bool vec = (reinterpret_cast<uintptr_t>(a.acc_src) & 15) == 0;
  launch_dependents();
  for (int i = tid; i < kBins; i += kEThreads) sm.hist[i] = 0;
  if (tid == 0) sm.listed = sm.gathered = 0;
  grid_wait();
  const Plan p = make_plan(a, b, rank == 0 && tid == 0 ? a.status : nullptr);
  int32_t* kept = a.kept + int64_t(b) * a.max_keep;
  for (int j = p.n + rank * kEThreads + tid; j < a.max_keep; j += C * kEThreads) kept[j] = -1;
  const int len = int(p.len), m0 = p.first, m1 = len - p.last;  // entries m0 .. m1-1 compete
  if (p.need == 0 || p.need == m1 - m0) {
    // only the protected entries stay, or all of them
    for (int j = rank * kEThreads + tid; j < p.n; j += C * kEThreads)
      kept[j] = p.need > 0 || j < p.first ? j : m1 + (j - p.first);
    cl.sync();  // every CTA has read the length (seq_len_out may be seq_len itself)
    if (rank == 0 && tid == 0) a.seq_len_out[b] = p.n;
    return;
  }
  // this warp's part of this CTA's run, in whole steps
  const int steps = (len + kStep - 1) / kStep;
  const int s0 = int(int64_t(steps) * rank / C), s1 = int(int64_t(steps) * (rank + 1) / C);
  const int w0 = (s0 + int(int64_t(s1 - s0) * warp / kEWarps)) * kStep;
  const int w1 = min(len, (s0 + int(int64_t(s1 - s0) * (warp + 1) / kEWarps)) * kStep);
  // ---- the keys, and how many lie above 0 and at 0 ----
  {
    uint32_t pos = 0, zer = 0;
    for (int q0 = w0; q0 < w1; q0 += kBatch * kStep) {
      float4 f[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int q = q0 + i * kStep + 4 * lane;
        f[i] = q < w1 ? load_acc(a, b, q, m0, m1, vec) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int q = q0 + i * kStep + 4 * lane;
        if (q < w1) {
          const uint4 k = keys4(f[i], q, m0, m1);
          if (q - w0 < warp_cap) *reinterpret_cast<uint4*>(mine + (q - w0)) = k;
          pos += uint32_t(k.x > kZeroKey) + uint32_t(k.y > kZeroKey) + uint32_t(k.z > kZeroKey) +
                 uint32_t(k.w > kZeroKey);
          zer += uint32_t(k.x == kZeroKey) + uint32_t(k.y == kZeroKey) + uint32_t(k.z == kZeroKey) +
                 uint32_t(k.w == kZeroKey);
        }
      }
    }
    pos = __reduce_add_sync(0xffffffffu, pos);
    zer = __reduce_add_sync(0xffffffffu, zer);
    if (lane == 0) {
      sm.warp_gt[warp] = pos;
      sm.warp_eq[warp] = zer;
    }
  }
  // every later pass over this warp's keys, the whole warp at a time:
  // fn(this lane's first position, its four keys); a key 0 does not compete
  auto each = [&](auto&& fn) {
    const int wc = min(w1, w0 + warp_cap);
    for (int q0 = w0; q0 < wc; q0 += kStep) {
      const int q = q0 + 4 * lane;
      fn(q, q < wc ? *reinterpret_cast<const uint4*>(mine + (q - w0)) : make_uint4(0, 0, 0, 0));
    }
    for (int q0 = w0 + warp_cap; q0 < w1; q0 += kBatch * kStep) {
      float4 f[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int q = q0 + i * kStep + 4 * lane;
        f[i] = q < w1 ? load_acc(a, b, q, m0, m1, vec) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int q = q0 + i * kStep + 4 * lane;
        if (q0 + i * kStep < w1) fn(q, q < w1 ? keys4(f[i], q, m0, m1) : make_uint4(0, 0, 0, 0));
      }
    }
  };
  // Sums sm.warp_gt / warp_eq over the cluster; slot 0: above and at 0, slot
  // 1: above and at the threshold.
  auto share = [&](int slot) {
    __syncthreads();
    if (warp == 0) {
      const uint32_t g = __reduce_add_sync(0xffffffffu, sm.warp_gt[lane]);
      const uint32_t e = __reduce_add_sync(0xffffffffu, sm.warp_eq[lane]);
      if (lane < C) {
        cl.map_shared_rank(&sm.gt[slot][0], lane)[rank] = g;
        cl.map_shared_rank(&sm.eq[slot][0], lane)[rank] = e;
      }
    }
    cl.sync();
  };
  share(0);
  int slot = 0;
  uint32_t left = uint32_t(p.need), thr = kZeroKey;
  {
    const uint32_t P = __reduce_add_sync(0xffffffffu, lane < C ? sm.gt[0][lane] : 0u);
    const uint32_t Z = __reduce_add_sync(0xffffffffu, lane < C ? sm.eq[0][lane] : 0u);
    if (left > P && left <= P + Z) {
      left -= P;  // the threshold is 0: so many of the zeros stay
    } else {
      // ---- the threshold's key, digit by digit among the keys of its sign ----
      slot = 1;
      const bool neg = left > P;
      if (neg) left -= P + Z;
      thr = neg ? 0u : kZeroKey;
      uint32_t mask = 0x80000000u;  // the bits of the threshold that are known
      auto in_bin = [&](uint32_t k) { return (k & mask) == thr && k != kZeroKey && k != 0u; };
      for (int digit = 0; digit < 3; ++digit) {
        const int shift = digit == 0 ? 20 : digit == 1 ? 10 : 0;
        const uint32_t width = digit == 0 ? 2047u : 1023u;
        each([&](int, uint4 k) {
          if (in_bin(k.x)) atomicAdd(&sm.hist[(k.x >> shift) & width], 1u);
          if (in_bin(k.y)) atomicAdd(&sm.hist[(k.y >> shift) & width], 1u);
          if (in_bin(k.z)) atomicAdd(&sm.hist[(k.z >> shift) & width], 1u);
          if (in_bin(k.w)) atomicAdd(&sm.hist[(k.w >> shift) & width], 1u);
        });
        // CTA r adds its share of the bins over the cluster and hands the sums to all
        cl.sync();
        const int per = (kBins + C - 1) / C;
        for (int i = tid; i < per && rank * per + i < kBins; i += kEThreads) {
          uint32_t v = 0;
#pragma unroll 4
          for (int c = 0; c < C; ++c) v += cl.map_shared_rank(sm.hist, c)[rank * per + i];
#pragma unroll 4
          for (int c = 0; c < C; ++c) cl.map_shared_rank(sm.total, c)[rank * per + i] = v;
        }
        cl.sync();
        // the bin that holds the left-th largest key: thread t owns bins 2047 - 2t and 2046 - 2t
        const uint32_t v0 = sm.total[kBins - 1 - 2 * tid], v1 = sm.total[kBins - 2 - 2 * tid];
        const uint32_t incl = warp_incl(v0 + v1, lane);
        if (lane == 31) sm.scan[warp] = incl;
        for (int i = tid; i < kBins; i += kEThreads) sm.hist[i] = 0;
        __syncthreads();
        const uint32_t part = warp_incl(sm.scan[lane], lane);
        uint32_t before = __shfl_sync(0xffffffffu, part, (warp + 31) & 31);
        before = (warp ? before : 0u) + incl - v0 - v1;
        if (before < left && before + v0 + v1 >= left) {
          const bool second = before + v0 < left;
          sm.bin = uint32_t(kBins - 1 - 2 * tid - (second ? 1 : 0));
          sm.above = before + (second ? v0 : 0u);
        }
        __syncthreads();
        left -= sm.above;
        thr |= sm.bin << shift;
        mask |= width << shift;
        if (digit == 2) break;
        const uint32_t inbin = sm.total[sm.bin];
        if (inbin <= uint32_t(kList)) {
          // few enough: every CTA gathers them and ranks one per thread
          each([&](int, uint4 k) {
            if (in_bin(k.x)) sm.list[atomicAdd(&sm.listed, 1u)] = k.x;
            if (in_bin(k.y)) sm.list[atomicAdd(&sm.listed, 1u)] = k.y;
            if (in_bin(k.z)) sm.list[atomicAdd(&sm.listed, 1u)] = k.z;
            if (in_bin(k.w)) sm.list[atomicAdd(&sm.listed, 1u)] = k.w;
          });
          cl.sync();
          const int group = kEThreads / C, src = tid / group;
          if (src < C) {
            const uint32_t n = *cl.map_shared_rank(&sm.listed, src);
            const uint32_t* from = cl.map_shared_rank(sm.list, src);
            for (uint32_t i = tid % group; i < n; i += group) sm.all[atomicAdd(&sm.gathered, 1u)] = from[i];
          }
          __syncthreads();
          if (tid < int(inbin)) {
            const uint32_t x = sm.all[tid];
            uint32_t gt = 0, eq = 0;
            for (uint32_t i = 0; i < inbin; ++i) {
              const uint32_t y = sm.all[i];
              gt += y > x;
              eq += y == x;
            }
            if (gt < left && gt + eq >= left) {  // (equal keys write the same values)
              sm.thr = x;
              sm.take = left - gt;
            }
          }
          __syncthreads();
          thr = sm.thr;
          left = sm.take;
          break;
        }
      }
      // ---- keys above and at the threshold ----
      uint32_t gt = 0, eq = 0;
      each([&](int, uint4 k) {
        gt += uint32_t(k.x > thr) + uint32_t(k.y > thr) + uint32_t(k.z > thr) + uint32_t(k.w > thr);
        eq += uint32_t(k.x == thr) + uint32_t(k.y == thr) + uint32_t(k.z == thr) + uint32_t(k.w == thr);
      });
      gt = __reduce_add_sync(0xffffffffu, gt);
      eq = __reduce_add_sync(0xffffffffu, eq);
      if (lane == 0) {
        sm.warp_gt[warp] = gt;
        sm.warp_eq[warp] = eq;
      }
      share(1);
    }
  }
  // (that barrier followed the last access to another CTA's memory, and every
  // CTA's read of the length: seq_len_out may be seq_len itself)
  if (rank == 0 && tid == 0) a.seq_len_out[b] = p.n;
  const uint32_t take_eq = left;  // of the keys equal to the threshold, how many stay
  // ---- the ordered list: what precedes this warp's part, then 32 positions at a time ----
  uint32_t ng = __reduce_add_sync(0xffffffffu, (lane < rank ? sm.gt[slot][lane] : 0u) +
                                                   (lane < warp ? sm.warp_gt[lane] : 0u));
  uint32_t ne = __reduce_add_sync(0xffffffffu, (lane < rank ? sm.eq[slot][lane] : 0u) +
                                                   (lane < warp ? sm.warp_eq[lane] : 0u));
  uint32_t at = ng + uint32_t(min(w0, m0)) + uint32_t(max(0, w0 - m1)) + min(ne, take_eq);  // kept before w0
  const uint32_t below = (1u << lane) - 1u;
  auto emit = [&](int q0, uint32_t k) {
    const int q = q0 + lane;
    bool stays = k > thr;
    if (q0 < m0 || q0 + 32 > m1) stays = stays || q < m0 || (q >= m1 && q < len);
    if (ne < take_eq) {
      const uint32_t same = __ballot_sync(0xffffffffu, k == thr);
      stays = stays || (k == thr && ne + __popc(same & below) < take_eq);
      ne += __popc(same);
    }
    const uint32_t all = __ballot_sync(0xffffffffu, stays);
    if (stays) kept[at + __popc(all & below)] = q;
    at += __popc(all);
  };
  const int wc = min(w1, w0 + warp_cap);
#pragma unroll 4
  for (int q0 = w0; q0 < wc; q0 += 32) emit(q0, q0 + lane < wc ? mine[q0 - w0 + lane] : 0u);
  for (int q0 = w0 + warp_cap; q0 < w1; q0 += 8 * 32) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int q = q0 + 32 * i + lane;
      f[i] = q >= m0 && q < min(w1, m1) ? __ldg(a.acc_src + seg_row(a.src, b, q, a.status)) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int q = q0 + 32 * i + lane;
      if (q0 + 32 * i < w1) emit(q0 + 32 * i, q >= m0 && q < min(w1, m1) ? rank_key(f[i]) : 0u);
    }
  }
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
  // CTAs per sequence: one for every 8192 positions while the clusters of all
  // sequences run at once.  The CTAs of a cluster share a GPC, so a B200's 148
  // SMs hold fewer clusters than 148 / C: kActive[C], as its occupancy query
  // gives it (another layout of the GPCs costs a second wave, nothing else).
  constexpr int kActive[kMaxCluster + 1] = {0, 148, 74, 45, 33, 26, 22, 15, 15, 15, 11, 7, 7, 7, 7, 7, 7};
  const int64_t want = (a.src.max_len + kRunKeys - 1) / kRunKeys;
  int C = int(std::max<int64_t>(1, std::min<int64_t>(kMaxCluster, want)));
  while (C > 1 && kActive[C] < a.B) --C;
  // keys of a warp that stay in shared memory: its part of the run, as far as there is room
  const int64_t steps = (a.src.max_len + kStep - 1) / kStep;
  const int64_t part = ((steps + C - 1) / C + kEWarps - 1) / kEWarps;
  const int64_t fit = (int64_t(224) * 1024 - int64_t(sizeof(SelSmem))) / (4 * kStep * kEWarps);
  const int warp_cap = int(std::min(part, fit)) * kStep;
  const size_t smem = sizeof(SelSmem) + size_t(warp_cap) * 4 * kEWarps;
  cudaFuncSetAttribute(k_evict_select, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  cudaFuncSetAttribute(k_evict_select, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  launch_k_cluster(k_evict_select, dim3(C, a.B), dim3(kEThreads), smem, st, C, a, warp_cap);
  const csa2_status rc = check_launch("csa2_cache_evict");
  if (rc != CSA2_OK) return rc;
  launch_k(k_evict_move, dim3(unsigned((a.max_keep + kMRows - 1) / kMRows), a.B), dim3(kMThreads), 0, st, a);
  return check_launch("csa2_cache_evict");
}

}  // namespace csa2
