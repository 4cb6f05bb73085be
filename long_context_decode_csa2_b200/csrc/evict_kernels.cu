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
// whose weights it holds in shared memory as far as there is room (the rest
// is read again, from L2 as a rule).  Most entries of a long cache were never
// selected and stand at exactly 0, so the first pass only counts the entries
// above 0 and at 0: where that puts the threshold at 0 it is known, and so
// are every warp's counts above and at it.  Otherwise the cluster counts the
// entries of the threshold's sign by digits of 11, 10 and 10 bits and adds
// the histograms through distributed shared memory; once the threshold's bin
// holds at most 1024 entries, every CTA collects them and goes on alone.
// Then each warp writes its kept positions in order.  Bound by instructions
// (an entry is 4 bytes): the passes compare floats, and the ordered write
// scans the flags of 128 positions at once, four counts to a register.
//
// The Full layers of a step that select in one candidate pool know an entry by
// its position, so all of them keep the same ones: one selection, by the sum of
// the layers' weights (added as they are read), and a move per layer.
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
constexpr int kList = kEThreads;              // entries of the threshold's bin that every CTA finishes alone
constexpr int kMaxCluster = 16;
constexpr int kSelSmem = 226 * 1024;          // shared memory of a selection's CTA, at most
constexpr int kRunKeys = 8192;                // positions per CTA that are worth a CTA

struct __align__(16) SelSmem {
  uint32_t hist[kBins];       // this CTA's counts of the current digit
  uint32_t total[kBins];      // the cluster's
  uint32_t list[kList];       // this CTA's entries of the threshold's bin
  uint8_t from[kList];        // and the warps that have them
  uint32_t all[kList];        // the cluster's
  uint32_t scan[kEWarps];
  uint32_t listed, gathered;
  uint32_t bin, above;
  uint32_t warp_gt[kEWarps], warp_eq[kEWarps];  // every warp's entries above the threshold (first: 0) and at it
  uint32_t gt[2][kMaxCluster], eq[2][kMaxCluster];  // every CTA's: above and at 0, above and at the threshold
};

static_assert(sizeof(SelSmem) % 16 == 0, "the weights behind it are read as 16-byte words");

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
                                : dst_off >= 0 && (dst_off & 7) == 0 && dst_off <= a.dst_rows - n;
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

// Inclusive sum over the lanes up to this one (the shuffle's own predicate says
// whether there is a lane d below).
__device__ __forceinline__ uint32_t warp_incl(uint32_t v) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b32 o;\n\tshfl.sync.up.b32 o|p, %0, %1, 0, 0xffffffff;\n\t@p add.u32 %0, %0, o;\n\t}"
        : "+r"(v)
        : "r"(d));
  return v;
}

// What an entry is ranked by: its accumulator, or the sum of its accumulators
// in several layers (fp32, in their order; NaN in one of them makes it NaN).
struct OneLayer {
  __device__ __forceinline__ float4 add4(float4 f, int64_t, bool) const { return f; }
  __device__ __forceinline__ float add(float f, int64_t) const { return f; }
};
struct MoreLayers {
  int n;
  const float* acc[kMaxEvictLayers - 1];  // behind EvictArgs::acc_src
  __device__ __forceinline__ float4 add4(float4 f, int64_t row, bool vec) const {
    for (int l = 0; l < n; ++l) {
      const float* src = acc[l] + row;
      const float4 x = vec ? __ldg(reinterpret_cast<const float4*>(src))
                           : make_float4(__ldg(src), __ldg(src + 1), __ldg(src + 2), __ldg(src + 3));
      f.x += x.x, f.y += x.y, f.z += x.z, f.w += x.w;
    }
    return f;
  }
  __device__ __forceinline__ float add(float f, int64_t row) const {
    for (int l = 0; l < n; ++l) f += __ldg(acc[l] + row);
    return f;
  }
};

template <class L>
__global__ void __launch_bounds__(kEThreads) k_evict_select(EvictArgs a, L layers, int warp_cap, bool vec) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  SelSmem& sm = *reinterpret_cast<SelSmem*>(smem_raw);
  cg::cluster_group cl = cg::this_cluster();
  const int C = int(cl.num_blocks()), rank = int(cl.block_rank());
  const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float* mine = reinterpret_cast<float*>(smem_raw + sizeof(SelSmem)) + warp * warp_cap;  // this warp's weights
  launch_dependents();
  // The cluster's CTAs write into one another's shared memory, which needs all
  // of them running: each arrives here and waits before its first such access
  // (the first pass over the weights lies between).
  cl.barrier_arrive();
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
    cl.barrier_wait();
    cl.sync();  // every CTA has read the length (seq_len_out may be seq_len itself)
    if (rank == 0 && tid == 0) a.seq_len_out[b] = p.n;
    return;
  }
  // this warp's part of this CTA's run, in whole steps
  const int steps = (len + kStep - 1) / kStep;
  const int s0 = int(int64_t(steps) * rank / C), s1 = int(int64_t(steps) * (rank + 1) / C);
  const int w0 = (s0 + int(int64_t(s1 - s0) * warp / kEWarps)) * kStep;
  const int w1 = min(len, (s0 + int(int64_t(s1 - s0) * (warp + 1) / kEWarps)) * kStep);
  const int wc = min(w1, w0 + warp_cap);
  const float* base = a.src.pages ? nullptr : a.acc_src + a.src.row_off[b];
  // (a step never crosses a page)
  auto step_at = [&](int q0) { return base ? base + q0 : a.acc_src + seg_row(a.src, b, q0, a.status); };
  auto one = [&](const float* src) { return layers.add(__ldg(src), src - a.acc_src); };
  // The whole warp over its part, 4 consecutive positions per lane and step:
  // fn(position, four weights), from the accumulators on (kBatch steps' loads
  // in flight) or from shared memory as far as it goes.  Entries that do not
  // compete (protected ones, positions behind the end) come as NaN.
  // Accumulators come in groups of 8, so a lane's four lie inside them.
  auto mask = [&](int q0, float4 f) {
    if (q0 < m0 || q0 + kStep > m1) {
      const int q = q0 + 4 * lane;
      const float no = __uint_as_float(0x7FC00000u);
      if (q < m0 || q >= m1) f.x = no;
      if (q + 1 < m0 || q + 1 >= m1) f.y = no;
      if (q + 2 < m0 || q + 2 >= m1) f.z = no;
      if (q + 3 < m0 || q + 3 >= m1) f.w = no;
    }
    return f;
  };
  auto from_global = [&](int from, auto&& fn) {
    for (int q0 = from; q0 < w1; q0 += kBatch * kStep) {
      float4 f[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (q0 + i * kStep + 4 * lane < w1) {
          const float* src = step_at(q0 + i * kStep) + 4 * lane;
          f[i] = vec ? __ldg(reinterpret_cast<const float4*>(src))
                     : make_float4(__ldg(src), __ldg(src + 1), __ldg(src + 2), __ldg(src + 3));
          f[i] = layers.add4(f[i], src - a.acc_src, vec);
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (q0 + i * kStep < w1) fn(q0 + i * kStep, f[i]);
    }
  };
  auto each = [&](auto&& fn) {
#pragma unroll 2
    for (int q0 = w0; q0 < wc; q0 += kStep)
      fn(mask(q0, *reinterpret_cast<const float4*>(mine + (q0 - w0) + 4 * lane)));
    from_global(w0 + warp_cap, [&](int q0, float4 f) { fn(mask(q0, f)); });
  };
  // Every warp's counts (sm.warp_gt / warp_eq) summed over the CTA and handed
  // to the cluster; slot 0: above and at 0, slot 1: above and at the threshold.
  auto put = [&](uint32_t gt, uint32_t eq) {
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) {
      sm.warp_gt[warp] = gt;
      sm.warp_eq[warp] = eq;
    }
    __syncthreads();
  };
  auto share = [&](int slot) {
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
  uint32_t gt = 0, eq = 0;
  // ---- the weights, and how many lie above 0 and at 0 ----
  from_global(w0, [&](int q0, float4 f) {
    if (q0 < wc) *reinterpret_cast<float4*>(mine + (q0 - w0) + 4 * lane) = f;
    f = mask(q0, f);
    gt += uint32_t(f.x > 0.0f) + uint32_t(f.y > 0.0f) + uint32_t(f.z > 0.0f) + uint32_t(f.w > 0.0f);
    eq += uint32_t(f.x == 0.0f) + uint32_t(f.y == 0.0f) + uint32_t(f.z == 0.0f) + uint32_t(f.w == 0.0f);
  });
  put(gt, eq);
  cl.barrier_wait();
  share(0);
  int slot = 0;
  uint32_t left = uint32_t(p.need);
  float thr = 0.0f;  // the threshold (NaN: NaN entries are the least that stay)
  const uint32_t above0 = __reduce_add_sync(0xffffffffu, lane < C ? sm.gt[0][lane] : 0u);
  const uint32_t at0 = __reduce_add_sync(0xffffffffu, lane < C ? sm.eq[0][lane] : 0u);
  if (left > above0 && left <= above0 + at0) {
    left -= above0;  // the threshold is 0: so many of the zeros stay
  } else {
    // ---- the threshold, digit by digit among the entries of its sign ----
    slot = 1;
    const bool neg = left > above0;
    if (neg) left -= above0 + at0;
    uint32_t known = 0, mask_bits = 0;  // the threshold's rank, and which bits of it are known
    // The bin of `counts` that holds the left-th largest, among bins that
    // thread t owns (2047 - 2t and 2046 - 2t); zeroes the histogram.
    auto find = [&](const uint32_t* counts, int shift, uint32_t width) {
      const uint32_t v0 = counts[kBins - 1 - 2 * tid], v1 = counts[kBins - 2 - 2 * tid];
      const uint32_t incl = warp_incl(v0 + v1);
      if (lane == 31) sm.scan[warp] = incl;
      sm.hist[kBins - 1 - 2 * tid] = sm.hist[kBins - 2 - 2 * tid] = 0;
      __syncthreads();
      const uint32_t part = warp_incl(sm.scan[lane]);
      uint32_t prior = __shfl_sync(0xffffffffu, part, (warp + 31) & 31);
      prior = (warp ? prior : 0u) + incl - v0 - v1;
      if (prior < left && prior + v0 + v1 >= left) {
        const bool second = prior + v0 < left;
        sm.bin = uint32_t(kBins - 1 - 2 * tid - (second ? 1 : 0));
        sm.above = prior + (second ? v0 : 0u);
      }
      __syncthreads();
      left -= sm.above;
      known |= sm.bin << shift;
      mask_bits |= width << shift;
    };
    // fn(rank) for the entries of the threshold's sign.  Among the negative
    // ones, NaN entries rank lowest, and those that do not compete have to be
    // told from them.
    auto ranks = [&](auto&& fn) {
      if (!neg) {
        each([&](float4 f) {
          if (f.x > 0.0f) fn(__float_as_uint(f.x));
          if (f.y > 0.0f) fn(__float_as_uint(f.y));
          if (f.z > 0.0f) fn(__float_as_uint(f.z));
          if (f.w > 0.0f) fn(__float_as_uint(f.w));
        });
      } else {
        for (int q = w0 + lane; q < w1; q += 32) {
          const float y = q < wc ? mine[q - w0] : one(step_at(q / kStep * kStep) + q % kStep);
          if (q >= m0 && q < m1 && !(y >= 0.0f)) fn(rank_key(y));
        }
      }
    };
    auto shift_of = [](int digit) { return digit == 0 ? 20 : digit == 1 ? 10 : 0; };
    int digit = 0;
    bool alone = false;
    uint32_t n = 0;  // alone: entries of the bin
    for (; digit < 3 && !alone; ++digit) {
      const int shift = shift_of(digit);
      const uint32_t width = digit == 0 ? 2047u : 1023u;
      if (digit == 0) {
        ranks([&](uint32_t k) { atomicAdd(&sm.hist[k >> 20], 1u); });
      } else {
        ranks([&](uint32_t k) {
          if ((k & mask_bits) == known) atomicAdd(&sm.hist[(k >> shift) & width], 1u);
        });
      }
      // CTA r adds its share of the bins over the cluster and hands the sums to all
      cl.sync();
      const int per = (kBins + C - 1) / C;
      for (int i = tid; i < per && rank * per + i < kBins; i += kEThreads) {
        uint32_t v = 0;
#pragma unroll 8
        for (int c = 0; c < C; ++c) v += cl.map_shared_rank(sm.hist, c)[rank * per + i];
#pragma unroll 8
        for (int c = 0; c < C; ++c) cl.map_shared_rank(sm.total, c)[rank * per + i] = v;
      }
      cl.sync();
      find(sm.total, shift, width);
      n = sm.total[sm.bin];
      alone = digit < 2 && n <= uint32_t(kList);
    }
    if (alone) {
      // list the bin's entries, count those above the bin on the way
      gt = 0;
      ranks([&](uint32_t k) {
        const uint32_t high = k & mask_bits;
        gt += high > known;
        if (high == known) {
          const uint32_t at = atomicAdd(&sm.listed, 1u);
          sm.list[at] = k;
          sm.from[at] = uint8_t(warp);
        }
      });
      put(gt, 0);
      cl.sync();
      const int group = kEThreads / C, src = tid / group;
      if (src < C) {
        const uint32_t m = *cl.map_shared_rank(&sm.listed, src);
        const uint32_t* from = cl.map_shared_rank(sm.list, src);
        for (uint32_t i = tid % group; i < m; i += group) sm.all[atomicAdd(&sm.gathered, 1u)] = from[i];
      }
      __syncthreads();
      const uint32_t x = uint32_t(tid) < n ? sm.all[tid] : 0u;
      for (; digit < 3; ++digit) {
        const int shift = shift_of(digit);
        if (uint32_t(tid) < n && (x & mask_bits) == known) atomicAdd(&sm.hist[(x >> shift) & 1023u], 1u);
        __syncthreads();
        find(sm.hist, shift, 1023u);
      }
      // this CTA's listed entries above and at the threshold
      if (uint32_t(tid) < sm.listed) {
        const uint32_t k = sm.list[tid];
        if (k >= known) atomicAdd(k > known ? &sm.warp_gt[sm.from[tid]] : &sm.warp_eq[sm.from[tid]], 1u);
      }
    } else {
      gt = eq = 0;
      ranks([&](uint32_t k) {
        gt += k > known;
        eq += k == known;
      });
      put(gt, eq);
    }
    if (neg) {
      // the entries at or above 0 are above the threshold too
      uint32_t up = 0;
      each([&](float4 f) {
        up += uint32_t(f.x >= 0.0f) + uint32_t(f.y >= 0.0f) + uint32_t(f.z >= 0.0f) + uint32_t(f.w >= 0.0f);
      });
      up = __reduce_add_sync(0xffffffffu, up);
      if (lane == 0) atomicAdd(&sm.warp_gt[warp], up);
    }
    __syncthreads();
    thr = neg ? (known == 1u ? __uint_as_float(0x7FC00000u) : __uint_as_float(~known)) : __uint_as_float(known);
    share(1);
  }
  // (that barrier followed the last access to another CTA's memory, and every
  // CTA's read of the length: seq_len_out may be seq_len itself)
  if (rank == 0 && tid == 0) a.seq_len_out[b] = p.n;
  const uint32_t take_eq = left;  // of the entries at the threshold, how many stay
  const bool nan_thr = thr != thr;
  // ---- the ordered list: what precedes this warp's part, then 128 positions at a time ----
  const uint32_t ng = __reduce_add_sync(0xffffffffu, (lane < rank ? sm.gt[slot][lane] : 0u) +
                                                         (lane < warp ? sm.warp_gt[lane] : 0u));
  uint32_t ne = __reduce_add_sync(0xffffffffu, (lane < rank ? sm.eq[slot][lane] : 0u) +
                                                   (lane < warp ? sm.warp_eq[lane] : 0u));
  uint32_t at = ng + uint32_t(min(w0, m0)) + uint32_t(max(0, w0 - m1)) + min(ne, take_eq);  // kept before w0
  const uint32_t below = (1u << lane) - 1u;
  // f[i]: the weight of position q0 + 32 i + lane (any value behind the end)
  auto emit = [&](int q0, const float (&f)[4]) {
    bool stays[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) stays[i] = f[i] > thr;
    if (nan_thr || q0 < m0 || q0 + kStep > m1) {
      // some of these 128 are protected or behind the end
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int q = q0 + 32 * i + lane;
        const bool in = q >= m0 && q < m1;
        const bool same = in && (nan_thr ? f[i] != f[i] : f[i] == thr);
        const uint32_t m = __ballot_sync(0xffffffffu, same);
        stays[i] = in ? (nan_thr ? f[i] == f[i] : stays[i]) || (same && ne + __popc(m & below) < take_eq) : q < len;
        ne += __popc(m);
      }
    } else if (ne < take_eq) {
      // the first entries at the threshold stay: as a rule all of these 128
      const uint32_t n = __reduce_add_sync(0xffffffffu, uint32_t(f[0] == thr) + uint32_t(f[1] == thr) +
                                                            uint32_t(f[2] == thr) + uint32_t(f[3] == thr));
      if (ne + n <= take_eq) {
#pragma unroll
        for (int i = 0; i < 4; ++i) stays[i] = f[i] >= thr;
        ne += n;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t m = __ballot_sync(0xffffffffu, f[i] == thr);
          stays[i] = stays[i] || (f[i] == thr && ne + __popc(m & below) < take_eq);
          ne += __popc(m);
        }
      }
    }
    const uint32_t flags = (stays[0] ? 1u : 0u) + (stays[1] ? 1u << 8 : 0u) + (stays[2] ? 1u << 16 : 0u) +
                           (stays[3] ? 1u << 24 : 0u);
    const uint32_t incl = warp_incl(flags), sum = __shfl_sync(0xffffffffu, incl, 31);
    // four indexes from `at` (each below 128): entries of earlier groups of 32, and of lanes below
    const uint32_t idx = incl - flags + sum * 0x01010100u;
    int32_t* to = kept + at;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (stays[i]) to[__byte_perm(idx, 0, 0x4440 + i)] = q0 + 32 * i + lane;
    at += (sum * 0x01010101u) >> 24;
  };
  for (int q0 = w0; q0 < wc; q0 += kStep) {
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = mine[q0 - w0 + 32 * i + lane];
    emit(q0, f);
  }
  for (int q0 = w0 + warp_cap; q0 < w1; q0 += 2 * kStep) {
    float f[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float* src = q0 + h * kStep < w1 ? step_at(q0 + h * kStep) : nullptr;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        f[h][i] = q0 + h * kStep + 32 * i + lane < w1 ? one(src + 32 * i + lane) : 0.0f;
    }
    emit(q0, f[0]);
    if (q0 + kStep < w1) emit(q0 + kStep, f[1]);
  }
}

constexpr int kMThreads = 256;
// Destination rows of a CTA: 64 measured 264 us at four sequences of 2^20 cut
// to half, 256 (fewer, longer CTAs with the same loads in flight) 296 us, and
// a persistent grid that looks rows up one tile ahead 320 us.
constexpr int kMRows = 64;

// Copies the kPerRow 16-byte words of each row (drow < 0: none), all of a thread's in flight.
template <int kPerRow>
__device__ __forceinline__ void move_plane(const uint8_t* src, uint8_t* dst, const int64_t (&srow)[kMRows],
                                           const int64_t (&drow)[kMRows], int tid) {
  constexpr int kN = (kMRows * kPerRow + kMThreads - 1) / kMThreads;
  uint4 v[kN];
#pragma unroll
  for (int m = 0; m < kN; ++m) {
    const int i = tid + m * kMThreads, r = i / kPerRow;
    if (r < kMRows && drow[r] >= 0) v[m] = __ldg(reinterpret_cast<const uint4*>(src) + srow[r] * kPerRow + i % kPerRow);
  }
#pragma unroll
  for (int m = 0; m < kN; ++m) {
    const int i = tid + m * kMThreads, r = i / kPerRow;
    if (r < kMRows && drow[r] >= 0) reinterpret_cast<uint4*>(dst)[drow[r] * kPerRow + i % kPerRow] = v[m];
  }
}

__global__ void __launch_bounds__(kMThreads, 8) k_evict_move(EvictArgs a) {
  __shared__ int64_t srow[kMRows], drow[kMRows];
  const int b = blockIdx.y, tid = threadIdx.x;
  launch_dependents();
  grid_wait();
  int64_t s = -1, d = -1;
  if (tid < kMRows) {
    const int64_t r = int64_t(blockIdx.x) * kMRows + tid;
    const int pos = r < a.max_keep ? __ldg(a.kept + int64_t(b) * a.max_keep + r) : -1;
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
  if (__syncthreads_and(d < 0)) return;
  move_plane<kMainCodeBytes / 16>(a.main_src.codes, a.main_dst.codes, srow, drow, tid);
  move_plane<kMainScaleBytes / 16>(a.main_src.scales, a.main_dst.scales, srow, drow, tid);
  if (a.idx_src.codes) {
    move_plane<kIdxCodeBytes / 16>(a.idx_src.codes, a.idx_dst.codes, srow, drow, tid);
    if (d >= 0)
      reinterpret_cast<uint32_t*>(a.idx_dst.scales)[d] = __ldg(reinterpret_cast<const uint32_t*>(a.idx_src.scales) + s);
  }
  if (d >= 0) a.acc_dst[d] = __ldg(a.acc_src + s);
}

template <class L>
csa2_status launch_select(const EvictArgs& a, const L& layers, bool vec, cudaStream_t st) {
  // CTAs per sequence: one for every 8192 positions while the clusters of all
  // sequences run at once.  The CTAs of a cluster share a GPC, so a B200's 148
  // SMs hold fewer clusters than 148 / C: kActive[C], as its occupancy query
  // gives it (another layout of the GPCs costs a second wave, nothing else).
  constexpr int kActive[kMaxCluster + 1] = {0, 148, 74, 45, 33, 26, 22, 15, 15, 15, 11, 7, 7, 7, 7, 7, 7};
  const int64_t want = (a.src.max_len + kRunKeys - 1) / kRunKeys;
  int C = int(std::max<int64_t>(1, std::min<int64_t>(kMaxCluster, want)));
  while (C > 1 && kActive[C] < a.B) --C;
  // weights of a warp that stay in shared memory: its part of the run, as far as there is room
  const int64_t steps = (a.src.max_len + kStep - 1) / kStep;
  const int64_t part = ((steps + C - 1) / C + kEWarps - 1) / kEWarps;
  const int64_t fit = (kSelSmem - int64_t(sizeof(SelSmem))) / (4 * kStep * kEWarps);
  const int warp_cap = int(std::min(part, fit)) * kStep;
  const size_t smem = sizeof(SelSmem) + size_t(warp_cap) * 4 * kEWarps;
  // (both are the kernel's, shared by all host threads: always the same values)
  cudaFuncSetAttribute(k_evict_select<L>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelSmem);
  if (C > 8) cudaFuncSetAttribute(k_evict_select<L>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  launch_k_cluster(k_evict_select<L>, dim3(C, a.B), dim3(kEThreads), smem, st, C, a, layers, warp_cap, vec);
  return check_launch("csa2_cache_evict");
}

}  // namespace

csa2_status launch_evict(const EvictArgs* a, int n, cudaStream_t st) {
  // accumulators that layers share count once
  MoreLayers more{};
  bool vec = aligned16(a[0].acc_src);
  for (int l = 1; l < n; ++l) {
    bool seen = a[l].acc_src == a[0].acc_src;
    for (int m = 0; m < more.n; ++m) seen |= a[l].acc_src == more.acc[m];
    if (seen) continue;
    more.acc[more.n++] = a[l].acc_src;
    vec = vec && aligned16(a[l].acc_src);
  }
  csa2_status rc = more.n ? launch_select(a[0], more, vec, st) : launch_select(a[0], OneLayer{}, vec, st);
  for (int l = 0; l < n && rc == CSA2_OK; ++l) {
    launch_k(k_evict_move, dim3(unsigned((int64_t(a[l].max_keep) + kMRows - 1) / kMRows), unsigned(a[l].B)),
             dim3(kMThreads), 0, st, a[l]);
    rc = check_launch("csa2_cache_evict");
  }
  return rc;
}

}  // namespace csa2
