// Accumulated attention weight of cache entries.
//
// The attention of query i gave entry j the weight
//   w_ij = sum_h exp(sm_scale q_ih . key_j - lse_ih)
// (lse over the whole softmax, window rows included, as the attention call
// returns it); acc[row of j] += w_ij for the queries that count.  Only the
// logits are needed again, not the values: the kernel reads the selected
// rows, multiplies and adds.
//
// k_weights.  A CTA takes chunks of 64 selected rows of one query.  The rows'
// 272 bytes come by cp.async while the query is converted; each of the four
// warps then multiplies its 16 rows with the 16 heads (mma m16n8k16, fp32
// accumulation): E2M1 codes are exact in fp16, each block's E8M0 scale
// multiplies the block's fp32 sum, and a head's query row is scaled by a
// power of two into [2^14, 2^15) at its largest element before it becomes
// fp16, so every bf16 query element down to 2^-39 of the row's largest is
// exact and no input leaves the fp16 range.  Inside a block the order of the
// 32 dims is permuted (the same way for both operands) so that a lane's
// 8 dims are one 32-bit word of codes.
//
// Order of the sums.  Entries are added in fp32 (weights of one query are at
// most 16, sums grow over a sequence's life).  Where one query of a sequence
// counts, k_weights adds itself.  Where several do, two of them may select
// the same entry, and k_accumulate adds them in the order of the queries:
// CTA p of a sequence owns the entries whose position falls into its part, a
// barrier separates the queries.  A position listed twice in one selection
// counts twice, as it does in the softmax; both additions have the same
// value, so their order does not matter.
#include <cuda_fp16.h>

#include <algorithm>

#include "device_common.cuh"
#include "sm100.cuh"

namespace csa2 {

namespace {

constexpr int kWKeys = 64;                    // selected rows per chunk
constexpr int kWThreads = 128;                // 4 warps of 16 rows
constexpr int kRow = kMainCodeBytes + kMainScaleBytes;  // 272 bytes: codes, then scales
constexpr int kQStride = kD + 32;             // halves: rows g and g+1 lie 4 of 8 16-byte columns apart
constexpr int kBlocks = kD / 32;              // 16 scale blocks

struct WSmem {
  __half q[kHq][kQStride];
  uint8_t raw[kWKeys][kRow];
  float qexp[kHq];                            // power of two that undoes the query row's scaling
  float lse[kHq];
  int64_t row[kWKeys];                        // cache row of a chunk's slot (-1: empty slot)
  int seq, counted, several;
  int64_t len;
};

__device__ __forceinline__ uint32_t e2m1x2_f16x2(uint32_t byte) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\tmov.b16 {t, _}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}" : "=r"(r) : "h"(uint16_t(byte)));
  return r;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 2^(byte - 127); byte 255 is E8M0's NaN.
__device__ __forceinline__ float e8m0(uint32_t byte) {
  return __uint_as_float(byte == 0u ? 0x00400000u : byte == 255u ? 0x7FC00000u : byte << 23);
}

// Cache row of position t of sequence b, or -1 (CSA2_DEV_ROW_LAYOUT) where the
// page table names a page outside the cache: such an entry has no weight.
__device__ __forceinline__ int64_t entry_row(const SegDesc& sd, int b, int64_t t, uint32_t* status) {
  if (sd.pages) {
    const int64_t pg = __ldg(sd.pages + int64_t(b) * sd.max_pages + (t >> sd.page_shift));
    if (pg < 0 || ((pg + 1) << sd.page_shift) > sd.cache_rows) {
      set_status(status, CSA2_DEV_ROW_LAYOUT);
      return -1;
    }
  }
  return seg_row(sd, b, t, status);
}

// The sequence of query i, whether it counts, and whether others of its
// sequence do.  q_off ascends, so the sequence is the number of sequences
// that end at or before i.  Whole warp.
struct QueryRef {
  int seq, counted, several;
};
__device__ __forceinline__ QueryRef query_ref(const WeightArgs& a, int i, int lane) {
  QueryRef r{i, 1, 0};
  if (a.q_off == nullptr) return r;
  int b = 0;
  for (int j0 = 1; j0 <= a.B; j0 += 32) {
    const int j = j0 + lane;
    const bool before = j <= a.B && __ldg(a.q_off + j) <= i;
    b += __popc(__ballot_sync(0xffffffffu, before));
  }
  if (b >= a.B || __ldg(a.q_off) > i) return QueryRef{-1, 0, 0};
  const int q0 = __ldg(a.q_off + b), q1 = __ldg(a.q_off + b + 1);
  const int most = a.n_accept ? min(max(__ldg(a.n_accept + b), 0), q1 - q0 - 1) : q1 - q0 - 1;
  r.seq = b;
  r.counted = i - q0 <= most;
  r.several = most > 0;
  return r;
}

__global__ void __launch_bounds__(kWThreads) k_weights(WeightArgs a) {
  __shared__ __align__(16) WSmem sm;
  const int i = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  launch_dependents();
  grid_wait();
  if (warp == 0) {
    const QueryRef r = query_ref(a, i, lane);
    if (lane == 0) {
      sm.seq = r.seq;
      sm.counted = r.counted;
      sm.several = r.several;
      sm.len = r.seq >= 0 ? seg_len_checked(a.sd, r.seq, a.status) : 0;
    }
  }
  if (tid >= 64 && tid < 64 + kHq) sm.lse[tid - 64] = a.lse[int64_t(i) * kHq + (tid - 64)];
  __syncthreads();
  const int b = sm.seq;
  float* wout = a.weights + int64_t(i) * a.k;
  if (!sm.counted) {
    for (int c = blockIdx.y * kWKeys; c < a.k; c += gridDim.y * kWKeys)
      if (tid < kWKeys && c + tid < a.k) wout[c + tid] = 0.0f;
    return;
  }
  const int64_t len = sm.len;
  bool first = true;
  for (int c0 = blockIdx.y * kWKeys; c0 < a.k; c0 += gridDim.y * kWKeys) {
    if (!first) __syncthreads();  // the last chunk's rows are read
    if (tid < kWKeys) {
      const int id = c0 + tid < a.k ? a.topk[int64_t(i) * a.k + c0 + tid] : -1;
      int64_t row = -1;
      if (id >= 0) {
        if (id < len) row = entry_row(a.sd, b, id, a.status);
        else set_status(a.status, CSA2_DEV_INDEX_RANGE);
      }
      sm.row[tid] = row;
    }
    __syncthreads();
    // 17 pieces of 16 bytes per row
    for (int p = tid; p < kWKeys * (kRow / 16); p += kWThreads) {
      const int r = p / (kRow / 16), part = p % (kRow / 16);
      const int64_t row = sm.row[r];
      uint8_t* dst = sm.raw[r] + 16 * part;
      if (row >= 0) {
        const uint8_t* src = part < kMainCodeBytes / 16 ? a.mcodes + row * kMainCodeBytes + 16 * part
                                                        : a.mscales + row * kMainScaleBytes;
        sm100::cp_async16(dst, src);
      } else {
        *reinterpret_cast<uint4*>(dst) = make_uint4(0, 0, 0, 0);
      }
    }
    sm100::cp_async_commit();
    if (first) {  // the query, while the rows are on their way: warp w converts heads 4w .. 4w+3
#pragma unroll
      for (int h0 = 0; h0 < 4; ++h0) {
        const int h = 4 * warp + h0;
        const uint4* src = reinterpret_cast<const uint4*>(a.q + (int64_t(i) * kHq + h) * kD);
        const uint4 v[2] = {__ldg(src + lane), __ldg(src + lane + 32)};
        const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
        float x[16], top = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[2 * j] = __uint_as_float(w[j] << 16);
          x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
          top = fmaxf(top, fmaxf(fabsf(x[2 * j]), fabsf(x[2 * j + 1])));
        }
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        // scale by 2^(14 - e), e the exponent of the largest element (kept where
        // both powers of two are normal numbers)
        const int e = min(max(int(__float_as_uint(top) >> 23) - 127, -112), 126);
        const float up = __uint_as_float(uint32_t(127 + 14 - e) << 23);
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const __half2 h2 = __floats2half2_rn(x[2 * j] * up, x[2 * j + 1] * up);
          o[j] = *reinterpret_cast<const uint32_t*>(&h2);
        }
        *reinterpret_cast<uint4*>(&sm.q[h][8 * lane]) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(&sm.q[h][8 * lane + 256]) = make_uint4(o[4], o[5], o[6], o[7]);
        if (lane == 0) sm.qexp[h] = __uint_as_float(uint32_t(127 - 14 + e) << 23);
      }
      first = false;
    }
    sm100::cp_async_wait<0>();
    __syncthreads();
    // ---- logits of the warp's 16 rows ----
    float acc[2][4] = {};
    const float qe0 = sm.qexp[g], qe1 = sm.qexp[g + 8];
    uint32_t sc[2][2][4];  // scale words of the rows of this lane's two accumulator columns, per n-tile
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        const uint4 v = *reinterpret_cast<const uint4*>(sm.raw[16 * warp + 8 * nt + 2 * t + cc] + kMainCodeBytes);
        sc[nt][cc][0] = v.x, sc[nt][cc][1] = v.y, sc[nt][cc][2] = v.z, sc[nt][cc][3] = v.w;
      }
#pragma unroll
    for (int j = 0; j < kBlocks; ++j) {
      const uint4 qa = *reinterpret_cast<const uint4*>(&sm.q[g][32 * j + 8 * t]);
      const uint4 qb = *reinterpret_cast<const uint4*>(&sm.q[g + 8][32 * j + 8 * t]);
      const uint32_t a0[4] = {qa.x, qb.x, qa.y, qb.y};
      const uint32_t a1[4] = {qa.z, qb.z, qa.w, qb.w};
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(sm.raw[16 * warp + 8 * nt + g] + 16 * j + 4 * t);
        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        mma_f16(d, a0, e2m1x2_f16x2(w & 255u), e2m1x2_f16x2((w >> 8) & 255u));
        mma_f16(d, a1, e2m1x2_f16x2((w >> 16) & 255u), e2m1x2_f16x2(w >> 24));
        const float s0 = e8m0((sc[nt][0][j / 4] >> (8 * (j % 4))) & 255u);
        const float s1 = e8m0((sc[nt][1][j / 4] >> (8 * (j % 4))) & 255u);
        acc[nt][0] = fmaf(d[0] * qe0, s0, acc[nt][0]);  // (qe: powers of two, so no rounding of its own)
        acc[nt][1] = fmaf(d[1] * qe0, s1, acc[nt][1]);
        acc[nt][2] = fmaf(d[2] * qe1, s0, acc[nt][2]);
        acc[nt][3] = fmaf(d[3] * qe1, s1, acc[nt][3]);
      }
    }
    // ---- weights: exp(logit - lse), summed over the heads (8 lanes of g, two heads each) ----
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      float w[2] = {0.0f, 0.0f};
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int h = g + 8 * (v >> 1);
        const float lse = sm.lse[h];
        // (no key at all: lse is -inf, and nothing has a weight)
        const float x = fmaf(acc[nt][v], a.sm_scale, -lse);
        w[v & 1] += lse == -INFINITY ? 0.0f : expf(x);
      }
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
#pragma unroll
        for (int d = 4; d <= 16; d <<= 1) w[cc] += __shfl_xor_sync(0xffffffffu, w[cc], d);
      }
      if (g < 2) {  // lane (g, t) writes column 2t + g
        const int r = 16 * warp + 8 * nt + 2 * t + g;
        const int64_t row = sm.row[r];
        float v = row >= 0 ? (g ? w[1] : w[0]) : 0.0f;
        if (v < 1.17549435e-38f) v = 0.0f;  // 2^-126: the fp32 atomics below flush subnormal numbers
        if (c0 + r < a.k) wout[c0 + r] = v;
        if (row >= 0 && !sm.several) atomicAdd(a.acc + row, v);
      }
    }
  }
}

// Sequences of which several queries count: their weights are added query by
// query.  CTA (p, b) owns positions [len p / P, len (p+1) / P) of sequence b.
constexpr int kAThreads = 256;

__global__ void __launch_bounds__(kAThreads) k_accumulate(WeightArgs a) {
  const int b = blockIdx.x, tid = threadIdx.x;
  launch_dependents();
  grid_wait();
  const int q0 = __ldg(a.q_off + b), q1 = __ldg(a.q_off + b + 1);
  const int most = a.n_accept ? min(max(__ldg(a.n_accept + b), 0), q1 - q0 - 1) : q1 - q0 - 1;
  if (q0 < 0 || q1 < q0 || q1 > a.Q) {
    if (blockIdx.y == 0 && tid == 0) set_status(a.status, CSA2_DEV_LENGTH);
    return;
  }
  if (most <= 0) return;
  const int64_t len = seg_len_checked(a.sd, b, nullptr);
  const int64_t lo = len * blockIdx.y / gridDim.y, hi = len * (blockIdx.y + 1) / gridDim.y;
  for (int i = q0; i <= q0 + most; ++i) {
    for (int j = tid; j < a.k; j += kAThreads) {
      const int id = a.topk[int64_t(i) * a.k + j];
      if (id >= lo && id < hi) {
        const int64_t row = entry_row(a.sd, b, id, nullptr);
        if (row >= 0) atomicAdd(a.acc + row, __ldcg(a.weights + int64_t(i) * a.k + j));
      }
    }
    __syncthreads();
  }
}

}  // namespace

void launch_weights(const WeightArgs& a, cudaStream_t st) {
  const int nchunk = (a.k + kWKeys - 1) / kWKeys;
  launch_k(k_weights, dim3(a.Q, nchunk), dim3(kWThreads), 0, st, a);
  if (a.q_off) launch_k(k_accumulate, dim3(a.B, 4), dim3(kAThreads), 0, st, a);
}

}  // namespace csa2
