// Accumulated attention weight of cache entries.
//
// The attention of query i gave entry j the weight
//   w_ij = sum_h exp(sm_scale q_ih . key_j - lse_ih)
// (lse over the whole softmax, window rows included, as the attention call
// returns it); acc[row of j] += w_ij for the queries that count.  Only the
// logits are needed again, not the values: the kernel reads the selected
// rows, multiplies and adds.
//
// k_weights.  A warp takes groups of 16 selected rows of one query; the CTA's
// four warps share the query, converted once, and nothing else: each streams
// its own groups, cp.async bringing the next group's 272-byte rows while it
// multiplies (no barrier after the first).  The product is 16 rows x 16 heads
// (mma m16n8k16, fp32 accumulation): E2M1 codes are exact in fp16, each
// block's E8M0 scale multiplies the block's fp32 sum, and a head's query row
// is scaled by a power of two into [2^14, 2^15) at its largest element before
// it becomes fp16, so every bf16 query element down to 2^-39 of the row's
// largest is exact and no input leaves the fp16 range.  Inside a block the
// order of the 32 dims is permuted (the same way for both operands) so that a
// lane's 8 dims are one 32-bit word of codes.  Bound by instructions: about
// 50 per row and warp, half of them to convert codes and apply scales.
//
// Order of the sums.  Entries are added in fp32 (weights of one query are at
// most 16, sums grow over a sequence's life).  Where one query of a sequence
// counts, k_weights adds itself.  Where several do, two of them may select
// the same entry, and k_accumulate adds them in the order of the queries:
// CTA p of a sequence owns the entries whose position falls into its part, a
// barrier separates the queries (the next query's ids and weights are on
// their way meanwhile).  A position listed twice in one selection
// counts twice, as it does in the softmax; both additions have the same
// value, so their order does not matter.
#include <cuda_fp16.h>

#include <algorithm>

#include "device_common.cuh"
#include "sm100.cuh"

namespace csa2 {

namespace {

constexpr int kWarps = 4;                     // per CTA; they share the query
constexpr int kWThreads = 32 * kWarps;
constexpr int kWRows = 16;                    // selected rows of a warp's group (MMA M)
constexpr int kWStages = 2;
constexpr int kRow = kMainCodeBytes + kMainScaleBytes;  // 272 bytes: codes, then scales
constexpr int kQStride = kD + 32;             // halves: rows g and g+1 lie 4 of 8 16-byte columns apart
constexpr uint32_t kBig = 224;                // scale bytes from here on take the slow path (2^97 and more)

struct WSmem {
  __half q[kHq][kQStride];
  uint8_t raw[kWarps][kWStages][kWRows][kRow];
  float qexp[kHq];                            // power of two that undoes the query row's scaling
  float lse[kHq];
};

__device__ __forceinline__ uint32_t e2m1x2_f16x2(uint32_t byte) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\tmov.b16 {t, _}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}" : "=r"(r) : "h"(uint16_t(byte)));
  return r;
}
// d = a b (from zero) and d += a b.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 16 bytes, or zeros where `valid` is false (src is then not read).
__device__ __forceinline__ void cp_async16_or_zero(void* dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sm100::smem_u32(dst)), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
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

// Scale byte j of word w as 2^(byte - 127 - sub).  Plain rows (no byte of kBig
// or more) have sub = 0; a byte of 0 stands on blocks of zeros there, and 0.0
// serves them.
template <bool kPlain>
__device__ __forceinline__ float e8m0(uint32_t w, int j, int sub) {
  const int bits = int((j == 3 ? w >> 1 : w << (23 - 8 * j)) & 0x7F800000u);
  return __int_as_float(kPlain ? bits : max(bits - (sub << 23), 0x00400000));
}

// Products of the warp's 16 rows with the 16 heads: acc[h][0..1] row g, heads
// 8h + 2t and + 1; acc[h][2..3] row g + 8 (lane = 4 g + t).
template <bool kPlain>
__device__ __forceinline__ void products(const WSmem& sm, const uint8_t (&raw)[kWRows][kRow], float (&acc)[2][4],
                                         int sub0, int sub1, int g, int t) {
#pragma unroll 1
  for (int j4 = 0; j4 < kD / 128; ++j4) {
    const uint32_t sw0 = *reinterpret_cast<const uint32_t*>(raw[g] + kMainCodeBytes + 4 * j4);
    const uint32_t sw1 = *reinterpret_cast<const uint32_t*>(raw[g + 8] + kMainCodeBytes + 4 * j4);
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) {
      const int j = 4 * j4 + jj;
      const uint32_t w0 = *reinterpret_cast<const uint32_t*>(raw[g] + 16 * j + 4 * t);
      const uint32_t w1 = *reinterpret_cast<const uint32_t*>(raw[g + 8] + 16 * j + 4 * t);
      const uint32_t a0[4] = {e2m1x2_f16x2(w0 & 255u), e2m1x2_f16x2(w1 & 255u), e2m1x2_f16x2((w0 >> 8) & 255u),
                              e2m1x2_f16x2((w1 >> 8) & 255u)};
      const uint32_t a1[4] = {e2m1x2_f16x2((w0 >> 16) & 255u), e2m1x2_f16x2((w1 >> 16) & 255u), e2m1x2_f16x2(w0 >> 24),
                              e2m1x2_f16x2(w1 >> 24)};
      const float s0 = e8m0<kPlain>(sw0, jj, sub0), s1 = e8m0<kPlain>(sw1, jj, sub1);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 q = *reinterpret_cast<const uint4*>(&sm.q[8 * h + g][32 * j + 8 * t]);
        float d[4];
        mma_f16_first(d, a0, q.x, q.y);
        mma_f16(d, a1, q.z, q.w);
        acc[h][0] = fmaf(d[0], s0, acc[h][0]);
        acc[h][1] = fmaf(d[1], s0, acc[h][1]);
        acc[h][2] = fmaf(d[2], s1, acc[h][2]);
        acc[h][3] = fmaf(d[3], s1, acc[h][3]);
      }
    }
  }
}

__global__ void __launch_bounds__(kWThreads) k_weights(WeightArgs a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  WSmem& sm = *reinterpret_cast<WSmem*>(smem_raw);
  const int i = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int groups = (a.k + kWRows - 1) / kWRows, stride = gridDim.y * kWarps;
  const int32_t* ids = a.topk + int64_t(i) * a.k;
  float* wout = a.weights + int64_t(i) * a.k;
  int grp = blockIdx.y * kWarps + warp;
  launch_dependents();
  grid_wait();
  // ids of a group (lanes 0 .. 15); a group behind the last has none
  auto load_ids = [&](int gr) {
    const int slot = gr * kWRows + lane;
    return lane < kWRows && slot < a.k ? __ldg(ids + slot) : -1;
  };
  int id = load_ids(grp);
  const QueryRef ref = query_ref(a, i, lane);
  if (!ref.counted) {
    for (int gr = grp; gr < groups; gr += stride)
      if (lane < kWRows && gr * kWRows + lane < a.k) wout[gr * kWRows + lane] = 0.0f;
    return;
  }
  const int64_t len = seg_len_checked(a.sd, ref.seq, lane == 0 ? a.status : nullptr);
  const int64_t base = a.sd.pages ? 0 : a.sd.row_off[ref.seq];
  // this lane's cache row of the group (-1: empty slot)
  auto row_of = [&](int pos) {
    if (pos < 0) return -1;
    if (pos >= len) {
      set_status(a.status, CSA2_DEV_INDEX_RANGE);
      return -1;
    }
    return int(a.sd.pages ? entry_row(a.sd, ref.seq, pos, a.status) : base + pos);
  };
  auto issue = [&](int stage, int row) {
    uint8_t(*raw)[kRow] = sm.raw[warp][stage];
#pragma unroll
    for (int p = 0; p < kWRows / 2; ++p) {  // two rows' codes
      const int r = 2 * p + (lane >> 4), from = __shfl_sync(0xffffffffu, row, r);
      cp_async16_or_zero(raw[r] + 16 * (lane & 15),
                         a.mcodes + int64_t(max(from, 0)) * kMainCodeBytes + 16 * (lane & 15), from >= 0);
    }
    if (lane < kWRows)
      cp_async16_or_zero(raw[lane] + kMainCodeBytes, a.mscales + int64_t(max(row, 0)) * kMainScaleBytes, row >= 0);
    sm100::cp_async_commit();
  };
  int row = row_of(id);
  if (grp < groups) issue(0, row);
  id = load_ids(grp + stride);
  // ---- the query: warp w converts heads 4w .. 4w+3 while its rows are on their way ----
  if (warp == 0 && lane < kHq) sm.lse[lane] = a.lse[int64_t(i) * kHq + lane];
#pragma unroll
  for (int h0 = 0; h0 < kHq / kWarps; ++h0) {
    const int h = kHq / kWarps * warp + h0;
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
  __syncthreads();
  float lse[4], qexp[4];  // of heads 2t, 2t+1, 8+2t, 8+2t+1
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    lse[h] = sm.lse[8 * (h >> 1) + 2 * t + (h & 1)];
    qexp[h] = sm.qexp[8 * (h >> 1) + 2 * t + (h & 1)];
  }
  for (int stage = 0; grp < groups; grp += stride, stage ^= 1) {
    const int next = row_of(id);
    if (grp + stride < groups) {
      issue(stage ^ 1, next);
      id = load_ids(grp + 2 * stride);
      sm100::cp_async_wait<1>();
    } else {
      sm100::cp_async_wait<0>();
    }
    __syncwarp();
    const uint8_t(&raw)[kWRows][kRow] = sm.raw[warp][stage];
    // rows with a scale byte of kBig or more: lane (g, t) looks at word t of rows g and g + 8
    const uint32_t b0 = *reinterpret_cast<const uint32_t*>(raw[g] + kMainCodeBytes + 4 * t);
    const uint32_t b1 = *reinterpret_cast<const uint32_t*>(raw[g + 8] + kMainCodeBytes + 4 * t);
    const uint32_t big0 = b0 & (b0 << 1) & (b0 << 2) & 0x80808080u, big1 = b1 & (b1 << 1) & (b1 << 2) & 0x80808080u;
    static_assert(kBig == 0xE0, "the three top bits");
    float acc[2][4] = {}, mul0 = 1.0f, mul1 = 1.0f;
    if (!__any_sync(0xffffffffu, big0 | big1)) {
      products<true>(sm, raw, acc, 0, 0, g, t);
    } else {
      // Such a row is multiplied with its scales 2^64 times smaller (blocks
      // that this takes below 2^-127 do not matter beside one of 2^97), and
      // one with an E8M0 NaN becomes NaN.
      auto row_any = [&](bool v) { return ((__ballot_sync(0xffffffffu, v) >> (4 * g)) & 15u) != 0u; };
      auto has_nan = [&](uint32_t w) { return (w & 255u) == 255u || (w >> 8 & 255u) == 255u || (w >> 16 & 255u) == 255u || w >> 24 == 255u; };
      const bool r0 = row_any(big0 != 0u), r1 = row_any(big1 != 0u), n0 = row_any(has_nan(b0)), n1 = row_any(has_nan(b1));
      products<false>(sm, raw, acc, r0 ? 64 : 0, r1 ? 64 : 0, g, t);
      mul0 = n0 ? __uint_as_float(0x7FC00000u) : r0 ? 1.8446744073709552e19f : 1.0f;  // 2^64
      mul1 = n1 ? __uint_as_float(0x7FC00000u) : r1 ? 1.8446744073709552e19f : 1.0f;
    }
    // ---- weights: exp(logit - lse), summed over the heads (four here, the others in lanes of other t) ----
    float w0 = 0.0f, w1 = 0.0f;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      // (no key at all: lse is -inf, and nothing has a weight)
      const bool none = lse[h] == -INFINITY;
      const float x0 = fmaf(acc[h >> 1][h & 1] * qexp[h] * mul0, a.sm_scale, -lse[h]);
      const float x1 = fmaf(acc[h >> 1][2 + (h & 1)] * qexp[h] * mul1, a.sm_scale, -lse[h]);
      w0 += none ? 0.0f : expf(x0);
      w1 += none ? 0.0f : expf(x1);
    }
#pragma unroll
    for (int d = 1; d <= 2; d <<= 1) {
      w0 += __shfl_xor_sync(0xffffffffu, w0, d);
      w1 += __shfl_xor_sync(0xffffffffu, w1, d);
    }
    // lane (g, 0) has row g, lane (g, 1) row g + 8
    const int r = g + 8 * (t & 1), at = __shfl_sync(0xffffffffu, row, r);
    if (t < 2) {
      float v = at >= 0 ? (t ? w1 : w0) : 0.0f;
      if (v < 1.17549435e-38f) v = 0.0f;  // 2^-126: the fp32 atomics below flush subnormal numbers
      const int slot = grp * kWRows + r;
      if (slot < a.k) wout[slot] = v;
      if (at >= 0 && !ref.several) atomicAdd(a.acc + at, v);
    }
    row = next;
    __syncwarp();  // this stage is read before its next copies
  }
}

// Sequences of which several queries count: their weights are added query by
// query.  CTA (p, b) owns positions [len p / P, len (p+1) / P) of sequence b.
constexpr int kAThreads = 256;
constexpr int kAPer = CSA2_MAX_TOPK / kAThreads;  // slots of a thread

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
  const int lo = int(len * blockIdx.y / gridDim.y), hi = int(len * (blockIdx.y + 1) / gridDim.y);
  // this thread's slots of query i that lie in this part: ids, then weights
  auto fetch = [&](int i, int (&id)[kAPer], float (&w)[kAPer]) {
    const int64_t at = int64_t(i) * a.k;
#pragma unroll
    for (int m = 0; m < kAPer; ++m) {
      const int j = tid + m * kAThreads;
      id[m] = j < a.k ? __ldg(a.topk + at + j) : -1;
    }
#pragma unroll
    for (int m = 0; m < kAPer; ++m) {
      if (id[m] < lo || id[m] >= hi) id[m] = -1;
      w[m] = id[m] >= 0 ? __ldcg(a.weights + at + tid + m * kAThreads) : 0.0f;
    }
  };
  int id[kAPer], id2[kAPer];
  float w[kAPer], w2[kAPer];
  fetch(q0, id, w);
  for (int i = q0; i <= q0 + most; ++i) {
    if (i < q0 + most) fetch(i + 1, id2, w2);
#pragma unroll
    for (int m = 0; m < kAPer; ++m) {
      if (id[m] >= 0) {
        const int64_t row = entry_row(a.sd, b, id[m], nullptr);
        if (row >= 0) atomicAdd(a.acc + row, w[m]);
      }
      id[m] = id2[m];
      w[m] = w2[m];
    }
    __syncthreads();
  }
}

}  // namespace

void launch_weights(const WeightArgs& a, cudaStream_t st) {
  // CTAs per query: one for every 64 slots while the SMs have room for all of
  // them, else enough for a few waves of four CTAs per SM
  const int most = (a.k + kWRows * kWarps - 1) / (kWRows * kWarps);
  const int64_t room = 16 * int64_t(num_sms());
  const int S = int(std::max<int64_t>(1, std::min<int64_t>(most, (room + a.Q - 1) / a.Q)));
  cudaFuncSetAttribute(k_weights, cudaFuncAttributeMaxDynamicSharedMemorySize, int(sizeof(WSmem)));
  launch_k(k_weights, dim3(a.Q, S), dim3(kWThreads), sizeof(WSmem), st, a);
  if (!a.q_off) return;
  // parts of a sequence: the ids are read by each of them
  const int P = int(std::max<int64_t>(1, std::min<int64_t>(16, 4 * int64_t(num_sms()) / a.B)));
  launch_k(k_accumulate, dim3(a.B, P), dim3(kAThreads), 0, st, a);
}

}  // namespace csa2
