// Accumulated attention weight of cache entries.
//
// The attention of query i gave entry j the weight
//   w_ij = sum_h exp(sm_scale q_ih . key_j - lse_ih)
// (lse over the whole softmax, window rows included, as the attention call
// returns it); acc[row of j] += w_ij for the queries that count.  Only the
// logits are needed again, not the values: the kernel reads the selected
// rows, multiplies and adds.
//
// k_weights.  A warp takes groups of 16 or 32 selected rows of one query; the
// CTA's four warps share the query, converted once, and nothing else: each
// streams its own groups, cp.async bringing the next group's 272-byte rows
// while it works on this one (no barrier after the first).  The product is 16
// rows x 16 heads (mma m16n8k16, fp32 accumulation): E2M1 codes are exact in
// fp16, each block's E8M0 scale (converted once per group, in shared memory)
// multiplies the block's fp32 sum, and a head's query row is scaled by a power
// of two into [2^14, 2^15) at its largest element before it becomes fp16: bf16
// elements down to 2^-31 of the row's largest are exact (their last bit is
// 2^-24 there, fp16's smallest number), those below are rounded by at most 2^-39
// of it, and no input leaves the fp16 range.  Inside a block the order of the 32 dims is
// permuted (the same way for both operands) so that a lane's 8 dims are one
// 32-bit word of codes.  Few rows: bound by the chain of dependent loads
// (offsets, ids, rows).  Many: by instructions and shared memory reads.
//
// Order of the sums.  Entries are added in fp32 (weights of one query are at
// most 16, sums grow over a sequence's life).  Where one query of a sequence
// counts, k_weights adds itself.  Where several do, two of them may select
// the same entry, and they are added in the order of the queries, a barrier
// between two: by the last CTA of the sequence to finish, or (many queries) by
// k_accumulate, whose CTA p of a sequence owns the entries whose position
// falls into its part.  A position listed twice in one selection counts twice,
// as it does in the softmax; both additions have the same value, so their
// order does not matter.
#include <cuda_fp16.h>

#include <algorithm>

#include "device_common.cuh"
#include "sm100.cuh"

namespace csa2 {

namespace {

constexpr int kRow = kMainCodeBytes + kMainScaleBytes;  // 272 bytes: codes, then scales
constexpr int kQStride = kD + 32;             // halves: rows g and g+1 lie 4 of 8 16-byte columns apart
constexpr int kBlocks = kD / 32;              // 16 scale blocks
constexpr int kLastK = 512;                   // longest selections that the last CTA of a sequence adds itself
constexpr uint32_t kBig = 224;                // scale bytes from here on take the slow path (2^97 and more)

// kTiles: MMA tiles (16 rows) of a warp's group.  Two tiles halve the shared
// memory reads of the query, which bound the kernel next to the instructions
// (48 sequences of up to 16 candidates, k = 2048: 94.1 us with one tile, 80.6
// with two); one tile spreads few rows over more warps (64 queries of k = 512:
// 7.5 against 9.5 us).
template <int kTiles>
struct Cfg {
  static constexpr int kWarps = 4;                   // per CTA; they share the query
  static constexpr int kStages = kTiles == 1 ? 2 : 1;      // groups of a warp in shared memory
  static constexpr int kBlocksPerSm = kTiles == 1 ? 4 : 3;
  static constexpr int kRows = 16 * kTiles;
  static constexpr int kThreads = 32 * kWarps;
};

template <int kTiles>
struct WSmem {
  using C = Cfg<kTiles>;
  __half q[kHq][kQStride];
  uint8_t raw[C::kWarps][C::kStages][C::kRows][kRow];
  float scale[C::kWarps][C::kRows][kBlocks];  // the current group's block scales
  float qexp[kHq];                            // power of two that undoes the query row's scaling
  float lse[kHq];
  int last;
};

// Eight E2M1 codes (element 0 in the low nibble) -> four f16x2, exact.
__device__ __forceinline__ void e2m1x8_f16(uint32_t w, uint32_t (&f)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3])
      : "r"(w));
}
// d = a b (from zero) and d += a b.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
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

// The sequence of query i, whether it counts, and the queries of its sequence
// that do (the first one and how many follow it).  q_off ascends, so the
// sequence is the number of sequences that end at or before i; offsets that do
// not ascend within [0, Q] are reported and no query counts.  Whole warp.
struct QueryRef {
  int seq, counted, q0, more;
};
__device__ __forceinline__ QueryRef query_ref(const WeightArgs& a, int i, int lane) {
  if (a.q_off == nullptr) return QueryRef{i, 1, i, 0};
  int b = 0, prior = __ldg(a.q_off);
  const int first = prior;
  bool bad = first < 0;
  for (int j0 = 1; j0 <= a.B; j0 += 32) {
    const int j = j0 + lane, end = __ldg(a.q_off + min(j, a.B)), left = __shfl_up_sync(0xffffffffu, end, 1);
    bad |= end < (lane ? left : prior) || end > a.Q;
    prior = __shfl_sync(0xffffffffu, end, 31);
    b += __popc(__ballot_sync(0xffffffffu, j <= a.B && end <= i));
  }
  if (__any_sync(0xffffffffu, bad)) {
    if (i == 0 && lane == 0) set_status(a.status, CSA2_DEV_LENGTH);
    return QueryRef{-1, 0, 0, 0};
  }
  if (b >= a.B || first > i) return QueryRef{-1, 0, 0, 0};
  const int q0 = __ldg(a.q_off + b), n = __ldg(a.q_off + b + 1) - q0;
  const int more = a.n_accept ? min(max(__ldg(a.n_accept + b), 0), n - 1) : n - 1;
  return QueryRef{b, i - q0 <= more, q0, more};
}

// Products of the warp's rows with the 16 heads: acc[m][h][0..1] row 16m + g,
// heads 8h + 2t and + 1; acc[m][h][2..3] row 16m + g + 8 (lane = 4 g + t).
template <int kTiles>
__device__ __forceinline__ void products(const __half (&qs)[kHq][kQStride], const uint8_t (&raw)[16 * kTiles][kRow],
                                         const float (&scale)[16 * kTiles][kBlocks], float (&acc)[kTiles][2][4], int g,
                                         int t) {
#pragma unroll
  for (int j4 = 0; j4 < kBlocks / 4; ++j4) {
    float s[kTiles][2][4];
#pragma unroll
    for (int m = 0; m < 2 * kTiles; ++m) {
      const float4 v = *reinterpret_cast<const float4*>(&scale[8 * m + g][4 * j4]);
      s[m / 2][m & 1][0] = v.x, s[m / 2][m & 1][1] = v.y, s[m / 2][m & 1][2] = v.z, s[m / 2][m & 1][3] = v.w;
    }
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) {
      const int j = 4 * j4 + jj;
      uint32_t a0[kTiles][4], a1[kTiles][4];
#pragma unroll
      for (int m = 0; m < kTiles; ++m) {
        uint32_t f0[4], f1[4];
        e2m1x8_f16(*reinterpret_cast<const uint32_t*>(raw[16 * m + g] + 16 * j + 4 * t), f0);
        e2m1x8_f16(*reinterpret_cast<const uint32_t*>(raw[16 * m + g + 8] + 16 * j + 4 * t), f1);
        a0[m][0] = f0[0], a0[m][1] = f1[0], a0[m][2] = f0[1], a0[m][3] = f1[1];
        a1[m][0] = f0[2], a1[m][1] = f1[2], a1[m][2] = f0[3], a1[m][3] = f1[3];
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 q = *reinterpret_cast<const uint4*>(&qs[8 * h + g][32 * j + 8 * t]);
#pragma unroll
        for (int m = 0; m < kTiles; ++m) {
          float d[4];
          mma_f16_first(d, a0[m], q.x, q.y);
          mma_f16(d, a1[m], q.z, q.w);
          acc[m][h][0] = fmaf(d[0], s[m][0][jj], acc[m][h][0]);
          acc[m][h][1] = fmaf(d[1], s[m][0][jj], acc[m][h][1]);
          acc[m][h][2] = fmaf(d[2], s[m][1][jj], acc[m][h][2]);
          acc[m][h][3] = fmaf(d[3], s[m][1][jj], acc[m][h][3]);
        }
      }
    }
  }
}

// The block scales of the warp's rows again, where some are 2^97 or more
// (bytes from kBig on): those 2^64 times smaller (255 is E8M0's NaN) and the
// others zero, or the others as they are and those zero.
template <int kTiles>
__device__ __forceinline__ void split_scales(const uint8_t (&raw)[16 * kTiles][kRow], float (&scale)[16 * kTiles][kBlocks],
                                             bool big, int g, int t) {
#pragma unroll 1
  for (int m = 0; m < 2 * kTiles; ++m) {
    const uint32_t word = *reinterpret_cast<const uint32_t*>(raw[8 * m + g] + kMainCodeBytes + 4 * t);
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      const uint32_t byte = word >> (8 * i) & 255u;
      uint32_t v = 0;
      if (big == (byte >= kBig))
        v = byte == 255u ? 0x7FC00000u : byte >= kBig ? (byte - 64u) << 23 : max(byte << 23, 0x00400000u);
      scale[8 * m + g][4 * t + i] = __uint_as_float(v);
    }
  }
}

// First half of the products of rows with such bytes: the other blocks' sums to
// `others`, the large ones' scales left for the second half.  Not inlined: the
// ordinary path keeps its registers (64 x 6 candidates 22.9 against 23.4 us).
template <int kTiles>
__device__ __noinline__ void products_of_others(const __half (&qs)[kHq][kQStride], const uint8_t (&raw)[16 * kTiles][kRow],
                                                float (&scale)[16 * kTiles][kBlocks], volatile float* others, int g, int t) {
  float acc[kTiles][2][4] = {};
  split_scales<kTiles>(raw, scale, false, g, t);
  __syncwarp();
  products<kTiles>(qs, raw, scale, acc, g, t);
#pragma unroll
  for (int r = 0; r < kTiles * 8; ++r) others[r] = acc[r >> 3][r >> 2 & 1][r & 3];
  __syncwarp();
  split_scales<kTiles>(raw, scale, true, g, t);
}

// Adds the weights of queries q0 .. q0 + more of sequence b, in their order, to
// the accumulators of positions lo .. hi-1.  Every thread of the CTA; at most
// kPer * kThreads slots.  A thread's ids are fetched two queries ahead, the
// cache rows and weights of those that lie in this part one ahead.
template <int kPer, int kThreads>
__device__ __forceinline__ void ordered_sums(const WeightArgs& a, int b, int q0, int more, int lo, int hi) {
  const int tid = threadIdx.x;
  auto fetch_ids = [&](int i, int (&id)[kPer]) {
#pragma unroll
    for (int m = 0; m < kPer; ++m) {
      const int j = tid + m * kThreads;
      id[m] = i <= q0 + more && j < a.k ? __ldg(a.topk + int64_t(i) * a.k + j) : -1;
    }
  };
  const int64_t base = a.sd.pages ? 0 : a.sd.row_off[b];
  auto fetch_rows = [&](int i, const int (&id)[kPer], int (&row)[kPer], float (&w)[kPer]) {
#pragma unroll
    for (int m = 0; m < kPer; ++m) {
      const bool here = id[m] >= lo && id[m] < hi;
      row[m] = here ? int(a.sd.pages ? entry_row(a.sd, b, id[m], nullptr) : base + id[m]) : -1;
      w[m] = here ? __ldcg(a.weights + int64_t(i) * a.k + tid + m * kThreads) : 0.0f;
    }
  };
  int row[kPer], row1[kPer], id1[kPer], id2[kPer];
  float w[kPer], w1[kPer];
  fetch_ids(q0, id2);
  fetch_ids(q0 + 1, id1);
  fetch_rows(q0, id2, row, w);
  for (int i = q0; i <= q0 + more; ++i) {
    fetch_ids(i + 2, id2);
    fetch_rows(i + 1, id1, row1, w1);
#pragma unroll
    for (int m = 0; m < kPer; ++m) {
      if (row[m] >= 0) atomicAdd(a.acc + row[m], w[m]);
      row[m] = row1[m];
      w[m] = w1[m];
      id1[m] = id2[m];
    }
    __syncthreads();
  }
}

template <int kTiles>
__global__ void __launch_bounds__(Cfg<kTiles>::kThreads, Cfg<kTiles>::kBlocksPerSm) k_weights(WeightArgs a) {
  constexpr int kWarps = Cfg<kTiles>::kWarps, kWRows = Cfg<kTiles>::kRows, kStages = Cfg<kTiles>::kStages;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  WSmem<kTiles>& sm = *reinterpret_cast<WSmem<kTiles>*>(smem_raw);
  const int i = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int groups = (a.k + kWRows - 1) / kWRows, stride = gridDim.y * kWarps;
  const int32_t* ids = a.topk + int64_t(i) * a.k;
  float* wout = a.weights + int64_t(i) * a.k;
  int grp = blockIdx.y * kWarps + warp;
  launch_dependents();
  grid_wait();
  // ids of a group, one per lane; a group behind the last has none
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
    if (lse[h] == -INFINITY) lse[h] = INFINITY;  // no key at all: nothing has a weight
  }
  for (int stage = 0; grp < groups; grp += stride, stage = (stage + 1) % kStages) {
    const int next = row_of(id);
    if (kStages > 1 && grp + stride < groups) {
      issue(stage ^ 1, next);
      id = load_ids(grp + 2 * stride);
      sm100::cp_async_wait<1>();
    } else {
      id = load_ids(grp + 2 * stride);
      sm100::cp_async_wait<0>();
    }
    __syncwarp();
    const uint8_t(&raw)[kWRows][kRow] = sm.raw[warp][stage];
    // ---- block scales as floats: lane (g, t) does words t of rows g, g + 8, .. ----
    uint32_t any = 0;
#pragma unroll
    for (int m = 0; m < 2 * kTiles; ++m) {
      const uint32_t word = *reinterpret_cast<const uint32_t*>(raw[8 * m + g] + kMainCodeBytes + 4 * t);
      static_assert(kBig == 0xE0, "the three top bits");
      any |= word & (word << 1) & (word << 2) & 0x80808080u;  // scale bytes of kBig or more
      // 2^(byte - 127), a byte of 0 as the subnormal 2^-127
      auto e8m0 = [](uint32_t byte) { return __int_as_float(max(int(byte << 23), 0x00400000)); };
      *reinterpret_cast<float4*>(&sm.scale[warp][8 * m + g][4 * t]) =
          make_float4(e8m0(word & 255u), e8m0(word >> 8 & 255u), e8m0(word >> 16 & 255u), e8m0(word >> 24));
    }
    const bool slow = __any_sync(0xffffffffu, any);
    float acc[kTiles][2][4] = {};
    // Scales of 2^97 and more could overflow the fp32 sums.  Where the warp's
    // rows hold such bytes, the other blocks are summed first and these then by
    // themselves with scales 2^64 times smaller: both sums are as exact as the
    // ordinary one, whatever the blocks' sizes.
    volatile float others[kTiles * 8];  // (volatile: in memory)
    if (slow) products_of_others<kTiles>(sm.q, raw, sm.scale[warp], others, g, t);
    __syncwarp();
    products<kTiles>(sm.q, raw, sm.scale[warp], acc, g, t);
    __syncwarp();  // this stage is read before its next copies
    const int here = row;
    if (kStages == 1 && grp + stride < groups) issue(0, next);
    row = next;
    // ---- weights: exp(logit - lse), summed over the heads (four here, the others in lanes of other t) ----
    float w[2 * kTiles];
#pragma unroll
    for (int m = 0; m < 2 * kTiles; ++m) {
      w[m] = 0.0f;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int at = 2 * (m & 1) + (h & 1);
        float x = acc[m >> 1][h >> 1][at] * qexp[h];
        if (slow) x = x * 1.8446744073709552e19f + others[8 * (m >> 1) + 4 * (h >> 1) + at] * qexp[h];  // 2^64
        w[m] += expf(fmaf(x, a.sm_scale, -lse[h]));
      }
#pragma unroll
      for (int d = 1; d <= 2; d <<= 1) w[m] += __shfl_xor_sync(0xffffffffu, w[m], d);
    }
    // lane (g, t) has row g + 8 t
    const int r = g + 8 * t, at = __shfl_sync(0xffffffffu, here, r % kWRows);
    if (r < kWRows) {
      float v = t == 0 ? w[0] : w[1];
      if (kTiles == 2 && t >= 2) v = t == 2 ? w[2 * kTiles - 2] : w[2 * kTiles - 1];
      // 2^-126: the fp32 atomics below flush subnormal numbers
      if (at < 0 || v < 1.17549435e-38f) v = 0.0f;
      const int slot = grp * kWRows + r;
      if (slot < a.k) wout[slot] = v;
      if (at >= 0 && ref.more == 0) atomicAdd(a.acc + at, v);
    }
  }
  if (kTiles == 1 && a.counters != nullptr && ref.more > 0) {
    // Few queries: the last CTA of the sequence adds its weights.  The barrier
    // orders every thread's stores before thread 0's release-acquire arrival.
    __syncthreads();
    if (tid == 0) {
      int old;
      asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(old) : "l"(a.counters + ref.seq) : "memory");
      sm.last = old == (ref.more + 1) * int(gridDim.y) - 1;
    }
    __syncthreads();
    if (!sm.last) return;
    if (tid == 0) a.counters[ref.seq] = 0;
    ordered_sums<kLastK / Cfg<kTiles>::kThreads, Cfg<kTiles>::kThreads>(a, ref.seq, ref.q0, ref.more, 0, int(len));
  }
}

// The same as a kernel of its own, for many queries: CTA (b, p) owns positions
// [len p / P, len (p+1) / P) of sequence b.
constexpr int kAThreads = 512;

__global__ void __launch_bounds__(kAThreads) k_accumulate(WeightArgs a) {
  const int b = blockIdx.x;
  launch_dependents();
  grid_wait();
  const int q0 = __ldg(a.q_off + b), q1 = __ldg(a.q_off + b + 1);
  if (q0 < 0 || q1 > a.Q) return;  // (k_weights has reported it, and every weight is 0)
  const int more = a.n_accept ? min(max(__ldg(a.n_accept + b), 0), q1 - q0 - 1) : q1 - q0 - 1;
  if (more <= 0) return;
  const int64_t len = seg_len_checked(a.sd, b, nullptr);
  ordered_sums<CSA2_MAX_TOPK / kAThreads, kAThreads>(a, b, q0, more, int(len * blockIdx.y / gridDim.y),
                                                     int(len * (blockIdx.y + 1) / gridDim.y));
}

// Zeroes the accumulators of positions from[b] .. to[b]-1 of every sequence.
// A decode step clears at most one entry per sequence (a launch); a bulk append
// streams 4 bytes per entry.
constexpr int kCThreads = 256;

__global__ void __launch_bounds__(kCThreads) k_clear(ClearArgs a) {
  const int b = blockIdx.x;
  launch_dependents();
  grid_wait();
  const int64_t to = seg_len_checked(a.sd, b, blockIdx.y == 0 && threadIdx.x == 0 ? a.status : nullptr);
  for (int64_t t = max(a.from[b], 0) + int64_t(blockIdx.y) * kCThreads + threadIdx.x; t < to;
       t += int64_t(gridDim.y) * kCThreads) {
    const int64_t row = entry_row(a.sd, b, t, a.status);
    if (row >= 0) a.acc[row] = 0.0f;
  }
}

template <int kTiles>
void launch_tiles(const WeightArgs& a, int64_t ctas, cudaStream_t st) {
  constexpr int kSlots = Cfg<kTiles>::kRows * Cfg<kTiles>::kWarps;  // of a CTA at a time
  const int most = (a.k + kSlots - 1) / kSlots;
  const int S = int(std::max<int64_t>(1, std::min<int64_t>(most, (ctas + a.Q - 1) / a.Q)));
  cudaFuncSetAttribute(k_weights<kTiles>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(sizeof(WSmem<kTiles>)));
  launch_k(k_weights<kTiles>, dim3(a.Q, S), dim3(Cfg<kTiles>::kThreads), sizeof(WSmem<kTiles>), st, a);
}

}  // namespace

void launch_clear(const ClearArgs& a, cudaStream_t st) {
  const int S = std::max(1, std::min(64, 2 * num_sms() / a.B));
  launch_k(k_clear, dim3(a.B, S), dim3(kCThreads), 0, st, a);
}

void launch_weights(const WeightArgs& args, cudaStream_t st) {
  WeightArgs a = args;
  // Two tiles per warp once there are more than 32 tiles per SM.  CTAs of a
  // query: as many as its slots allow while the grid stays at 16 (one tile)
  // or 4 (two) CTAs per SM, about a wave of those that run together.
  const int64_t tiles = int64_t(a.Q) * ((a.k + 15) / 16), sms = num_sms();
  if (tiles <= 32 * sms) {
    // The last CTA of a sequence adds its weights where few slots make that
    // short; else, and for many queries, a kernel of its own with several CTAs
    // per sequence does (a second launch costs a caller about 2 us).
    const bool last = a.k <= kLastK && a.B <= kArrivalCounters;
    if (!last) a.counters = nullptr;
    launch_tiles<1>(a, 16 * sms, st);
    if (last) return;
  } else {
    a.counters = nullptr;
    launch_tiles<2>(a, 4 * sms, st);
  }
  if (!a.q_off) return;
  // parts of a sequence: the ids are read by each of them
  const int P = int(std::max<int64_t>(1, std::min<int64_t>(16, 2 * sms / a.B)));
  launch_k(k_accumulate, dim3(a.B, P), dim3(kAThreads), 0, st, a);
}

}  // namespace csa2
