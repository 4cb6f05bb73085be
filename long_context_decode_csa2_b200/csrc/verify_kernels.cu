// Verification of drafted tokens against the target's probabilities.
//
// Sequence b owns candidates q_off[b] .. q_off[b+1]-1: candidate 0 is its last
// known token, the others are drafts.  Row i of `target` is the target's
// distribution p_i behind candidate i, row i of `draft` the distribution q_i
// that candidate i+1 was drawn from.  Speculative sampling keeps candidate
// i+1 (token x) with probability min(1, p_i(x) / q_i(x)), here as the test
// u_i q_i(x) < p_i(x) (no division, and q = 0 needs no case of its own), and
// where the first one fails draws the next token from max(p_i - q_i, 0): the
// outcome is distributed as if it were drawn from p alone.  Behind the last
// candidate the token is drawn from p.  The draw inverts the running sum:
// the first j with C_j > r C_V.
//
// A border between two tokens is a value of the running sum, so the sums are
// fp64: in fp32 a vocabulary of 131072 puts a border within the rounding of
// r C_V about once in a hundred draws, in fp64 about once in 10^11.
//
// Work split.  Only the stop row of a sequence is read (n - 1 tests read
// single elements), by S CTAs, all sequences' at once: a warp takes a segment
// of 256 elements at a time and leaves its fp64 sum in the workspace; the last
// CTA of the sequence to finish scans them, and one of its warps reads the
// segment that holds r C_V again (from L2) to find the token.  The sums do not
// depend on S or on the order of arrival.  Bound by the chain of dependent steps (tests 2 us, arrival
// 1 us, scan and second read 3 us) until the rows are tens of MB.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "device_common.cuh"
#include "sm100.cuh"

namespace csa2 {

namespace {

constexpr int kVThreads = 256;
constexpr int kVWarps = kVThreads / 32;
constexpr int kVec = 8;                       // consecutive elements per lane and step
constexpr int kSeg = kVerifySegment;          // elements of one partial sum: 8 per lane
static_assert(kSeg == 32 * kVec, "a segment is one vector per lane");

struct NoDraft {};  // drafts without probabilities

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float as_float(__half x) { return __half2float(x); }

// A probability that is negative or NaN counts as 0.
__device__ __forceinline__ float prob(float x) { return x > 0.0f ? x : 0.0f; }

// Eight consecutive elements of a row as they lie in memory.  Rows start at
// any multiple of their element size: the vector is read as the aligned
// 16-byte words that cover it (one more than it fills where it is not aligned
// itself) and shifted into place.
template <class T>
struct Raw8 {
  static constexpr int kWords = kVec * int(sizeof(T)) / 4;  // 32-bit words of the vector
  uint32_t w[kWords + 4];

  // Elements of row that the covering words take from before e and behind e+7.
  static __device__ __forceinline__ int misalignment(const T* at) {
    return int(reinterpret_cast<uintptr_t>(at) & 15);
  }
  static __device__ __forceinline__ bool inside(const T* row, int64_t e, int64_t n, int64_t V) {
    const int mis = misalignment(row + e);
    const int pad = mis / int(sizeof(T)), tail = mis ? 16 / int(sizeof(T)) - pad : 0;
    return e - pad >= 0 && e + n + tail <= V;
  }
  __device__ __forceinline__ void load(const T* at, int mis) {
    const uint4* g = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(at) - mis);
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) {
      const uint4 v = __ldg(g + i);
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
    if (mis) {
      const uint4 v = __ldg(g + kWords / 4);
      w[kWords] = v.x, w[kWords + 1] = v.y, w[kWords + 2] = v.z, w[kWords + 3] = v.w;
    }
  }
  __device__ __forceinline__ void unpack(int mis, float (&x)[kVec]) {
    if (mis) {
      if (mis & 8) {
#pragma unroll
        for (int i = 0; i < kWords + 2; ++i) w[i] = w[i + 2];
      }
      if (mis & 4) {
#pragma unroll
        for (int i = 0; i < kWords + 1; ++i) w[i] = w[i + 1];
      }
      if (mis & 2) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
      }
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      if constexpr (sizeof(T) == 4) {
        x[i] = __uint_as_float(w[i]);
      } else {
        const uint16_t h = uint16_t(w[i / 2] >> (16 * (i & 1)));
        x[i] = as_float(*reinterpret_cast<const T*>(&h));
      }
    }
  }
};

// Elements e .. e+7 of a row (0 behind its end), one by one.
template <class T>
__device__ __forceinline__ void load8_edge(const T* row, int64_t e, int64_t V, float (&x)[kVec]) {
#pragma unroll
  for (int i = 0; i < kVec; ++i) x[i] = e + i < V ? as_float(row[e + i]) : 0.0f;
}

// What the next token is drawn from: p where every draft stood or the
// residual is empty, else max(p - q, 0).
template <class TQ>
struct StopRow {
  const TQ* q;      // draft row (null: p itself)
  int drafted;      // drafts without probabilities: the rejected token (-1: p itself)
};

// Weight of element e from its probabilities.
template <class TQ>
__device__ __forceinline__ double weight_of(float x, float y, const StopRow<TQ>& s, int64_t e) {
  const float a = prob(x);
  if constexpr (std::is_same<TQ, NoDraft>::value) {
    return double(e == s.drafted ? prob(a - 1.0f) : a);  // the draft's distribution is 1 at its token
  } else {
    const float b = prob(y);  // (0 where there is no draft row)
    return a > b ? double(a) - double(b) : 0.0;
  }
}

// fn(i, weights): this lane's 8 weights of segment seg + i, the loads of all kN
// segments in flight together.  Segments at an edge, whose covering words would
// leave the row (or that lie behind it), are read element by element.
template <int kN, class TP, class TQ, class F>
__device__ __forceinline__ void each_segment(const TP* p, const StopRow<TQ>& s, int seg, int64_t V, int lane, F&& fn) {
  constexpr bool kDraft = !std::is_same<TQ, NoDraft>::value;
  using QT = typename std::conditional<kDraft, TQ, float>::type;
  const int64_t e0 = int64_t(seg) * kSeg;
  const QT* q = nullptr;
  if constexpr (kDraft) q = s.q;
  if (Raw8<TP>::inside(p, e0, kN * kSeg, V) && (q == nullptr || Raw8<QT>::inside(q, e0, kN * kSeg, V))) {
    const TP* pe = p + e0 + lane * kVec;
    const QT* qe = q + e0 + lane * kVec;
    const int pm = Raw8<TP>::misalignment(pe), qm = q ? Raw8<QT>::misalignment(qe) : 0;
    Raw8<TP> pr[kN];
    Raw8<QT> qr[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) pr[i].load(pe + i * kSeg, pm);
    if (kDraft && q != nullptr) {
#pragma unroll
      for (int i = 0; i < kN; ++i) qr[i].load(qe + i * kSeg, qm);
    }
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      float x[kVec], y[kVec] = {};
      double w[kVec];
      pr[i].unpack(pm, x);
      if (kDraft && q != nullptr) qr[i].unpack(qm, y);
#pragma unroll
      for (int j = 0; j < kVec; ++j) w[j] = weight_of(x[j], y[j], s, e0 + i * kSeg + lane * kVec + j);
      fn(i, w);
    }
  } else {
#pragma unroll 1
    for (int i = 0; i < kN; ++i) {
      float x[kVec], y[kVec] = {};
      double w[kVec];
      const int64_t e = e0 + i * kSeg + lane * kVec;
      load8_edge(p, e, V, x);
      if (kDraft && q != nullptr) load8_edge(q, e, V, y);
#pragma unroll
      for (int j = 0; j < kVec; ++j) w[j] = weight_of(x[j], y[j], s, e + j);
      fn(i, w);
    }
  }
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}
__device__ __forceinline__ double warp_scan(double v, int lane) {  // inclusive
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const double o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// Segments of a warp whose loads are in flight together, with 32 warps per SM
// (64 x 131072 fp32 p and q: 19.3 us with one, 18.0 with two, spills with more;
// 256 x 50001 fp16 p: 17.6, 17.2 and 16.5 us with one, two and three).
template <class TP, class TQ>
constexpr int fly() {
  constexpr int bytes = int(sizeof(TP)) + (std::is_same<TQ, NoDraft>::value ? 0 : int(sizeof(TQ)));
  return bytes >= 4 ? 2 : 3;
}

// Sums of segments seg .. seg + fly - 1 (those below nseg) to part.
template <class TP, class TQ>
__device__ __forceinline__ void segment_sums(const TP* p, const StopRow<TQ>& s, int seg, int nseg, int64_t V, int lane,
                                             double* part) {
  constexpr int kFly = fly<TP, TQ>();
  double mine = 0.0;
  each_segment<kFly>(p, s, seg, V, lane, [&](int i, const double (&w)[kVec]) {
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < kVec; ++j) sum += w[j];
    sum = warp_sum(sum);
    if (lane == i) mine = sum;
  });
  if (lane < kFly && seg + lane < nseg) __stcg(part + seg + lane, mine);
}

// The first token of segment `seg` whose running sum (from `base`) passes
// `want`; where rounding lets none pass, the last one with a weight (-1: none).
template <class TP, class TQ>
__device__ __forceinline__ int segment_find(const TP* p, const StopRow<TQ>& s, int seg, int64_t V, double base,
                                            double want, int lane) {
  double w[kVec], sum = 0.0;
  each_segment<1>(p, s, seg, V, lane, [&](int, const double (&v)[kVec]) {
#pragma unroll
    for (int j = 0; j < kVec; ++j) w[j] = v[j];
  });
#pragma unroll
  for (int j = 0; j < kVec; ++j) sum += w[j];
  const double incl = warp_scan(sum, lane);
  double c = __shfl_up_sync(0xffffffffu, incl, 1);
  c = base + (lane == 0 ? 0.0 : c);
  int hit = -1, last = -1;
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    c += w[j];
    if (w[j] > 0.0) {
      last = seg * kSeg + lane * kVec + j;
      if (hit < 0 && c > want) hit = last;
    }
  }
  const unsigned any = __ballot_sync(0xffffffffu, hit >= 0);
  if (any) return __shfl_sync(0xffffffffu, hit, __ffs(any) - 1);
  return __reduce_max_sync(0xffffffffu, last);
}

struct Shared {
  int n, accepted, row0, drafted, last, seg;
  double base, want, total;
  double scan[kVWarps];
  int lastpos[kVWarps];
};

// Scans the segment sums: the first segment whose running sum passes r C_V
// (the last one with a weight where none does), what lies before it, and the
// total.  Every thread of the CTA.
__device__ __forceinline__ void find_segment(const double* part, int nseg, float r, Shared& sm) {
  constexpr int kKeep = 4;                             // sums of a thread in registers (vocabularies up to 2^18)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (nseg + kVThreads - 1) / kVThreads;  // consecutive segments of this thread
  const int s0 = min(nseg, tid * per), s1 = min(nseg, s0 + per);
  double v[kKeep], mine = 0.0;
  int pos = -1;
#pragma unroll
  for (int k = 0; k < kKeep; ++k) v[k] = s0 + k < s1 ? __ldcg(part + s0 + k) : 0.0;
#pragma unroll
  for (int k = 0; k < kKeep; ++k) {
    mine += v[k];
    if (v[k] > 0.0) pos = s0 + k;
  }
  for (int s = s0 + kKeep; s < s1; ++s) {
    const double x = __ldcg(part + s);
    mine += x;
    if (x > 0.0) pos = s;
  }
  const double incl = warp_scan(mine, lane);
  pos = __reduce_max_sync(0xffffffffu, pos);
  if (lane == 31) sm.scan[warp] = incl;
  if (lane == 0) sm.lastpos[warp] = pos;
  if (tid == 0) sm.seg = 0x7fffffff;
  __syncthreads();
  double before = 0.0, total = 0.0;
  int lastpos = -1;
#pragma unroll
  for (int w = 0; w < kVWarps; ++w) {
    if (w < warp) before += sm.scan[w];
    total += sm.scan[w];
    lastpos = max(lastpos, sm.lastpos[w]);
  }
  const double want = r >= 1.0f ? double(INFINITY) : double(r) * total;  // (from 1 on: the last weighted token)
  double c = __shfl_up_sync(0xffffffffu, incl, 1);
  c = before + (lane == 0 ? 0.0 : c);
  // this thread's first segment that passes, and what lies before it (or
  // before segment lastpos, which is taken where none passes).  Only segments
  // with a weight pass: c comes from the scan's grouping of the sums, `total`
  // from another, so behind the last weight c may lie an ulp above it.
  int hit = -1;
  double base = 0.0, base_last = 0.0;
  auto step = [&](int s, double x) {
    if (s == lastpos) base_last = c;
    if (hit < 0 && x > 0.0 && c + x > want) hit = s, base = c;
    c += x;
  };
#pragma unroll
  for (int k = 0; k < kKeep; ++k)
    if (s0 + k < s1) step(s0 + k, v[k]);
  for (int s = s0 + kKeep; s < s1; ++s) step(s, __ldcg(part + s));
  if (hit >= 0) atomicMin(&sm.seg, hit);
  __syncthreads();
  const bool none = sm.seg == 0x7fffffff;
  const int seg = none ? lastpos : sm.seg;
  __syncthreads();
  if (none ? lastpos >= s0 && lastpos < s1 : hit == seg) {
    sm.base = none ? base_last : base;
    sm.seg = seg;
  }
  if (tid == 0) {
    if (none && lastpos < 0) sm.seg = -1;
    sm.total = total;
    sm.want = want;
  }
  __syncthreads();
}

template <class TP, class TQ>
__global__ void __launch_bounds__(kVThreads, 4) k_verify(VerifyArgs a) {
  constexpr bool kDraft = !std::is_same<TQ, NoDraft>::value;
  using QT = typename std::conditional<kDraft, TQ, float>::type;
  __shared__ Shared sm;
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  launch_dependents();
  grid_wait();
  // ---- the accepted prefix (every CTA of the sequence finds it for itself) ----
  if (warp == 0) {
    int lo = a.q_off[b], hi = a.q_off[b + 1];
    if (lo < 0 || hi < lo || hi > a.Q) {
      if (lane == 0) set_status(a.status, CSA2_DEV_LENGTH);
      lo = hi = 0;
    }
    const int n = hi - lo;
    int acc = 0, drafted = -1;
    for (int i0 = 0; i0 < n - 1; i0 += 32) {
      const int i = i0 + lane;
      bool ok = false;
      int x = -1;
      if (i < n - 1) {
        const int64_t row = int64_t(lo) + i;
        x = a.tokens[row + 1];
        const float u = a.u[row];
        if (x < 0 || x >= a.V) {
          set_status(a.status, CSA2_DEV_INDEX_RANGE);
        } else {
          const float p = prob(as_float(static_cast<const TP*>(a.target)[row * a.target_stride + x]));
          float q = 1.0f;
          if constexpr (kDraft) q = prob(as_float(static_cast<const QT*>(a.draft)[row * a.draft_stride + x]));
          ok = double(u) * double(q) < double(p);
        }
      }
      const unsigned stop = __ballot_sync(0xffffffffu, i < n - 1 && !ok);
      if (stop) {
        const int l = __ffs(stop) - 1;
        acc = i0 + l;
        drafted = __shfl_sync(0xffffffffu, x, l);
        if (drafted < 0 || drafted >= a.V) drafted = -2;  // rejected, no token of the vocabulary
        break;
      }
      acc = min(n - 1, i0 + 32);
    }
    if (lane == 0) {
      sm.n = n;
      sm.accepted = n > 0 ? acc : 0;
      sm.row0 = lo;
      sm.drafted = drafted;
    }
  }
  __syncthreads();
  const int n = sm.n, acc = sm.accepted, row0 = sm.row0;
  int32_t* out = a.out_tokens ? a.out_tokens + int64_t(b) * a.out_stride : nullptr;
  if (n == 0) {
    if (blockIdx.y == 0) {
      if (tid == 0) {
        a.n_accept[b] = 0;
        a.next_tok[b] = -1;
        if (a.seq_len_out) a.seq_len_out[b] = a.seq_len_in[b];
      }
      if (out)
        for (int j = tid; j < a.out_stride; j += kVThreads) out[j] = -1;
    }
    return;
  }
  // ---- the stop row's segment sums ----
  const bool rejected = acc < n - 1;
  const int64_t row = int64_t(row0) + acc;
  const TP* p = static_cast<const TP*>(a.target) + row * a.target_stride;
  StopRow<TQ> s{nullptr, -1};
  if constexpr (kDraft) {
    if (rejected) s.q = static_cast<const TQ*>(a.draft) + row * a.draft_stride;
  } else {
    if (rejected) s.drafted = sm.drafted;
  }
  const int nseg = (a.V + kSeg - 1) / kSeg;
  double* part = a.part + int64_t(b) * nseg;
  constexpr int kFly = fly<TP, TQ>();
  for (int g = (blockIdx.y * kVWarps + warp) * kFly; g < nseg; g += gridDim.y * kVWarps * kFly)
    segment_sums(p, s, g, nseg, a.V, lane, part);
  __syncthreads();
  if (gridDim.y > 1) {
    if (tid == 0) {
      int old;
      asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(old) : "l"(a.counters + b) : "memory");
      sm.last = old == int(gridDim.y) - 1;
    }
    __syncthreads();
    if (!sm.last) return;
  }
  // ---- the last CTA draws the token ----
  const float r = fmaxf(a.r[b], 0.0f);  // (NaN draws as 0)
  find_segment(part, nseg, r, sm);
  if (!(sm.total > 0.0) && rejected) {
    // p <= q everywhere: the residual is empty, the token comes from p (one
    // CTA sums the row again; the test above fails on p = q only where u >= 1
    // or p(x) = 0, so this is rare)
    s = StopRow<TQ>{nullptr, -1};
    for (int g = warp * kFly; g < nseg; g += kVWarps * kFly) segment_sums(p, s, g, nseg, a.V, lane, part);
    __syncthreads();
    find_segment(part, nseg, r, sm);
  }
  if (warp == 0) {
    int tok = -1;
    if (sm.seg >= 0) tok = segment_find(p, s, sm.seg, a.V, sm.base, sm.want, lane);
    if (lane == 0) {
      if (tok < 0) set_status(a.status, CSA2_DEV_NO_TOKEN);
      a.n_accept[b] = acc;
      a.next_tok[b] = tok;
      if (a.seq_len_out) a.seq_len_out[b] = a.seq_len_in[b] - (n - 1 - acc);
      if (gridDim.y > 1) a.counters[b] = 0;
      if (out && acc < a.out_stride) out[acc] = tok;
      if (out && acc >= a.out_stride) set_status(a.status, CSA2_DEV_LENGTH);
    }
  }
  if (out)
    for (int j = tid; j < a.out_stride; j += kVThreads)
      if (j != acc) out[j] = j < acc ? a.tokens[row0 + 1 + j] : -1;
}

template <class TP, class TQ>
void launch_typed(const VerifyArgs& a, int S, cudaStream_t st) {
  launch_k(k_verify<TP, TQ>, dim3(a.B, S), dim3(kVThreads), 0, st, a);
}
template <class TP>
void launch_target(const VerifyArgs& a, int S, cudaStream_t st) {
  if (!a.draft) return launch_typed<TP, NoDraft>(a, S, st);
  switch (a.draft_type) {
    case CSA2_TYPE_F32: return launch_typed<TP, float>(a, S, st);
    case CSA2_TYPE_BF16: return launch_typed<TP, __nv_bfloat16>(a, S, st);
    default: return launch_typed<TP, __half>(a, S, st);
  }
}

}  // namespace

void launch_verify(const VerifyArgs& a, cudaStream_t st) {
  // CTAs per sequence: as many as its segments keep busy, while those of all
  // sequences run at once (four CTAs per SM): a second wave would repeat the
  // tests' chain of loads (64 rows of 131072: 23.5 us in three waves)
  const int nseg = (a.V + kSeg - 1) / kSeg;
  const int S = a.B > kArrivalCounters
                    ? 1
                    : std::max(1, std::min(4 * num_sms() / a.B, (nseg + kVWarps - 1) / kVWarps));
  switch (a.target_type) {
    case CSA2_TYPE_F32: return launch_target<float>(a, S, st);
    case CSA2_TYPE_BF16: return launch_target<__nv_bfloat16>(a, S, st);
    default: return launch_target<__half>(a, S, st);
  }
}

}  // namespace csa2
