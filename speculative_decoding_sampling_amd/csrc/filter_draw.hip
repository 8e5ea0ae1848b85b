// Filtered distributions and draws with each request's own parameters
// (specv_filter).
//
// A row's kept set is {z >= tau}: top-k, top-p and min-p each keep the tokens
// from some logit up, so the set is the one of the highest of their
// thresholds.
//   tau_k: the largest value with count{z >= tau_k} >= k
//   tau_p: the largest value with mass{z >= tau_p} >= p mass{z >= tau_k}
//   tau_m: the smallest logit whose weight is at least min_p
// with weights w = exp((z - m) / T), m the row's maximum.  A token is therefore
// kept by top-k if fewer than k lie above it, by top-p if those above it hold
// less than p of the mass: both are a search, from the top, for the value at
// which a running count or mass reaches a target.
//
// Numerics.  Weights are float64, good to 1e-13 of their size up to 100 T below the
// maximum (4e-14 the coarser of the two exponentials, the rest the argument's
// roundings).  A mass that decides tau_p is a sum of whole
// multiples of 2^-s, s = 62 - ceil(log2 V) but at most 51: integer sums do not
// depend on their order, so that the histograms may be built with atomics, and n
// tokens are off by at most n 2^-(s+1) of the largest weight.  The sums of a draw are
// float64 in a fixed order.  Probabilities are float64 up to their rounding.
//
// Split.  A row is cut into groups, one 16-byte vector for each lane of a wave,
// and segments of four groups.
//  stats    streams all rows, one wave a segment: each group's largest logit and,
//           where they will be needed, each segment's sum of weights.
//  plan     one workgroup a row: its maximum and total; finishes greedy and
//           unfiltered rows; for the others a bracket [lo, hi) of logits that
//           holds the threshold: from the groups' maxima for top-k, from a sample of
//           the row for top-p, the threshold itself for min-p.
//  collect  one wave a segment, those that reach the bracket: the sum of weights
//           from hi up, and the logits in the bracket.
//  row      one workgroup a row: the threshold among the collected logits, checked
//           against the sums (where the sample misled, the search runs over the
//           row itself, from a bound that holds always), and the draw.
//  probs    writes the probabilities, reading the groups that hold kept tokens.
#include "common.h"
#include "exp64.h"
#include "fp8.h"
#include "grid.h"
#include "specverify_draft.h"
#include "wave_scan.h"

namespace specv {

constexpr int kFdThreads = 1024;
constexpr int kFdWaves = kFdThreads / kWave;
constexpr int kFdBins = 2 * kFdThreads;             // of a round of the search
constexpr int kFdGroups = 4;                        // groups of a segment
constexpr int kFdSegVecs = kFdGroups * kWave;       // 4 KB of logits
constexpr int kFdStatThreads = 256;
constexpr int kFdPlanThreads = 512;
constexpr int kFdCollectBlocks = 8 * 256;           // eight to a CU
constexpr int kFdListCap = 16384;                   // collected logits of a row
constexpr int kFdSampleBins = 2 * kFdPlanThreads;
// The most LDS that a kernel asks for, of the 160 KB of a CU.
constexpr int kFdLds = 159 * 1024;

enum FdKind : int { kFdError = 0, kFdGreedy = 1, kFdDraw = 2 };
// What is left to do for a row after its plan.
enum FdNeed : int { kFdDone = 0, kFdSums = 1, kFdTopK = 2, kFdTopP = 4 };

// A row's plan, and what the kernel that writes the probabilities reads.  The row
// kernel's waves read the plan each for itself, and its first may be done before the
// others have: what it finds has fields of its own, which no wave of it reads.
struct FdPlan {
  int kind;
  int need;
  int best;          // greedy: the token
  float m, tau;      // largest logit; min-p keeps a token iff its logit >= tau
  float lo, hi;      // the bracket
  float bound;       // no token below it is kept by top-p
  uint32_t listed;   // logits collected for the row
  float cut;         // found: a token is kept iff its logit >= cut
  double invT;
  double invS;       // found
  double Z;
};
static_assert(sizeof(FdPlan) == 64, "FdPlan is 64 bytes");

struct FdArgs {
  const void* z;
  long long zsb, zsl;               // strides in elements
  int L, V;
  specv_filters_t f;
  const float* u;
  long long usb, usl;
  int* tokens;
  long long tsb, tsl;
  void* probs;
  long long psb, psl;
  FdPlan* plans;                    // [B L]
  float4* gmax;                     // [B L][nseg] largest logit of each group, NaN for a bad one
  double* ssum;                     // [B L][nseg] weights against the segment's largest logit, then
                                    // (collect) against the row's, from hi up
  uint2* part;                      // [B L][nseg] where a segment's logits of the bracket stand in
                                    // the row's list, and how many they are
  uint2* list;                      // [B L][cap] those logits, with their ids
  int* nitem;                       // what there is to collect: how many segments,
  uint2* items;                     // and which (row; segment and groups as fd_pick has them)
  int nseg, cap;
};

// A row as aligned 16-byte vectors.  The row may start inside the first one:
// vector q holds elements q N - off .. + N - 1.  Vectors inside the row are one
// load; those at its two ends are read element by element, so that nothing
// outside the row is.  Elements outside read as -inf.
template <typename T>
struct FdRow {
  static constexpr int N = Elem<T>::kPerVec;
  const T* p;
  int off, V;
  __device__ __forceinline__ FdRow(const T* row, int V) : p(row), V(V) {
    off = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
  }
  __device__ __forceinline__ int vecs() const { return (V + off + N - 1) / N; }
  __device__ __forceinline__ int first(int q) const { return q * N - off; }
  __device__ __forceinline__ uint4 nothing() const {
    const uint32_t x = N == 4 ? 0xff800000u : 0xff80ff80u;
    return make_uint4(x, x, x, x);
  }
  __device__ __forceinline__ uint4 raw(int q) const {
    const int e = first(q);
    if (e >= 0 && e + N <= V) return *reinterpret_cast<const uint4*>(p + e);
    uint32_t x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = e + i >= 0 && e + i < V ? elem_bits(p, e + i) : neg_inf_bits(T{});
    if constexpr (N == 4) return make_uint4(x[0], x[1], x[2], x[3]);
    else return make_uint4(x[0] | x[1] << 16, x[2] | x[3] << 16, x[4] | x[5] << 16, x[6] | x[7] << 16);
  }
  __device__ __forceinline__ void load(int q, float* out) const { unpack(raw(q), out, T{}); }
  // Whether all of a segment's vectors lie in the row: its loads then need no
  // bounds, each of which would part them.
  __device__ __forceinline__ bool whole(int seg) const {
    return first(seg * kFdSegVecs) >= 0 && first((seg + 1) * kFdSegVecs) <= V;
  }
};

// The parameters of a request.
struct FdParams {
  float T, p, mp;
  int k;
  bool ok;
};
__device__ __forceinline__ FdParams fd_params(const specv_filters_t& f, int b) {
  FdParams r;
  r.T = f.temperature_array ? f.temperature_array[b] : f.temperature;
  r.k = f.top_k_array ? f.top_k_array[b] : f.top_k;
  r.p = f.top_p_array ? f.top_p_array[b] : f.top_p;
  r.mp = f.min_p_array ? f.min_p_array[b] : f.min_p;
  r.ok = r.T >= 0.f && r.T <= 3.402823466e38f && r.k >= 0 && r.p > 0.f && r.p <= 1.f &&
         r.mp >= 0.f && r.mp <= 1.f;                 // false for NaN
  return r;
}

// Whether a row's sums of weights are wanted: for the mass that top-p is a part
// of, or for a draw from all tokens.
__device__ __forceinline__ bool fd_wants_sums(const FdParams& f, int V) {
  return f.ok && f.T > 0.f && (f.k == 0 || f.k >= V) && (f.p < 1.f || f.mp == 0.f);
}

// Weights exp((z - m) / T), at most 1: exp64.h's method and table.  The entries
// have their index taken from the exponent's place, so that adding k there leaves
// 2^(k / N) in one operation.  What would be below e^-700 stays there, -inf too.
//
// A weight of at most kFdNothing counts as nothing, in a segment's mass too: it has
// one only where a token in it counts, however many others there are (at u = 0 a draw
// ends in the first that has one).
constexpr double kFdNothing = 1e-290;
template <int BITS>                                  // of the 9 of the table's index
__device__ __forceinline__ double fd_table_entry(int i) {
  const double v = kExp64Table[i << (SPECV_EXP64_LOG2N - BITS)];
  return __hiloint2double(__double2hiint(v) - (i << (20 - BITS)), __double2loint(v));
}

// The sum of the weights at or above tau that count.  No branches: the weights'
// chains of dependent operations and table reads overlap.
template <typename E, int N>
__device__ __forceinline__ double fd_sum(const E& weight, const float (&v)[N], float tau) {
  double w[N], s = 0.0;
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] = weight(v[i]);
#pragma unroll
  for (int i = 0; i < N; ++i) s += v[i] >= tau && w[i] > kFdNothing ? w[i] : 0.0;
  return s;
}

// With the table of 512 in LDS.
template <int NT>
__device__ __forceinline__ void fd_stage_table(double* tbl) {
  for (int i = threadIdx.x; i < SPECV_EXP64_N; i += NT) tbl[i] = fd_table_entry<SPECV_EXP64_LOG2N>(i);
}
struct FdExp {
  double m, invT;
  const double* tbl;
  __device__ __forceinline__ FdExp(double m, double invT, const double* tbl)
      : m(m), invT(invT), tbl(tbl) {}
  // x = (z - m) / T, and its weight
  __device__ __forceinline__ double arg(float z) const { return ((double)z - m) * invT; }
  __device__ __forceinline__ double of(double x) const {
    x = fmax(x, -700.0);
    const double t = fma(x, SPECV_EXP64_INV_L, SPECV_EXP64_SHIFT);
    const double r = fma(-(t - SPECV_EXP64_SHIFT), SPECV_EXP64_L, x);
    double q = fma(r, SPECV_EXP64_C3, 0.5);
    q = fma(r, q, 1.0);
    const int k = __double2loint(t);
    const double e = tbl[k & (SPECV_EXP64_N - 1)];
    const double tj = __hiloint2double(__double2hiint(e) + (k << (20 - SPECV_EXP64_LOG2N)), __double2loint(e));
    return fma(tj, r * q, tj);
  }
  __device__ __forceinline__ double operator()(float z) const { return of(arg(z)); }
};

// With every eighth entry of the table, one in each lane of a wave, read across
// lanes: nothing to stage and no barrier, one degree more (truncation r^5 / 120 <
// 4e-14).  All lanes call it together: a lane that is off gives zeros.
struct FdWaveExp {
  double m, invT;
  int lo, hi;
  __device__ __forceinline__ FdWaveExp(double m, double invT) : m(m), invT(invT) {
    const double v = fd_table_entry<6>(threadIdx.x % kWave);
    lo = __double2loint(v);
    hi = __double2hiint(v);
  }
  __device__ __forceinline__ double operator()(float z) const {
    const double x = fmax(((double)z - m) * invT, -700.0);
    const double t = fma(x, SPECV_EXP64_INV_L / 8, SPECV_EXP64_SHIFT);
    const double r = fma(-(t - SPECV_EXP64_SHIFT), SPECV_EXP64_L * 8, x);
    double q = fma(r, 1.0 / 24, SPECV_EXP64_C3);
    q = fma(r, q, 0.5);
    q = fma(r, q, 1.0);
    const int k = __double2loint(t);                 // (lane k % 64)
    const double tj = __hiloint2double(__builtin_amdgcn_ds_bpermute(k << 2, hi) + (k << 14),
                                       __builtin_amdgcn_ds_bpermute(k << 2, lo));
    return fma(tj, r * q, tj);
  }
};

// Weights as whole multiples of 2^-s: the sum with 2^52 leaves them in its low
// bits, rounded to nearest.
__device__ __forceinline__ double fd_unit(int V) {
  return __hiloint2double((1023 + min(62 - (32 - __clz((V - 1) | 1)), 51)) << 20, 0);
}
__device__ __forceinline__ unsigned long long fd_fixed(double w, double unit) {
  return (unsigned long long)__double_as_longlong(fma(w, unit, 4503599627370496.0)) & 0xfffffffffffffull;
}

// A row's groups: one wave a segment.  Without sums it reads 5.8 TB/s (27 us for
// 156 MB); float64 weights of all tokens add 10 us there.  (A table staged for each
// workgroup cost 7 us more; workgroups that stay and fetch ahead, or neighbouring
// ones on different rows, read slower.)
template <typename T>
__global__ __launch_bounds__(kFdStatThreads) void filter_stats_kernel(FdArgs a, int nblk) {
  constexpr int N = FdRow<T>::N;
  const int r = blockIdx.x / nblk, b = r / a.L, l = r % a.L;
  const int lane = threadIdx.x % kWave;
  const int g = (blockIdx.x % nblk) * (kFdStatThreads / kWave) +
                __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const FdRow<T> row(static_cast<const T*>(a.z) + (size_t)b * a.zsb + (size_t)l * a.zsl, a.V);
  uint4 raw[kFdGroups];
  if (row.whole(g)) {
#pragma unroll
    for (int j = 0; j < kFdGroups; ++j)
      raw[j] = *reinterpret_cast<const uint4*>(row.p + row.first(g * kFdSegVecs + j * kWave + lane));
  } else {
#pragma unroll
    for (int j = 0; j < kFdGroups; ++j) raw[j] = row.raw(g * kFdSegVecs + j * kWave + lane);
  }
  const FdParams f = fd_params(a.f, b);
  const bool sums = fd_wants_sums(f, a.V);
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.nitem = 0;     // for the plans, which follow
  if (g >= a.nseg) return;
  float top[kFdGroups], m = -INFINITY;
#pragma unroll
  for (int j = 0; j < kFdGroups; ++j) {
    float v[N];
    unpack(raw[j], v, T{});
    bool fine = true;
    top[j] = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      top[j] = fmaxf(top[j], v[i]);
      fine = fine && v[i] < INFINITY;                // neither NaN nor +inf
    }
    top[j] = wave_max(top[j]);
    m = fmaxf(m, top[j]);
    if (!__all(fine)) top[j] = __builtin_nanf("");
  }
  double w = 0.0;
  if (sums && m > -INFINITY) {
    const FdWaveExp e(m, 1.0 / (double)f.T);
#pragma unroll
    for (int j = 0; j < kFdGroups; ++j) {
      float v[N];
      unpack(raw[j], v, T{});
#pragma unroll
      for (int i = 0; i < N; ++i) w += e(v[i]);
    }
    w = wave_sum(w);
  }
  if (lane == 0) {
    a.gmax[(size_t)r * a.nseg + g] = make_float4(top[0], top[1], top[2], top[3]);
    if (sums) a.ssum[(size_t)r * a.nseg + g] = w;
  }
}

// LDS of the plan and row kernels; behind it, sized by the call: seg[nseg]
// (double), picks[nseg] (uint32) and, for the row kernel, list[cap] (float).
struct FdShared {
  double tbl[SPECV_EXP64_N];
  unsigned long long mass[kFdBins];
  uint32_t count[kFdBins];
  unsigned long long wave_u64[kFdWaves];
  uint32_t wave_u32[kFdWaves];
  int found[2 * kFdGroups];
  uint32_t npick;
  unsigned long long above;
};

template <int WAVES>
__device__ __forceinline__ uint32_t fd_block_max(FdShared& s, uint32_t v) {
  v = wave_max_u32(v);
  if (threadIdx.x % kWave == 0) s.wave_u32[threadIdx.x / kWave] = v;
  __syncthreads();
  uint32_t r = s.wave_u32[0];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) r = max(r, s.wave_u32[w]);
  __syncthreads();
  return r;
}
// The sum of all threads' values before this one's, and of all.
template <int WAVES>
__device__ __forceinline__ unsigned long long fd_block_scan(FdShared& s, unsigned long long v,
                                                            unsigned long long& total) {
  const unsigned long long incl = wave_incl_scan_u64(v);
  const int wave = threadIdx.x / kWave;
  if (threadIdx.x % kWave == kWave - 1) s.wave_u64[wave] = incl;
  __syncthreads();
  unsigned long long before = incl - v, sum = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    const unsigned long long x = s.wave_u64[w];
    if (w < wave) before += x;
    sum += x;
  }
  __syncthreads();
  total = sum;
  return before;
}
template <int WAVES>
__device__ __forceinline__ double fd_block_sum(FdShared& s, double v) {
  v = wave_sum(v);
  if (threadIdx.x % kWave == 0) s.wave_u64[threadIdx.x / kWave] = __double_as_longlong(v);
  __syncthreads();
  double r = 0.0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) r += __longlong_as_double(s.wave_u64[w]);
  __syncthreads();
  return r;
}

// Order-preserving key of a logit: 32 bits, or the 16 that a bfloat16 one has.
// unkey of a 16-bit one is a threshold that parts it from the value below.
template <typename T>
__device__ __forceinline__ uint32_t fd_key(float f) {
  return sizeof(T) == 2 ? fkey(f) >> 16 : fkey(f);
}
template <typename T>
__device__ __forceinline__ float fd_unkey(uint32_t k) {
  return unkey(sizeof(T) == 2 ? k << 16 : k);
}
// The logit of a key.
template <typename T>
__device__ __forceinline__ float fd_value(uint32_t k) {
  return unkey(sizeof(T) == 4 ? k : k < 0x8000u ? k << 16 | 0xffffu : k << 16);
}
template <typename T>
constexpr uint32_t kFdLowest = sizeof(T) == 2 ? (kNegInfKey >> 16) + 1 : kNegInfKey + 1;

// Which of a segment's groups reach tau, as four bits.
__device__ __forceinline__ uint32_t fd_reach(const float4& t, float tau) {
  return (t.x >= tau ? 1u : 0u) | (t.y >= tau ? 2u : 0u) | (t.z >= tau ? 4u : 0u) |
         (t.w >= tau ? 8u : 0u);
}

// The segments that hold a group reaching tau, in any order: the segment's
// number above the four bits.
__device__ __forceinline__ uint32_t fd_pick(FdShared& s, uint32_t* picks, const float4* gmax,
                                            int nseg, float tau) {
  if (threadIdx.x == 0) s.npick = 0;
  __syncthreads();
  for (int g = threadIdx.x; g < nseg; g += kFdThreads) {
    const uint32_t bits = fd_reach(gmax[g], tau);
    if (bits) picks[atomicAdd(&s.npick, 1u)] = (uint32_t)g << 4 | bits;
  }
  __syncthreads();
  return s.npick;
}

// The vectors of a picked segment, those of groups that were not picked as -inf.
// Their loads repeat a picked group's, so that all are in flight at once.
template <typename T>
__device__ __forceinline__ void fd_load(const FdRow<T>& row, uint32_t pick, int lane,
                                        float (&v)[kFdGroups][FdRow<T>::N]) {
  const int q = (int)(pick >> 4) * kFdSegVecs + lane, any = __ffs((int)(pick & 15u)) - 1;
#pragma unroll
  for (int j = 0; j < kFdGroups; ++j) row.load(q + (pick >> j & 1u ? j : any) * kWave, v[j]);
#pragma unroll
  for (int j = 0; j < kFdGroups; ++j)
    if (!(pick >> j & 1u)) {
#pragma unroll
      for (int i = 0; i < FdRow<T>::N; ++i) v[j][i] = -INFINITY;
    }
}

// The logits that a search is about: the list, or the picked segments again.
template <typename T>
struct FdSource {
  FdRow<T> row;
  const uint32_t* picks;
  uint32_t npick;
  const float* list;
  uint32_t n;
  bool listed;
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    if (listed) {
      for (uint32_t i = threadIdx.x; i < n; i += kFdThreads) f(list[i]);
    } else {
      for (uint32_t e = threadIdx.x / kWave; e < npick; e += kFdWaves) {
        float v[kFdGroups][FdRow<T>::N];
        fd_load(row, picks[e], threadIdx.x % kWave, v);
#pragma unroll
        for (int j = 0; j < kFdGroups; ++j)
#pragma unroll
          for (int i = 0; i < FdRow<T>::N; ++i) f(v[j][i]);
      }
    }
  }
};

// What a search finds: the key of the lowest kept value, and whether the target
// is reached there (if not all of the bracket is kept).
struct FdFound {
  uint32_t low;
  bool reached;
};

// The search for a threshold, by a block of THREADS: a value is kept if what lies
// above it (`above` before the bracket) is below the target.  Each round sorts
// the keys of the bracket [lo, hi] into bins by count, and by mass where that is
// what the target is about, finds the bin where the running sum from the top
// reaches the target and goes on inside it, until it holds one value (or one key:
// ties go together).  A BOUND takes one round.  Where a bin is one key, its mass is
// its count times that key's weight: bfloat16 logits share few keys, whose masses
// would all be added at the same places.
template <int THREADS, bool MASS, bool BOUND, typename T, typename Each, typename W>
__device__ __forceinline__ FdFound fd_search(FdShared& s, uint32_t lo, uint32_t hi,
                                             unsigned long long above, double target, Each each,
                                             W weight) {
  constexpr int kBins = 2 * THREADS, kBits = THREADS == 1024 ? 11 : 10, kWaves = THREADS / kWave;
  static_assert(kBins == 1 << kBits && kBins <= kFdBins, "two bins to a thread");
  const int t = threadIdx.x, lane = t % kWave, wave = t / kWave;
  bool reached = false;
  for (bool first_round = true;; first_round = false) {
    const int sh = max(32 - __clz((int)((hi - lo) | 1u)) - kBits, 0);
    for (int i = t; i < kBins; i += THREADS) {
      s.count[i] = 0;
      if (MASS && sh) s.mass[i] = 0;
    }
    __syncthreads();
    each([&](uint32_t key, float z) {
      if (key >= lo && key <= hi) {
        const int b = (int)((key - lo) >> sh);
        atomicAdd(&s.count[b], 1u);
        if (MASS && sh) atomicAdd(&s.mass[b], weight(z));
      }
    });
    __syncthreads();
    // thread t owns bins top - 2 t and the one below: running sums from the top
    const int b0 = kBins - 1 - 2 * t, b1 = b0 - 1;
    const uint32_t c0 = s.count[b0], c1 = s.count[b1];
    unsigned long long x0 = c0, x1 = c1;
    if (MASS) {
      x0 = sh ? s.mass[b0] : c0 ? c0 * weight(fd_value<T>(lo + b0)) : 0ull;
      x1 = sh ? s.mass[b1] : c1 ? c1 * weight(fd_value<T>(lo + b1)) : 0ull;
    }
    const unsigned long long incl = wave_incl_scan_u64(x0 + x1);
    if (lane == kWave - 1) s.wave_u64[wave] = incl;
    __syncthreads();
    unsigned long long before = above + incl - (x0 + x1);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) before += w < wave ? s.wave_u64[w] : 0ull;
    // the lowest bin that holds something and has less than the target above:
    // its number, in bit 31 whether it holds one value only, in bit 30 whether
    // the target is reached with it
    uint32_t mine = 0xffffffffu;
    unsigned long long mine_above = 0;
    auto take = [&](int bin, uint32_t c, unsigned long long x, unsigned long long over) {
      if (c == 0 || !((double)over < target)) return;
      mine = (uint32_t)bin | (c == 1u ? 1u << 31 : 0u) | ((double)(over + x) >= target ? 1u << 30 : 0u);
      mine_above = over;
    };
    take(b0, c0, x0, before);
    take(b1, c1, x1, before + x0);
    const uint64_t some = __ballot(mine != 0xffffffffu);
    const int src = some ? 63 - __clzll((long long)some) : 0;
    if (lane == src) s.wave_u32[wave] = mine;
    __syncthreads();
    uint32_t found = 0xffffffffu;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const uint32_t x = s.wave_u32[w];
      if (x != 0xffffffffu) found = x;
    }
    if (found != 0xffffffffu && mine == found) s.above = mine_above;
    __syncthreads();
    if (found == 0xffffffffu) return {lo, reached};  // nothing in the bracket
    if (first_round) reached = found >> 30 & 1u;
    const uint32_t base = lo + ((found & (kFdBins - 1)) << sh);
    above = s.above;
    if (BOUND || sh == 0 || found >> 31) return {base, reached};
    lo = base;
    hi = base + ((1u << sh) - 1u);
  }
}

// The smallest float whose weight is at least mp, in (0, 1]: a search over keys
// in which each lane of a wave tries one of 64, first those around m + T log mp,
// then, where that is too far off, of all (6 rounds for 32 bits).
__device__ __forceinline__ float fd_min_p_threshold(float m, float T, const FdExp& e, float mp) {
  const int lane = threadIdx.x % kWave;
  uint32_t lo = kNegInfKey + 1, hi = fkey(m);        // the maximum itself has weight 1
  auto weighs = [&](uint32_t key) { return e(unkey(key)) >= (double)mp; };
  const uint32_t guess = fkey((float)fmax((double)m + (double)T * log((double)mp), -3e38));
  const uint32_t near = min(max(guess + lane - 32u, lo), hi);
  const uint64_t yes = __ballot(weighs(near));
  if (yes != 0 && !(yes & 1ull)) return unkey((uint32_t)lane_value((int)near, __ffsll((unsigned long long)yes) - 1));
  while (lo < hi) {
    const uint32_t step = (hi - lo) / kWave + 1;
    auto key = [&](int i) { return lo + min((uint32_t)i * step, hi - lo); };
    const uint64_t some = __ballot(weighs(key(lane)));
    if (some == 0) {
      lo = key(kWave - 1) + 1;
    } else {
      const int i = __ffsll((unsigned long long)some) - 1;
      hi = key(i);
      if (i > 0) lo = key(i - 1) + 1;
    }
  }
  return unkey(hi);
}

// A short list's threshold and draw, by one wave without barriers: lane i holds
// entry i of n.  The entries are all the tokens that top-k and top-p are about
// (want_k, want_p: the filters that are on; target: top-p's, where top-k is off).
struct FdShort {
  bool reached;      // top-p's target, with the whole list
  bool kept;         // this lane's entry
};
__device__ __forceinline__ FdShort fd_short(uint32_t key, unsigned long long mass, int n, bool want_k,
                                            int k, bool want_p, double p, double target) {
  const int lane = threadIdx.x % kWave;
  FdShort r = {true, lane < n};
  if (want_k) {
    int above = 0;
    for (int j = 0; j < n; ++j) above += (uint32_t)lane_value((int)key, j) > key ? 1 : 0;
    r.kept = r.kept && above < k;
  }
  if (want_p) {
    const unsigned long long mine = r.kept ? mass : 0ull;
    const int lo = (int)(uint32_t)mine, hi = (int)(uint32_t)(mine >> 32);
    unsigned long long above = 0, all = 0;
    for (int j = 0; j < n; ++j) {
      const unsigned long long w =
          (unsigned long long)(uint32_t)lane_value(hi, j) << 32 | (uint32_t)lane_value(lo, j);
      all += w;
      above += (uint32_t)lane_value((int)key, j) > key ? w : 0ull;
    }
    if (want_k) target = p * (double)all;
    r.reached = (double)all >= target;
    r.kept = r.kept && (double)above < target;
  }
  return r;
}
// The token drawn at u from the kept entries in order of their ids (their sum in
// S), -1 where none is wanted.
__device__ __forceinline__ int fd_short_draw(bool kept, int id, double w, int n, bool token, float u,
                                             double& S) {
  const int lane = threadIdx.x % kWave;
  const uint64_t in = __ballot(kept);
  const uint32_t mine = kept ? (uint32_t)id : 0xffffffffu;
  int rank = 0;
  for (int j = 0; j < n; ++j) rank += (uint32_t)lane_value((int)mine, j) < mine ? 1 : 0;
  // the others behind them: every lane's entry moves to a lane of its own
  if (!kept) rank = __popcll(in) + __popcll(~in & ((1ull << lane) - 1ull));
  w = kept ? w : 0.0;
  const int lo = __builtin_amdgcn_ds_permute(rank * 4, __double2loint(w));
  const int hi = __builtin_amdgcn_ds_permute(rank * 4, __double2hiint(w));
  id = __builtin_amdgcn_ds_permute(rank * 4, id);
  w = __hiloint2double(hi, lo);
  const double incl = wave_incl_scan(w);
  S = lane_value(incl, kWave - 1);
  if (!token) return -1;
  const uint64_t over = __ballot(w > kFdNothing && incl > (double)u * S), some = __ballot(w > kFdNothing);
  return lane_value(id, over ? __ffsll((unsigned long long)over) - 1 : 63 - __clzll((long long)some));
}

// The draw from a row's segment masses seg (in LDS), by the whole block: S their
// sum, and where a token is wanted the first whose running sum exceeds u S, or
// where rounding leaves none the last with weight.  Every wave finds the segment;
// the first four take one of its groups each.
template <typename T>
__device__ __forceinline__ int fd_draw(FdShared& s, const FdRow<T>& row, const double* seg, int nseg,
                                       bool token, float u, float tau, const FdExp& weight,
                                       double& S) {
  constexpr int N = FdRow<T>::N;
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  // lane l sums segments l per .. l per + per - 1
  const int per = (nseg + kWave - 1) / kWave;
  const int g0 = min(lane * per, nseg), g1 = min(g0 + per, nseg);
  double mine = 0.0;
  for (int g = g0; g < g1; ++g) mine += seg[g];
  const double incl = wave_incl_scan(mine);
  S = lane_value(incl, kWave - 1);
  if (!token) return -1;
  const double target = (double)u * S;
  double run = wave_shr1(incl), at = 0.0, last_at = 0.0;
  int pick = -1, last = -1;
  for (int g = g0; g < g1; ++g) {
    const double w = seg[g];
    if (w > kFdNothing) {
      last = g;
      last_at = run;
      if (pick < 0 && run + w > target) {
        pick = g;
        at = run;
      }
    }
    run += w;
  }
  const uint64_t over = __ballot(pick >= 0), some = __ballot(last >= 0);
  const int src = over ? __ffsll((unsigned long long)over) - 1 : 63 - __clzll((long long)some);
  const int g = lane_value(over ? pick : last, src);
  const double base = lane_value(over ? at : last_at, src);
  // inside it: sums of the groups, then over lanes, then over a lane's elements
  const int q = g * kFdSegVecs + wave * kWave + lane, e = row.first(q);
  double w[N], sum = 0.0;
  if (wave < kFdGroups) {
    float v[N];
    row.load(q, v);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      w[i] = v[i] >= tau && v[i] > -INFINITY ? weight(v[i]) : 0.0;
      sum += w[i];
    }
    sum = wave_incl_scan(sum);
    if (lane == kWave - 1) s.wave_u64[wave] = __double_as_longlong(sum);
  }
  __syncthreads();
  if (wave < kFdGroups) {
    double here = base;
    for (int i = 0; i < wave; ++i) here += __longlong_as_double(s.wave_u64[i]);
    here += wave_shr1(sum);
    int first = -1, tail = -1;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      here += w[i];
      if (w[i] > kFdNothing) {
        tail = e + i;
        if (first < 0 && here > target) first = tail;
      }
    }
    const uint64_t hit = __ballot(first >= 0), any = __ballot(tail >= 0);
    if (lane == 0) {
      s.found[wave] = hit ? lane_value(first, __ffsll((unsigned long long)hit) - 1) : -1;
      s.found[kFdGroups + wave] = any ? lane_value(tail, 63 - __clzll((long long)any)) : -1;
    }
  }
  __syncthreads();
  int y = -1, end = -1;
#pragma unroll
  for (int i = 0; i < kFdGroups; ++i) {
    if (y < 0) y = s.found[i];
    if (s.found[kFdGroups + i] >= 0) end = s.found[kFdGroups + i];
  }
  return y < 0 ? end : y;
}

// Masses put into bins of their distance from the maximum (so many bins to a unit
// of (m - z) / T), past the last into tail.
template <int N>
__device__ __forceinline__ void fd_spread(FdShared& s, const FdExp& weight, const float (&v)[N],
                                          double unit, double bins, int nbin,
                                          unsigned long long& tail) {
  unsigned long long w[N];
  double b[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const double x = weight.arg(v[i]);
    w[i] = fd_fixed(weight.of(x), unit);
    b[i] = -x * bins;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (b[i] < nbin) atomicAdd(&s.mass[(int)b[i]], w[i]);
    else tail += w[i];
  }
}

// The bracket of a top-p threshold from a sample of the row.  With M(x) the mass
// of the tokens x or more below the maximum (in units of T), the threshold lies
// where M falls below B = (1 - p) Z.  The sample gives M as scale sum w; tokens
// that weigh at most w = exp(-x) leave it uncertain by some sqrt(scale w M), and by
// a few of those tokens where there are few: lo is the highest x at which M and
// four deviations and eight tokens are below B, hi the lowest at which M less
// those is above it.  Nothing rests on it but the time: the row kernel checks.
template <typename T>
__device__ __forceinline__ void fd_sample(FdShared& s, const FdRow<T>& row, const FdExp& weight,
                                          double T64, double B, double width, double unit, float& lo,
                                          float& hi) {
  constexpr int N = FdRow<T>::N, kChunk = 16, kWaves = kFdPlanThreads / kWave;
  const int t = threadIdx.x, chunks = (row.vecs() + kChunk - 1) / kChunk;
  constexpr int kChunks = 8192 / (kChunk * N);       // 8192 tokens, in pieces of 256 bytes
  const int n = min(chunks, kChunks);
  for (int i = t; i < kFdSampleBins; i += kFdPlanThreads) s.mass[i] = 0;
  __syncthreads();
  const double per = kFdSampleBins / width;
  unsigned long long tail = 0;
  constexpr int kSweeps = kChunks * kChunk / kFdPlanThreads;
  float v[kSweeps][N];
#pragma unroll
  for (int i = 0; i < kSweeps; ++i) {
    const int c = i * (kFdPlanThreads / kChunk) + t / kChunk;
    const int q = (int)((long long)c * chunks / n) * kChunk + t % kChunk;
    row.load(c < n ? q : row.vecs(), v[i]);          // past the row: -inf
  }
#pragma unroll
  for (int i = 0; i < kSweeps; ++i) fd_spread(s, weight, v[i], unit, per, kFdSampleBins, tail);
  unsigned long long all;
  fd_block_scan<kWaves>(s, tail, all);
  // thread t owns bins top - 2 t and the one below: sums from the far end
  const int b0 = kFdSampleBins - 1 - 2 * t, b1 = b0 - 1;
  const unsigned long long x0 = s.mass[b0], x1 = s.mass[b1];
  unsigned long long ignore;
  const unsigned long long before = fd_block_scan<kWaves>(s, x0 + x1, ignore) + all;
  const double scale = (double)chunks / n / unit;
  uint32_t low = 0, high = 0;                        // ~b of lo, b + 1 of hi
  auto look = [&](int b, unsigned long long sum) {   // tokens from bin b on
    const double M = scale * (double)sum, q = scale * unit * weight.of(-b / per);
    const double off = 4.0 * sqrt(q * M) + 8.0 * q;
    if (M + off <= B) low = max(low, ~(uint32_t)b);
    if (M - off >= B) high = max(high, (uint32_t)b + 1u);
  };
  look(b0, before + x0);
  look(b1, before + x0 + x1);
  low = fd_block_max<kWaves>(s, low);
  high = fd_block_max<kWaves>(s, high);
  if (low) lo = fmaxf(lo, (float)(weight.m - T64 * ((double)~low / per)));
  if (high) hi = (float)(weight.m - T64 * ((double)(high - 1u) / per));
}

// One workgroup a row: the plan.  A chain of short phases: 10 us for 64 or 256 rows
// (a row's maxima, its total, the sample's loads and table reads, two scans of its
// bins), half of it the sample.
template <typename T>
__global__ __launch_bounds__(kFdPlanThreads) void filter_plan_kernel(FdArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
  FdShared& s = *reinterpret_cast<FdShared*>(dyn);
  double* seg = reinterpret_cast<double*>(dyn + sizeof(FdShared));
  uint32_t* picks = reinterpret_cast<uint32_t*>(seg + a.nseg);
  constexpr int N = FdRow<T>::N, kWaves = kFdPlanThreads / kWave;
  const int r = blockIdx.x, b = r / a.L, l = r % a.L, t = threadIdx.x;
  const int lane = t % kWave, wave = t / kWave;
  const float4* gmax = a.gmax + (size_t)r * a.nseg;
  const double* ssum = a.ssum + (size_t)r * a.nseg;
  const float u = a.tokens ? a.u[(size_t)b * a.usb + (size_t)l * a.usl] : 0.f;
  const FdParams f = fd_params(a.f, b);
  fd_stage_table<kFdPlanThreads>(s.tbl);
  const FdRow<T> row(static_cast<const T*>(a.z) + (size_t)b * a.zsb + (size_t)l * a.zsl, a.V);

  // the row's largest logit; NaN or +inf anywhere shows as the largest key
  uint32_t top = 0;
  for (int g = t; g < a.nseg; g += kFdPlanThreads) {
    const float4 x = gmax[g];
    const float big = fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w));
    const bool fine = x.x < INFINITY && x.y < INFINITY && x.z < INFINITY && x.w < INFINITY;
    top = max(top, fine ? fkey(big) : 0xffffffffu);
  }
  top = fd_block_max<kWaves>(s, top);
  const bool ok = f.ok && top > kNegInfKey && top != 0xffffffffu && u >= 0.f && u < 1.f;
  const float m = ok ? unkey(top) : 0.f;
  FdPlan plan = {kFdError, kFdDone, -1, m, -INFINITY, -INFINITY, INFINITY, -INFINITY, 0u, -INFINITY, 0.0, 0.0, 0.0};
  int y = -1;
  if (ok && f.T == 0.f) {
    // the first group that reaches the maximum, and in it the first token
    uint32_t first = 0;
    for (int g = t; g < a.nseg; g += kFdPlanThreads) {
      const uint32_t bits = fd_reach(gmax[g], m);
      if (bits) first = max(first, ~(uint32_t)(g * kFdGroups + __ffs((int)bits) - 1));
    }
    first = ~fd_block_max<kWaves>(s, first);
    if (wave == 0) {
      float v[N];
      const int q = (int)first * kWave + lane;
      row.load(q, v);
      int at = -1;
#pragma unroll
      for (int i = N - 1; i >= 0; --i)
        if (v[i] == m) at = row.first(q) + i;
      y = lane_value(at, __ffsll((unsigned long long)__ballot(at >= 0)) - 1);
    }
    plan.kind = kFdGreedy;
    plan.best = y;
  } else if (ok) {
    plan.kind = kFdDraw;
    plan.invT = 1.0 / (double)f.T;
    const FdExp weight(m, plan.invT, s.tbl);
    const bool by_k = f.k > 0 && f.k < a.V, by_p = f.p < 1.f;
    if (fd_wants_sums(f, a.V)) {
      double mine = 0.0;
      for (int g = t; g < a.nseg; g += kFdPlanThreads) {
        const float4 x = gmax[g];
        const float big = fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w));
        const double top = weight(big), w = top > kFdNothing ? ssum[g] * top : 0.0;
        seg[g] = w;
        mine += w;
      }
      plan.Z = fd_block_sum<kWaves>(s, mine);
    }
    if (!by_k && !by_p && f.mp == 0.f) {
      double S;
      y = fd_draw(s, row, seg, a.nseg, a.tokens != nullptr, u, -INFINITY, weight, S);
      plan.invS = 1.0 / S;
    } else {
      if (f.mp > 0.f) plan.tau = fd_min_p_threshold(m, f.T, weight, f.mp);
      plan.need = by_k ? kFdTopK | (by_p ? kFdTopP : 0) : by_p ? kFdTopP : kFdSums;
      if (by_k) {
        // at least k tokens reach the k-th largest of the groups' maxima
        if (f.k <= a.nseg * kFdGroups) {
          auto maxima = [&](auto put) {
            for (int g = t; g < a.nseg; g += kFdPlanThreads) {
              const float4 x = gmax[g];
              put(fd_key<T>(x.x), x.x);
              put(fd_key<T>(x.y), x.y);
              put(fd_key<T>(x.z), x.z);
              put(fd_key<T>(x.w), x.w);
            }
          };
          // (from the lowest of these, so that the bins are fine)
          uint32_t least = 0;
          maxima([&](uint32_t key, float x) { least = max(least, x > -INFINITY ? ~key : 0u); });
          least = ~fd_block_max<kWaves>(s, least);
          const FdFound k = fd_search<kFdPlanThreads, false, true, T>(
              s, least, fd_key<T>(m), 0, (double)f.k, maxima, [](float) { return 0ull; });
          if (k.reached) plan.lo = fd_unkey<T>(k.low);
        }
        // top-p is a part of the whole top-k set's mass
        if (!by_p) plan.lo = fmaxf(plan.lo, plan.tau);
      } else if (by_p) {
        // Tokens below w hold less than V w: with V w = (1 - p) Z all that
        // top-p keeps lies above w.  (Both sides with room for rounding.)
        const double B = (1.0 - (double)f.p) * plan.Z, width = 1e-6 - log(B / a.V);
        const double z = (double)m - (double)f.T * width;
        const float bound = (float)(z - fabs(z) * 1e-6);
        if (bound > -3e38f) plan.bound = bound;
        plan.lo = plan.bound;
        if (width > 0.0)
          fd_sample(s, row, weight, (double)f.T, B, width, fd_unit(a.V), plan.lo, plan.hi);
        // what min-p drops need not be looked at
        plan.lo = fmaxf(plan.lo, plan.tau);
        plan.hi = fmaxf(plan.hi, plan.lo);
      } else {
        plan.lo = plan.hi = plan.tau;
      }
    }
  }
  if (t == 0) {
    a.plans[r] = plan;
    if (a.tokens) a.tokens[(size_t)b * a.tsb + (size_t)l * a.tsl] = y;
    s.npick = 0;
  }
  if (plan.need == kFdDone) return;
  // the segments that reach the bracket; the others have nothing
  __syncthreads();
  for (int g = t; g < a.nseg; g += kFdPlanThreads) {
    const float4 x = gmax[g];
    const bool some = fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)) > -INFINITY;
    const uint32_t bits = some ? fd_reach(x, plan.lo) : 0u;
    if (bits) {
      picks[atomicAdd(&s.npick, 1u)] = (uint32_t)g << 4 | bits;
    } else {
      a.ssum[(size_t)r * a.nseg + g] = 0.0;
      a.part[(size_t)r * a.nseg + g] = make_uint2(0u, 0u);
    }
  }
  __syncthreads();
  if (t == 0) s.above = (unsigned long long)atomicAdd(a.nitem, (int)s.npick);
  __syncthreads();
  for (uint32_t i = t; i < s.npick; i += kFdPlanThreads) a.items[s.above + i] = make_uint2((uint32_t)r, picks[i]);
}

// One wave a segment that reaches its row's bracket: as many waves as the chip
// holds take them in turn from the plans' list, as rows differ in what they leave
// (256 x 152064 float32, filters mixed: 73 us for the call at the time, 77 with one
// wave for every segment, most of which ended at once).  12 us there, 10 at 64 x
// 128256 bfloat16: two dependent loads, then the logits.
template <typename T>
__global__ __launch_bounds__(kFdStatThreads) void filter_collect_kernel(FdArgs a) {
  constexpr int N = FdRow<T>::N, kWaves = kFdStatThreads / kWave;
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int items = *a.nitem;
  if ((int)blockIdx.x * kWaves >= items) return;
  for (int i = blockIdx.x * kWaves + wave; i < items; i += gridDim.x * kWaves) {
    const uint2 item = a.items[i];
    const int r = (int)item.x, b = r / a.L, l = r % a.L, g = (int)(item.y >> 4);
    const size_t at = (size_t)r * a.nseg + g;
    FdPlan* plan = a.plans + r;
    const FdRow<T> row(static_cast<const T*>(a.z) + (size_t)b * a.zsb + (size_t)l * a.zsl, a.V);
    float v[kFdGroups][N];
    fd_load(row, item.y, lane, v);
    const float lo = plan->lo, hi = plan->hi;
    const uint32_t over = fd_reach(a.gmax[at], hi);
    double w = 0.0;
    if (over) {
      const FdWaveExp weight(plan->m, plan->invT);
#pragma unroll
      for (int j = 0; j < kFdGroups; ++j)
        if (over >> j & 1u) w += fd_sum(weight, v[j], hi);
      w = wave_sum(w);
    }
    uint32_t n = 0, from = 0;
#pragma unroll
    for (int j = 0; j < kFdGroups; ++j)
#pragma unroll
      for (int i = 0; i < N; ++i) n += v[j][i] >= lo && v[j][i] < hi && v[j][i] > -INFINITY ? 1u : 0u;
    const uint32_t incl = wave_incl_scan_u32(n);
    uint32_t mine = incl - n;
    n = (uint32_t)lane_value((int)incl, kWave - 1);
    if (n) {
      // a piece of the row's list, its entries in order of lanes
      if (lane == 0) from = atomicAdd(&plan->listed, n);
      from = (uint32_t)lane_value((int)from, 0);
      uint2* list = a.list + (size_t)r * a.cap;
      mine += from;
#pragma unroll
      for (int j = 0; j < kFdGroups; ++j)
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (v[j][i] >= lo && v[j][i] < hi && v[j][i] > -INFINITY) {
            if (mine < (uint32_t)a.cap)
              list[mine] = make_uint2(__float_as_uint(v[j][i]),
                                      (uint32_t)(row.first(g * kFdSegVecs + j * kWave + lane) + i));
            ++mine;
          }
    }
    if (lane == 0) {
      a.ssum[at] = w;
      a.part[at] = make_uint2(from, n);
    }
  }
}

// One workgroup a row: its threshold and its draw.  A chain of rounds, each some
// barriers: 11.6 us at 64 x 128256 bfloat16, 16 at 256 x 152064 float32, whose
// brackets hold more keys; a row with up to 64 collected logits, as top-k leaves,
// takes one wave without barriers.  Rows searched whole cost more: a top-k past the
// groups of a row with top-p 190 us for 64 x 129279 float32, equal logits 620, whose
// masses are added at one place.
template <typename T>
__global__ __launch_bounds__(kFdThreads) void filter_row_kernel(FdArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
  FdShared& s = *reinterpret_cast<FdShared*>(dyn);
  double* seg = reinterpret_cast<double*>(dyn + sizeof(FdShared));
  uint32_t* picks = reinterpret_cast<uint32_t*>(seg + a.nseg);
  float* list = reinterpret_cast<float*>(picks + a.nseg);
  constexpr int N = FdRow<T>::N;
  const int r = blockIdx.x, b = r / a.L, l = r % a.L, t = threadIdx.x;
  const int lane = t % kWave, wave = __builtin_amdgcn_readfirstlane(t / kWave);
  const FdPlan plan = a.plans[r];
  const uint2* found = a.list + (size_t)r * a.cap;
  uint2 entry = make_uint2(0u, 0u);
  if (lane < a.cap) entry = found[lane];             // (what stands there, if not enough was collected)
  const float u = a.tokens ? a.u[(size_t)b * a.usb + (size_t)l * a.usl] : 0.f;
  const FdParams f = fd_params(a.f, b);
  if (plan.need == kFdDone) return;
  const bool by_k = plan.need & kFdTopK, by_p = plan.need & kFdTopP;
  const uint32_t n = plan.listed;
  const float m = plan.m;
  const double invT = plan.invT, unit = fd_unit(a.V);
  float tau = plan.tau;

  // all that matters in one wave's hands
  if (n >= 1 && n <= (uint32_t)kWave && plan.hi == INFINITY) {
    const float z = __uint_as_float(entry.x);
    const double w = exp(((double)z - (double)m) * invT);
    FdShort k = fd_short(fkey(z), lane < (int)n ? fd_fixed(w, unit) : 0ull, (int)n, by_k, f.k, by_p,
                         (double)f.p, (double)f.p * plan.Z * unit);
    if (k.reached || by_k || plan.lo == plan.tau) {
      if (wave != 0) return;
      k.kept = k.kept && z >= tau;
      double S;
      const int y = fd_short_draw(k.kept, (int)entry.y, w, (int)n, a.tokens != nullptr, u, S);
      const uint32_t low = ~wave_max_u32(k.kept ? ~fkey(z) : 0u);
      if (lane == 0) {
        a.plans[r].cut = unkey(low);
        a.plans[r].invS = 1.0 / S;
        if (a.tokens) a.tokens[(size_t)b * a.tsb + (size_t)l * a.tsl] = y;
      }
      return;
    }
  }

  const float4* gmax = a.gmax + (size_t)r * a.nseg;
  const double* ssum = a.ssum + (size_t)r * a.nseg;
  const uint2* part = a.part + (size_t)r * a.nseg;
  fd_stage_table<kFdThreads>(s.tbl);
  const FdRow<T> row(static_cast<const T*>(a.z) + (size_t)b * a.zsb + (size_t)l * a.zsl, a.V);
  const FdExp weight(m, invT, s.tbl);
  auto fixed = [&](float z) { return fd_fixed(weight(z), unit); };
  bool whole = n <= (uint32_t)a.cap;
  double high = 0.0;
  for (int g = t; g < a.nseg; g += kFdThreads) {
    seg[g] = ssum[g];
    high += seg[g];
  }
  if (whole) {
#pragma unroll 4
    for (uint32_t e = t; e < n; e += kFdThreads) list[e] = __uint_as_float(found[e].x);
  }
  high = fd_block_sum<kFdWaves>(s, high);            // (its barriers serve the list too)
  if (by_k || by_p) {
    FdSource<T> src = {row, picks, 0u, list, n, true};
    auto each = [&](auto put) { src.each([&](float z) { put(fd_key<T>(z), z); }); };
    const double share = (double)f.p * plan.Z * unit;    // top-p's, where top-k is off
    auto search = [&](float from, uint32_t top, unsigned long long above) -> FdFound {
      FdFound k = {from > -INFINITY ? fd_key<T>(from) : kFdLowest<T>, true};
      if (by_k)
        k = fd_search<kFdThreads, false, false, T>(s, k.low, top, 0, (double)f.k, each,
                                                [](float) { return 0ull; });
      if (by_p) {
        double target = share;
        if (by_k) {
          unsigned long long sum = 0, all;
          each([&](uint32_t key, float z) {
            if (key >= k.low) sum += fixed(z);
          });
          fd_block_scan<kFdWaves>(s, sum, all);
          target = (double)f.p * (double)all;
        }
        k = fd_search<kFdThreads, true, false, T>(s, k.low, top, above, target, each, fixed);
      }
      k.reached = k.reached || by_k;
      return k;
    };
    FdFound k = {0u, false};
    const unsigned long long above = (unsigned long long)__double2ll_rn(high * unit);
    if (whole && (by_k || (double)above < share)) {
      // (the range that the list covers, so that its bins are fine)
      k = search(plan.lo, fd_key<T>(fminf(plan.hi, m)), above);
      // not reached, with less than the share above: the threshold lies below the
      // bracket, and below min-p's if the bracket starts there
      if (!k.reached && plan.lo == plan.tau)
        k = {plan.lo > -INFINITY ? fd_key<T>(plan.lo) : kFdLowest<T>, true};
    }
    if (!k.reached) {
      // the sample misled, or a list is too short for it: all of the row that matters
      const float from = by_k ? plan.lo : fmaxf(plan.bound, plan.tau);
      __syncthreads();
      src.npick = fd_pick(s, picks, gmax, a.nseg, from);
      src.listed = whole = false;
      k = search(from, fd_key<T>(m), 0ull);
    }
    tau = fmaxf(tau, fd_unkey<T>(k.low));
  }

  // the kept mass of each segment
  __syncthreads();
  if (whole) {
    // 16 lanes a segment
    if (n)
      for (int g = t / 16; g < a.nseg; g += kFdThreads / 16) {
        const uint2 p = part[g];
        double w = 0.0;
        for (uint32_t e = t % 16; e < p.y; e += 16) {
          const float z = list[p.x + e];
          const double x = weight(z);
          w += z >= tau && x > kFdNothing ? x : 0.0;
        }
        w += dpp_f64<0xb1>(w);
        w += dpp_f64<0x4e>(w);
        w += dpp_f64<0x141>(w);
        w += dpp_f64<0x140>(w);
        if (t % 16 == 0) seg[g] += w;
      }
  } else {
    for (int g = t; g < a.nseg; g += kFdThreads) seg[g] = 0.0;
    const uint32_t np = fd_pick(s, picks, gmax, a.nseg, tau);
    for (uint32_t e = wave; e < np; e += kFdWaves) {
      const uint32_t pick = picks[e];
      float v[kFdGroups][N];
      fd_load(row, pick, lane, v);
      double w = 0.0;
#pragma unroll
      for (int j = 0; j < kFdGroups; ++j) w += fd_sum(weight, v[j], tau);
      w = wave_sum(w);
      if (lane == 0) seg[pick >> 4] = w;
    }
  }
  __syncthreads();
  double S;
  const int y = fd_draw(s, row, seg, a.nseg, a.tokens != nullptr, u, tau, weight, S);
  if (t == 0) {
    a.plans[r].cut = tau;
    a.plans[r].invS = 1.0 / S;
    if (a.tokens) a.tokens[(size_t)b * a.tsb + (size_t)l * a.tsl] = y;
  }
}

__device__ __forceinline__ void fd_put(float* p, float v) { *p = v; }
__device__ __forceinline__ void fd_put(bf16_t* p, float v) { *p = bf16_bits(v); }

// The probabilities of one vector: whole 16- or 8-byte stores where the row's
// place allows.
template <typename O, int N>
__device__ __forceinline__ void fd_put_all(O* out, int e, int V, const float (&w)[N]) {
  constexpr int kBytes = N * (int)sizeof(O);
  if (e >= 0 && e + N <= V && (reinterpret_cast<uintptr_t>(out + e) & (kBytes < 16 ? kBytes - 1 : 15)) == 0) {
    uint32_t word[kBytes / 4];
#pragma unroll
    for (int i = 0; i < kBytes / 4; ++i)
      word[i] = sizeof(O) == 4 ? __float_as_uint(w[i]) : bf16_pair(w[2 * i % N], w[(2 * i + 1) % N]);
    if constexpr (kBytes == 8) {
      *reinterpret_cast<uint2*>(out + e) = make_uint2(word[0], word[1]);
    } else {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i)
        *(reinterpret_cast<uint4*>(out + e) + i) =
            make_uint4(word[4 * i], word[4 * i + 1], word[4 * i + 2], word[4 * i + 3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (e + i >= 0 && e + i < V) fd_put(out + e + i, w[i]);
  }
}

// The probabilities: one wave a segment, which reads the groups that reach the cut.
// Memory: 320 x 128256 float32, filters mixed, 31 us for 164 MB of writes, 5.3 TB/s,
// with the kept logits' reads beside them.  (Probabilities by the hardware's float32
// exp2 take a microsecond less, 3 where nothing is filtered, and are off by up to 2.7
// half steps.)
template <typename T, typename O>
__global__ __launch_bounds__(kFdStatThreads) void filter_probs_kernel(FdArgs a, int nblk) {
  constexpr int N = FdRow<T>::N;
  const int r = blockIdx.x / nblk, b = r / a.L, l = r % a.L, lane = threadIdx.x % kWave;
  const int g = (blockIdx.x % nblk) * (kFdStatThreads / kWave) + threadIdx.x / kWave;
  if (g >= a.nseg) return;
  const FdRow<T> row(static_cast<const T*>(a.z) + (size_t)b * a.zsb + (size_t)l * a.zsl, a.V);
  const FdPlan p = a.plans[r];
  const float4 x = a.gmax[(size_t)r * a.nseg + g];
  O* out = static_cast<O*>(a.probs) + (size_t)b * a.psb + (size_t)l * a.psl;
  const FdWaveExp weight(p.m, p.invT);
  const bool draws = p.kind == kFdDraw;
  const uint32_t bits = draws ? fd_reach(x, p.cut) : 0u;
  float v[kFdGroups][N];
  if (bits) fd_load(row, (uint32_t)g << 4 | bits, lane, v);
#pragma unroll
  for (int j = 0; j < kFdGroups; ++j) {
    const int e = row.first(g * kFdSegVecs + j * kWave + lane);
    float w[N];
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = 0.f;
    if (bits >> j & 1u) {                            // (all lanes: the table is spread over them)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float x = (float)(weight(v[j][i]) * p.invS);
        w[i] = v[j][i] >= p.cut ? x : 0.f;
      }
    }
    if (p.kind == kFdGreedy) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (e + i == p.best) w[i] = 1.f;
    }
    fd_put_all(out, e, a.V, w);
  }
}

// The whole call for a short row: one workgroup, the row in LDS (each thread reads
// its own vectors again, so without barriers), one read of the logits and no
// workspace.
//
// For top-p the masses are sorted into bins of equal width in (m - z) / T, over the
// range that holds all that top-p may keep: tokens that weigh less than (1 - p) /
// V together hold less than (1 - p) of a mass that is at least 1.  One pass of
// exponentials gives the total and the bin of the threshold; fd_search finds the
// value in it.
//
// For top-k, and in top-p's bin, what is left goes on a list of places in the row:
// up to 64 are one wave's, up to 512 are searched in the row's stead (one of 16000
// with all three filters 19.6 -> 15.8 us at 64 rows).
//
// Bound by one CU: 32000 bfloat16 logits with top-p take 20 to 30 us, 10 to 19 of
// them that pass, as few or most tokens lie in the bins (their LDS atomics; bins by
// whole steps of the exponential's table, with three float64 operations fewer a
// token, changed nothing); with top-k 13, with min-p 9; 69 rows of 20001 without
// filters 15.  Spread over workgroups, as longer rows are, a row of 33000 takes 20
// to 30, 23 and 17.
constexpr int kFdOneGroups = 144;                   // groups of 64 vectors
constexpr int kFdOneV = 32768;
constexpr int kFdOneList = 512;                     // one to a thread

struct FdOneShared {
  FdShared s;
  double group[kFdOneGroups];                       // their kept masses
  uint16_t few[kFdOneList];                         // a list of places in the row
  double S;
  float tau;
};
static_assert(((kFdOneV + 6) / 4 + 63) / 64 <= kFdOneGroups, "every group has its mass");
static_assert((sizeof(FdOneShared) + 15) / 16 * 16 + (kFdOneV + 6) / 4 * 16 <= kFdLds, "the row fits");
static_assert(kFdOneList <= kFdThreads && kFdOneV + 14 < 65536, "a thread to an entry, 16 bits to a place");

template <typename T, typename O>
__global__ __launch_bounds__(kFdThreads) void filter_one_kernel(FdArgs a) {
  constexpr int N = FdRow<T>::N;
  extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
  FdOneShared& o = *reinterpret_cast<FdOneShared*>(dyn);
  FdShared& s = o.s;
  uint4* kept = reinterpret_cast<uint4*>(dyn + (sizeof(FdOneShared) + 15) / 16 * 16);
  const int r = blockIdx.x, b = r / a.L, l = r % a.L, t = threadIdx.x;
  const int lane = t % kWave, wave = t / kWave;
  const FdRow<T> row(static_cast<const T*>(a.z) + (size_t)b * a.zsb + (size_t)l * a.zsl, a.V);
  const int nv = row.vecs();
  const float u = a.tokens ? a.u[(size_t)b * a.usb + (size_t)l * a.usl] : 0.f;
  const FdParams f = fd_params(a.f, b);
  fd_stage_table<kFdThreads>(s.tbl);
  float big = -INFINITY;
  bool fine = true;
#pragma unroll 4
  for (int q = t; q < nv; q += kFdThreads) {
    const uint4 raw = row.raw(q);
    kept[q] = raw;
    float v[N];
    unpack(raw, v, T{});
#pragma unroll
    for (int j = 0; j < N; ++j) {
      big = fmaxf(big, v[j]);
      fine = fine && v[j] < INFINITY;                // neither NaN nor +inf
    }
  }
  const uint32_t top = fd_block_max<kFdWaves>(s, fine ? fkey(big) : 0xffffffffu);
  const bool ok = f.ok && top > kNegInfKey && top != 0xffffffffu && u >= 0.f && u < 1.f;
  const float m = ok ? unkey(top) : 0.f;
  int y = -1;
  float tau = INFINITY;
  double invT = 0.0, invS = 0.0;
  if (ok && f.T == 0.f) {
    uint32_t first = 0;                              // ~ of the first id
    for (int q = t; q < nv; q += kFdThreads) {
      float v[N];
      unpack(kept[q], v, T{});
#pragma unroll
      for (int j = N - 1; j >= 0; --j)
        if (v[j] == m) first = max(first, ~(uint32_t)(row.first(q) + j));
    }
    y = (int)~fd_block_max<kFdWaves>(s, first);
  } else if (ok) {
    invT = 1.0 / (double)f.T;
    const bool by_k = f.k > 0 && f.k < a.V, by_p = f.p < 1.f;
    const double unit = fd_unit(a.V);
    const FdExp weight(m, invT, s.tbl);
    auto fixed = [&](float z) { return fd_fixed(weight(z), unit); };
    auto each = [&](auto put) {
      for (int q = t; q < nv; q += kFdThreads) {
        float v[N];
        unpack(kept[q], v, T{});
#pragma unroll
        for (int j = 0; j < N; ++j) put(fd_key<T>(v[j]), v[j]);
      }
    };
    const uint32_t high = fd_key<T>(m);
    tau = -INFINITY;
    if (f.mp > 0.f) tau = fd_min_p_threshold(m, f.T, weight, f.mp);
    // logits put on a list (in any order), how many in s.npick
    if (t == 0) s.npick = 0;
    auto put = [&](int place) {
      const uint32_t at = atomicAdd(&s.npick, 1u);
      if (at < (uint32_t)kFdOneList) o.few[at] = (uint16_t)place;
    };
    auto held = [&](int place) {
      const uint32_t word = reinterpret_cast<const uint32_t*>(kept)[place * (int)sizeof(T) / 4];
      return __uint_as_float(sizeof(T) == 4 ? word : place & 1 ? word & 0xffff0000u : word << 16);
    };
    auto listed = [&](int n, auto put) {             // those of a list
      if (t < n) {
        const float z = held(o.few[t]);
        put(fd_key<T>(z), z);
      }
    };
    bool done = false;
    int nlist = kFdOneList + 1;                      // top-k's list, if it fits
    uint32_t low = kFdLowest<T>;
    if (by_k) {
      if (f.k <= kFdThreads) {
        // at least k tokens reach the k-th largest of the threads' maxima
        // (from the lowest of these, so that the bins are fine)
        const uint32_t least = ~fd_block_max<kFdWaves>(s, big > -INFINITY ? ~fd_key<T>(big) : 0u);
        const FdFound k = fd_search<kFdThreads, false, true, T>(
            s, least, high, 0, (double)f.k, [&](auto add) { add(fd_key<T>(big), big); },
            [](float) { return 0ull; });
        if (k.reached) low = k.low;
        if (fd_key<T>(big) >= low)
          for (int q = t; q < nv; q += kFdThreads) {
            float v[N];
            unpack(kept[q], v, T{});
#pragma unroll
            for (int j = 0; j < N; ++j)
              if (fd_key<T>(v[j]) >= low) put(q * N + j);
          }
        __syncthreads();
        const int n = nlist = (int)s.npick;
        if (n <= kWave) {
          // all that matters in one wave's hands
          done = true;
          if (wave == 0) {
            const int place = lane < n ? o.few[lane] : 0;
            const float z = lane < n ? held(place) : m;
            const double w = weight(z);
            const FdShort k1 = fd_short(fkey(z), lane < n ? fd_fixed(w, unit) : 0ull, n, true, f.k, by_p,
                                        (double)f.p, 0.0);
            const bool in = k1.kept && z >= tau;
            double S;
            y = fd_short_draw(in, place - row.off, w, n, a.tokens != nullptr, u, S);
            const uint32_t least = ~wave_max_u32(in ? ~fkey(z) : 0u);
            if (lane == 0) {
              o.tau = unkey(least);
              o.S = S;
            }
          }
          __syncthreads();
          tau = o.tau;
          invS = 1.0 / o.S;
        }
      }
    }
    if (by_k && !done) {
      // all that matters is on the list, or in the row
      auto some = [&](auto put) {
        if (nlist <= kFdOneList) listed(nlist, put);
        else each(put);
      };
      low = fd_search<kFdThreads, false, false, T>(s, low, high, 0, (double)f.k, some,
                                                [](float) { return 0ull; }).low;
      if (by_p) {
        unsigned long long sum = 0, all;
        some([&](uint32_t key, float z) {
          if (key >= low) sum += fixed(z);
        });
        fd_block_scan<kFdWaves>(s, sum, all);
        low = fd_search<kFdThreads, true, false, T>(s, low, high, 0, (double)f.p * (double)all, some,
                                                 fixed).low;
      }
    } else if (by_p && !by_k) {
      const double width = 1e-6 - log((1.0 - (double)f.p) / a.V);
      const double per = kFdBins / width;
      for (int i = t; i < kFdBins; i += kFdThreads) s.mass[i] = 0;
      __syncthreads();
      unsigned long long tail = 0, all, rest;
      for (int q = t; q < nv; q += kFdThreads) {
        float v[N];
        unpack(kept[q], v, T{});
        fd_spread(s, weight, v, unit, per, kFdBins, tail);
      }
      fd_block_scan<kFdWaves>(s, tail, rest);        // (its barriers serve the bins too)
      const unsigned long long x0 = s.mass[2 * t], x1 = s.mass[2 * t + 1];
      const unsigned long long before = fd_block_scan<kFdWaves>(s, x0 + x1, all);
      const double target = (double)f.p * (double)(all + rest);
      // the last bin that holds something and has less than the target before it
      uint32_t mine = 0;
      if (x0 && (double)before < target) mine = 2u * t + 1u;
      if (x1 && (double)(before + x0) < target) mine = 2u * t + 2u;
      const uint32_t found = fd_block_max<kFdWaves>(s, mine);
      if (mine == found && found) s.above = found & 1u ? before : before + x0;
      // its logits
      const int at = (int)found - 1;
      auto in_bin = [&](float z) {
        const double bin = -weight.arg(z) * per;
        return bin >= at && bin < at + 1;
      };
      // (a cheap look first: their range, with room for the edges' rounding)
      const double z1 = (double)m - (double)f.T * (at / per), z0 = (double)m - (double)f.T * ((at + 1) / per);
      const double room = 1e-12 * (fabs((double)m) + fabs(z0) + fabs(z1));
      const uint32_t e0 = fd_key<T>((float)(z0 - room)), e1 = fd_key<T>((float)(z1 + room));
      const uint32_t k0 = max(kFdLowest<T>, e0 - min(e0, 1u)), k1 = min(high, e1 + 1u);
      for (int q = t; q < nv; q += kFdThreads) {
        float v[N];
        unpack(kept[q], v, T{});
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const uint32_t key = fd_key<T>(v[j]);
          if (key >= k0 && key <= k1 && in_bin(v[j])) put(q * N + j);
        }
      }
      __syncthreads();
      const int n = (int)s.npick;
      const unsigned long long above = s.above;
      if (n <= kWave) {                              // every wave for itself
        const float z = lane < n ? held(o.few[lane]) : m;
        const unsigned long long w = lane < n ? fixed(z) : 0ull;
        const int lo32 = (int)(uint32_t)w, hi32 = (int)(uint32_t)(w >> 32);
        const uint32_t key = fd_key<T>(z);
        unsigned long long over = above;
        for (int j = 0; j < n; ++j) {
          const unsigned long long x =
              (unsigned long long)(uint32_t)lane_value(hi32, j) << 32 | (uint32_t)lane_value(lo32, j);
          over += (uint32_t)lane_value((int)key, j) > key ? x : 0ull;
        }
        low = ~wave_max_u32(lane < n && (double)over < target ? ~key : 0u);
      } else {
        low = fd_search<kFdThreads, true, false, T>(
                  s, k0, k1, above, target,
                  [&](auto add) {
                    if (n <= kFdOneList) listed(n, add);
                    else
                      each([&](uint32_t key, float z) {
                        if (key >= k0 && key <= k1 && in_bin(z)) add(key, z);
                      });
                  },
                  fixed).low;
      }
    }
    if ((by_k || by_p) && !done) tau = fmaxf(tau, fd_unkey<T>(low));

    if (!done) {
    // kept mass of each group of 64 vectors
    const int ngroup = (nv + kWave - 1) / kWave;
    for (int g = wave; g < ngroup; g += kFdWaves) {
      const int q = g * kWave + lane;
      float v[N];
      unpack(q < nv ? kept[q] : row.nothing(), v, T{});
      double w = 0.0;
      bool some = false;
#pragma unroll
      for (int j = 0; j < N; ++j) some = some || (v[j] >= tau && v[j] > -INFINITY);
      if (__any(some)) w = wave_sum(fd_sum(weight, v, tau));
      if (lane == 0) o.group[g] = w;
    }
    __syncthreads();
    // every wave finds the group of the draw, the first draws
    constexpr int kPer = (kFdOneGroups + kWave - 1) / kWave;
    double w[kPer], mine = 0.0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      w[i] = lane * kPer + i < ngroup ? o.group[lane * kPer + i] : 0.0;
      mine += w[i];
    }
    const double incl = wave_incl_scan(mine), S = lane_value(incl, kWave - 1);
    invS = 1.0 / S;
    if (a.tokens) {
      const double target = (double)u * S;
      double run = wave_shr1(incl), at = 0.0, last_at = 0.0;
      int pick = -1, last = -1;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (w[i] > kFdNothing) {
          last = lane * kPer + i;
          last_at = run;
          if (pick < 0 && run + w[i] > target) {
            pick = last;
            at = run;
          }
        }
        run += w[i];
      }
      const uint64_t over = __ballot(pick >= 0), some = __ballot(last >= 0);
      const int src = over ? __ffsll((unsigned long long)over) - 1 : 63 - __clzll((long long)some);
      const int g = lane_value(over ? pick : last, src);
      const double base = lane_value(over ? at : last_at, src);
      if (wave == 0) {
        const int q = g * kWave + lane;
        float v[N];
        unpack(q < nv ? kept[q] : row.nothing(), v, T{});
        double x[N], sum = 0.0;
#pragma unroll
        for (int j = 0; j < N; ++j) {
          x[j] = v[j] >= tau && v[j] > -INFINITY ? weight(v[j]) : 0.0;
          sum += x[j];
        }
        double here = base + wave_shr1(wave_incl_scan(sum));
        int first = -1, tail = -1;
#pragma unroll
        for (int j = 0; j < N; ++j) {
          here += x[j];
          if (x[j] > kFdNothing) {
            tail = row.first(q) + j;
            if (first < 0 && here > target) first = tail;
          }
        }
        const uint64_t hit = __ballot(first >= 0), any = __ballot(tail >= 0);
        y = hit ? lane_value(first, __ffsll((unsigned long long)hit) - 1)
                : lane_value(tail, 63 - __clzll((long long)any));
      }
    }
    }
  }
  if (t == 0 && a.tokens) a.tokens[(size_t)b * a.tsb + (size_t)l * a.tsl] = y;
  if (a.probs) {
    O* out = static_cast<O*>(a.probs) + (size_t)b * a.psb + (size_t)l * a.psl;
    const FdExp weight(m, invT, s.tbl);
    for (int q = t; q < nv; q += kFdThreads) {
      const int e = row.first(q);
      float v[N], w[N];
      unpack(kept[q], v, T{});
#pragma unroll
      for (int j = 0; j < N; ++j) {
        w[j] = 0.f;
        if (ok && v[j] >= tau) w[j] = (float)(weight(v[j]) * invS);
        if (ok && f.T == 0.f) w[j] = e + j == y ? 1.f : 0.f;
      }
      fd_put_all(out, e, a.V, w);
    }
  }
}

// Segments of the longest row of V logits: it may start inside a vector.
int fd_segs(int V, bool bf16) {
  const int n = bf16 ? 8 : 4;
  return ((V + 2 * (n - 1)) / n + kFdSegVecs - 1) / kFdSegVecs;
}
int fd_blocks(int V, bool bf16) {
  return (fd_segs(V, bf16) + kFdStatThreads / kWave - 1) / (kFdStatThreads / kWave);
}

bool filter_fits(int B, int L, int V, bool bf16) {
  const size_t rows = (size_t)B * L;
  return grid_fits(rows, kFdThreads) && grid_fits(rows * fd_blocks(V, bf16), kFdStatThreads);
}

// Parts of the workspace, 16-byte aligned.
struct FdLayout {
  size_t gmax, ssum, part, list, items, nitem, bytes;
  int cap;
};
FdLayout fd_layout(size_t rows, int V, int nseg) {
  const size_t segs = (rows * nseg + 1) / 2 * 2;
  FdLayout w;
  w.cap = min(V, kFdListCap);
  w.gmax = rows * sizeof(FdPlan);
  w.ssum = w.gmax + segs * sizeof(float4);
  w.part = w.ssum + segs * sizeof(double);
  w.list = w.part + segs * sizeof(uint2);
  w.items = w.list + rows * w.cap * sizeof(uint2);
  w.nitem = w.items + segs * sizeof(uint2);
  w.bytes = w.nitem + 16;
  return w;
}

size_t filter_workspace_bytes(int B, int L, int V, bool bf16) {
  if (V <= kFdOneV) return 0;
  return fd_layout((size_t)B * L, V, fd_segs(V, bf16)).bytes;
}

template <typename F>
hipError_t fd_allow_lds(F* kernel) {
  return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                             hipFuncAttributeMaxDynamicSharedMemorySize, kFdLds);
}

template <typename T>
hipError_t fd_run(const FdArgs& a, size_t rows, bool probs_bf16, hipStream_t stream) {
  if (a.V <= kFdOneV) {
    const auto one = probs_bf16 ? filter_one_kernel<T, bf16_t> : filter_one_kernel<T, float>;
    constexpr int N = Elem<T>::kPerVec;
    const int lds = ((int)sizeof(FdOneShared) + 15) / 16 * 16 + (a.V + 2 * (N - 1)) / N * 16;
    const hipError_t e = fd_allow_lds(one);
    if (e != hipSuccess) return e;
    one<<<dim3((unsigned)rows), dim3(kFdThreads), lds, stream>>>(a);
    return hipGetLastError();
  }
  const int nblk = fd_blocks(a.V, sizeof(T) == 2);
  const dim3 grid((unsigned)(rows * nblk));
  filter_stats_kernel<T><<<grid, dim3(kFdStatThreads), 0, stream>>>(a, nblk);
  const int fixed = (int)sizeof(FdShared) + a.nseg * (int)sizeof(double);
  hipError_t e = fd_allow_lds(filter_plan_kernel<T>);
  if (e != hipSuccess) return e;
  const int lds_plan = fixed + a.nseg * (int)sizeof(uint32_t);
  filter_plan_kernel<T><<<dim3((unsigned)rows), dim3(kFdPlanThreads), lds_plan, stream>>>(a);
  // one setting for all rows that leaves nothing to collect ends here
  const specv_filters_t& f = a.f;
  const bool plain = !f.top_k_array && !f.top_p_array && !f.min_p_array &&
                     (f.top_k == 0 || f.top_k >= a.V) && f.top_p == 1.f && f.min_p == 0.f;
  const bool greedy = !f.temperature_array && f.temperature == 0.f;
  if (!plain && !greedy) {
    const size_t blocks = min(rows * nblk, (size_t)kFdCollectBlocks);
    filter_collect_kernel<T><<<dim3((unsigned)blocks), dim3(kFdStatThreads), 0, stream>>>(a);
    e = fd_allow_lds(filter_row_kernel<T>);
    if (e != hipSuccess) return e;
    const int lds = lds_plan + a.cap * (int)sizeof(float);
    filter_row_kernel<T><<<dim3((unsigned)rows), dim3(kFdThreads), lds, stream>>>(a);
  }
  if (a.probs) {
    if (probs_bf16) filter_probs_kernel<T, bf16_t><<<grid, dim3(kFdStatThreads), 0, stream>>>(a, nblk);
    else filter_probs_kernel<T, float><<<grid, dim3(kFdStatThreads), 0, stream>>>(a, nblk);
  }
  return hipGetLastError();
}

hipError_t launch_filter(const void* logits, long long zsb, long long zsl, bool bf16, int B, int L,
                         int V, const specv_filters_t& f, const float* u, long long usb,
                         long long usl, int* tokens, long long tsb, long long tsl, void* probs,
                         long long psb, long long psl, bool probs_bf16, void* workspace,
                         hipStream_t stream) {
  FdArgs a = {logits, zsb, zsl, L, V, f, u, usb, usl, tokens, tsb, tsl, probs, psb, psl};
  const size_t rows = (size_t)B * L;
  a.nseg = fd_segs(V, bf16);
  const FdLayout w = fd_layout(rows, V, a.nseg);
  char* base = static_cast<char*>(workspace);
  a.plans = reinterpret_cast<FdPlan*>(base);
  a.gmax = reinterpret_cast<float4*>(base + w.gmax);
  a.ssum = reinterpret_cast<double*>(base + w.ssum);
  a.part = reinterpret_cast<uint2*>(base + w.part);
  a.list = reinterpret_cast<uint2*>(base + w.list);
  a.items = reinterpret_cast<uint2*>(base + w.items);
  a.nitem = reinterpret_cast<int*>(base + w.nitem);
  a.cap = w.cap;
  return bf16 ? fd_run<bf16_t>(a, rows, probs_bf16, stream)
              : fd_run<float>(a, rows, probs_bf16, stream);
}

}  // namespace specv
