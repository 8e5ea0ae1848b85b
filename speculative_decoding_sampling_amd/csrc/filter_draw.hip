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
// Numerics.  Weights are float64 (exp64).  A mass that decides tau_p is a sum of
// whole multiples of 2^-s, s = 62 - ceil(log2 V): integer sums do not depend on
// their order, so that the histograms may be built with atomics, and n tokens
// are off by at most n 2^-(s+1) of the largest weight.  The sums of a draw are
// float64 in a fixed order.
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
constexpr int kFdGroups = 4;                        // vectors per lane of a segment
constexpr int kFdSegVecs = kFdGroups * kWave;       // a segment: one wave's load of 4 KB
// segments of the longest row, which may start inside a vector (float32 has more)
constexpr int kFdMaxSegs = SPECV_MAX_V / (kFdSegVecs * 4) + 1;

enum FdKind : int { kFdError = 0, kFdGreedy = 1, kFdDraw = 2 };

// What the row kernel leaves for the kernel that writes the probabilities.
struct FdPlan {
  int kind;
  int best;          // greedy: the token
  float m, tau;      // largest logit; a token is kept iff its logit >= tau
  double invT, invS;
};
static_assert(sizeof(FdPlan) == 32, "FdPlan is 32 bytes");

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
  __device__ __forceinline__ void load(int q, float* out) const {
    const int e = first(q);
    if (e >= 0 && e + N <= V) {
      load_vec_fast(p, e, out);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) out[i] = e + i >= 0 && e + i < V ? to_f32(p[e + i]) : -INFINITY;
    }
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

struct FdShared {
  double tbl[SPECV_EXP64_N];
  unsigned long long mass[kFdBins];
  uint32_t count[kFdBins];
  double seg[kFdMaxSegs];
  unsigned long long wave_u64[kFdWaves];
  uint32_t wave_u32[kFdWaves];
  float wave_f32[kFdWaves];
  int found;
  unsigned long long above;
};

__device__ __forceinline__ float fd_block_max(FdShared& s, float v) {
  v = wave_max(v);
  if (threadIdx.x % kWave == 0) s.wave_f32[threadIdx.x / kWave] = v;
  __syncthreads();
  float r = s.wave_f32[0];
#pragma unroll
  for (int w = 1; w < kFdWaves; ++w) r = fmaxf(r, s.wave_f32[w]);
  __syncthreads();
  return r;
}
__device__ __forceinline__ uint32_t fd_block_min(FdShared& s, uint32_t v) {
  v = wave_reduce_u32(v, [](uint32_t x, uint32_t y) { return x < y ? x : y; });
  if (threadIdx.x % kWave == 0) s.wave_u32[threadIdx.x / kWave] = v;
  __syncthreads();
  uint32_t r = s.wave_u32[0];
#pragma unroll
  for (int w = 1; w < kFdWaves; ++w) r = min(r, s.wave_u32[w]);
  __syncthreads();
  return r;
}
__device__ __forceinline__ unsigned long long fd_block_sum(FdShared& s, unsigned long long v) {
  v = wave_incl_scan_u64(v);
  if (threadIdx.x % kWave == kWave - 1) s.wave_u64[threadIdx.x / kWave] = v;
  __syncthreads();
  unsigned long long r = 0;
#pragma unroll
  for (int w = 0; w < kFdWaves; ++w) r += s.wave_u64[w];
  __syncthreads();
  return r;
}

// exp((z - m) / T), at most 1.
__device__ __forceinline__ double fd_weight(float z, double m, double invT, const double* tbl) {
  return exp64(((double)z - m) * invT, tbl);
}

// The block's pass over a row: f(vector, elements, first id).
template <typename T, typename F>
__device__ __forceinline__ void fd_scan(const FdRow<T>& row, F f) {
  const int nv = row.vecs();
  for (int q = threadIdx.x; q < nv; q += kFdThreads) {
    float v[FdRow<T>::N];
    row.load(q, v);
    f(v, row.first(q));
  }
}

// The search for a threshold, by the whole block: the key of the lowest kept
// value, where a value is kept if what lies above it is below the target.
// Each round sorts the keys of the bracket [lo, hi] into bins by count, and by
// mass where that is what the target is about, finds the bin where the running
// sum from the top reaches the target and goes on inside it, until it holds one
// value (or one key: ties go together).
template <bool MASS, typename T, typename W>
__device__ uint32_t fd_search(FdShared& s, const FdRow<T>& row, uint32_t lo, uint32_t hi,
                              double target, W weight) {
  unsigned long long above = 0;
  const int t = threadIdx.x, lane = t % kWave, wave = t / kWave;
  for (;;) {
    const int bits = 32 - __clz((int)((hi - lo) | 1u));
    const int sh = max(bits - 11, 0);
    static_assert(kFdBins == 1 << 11, "a round takes 11 bits of the key");
    for (int i = t; i < kFdBins; i += kFdThreads) {
      s.count[i] = 0;
      if (MASS) s.mass[i] = 0;
    }
    if (t == 0) s.found = -1;
    __syncthreads();
    fd_scan(row, [&](const float* v, int) {
#pragma unroll
      for (int i = 0; i < FdRow<T>::N; ++i) {
        const uint32_t key = fkey(v[i]);
        if (key >= lo && key <= hi) {
          const int b = (int)((key - lo) >> sh);
          atomicAdd(&s.count[b], 1u);
          if (MASS) atomicAdd(&s.mass[b], weight(v[i]));
        }
      }
    });
    __syncthreads();
    // thread t owns bins top - 2 t and the one below: running sums from the top
    const int b0 = kFdBins - 1 - 2 * t, b1 = b0 - 1;
    const unsigned long long x0 = MASS ? s.mass[b0] : s.count[b0];
    const unsigned long long x1 = MASS ? s.mass[b1] : s.count[b1];
    const unsigned long long incl = wave_incl_scan_u64(x0 + x1);
    if (lane == kWave - 1) s.wave_u64[wave] = incl;
    __syncthreads();
    unsigned long long before = above + incl - (x0 + x1);
    for (int w = 0; w < wave; ++w) before += s.wave_u64[w];
    // the lowest bin that holds something and has less than the target above
    int mine = -1;
    unsigned long long mine_above = 0;
    if (s.count[b0] && (double)before < target) {
      mine = b0;
      mine_above = before;
    }
    if (s.count[b1] && (double)(before + x0) < target) {
      mine = b1;
      mine_above = before + x0;
    }
    const uint64_t some = __ballot(mine >= 0);
    if (some && lane == 63 - __clzll((long long)some)) s.wave_u32[wave] = (uint32_t)mine;
    if (!some && lane == 0) s.wave_u32[wave] = 0xffffffffu;
    __syncthreads();
    int bin = -1;
    for (int w = 0; w < kFdWaves; ++w)
      if (s.wave_u32[w] != 0xffffffffu) bin = (int)s.wave_u32[w];
    if (bin >= 0 && mine == bin) s.above = mine_above;
    __syncthreads();
    if (bin < 0) return lo;                          // nothing in the bracket
    const uint32_t base = lo + ((uint32_t)bin << sh);
    const bool last = sh == 0 || s.count[bin] == 1u;
    above = s.above;
    __syncthreads();
    if (last) return base;
    lo = base;
    hi = base + ((1u << sh) - 1u);
  }
}

// The smallest float whose weight is at least mp, in (0, 1]: a search over keys
// in which each lane of a wave tries one of 64 (6 rounds for 32 bits).
__device__ __forceinline__ float fd_min_p_threshold(float m, double invT, float mp,
                                                    const double* tbl) {
  const int lane = threadIdx.x % kWave;
  uint32_t lo = kNegInfKey + 1, hi = fkey(m);        // the maximum itself has weight 1
  while (lo < hi) {
    const uint32_t step = (hi - lo) / kWave + 1;
    auto key = [&](int i) { return lo + min((uint32_t)i * step, hi - lo); };
    const uint64_t yes = __ballot(fd_weight(unkey(key(lane)), m, invT, tbl) >= (double)mp);
    if (yes == 0) {
      lo = key(kWave - 1) + 1;
    } else {
      const int i = __ffsll((unsigned long long)yes) - 1;
      hi = key(i);
      if (i > 0) lo = key(i - 1) + 1;
    }
  }
  return unkey(hi);
}

// One workgroup a row.
template <typename T>
__global__ __launch_bounds__(kFdThreads) void filter_row_kernel(FdArgs a) {
  __shared__ FdShared s;
  const int r = blockIdx.x, b = r / a.L, l = r % a.L;
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  constexpr int N = FdRow<T>::N;
  if (threadIdx.x < SPECV_EXP64_N) s.tbl[threadIdx.x] = kExp64Table[threadIdx.x];
  const FdRow<T> row(static_cast<const T*>(a.z) + (size_t)b * a.zsb + (size_t)l * a.zsl, a.V);
  const FdParams f = fd_params(a.f, b);
  const float u = a.tokens ? a.u[(size_t)b * a.usb + (size_t)l * a.usl] : 0.f;

  float m = -INFINITY;
  bool bad = false;
  fd_scan(row, [&](const float* v, int) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      m = fmaxf(m, v[i]);
      bad = bad || !(v[i] < INFINITY);               // NaN or +inf
    }
  });
  bad = __syncthreads_or(bad);
  m = fd_block_max(s, m);
  const bool ok = f.ok && !bad && m > -INFINITY && u >= 0.f && u < 1.f;
  FdPlan plan = {kFdError, -1, m, m, 0.0, 0.0};
  int y = -1;
  if (ok && f.T == 0.f) {
    uint32_t best = 0xffffffffu;
    fd_scan(row, [&](const float* v, int e) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (v[i] == m) best = min(best, (uint32_t)(e + i));
    });
    y = (int)fd_block_min(s, best);
    plan.kind = kFdGreedy;
    plan.best = y;
  } else if (ok) {
    const double invT = 1.0 / (double)f.T;
    const int shift = 62 - (32 - __clz(a.V - 1 | 1));
    const double unit = ldexp(1.0, shift);
    auto fixed = [&](float z) {
      return (unsigned long long)__double2ll_rn(fd_weight(z, m, invT, s.tbl) * unit);
    };
    const uint32_t top = fkey(m);
    uint32_t low = kNegInfKey + 1;
    if (f.k > 0 && f.k < a.V)
      low = fd_search<false>(s, row, low, top, (double)f.k, [](float) { return 0ull; });
    if (f.p < 1.f) {
      unsigned long long sum = 0;
      fd_scan(row, [&](const float* v, int) {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (fkey(v[i]) >= low) sum += fixed(v[i]);
      });
      sum = fd_block_sum(s, sum);
      low = fd_search<true>(s, row, low, top, (double)f.p * (double)sum, fixed);
    }
    float tau = low == kNegInfKey + 1 ? -INFINITY : unkey(low);
    if (f.mp > 0.f) tau = fmaxf(tau, fd_min_p_threshold(m, invT, f.mp, s.tbl));

    // kept mass of each segment, then of all before it
    const int nv = row.vecs(), nseg = (nv + kFdSegVecs - 1) / kFdSegVecs;
    for (int g = wave; g < nseg; g += kFdWaves) {
      double w = 0.0;
      for (int j = 0; j < kFdGroups; ++j) {
        const int q = g * kFdSegVecs + j * kWave + lane;
        if (q < nv) {
          float v[N];
          row.load(q, v);
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (v[i] >= tau) w += fd_weight(v[i], m, invT, s.tbl);
        }
      }
      w = wave_sum(w);
      if (lane == 0) s.seg[g] = w;
    }
    __syncthreads();
    if (wave == 0) {
      // lane l sums segments l per .. l per + per - 1
      const int per = (nseg + kWave - 1) / kWave;
      const int g0 = min(lane * per, nseg), g1 = min(g0 + per, nseg);
      double mine = 0.0;
      for (int g = g0; g < g1; ++g) mine += s.seg[g];
      const double incl = wave_incl_scan(mine);
      const double S = lane_value(incl, kWave - 1);
      plan = {kFdDraw, -1, m, tau, invT, 1.0 / S};
      if (a.tokens) {
        const double t = (double)u * S;
        // the first segment with weight whose running sum exceeds t, or where
        // rounding leaves none the last with weight
        double run = wave_shr1(incl), at = 0.0, last_at = 0.0;
        int pick = -1, last = -1;
        for (int g = g0; g < g1; ++g) {
          const double w = s.seg[g];
          if (w > 0.0) {
            last = g;
            last_at = run;
            if (pick < 0 && run + w > t) {
              pick = g;
              at = run;
            }
          }
          run += w;
        }
        const uint64_t over = __ballot(pick >= 0), some = __ballot(last >= 0);
        const int src = over ? __ffsll((unsigned long long)over) - 1 : 63 - __clzll((long long)some);
        const int seg = lane_value(over ? pick : last, src);
        double base = lane_value(over ? at : last_at, src);
        // inside it: the same over lanes, then over a lane's elements
        int end = -1;
        for (int j = 0; j < kFdGroups && y < 0; ++j) {
          const int q = seg * kFdSegVecs + j * kWave + lane;
          float v[N];
          double w[N], sum = 0.0;
          if (q < nv) row.load(q, v);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            w[i] = q < nv && v[i] >= tau ? fd_weight(v[i], m, invT, s.tbl) : 0.0;
            sum += w[i];
          }
          const double in = wave_incl_scan(sum);
          double run = base + wave_shr1(in);
          int first = -1, tail = -1;
#pragma unroll
          for (int i = 0; i < N; ++i) {
            run += w[i];
            if (w[i] > 0.0) {
              tail = row.first(q) + i;
              if (first < 0 && run > t) first = tail;
            }
          }
          const uint64_t hit = __ballot(first >= 0), any = __ballot(tail >= 0);
          if (hit) y = lane_value(first, __ffsll((unsigned long long)hit) - 1);
          if (any) end = lane_value(tail, 63 - __clzll((long long)any));
          base += lane_value(in, kWave - 1);
        }
        if (y < 0) y = end;
      }
    }
  }
  if (threadIdx.x == 0) {
    a.plans[r] = plan;
    if (a.tokens) a.tokens[(size_t)b * a.tsb + (size_t)l * a.tsl] = y;
  }
}

// 2^x / S for x = (z - m) / (T ln 2): the argument in float64, its fraction's
// power by the hardware's exp2 (1 ulp).
__device__ __forceinline__ float fd_prob(float z, double m, double c, float invS) {
  const double x = fmax(((double)z - m) * c, -1000.0);
  const double k = rint(x);
  return ldexpf(__builtin_amdgcn_exp2f((float)(x - k)) * invS, (int)k);
}

__device__ __forceinline__ void fd_put(float* p, float v) { *p = v; }
__device__ __forceinline__ void fd_put(bf16_t* p, float v) { *p = bf16_bits(v); }

// The probabilities: each thread one vector of logits.
template <typename T, typename O>
__global__ __launch_bounds__(256) void filter_probs_kernel(FdArgs a, int nblk) {
  constexpr int N = FdRow<T>::N;
  const int r = blockIdx.x / nblk, b = r / a.L, l = r % a.L;
  const int q = (blockIdx.x % nblk) * 256 + threadIdx.x;
  const FdRow<T> row(static_cast<const T*>(a.z) + (size_t)b * a.zsb + (size_t)l * a.zsl, a.V);
  if (q >= row.vecs()) return;
  const FdPlan p = a.plans[r];
  O* out = static_cast<O*>(a.probs) + (size_t)b * a.psb + (size_t)l * a.psl;
  const int e = row.first(q);
  float v[N];
  row.load(q, v);
  const double c = p.invT * 1.4426950408889634, m = p.m;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float w = 0.f;
    if (p.kind == kFdDraw && v[i] >= p.tau) w = fd_prob(v[i], m, c, (float)p.invS);
    if (p.kind == kFdGreedy && e + i == p.best) w = 1.f;
    if (e + i >= 0 && e + i < a.V) fd_put(out + e + i, w);
  }
}

int fd_vecs(int V, bool bf16) { return bf16 ? (V + 7 + 7) / 8 : (V + 3 + 3) / 4; }

bool filter_fits(int B, int L, int V, bool bf16) {
  const size_t rows = (size_t)B * L;
  return grid_fits(rows, kFdThreads) && grid_fits(rows * ((fd_vecs(V, bf16) + 255) / 256), 256);
}

size_t filter_workspace_bytes(int B, int L, int V, bool bf16) {
  return (size_t)B * L * sizeof(FdPlan);
}

template <typename T>
hipError_t fd_run(const FdArgs& a, size_t rows, bool probs_bf16, hipStream_t stream) {
  filter_row_kernel<T><<<dim3((unsigned)rows), dim3(kFdThreads), 0, stream>>>(a);
  if (a.probs) {
    const int nblk = (fd_vecs(a.V, sizeof(T) == 2) + 255) / 256;
    const dim3 grid((unsigned)(rows * nblk));
    if (probs_bf16) filter_probs_kernel<T, bf16_t><<<grid, dim3(256), 0, stream>>>(a, nblk);
    else filter_probs_kernel<T, float><<<grid, dim3(256), 0, stream>>>(a, nblk);
  }
  return hipGetLastError();
}

hipError_t launch_filter(const void* logits, long long zsb, long long zsl, bool bf16, int B, int L,
                         int V, const specv_filters_t& f, const float* u, long long usb,
                         long long usl, int* tokens, long long tsb, long long tsl, void* probs,
                         long long psb, long long psl, bool probs_bf16, void* workspace,
                         hipStream_t stream) {
  const FdArgs a = {logits, zsb, zsl, L, V, f, u, usb, usl, tokens, tsb, tsl, probs, psb, psl,
                    static_cast<FdPlan*>(workspace)};
  const size_t rows = (size_t)B * L;
  return bf16 ? fd_run<bf16_t>(a, rows, probs_bf16, stream)
              : fd_run<float>(a, rows, probs_bf16, stream);
}

}  // namespace specv
