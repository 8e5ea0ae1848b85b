// Verification from probabilities (specv_verify_probs).
//
// Per request: the accept scan u_k q_k(x_k) < p_k(x_k) over the drafted
// positions, then one inverse-CDF draw from max(p_j - q_j, 0) at the first
// rejection j, or from p_n when every draft was accepted (nickwang.xyz
// "推测解码：草稿、验证与实际加速", sections "接受与拒绝怎样保住分布" and
// "算完三个 token 的全部概率").  A request therefore needs two gathered values
// per draft and one row (bonus) or a pair of rows (rejection): that is all
// the call reads.
//
// Numerics.  u, p and q are float32 (or bfloat16) values, so u q is exact in
// float64 and the accept test is decided without rounding; p - q is exact in
// float64 too wherever it matters (their exponents differ by less than 29).
// Sums are float64 in a fixed order: results do not change from run to run.
//
// Split.  A chunk is kProbChunk tokens, summed by one wave.  Each wave makes
// the request's accept scan for itself (lane k owns position k, two dependent
// loads) rather than wait for a scan kernel's plan: the scans run side by
// side, a kernel boundary would not.  The wave of chunk 0 writes everything but
// the drawn token, and the plan; then one wave per request walks the chunk
// sums to the chunk that holds the draw and scans that chunk.  Small
// vocabularies do both in one workgroup per request, the chunk sums in LDS.
#include "common.h"
#include "grid.h"
#include "specverify.h"
#include "wave_scan.h"

namespace specv {

constexpr int kProbChunk = 1024;
constexpr int kProbPer = kProbChunk / kWave;       // 16 tokens per lane
constexpr int kProbBatch = kWave;                  // chunk records a wave takes at once
constexpr int kProbPassThreads = 256;
constexpr int kProbOneThreads = 1024;
constexpr int kProbOneChunks = 64;                 // LDS records of the one-kernel form
static_assert(SPECV_MAX_V <= kProbChunk * kProbBatch * kWave,
              "one lane per batch of chunk records");

// What the draw of a scanned request needs.
struct ProbPlan {
  int path, stop;
  float uf;
  int hot;            // the drafted token of a rejection without draft rows, else -1
};
static_assert(sizeof(ProbPlan) == 16, "ProbPlan is 16 bytes");

struct ProbArgs {
  const void* tgt;
  const void* dft;                  // null: one at the drafted token
  long long tsb, tsk, dsb, dsk;     // strides in elements
  const int* tokens;
  const int* draft_len;
  const float* u;
  const float* u_final;
  int K, V, nch, eos_id;
  ProbPlan* plans;                  // [B]
  double* recs;                     // [B][nch] chunk sums of the weights, NaN if invalid
  int* out_tokens;
  int* n_emitted;
  float* alpha_out;
  double* rmass_out;
  int* stop_out;
  int* path_out;
};

// A probability the call may use: finite and not negative (false for NaN).
__device__ __forceinline__ bool prob_ok(float p) { return p >= 0.f && p <= 3.402823466e38f; }

// The accept scan of request b, by one wave.
struct ProbScan {
  int path, stop, nb;
  float uf;
  int x;              // lane k: drafted token k (lane < nb)
  double alpha;       // lane k: min(1, p/q), -1 where not drafted
};

template <typename T>
__device__ __forceinline__ ProbScan prob_scan(const ProbArgs& a, int b, int lane) {
  ProbScan s;
  const int nraw = a.draft_len[b];
  s.uf = a.u_final[b];
  int x = -1;
  float uk = 0.f;
  if (lane < a.K) {
    x = a.tokens[(size_t)b * a.K + lane];
    uk = a.u[(size_t)b * a.K + lane];
  }
  bool bad = nraw < 0 || nraw > a.K || !(s.uf >= 0.f && s.uf < 1.f);
  const int nb = bad ? 0 : nraw;
  bool ok = true, accept = false;
  s.alpha = -1.0;
  if (lane < nb) {
    ok = x >= 0 && x < a.V && uk >= 0.f && uk < 1.f;
    if (ok) {
      const T* t = static_cast<const T*>(a.tgt);
      const T* d = static_cast<const T*>(a.dft);
      const float p = to_f32(t[(size_t)b * a.tsb + (size_t)lane * a.tsk + x]);
      const float q = d ? to_f32(d[(size_t)b * a.dsb + (size_t)lane * a.dsk + x]) : 1.f;
      ok = prob_ok(p) && prob_ok(q) && q > 0.f;
      accept = (double)uk * (double)q < (double)p;
      const double ratio = (double)p / (double)q;
      s.alpha = ratio < 1.0 ? ratio : 1.0;
    }
  }
  bad = bad || __ballot(!ok) != 0;
  const uint64_t rej = __ballot(lane < nb && !accept);
  s.stop = rej ? __ffsll((unsigned long long)rej) - 1 : nb;
  s.path = rej ? kPathReject : kPathBonus;
  const uint64_t eos = __ballot(lane < nb && accept && x == a.eos_id);
  if (eos) {
    const int e = __ffsll((unsigned long long)eos) - 1;
    if (e < s.stop) {
      s.stop = e;
      s.path = kPathEos;
    }
  }
  if (bad) s.path = kPathError;
  s.nb = nb;
  s.x = x;
  return s;
}

__device__ __forceinline__ ProbPlan prob_plan(const ProbArgs& a, const ProbScan& s) {
  ProbPlan p = {s.path, s.stop, s.uf, -1};
  if (s.path == kPathReject && !a.dft) p.hot = lane_value(s.x, s.stop);
  return p;
}
__device__ __forceinline__ bool prob_draws(int path) {
  return path == kPathReject || path == kPathBonus;
}

// The rows the draw of a planned request reads.
template <typename T>
struct ProbRows {
  const T* p;
  const T* q;         // null: none, or one at token hot
  int hot;
};

template <typename T>
__device__ __forceinline__ ProbRows<T> prob_rows(const ProbArgs& a, int b, const ProbPlan& s) {
  ProbRows<T> r;
  r.p = static_cast<const T*>(a.tgt) + (size_t)b * a.tsb + (size_t)s.stop * a.tsk;
  r.q = s.path == kPathReject && a.dft
            ? static_cast<const T*>(a.dft) + (size_t)b * a.dsb + (size_t)s.stop * a.dsk
            : nullptr;
  r.hot = s.hot;
  return r;
}

// The weight of one token.  max(p - q, 0) of valid entries is p itself where
// there is no q.
__device__ __forceinline__ double prob_weight(float p, float q) {
  return fmax((double)p - (double)q, 0.0);
}

// Validity of a batch of entries: the largest of their bits as unsigned
// integers is below those of infinity unless one is negative, infinite or NaN
// (or -0, which only the full test below tells).
__device__ __forceinline__ uint32_t prob_bits(float p) { return __float_as_uint(p); }

// 16 entries of a row as floats.  striped: entries base + (64 j + lane) N + i
// (N per 16-byte vector, whole cache lines per load); otherwise the lane's
// own base + 16 lane + i, in order.  Entries at or past V read as 0.
template <typename T, bool STRIPED>
__device__ __forceinline__ void prob_load(const T* __restrict__ row, int base, int lane, int V,
                                          float* out) {
  constexpr int N = Elem<T>::kPerVec;
  constexpr int J = kProbPer / N;
  if (aligned16(row) && base + kProbChunk <= V) {          // uniform over the wave
#pragma unroll
    for (int j = 0; j < J; ++j)
      load_vec_fast(row, STRIPED ? base + (j * kWave + lane) * N : base + lane * kProbPer + j * N,
                    out + j * N);
  } else {
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int v = STRIPED ? base + (j * kWave + lane) * N + i : base + lane * kProbPer + j * N + i;
        const float p = to_f32(row[min(v, V - 1)]);         // no branch: all loads in flight
        out[j * N + i] = v < V ? p : 0.f;
      }
  }
}

// Sum of chunk c's weights, by one wave (every lane gets it); NaN where an
// entry is invalid.
template <typename T>
__device__ __forceinline__ double prob_chunk(const ProbRows<T>& r, int c, int lane, int V) {
  const int base = c * kProbChunk;
  constexpr int N = Elem<T>::kPerVec;
  float p[kProbPer], q[kProbPer];
  prob_load<T, true>(r.p, base, lane, V, p);
  const bool has_q = r.q || (r.hot >= base && r.hot < base + kProbChunk);   // uniform
  if (r.q) {
    prob_load<T, true>(r.q, base, lane, V, q);
  } else {
#pragma unroll
    for (int j = 0; j < kProbPer / N; ++j)
#pragma unroll
      for (int i = 0; i < N; ++i) q[j * N + i] = base + (j * kWave + lane) * N + i == r.hot ? 1.f : 0.f;
  }
  uint32_t top = 0;
  double w = 0.0;
  if (has_q) {
#pragma unroll
    for (int e = 0; e < kProbPer; ++e) {
      top = max(top, max(prob_bits(p[e]), prob_bits(q[e])));
      w += prob_weight(p[e], q[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < kProbPer; ++e) {
      top = max(top, prob_bits(p[e]));
      w += (double)p[e];
    }
  }
  if (top >= 0x7f800000u) {
    bool ok = true;
#pragma unroll
    for (int e = 0; e < kProbPer; ++e) ok = ok && prob_ok(p[e]) && prob_ok(q[e]);
    if (!ok) w = __builtin_nan("");
  }
  return wave_sum(w);
}

// The first lane whose running sum exceeds t, or where rounding leaves none
// the last with a positive term.
__device__ __forceinline__ int prob_lane(double incl, double term, double t) {
  const uint64_t over = __ballot(incl > t && term > 0.0);
  const uint64_t some = __ballot(term > 0.0);
  return over ? __ffsll((unsigned long long)over) - 1 : 63 - __clzll((long long)some);
}

// The token of chunk c at t, base being the weights before the chunk: the
// first with a positive weight whose running sum exceeds t, or where rounding
// leaves none the last with one.  The weight is looked at because the scans
// add in an order of each lane's own: base and the sum before a lane may be a
// rounding above that of the last lane with weight, and so above t already.
template <typename T>
__device__ __forceinline__ int prob_draw(const ProbRows<T>& r, int c, int lane, int V, double base,
                                         double t) {
  const int v0 = c * kProbChunk + lane * kProbPer;
  float p[kProbPer], q[kProbPer];
  prob_load<T, false>(r.p, c * kProbChunk, lane, V, p);
  if (r.q) prob_load<T, false>(r.q, c * kProbChunk, lane, V, q);
  else
#pragma unroll
    for (int i = 0; i < kProbPer; ++i) q[i] = v0 + i == r.hot ? 1.f : 0.f;
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < kProbPer; ++i) sum += prob_weight(p[i], q[i]);
  const double incl = wave_incl_scan(sum);
  double run = base + wave_shr1(incl);
  int first = kProbPer, last = 0;
#pragma unroll
  for (int i = 0; i < kProbPer; ++i) {
    const double w = prob_weight(p[i], q[i]);
    run += w;
    if (first == kProbPer && w > 0.0 && run > t) first = i;
    if (w > 0.0) last = i;
  }
  const int L = prob_lane(base + incl, sum, t) & (kWave - 1);
  const int pick = first < kProbPer ? first : last;
  return c * kProbChunk + L * kProbPer + lane_value(pick, L);
}

// The outputs of a scanned request by one wave: y the drawn token, mass the
// residual's.
__device__ __forceinline__ void prob_outputs(const ProbArgs& a, int b, int lane,
                                             const ProbScan& s, int y, double mass) {
  const bool err = s.path == kPathError;
  for (int k = lane; k <= a.K; k += kWave) {
    int v = -1;
    if (!err) {
      // a position before the stop is one of the first 64: k = lane there
      if (k < s.stop || (k == s.stop && s.path == kPathEos)) v = s.x;
      else if (k == s.stop) v = y;
    }
    a.out_tokens[(size_t)b * (a.K + 1) + k] = v;
  }
  if (a.alpha_out && lane < a.K)
    a.alpha_out[(size_t)b * a.K + lane] = !err && lane < s.nb ? (float)s.alpha : -1.f;
  if (lane == 0) {
    a.n_emitted[b] = err ? -1 : s.stop + 1;
    if (a.rmass_out) a.rmass_out[b] = err ? 0.0 : mass;
    if (a.stop_out) a.stop_out[b] = err ? -1 : s.stop;
    if (a.path_out) a.path_out[b] = s.path;
  }
}
__device__ __forceinline__ void prob_error(const ProbArgs& a, int b, int lane) {
  ProbScan e = {};
  e.path = kPathError;
  prob_outputs(a, b, lane, e, -1, 0.0);
}

// A walk over chunk sums, 64 at a time: rec(i), called by the whole wave, is
// lane l's sum of chunk 64 i + l (0 past the last).  Lane i keeps the total of
// batch i.
struct ProbWalk {
  double batch, total;
};
template <typename F>
__device__ __forceinline__ ProbWalk prob_total(int nch, int lane, F rec) {
  double mine = 0.0;
  for (int i = 0; i * kProbBatch < nch; ++i) {
    const double s = wave_sum(rec(i));
    if (lane == i) mine = s;
  }
  return {mine, wave_sum(mine)};
}
// The chunk that holds t and the weights before it (total > 0).
template <typename F>
__device__ __forceinline__ int prob_find(const ProbWalk& w, int lane, double t, F rec,
                                         double& before) {
  const double bincl = wave_incl_scan(w.batch);
  const int bi = prob_lane(bincl, w.batch, t);
  const double start = lane_value(wave_shr1(bincl), bi);
  const double r = rec(bi);
  const double cincl = start + wave_incl_scan(r);
  const int ci = prob_lane(cincl, r, t);
  before = ci ? lane_value(cincl, ci - 1) : start;
  return bi * kProbBatch + ci;
}

// The draw of a planned request from its chunk records, a walk over them and
// their access, by one wave: the token, -1 where an entry is invalid or there is
// no mass.
template <typename T, typename F>
__device__ __forceinline__ int prob_pick(const ProbArgs& a, int b, int lane, const ProbPlan& s,
                                         const ProbWalk& w, F rec, double& mass) {
  ProbRows<T> rows = prob_rows<T>(a, b, s);
  double before;
  mass = s.path == kPathReject ? w.total : 0.0;
  if (w.total > 0.0) {
    const double t = (double)s.uf * w.total;
    const int c = prob_find(w, lane, t, rec, before);
    return prob_draw<T>(rows, c, lane, a.V, before, t);
  }
  if (!(w.total == 0.0) || s.path != kPathReject) return -1;
  // An empty residual: the correction is drawn from p itself, whose chunks
  // this wave sums on the spot (only the rounding of the caller's
  // probabilities leads here).
  rows.q = nullptr;
  rows.hot = -1;
  auto sum = [&](int i) {
    double mine = 0.0;
    for (int l = 0; l < kProbBatch && i * kProbBatch + l < a.nch; ++l) {
      const double v = prob_chunk<T>(rows, i * kProbBatch + l, lane, a.V);
      if (lane == l) mine = v;
    }
    return mine;
  };
  const ProbWalk wp = prob_total(a.nch, lane, sum);
  if (!(wp.total > 0.0)) return -1;
  const double t = (double)s.uf * wp.total;
  const int c = prob_find(wp, lane, t, sum, before);
  return prob_draw<T>(rows, c, lane, a.V, before, t);
}

// Chunk sums: one wave per (request, chunk).  Bound by memory where there is
// enough of it: 31 us for the 156 MB of 256 x 8 x 152064 float32 without draft rows
// (5.1 TB/s with what it reads twice; the fastest read of this card is 6.9), 12.2 us
// at 64 x 4 x 128256 float32 (52 MB read, 4.3 TB/s) and 8.8 us at 64 x 8 x 129279
// bfloat16 (26 MB read, 2.9 TB/s), of which the scan's two dependent round trips
// before the rows are some 3 us.  Registers allow seven waves a SIMD; eight spill (15.9 us
// instead of 12.0), chunks of 2048 leave too few waves (21.9 us instead of 18.8 for
// this kernel and the draw).
template <typename T>
__global__ __launch_bounds__(kProbPassThreads) void prob_pass_kernel(ProbArgs a, int nblk) {
  const int b = blockIdx.x / nblk;
  const int c = (blockIdx.x % nblk) * (kProbPassThreads / kWave) + threadIdx.x / kWave;
  const int lane = threadIdx.x % kWave;
  if (c >= a.nch) return;
  const ProbScan s = prob_scan<T>(a, b, lane);
  const ProbPlan p = prob_plan(a, s);
  if (prob_draws(s.path)) {
    const double w = prob_chunk<T>(prob_rows<T>(a, b, p), c, lane, a.V);
    if (lane == 0) a.recs[(size_t)b * a.nch + c] = w;
  }
  if (c == 0) {
    prob_outputs(a, b, lane, s, -1, 0.0);
    if (lane == 0) a.plans[b] = p;
  }
}

// The draws: one wave per request, a chain of round trips (records, the chunk).
// HELD: up to four batches of records are fetched at once, beside the plan, and
// kept in registers for both walks: 4.7 -> 4.2 us at 64 x 8 x 129279 bfloat16, 4.2 ->
// 3.9 us at 64 x 4 x 128256 float32.  (Four variables: an array that is indexed at
// run time leaves the registers, 8.7 us.)
constexpr int kProbHeld = 4;
template <typename T, bool HELD>
__global__ __launch_bounds__(kWave) void prob_draw_kernel(ProbArgs a) {
  const int b = blockIdx.x, lane = threadIdx.x;
  const double* recs = a.recs + (size_t)b * a.nch;
  auto load = [&](int i) {
    const int c = i * kProbBatch + lane;
    const double v = recs[min(c, a.nch - 1)];
    return c < a.nch ? v : 0.0;
  };
  double h0 = 0.0, h1 = 0.0, h2 = 0.0, h3 = 0.0;
  if constexpr (HELD) {
    h0 = load(0);
    h1 = load(1);
    h2 = load(2);
    h3 = load(3);
  }
  const ProbPlan p = a.plans[b];
  if (!prob_draws(p.path)) return;
  double mass;
  int y;
  if constexpr (HELD) {
    const double s0 = wave_sum(h0), s1 = wave_sum(h1), s2 = wave_sum(h2), s3 = wave_sum(h3);
    const double batch = lane == 0 ? s0 : lane == 1 ? s1 : lane == 2 ? s2 : lane == 3 ? s3 : 0.0;
    auto rec = [=](int i) { return i == 0 ? h0 : i == 1 ? h1 : i == 2 ? h2 : h3; };
    y = prob_pick<T>(a, b, lane, p, {batch, wave_sum(batch)}, rec, mass);
  } else {
    y = prob_pick<T>(a, b, lane, p, prob_total(a.nch, lane, load), load, mass);
  }
  if (y < 0) {
    prob_error(a, b, lane);
  } else if (lane == 0) {
    a.out_tokens[(size_t)b * (a.K + 1) + p.stop] = y;
    if (a.rmass_out) a.rmass_out[b] = mass;
  }
}

// Both in one workgroup per request: 7 us at 1 x 5 x 32000 float32, five dependent
// round trips; two chunks in flight a wave change nothing (6.8 us).
template <typename T>
__global__ __launch_bounds__(kProbOneThreads) void prob_one_kernel(ProbArgs a) {
  __shared__ double recs[kProbOneChunks];
  const int b = blockIdx.x, lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const ProbScan s = prob_scan<T>(a, b, lane);
  const ProbPlan p = prob_plan(a, s);
  if (prob_draws(s.path)) {
    const ProbRows<T> rows = prob_rows<T>(a, b, p);
    for (int c = wave; c < a.nch; c += kProbOneThreads / kWave) {
      const double w = prob_chunk<T>(rows, c, lane, a.V);
      if (lane == 0) recs[c] = w;
    }
  }
  __syncthreads();
  if (wave != 0) return;
  int y = -1;
  double mass = 0.0;
  if (prob_draws(s.path)) {
    auto rec = [&](int i) { return i * kProbBatch + lane < a.nch ? recs[i * kProbBatch + lane] : 0.0; };
    y = prob_pick<T>(a, b, lane, p, prob_total(a.nch, lane, rec), rec, mass);
    if (y < 0) {
      prob_error(a, b, lane);
      return;
    }
  }
  prob_outputs(a, b, lane, s, y, mass);
}

// Largest vocabulary the one-kernel form takes.  One kernel against two, us a
// call: 1 x 4096 4.5 / 6.6, 1 x 32000 7.4 / 7.4, 64 x 32000 9.7 / 10.7, then
// 1 x 65000 9.6 / 7.5 and 64 x 65000 15.2 / 12.8 (float32, 5 and 4 drafts): past
// some 32000 values one workgroup's pass over its row takes longer than a second
// launch and its wait.
constexpr int kProbOneV = 32768;
static_assert(kProbOneV <= kProbOneChunks * kProbChunk, "records fit LDS");

// Whether the launches of a call fit.
bool probs_fits(int B, int V) {
  if (V <= kProbOneV) return grid_fits(B, kProbOneThreads);
  const size_t nch = (size_t)((V + kProbChunk - 1) / kProbChunk);
  const size_t waves = kProbPassThreads / kWave;
  return grid_fits(B * ((nch + waves - 1) / waves), kProbPassThreads);
}

// 0: the one-kernel form needs none.
size_t probs_workspace_bytes(int B, int V) {
  if (V <= kProbOneV) return 0;
  const size_t nch = (size_t)((V + kProbChunk - 1) / kProbChunk);
  return (size_t)B * (sizeof(ProbPlan) + nch * sizeof(double));
}

hipError_t launch_verify_probs(bool bf16, const void* tgt, long long tsb, long long tsk,
                               const void* dft, long long dsb, long long dsk, const int* tokens,
                               const int* draft_len, const float* u, const float* u_final, int B,
                               int K, int V, int eos_id, int* out_tokens, int* n_emitted,
                               void* workspace, float* alpha_out, double* rmass_out, int* stop_out,
                               int* path_out, hipStream_t stream) {
  ProbArgs a;
  a.tgt = tgt;
  a.dft = dft;
  a.tsb = tsb;
  a.tsk = tsk;
  a.dsb = dsb;
  a.dsk = dsk;
  a.tokens = tokens;
  a.draft_len = draft_len;
  a.u = u;
  a.u_final = u_final;
  a.K = K;
  a.V = V;
  a.nch = (V + kProbChunk - 1) / kProbChunk;
  a.eos_id = eos_id;
  a.plans = static_cast<ProbPlan*>(workspace);
  a.recs = reinterpret_cast<double*>(a.plans + B);
  a.out_tokens = out_tokens;
  a.n_emitted = n_emitted;
  a.alpha_out = alpha_out;
  a.rmass_out = rmass_out;
  a.stop_out = stop_out;
  a.path_out = path_out;
  if (V <= kProbOneV) {
    if (bf16) prob_one_kernel<bf16_t><<<dim3(B), dim3(kProbOneThreads), 0, stream>>>(a);
    else prob_one_kernel<float><<<dim3(B), dim3(kProbOneThreads), 0, stream>>>(a);
    return hipGetLastError();
  }
  constexpr int kWaves = kProbPassThreads / kWave;
  const int nblk = (a.nch + kWaves - 1) / kWaves;
  const dim3 grid((unsigned)((size_t)B * nblk));
  if (bf16) prob_pass_kernel<bf16_t><<<grid, dim3(kProbPassThreads), 0, stream>>>(a, nblk);
  else prob_pass_kernel<float><<<grid, dim3(kProbPassThreads), 0, stream>>>(a, nblk);
  const bool held = a.nch <= kProbHeld * kProbBatch;
  auto draw = bf16 ? held ? prob_draw_kernel<bf16_t, true> : prob_draw_kernel<bf16_t, false>
                   : held ? prob_draw_kernel<float, true> : prob_draw_kernel<float, false>;
  draw<<<dim3(B), dim3(kWave), 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace specv
