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
// side, a kernel boundary would not.  Then one wave per request walks the
// chunk sums to the chunk that holds the draw and scans that chunk.  Small
// vocabularies do both in one workgroup per request, the chunk sums in LDS.
#include "common.h"
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

// Sums over a chunk: w the weights the draw uses (the residual after a
// rejection, p otherwise), p the target row.  NaN marks an invalid entry.
struct ProbRec {
  double w, p;
};

struct ProbArgs {
  const void* tgt;
  const void* dft;                  // null: one at the drafted token
  long long tsb, tsk, dsb, dsk;     // strides in elements
  const int* tokens;
  const int* draft_len;
  const float* u;
  const float* u_final;
  int K, V, nch, eos_id;
  ProbRec* recs;                    // [B][nch]
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

// The rows the draw of a scanned request reads.
template <typename T>
struct ProbRows {
  const T* p;
  const T* q;         // null: none, or one at token hot
  int hot;            // the drafted token of a rejection without draft rows, else -1
};

template <typename T>
__device__ __forceinline__ ProbRows<T> prob_rows(const ProbArgs& a, int b, const ProbScan& s) {
  ProbRows<T> r;
  r.p = static_cast<const T*>(a.tgt) + (size_t)b * a.tsb + (size_t)s.stop * a.tsk;
  r.q = nullptr;
  r.hot = -1;
  if (s.path == kPathReject) {
    if (a.dft) r.q = static_cast<const T*>(a.dft) + (size_t)b * a.dsb + (size_t)s.stop * a.dsk;
    else r.hot = lane_value(s.x, s.stop);
  }
  return r;
}

// The weight of one token; NaN for an invalid entry.
__device__ __forceinline__ double prob_weight(float p, float q) {
  const double d = (double)p - (double)q;
  const double w = d > 0.0 ? d : 0.0;
  return prob_ok(p) && prob_ok(q) ? w : __builtin_nan("");
}

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
        out[j * N + i] = v < V ? to_f32(row[v]) : 0.f;
      }
  }
}

// Sums of chunk c, by one wave (every lane gets them).
template <typename T>
__device__ __forceinline__ ProbRec prob_chunk(const ProbRows<T>& r, int c, int lane, int V) {
  const int base = c * kProbChunk;
  float p[kProbPer], q[kProbPer];
  prob_load<T, true>(r.p, base, lane, V, p);
  if (r.q) prob_load<T, true>(r.q, base, lane, V, q);
  else
#pragma unroll
    for (int i = 0; i < kProbPer; ++i) q[i] = 0.f;
  constexpr int N = Elem<T>::kPerVec;
  double w = 0.0, sp = 0.0;
#pragma unroll
  for (int j = 0; j < kProbPer / N; ++j)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = j * N + i;
      float qe = q[e];
      if (base + (j * kWave + lane) * N + i == r.hot) qe = 1.f;
      w += prob_weight(p[e], qe);
      sp += (double)p[e];
    }
  ProbRec rec;
  rec.w = wave_sum(w);
  rec.p = wave_sum(sp);
  return rec;
}

// The token of chunk c at t, base being the weights before the chunk: the
// first whose running sum exceeds t, or where rounding leaves none the last
// with a positive weight.
template <typename T>
__device__ __forceinline__ int prob_draw(const ProbRows<T>& r, int c, int lane, int V, bool use_p,
                                         double base, double t) {
  const int v0 = c * kProbChunk;
  float p[kProbPer], q[kProbPer];
  prob_load<T, false>(r.p, v0, lane, V, p);
  if (r.q && !use_p) prob_load<T, false>(r.q, v0, lane, V, q);
  else
#pragma unroll
    for (int i = 0; i < kProbPer; ++i) q[i] = 0.f;
  if (!use_p && r.hot >= v0 + lane * kProbPer && r.hot < v0 + (lane + 1) * kProbPer) {
#pragma unroll
    for (int i = 0; i < kProbPer; ++i)
      if (v0 + lane * kProbPer + i == r.hot) q[i] = 1.f;
  }
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
    if (first == kProbPer && run > t) first = i;
    if (w > 0.0) last = i;
  }
  const uint64_t over = __ballot(base + incl > t && sum > 0.0);
  const uint64_t some = __ballot(sum > 0.0);
  const int L = over ? __ffsll((unsigned long long)over) - 1
                     : some ? 63 - __clzll((long long)some) : 0;
  const int pick = first < kProbPer && over ? first : last;
  return v0 + L * kProbPer + lane_value(pick, L);
}

// The draw of a scanned request from its chunk records, and the request's
// outputs, by one wave.
template <typename T>
__device__ __forceinline__ void prob_finish(const ProbArgs& a, int b, int lane, ProbScan s,
                                            const ProbRec* recs) {
  int y = -1;
  double mass = 0.0;
  if (s.path == kPathReject || s.path == kPathBonus) {
    const ProbRows<T> rows = prob_rows<T>(a, b, s);
    // lane i keeps the totals of record batch i
    const int nbatch = (a.nch + kProbBatch - 1) / kProbBatch;
    double bw = 0.0, bp = 0.0;
    for (int i = 0; i < nbatch; ++i) {
      const int c = i * kProbBatch + lane;
      ProbRec r = {0.0, 0.0};
      if (c < a.nch) r = recs[c];
      const double sw = wave_sum(r.w), sp = wave_sum(r.p);
      if (lane == i) {
        bw = sw;
        bp = sp;
      }
    }
    const double W = wave_sum(bw), P = wave_sum(bp);
    if (s.path == kPathReject) mass = W;
    // an empty residual: the correction is drawn from p itself
    const bool use_p = s.path == kPathReject && W == 0.0;
    const double total = use_p ? P : W;
    if (!(total > 0.0) || !(W >= 0.0)) {                   // zero or NaN
      s.path = kPathError;
    } else {
      const double t = (double)s.uf * total;
      const double bt = use_p ? bp : bw;
      const double bincl = wave_incl_scan(bt);
      const uint64_t bover = __ballot(bincl > t && bt > 0.0);
      const uint64_t bsome = __ballot(bt > 0.0);
      const int bi = bover ? __ffsll((unsigned long long)bover) - 1
                           : 63 - __clzll((long long)bsome);
      const double before = lane_value(wave_shr1(bincl), bi);
      const int c = bi * kProbBatch + lane;
      ProbRec r = {0.0, 0.0};
      if (c < a.nch) r = recs[c];
      const double ct = use_p ? r.p : r.w;
      const double cincl = before + wave_incl_scan(ct);
      const uint64_t cover = __ballot(cincl > t && ct > 0.0);
      const uint64_t csome = __ballot(ct > 0.0);
      const int ci = cover ? __ffsll((unsigned long long)cover) - 1
                           : 63 - __clzll((long long)csome);
      const double base = ci ? lane_value(cincl, ci - 1) : before;
      y = prob_draw<T>(rows, bi * kProbBatch + ci, lane, a.V, use_p, base, t);
    }
  }
  const bool err = s.path == kPathError;
  for (int k = lane; k <= a.K; k += kWave) {
    int v = -1;
    if (!err) {
      if (k < s.stop || (k == s.stop && s.path == kPathEos)) v = s.x;   // k = lane < 64 here
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

// Chunk sums: one wave per (request, chunk).
template <typename T>
__global__ __launch_bounds__(kProbPassThreads) void prob_pass_kernel(ProbArgs a, int nblk) {
  const int b = blockIdx.x / nblk;
  const int c = (blockIdx.x % nblk) * (kProbPassThreads / kWave) + threadIdx.x / kWave;
  const int lane = threadIdx.x % kWave;
  if (c >= a.nch) return;
  const ProbScan s = prob_scan<T>(a, b, lane);
  if (s.path != kPathReject && s.path != kPathBonus) return;
  const ProbRec r = prob_chunk<T>(prob_rows<T>(a, b, s), c, lane, a.V);
  if (lane == 0) a.recs[(size_t)b * a.nch + c] = r;
}

// The draws: one wave per request.
template <typename T>
__global__ __launch_bounds__(kWave) void prob_draw_kernel(ProbArgs a) {
  const int b = blockIdx.x, lane = threadIdx.x;
  const ProbScan s = prob_scan<T>(a, b, lane);
  prob_finish<T>(a, b, lane, s, a.recs + (size_t)b * a.nch);
}

// Both in one workgroup per request.
template <typename T>
__global__ __launch_bounds__(kProbOneThreads) void prob_one_kernel(ProbArgs a) {
  __shared__ ProbRec recs[kProbOneChunks];
  const int b = blockIdx.x, lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const ProbScan s = prob_scan<T>(a, b, lane);
  if (s.path == kPathReject || s.path == kPathBonus) {
    const ProbRows<T> rows = prob_rows<T>(a, b, s);
    for (int c = wave; c < a.nch; c += kProbOneThreads / kWave) {
      const ProbRec r = prob_chunk<T>(rows, c, lane, a.V);
      if (lane == 0) recs[c] = r;
    }
  }
  __syncthreads();
  if (wave == 0) prob_finish<T>(a, b, lane, s, recs);
}

// Largest vocabulary the one-kernel form takes.
constexpr int kProbOneV = 32768;
static_assert(kProbOneV <= kProbOneChunks * kProbChunk, "records fit LDS");

size_t probs_workspace_bytes(int B, int V) {
  const size_t nch = (size_t)((V + kProbChunk - 1) / kProbChunk);
  return (size_t)B * nch * sizeof(ProbRec);
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
  a.recs = static_cast<ProbRec*>(workspace);
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
  if ((size_t)B * nblk > 0x7fffffffu) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)((size_t)B * nblk));
  if (bf16) {
    prob_pass_kernel<bf16_t><<<grid, dim3(kProbPassThreads), 0, stream>>>(a, nblk);
    prob_draw_kernel<bf16_t><<<dim3(B), dim3(kWave), 0, stream>>>(a);
  } else {
    prob_pass_kernel<float><<<grid, dim3(kProbPassThreads), 0, stream>>>(a, nblk);
    prob_draw_kernel<float><<<dim3(B), dim3(kWave), 0, stream>>>(a);
  }
  return hipGetLastError();
}

}  // namespace specv
