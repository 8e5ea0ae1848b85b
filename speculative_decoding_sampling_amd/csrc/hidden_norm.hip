// The norms around the target's last block, its gate and its residual scale
// in one pass (specv_hidden_norm):
//
//   r' = r + scale * g * N(x; w1),  y = N(r'; w2),  N(v; w) = w v / sqrt(mean(v^2) + eps)
//
// Every row is read once, kept in registers through both reductions and
// written once (r' and y), so the bytes moved are the floor.  A workgroup owns
// a row, each thread 8 values, up to 1024 threads: a row's latency is two
// reductions and is shortest with the fewest values a thread (5 x 4096 bfloat16:
// 512 threads 4.2 us, 256 5.4, 128 8.1), and many rows keep two to four
// workgroups on a compute unit.  The sums of squares are float32: per thread
// in order, then the wave and the waves' sums on DPP moves, a fixed order.
//
// 2304 x 8192: 30.2 us from bfloat16 to 8-bit values (4.4 TB/s), 44.6 us with a
// float32 residual (4.7 TB/s; a large copy reaches 4.9).  The narrow types are
// bound by their instructions as much as by memory: packed conversions, one
// reciprocal root and DPP sums took the first from 37.9 to 33.0 us.  Workgroups
// that stay and fetch the next row ahead gained 6 % there before that and lost
// 24 % with a float32 residual (registers); loads past the caches gained 8 % there
// and lost 9 % at 1024 x 8192, where the rows still lie in them; weights fetched
// before the first reduction gained 6 % at 320 x 4096 and lost 11 % at 2304 x 8192.
// Rows of other than whole 8s, element by element: 2304 x 8191 bfloat16 36.8 us
// (4.1 TB/s).  Past 16384 values every row takes the kernel of eight groups a
// thread, those past its end masked: 1152 x 16384 bfloat16 32.5 us (4.6 TB/s),
// 16392 63 us, 32768 86 us (3.5 TB/s), 576 x 65536 80 us (3.8 TB/s).
//
// y is formed from r' before r' is rounded to its own type: one rounding less
// between the residual stream and the logits.
#include "fp8.h"
#include "grid.h"
#include "specverify_ops.h"

namespace specv {

constexpr int kNormMaxThreads = 1024;

struct NormArgs {
  const void* x;
  const void* r;
  const void* w1;       // null: x as it is
  const void* gate;     // null: a factor of one
  const void* w2;
  void* r_out;
  void* out;
  uint8_t* out_scale;
  int D, rows_per_gate;
  bool w_bf16;          // type of w1, gate and w2
  float scale, eps, inv_d;
};

// How a thread's 8 values of a group lie in the row: 8 neighbours in 16-byte
// loads; 8 neighbours one at a time (8-bit output of arrays off 16 bytes, whose
// runs of 128 are 16 threads'); or a workgroup's width apart, one at a time, so
// that neighbouring threads read neighbouring values (rows of any length: 8.8
// -> 4.6 us at 37 x 2047 float32 against 8 neighbours).
enum NormLayout { kWide, kNeighbours, kApart };

// Values e0, e0 + es, .. of a row as floats; those at or past D read as 0.  No
// branches: each would make the loads behind it wait for those before it.
template <typename T, int LAYOUT>
__device__ __forceinline__ void norm_load(const T* row, int e0, int es, int D, float* v) {
  if constexpr (LAYOUT == kWide) {                       // D is a multiple of 8
    const int e = min(e0, D - 8);
#pragma unroll
    for (int i = 0; i < 8; i += Elem<T>::kPerVec) load_vec_fast(row, e + i, v + i);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(row[min(e0 + i * es, D - 1)]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = e0 + i * es < D ? v[i] : 0.f;
}

// The same for a weight row of either type (uniform over the grid).
template <int LAYOUT>
__device__ __forceinline__ void norm_load_w(const void* w, bool w_bf16, size_t off, int e0, int es,
                                            int D, float* v) {
  if (w_bf16) norm_load<bf16_t, LAYOUT>(static_cast<const bf16_t*>(w) + off, e0, es, D, v);
  else norm_load<float, LAYOUT>(static_cast<const float*>(w) + off, e0, es, D, v);
}

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(bf16_t* p, float v) { *p = bf16_bits(v); }

template <typename T, int LAYOUT>
__device__ __forceinline__ void norm_store(T* row, int e0, int es, int D, const float* v) {
  if constexpr (LAYOUT == kWide) {
    if (e0 >= D) return;
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(row + e0) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(row + e0 + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      uint4 w;
      w.x = bf16_pair(v[0], v[1]);
      w.y = bf16_pair(v[2], v[3]);
      w.z = bf16_pair(v[4], v[5]);
      w.w = bf16_pair(v[6], v[7]);
      *reinterpret_cast<uint4*>(row + e0) = w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (e0 + i * es < D) put(row + e0 + i * es, v[i]);
  }
}

// Sum over each row of 16 lanes, the same bits in all of them: every step adds
// two partial sums that both lanes hold.
__device__ __forceinline__ float row16_sum(float v) {
  v += dpp_f32<0xb1>(v);
  v += dpp_f32<0x4e>(v);
  v += dpp_f32<0x141>(v);
  return v + dpp_f32<0x140>(v);
}

// Sum over the workgroup, the same value in every thread.  Two calls use two
// arrays, so the second needs no barrier before it.
static_assert(kNormMaxThreads / kWave <= 16, "a row of lanes sums the waves");
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = wave_sum(v);
  const int nw = blockDim.x / kWave, i = threadIdx.x % 16;
  if (nw == 1) return v;
  if (threadIdx.x % kWave == 0) red[threadIdx.x / kWave] = v;
  __syncthreads();
  return row16_sum(i < nw ? red[i] : 0.f);
}

// 1 / sqrt(v) for v >= 0.  The instruction is within a step of it, but takes
// subnormal numbers as 0.
__device__ __forceinline__ float inv_root(float v) {
  const bool tiny = v < 0x1p-100f;
  const float r = __builtin_amdgcn_rsqf(tiny ? v * 0x1p100f : v);
  return tiny ? r * 0x1p50f : r;
}

// Rows of more than 2 groups per thread leave the residual in memory until
// the first reduction is done: with both rows in registers 1024 threads
// would spill.
template <typename X, typename R, int OUT, int NV, int LAYOUT>
__global__ __launch_bounds__(kNormMaxThreads) void hidden_norm_kernel(NormArgs a) {
  constexpr bool kEarly = NV <= 2;
  __shared__ float red[2][kNormMaxThreads / kWave];
  const int m = blockIdx.x, D = a.D;
  const size_t off = (size_t)m * D;
  const X* x = static_cast<const X*>(a.x) + off;
  const R* r = static_cast<const R*>(a.r) + off;
  const size_t goff = (size_t)(m / a.rows_per_gate) * D;

  // group j's first value and the distance to the next
  const int es = LAYOUT == kApart ? (int)blockDim.x : 1;
  auto at = [&](int j) {
    return LAYOUT == kApart ? (int)(j * 8 * blockDim.x + threadIdx.x)
                            : (int)(threadIdx.x + j * blockDim.x) * 8;
  };

  float h[NV][8], res[kEarly ? NV : 1][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e0 = at(j);
    norm_load<X, LAYOUT>(x, e0, es, D, h[j]);
  }
  float f = a.scale, ss = 0.f;
  if (a.w1) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(h[j][i], h[j][i], ss);
  }
  // The residual is fetched while the first reduction runs: before it, its
  // reads delay those that the reduction waits for (2304 x 8192 bfloat16 to 8
  // bits 32.2 -> 30.2 us, 320 x 4096 with a float32 residual 6.0 -> 5.6 us).
  __builtin_amdgcn_sched_barrier(0);
  if constexpr (kEarly) {
#pragma unroll
    for (int j = 0; j < NV; ++j) norm_load<R, LAYOUT>(r, at(j), es, D, res[j]);
  }
  __builtin_amdgcn_sched_barrier(0);
  if (a.w1) f = a.scale * inv_root(fmaf(block_sum(ss, red[0]), a.inv_d, a.eps));
  ss = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e0 = at(j);
    float c[8];
    if (a.w1) {
      norm_load_w<LAYOUT>(a.w1, a.w_bf16, 0, e0, es, D, c);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[j][i] *= c[i];
    }
    if (a.gate) {
      norm_load_w<LAYOUT>(a.gate, a.w_bf16, goff, e0, es, D, c);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[j][i] *= c[i];
    }
    float* rj = res[kEarly ? j : 0];
    if constexpr (!kEarly) norm_load<R, LAYOUT>(r, e0, es, D, rj);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      h[j][i] = fmaf(f, h[j][i], rj[i]);
      ss = fmaf(h[j][i], h[j][i], ss);
    }
    norm_store<R, LAYOUT>(static_cast<R*>(a.r_out) + off, e0, es, D, h[j]);
  }
  f = inv_root(fmaf(block_sum(ss, red[1]), a.inv_d, a.eps));
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e0 = at(j);
    float c[8];
    norm_load_w<LAYOUT>(a.w2, a.w_bf16, 0, e0, es, D, c);
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] *= h[j][i] * f;
    if constexpr (OUT == SPECV_OUT_E4M3) {
      // 16 lanes hold a run of 128; D is a multiple of it, so a run is wholly
      // inside the row or wholly past it
      uint32_t byte;
      const uint2 q = fp8_pack8(c, byte);
      if (e0 < D) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + off + e0) = q;
        if (threadIdx.x % kFp8Lanes == 0) a.out_scale[(off + e0) / kFp8Block] = (uint8_t)byte;
      }
    } else if constexpr (OUT == SPECV_OUT_F32) {
      norm_store<float, LAYOUT>(static_cast<float*>(a.out) + off, e0, es, D, c);
    } else {
      norm_store<bf16_t, LAYOUT>(static_cast<bf16_t*>(a.out) + off, e0, es, D, c);
    }
  }
}

template <typename X, typename R, int OUT, int NV>
void norm_launch(const NormArgs& a, int M, int threads, bool vec, hipStream_t stream) {
  constexpr int kNarrow = OUT == SPECV_OUT_E4M3 ? kNeighbours : kApart;
  if (vec) hidden_norm_kernel<X, R, OUT, NV, kWide><<<dim3(M), dim3(threads), 0, stream>>>(a);
  else hidden_norm_kernel<X, R, OUT, NV, kNarrow><<<dim3(M), dim3(threads), 0, stream>>>(a);
}

int norm_threads(int D) {
  const int groups = (D + 7) / 8;
  return groups >= kNormMaxThreads ? kNormMaxThreads : (groups + kWave - 1) / kWave * kWave;
}
bool hidden_norm_fits(int M, int D) { return grid_fits(M, norm_threads(D)); }

template <typename X, typename R, int OUT>
void norm_by_size(const NormArgs& a, int M, bool vec, hipStream_t stream) {
  const int groups = (a.D + 7) / 8, threads = norm_threads(a.D);
  const int nv = (groups + threads - 1) / threads;
  if (nv == 1) norm_launch<X, R, OUT, 1>(a, M, threads, vec, stream);
  else if (nv == 2) norm_launch<X, R, OUT, 2>(a, M, threads, vec, stream);
  else norm_launch<X, R, OUT, 8>(a, M, threads, vec, stream);
}
static_assert(SPECV_MAX_D <= 8 * 8 * kNormMaxThreads, "a row fits a workgroup's registers");

template <typename X, typename R>
void norm_by_out(const NormArgs& a, int M, int out, bool vec, hipStream_t stream) {
  if (out == SPECV_OUT_E4M3) norm_by_size<X, R, SPECV_OUT_E4M3>(a, M, vec, stream);
  else if (out == SPECV_OUT_BF16) norm_by_size<X, R, SPECV_OUT_BF16>(a, M, vec, stream);
  else norm_by_size<X, R, SPECV_OUT_F32>(a, M, vec, stream);
}

hipError_t launch_hidden_norm(const void* x, bool xb, const void* r, bool rb, const void* w1,
                              const void* gate, int gate_rows, const void* w2, bool wb, int M,
                              int D, float scale, float eps, void* r_out, void* out, int out_dtype,
                              uint8_t* out_scale, hipStream_t stream) {
  NormArgs a;
  a.x = x;
  a.r = r;
  a.w1 = w1;
  a.gate = gate;
  a.w2 = w2;
  a.r_out = r_out;
  a.out = out;
  a.out_scale = out_scale;
  a.D = D;
  a.rows_per_gate = gate ? M / gate_rows : 1;
  a.w_bf16 = wb;
  a.scale = scale;
  a.eps = eps;
  a.inv_d = 1.f / (float)D;
  auto al = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  const bool vec = D % 8 == 0 && al(x) && al(r) && al(w1) && al(gate) && al(w2) && al(r_out) &&
                   (out_dtype == SPECV_OUT_E4M3 || al(out));
  if (xb) {
    if (rb) norm_by_out<bf16_t, bf16_t>(a, M, out_dtype, vec, stream);
    else norm_by_out<bf16_t, float>(a, M, out_dtype, vec, stream);
  } else {
    if (rb) norm_by_out<float, bf16_t>(a, M, out_dtype, vec, stream);
    else norm_by_out<float, float>(a, M, out_dtype, vec, stream);
  }
  return hipGetLastError();
}

}  // namespace specv
