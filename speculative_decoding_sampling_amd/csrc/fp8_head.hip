// The LM head on 8-bit floats (specv_fp8_lm_head), its weight layout and the
// quantiser of its operands.
//
//   logits[m][v] = sum_b hs[m][b] ws[v][b] sum_{d in run b} hq[m][d] wq[v][d]
//
// Elements are e4m3, each run of 128 along the hidden size has a power-of-two
// scale, and v_mfma_scale_f32_32x32x64_f8f6f4 applies both scales inside the
// matrix core: the running sum stays in the accumulators (float32), no vector
// instruction touches it between the runs.
//
// Orientation.  C^T = W H^T: the weights are the A operand (32 vocabulary
// rows), the hidden states the B operand (32 hidden rows).  A lane of the
// result holds one hidden row, col l % 32, and vocabulary rows 8 (i / 4) +
// i % 4 + 4 (l / 32) of accumulator register i.
//
// k order.  Per run of 128 lane l supplies bytes 64 (l / 32) .. + 63 of its
// row, 32 for each of the two products of the run; both operands share that
// order, and any order of k shared by both gives the same sum.  Both products
// lie in one run, so a lane's scale byte is that of its row and run whatever
// the matrix core's own 32-wide blocks are.
#include "fp8.h"
#include "specverify_ops.h"

namespace specv {

typedef int fp8_i32x8 __attribute__((ext_vector_type(8)));
typedef float fp8_f32x16 __attribute__((ext_vector_type(16)));

constexpr int kF8Group = 32;                       // vocabulary rows of a packed group
constexpr int kF8RunBytes = kF8Group * kFp8Block;  // packed bytes of one group's run (4 KB)
constexpr int kF8Waves = 4;
constexpr int kF8Threads = kF8Waves * kWave;

int fp8_groups(int V) { return (V + kF8Group - 1) / kF8Group; }
size_t fp8_packed_scale_off(int V, int D) {
  return (size_t)fp8_groups(V) * (D / kFp8Block) * kF8RunBytes;
}
size_t fp8_packed_bytes(int V, int D) {
  const int nk4 = (D / kFp8Block + 3) / 4;
  return fp8_packed_scale_off(V, D) + (size_t)fp8_groups(V) * nk4 * kF8Group * 4;
}

// ------------------------------------------------------------- quantise

// 8 values per thread, 16 lanes per run; rows are whole runs, so the array is
// one sequence of runs.
template <typename T>
__global__ __launch_bounds__(256) void fp8_quantize_kernel(const T* __restrict__ x, size_t n8,
                                                           uint8_t* __restrict__ q,
                                                           uint8_t* __restrict__ scale) {
  const size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
  const bool in = i < n8;                          // n8 is a multiple of 16: whole runs
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.f;
  if (in) {
#pragma unroll
    for (int j = 0; j < 8; j += Elem<T>::kPerVec) load_vec_fast(x + i * 8, j, v + j);
  }
  uint32_t byte;
  const uint2 w = fp8_pack8(v, byte);
  if (in) {
    *reinterpret_cast<uint2*>(q + i * 8) = w;
    if (threadIdx.x % kFp8Lanes == 0) scale[i / kFp8Lanes] = (uint8_t)byte;
  }
}

hipError_t launch_fp8_quantize(const void* x, bool bf16, int rows, int D, uint8_t* q,
                               uint8_t* scale, hipStream_t stream) {
  const size_t n8 = (size_t)rows * D / 8;
  const size_t blocks = (n8 + 255) / 256;
  if (blocks > 0x7fffffffu) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks);
  if (bf16)
    fp8_quantize_kernel<<<grid, dim3(256), 0, stream>>>(static_cast<const bf16_t*>(x), n8, q, scale);
  else
    fp8_quantize_kernel<<<grid, dim3(256), 0, stream>>>(static_cast<const float*>(x), n8, q, scale);
  return hipGetLastError();
}

// ----------------------------------------------------------------- pack

// One thread per 16-byte piece, then one per scale word.
__global__ __launch_bounds__(256) void fp8_pack_kernel(const uint8_t* __restrict__ q,
                                                       const uint8_t* __restrict__ scale,
                                                       uint8_t* __restrict__ packed, int V, int D,
                                                       size_t pieces, size_t words) {
  const size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int nkb = D / kFp8Block;
  if (i < pieces) {
    const int lane = (int)(i % kWave);
    size_t r = i / kWave;
    const int s = (int)(r % 4);
    r /= 4;
    const int kb = (int)(r % nkb);
    const size_t v = r / nkb * kF8Group + lane % 32;
    const int k = kb * kFp8Block + 64 * (lane / 32) + 16 * s;
    uint4 val = make_uint4(0u, 0u, 0u, 0u);
    if (v < (size_t)V) val = *reinterpret_cast<const uint4*>(q + v * D + k);
    *reinterpret_cast<uint4*>(packed + i * 16) = val;
  } else if (i - pieces < words) {
    const size_t w = i - pieces;
    const int nk4 = (nkb + 3) / 4;
    const int row = (int)(w % kF8Group);
    const int j = (int)(w / kF8Group % nk4);
    const size_t v = w / kF8Group / nk4 * kF8Group + row;
    uint32_t word = 0;
    for (int e = 0; e < 4; ++e) {
      const uint32_t byte = v < (size_t)V && 4 * j + e < nkb ? scale[v * nkb + 4 * j + e] : 127u;
      word |= byte << (8 * e);
    }
    *reinterpret_cast<uint32_t*>(packed + pieces * 16 + w * 4) = word;
  }
}

hipError_t launch_fp8_pack(const uint8_t* q, const uint8_t* scale, void* packed, int V, int D,
                           hipStream_t stream) {
  const size_t pieces = fp8_packed_scale_off(V, D) / 16;
  const size_t words = (fp8_packed_bytes(V, D) - pieces * 16) / 4;
  const size_t blocks = (pieces + words + 255) / 256;
  if (blocks > 0x7fffffffu) return hipErrorInvalidConfiguration;
  fp8_pack_kernel<<<dim3((unsigned)blocks), dim3(256), 0, stream>>>(
      q, scale, static_cast<uint8_t*>(packed), V, D, pieces, words);
  return hipGetLastError();
}

// -------------------------------------------------------------- product

__device__ __forceinline__ fp8_i32x8 fp8_operand(uint4 lo, uint4 hi) {
  fp8_i32x8 r = {(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w,
                 (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
  return r;
}

// One product step of run i (0..3, its byte of the scale words).
template <int I>
__device__ __forceinline__ fp8_f32x16 fp8_mfma(fp8_i32x8 a, fp8_i32x8 b, fp8_f32x16 c, uint32_t sa,
                                               uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, I, (int)sa, I, (int)sb);
}

__device__ __forceinline__ void f8_put(float* p, float v) { *p = v; }
__device__ __forceinline__ void f8_put(bf16_t* p, float v) { *p = (bf16_t)bf16_bits(v); }

// Few hidden rows: the weights are read straight into registers, once, and
// the kernel is bound by them.  A workgroup owns 32 vocabulary rows and up to
// 32 MT hidden rows; its four waves split the runs (groups of four, one scale
// word) and add their sums through LDS in a fixed order.
template <int MT, typename O>
__global__ __launch_bounds__(kF8Threads) void fp8_skinny_kernel(
    const uint8_t* __restrict__ H, const uint8_t* __restrict__ hs, const uint8_t* __restrict__ P,
    const uint32_t* __restrict__ ws, int M, int D, int V, int ngroup, O* __restrict__ out) {
  __shared__ float red[kF8Waves][MT * 32][33];
  const int group = blockIdx.x % ngroup;
  const int m0 = (blockIdx.x / ngroup) * (32 * MT);
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int h = lane / 32, l32 = lane % 32;
  const int nkb = D / kFp8Block, nk4 = (nkb + 3) / 4;
  const uint8_t* wrow = P + (size_t)group * nkb * kF8RunBytes + lane * 16;
  const uint32_t* wsc = ws + (size_t)group * nk4 * kF8Group + l32;
  const uint8_t* hrow[MT];
  const uint8_t* hsc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const size_t m = (size_t)min(m0 + 32 * t + l32, M - 1);   // rows past M repeat the last
    hrow[t] = H + m * D + 64 * h;
    hsc[t] = hs + m * nkb;
  }
  fp8_f32x16 acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[t][r] = 0.f;

  auto run = [&](auto idx, int kb, uint32_t sa, const uint32_t* sb) {
    constexpr int I = decltype(idx)::value;
    uint4 a[4];
#pragma unroll
    for (int s = 0; s < 4; ++s)
      a[s] = *reinterpret_cast<const uint4*>(wrow + (size_t)kb * kF8RunBytes + s * 1024);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      uint4 b[4];
#pragma unroll
      for (int s = 0; s < 4; ++s)
        b[s] = *reinterpret_cast<const uint4*>(hrow[t] + kb * kFp8Block + 16 * s);
      acc[t] = fp8_mfma<I>(fp8_operand(a[0], a[1]), fp8_operand(b[0], b[1]), acc[t], sa, sb[t]);
      acc[t] = fp8_mfma<I>(fp8_operand(a[2], a[3]), fp8_operand(b[2], b[3]), acc[t], sa, sb[t]);
    }
  };
  for (int g = wave; g < nk4; g += kF8Waves) {
    const uint32_t sa = wsc[g * kF8Group];
    const int left = nkb - 4 * g;
    uint32_t sb[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      sb[t] = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < left) sb[t] |= (uint32_t)hsc[t][4 * g + e] << (8 * e);
    }
    run(std::integral_constant<int, 0>{}, 4 * g, sa, sb);
    if (left > 1) run(std::integral_constant<int, 1>{}, 4 * g + 1, sa, sb);
    if (left > 2) run(std::integral_constant<int, 2>{}, 4 * g + 2, sa, sb);
    if (left > 3) run(std::integral_constant<int, 3>{}, 4 * g + 3, sa, sb);
  }
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r)
      red[wave][32 * t + l32][8 * (r / 4) + r % 4 + 4 * h] = acc[t][r];
  __syncthreads();
  for (int i = threadIdx.x; i < MT * 32 * 32; i += kF8Threads) {
    const int m = i / 32, v = i % 32;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kF8Waves; ++w) s += red[w][m][v];
    if (m0 + m < M && group * kF8Group + v < V)
      f8_put(out + (size_t)(m0 + m) * V + group * kF8Group + v, s);
  }
}

template <typename O>
hipError_t fp8_head(const uint8_t* H, const uint8_t* hs, const uint8_t* P, int M, int D, int V,
                    O* out, hipStream_t stream) {
  const uint32_t* ws = reinterpret_cast<const uint32_t*>(P + fp8_packed_scale_off(V, D));
  const int ng = fp8_groups(V);
  const int mt = M <= 32 ? 1 : 2;
  const size_t blocks = (size_t)ng * ((M + 32 * mt - 1) / (32 * mt));
  if (blocks > 0x7fffffffu) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks), thr(kF8Threads);
  if (mt == 1) fp8_skinny_kernel<1, O><<<grid, thr, 0, stream>>>(H, hs, P, ws, M, D, V, ng, out);
  else fp8_skinny_kernel<2, O><<<grid, thr, 0, stream>>>(H, hs, P, ws, M, D, V, ng, out);
  return hipGetLastError();
}

hipError_t launch_fp8_head(const uint8_t* hidden, const uint8_t* hscale, const void* packed, int M,
                           int D, int V, void* logits, bool bf16, hipStream_t stream) {
  const uint8_t* P = static_cast<const uint8_t*>(packed);
  if (bf16)
    return fp8_head(hidden, hscale, P, M, D, V, static_cast<bf16_t*>(logits), stream);
  return fp8_head(hidden, hscale, P, M, D, V, static_cast<float*>(logits), stream);
}

// Largest grid of any product (workgroups), for the host's size check.
size_t fp8_head_blocks(int M, int V) { return (size_t)fp8_groups(V) * ((M + 31) / 32); }

}  // namespace specv
