// The LM head on 4-bit floats (specv_fp4_lm_head), its weight layout and the
// quantiser of its operands.
//
//   logits[m][v] = sum_d h[m][d] w[v][d]
//
// Weights are e2m1 codes with a power-of-two scale for each 32 along the hidden
// size; hidden states are the same, or e4m3 bytes with a scale for each 128.
// v_mfma_scale_f32_32x32x64_f8f6f4 takes either pair and applies both scales.
//
// Orientation.  C^T = W H^T: the weights are the A operand (32 vocabulary
// rows), the hidden states the B operand (32 hidden rows).  A lane of the
// result holds one hidden row, col l % 32, and vocabulary rows 8 (i / 4) +
// i % 4 + 4 (l / 32) of accumulator register i.
//
// k order.  Of a step's 64 columns lane l holds, in 4 bits, 32 (l / 32) .. + 31,
// one block, and supplies that block's scale.  In 8 bits its first 16 bytes are
// columns 16 (l / 32) .. + 15 and its last 16 columns 32 + 16 (l / 32) .. + 15
// (measured with single products); the scale that it supplies is still that of
// columns 32 (l / 32) .. + 31, the same byte for all 64 as an e4m3 run is 128.
#include "fp4.h"
#include "fp8.h"
#include "grid.h"
#include "specverify_draft.h"

namespace specv {

typedef int fp4_i32x8 __attribute__((ext_vector_type(8)));
typedef float fp4_f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 fp4_bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 fp4_bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kF4Group = 32;                       // vocabulary rows of a packed group
constexpr int kF4Step = 64;                        // columns of one product
constexpr int kF4StepBytes = kF4Group * kF4Step / 2;   // packed bytes of a group's step (1 KB)
constexpr int kF4Waves = 4;
constexpr int kF4Threads = kF4Waves * kWave;

int fp4_groups(int V) { return (V + kF4Group - 1) / kF4Group; }
size_t fp4_packed_scale_off(int V, int D) {
  return (size_t)fp4_groups(V) * (D / kF4Step) * kF4StepBytes;
}
size_t fp4_packed_bytes(int V, int D) {
  const int nj = (D / kF4Step + 3) / 4;
  return fp4_packed_scale_off(V, D) + (size_t)fp4_groups(V) * nj * kWave * 4;
}

// ------------------------------------------------------------- quantise

// 8 values per thread, 4 lanes per block; rows are whole blocks, so the array
// is one sequence of blocks.
template <typename T>
__global__ __launch_bounds__(256) void fp4_quantize_kernel(const T* __restrict__ x, size_t n8,
                                                           uint32_t* __restrict__ q,
                                                           uint8_t* __restrict__ scale) {
  const size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
  const bool in = i < n8;                          // n8 is a multiple of 4: whole blocks
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.f;
  if (in) {
#pragma unroll
    for (int j = 0; j < 8; j += Elem<T>::kPerVec) load_vec_fast(x + i * 8, j, v + j);
  }
  uint32_t byte;
  const uint32_t w = fp4_pack8(v, byte);
  if (in) {
    q[i] = w;
    if (threadIdx.x % kFp4Lanes == 0) scale[i / kFp4Lanes] = (uint8_t)byte;
  }
}

bool fp4_quantize_fits(int rows, int D) { return grid_fits(((size_t)rows * D / 8 + 255) / 256, 256); }

hipError_t launch_fp4_quantize(const void* x, bool bf16, int rows, int D, uint8_t* q,
                               uint8_t* scale, hipStream_t stream) {
  const size_t n8 = (size_t)rows * D / 8;
  const dim3 grid((unsigned)((n8 + 255) / 256));
  uint32_t* q4 = reinterpret_cast<uint32_t*>(q);
  if (bf16)
    fp4_quantize_kernel<<<grid, dim3(256), 0, stream>>>(static_cast<const bf16_t*>(x), n8, q4, scale);
  else
    fp4_quantize_kernel<<<grid, dim3(256), 0, stream>>>(static_cast<const float*>(x), n8, q4, scale);
  return hipGetLastError();
}

// ----------------------------------------------------------------- pack

// One thread per 16-byte piece, then one per scale word.
__global__ __launch_bounds__(256) void fp4_pack_kernel(const uint8_t* __restrict__ q,
                                                       const uint8_t* __restrict__ scale,
                                                       uint8_t* __restrict__ packed, int V, int D,
                                                       size_t pieces, size_t words) {
  const size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int lane = (int)(i % kWave);               // pieces are a multiple of 64: words' too
  const int steps = D / kF4Step, nb = D / kFp4Block;
  if (i < pieces) {
    const size_t r = i / kWave;
    const size_t v = r / steps * kF4Group + lane % 32;
    const int k = (int)(r % steps) * kF4Step + 32 * (lane / 32);
    uint4 val = make_uint4(0u, 0u, 0u, 0u);
    if (v < (size_t)V) val = *reinterpret_cast<const uint4*>(q + (v * D + k) / 2);
    *reinterpret_cast<uint4*>(packed + i * 16) = val;
  } else if (i - pieces < words) {
    const size_t r = (i - pieces) / kWave;
    const int nj = (steps + 3) / 4;
    const int j = (int)(r % nj);
    const size_t v = r / nj * kF4Group + lane % 32;
    uint32_t word = 0;
    for (int e = 0; e < 4; ++e) {
      const int b = 8 * j + 2 * e + lane / 32;
      const uint32_t byte = v < (size_t)V && b < nb ? scale[v * nb + b] : 127u;
      word |= byte << (8 * e);
    }
    *reinterpret_cast<uint32_t*>(packed + pieces * 16 + (i - pieces) * 4) = word;
  }
}

bool fp4_pack_fits(int V, int D) {
  const size_t pieces = fp4_packed_scale_off(V, D) / 16;
  return grid_fits((pieces + (fp4_packed_bytes(V, D) - pieces * 16) / 4 + 255) / 256, 256);
}

hipError_t launch_fp4_pack(const uint8_t* q, const uint8_t* scale, void* packed, int V, int D,
                           hipStream_t stream) {
  const size_t pieces = fp4_packed_scale_off(V, D) / 16;
  const size_t words = (fp4_packed_bytes(V, D) - pieces * 16) / 4;
  const size_t blocks = (pieces + words + 255) / 256;
  fp4_pack_kernel<<<dim3((unsigned)blocks), dim3(256), 0, stream>>>(
      q, scale, static_cast<uint8_t*>(packed), V, D, pieces, words);
  return hipGetLastError();
}

// -------------------------------------------------------------- product

// How the hidden states are held, and what their product with the weights
// takes.  kExact: 8-bit states whose logits leave as float32 take the bfloat16
// product on operands that hold the same values exactly, as the mixed one
// drops, of each 8 products that it adds at once, what lies below 2^-13 of the
// largest.  Of 4-bit operands, whose blocks have one scale, it drops nothing:
// their products lie between 2^-2 and 36.
template <bool H8, typename O>
constexpr bool kFp4Exact = H8 && sizeof(O) == 4;

__device__ __forceinline__ uint4 load16(const uint8_t* p) {
  return *reinterpret_cast<const uint4*>(p);
}

// A lane's part of a step of its hidden row: h is l / 32.
template <bool H8, bool EXACT>
struct Fp4Hidden {
  uint4 lo, hi;                                    // 4 bits: lo alone
  __device__ __forceinline__ void load(const uint8_t* row, int step, int h) {
    if constexpr (!H8) {
      lo = load16(row + step * (kF4Step / 2) + 16 * h);
      hi = make_uint4(0u, 0u, 0u, 0u);
    } else if constexpr (EXACT) {                  // the weights' own order
      lo = load16(row + step * kF4Step + 32 * h);
      hi = load16(row + step * kF4Step + 32 * h + 16);
    } else {
      lo = load16(row + step * kF4Step + 16 * h);
      hi = load16(row + step * kF4Step + 32 + 16 * h);
    }
  }
};

// c += w h over one step: byte IA of sa and byte IB of sb are the scales.
template <bool H8, bool EXACT, int IA, int IB>
__device__ __forceinline__ fp4_f32x16 fp4_step(const uint4& a, const uint4& lo, const uint4& hi,
                                               fp4_f32x16 c, uint32_t sa, uint32_t sb) {
  if constexpr (!EXACT) {
    const fp4_i32x8 av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    const fp4_i32x8 bv = {(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w,
                          (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, H8 ? 0 : 4, IA, (int)sa, IB,
                                                           (int)sb);
  } else {
    const uint32_t aw[4] = {a.x, a.y, a.z, a.w};
    const uint32_t bw[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    const float fa = __uint_as_float(((sa >> (8 * IA)) & 255u) << 23);
    const float fb = __uint_as_float(((sb >> (8 * IB)) & 255u) << 23);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const fp4_bf16x2 x0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(aw[s], fa, 0);
      const fp4_bf16x2 x1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(aw[s], fa, 1);
      const fp4_bf16x2 x2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(aw[s], fa, 2);
      const fp4_bf16x2 x3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(aw[s], fa, 3);
      const fp4_bf16x2 y0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(bw[2 * s], fb, false);
      const fp4_bf16x2 y1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(bw[2 * s], fb, true);
      const fp4_bf16x2 y2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(bw[2 * s + 1], fb, false);
      const fp4_bf16x2 y3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(bw[2 * s + 1], fb, true);
      const fp4_bf16x8 x = {x0[0], x0[1], x1[0], x1[1], x2[0], x2[1], x3[0], x3[1]};
      const fp4_bf16x8 y = {y0[0], y0[1], y1[0], y1[1], y2[0], y2[1], y3[0], y3[1]};
      c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, y, c, 0, 0, 0);
    }
    return c;
  }
}

__device__ __forceinline__ void f4_put(float* p, float v) { *p = v; }
__device__ __forceinline__ void f4_put(bf16_t* p, float v) { *p = bf16_bits(v); }

// A workgroup owns 32 vocabulary rows and up to 32 hidden rows; its four waves
// split the runs of 128 columns (every fourth one each) and add their sums
// through LDS in a fixed order.
template <bool H8, typename O>
__global__ __launch_bounds__(kF4Threads) void fp4_skinny_kernel(
    const uint8_t* __restrict__ H, const uint8_t* __restrict__ hs, const uint8_t* __restrict__ P,
    const uint8_t* __restrict__ ws, int M, int D, int V, int ngroup, O* __restrict__ out) {
  constexpr bool EXACT = kFp4Exact<H8, O>;
  __shared__ float red[kF4Waves][32][33];
  const int group = blockIdx.x % ngroup;
  const int m0 = (blockIdx.x / ngroup) * 32;
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int h = lane / 32, l32 = lane % 32;
  const int runs = D / kFp8Block, steps = 2 * runs, nj = (steps + 3) / 4;
  const uint8_t* wrow = P + (size_t)group * steps * kF4StepBytes + lane * 16;
  const uint8_t* wsc = ws + ((size_t)group * nj * kWave + lane) * 4;
  const size_t hm = (size_t)min(m0 + l32, M - 1);            // rows past M repeat the last
  const uint8_t* hrow = H + hm * (H8 ? D : D / 2);
  const uint8_t* hsc = hs + hm * (H8 ? D / kFp8Block : D / kFp4Block);
  fp4_f32x16 acc;
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[r] = 0.f;

  for (int r = wave; r < runs; r += kF4Waves) {
    const int s = 2 * r;
    const uint4 a0 = load16(wrow + (size_t)s * kF4StepBytes);
    const uint4 a1 = load16(wrow + (size_t)(s + 1) * kF4StepBytes);
    const uint32_t sa = *reinterpret_cast<const uint16_t*>(wsc + (s / 4) * (kWave * 4) + s % 4);
    Fp4Hidden<H8, EXACT> b0, b1;
    b0.load(hrow, s, h);
    b1.load(hrow, s + 1, h);
    const uint32_t sb0 = H8 ? hsc[r] : hsc[2 * s + h], sb1 = H8 ? sb0 : hsc[2 * s + 2 + h];
    acc = fp4_step<H8, EXACT, 0, 0>(a0, b0.lo, b0.hi, acc, sa, sb0);
    acc = fp4_step<H8, EXACT, 1, 0>(a1, b1.lo, b1.hi, acc, sa, sb1);
  }
#pragma unroll
  for (int r = 0; r < 16; ++r) red[wave][l32][8 * (r / 4) + r % 4 + 4 * h] = acc[r];
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * 32; i += kF4Threads) {
    const int m = i / 32, v = i % 32;
    if (m0 + m >= M) break;                                  // m only grows
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kF4Waves; ++w) s += red[w][m][v];
    if (group * kF4Group + v < V) f4_put(out + (size_t)(m0 + m) * V + group * kF4Group + v, s);
  }
}

struct Fp4Args {
  const uint8_t *H, *hs, *P, *ws;
  int M, D, V;
  hipStream_t stream;
};

template <bool H8, typename O>
hipError_t fp4_head(const Fp4Args& a, O* out) {
  const int ng = fp4_groups(a.V);
  const size_t blocks = (size_t)ng * ((a.M + 31) / 32);
  fp4_skinny_kernel<H8, O><<<dim3((unsigned)blocks), dim3(kF4Threads), 0, a.stream>>>(
      a.H, a.hs, a.P, a.ws, a.M, a.D, a.V, ng, out);
  return hipGetLastError();
}

hipError_t launch_fp4_head(const uint8_t* hidden, bool h8, const uint8_t* hscale, const void* packed,
                           int M, int D, int V, void* logits, bool bf16, hipStream_t stream) {
  const uint8_t* P = static_cast<const uint8_t*>(packed);
  const Fp4Args a = {hidden, hscale, P, P + fp4_packed_scale_off(V, D), M, D, V, stream};
  if (bf16)
    return h8 ? fp4_head<true>(a, static_cast<bf16_t*>(logits))
              : fp4_head<false>(a, static_cast<bf16_t*>(logits));
  return h8 ? fp4_head<true>(a, static_cast<float*>(logits))
            : fp4_head<false>(a, static_cast<float*>(logits));
}

// Whether a product's grid fits, by the one with the most workgroups.
bool fp4_head_fits(int M, int V) {
  return grid_fits((size_t)fp4_groups(V) * ((M + 31) / 32), kF4Threads);
}

}  // namespace specv
