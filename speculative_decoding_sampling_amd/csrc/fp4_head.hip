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
#include "head_tile.h"
#include "specverify_draft.h"

namespace specv {

typedef int fp4_i32x8 __attribute__((ext_vector_type(8)));
using fp4_f32x16 = HeadF32x16;
typedef __bf16 fp4_bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 fp4_bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t fp4_word __attribute__((aligned(1), may_alias));   // scale bytes start anywhere

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
// is one sequence of blocks.  Memory: 128256 x 4096 of bfloat16 take 236 us, 5.6
// TB/s read and written; 320 x 4096 5 us, one load's and a launch's latency.
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

// A workgroup owns 32 vocabulary rows and up to 32 hidden rows; its four waves
// split the runs of 128 columns (every fourth one each) and add their sums
// through LDS in a fixed order.  Bound by reading the weights: 6 x 32000 x 4096
// takes 12.6 us, 5.5 TB/s (70 MB, partly from the memory-side cache).  The loads of
// two, four or eight runs issued together change nothing (17.0, 16.7 and 16.5 us
// against 17.7 where no weights are cached): other workgroups cover a wait.
template <bool ONCE, bool H8, typename O>
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
    const uint4 a0 = load16_weight<ONCE>(wrow + (size_t)s * kF4StepBytes);
    const uint4 a1 = load16_weight<ONCE>(wrow + (size_t)(s + 1) * kF4StepBytes);
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
    if (group * kF4Group + v < V) head_put(out + (size_t)(m0 + m) * V + group * kF4Group + v, s);
  }
}

// Many hidden rows.  A workgroup of four waves owns 256 vocabulary rows (64 a
// wave) and 32 MT hidden rows; two workgroups share a CU.  Each wave reads its
// weights straight into registers, runs ahead; the hidden rows of a run, 128
// bytes of each, are staged in LDS a run ahead, and every wave reads all of
// them, each fragment feeding two products.  A run is two steps of 8-bit or
// four of 4-bit states.
//
// Bound by operands on their way to the products and by the stores.  1152 x 152064 x
// 4096 takes 590 us with 8-bit states, 2.4 PFLOP/s, the matrix cores busy 65 % of
// the cycles at 1.8 GHz: without its weight loads 505, without those of the hidden
// rows 527, without either 455, without the stores of the logits 543.  With 4-bit
// states 451 us, 3.2 PFLOP/s, busy 39 % at 2.0 GHz, and 352, 409, 317 and 388; at 320
// x 128256 132 us, and 90, 121, 81 and 115.  (A loop of nothing but such products does
// 4.0 and 7.3 PFLOP/s, on zeros and ones.)  Float32 logits: of 8-bit states 1130 us,
// and 305 at 320 x 128256, a large library product's rate in bfloat16, the type that
// they take; of 4-bit states 522 and 150.
//
// Weights three runs ahead instead of one (96 rows, which have the registers) took 536
// us against 517; a wave's priority raised over its products changed nothing, steps
// kept apart cost 3 %.
//
// Rows of a staged run have their eight 16-byte pieces swapped by row pair (row
// r's piece p at slot p ^ ((r >> 1) & 7)), so that 16 consecutive rows cover
// every bank once.
//
// Workgroups are numbered so that one XCD (every eighth block) takes
// consecutive (vocabulary tile, row block) pairs, row blocks first: the
// blocks that share weights run side by side under one L2.
constexpr int kF4RowBytes = 128;                   // staged bytes of a hidden row
constexpr int kF4TileGroups = kTileVocab / kF4Group;
static_assert(kF4TileGroups == 2 * kF4Waves && kF4Threads == kHeadThreads, "two groups to a wave");

template <int MT, bool H8, typename O>
struct Fp4Tile {
  static constexpr int kRows = MT * 32;
  static constexpr int kBuf = kRows * kF4RowBytes;
  static constexpr int kTrBytes = HeadStore<MT, O>::kBytes;
  static constexpr int kBytes = 2 * kBuf > kTrBytes ? 2 * kBuf : kTrBytes;
  static constexpr int kSteps = H8 ? 2 : 4;        // of a run
  static constexpr int kRing = MT <= 1 || H8 ? 4 : 2;   // runs of weights in registers
};

// The tile of 256 vocabulary ids and hidden rows m0 .. m0 + 32 MT - 1.
template <int MT, bool ONCE, bool H8, typename O>
__device__ __forceinline__ void fp4_tile(uint8_t* lds, uint32_t (&lsc)[2][2 * kF4Threads],
                                         const uint8_t* __restrict__ H,
                                         const uint8_t* __restrict__ hs,
                                         const uint8_t* __restrict__ P,
                                         const uint32_t* __restrict__ ws, int M, int D, int V,
                                         int ngroup, int tile, int m0, O* __restrict__ out) {
  using T = Fp4Tile<MT, H8, O>;
  constexpr bool EXACT = kFp4Exact<H8, O>;
  constexpr int kBuf = T::kBuf, RING = T::kRing, STEPS = T::kSteps;
  static_assert(T::kRows <= kF4Threads, "one row's scales to a thread");
  const int tid = threadIdx.x, lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int h = lane / 32, l32 = lane % 32;
  const int steps = D / kF4Step, nj = (steps + 3) / 4;
  const int nrun = (steps + STEPS - 1) / STEPS;
  const int row_bytes = H8 ? D : D / 2;

  // this wave's two packed groups; groups past V repeat the last (dropped)
  const int g0 = min(tile * kF4TileGroups + wave * 2, ngroup - 1), g1 = min(g0 + 1, ngroup - 1);
  const uint8_t* w0 = P + (size_t)g0 * steps * kF4StepBytes;
  const uint8_t* w1 = P + (size_t)g1 * steps * kF4StepBytes;
  const uint32_t* s0 = ws + (size_t)g0 * nj * kWave + lane;
  const uint32_t* s1 = ws + (size_t)g1 * nj * kWave + lane;
  const uint32_t lane16 = lane * 16;

  // staging: this thread's pieces are tid + 256 j, eight to a row; rows past
  // M repeat the last (dropped).  The last run of 4-bit states may be half one:
  // their pieces past the row's end are zeros, whatever weights they meet.
  const uint8_t* hb = H + (size_t)m0 * row_bytes;
  const int left = M - 1 - m0;
  uint32_t hoff[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) hoff[j] = (uint32_t)min(tid / 8 + 32 * j, left) * row_bytes;
  const uint32_t piece = (tid % 8) * 16;
  const int slot = (tid / 8) * kF4RowBytes + (((tid % 8) ^ ((tid / 16) & 7)) * 16);
  const int nblock = H8 ? D / kFp8Block : D / kFp4Block;
  const uint8_t* hsrow = hs + (size_t)(m0 + min(tid, left)) * nblock;

  fp4_f32x16 acc[2][MT];
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[a][t][r] = 0.f;

  constexpr int kW = 2 * STEPS;                    // weight loads of a run
  uint4 wr[RING][2][STEPS], st[MT];
  // load i of the MT + kW of a run: staged hidden rows of run kb, then weights
  // of run kbw (past the end: the last step again)
  auto load = [&](int i, int kb, int kbw, uint4 (&d)[2][STEPS]) {
    if (i < MT) {
      const uint32_t at = (uint32_t)kb * kF4RowBytes + piece;
      st[i] = load16(hb + hoff[i] + min(at, (uint32_t)row_bytes - 16));
    } else {
      const int a = (i - MT) / STEPS, s = (i - MT) % STEPS;
      d[a][s] = load16_weight<ONCE>((a ? w1 : w0) + (size_t)min(kbw * STEPS + s, steps - 1) * kF4StepBytes +
                                    lane16);
    }
  };
  auto store_h = [&](int b, int kb) {
    // (a mask: a branch would cut the product loop into blocks)
    const uint32_t in = (uint32_t)kb * kF4RowBytes + piece < (uint32_t)row_bytes ? ~0u : 0u;
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      uint4 v = st[j];
      if constexpr (!H8) v = make_uint4(v.x & in, v.y & in, v.z & in, v.w & in);
      *reinterpret_cast<uint4*>(lds + b * kBuf + slot + j * 32 * kF4RowBytes) = v;
    }
  };
  // The rows' scales: 8 bits, bytes 4 g .. 4 g + 3 of a row as a word, one a
  // run; 4 bits, the bytes of run g, those of each half of a wave as a word.
  struct Scales {
    uint32_t b[H8 ? 4 : 2];
  };
  auto scale_load = [&](int g) {
    Scales x;
    if constexpr (H8) {
#pragma unroll
      for (int e = 0; e < 4; ++e) x.b[e] = hsrow[min(4 * g + e, nblock - 1)];
    } else {
      const fp4_word* p = reinterpret_cast<const fp4_word*>(hsrow);
#pragma unroll
      for (int e = 0; e < 2; ++e) x.b[e] = p[min(2 * g + e, nblock / 4 - 1)];
    }
    return x;
  };
  auto scale_store = [&](int buf, const Scales& x) {
    if constexpr (H8) {
      lsc[buf][tid] = x.b[0] | x.b[1] << 8 | x.b[2] << 16 | x.b[3] << 24;
    } else {
      lsc[buf][tid] = __builtin_amdgcn_perm(x.b[1], x.b[0], 0x06040200u);
      lsc[buf][tid + kF4Threads] = __builtin_amdgcn_perm(x.b[1], x.b[0], 0x07050301u);
    }
  };

#pragma unroll
  for (int i = 0; i < MT; ++i) load(i, 0, 0, wr[0]);
  scale_store(0, scale_load(0));
#pragma unroll
  for (int r = 0; r < RING - 1; ++r)
#pragma unroll
    for (int i = MT; i < MT + kW; ++i) load(i, 0, r, wr[r]);
  store_h(0, 0);
  lds_barrier();

  uint32_t sa0 = 0, sa1 = 0, sb[MT];
  // run kb, the I-th of its group
  auto run = [&](auto idx, int kb) {
    constexpr int I = decltype(idx)::value;
    const uint8_t* buf = lds + (I % 2) * kBuf + l32 * kF4RowBytes;
    const uint4(&w)[2][STEPS] = wr[I % RING];
    const int sw = (l32 >> 1) & 7;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {              // a step's products are kept together
#pragma unroll
      for (int l = s * (MT + kW) / STEPS; l < (s + 1) * (MT + kW) / STEPS; ++l)
        load(l, kb + 1, kb + RING - 1, wr[(I + RING - 1) % RING]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const uint8_t* row = buf + t * 32 * kF4RowBytes;
        uint4 lo, hi = make_uint4(0u, 0u, 0u, 0u);
        if constexpr (!H8) {
          lo = load16(row + (((2 * s + h) ^ sw) * 16));
        } else {
          lo = load16(row + (((4 * s + (EXACT ? 2 : 1) * h) ^ sw) * 16));
          hi = load16(row + (((4 * s + (EXACT ? 2 * h + 1 : 2 + h)) ^ sw) * 16));
        }
        constexpr int IA = H8 ? 2 * (I % 2) : 0, IB = H8 ? I : 0;
        if constexpr (H8) {
          if (s == 0) {
            acc[0][t] = fp4_step<H8, EXACT, IA, IB>(w[0][s], lo, hi, acc[0][t], sa0, sb[t]);
            acc[1][t] = fp4_step<H8, EXACT, IA, IB>(w[1][s], lo, hi, acc[1][t], sa1, sb[t]);
          } else {
            acc[0][t] = fp4_step<H8, EXACT, IA + 1, IB>(w[0][s], lo, hi, acc[0][t], sa0, sb[t]);
            acc[1][t] = fp4_step<H8, EXACT, IA + 1, IB>(w[1][s], lo, hi, acc[1][t], sa1, sb[t]);
          }
        } else {
          auto both = [&](auto S) {
            constexpr int B = decltype(S)::value;
            acc[0][t] = fp4_step<H8, EXACT, B, B>(w[0][s], lo, hi, acc[0][t], sa0, sb[t]);
            acc[1][t] = fp4_step<H8, EXACT, B, B>(w[1][s], lo, hi, acc[1][t], sa1, sb[t]);
          };
          if (s == 0) both(std::integral_constant<int, 0>{});
          else if (s == 1) both(std::integral_constant<int, 1>{});
          else if (s == 2) both(std::integral_constant<int, 2>{});
          else both(std::integral_constant<int, 3>{});
        }
      }
    }
    store_h((I + 1) % 2, kb + 1);
  };
  using std::integral_constant;
  if constexpr (H8) {
    // groups of four runs: one word of the hidden rows' scales, two of the weights'
    uint32_t n0[2] = {s0[0], s0[min(1, nj - 1) * kWave]}, n1[2] = {s1[0], s1[min(1, nj - 1) * kWave]};
    for (int g = 0;; ++g) {
      const Scales next = scale_load(g + 1);       // past the end: the last bytes (not used)
#pragma unroll
      for (int t = 0; t < MT; ++t) sb[t] = lsc[g & 1][t * 32 + l32];
      sa0 = n0[0];
      sa1 = n1[0];
      run(integral_constant<int, 0>{}, 4 * g);
      lds_barrier();
      if (4 * g + 1 == nrun) break;
      run(integral_constant<int, 1>{}, 4 * g + 1);
      lds_barrier();
      if (4 * g + 2 == nrun) break;
      sa0 = n0[1];
      sa1 = n1[1];
      n0[0] = s0[min(2 * g + 2, nj - 1) * kWave];
      n1[0] = s1[min(2 * g + 2, nj - 1) * kWave];
      run(integral_constant<int, 2>{}, 4 * g + 2);
      lds_barrier();
      if (4 * g + 3 == nrun) break;
      n0[1] = s0[min(2 * g + 3, nj - 1) * kWave];
      n1[1] = s1[min(2 * g + 3, nj - 1) * kWave];
      run(integral_constant<int, 3>{}, 4 * g + 3);
      scale_store((g + 1) & 1, next);
      lds_barrier();
      if (4 * g + 4 == nrun) break;
    }
  } else {
    // every run has its own words
    uint32_t n0 = s0[0], n1 = s1[0];
    auto turn = [&](auto idx, int kb) {
      constexpr int I = decltype(idx)::value;
      const int next = min(kb + 1, nrun - 1);
      const Scales nh = scale_load(next);
#pragma unroll
      for (int t = 0; t < MT; ++t) sb[t] = lsc[I % 2][h * kF4Threads + t * 32 + l32];
      sa0 = n0;
      sa1 = n1;
      n0 = s0[next * kWave];
      n1 = s1[next * kWave];
      run(idx, kb);
      scale_store((I + 1) % 2, nh);
      lds_barrier();
    };
    for (int kb = 0;; kb += RING) {
      turn(integral_constant<int, 0>{}, kb);
      if (kb + 1 == nrun) break;
      turn(integral_constant<int, 1>{}, kb + 1);
      if (kb + 2 == nrun) break;
      if constexpr (RING == 4) {
        turn(integral_constant<int, 2>{}, kb + 2);
        if (kb + 3 == nrun) break;
        turn(integral_constant<int, 3>{}, kb + 3);
        if (kb + 4 == nrun) break;
      }
    }
  }
  head_store<MT>(lds, acc, tile, m0, M, V, out);
}

// The row blocks share the 32-row steps evenly, at most MT each.
template <int MT, bool ONCE, bool H8, typename O>
__global__ __launch_bounds__(kF4Threads, 2) void fp4_tile_kernel(
    const uint8_t* __restrict__ H, const uint8_t* __restrict__ hs, const uint8_t* __restrict__ P,
    const uint32_t* __restrict__ ws, int M, int D, int V, int ngroup, int nrb, int nwork,
    O* __restrict__ out) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[Fp4Tile<MT, H8, O>::kBytes];
  __shared__ uint32_t lsc[2][2 * kF4Threads];                // words past the rows are not read
  const int per = (nwork + kXcds - 1) / kXcds;
  const int work = (int)(blockIdx.x % kXcds) * per + (int)(blockIdx.x / kXcds);
  if (work >= nwork) return;                                 // blockIdx.x / kXcds < per
  const int tile = work / nrb, rb = work % nrb, all = (M + 31) / 32;
  const int m0 = 32 * (rb * (all / nrb) + min(rb, all % nrb));
  const int steps = all / nrb + (rb < all % nrb ? 1 : 0);
  if (MT > 3 && steps == 3)
    fp4_tile<MT < 3 ? MT : 3, ONCE, H8>(lds, lsc, H, hs, P, ws, M, D, V, ngroup, tile, m0, out);
  else if (MT > 2 && steps == 2)
    fp4_tile<MT < 2 ? MT : 2, ONCE, H8>(lds, lsc, H, hs, P, ws, M, D, V, ngroup, tile, m0, out);
  else if (MT > 1 && steps == 1)
    fp4_tile<1, ONCE, H8>(lds, lsc, H, hs, P, ws, M, D, V, ngroup, tile, m0, out);
  else
    fp4_tile<MT, ONCE, H8>(lds, lsc, H, hs, P, ws, M, D, V, ngroup, tile, m0, out);
}

struct Fp4Args {
  const uint8_t *H, *hs, *P, *ws;
  int M, D, V;
  hipStream_t stream;
};

template <int MT, bool ONCE, bool H8, typename O>
hipError_t fp4_tiles(const Fp4Args& a, O* out) {
  const int nrb = (a.M + 32 * MT - 1) / (32 * MT);
  const size_t nwork = (size_t)((a.V + kTileVocab - 1) / kTileVocab) * nrb;
  const size_t blocks = (nwork + kXcds - 1) / kXcds * kXcds;
  fp4_tile_kernel<MT, ONCE, H8, O><<<dim3((unsigned)blocks), dim3(kF4Threads), 0, a.stream>>>(
      a.H, a.hs, a.P, reinterpret_cast<const uint32_t*>(a.ws), a.M, a.D, a.V, fp4_groups(a.V), nrb,
      (int)nwork, out);
  return hipGetLastError();
}

template <bool ONCE, bool H8, typename O>
hipError_t fp4_skinny(const Fp4Args& a, O* out) {
  const int ng = fp4_groups(a.V);
  const size_t blocks = (size_t)ng * ((a.M + 31) / 32);
  fp4_skinny_kernel<ONCE, H8, O><<<dim3((unsigned)blocks), dim3(kF4Threads), 0, a.stream>>>(
      a.H, a.hs, a.P, a.ws, a.M, a.D, a.V, ng, out);
  return hipGetLastError();
}

constexpr double kFp4CacheBytes = 256.0 * (1 << 20);

// Which product: 0 the skinny one, 1 .. 4 tiles of at most 32 times as many
// hidden rows.
//
// The skinny one has eight times the workgroups, each a chain an eighth as long,
// but reads the weights once for every 32 rows.  It is taken where its
// workgroups (an empty row block counts half) are at most four a CU for 64 rows,
// two for more: at D = 4096 and 8-bit states 8000 x 64 takes 14.6 us and by tiles
// 20.2, 20001 x 17 14.8 and 22.8; beyond, 20001 x 64 31.0 and 24.2, 8000 x 100
// 22.4 and 20.3, 128256 x 1 52.3 and 49.2, 128256 x 32 98 and 52.
//
// Among tiles: a CU does its share of them at the pace of one, whose time grows
// as 2 D for the weights and D + 640 for each 32 rows and their logits.  At
// 32000 x 4096 and 160 rows 32, 64, 96 and 128 rows take 39, 34, 30 and 30 us, at
// 128256 and 100 rows 100, 83, 85 and 70, at 20001 and 64 rows 24, 30, 30 and 30;
// over 250 sizes, M from 1 to 1152, the rule's choice takes 1.4 % more than the
// best one (geometric mean; 30 % at most, 20001 x 1024 with 200 rows).
int fp4_choice(int M, int D, int V, bool exact) {
  constexpr long long kCus = 256;
  const long long groups = fp4_groups(V), blocks = (M + 31) / 32;
  if (groups * blocks <= 2 * kCus || (M <= 64 && groups * (32 * blocks + M) <= 64 * 4 * kCus))
    return 0;
  const long long tiles = ((long long)V + kTileVocab - 1) / kTileVocab;
  int best = 1;
  long long least = 0;
  for (int mt = 1; mt <= (exact ? 3 : 4); ++mt) {
    const long long work = tiles * ((M + 32 * mt - 1) / (32 * mt));
    const long long cost = (work + kCus - 1) / kCus * (2 * D + mt * (D + 640));
    if (mt == 1 || cost < least) best = mt, least = cost;
  }
  return best;
}

template <bool ONCE, bool H8, typename O>
hipError_t fp4_run(const Fp4Args& a, int choice, O* out) {
  if (choice == 0) return fp4_skinny<ONCE, H8>(a, out);
  if (choice == 1) return fp4_tiles<1, ONCE, H8>(a, out);
  if (choice == 2) return fp4_tiles<2, ONCE, H8>(a, out);
  if constexpr (!kFp4Exact<H8, O>)                           // bfloat16 operands: 4 would spill
    if (choice == 4) return fp4_tiles<4, ONCE, H8>(a, out);
  return fp4_tiles<3, ONCE, H8>(a, out);
}
template <bool H8, typename O>
hipError_t fp4_head(const Fp4Args& a, O* out) {
  const int choice = fp4_choice(a.M, a.D, a.V, kFp4Exact<H8, O>);
  const int rows = choice == 0 ? 32 : 32 * choice;
  return a.M <= rows && (double)a.V * a.D / 2 > kFp4CacheBytes ? fp4_run<true, H8>(a, choice, out)
                                                                  : fp4_run<false, H8>(a, choice, out);
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
