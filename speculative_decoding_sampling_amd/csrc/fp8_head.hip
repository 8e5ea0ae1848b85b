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
// k order.  A run of 128 is two products of 64; in product j lane l supplies
// bytes 64 j + 32 (l / 32) .. + 31 of its row.  Both operands share that order,
// and any order of k shared by both gives the same sum.  Both products lie in
// one run, so a lane's scale byte is that of its row and run whatever the
// matrix core's own 32-wide blocks are.
#include "fp8.h"
#include "grid.h"
#include "specverify_ops.h"

namespace specv {

typedef int fp8_i32x8 __attribute__((ext_vector_type(8)));
typedef float fp8_f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 fp8_bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 fp8_bf16x8 __attribute__((ext_vector_type(8)));

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
// one sequence of runs.  Memory-bound where there is enough of it: 2304 x 8192
// bfloat16 10.9 us (5.2 TB/s); 320 x 4096 is one wait of its loads, 3.6 to 5.3 us.
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

bool fp8_quantize_fits(int rows, int D) { return grid_fits(((size_t)rows * D / 8 + 255) / 256, 256); }

hipError_t launch_fp8_quantize(const void* x, bool bf16, int rows, int D, uint8_t* q,
                               uint8_t* scale, hipStream_t stream) {
  const size_t n8 = (size_t)rows * D / 8;
  const dim3 grid((unsigned)((n8 + 255) / 256));
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
    const int k = kb * kFp8Block + 64 * (s / 2) + 32 * (lane / 32) + 16 * (s % 2);
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

bool fp8_pack_fits(int V, int D) {
  const size_t pieces = fp8_packed_scale_off(V, D) / 16;
  return grid_fits((pieces + (fp8_packed_bytes(V, D) - pieces * 16) / 4 + 255) / 256, 256);
}

hipError_t launch_fp8_pack(const uint8_t* q, const uint8_t* scale, void* packed, int V, int D,
                           hipStream_t stream) {
  const size_t pieces = fp8_packed_scale_off(V, D) / 16;
  const size_t words = (fp8_packed_bytes(V, D) - pieces * 16) / 4;
  const size_t blocks = (pieces + words + 255) / 256;
  fp8_pack_kernel<<<dim3((unsigned)blocks), dim3(256), 0, stream>>>(
      q, scale, static_cast<uint8_t*>(packed), V, D, pieces, words);
  return hipGetLastError();
}

// -------------------------------------------------------------- product

// 32 bytes of a lane's row, one operand of a 64-wide product step.
struct Fp8Bytes {
  uint4 lo, hi;
};

// c += a b over one 64-wide step of run I of its group (byte I of the scale
// words).
//
// The 8-bit matrix product keeps, of each 8 products it adds at once, what
// lies within 2^-13 of the largest (measured on single products): before their
// rounding the logits come out 1e-5 to 6e-5 of their rms off, 0.3 to 1.5 % of
// 2^-8.  That is enough where they are rounded to bfloat16: their error against
// 64 bits stays 1.66e-3 of the rms, 1.1 to 1.7 % of them round the other way.
// Where large products cancel it is up to 2^-10 of the sum of magnitudes, as
// the header says.  Float32 logits (EXACT) take the bfloat16 product instead,
// on operands that hold the same values exactly with their scales applied: 1e-8
// to 1e-7 of the rms off (D from 128 to 16384), at half the rate.
template <bool EXACT, int I>
__device__ __forceinline__ fp8_f32x16 fp8_step(const Fp8Bytes& a, const Fp8Bytes& b, fp8_f32x16 c,
                                               uint32_t sa, uint32_t sb) {
  const uint32_t aw[8] = {a.lo.x, a.lo.y, a.lo.z, a.lo.w, a.hi.x, a.hi.y, a.hi.z, a.hi.w};
  const uint32_t bw[8] = {b.lo.x, b.lo.y, b.lo.z, b.lo.w, b.hi.x, b.hi.y, b.hi.z, b.hi.w};
  if constexpr (!EXACT) {
    fp8_i32x8 av, bv;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      av[i] = (int)aw[i];
      bv[i] = (int)bw[i];
    }
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 0, 0, I, (int)sa, I, (int)sb);
  } else {
    const float fa = __uint_as_float(((sa >> (8 * I)) & 255u) << 23);
    const float fb = __uint_as_float(((sb >> (8 * I)) & 255u) << 23);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      fp8_bf16x8 x, y;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const fp8_bf16x2 x0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(aw[2 * s + w], fa, false);
        const fp8_bf16x2 x1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(aw[2 * s + w], fa, true);
        const fp8_bf16x2 y0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(bw[2 * s + w], fb, false);
        const fp8_bf16x2 y1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(bw[2 * s + w], fb, true);
        x[4 * w] = x0[0];
        x[4 * w + 1] = x0[1];
        x[4 * w + 2] = x1[0];
        x[4 * w + 3] = x1[1];
        y[4 * w] = y0[0];
        y[4 * w + 1] = y0[1];
        y[4 * w + 2] = y1[0];
        y[4 * w + 3] = y1[1];
      }
      c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, y, c, 0, 0, 0);
    }
    return c;
  }
}

template <typename O>
constexpr bool kFp8Exact = sizeof(O) == 4;

__device__ __forceinline__ void f8_put(float* p, float v) { *p = v; }
__device__ __forceinline__ void f8_put(bf16_t* p, float v) { *p = bf16_bits(v); }
// Four consecutive logits, registers r .. r + 3 of an accumulator.
__device__ __forceinline__ void f8_put4(float* p, const fp8_f32x16& c, int r) {
  *reinterpret_cast<float4*>(p) = make_float4(c[r], c[r + 1], c[r + 2], c[r + 3]);
}
__device__ __forceinline__ void f8_put4(bf16_t* p, const fp8_f32x16& c, int r) {
  uint2 w;
  w.x = bf16_pair(c[r], c[r + 1]);
  w.y = bf16_pair(c[r + 2], c[r + 3]);
  *reinterpret_cast<uint2*>(p) = w;
}

__device__ __forceinline__ uint4 load16(const uint8_t* p) {
  return *reinterpret_cast<const uint4*>(p);
}

// 16 bytes of a weight, past the caches where the call reads it only once.
template <bool ONCE>
__device__ __forceinline__ uint4 load16_weight(const uint8_t* p) {
  if constexpr (!ONCE) {
    return load16(p);
  } else {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
    return make_uint4(v.x, v.y, v.z, v.w);
  }
}

// Bytes 4 g .. 4 g + 3 of a row of nkb scale bytes as a word, 127 past the
// end.  No branches: a product loop that holds one is cut into blocks, and the
// compiler then moves products across them and spills their accumulators.
// Load and use are apart, so that a loop can wait for the bytes where it needs
// them.
struct Fp8ScaleBytes {
  uint32_t b[4];
};
__device__ __forceinline__ Fp8ScaleBytes fp8_scale_load(const uint8_t* row, int g, int nkb) {
  Fp8ScaleBytes s;
#pragma unroll
  for (int e = 0; e < 4; ++e) s.b[e] = row[min(4 * g + e, nkb - 1)];
  return s;
}
__device__ __forceinline__ uint32_t fp8_scale_word(const Fp8ScaleBytes& s, int g, int nkb) {
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) w |= (4 * g + e < nkb ? s.b[e] : 127u) << (8 * e);
  return w;
}

// Few hidden rows: the weights are read straight into registers, once, and
// the kernel is bound by them (76 us for the 529 MB of 1 x 128256 x 4096, 6.9
// TB/s).  A workgroup owns 32 vocabulary rows and up to 32 hidden rows; its
// four waves split the runs (every fourth one each, so that together they read
// 16 KB in a row) and add their sums through LDS in a fixed order.
template <bool ONCE, typename O>
__global__ __launch_bounds__(kF8Threads) void fp8_skinny_kernel(
    const uint8_t* __restrict__ H, const uint8_t* __restrict__ hs, const uint8_t* __restrict__ P,
    const uint8_t* __restrict__ ws, int M, int D, int V, int ngroup, O* __restrict__ out) {
  __shared__ float red[kF8Waves][32][33];
  const int group = blockIdx.x % ngroup;
  const int m0 = (blockIdx.x / ngroup) * 32;
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int h = lane / 32, l32 = lane % 32;
  const int nkb = D / kFp8Block, nk4 = (nkb + 3) / 4;
  const uint8_t* wrow = P + (size_t)group * nkb * kF8RunBytes + lane * 16;
  const uint8_t* wsc = ws + (size_t)group * nk4 * (kF8Group * 4) + l32 * 4;
  const size_t hm = (size_t)min(m0 + l32, M - 1);            // rows past M repeat the last
  const uint8_t* hrow = H + hm * D + 32 * h;
  const uint8_t* hsc = hs + hm * nkb;
  fp8_f32x16 acc;
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[r] = 0.f;

#pragma unroll 4
  for (int kb = wave; kb < nkb; kb += kF8Waves) {
    uint4 a[4];
#pragma unroll
    for (int s = 0; s < 4; ++s)
      a[s] = load16_weight<ONCE>(wrow + (size_t)kb * kF8RunBytes + s * 1024);
    const uint32_t sa = wsc[(kb / 4) * (kF8Group * 4) + kb % 4];
    uint4 b[4];
#pragma unroll
    for (int s = 0; s < 4; ++s)
      b[s] = load16(hrow + kb * kFp8Block + 64 * (s / 2) + 16 * (s % 2));
    const uint32_t sb = hsc[kb];
    acc = fp8_step<kFp8Exact<O>, 0>({a[0], a[1]}, {b[0], b[1]}, acc, sa, sb);
    acc = fp8_step<kFp8Exact<O>, 0>({a[2], a[3]}, {b[2], b[3]}, acc, sa, sb);
  }
#pragma unroll
  for (int r = 0; r < 16; ++r) red[wave][l32][8 * (r / 4) + r % 4 + 4 * h] = acc[r];
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * 32; i += kF8Threads) {
    const int m = i / 32, v = i % 32;
    if (m0 + m >= M) break;                                  // m only grows
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kF8Waves; ++w) s += red[w][m][v];
    if (group * kF8Group + v < V) f8_put(out + (size_t)(m0 + m) * V + group * kF8Group + v, s);
  }
}

// LDS writes of this workgroup made visible at a barrier, global loads left
// in flight.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Many hidden rows.  A workgroup of four waves owns 256 vocabulary rows (64 a
// wave) and 32 MT hidden rows; two workgroups share a CU and cover each
// other's waits.  Each wave reads its weights straight into registers, a run
// ahead; the hidden rows of a run are staged in LDS, a run ahead, and every
// wave reads all of them, each fragment feeding two products (64 vocabulary
// rows a wave halve the LDS reads of 32).  The products of kPin fragments are
// kept together (sched_barrier), the compiler orders them.
//
// Rows of a staged run are 128 bytes, their eight 16-byte pieces swapped by
// row pair (row r's piece p at slot p ^ ((r >> 1) & 7)), so that 16
// consecutive rows cover every bank once.
//
// At 1152 x 152064 x 4096 it takes 685 us, 2.09 PFLOP/s: the matrix cores are busy
// 55 % of the cycles at a clock that power holds near 1.8 GHz; without the weights'
// loads it would take 525 us.
//
// Workgroups are numbered so that one XCD (every eighth block) takes
// consecutive (vocabulary tile, row block) pairs, row blocks first: the
// blocks that share weights run side by side under one L2.
constexpr int kTileVocab = 256;
constexpr int kTileGroups = kTileVocab / kF8Group;
constexpr int kXcds = 8;
static_assert(kTileGroups == 2 * kF8Waves, "two packed groups to a wave");

// A tile's LDS: two runs of staged hidden rows, in whose place the epilogue
// moves 32 rows of bfloat16 logits or 16 of float32 at a time; two words of the
// rows' scales.
template <int MT, typename O>
struct Fp8Tile {
  static constexpr int kRows = MT * 32;
  static constexpr int kBuf = kRows * kFp8Block;
  static constexpr int kTrStride = kTileVocab + 16 / (int)sizeof(O);
  static constexpr int kTrRows = 64 / (int)sizeof(O);
  static constexpr int kTrBytes = kTrRows * kTrStride * (int)sizeof(O);
  static constexpr int kBytes = 2 * kBuf > kTrBytes ? 2 * kBuf : kTrBytes;
  static constexpr int kRing = MT <= 2 ? 4 : 2;              // runs of weights in registers
};

// The tile of 256 vocabulary ids and hidden rows m0 .. m0 + 32 MT - 1.
template <int MT, bool ONCE, typename O>
__device__ __forceinline__ void fp8_tile(uint8_t* lds, uint32_t (&lsc)[2][kF8Threads],
                                         const uint8_t* __restrict__ H,
                                         const uint8_t* __restrict__ hs,
                                         const uint8_t* __restrict__ P,
                                         const uint32_t* __restrict__ ws, int M, int D, int V,
                                         int ngroup, int tile, int m0, O* __restrict__ out) {
  using T = Fp8Tile<MT, O>;
  constexpr int kBuf = T::kBuf, kTrStride = T::kTrStride, kTrRows = T::kTrRows, RING = T::kRing;
  static_assert(T::kRows <= kF8Threads, "one row's scales to a thread");
  static_assert(4 % RING == 0, "the weight ring indexes statically over a group of runs");
  const int tid = threadIdx.x, lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int h = lane / 32, l32 = lane % 32;
  const int nkb = D / kFp8Block, nk4 = (nkb + 3) / 4;

  // this wave's two packed groups; groups past V repeat the last (dropped)
  const int g0 = min(tile * kTileGroups + wave * 2, ngroup - 1), g1 = min(g0 + 1, ngroup - 1);
  const uint8_t* w0 = P + (size_t)g0 * nkb * kF8RunBytes;
  const uint8_t* w1 = P + (size_t)g1 * nkb * kF8RunBytes;
  const uint32_t* s0 = ws + (size_t)g0 * nk4 * kF8Group;
  const uint32_t* s1 = ws + (size_t)g1 * nk4 * kF8Group;
  const uint32_t lane16 = lane * 16;

  // staging: this thread's pieces are tid + 256 j, eight to a row; rows past
  // M repeat the last (dropped)
  const uint8_t* hb = H + (size_t)m0 * D;
  const int left = M - 1 - m0;
  uint32_t hoff[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j)
    hoff[j] = (uint32_t)min(tid / 8 + 32 * j, left) * D + (tid % 8) * 16;
  const int slot = (tid / 8) * kFp8Block + (((tid % 8) ^ ((tid / 16) & 7)) * 16);
  const uint8_t* hsrow = hs + (size_t)(m0 + min(tid, left)) * nkb;

  fp8_f32x16 acc[2][MT];
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[a][t][r] = 0.f;

  uint4 wr[RING][2][4], st[MT];
  // load i of the MT + 8 of a run: staged hidden rows of run kb, then weights of
  // run kbw (past the end: the last run again)
  auto load = [&](int i, int kb, int kbw, uint4 (&d)[2][4]) {
    if (i < MT) {
      st[i] = load16(hb + (size_t)min(kb, nkb - 1) * kFp8Block + hoff[i]);
    } else {
      const int a = (i - MT) / 4, s = (i - MT) % 4;
      d[a][s] = load16_weight<ONCE>((a ? w1 : w0) + (size_t)min(kbw, nkb - 1) * kF8RunBytes +
                                    s * 1024 + lane16);
    }
  };
  auto store_h = [&](int b) {
#pragma unroll
    for (int j = 0; j < MT; ++j)
      *reinterpret_cast<uint4*>(lds + b * kBuf + slot + j * 32 * kFp8Block) = st[j];
  };

  uint32_t sa0 = s0[l32], sa1 = s1[l32], sb[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) load(i, 0, 0, wr[0]);
  lsc[0][tid] = fp8_scale_word(fp8_scale_load(hsrow, 0, nkb), 0, nkb);
#pragma unroll
  for (int r = 0; r < RING - 1; ++r)
#pragma unroll
    for (int i = MT; i < MT + 8; ++i) load(i, 0, r, wr[r]);
  store_h(0);
  lds_barrier();

  auto run = [&](auto idx, int kb) {
    constexpr int I = decltype(idx)::value;
    const uint8_t* buf = lds + (I % 2) * kBuf + l32 * kFp8Block;
    const uint4(&w)[2][4] = wr[I % RING];
    const int sw = (l32 >> 1) & 7;
    constexpr int kPin = MT;                               // products kept together
    constexpr int kParts = 2 * MT / kPin;
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) {
      const int s = i / MT, t = i % MT;
      if (i % kPin == 0) {
#pragma unroll
        for (int l = (i / kPin) * (MT + 8) / kParts; l < (i / kPin + 1) * (MT + 8) / kParts; ++l)
          load(l, kb + 1, kb + RING - 1, wr[(I + RING - 1) % RING]);
        __builtin_amdgcn_sched_barrier(0);
      }
      const Fp8Bytes b = {load16(buf + t * 32 * kFp8Block + (((4 * s + 2 * h) ^ sw) * 16)),
                          load16(buf + t * 32 * kFp8Block + (((4 * s + 2 * h + 1) ^ sw) * 16))};
      acc[0][t] = fp8_step<kFp8Exact<O>, I>({w[0][2 * s], w[0][2 * s + 1]}, b, acc[0][t], sa0, sb[t]);
      acc[1][t] = fp8_step<kFp8Exact<O>, I>({w[1][2 * s], w[1][2 * s + 1]}, b, acc[1][t], sa1, sb[t]);
      if (i % kPin == kPin - 1) __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_sched_barrier(0);
    store_h((I + 1) % 2);
  };
  // groups of four runs, one scale word
  for (int g = 0;; ++g) {
    const int next = min(g + 1, nk4 - 1);
    const uint32_t n0 = s0[next * kF8Group + l32], n1 = s1[next * kF8Group + l32];
    const Fp8ScaleBytes nh = fp8_scale_load(hsrow, next, nkb);
#pragma unroll
    for (int t = 0; t < MT; ++t) sb[t] = lsc[g & 1][t * 32 + l32];
    run(std::integral_constant<int, 0>{}, 4 * g);
    lds_barrier();
    if (4 * g + 1 == nkb) break;
    run(std::integral_constant<int, 1>{}, 4 * g + 1);
    lds_barrier();
    if (4 * g + 2 == nkb) break;
    run(std::integral_constant<int, 2>{}, 4 * g + 2);
    lds_barrier();
    if (4 * g + 3 == nkb) break;
    run(std::integral_constant<int, 3>{}, 4 * g + 3);
    lsc[(g + 1) & 1][tid] = fp8_scale_word(nh, next, nkb);
    lds_barrier();
    if (4 * g + 4 == nkb) break;
    sa0 = n0;
    sa1 = n1;
  }

  // acc[a][t][r] is the logit of row 32 t + l32 of the block and vocabulary id
  // 64 wave + 32 a + 8 (r / 4) + r % 4 + 4 h of the tile.
  // They leave through LDS, so that a wave's stores cover consecutive ids: 16
  // bytes a lane where every row starts 16-byte aligned, else two bfloat16
  // logits that share an aligned word, or one float32 logit (stored straight
  // from the accumulators an odd V cost 31 instead of 17 us at 320 x 20001 x
  // 1152).
  const int vb = wave * 64 + 4 * h;
  const int v0 = tile * kTileVocab, nv = min(kTileVocab, V - v0);
  constexpr int kVec = 16 / sizeof(O);
  const bool whole = V % kVec == 0 && (reinterpret_cast<uintptr_t>(out) & 15) == 0;
  O* tr = reinterpret_cast<O*>(lds);
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int part = 0; part < 32 / kTrRows; ++part) {
      const int r0 = t * 32 + part * kTrRows;               // first row of the part in the block
      if (32 == kTrRows || l32 / kTrRows == part) {
        O* row = tr + (l32 % kTrRows) * kTrStride + vb;
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int q = 0; q < 4; ++q) f8_put4(row + 32 * a + 8 * q, acc[a][t], 4 * q);
      }
      lds_barrier();
      if (whole) {
#pragma unroll
        for (int i = 0; i < kTrRows * kTileVocab / kVec / kF8Threads; ++i) {
          const int p = tid + i * kF8Threads, row = p / (kTileVocab / kVec);
          const int c = p % (kTileVocab / kVec) * kVec;
          if (m0 + r0 + row < M && c < nv)
            *reinterpret_cast<uint4*>(out + (size_t)(m0 + r0 + row) * V + v0 + c) =
                *reinterpret_cast<const uint4*>(tr + row * kTrStride + c);
        }
      } else {
        constexpr int kLog = 4 / sizeof(O);                  // logits of a 4-byte store
#pragma unroll
        for (int i = 0; i < kTrRows * kTileVocab / kLog / kF8Threads; ++i) {
          const int p = tid + i * kF8Threads, row = p / (kTileVocab / kLog);
          if (m0 + r0 + row >= M) continue;
          O* dst = out + (size_t)(m0 + r0 + row) * V + v0;
          const O* src = tr + row * kTrStride;
          if constexpr (sizeof(O) == 4) {
            const int c = p % kTileVocab;
            if (c < nv) dst[c] = src[c];
          } else {
            // aligned words start at the row's first logit or its second; a
            // first or last logit without a partner is stored alone
            const int odd = (int)(reinterpret_cast<uintptr_t>(dst) >> 1) & 1;
            const int c = odd + 2 * (p % (kTileVocab / 2));
            if (odd && c == 1) dst[0] = src[0];
            if (c + 1 < nv)
              *reinterpret_cast<uint32_t*>(dst + c) = (uint32_t)src[c] | (uint32_t)src[c + 1] << 16;
            else if (c < nv)
              dst[c] = src[c];
          }
        }
      }
      lds_barrier();
    }
}

// The row blocks share the 32-row steps evenly, at most MT each: as many rows
// as there are, and blocks that share weights keep in step, so that more of them
// are found in L2.  bfloat16, us, against whole tiles / a short last block: 320 x
// 128256 x 4096 219 / 213 -> 206, 257 rows 203 / 204 -> 186, 200 rows 156 / 150 ->
// 149, 160 x 64000 x 4096 75 / 66 -> 65; float32 97 x 128256 x 4096 205 / 195 -> 176.
template <int MT, bool ONCE, typename O>
__global__ __launch_bounds__(kF8Threads, 2) void fp8_tile_kernel(
    const uint8_t* __restrict__ H, const uint8_t* __restrict__ hs, const uint8_t* __restrict__ P,
    const uint32_t* __restrict__ ws, int M, int D, int V, int ngroup, int nrb, int nwork,
    O* __restrict__ out) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[Fp8Tile<MT, O>::kBytes];
  __shared__ uint32_t lsc[2][kF8Threads];                    // words past the rows are not read
  const int per = (nwork + kXcds - 1) / kXcds;
  const int work = (int)(blockIdx.x % kXcds) * per + (int)(blockIdx.x / kXcds);
  if (work >= nwork) return;                                 // blockIdx.x / kXcds < per
  const int tile = work / nrb, rb = work % nrb, all = (M + 31) / 32;
  const int m0 = 32 * (rb * (all / nrb) + min(rb, all % nrb));
  const int steps = all / nrb + (rb < all % nrb ? 1 : 0);
  if (MT > 3 && steps == 3)
    fp8_tile<MT < 3 ? MT : 3, ONCE>(lds, lsc, H, hs, P, ws, M, D, V, ngroup, tile, m0, out);
  else if (MT > 2 && steps == 2)
    fp8_tile<MT < 2 ? MT : 2, ONCE>(lds, lsc, H, hs, P, ws, M, D, V, ngroup, tile, m0, out);
  else if (MT > 1 && steps == 1)
    fp8_tile<1, ONCE>(lds, lsc, H, hs, P, ws, M, D, V, ngroup, tile, m0, out);
  else
    fp8_tile<MT, ONCE>(lds, lsc, H, hs, P, ws, M, D, V, ngroup, tile, m0, out);
}

struct Fp8Args {
  const uint8_t *H, *hs, *P, *ws;
  int M, D, V;
  hipStream_t stream;
};

template <int MT, bool ONCE, typename O>
hipError_t fp8_tiles(const Fp8Args& a, O* out) {
  const int nrb = (a.M + 32 * MT - 1) / (32 * MT);
  const size_t nwork = (size_t)((a.V + kTileVocab - 1) / kTileVocab) * nrb;
  const size_t blocks = (nwork + kXcds - 1) / kXcds * kXcds;
  fp8_tile_kernel<MT, ONCE, O><<<dim3((unsigned)blocks), dim3(kF8Threads), 0, a.stream>>>(
      a.H, a.hs, a.P, reinterpret_cast<const uint32_t*>(a.ws), a.M, a.D, a.V, fp8_groups(a.V), nrb,
      (int)nwork, out);
  return hipGetLastError();
}

template <bool ONCE, typename O>
hipError_t fp8_skinny(const Fp8Args& a, O* out) {
  const int ng = fp8_groups(a.V);
  const size_t blocks = (size_t)ng * ((a.M + 31) / 32);
  fp8_skinny_kernel<ONCE, O><<<dim3((unsigned)blocks), dim3(kF8Threads), 0, a.stream>>>(
      a.H, a.hs, a.P, a.ws, a.M, a.D, a.V, ng, out);
  return hipGetLastError();
}

constexpr double kFp8CacheBytes = 256.0 * (1 << 20);

// Which product: 0 the skinny one, MT = 1..4 row blocks of at most 32 MT hidden
// rows, by an estimate of each one's time in nanoseconds.  Its constants are
// rates measured from 1 x 128256 x 4096 to 1152 x 152064 x 4096, start-up times
// fitted over 517 random sizes (1 to 1152 rows, 1000 to 150000 ids, D from 128
// to 8192, both logit types): the choice takes 1.6 % more than the best product
// on average.
//  - The skinny product reads the weights once for every 32 rows: 6.5 TB/s (4.3
//    from memory with more than 16 rows, where the hidden rows' reads tell), 5.8
//    for the blocks after the first.
//  - A tile takes 0.65 to 1.06 us a run, two on a CU as long as one after the
//    other, one alone 0.7 of that; a little more than one to a CU on average is
//    two on some.  All of them take at least the weights' time, 34 GB/s to a busy
//    CU and 5.4 TB/s, 4.3 where more than one row block reads them.
int fp8_choice(int M, int D, int V, bool exact) {
  const double bytes = (double)V * D, runs = D / kFp8Block;
  const double tiles = (V + kTileVocab - 1) / kTileVocab;
  const double first = M > 16 && bytes > kFp8CacheBytes ? 4300 : 6500;
  double best = 2000 + bytes / first + ((M + 31) / 32 - 1) * bytes / 5800;
  int choice = 0;
  const double run_ns[5] = {0, 650, 730, 870, 1060};
  for (int mt = 1; mt <= (exact ? 3 : 4); ++mt) {
    const int nrb = (M + 32 * mt - 1) / (32 * mt);
    const double cus = tiles * nrb / 256;
    const double load = cus <= 1 ? 0.7 : cus <= 1.55 ? 1.55 : cus < 3 ? 1.12 * cus : cus;
    const int steps = (M + 31) / 32, low = steps / nrb, more = steps % nrb;
    const double mean = (more * run_ns[more ? low + 1 : low] + (nrb - more) * run_ns[low]) / nrb;
    const double work = load * runs * mean * (exact ? 1.6 : 1);
    double rate = nrb == 1 ? 5400 : 4300;
    if (rate > 34 * tiles * nrb) rate = 34 * tiles * nrb;
    const double t = 6000 + (work > bytes / rate ? work : bytes / rate);
    if (t < best) {
      best = t;
      choice = mt;
    }
  }
  return choice;
}

// Weights larger than the memory-side cache (256 MB) and read once go past
// the caches: 88 -> 76 us at 1 x 128256 x 4096, 117 -> 101 us at 128 rows.
// Smaller ones may still be there from the last call (20 instead of 22 us at
// 6 x 32000 x 4096), and with several row blocks all but the first find them
// in L2 (at 320 rows 256 us past the caches, 218 through them, whole tiles).
template <bool ONCE, typename O>
hipError_t fp8_run(const Fp8Args& a, int choice, O* out) {
  if (choice == 0) return fp8_skinny<ONCE>(a, out);
  if (choice == 1) return fp8_tiles<1, ONCE>(a, out);
  if (choice == 2) return fp8_tiles<2, ONCE>(a, out);
  if constexpr (!kFp8Exact<O>)                               // float32: 4 would spill
    if (choice == 4) return fp8_tiles<4, ONCE>(a, out);
  return fp8_tiles<3, ONCE>(a, out);
}
template <typename O>
hipError_t fp8_head(const Fp8Args& a, O* out) {
  const int choice = fp8_choice(a.M, a.D, a.V, kFp8Exact<O>);
  const int rows = choice == 0 ? 32 : 32 * choice;
  return a.M <= rows && (double)a.V * a.D > kFp8CacheBytes ? fp8_run<true>(a, choice, out)
                                                              : fp8_run<false>(a, choice, out);
}

hipError_t launch_fp8_head(const uint8_t* hidden, const uint8_t* hscale, const void* packed, int M,
                           int D, int V, void* logits, bool bf16, hipStream_t stream) {
  const uint8_t* P = static_cast<const uint8_t*>(packed);
  const Fp8Args a = {hidden, hscale, P, P + fp8_packed_scale_off(V, D), M, D, V, stream};
  return bf16 ? fp8_head(a, static_cast<bf16_t*>(logits)) : fp8_head(a, static_cast<float*>(logits));
}

// Whether a product's grid fits, by the one with the most workgroups.
bool fp8_head_fits(int M, int V) {
  return grid_fits((size_t)fp8_groups(V) * ((M + 31) / 32), kF8Threads);
}

}  // namespace specv
