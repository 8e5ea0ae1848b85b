// What the LM heads on 8- and 4-bit floats share: loads, the barrier of a
// product loop and the way of a tile's logits to memory.
#pragma once

#include <type_traits>

#include "common.h"
#include "fp8.h"

namespace specv {

typedef float HeadF32x16 __attribute__((ext_vector_type(16)));

constexpr int kTileVocab = 256;                    // vocabulary rows of a tile, 64 a wave
constexpr int kHeadThreads = 256;
constexpr int kXcds = 8;

__device__ __forceinline__ void head_put(float* p, float v) { *p = v; }
__device__ __forceinline__ void head_put(bf16_t* p, float v) { *p = bf16_bits(v); }
// Four consecutive logits, registers r .. r + 3 of an accumulator.
__device__ __forceinline__ void head_put4(float* p, const HeadF32x16& c, int r) {
  *reinterpret_cast<float4*>(p) = make_float4(c[r], c[r + 1], c[r + 2], c[r + 3]);
}
__device__ __forceinline__ void head_put4(bf16_t* p, const HeadF32x16& c, int r) {
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

// LDS writes of this workgroup made visible at a barrier, global loads left
// in flight.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// The LDS that a tile's logits leave through: up to 128 rows of bfloat16 or 64 of
// float32 at a time, 70 KB (two workgroups a CU have 80 each), so that few barriers
// part the stores.  At 1152 x 152064 x 4096 of 4-bit weights and states this takes
// 469 us; 32 rows at a time took 479, and no stores at all 435.  At 8-bit states,
// bound by the products, both take the same.
template <int MT, typename O>
struct HeadStore {
  static constexpr int kStride = kTileVocab + 16 / (int)sizeof(O);
  static constexpr int kMost = 8 / (int)sizeof(O);         // 32-row steps of a pass
  static constexpr int kSteps = MT < kMost ? MT : kMost;
  static constexpr int kBytes = 32 * kSteps * kStride * (int)sizeof(O);
};

// A tile's logits, by its four waves, to rows m0 .. and ids 256 tile ..; lds is
// free at the call (HeadStore<MT, O>::kBytes of it are used).
template <int MT, typename O>
__device__ __forceinline__ void head_store(uint8_t* lds, const HeadF32x16 (&acc)[2][MT], int tile,
                                           int m0, int M, int V, O* __restrict__ out) {
  constexpr int kTrStride = HeadStore<MT, O>::kStride, kSteps = HeadStore<MT, O>::kSteps;
  const int tid = threadIdx.x, lane = tid % kWave, h = lane / 32, l32 = lane % 32;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
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
  auto pass = [&](auto first) {
    constexpr int t0 = decltype(first)::value, kT = kSteps < MT - t0 ? kSteps : MT - t0;
    constexpr int kPassRows = 32 * kT, r0 = t0 * 32;         // its rows, the first in the block
    // float32 in two halves of the lanes: written by all at once, the compiler
    // spills the accumulators (52 to 208 registers)
    constexpr int kHalves = sizeof(O) / 2;
#pragma unroll
    for (int i = 0; i < kT * kHalves; ++i) {
      const int t = i / kHalves;
      if (kHalves > 1 && l32 / 16 != i % kHalves) continue;
      O* row = tr + (t * 32 + l32) * kTrStride + vb;
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int q = 0; q < 4; ++q) head_put4(row + 32 * a + 8 * q, acc[a][t0 + t], 4 * q);
    }
    lds_barrier();
    if (whole) {
#pragma unroll 4
      for (int i = 0; i < kPassRows * kTileVocab / kVec / kHeadThreads; ++i) {
        const int p = tid + i * kHeadThreads, row = p / (kTileVocab / kVec);
        const int c = p % (kTileVocab / kVec) * kVec;
        if (m0 + r0 + row < M && c < nv)
          *reinterpret_cast<uint4*>(out + (size_t)(m0 + r0 + row) * V + v0 + c) =
              *reinterpret_cast<const uint4*>(tr + row * kTrStride + c);
      }
    } else {
      constexpr int kLog = 4 / sizeof(O);                  // logits of a 4-byte store
#pragma unroll 4
      for (int i = 0; i < kPassRows * kTileVocab / kLog / kHeadThreads; ++i) {
        const int p = tid + i * kHeadThreads, row = p / (kTileVocab / kLog);
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
  };
  pass(std::integral_constant<int, 0>{});
  if constexpr (MT > kSteps) pass(std::integral_constant<int, kSteps>{});
  static_assert(MT <= 2 * kSteps, "two passes at most");
}

}  // namespace specv
