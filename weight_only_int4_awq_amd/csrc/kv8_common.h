// Shared by the kernels of the 8-bit paged KV cache (kv8_append.hip,
// attn_kv8.hip): the cache's description on the device, the batch's metadata,
// and the conversions of e4m3 codes.
//
// Layout: page id `pid` of head h holds P tokens:
//   k codes  kc[((pid * hkv + h) * P + slot) * D + d]     (channels contiguous)
//   v codes  vc[((pid * hkv + h) * D + d) * P + slot]     (tokens contiguous)
//   scales   ks[pid * hkv + h], vs[pid * hkv + h]
// K rows feed the score product and V columns the output product straight from
// global memory as MFMA operands: both products contract over the axis that is
// contiguous in memory, so no transposition stands between the cache and the
// matrix instruction.
#pragma once

#include "awq_common.h"

namespace awq {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

struct Kv8View {
  uint8_t* kc;
  uint8_t* vc;
  float* ks;
  float* vs;
  const int32_t* bt;       // [b][max_pages]
  const int32_t* cu;       // [b + 1] or null: one row per sequence
  const int32_t* ctx;      // [b]
  int64_t pages;           // pages of the cache
  int64_t rows;            // rows of q, k, v
  int32_t max_pages, shift, hkv, b;   // page = 1 << shift
};

// Rows [r0, r0 + n) and tokens with them of sequence i.  Whatever the arrays
// hold, r0 and n stay within the rows there are.
struct SeqRows {
  int32_t r0, n, ctx;
};
__device__ __forceinline__ SeqRows seq_rows(const Kv8View& v, int i) {
  SeqRows s;
  if (v.cu) {
    const int rows = (int)v.rows;
    int a = v.cu[i], z = v.cu[i + 1];
    a = a < 0 ? 0 : (a > rows ? rows : a);
    z = z < a ? a : (z > rows ? rows : z);
    s.r0 = a;
    s.n = z - a;
  } else {
    s.r0 = i;
    s.n = i < v.rows ? 1 : 0;
  }
  const int c = v.ctx[i];
  s.ctx = c < 0 ? 0 : c;
  return s;
}

// Inclusive sum over the lanes of a wave, in six register moves.
__device__ __forceinline__ int wave_scan(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);   // lane - 1 of the row of 16
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);   // - 2
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);   // - 4
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);   // - 8
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);   // the row before's last
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);   // the half before's last
  return x;
}

// Largest and sum over the lanes of a wave, the same way; the same in all lanes.
template <class Op>
__device__ __forceinline__ float wave_fold(float x, float none, Op op) {
  const int n = __builtin_bit_cast(int, none);
  auto from = [&](float v, int moved) { return op(v, __builtin_bit_cast(float, moved)); };
#define AWQ_FOLD(CTRL, ROWS) \
  x = from(x, __builtin_amdgcn_update_dpp(n, __builtin_bit_cast(int, x), CTRL, ROWS, 0xf, false))
  AWQ_FOLD(0x111, 0xf);
  AWQ_FOLD(0x112, 0xf);
  AWQ_FOLD(0x114, 0xf);
  AWQ_FOLD(0x118, 0xf);
  AWQ_FOLD(0x142, 0xa);
  AWQ_FOLD(0x143, 0xc);
#undef AWQ_FOLD
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 63));
}

// 8 e4m3 codes (two 32-bit words) as the MFMA operand type: exact in fp16 and
// in bf16 (4 significant bits, |code| <= 448, least 2^-9); NaN codes stay NaN.
template <bool BF>
struct Mma;
template <>
struct Mma<false> {
  typedef half8_t frag;
  static __device__ __forceinline__ frag from_fp8(uint32_t lo, uint32_t hi) {
    const half2_t a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
    const half2_t b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
    const half2_t c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
    const half2_t d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
    return frag{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
  }
  static __device__ __forceinline__ floatx4_t mma16(frag a, frag b, floatx4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ floatx16_t mma32(frag a, frag b, floatx16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Mma<true> {
  typedef bf16x8_t frag;
  static __device__ __forceinline__ frag from_fp8(uint32_t lo, uint32_t hi) {
    const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    return frag{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
  }
  static __device__ __forceinline__ floatx4_t mma16(frag a, frag b, floatx4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ floatx16_t mma32(frag a, frag b, floatx16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
};

template <bool BF>
__device__ __forceinline__ float act2f(uint16_t b) {
  return BF ? bf2f(b) : h2f(b);
}
// two values rounded once each (nearest, ties to even) to fp16 or bf16
template <bool BF>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (BF) return __builtin_bit_cast(uint32_t, (bf16x2_t){(__bf16)a, (__bf16)b});
  else return __builtin_bit_cast(uint32_t, (half2_t){(half_t)a, (half_t)b});
}
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
// A value at an address that is the same in all lanes and that the launch does not
// write, by a scalar load: it waits for no vector load asked for before it.
template <class T>
__device__ __forceinline__ T scalar_load(const T* p) {
  typedef const T __attribute__((address_space(4))) constant_t;
  const uint64_t a = (uint64_t)(uintptr_t)p;
  const uint64_t u = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a) |
                     (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32)) << 32;
  return *(constant_t*)u;
}

}  // namespace awq
