// Rotary tables, and appending keys and values to the 8-bit paged cache with
// the rotation of queries and keys applied on the way.
#include <math.h>

#include "awq_internal.h"
#include "kv8_common.h"

namespace awq {
namespace {

// ---------------------------------------------------------------- rotary table

// Rotations per position (radians / 2 pi) of pair j, in float64.
__device__ double rope_turns(int j, int rot, double base, RopeScaling sc) {
  const double two_pi = 6.283185307179586476925286766559;
  double f = pow(base, -2.0 * j / rot);
  if (sc.kind == 1) {
    f /= sc.factor;
  } else if (sc.kind == 2) {
    // by bands: pairs that turn more than `high` times over the trained length
    // stay, those below `low` turns are divided, linear in the turns between
    double w = (sc.trained * f / two_pi - sc.low) / (sc.high - sc.low);
    w = w < 0 ? 0 : (w > 1 ? 1 : w);
    f = w * f + (1 - w) * f / sc.factor;
  } else if (sc.kind == 3) {
    // the same ends, linear in the pair's number between them
    const double a = rot * log(sc.trained / (sc.high * two_pi)) / (2 * log(base));
    const double z = rot * log(sc.trained / (sc.low * two_pi)) / (2 * log(base));
    const double lo = fmax(floor(a), 0.0), hi = fmin(ceil(z), (double)(rot - 1));
    double w = (j - lo) / fmax(hi - lo, 0.001);
    w = w < 0 ? 0 : (w > 1 ? 1 : w);
    f = (1 - w) * f + w * f / sc.factor;
  }
  return f / two_pi;
}

// Sine and cosine of |y| <= pi / 4 from their power series: the terms left out are
// below 2^-29 and 2^-31, the fp32 roundings below one ulp of 1.
__device__ __forceinline__ float sin_eighth(float y) {
  const float z = y * y;
  float r = __builtin_fmaf(z, 1.0f / 362880, -1.0f / 5040);
  r = __builtin_fmaf(z, r, 1.0f / 120);
  r = __builtin_fmaf(z, r, -1.0f / 6);
  return __builtin_fmaf(y * z, r, y);
}
__device__ __forceinline__ float cos_eighth(float y) {
  const float z = y * y;
  float r = __builtin_fmaf(z, -1.0f / 3628800, 1.0f / 40320);
  r = __builtin_fmaf(z, r, -1.0f / 720);
  r = __builtin_fmaf(z, r, 1.0f / 24);
  r = __builtin_fmaf(z, r, -0.5f);
  return __builtin_fmaf(z, r, 1.0f);
}

// table[p][j] = m cos(p f_j), table[p][rot / 2 + j] = m sin(p f_j).  The angle is
// reduced in float64, in turns (p f / 2 pi less its nearest quarter), so that a
// position of 10^6 loses nothing; the eighth of a turn that is left goes through
// the fp32 series.  f (the power, its scaling), its quotient by 2 pi and the product
// with p are off by some 14 * 2^-53 of the angle together: 2^-25 at an angle of 2^24, but
// entries 2.8 ulp of 1 off at 2^31 (f = 1).  Bound by the 4 * positions * rot bytes written (131072 x 128: 14.2 us,
// 4.7 TB/s; 18.6 us with the library's sinpi and cospi).
__global__ __launch_bounds__(256) void rope_table_kernel(int64_t positions, int32_t rot, double base,
                                                         RopeScaling sc, float mag, int32_t per,
                                                         float* table) {
  __shared__ double turns[128];
  const int half = rot / 2;
  if (threadIdx.x < half) turns[threadIdx.x] = rope_turns(threadIdx.x, rot, base, sc);
  __syncthreads();
  const int64_t p0 = (int64_t)blockIdx.x * per, p1 = p0 + per < positions ? p0 + per : positions;
  const int step = 256 / half;
  const int j = threadIdx.x % half, at = threadIdx.x / half;
  if (at >= step) return;
  const double t = turns[j];
  for (int64_t p = p0 + at; p < p1; p += step) {
    const double a = (double)p * t;
    const double q4 = __builtin_rint(4.0 * a);
    const float y = (float)(6.283185307179586476925286766559 * (a - 0.25 * q4));     // |y| <= pi / 4
    const int q = (int)((int64_t)q4 & 3);
    const float sn = sin_eighth(y), cs = cos_eighth(y);
    const float s = q & 1 ? cs : sn, c = q & 1 ? sn : cs;
    table[p * rot + j] = mag * (q == 1 || q == 2 ? -c : c);
    table[p * rot + half + j] = mag * (q & 2 ? -s : s);
  }
}

// ---------------------------------------------------------------- append

struct AppendP {
  Kv8View v;
  const uint16_t *q, *k, *vv;
  int64_t q_stride, k_stride, v_stride, o_stride;
  const float* rope;                 // [positions][rot] or null
  int64_t positions;
  int32_t rot, inter, hq, hpt;       // hpt: query heads per work-group
  uint16_t* q_out;
  int32_t n_kv;                      // work-groups of the cache's part, which come last
};

// Channels of a head in units of 8 values that one lane holds: two runs of four,
// from a and from b.  A rotated unit u holds the pairs 4 u .. 4 u + 3 whole (both halves of
// the split layout, or eight neighbours of the interleaved one), so that a
// rotation needs nothing from another lane.
struct Runs {
  int a, b;
  bool turn;
};
__device__ __forceinline__ Runs runs_of(int u, int rot, bool inter) {
  Runs r;
  r.turn = 8 * u < rot;
  const bool split = r.turn && !inter;
  r.a = split ? 4 * u : 8 * u;
  r.b = split ? rot / 2 + 4 * u : 8 * u + 4;
  return r;
}
struct Raw {
  uint2 a, b;
};
// Each value is read once by the launch (but for pages of more than 64 slots).
__device__ __forceinline__ Raw load_raw(const uint16_t* row, const Runs& r) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  return Raw{__builtin_bit_cast(uint2, __builtin_nontemporal_load((const u32x2*)(row + r.a))),
             __builtin_bit_cast(uint2, __builtin_nontemporal_load((const u32x2*)(row + r.b)))};
}
template <bool BF>
__device__ __forceinline__ void widen(const Raw& w, float* x) {
  const uint32_t r[4] = {w.a.x, w.a.y, w.b.x, w.b.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = act2f<BF>((uint16_t)r[i]);
    x[2 * i + 1] = act2f<BF>((uint16_t)(r[i] >> 16));
  }
}
// The angles of a unit's four pairs at the table's row cs.
struct Angles {
  float c[4], s[4];
};
__device__ __forceinline__ Angles load_angles(const float* cs, int u, int rot, const Runs& r) {
  Angles g;
  const int j = r.turn ? 4 * u : 0;
  const float4 c = *(const float4*)(cs + j), s = *(const float4*)(cs + rot / 2 + j);
  g.c[0] = c.x, g.c[1] = c.y, g.c[2] = c.z, g.c[3] = c.w;
  g.s[0] = s.x, g.s[1] = s.y, g.s[2] = s.z, g.s[3] = s.w;
  return g;
}
// The rotation is one product, one product and one sum, each rounded once to
// fp32 (no fused multiply-add), so that the codes do not hang on contraction.
__device__ __forceinline__ void rotate(float* x, const Angles& g, const Runs& r, bool inter) {
  if (!r.turn) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float& p = x[inter ? 2 * i : i];
    float& q = x[inter ? 2 * i + 1 : 4 + i];
    const float a = p * g.c[i] - q * g.s[i], b = q * g.c[i] + p * g.s[i];
    p = a;
    q = b;
  }
}

// The block scale of a largest magnitude: 2^e with the least e >= -64 for which
// amax <= 448 * 2^e (448 = 0.875 * 2^9 is the largest e4m3 value).
__device__ __forceinline__ float scale_of(float amax) {
  const uint32_t u = __builtin_bit_cast(uint32_t, amax);
  // amax = 1.f * 2^x: 448 * 2^e = 1.75 * 2^(8 + e)
  int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = e < -64 ? -64 : e;
  return __builtin_bit_cast(float, (uint32_t)(e + 127) << 23);
}

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  return (uint32_t)w;
}

// Four codes rescaled by r <= 1: exact for a power of two but where the result is
// subnormal, and then the nearest code (ties to even).
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float r) {
  return codes4(__builtin_amdgcn_cvt_f32_fp8(w, 0) * r, __builtin_amdgcn_cvt_f32_fp8(w, 1) * r,
                __builtin_amdgcn_cvt_f32_fp8(w, 2) * r, __builtin_amdgcn_cvt_f32_fp8(w, 3) * r);
}

// Sequence of unit j of the cache's part.  Sequence i owns the numbers from
// cu[i] / page + 2 i on, of which it uses one for each page that its rows
// touch: n rows touch at most (n - 2) / page + 2 pages (n >= 2; one for n = 1),
// and it owns at least floor(n / page) + 2.  Ascending in i, so the sequence is
// found by counting the firsts <= j.
__device__ __forceinline__ int seq_of_unit(const Kv8View& v, int j, int lane) {
  int count = 0;
  for (int i0 = 0; i0 < v.b; i0 += 64) {
    const int i = i0 + lane;
    bool le = false;
    if (i < v.b) {
      const SeqRows r = seq_rows(v, i);
      le = (r.r0 >> v.shift) + 2 * i <= j;
    }
    count += __popcll(__ballot(le));
  }
  return count - 1;
}
// Sequences of the rows row0 .. row0 + N - 1 (-1: none); this lane gets that of row
// row0 + lane / (64 / N).
template <int N>
__device__ __forceinline__ int seq_of_rows(const Kv8View& v, int row0, int lane) {
  const int mine = lane / (64 / N);
  if (!v.cu) return row0 + mine < v.b && row0 + mine < v.rows ? row0 + mine : -1;
  int count = 0;
  for (int i0 = 0; i0 < v.b; i0 += 64) {
    int end = 0x7FFFFFFF;
    if (i0 + lane < v.b) {
      const SeqRows r = seq_rows(v, i0 + lane);
      end = r.r0 + r.n;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int n = __popcll(__ballot(end <= row0 + i));
      count += mine == i ? n : 0;
    }
  }
  return count < v.b ? count : -1;
}

// Cache part: one work-group per (page that a sequence's new rows touch, head).
// It alone writes that page's codes and scales of the head, so growing a
// part-filled page's scale and requantizing its older codes needs no atomic
// and its result does not hang on any order.  Slots are taken 64 at a time: first
// the largest magnitudes and the rows that hold inf or NaN, then the codes.  The
// 64 slots' rows are asked for at once and stay in registers between the two;
// pages of more slots read them again.  V's codes turn through LDS to lie token by
// token.
// Query part: rows x groups of heads, the angles kept over the heads.
// Bound by the bytes: 2 read per value of q, k and v, 2 written for q, 1 for k and v.
template <int D, bool BF>
__global__ __launch_bounds__(256) void kv8_append_kernel(AppendP p) {
  constexpr int LPT = D / 8;                 // lanes per token
  constexpr int TPI = 256 / LPT;             // tokens per pass of the work-group
  constexpr int SL = 64, NI = SL / TPI;      // slots of a chunk, passes for it
  const Kv8View& v = p.v;
  const int lane = threadIdx.x & 63;
  const int at = threadIdx.x / LPT, u = threadIdx.x % LPT;
  const bool inter = p.inter != 0;
  const Runs ru = runs_of(u, p.rot, inter);
  const int n_q = (int)gridDim.x - p.n_kv;
  if ((int)blockIdx.x < n_q) {
    const int groups = (p.hq + p.hpt - 1) / p.hpt;
    const int w = blockIdx.x;
    const int row0 = (w / groups) * TPI, h0 = (w % groups) * p.hpt;
    const int h1 = h0 + p.hpt < p.hq ? h0 + p.hpt : p.hq;
    constexpr int RPW = 64 / LPT;            // rows of a wave
    const int seq = seq_of_rows<RPW>(v, row0 + (threadIdx.x / 64) * RPW, lane);
    const int row = row0 + at;
    if (seq < 0) return;
    const SeqRows r = seq_rows(v, seq);
    if (row < r.r0 || row >= r.r0 + r.n) return;
    const int64_t pos = (int64_t)r.ctx - r.n + (row - r.r0);
    const bool out_of = p.rope && (pos < 0 || pos >= p.positions);
    Angles g = {};
    if (p.rope) g = load_angles(p.rope + (out_of ? 0 : pos) * p.rot, u, p.rot, ru);
    const uint16_t* src = p.q + row * p.q_stride + (int64_t)h0 * D;
    uint16_t* dst = p.q_out + row * p.o_stride + (int64_t)h0 * D;
#pragma unroll 8
    for (int h = h0; h < h1; ++h, src += D, dst += D) {
      float y[8];
      widen<BF>(load_raw(src, ru), y);
      rotate(y, g, ru, inter);
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float nan = __builtin_nanf("");
        o[i] = out_of ? pack2<BF>(nan, nan) : pack2<BF>(y[2 * i], y[2 * i + 1]);
      }
      *(uint2*)(dst + ru.a) = make_uint2(o[0], o[1]);
      *(uint2*)(dst + ru.b) = make_uint2(o[2], o[3]);
    }
    return;
  }

  const int h = (blockIdx.x - n_q) % v.hkv, unit = (blockIdx.x - n_q) / v.hkv;
  const int seq = seq_of_unit(v, unit, lane);
  if (seq < 0) return;
  const SeqRows r = seq_rows(v, seq);
  const int page = 1 << v.shift;
  const int64_t first = (int64_t)r.ctx - r.n;                 // position of the first new row
  const int64_t lo_pos = first < 0 ? 0 : first;
  const int nth = unit - ((r.r0 >> v.shift) + 2 * seq);
  const int64_t j = (lo_pos >> v.shift) + nth;
  if (nth < 0 || r.n == 0 || (j << v.shift) >= r.ctx || j >= v.max_pages) return;
  const int pid = v.bt[(int64_t)seq * v.max_pages + j];
  if ((uint32_t)pid >= (uint64_t)v.pages) return;             // not in the cache: dropped
  const int64_t page0 = j << v.shift;
  const int a = (int)(lo_pos > page0 ? lo_pos - page0 : 0);  // older tokens of the page
  const int z = (int)(r.ctx - page0 < page ? r.ctx - page0 : page);
  const int64_t ph = (int64_t)pid * v.hkv + h;
  const int64_t row0 = r.r0 + page0 - first;                  // row of the page's slot 0
  const Runs rv = runs_of(u, 0, false);
  const uint16_t* ksrc = p.k + row0 * p.k_stride + (int64_t)h * D;
  const uint16_t* vsrc = p.vv + row0 * p.v_stride + (int64_t)h * D;

  __shared__ uint32_t bad[256 / 32];
  __shared__ uint32_t kmax[4], vmax[4];
  __shared__ uint32_t turn[SL][D / 4 + 1];                    // V codes [slot][channel]
  if (threadIdx.x < 256 / 32) bad[threadIdx.x] = 0;
  const float kold = a ? v.ks[ph] : 0.0f, vold = a ? v.vs[ph] : 0.0f;
  float y[NI][8];                                             // rotated keys
  Raw x[NI];                                                  // values
  const int cfirst = a / SL * SL;
  auto fetch = [&](int c0) {
    const uint16_t* kp = ksrc + (c0 + at) * p.k_stride;
    const uint16_t* vp = vsrc + (c0 + at) * p.v_stride;
    Raw kk[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int s = c0 + i * TPI + at;
      if (s >= a && s < z) {
        kk[i] = load_raw(kp + i * TPI * p.k_stride, ru);
        x[i] = load_raw(vp + i * TPI * p.v_stride, rv);
      }
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int s = c0 + i * TPI + at;
      if (s >= a && s < z) {
        widen<BF>(kk[i], y[i]);
        if (p.rope) {
          const int64_t pos = page0 + s;
          rotate(y[i], load_angles(p.rope + (pos < p.positions ? pos : 0) * p.rot, u, p.rot, ru), ru, inter);
        }
      }
    }
  };
  fetch(cfirst);
  __syncthreads();
  // Magnitudes are compared as their bits: inf and NaN are above every finite value.
  constexpr uint32_t kInf16 = BF ? 0x7F80u : 0x7C00u;
  uint32_t km = 0, vm = 0;
  for (int c0 = cfirst; c0 < z; c0 += SL) {
    if (c0 > cfirst) fetch(c0);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int s = c0 + i * TPI + at;
      const bool here = s >= a && s < z;
      uint32_t ka = 0, va = 0;
      if (here) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t m = __builtin_bit_cast(uint32_t, y[i][e]) & 0x7FFFFFFFu;
          ka = ka > m ? ka : m;
        }
        const uint32_t r[4] = {x[i].a.x, x[i].a.y, x[i].b.x, x[i].b.y};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t lo = r[e] & 0x7FFFu, hi = r[e] >> 16 & 0x7FFFu;
          va = va > lo ? va : lo;
          va = va > hi ? va : hi;
        }
      }
      bool ok = ka < 0x7F800000u && va < kInf16 && (!p.rope || page0 + s < p.positions || !here);
      const uint64_t group = ((1ull << LPT) - 1) << (lane & ~(LPT - 1));
      ok = (__ballot(!ok) & group) == 0;
      if (!ok && u == 0) atomicOr(&bad[s >> 5], 1u << (s & 31));
      if (ok) {
        km = km > ka ? km : ka;
        vm = vm > va ? vm : va;
      }
    }
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) {
    const uint32_t k2 = __shfl_xor(km, o, 64), v2 = __shfl_xor(vm, o, 64);
    km = km > k2 ? km : k2;
    vm = vm > v2 ? vm : v2;
  }
  if (lane == 0) {
    kmax[threadIdx.x >> 6] = km;
    vmax[threadIdx.x >> 6] = vm;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    km = km > kmax[i] ? km : kmax[i];
    vm = vm > vmax[i] ? vm : vmax[i];
  }
  const float ks = __builtin_fmaxf(scale_of(__builtin_bit_cast(float, km)), kold);
  const float vs = __builtin_fmaxf(scale_of(act2f<BF>((uint16_t)vm)), vold);
  const float kr = kold / ks, vr = vold / vs;
  if (threadIdx.x == 0) {
    v.ks[ph] = ks;
    v.vs[ph] = vs;
  }
  // x / scale is x * (1 / scale) for the powers of two that this kernel writes; a scale
  // that another writer left in the page need not be one
  const bool exact = ((__builtin_bit_cast(uint32_t, ks) | __builtin_bit_cast(uint32_t, vs)) & 0x7FFFFFu) == 0;
  const float ki = 1.0f / ks, vi = 1.0f / vs;
  uint8_t* kp = v.kc + (ph << v.shift) * D;
  uint8_t* vp = v.vc + ((ph * D) << v.shift);
  if (a && kr != 1.0f)
    for (int i = threadIdx.x; i < a * D / 4; i += 256) ((uint32_t*)kp)[i] = rescale4(((uint32_t*)kp)[i], kr);
  for (int c0 = vr != 1.0f ? 0 : cfirst; c0 < z; c0 += SL) {
    const int c1 = c0 + SL < z ? c0 + SL : z;
    if (z - cfirst > SL && c1 > a) fetch(c0);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int s = c0 + i * TPI + at;
      if (s < a || s >= z) continue;
      uint32_t k0 = 0x7F7F7F7Fu, k1 = 0x7F7F7F7Fu, v0 = 0, v1 = 0;
      if (!(bad[s >> 5] >> (s & 31) & 1)) {
        float e[8], f[8];
        widen<BF>(x[i], f);
        if (exact) {
#pragma unroll
          for (int c = 0; c < 8; ++c) e[c] = y[i][c] * ki, f[c] = f[c] * vi;
        } else {
#pragma unroll
          for (int c = 0; c < 8; ++c) e[c] = y[i][c] / ks, f[c] = f[c] / vs;
        }
        k0 = codes4(e[0], e[1], e[2], e[3]);
        k1 = codes4(e[4], e[5], e[6], e[7]);
        v0 = codes4(f[0], f[1], f[2], f[3]);
        v1 = codes4(f[4], f[5], f[6], f[7]);
      }
      *(uint32_t*)(kp + s * D + ru.a) = k0;
      *(uint32_t*)(kp + s * D + ru.b) = k1;
      turn[s % SL][2 * u] = v0;
      turn[s % SL][2 * u + 1] = v1;
    }
    __syncthreads();
    // V: a thread turns 4 channels x 8 slots; eight neighbours write 64 bytes of a
    // channel.  Slots that are not new keep what they held.
    const int from = vr != 1.0f || a < c0 ? c0 : a;
    for (int i = threadIdx.x; i < D / 4 * (SL / 8); i += 256) {
      const int c = i / (SL / 8), s0 = c0 + i % (SL / 8) * 8;
      if (s0 + 8 <= from || s0 >= c1) continue;
      uint32_t t[8], w[4][2];
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] = turn[s0 % SL + e][c];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t* r = t + 4 * q;
        const uint32_t ab0 = __builtin_amdgcn_perm(r[1], r[0], 0x05010400), ab1 = __builtin_amdgcn_perm(r[1], r[0], 0x07030602);
        const uint32_t cd0 = __builtin_amdgcn_perm(r[3], r[2], 0x05010400), cd1 = __builtin_amdgcn_perm(r[3], r[2], 0x07030602);
        w[0][q] = __builtin_amdgcn_perm(cd0, ab0, 0x05040100);
        w[1][q] = __builtin_amdgcn_perm(cd0, ab0, 0x07060302);
        w[2][q] = __builtin_amdgcn_perm(cd1, ab1, 0x05040100);
        w[3][q] = __builtin_amdgcn_perm(cd1, ab1, 0x07060302);
      }
      const bool all = s0 >= a && s0 + 8 <= z;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t* g = (uint32_t*)(vp + ((4 * c + q) << v.shift) + s0);
        if (all) {
          *(uint2*)g = make_uint2(w[q][0], w[q][1]);
          continue;
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int s = s0 + 4 * half, lo = a - s, hi = z - s;      // slots lo .. hi - 1 of the word are new
          if (s + 4 <= from || hi <= 0) continue;
          const uint32_t older = lo <= 0 ? 0u : lo >= 4 ? ~0u : (1u << (8 * lo)) - 1u;
          const uint32_t keep = hi >= 4 ? 0u : ~((1u << (8 * hi)) - 1u);
          const uint32_t was = older | keep ? g[half] : 0u;
          g[half] = (w[q][half] & ~(older | keep)) | (was & keep) |
                    ((vr != 1.0f && older ? rescale4(was, vr) : was) & older);
        }
      }
    }
    __syncthreads();
  }
}

}  // namespace

hipError_t launch_rope_table(int64_t positions, int32_t rot, double base, const RopeScaling& sc,
                             float* table, hipStream_t stream) {
  const int step = 256 / (rot / 2);
  // about eight work-groups per CU, each at least one round of its threads
  int64_t per = (positions + 2047) / 2048;
  per = (per + step - 1) / step * step;
  const float mag = sc.kind == 3 && sc.factor > 1 ? (float)(0.1 * log(sc.factor) + 1.0) : 1.0f;
  rope_table_kernel<<<(unsigned)((positions + per - 1) / per), 256, 0, stream>>>(positions, rot, base, sc, mag,
                                                                                (int32_t)per, table);
  return hipGetLastError();
}

hipError_t launch_kv8_append(const Kv8Args& a, const uint16_t* q, int64_t q_stride, const uint16_t* k,
                             int64_t k_stride, const uint16_t* v, int64_t v_stride, int32_t hq,
                             const float* rope, int64_t positions, int32_t rot, bool interleaved,
                             bool bf, uint16_t* q_out, int64_t q_out_stride, hipStream_t stream) {
  if (a.rows < 1 || a.b < 1) return hipSuccess;
  AppendP p;
  p.v = Kv8View{a.k, a.v, a.k_scale, a.v_scale, a.block_table, a.cu_q, a.ctx, a.pages, a.rows,
                (int32_t)a.max_pages, __builtin_ctz((unsigned)a.page), a.hkv, (int32_t)a.b};
  p.q = q;
  p.k = k;
  p.vv = v;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.o_stride = q_out_stride;
  p.rope = rope;
  p.positions = positions;
  p.rot = rope ? rot : 0;
  p.inter = interleaved;
  p.hq = hq;
  p.q_out = q_out;
  const int64_t units = (a.rows >> p.v.shift) + 2 * a.b;
  p.n_kv = (int32_t)(units * a.hkv);
  int64_t nq = 0;
  p.hpt = 1;
  if (q) {
    const int64_t rowgroups = (a.rows + 2048 / a.d - 1) / (2048 / a.d);
    // heads that share one reading of the angles: as many as leave four
    // work-groups per CU
    while (p.hpt < 8 && p.hpt < hq && rowgroups * ((hq + 2 * p.hpt - 1) / (2 * p.hpt)) >= 1024) p.hpt *= 2;
    nq = rowgroups * ((hq + p.hpt - 1) / p.hpt);
  }
  const unsigned grid = (unsigned)(p.n_kv + nq);
  if (a.d == 64) {
    if (bf) kv8_append_kernel<64, true><<<grid, 256, 0, stream>>>(p);
    else kv8_append_kernel<64, false><<<grid, 256, 0, stream>>>(p);
  } else {
    if (bf) kv8_append_kernel<128, true><<<grid, 256, 0, stream>>>(p);
    else kv8_append_kernel<128, false><<<grid, 256, 0, stream>>>(p);
  }
  return hipGetLastError();
}

}  // namespace awq
