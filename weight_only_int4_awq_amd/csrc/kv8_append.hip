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

// table[p][j] = m cos(p f_j), table[p][rot / 2 + j] = m sin(p f_j).  The angle is
// reduced in float64, in turns (p f / 2 pi less its nearest quarter), so that a
// position of 10^6 loses nothing; the eighth of a turn that is left goes through
// fp32 sine and cosine.  Bound by the 4 * positions * rot bytes written.
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
    const float x = (float)(2.0 * (a - 0.25 * q4));         // half turns, |x| <= 1/4
    const int q = (int)((int64_t)q4 & 3);
    const float sn = sinpif(x), cs = cospif(x);
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
  int32_t n_kv;                      // work-groups of the cache's part
};

// 8 values of a row's head, channels d0 .. d0 + 7, rotated at position pos.
// The rotation is one product, one product and one sum, each rounded once to
// fp32 (no fused multiply-add), so that the codes do not hang on contraction.
template <bool BF>
__device__ __forceinline__ void load_rotated(const uint16_t* row, int d0, const float* cs, int rot,
                                             bool inter, float* y) {
  const uint4 raw = *(const uint4*)(row + d0);
  const uint32_t* r = (const uint32_t*)&raw;
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = act2f<BF>((uint16_t)r[i]);
    x[2 * i + 1] = act2f<BF>((uint16_t)(r[i] >> 16));
  }
  if (d0 >= rot) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i];
    return;
  }
  const int half = rot / 2;
  if (inter) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float c = cs[d0 / 2 + i], s = cs[half + d0 / 2 + i];
      y[2 * i] = x[2 * i] * c - x[2 * i + 1] * s;
      y[2 * i + 1] = x[2 * i + 1] * c + x[2 * i] * s;
    }
    return;
  }
  const bool hi = d0 >= half;
  const int j = hi ? d0 - half : d0;
  const uint4 mate = *(const uint4*)(row + (hi ? d0 - half : d0 + half));
  const uint32_t* mr = (const uint32_t*)&mate;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float z = act2f<BF>((uint16_t)(mr[i / 2] >> (16 * (i & 1))));
    const float c = cs[j + i], s = cs[half + j + i];
    y[i] = hi ? x[i] * c + z * s : x[i] * c - z * s;
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

__device__ __forceinline__ bool finite(float x) {
  return (__builtin_bit_cast(uint32_t, x) & 0x7F800000u) != 0x7F800000u;
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
__device__ __forceinline__ int seq_of_row(const Kv8View& v, int row, int lane) {
  if (!v.cu) return row < v.b ? row : -1;
  int count = 0;
  for (int i0 = 0; i0 < v.b; i0 += 64) {
    const int i = i0 + lane;
    bool le = false;
    if (i < v.b) {
      const SeqRows r = seq_rows(v, i);
      le = r.r0 + r.n <= row;
    }
    count += __popcll(__ballot(le));
  }
  return count < v.b ? count : -1;
}

// Cache part: one work-group per (page that a sequence's new rows touch, head).
// It alone writes that page's codes and scales of the head, so growing a
// part-filled page's scale and requantizing its older codes needs no atomic
// and its result does not hang on any order.  Two passes over the new rows
// (the second from the caches): largest magnitudes and rows that hold inf or
// NaN, then the codes.  V's codes turn through LDS to lie token by token.
// Query part: rows x groups of heads, the angles kept over the heads.
template <int D, bool BF>
__global__ __launch_bounds__(256) void kv8_append_kernel(AppendP p) {
  constexpr int LPT = D / 8;                 // lanes per token
  constexpr int TPI = 256 / LPT;             // tokens per pass of the work-group
  const Kv8View& v = p.v;
  const int lane = threadIdx.x & 63;
  const int at = threadIdx.x / LPT, d0 = (threadIdx.x % LPT) * 8;
  if ((int)blockIdx.x >= p.n_kv) {
    const int groups = (p.hq + p.hpt - 1) / p.hpt;
    const int u = blockIdx.x - p.n_kv;
    const int row0 = (u / groups) * TPI, h0 = (u % groups) * p.hpt;
    const int h1 = h0 + p.hpt < p.hq ? h0 + p.hpt : p.hq;
    // the rows of this wave, one after another: all lanes vote on each
    constexpr int RPW = 64 / LPT;
    const int wrow = row0 + (threadIdx.x / 64) * RPW;
    int seq = -1;
#pragma unroll
    for (int i = 0; i < RPW; ++i) {
      const int s = wrow + i < v.rows ? seq_of_row(v, wrow + i, lane) : -1;
      if (lane / LPT == i) seq = s;
    }
    const int row = row0 + at;
    if (seq < 0) return;
    const SeqRows r = seq_rows(v, seq);
    if (row < r.r0 || row >= r.r0 + r.n) return;
    const int64_t pos = (int64_t)r.ctx - r.n + (row - r.r0);
    const bool out_of = p.rope && (pos < 0 || pos >= p.positions);
    const float* cs = p.rope ? p.rope + (out_of ? 0 : pos) * p.rot : nullptr;
    for (int h = h0; h < h1; ++h) {
      float y[8];
      load_rotated<BF>(p.q + row * p.q_stride + (int64_t)h * D, d0, cs, p.rot, p.inter, y);
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = (uint32_t)f2act(out_of ? __builtin_nanf("") : y[2 * i], BF) |
               (uint32_t)f2act(out_of ? __builtin_nanf("") : y[2 * i + 1], BF) << 16;
      // the pair's other half is read by other lanes of this wave: with q_out = q
      // all of them have read it before any writes
      __builtin_amdgcn_wave_barrier();
      *(uint4*)(p.q_out + row * p.o_stride + (int64_t)h * D + d0) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return;
  }

  const int h = blockIdx.x % v.hkv, unit = blockIdx.x / v.hkv;
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

  __shared__ uint32_t bad[256 / 32];
  __shared__ float kmax[4], vmax[4];
  __shared__ uint8_t turn[256][D + 4];                        // V codes [slot][channel]
  if (threadIdx.x < 256 / 32) bad[threadIdx.x] = 0;
  __syncthreads();
  float km = 0.0f, vm = 0.0f;
  for (int s0 = a; s0 < z; s0 += TPI) {
    const int s = s0 + at;
    float y[8], x[8], ka = 0.0f, va = 0.0f;
    bool ok = true;
    if (s < z) {
      const int64_t row = row0 + s, pos = page0 + s;
      const bool out_of = p.rope && pos >= p.positions;
      const float* cs = p.rope ? p.rope + (out_of ? 0 : pos) * p.rot : nullptr;
      load_rotated<BF>(p.k + row * p.k_stride + (int64_t)h * D, d0, cs, p.rot, p.inter, y);
      load_rotated<BF>(p.vv + row * p.v_stride + (int64_t)h * D, d0, nullptr, 0, false, x);
      ok = !out_of;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ok = ok && finite(y[i]) && finite(x[i]);
        ka = __builtin_fmaxf(ka, __builtin_fabsf(y[i]));
        va = __builtin_fmaxf(va, __builtin_fabsf(x[i]));
      }
    }
    const uint64_t group = ((1ull << LPT) - 1) << (lane & ~(LPT - 1));
    ok = (__ballot(!ok) & group) == 0;
    if (!ok && s < z && d0 == 0) atomicOr(&bad[s >> 5], 1u << (s & 31));
    if (ok) {
      km = __builtin_fmaxf(km, ka);
      vm = __builtin_fmaxf(vm, va);
    }
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) {
    km = __builtin_fmaxf(km, __shfl_xor(km, o, 64));
    vm = __builtin_fmaxf(vm, __shfl_xor(vm, o, 64));
  }
  if (lane == 0) {
    kmax[threadIdx.x >> 6] = km;
    vmax[threadIdx.x >> 6] = vm;
  }
  const float kold = a ? v.ks[ph] : 0.0f, vold = a ? v.vs[ph] : 0.0f;
  __syncthreads();
  km = __builtin_fmaxf(__builtin_fmaxf(kmax[0], kmax[1]), __builtin_fmaxf(kmax[2], kmax[3]));
  vm = __builtin_fmaxf(__builtin_fmaxf(vmax[0], vmax[1]), __builtin_fmaxf(vmax[2], vmax[3]));
  const float ks = __builtin_fmaxf(scale_of(km), kold), vs = __builtin_fmaxf(scale_of(vm), vold);
  const float kr = kold / ks, vr = vold / vs;
  if (threadIdx.x == 0) {
    v.ks[ph] = ks;
    v.vs[ph] = vs;
  }
  uint8_t* kp = v.kc + (ph << v.shift) * D;
  uint8_t* vp = v.vc + ((ph * D) << v.shift);
  if (a && kr != 1.0f)
    for (int i = threadIdx.x; i < a * D / 4; i += 256) ((uint32_t*)kp)[i] = rescale4(((uint32_t*)kp)[i], kr);
  for (int s0 = a; s0 < z; s0 += TPI) {
    const int s = s0 + at;
    if (s >= z) continue;
    const int64_t row = row0 + s, pos = page0 + s;
    uint2 kw = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu), vw = make_uint2(0, 0);
    if (!(bad[s >> 5] >> (s & 31) & 1)) {
      float y[8], x[8];
      const float* cs = p.rope ? p.rope + pos * p.rot : nullptr;
      load_rotated<BF>(p.k + row * p.k_stride + (int64_t)h * D, d0, cs, p.rot, p.inter, y);
      load_rotated<BF>(p.vv + row * p.v_stride + (int64_t)h * D, d0, nullptr, 0, false, x);
      // true quotients: a scale that another writer left need not be a power of two
      kw = make_uint2(codes4(y[0] / ks, y[1] / ks, y[2] / ks, y[3] / ks),
                      codes4(y[4] / ks, y[5] / ks, y[6] / ks, y[7] / ks));
      vw = make_uint2(codes4(x[0] / vs, x[1] / vs, x[2] / vs, x[3] / vs),
                      codes4(x[4] / vs, x[5] / vs, x[6] / vs, x[7] / vs));
    }
    *(uint2*)(kp + s * D + d0) = kw;
    uint32_t* t = (uint32_t*)&turn[s][d0];
    t[0] = vw.x;
    t[1] = vw.y;
  }
  __syncthreads();
  // V: whole words of four slots; slots that are not new keep what they held
  const int w0 = vr != 1.0f ? 0 : a >> 2, w1 = (z + 3) >> 2, nw = w1 - w0;
  for (int i = threadIdx.x; i < nw * D; i += 256) {
    const int d = i / nw, w = w0 + i % nw;
    uint32_t* g = (uint32_t*)(vp + (d << v.shift)) + w;
    uint32_t word = 0, keep = 0, older = 0;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int s = 4 * w + x;
      const uint32_t m = 0xFFu << (8 * x);
      if (s < a) older |= m;
      else if (s >= z) keep |= m;
      else word |= (uint32_t)turn[s][d] << (8 * x);
    }
    if (older | keep) {
      const uint32_t was = *g;
      word |= was & keep;
      word |= (vr != 1.0f ? rescale4(was, vr) : was) & older;
    }
    *g = word;
  }
}

}  // namespace

hipError_t launch_rope_table(int64_t positions, int32_t rot, double base, const RopeScaling& sc,
                             float* table, hipStream_t stream) {
  const int step = 256 / (rot / 2);
  // about eight work-groups per CU, each at least one round of its threads
  int64_t per = (positions + 2047) / 2048;
  per = (per + step - 1) / step * step;
  const float mag = sc.kind == 3 ? (float)(0.1 * log(sc.factor) + 1.0) : 1.0f;
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
