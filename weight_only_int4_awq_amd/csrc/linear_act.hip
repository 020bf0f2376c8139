// The 4-bit linear with an epilogue, alone or grouped by expert:
//
//   acc[r][c] = sum_k x~[r][k] (q[c][k] - z[c][k / g]) D[c][k / g]        x~ = fp16(x inv_s) or x
//   y[r][o]   = act(acc[r][o] + bias[o]) (+ res[r][o])
//   y[r][o]   = act(acc[r][o] + bias[o]) (acc[r][n + o] + bias[n + o]) (+ res[r][o])    gated
//
// Rows of expert i are offsets[i] .. offsets[i + 1] - 1 and use its weights; the row counts
// are device data, so work-groups find their expert and rows themselves and the grid is an
// upper bound.  Roundings: bf16 activations once to fp16 (exact within fp16's normal range: the
// matrix instructions take one type, and neither x inv_s nor weights times their scale fit bf16's
// 8 bits); x inv_s once to fp16, which is what all linears here take (by pairs without loss where
// four rows or fewer stream, see there; for more the rest would be a second product of its own,
// twice the matrix work of the tiles, for 1.7e-4 of a result); weights exactly.  Sums, bias,
// activation and residual are fp32 with one rounding at the end.
#include "decode_common.h"
#include "moe_common.h"

namespace awq {

// ---------------------------------------------------------------- which rows a work-group has

struct Place {
  int expert, row0, rows;      // rows of the tile: row0 .. row0 + rows - 1, at least one
  int all;                     // rows of the expert
  int col, sl;                 // column block, slice of K
};

// Rows of expert i (none behind the last).  Every lane loads, so that loads of several runs of
// experts fly together.  False: the offsets do not ascend within the rows there are.
__device__ __forceinline__ bool expert_rows(const ActArgs& a, int i, int& r0, int& n) {
  const int j = i < a.e ? i : a.e - 1;
  const int s = a.offsets[j], t = a.offsets[j + 1];
  r0 = s;
  n = i < a.e ? t - s : 0;
  return s >= 0 && t >= s && t <= (int)a.rows;
}

// Units of a launch are fewer.
constexpr int64_t kMaxUnits = 1 << 22;

// x / y for 0 <= x < kMaxUnits, 0 < y < 2^24: x and y are exact in fp32; for y of 1 and 2 so is the
// quotient, from 3 on it is below 2^21 and off by 1.5 2^-23 of it, less than one: one step either way.
__device__ __forceinline__ int quot(int x, int y) {
  int q = (int)((float)x * __builtin_amdgcn_rcpf((float)y));
  const int rem = x - q * y;
  q += rem >= y ? 1 : 0;
  q -= rem < 0 ? 1 : 0;
  return uniform(q);
}

// The units of a launch: tiles of 2^lt rows of each expert x column blocks x K slices, in an
// order in which the tiles of an expert follow one another (bands of four row tiles, column by
// column), so that work-groups next to one another share weights or rows.  Units are below
// kMaxUnits (the host checks).
struct Units {
  int lt;                                                // tiles of 2^lt rows
  static constexpr int KEEP = 2;                         // experts 0 .. 127 are looked up once
  int r0[KEEP], n[KEEP], inc[KEEP];                      // lane l: experts l, l + 64: rows, tiles up to it
  int tiles_all;

  __device__ __forceinline__ int tiles_of(int rows_) const { return (rows_ + (1 << lt) - 1) >> lt; }

  // How many there are; none under offsets that do not ascend within the rows (ascending ones
  // share the rows out, so the sums below stay within the host's bound).
  __device__ __forceinline__ int count(const ActArgs& a, int lane) {
    if (!a.offsets) {
      tiles_all = tiles_of((int)a.rows);
    } else {
      tiles_all = 0;
      bool ok = true;
#pragma unroll
      for (int j = 0; j < KEEP; ++j) ok &= expert_rows(a, 64 * j + lane, r0[j], n[j]);
      for (int b = 64 * KEEP; b < a.e; b += 64) {
        int first, cnt;
        ok &= expert_rows(a, b + lane, first, cnt);
      }
      if (__ballot(!ok)) return 0;
#pragma unroll
      for (int j = 0; j < KEEP; ++j) {
        inc[j] = wave_scan(tiles_of(n[j])) + tiles_all;
        tiles_all = __builtin_amdgcn_readlane(inc[j], 63);
      }
      for (int b = 64 * KEEP; b < a.e; b += 64) {
        int first, cnt;
        expert_rows(a, b + lane, first, cnt);
        tiles_all += __builtin_amdgcn_readlane(wave_scan(tiles_of(cnt)), 63);
      }
    }
    return tiles_all * a.ncol * a.ks;
  }

  __device__ __forceinline__ void at(const ActArgs& a, int lane, int o, Place& p) const {
    p.sl = 0;
    if (a.ks > 1) {
      const int q = quot(o, a.ks);
      p.sl = o - q * a.ks;
      o = q;
    }
    int tiles = tiles_all, first = 0, rows = (int)a.rows;
    p.expert = 0;
    p.row0 = 0;
    if (a.offsets) {
      const int t = quot(o, a.ncol);
      bool found = false;
      int last = 0;
      auto take = [&](int base, int r, int cnt, int sum) {   // the first lane whose sum passes t
        const uint64_t here = __ballot(t < sum);
        if (here && !found) {
          const int l = __builtin_ctzll(here);
          found = true;
          p.expert = base + l;
          rows = __builtin_amdgcn_readlane(cnt, l);
          tiles = tiles_of(rows);
          first = __builtin_amdgcn_readlane(sum, l) - tiles;
          p.row0 = __builtin_amdgcn_readlane(r, l);
        }
        last = __builtin_amdgcn_readlane(sum, 63);
      };
#pragma unroll
      for (int j = 0; j < KEEP; ++j) take(64 * j, r0[j], n[j], inc[j]);
      for (int b = 64 * KEEP; !found && b < a.e; b += 64) {
        int f, cnt;
        expert_rows(a, b + lane, f, cnt);
        take(b, f, cnt, wave_scan(tiles_of(cnt)) + last);
      }
    }
    const int local = o - first * a.ncol;
    int tm, tn;
    if (tiles <= 4) {
      tn = tiles == 1 ? local : quot(local, tiles);
      tm = local - tn * tiles;
    } else {
      const int band = quot(local, 4 * a.ncol), left = tiles - 4 * band;
      const int wide = left < 4 ? left : 4, in = local - band * 4 * a.ncol;
      tn = quot(in, wide);
      tm = 4 * band + in - tn * wide;
    }
    p.col = tn;
    p.row0 += tm << lt;
    p.all = rows;
    rows -= tm << lt;
    p.rows = rows < 1 << lt ? rows : 1 << lt;
  }
};

// The one unit of this work-group: every XCD takes a contiguous run of the order.  False:
// nothing to do.
__device__ __forceinline__ bool find_place(const ActArgs& a, int lane, int lt, Place& p) {
  Units units;
  units.lt = lt;
  const int total = units.count(a, lane);
  const int per = (total + 7) / 8, slot = blockIdx.x >> 3;
  const int o = (blockIdx.x & 7) * per + slot;
  if (slot >= per || o >= total) return false;
  units.at(a, lane, o, p);
  return true;
}

// The row of x that a slot reads, held within the rows there are whatever the plan says.
// slot / topk as the upper half of slot * ceil(2^32 / topk): exact where slot times the
// rounding of the second (below topk <= 32) stays below 2^32, so for all slots up to 2^27.
__device__ __forceinline__ int slot_token(const ActArgs& a, int slot) {
  const uint32_t s = (uint32_t)(slot < 0 ? 0 : slot);
  const uint32_t t = a.topk == 1 ? s : __umulhi(s, a.topk_inv);
  const uint32_t last = (uint32_t)a.x_rows - 1;
  return (int)(t < last ? t : last);
}

// ---------------------------------------------------------------- epilogue

// erfc(x) = t exp(P(t) - x^2), t = 1 / (1 + |x| / 2), and 2 minus that below zero: the form that
// Press et al., Numerical Recipes, give for the complementary error function.  P: a polynomial
// fitted here at Chebyshev nodes to log(exp(x^2) erfc(x) / t) over x in [0, 14.6], off by 1.2e-7;
// with the rounding of the exponent 3e-6 relative up to x = 5, 8e-6 up to 9.2.  1 + erf(x) would
// lose the lower tail's digits.
__device__ __forceinline__ float erfc_tail(float x) {
  const float z = __builtin_fabsf(x);
  const float t = __builtin_amdgcn_rcpf(1.0f + 0.5f * z);
  float q = 0.16738100f;
  q = __builtin_fmaf(q, t, -0.80132526f);
  q = __builtin_fmaf(q, t, 1.43554544f);
  q = __builtin_fmaf(q, t, -1.06009936f);
  q = __builtin_fmaf(q, t, 0.21378274f);
  q = __builtin_fmaf(q, t, -0.15077300f);
  q = __builtin_fmaf(q, t, 0.08468209f);
  q = __builtin_fmaf(q, t, 0.37655020f);
  q = __builtin_fmaf(q, t, 0.99975681f);
  q = __builtin_fmaf(q, t, -1.26550055f);
  const float e = t * __expf(__builtin_fmaf(-z, z, q));
  return x < 0.0f ? 2.0f - e : e;
}

__device__ __forceinline__ float activate(float v, int act) {
  // v / (1 + exp(-u)), 1 / (1 + exp) by the hardware reciprocal (1 ulp)
  if (act == 1) return v * __builtin_amdgcn_rcpf(1.0f + __expf(-v));
  if (act == 2) return 0.5f * v * erfc_tail(v * -0.70710678118654752f);
  if (act == 3) {                                      // 1 + tanh(u) = 2 / (1 + exp(-2 u))
    const float u = 1.5957691216057308f * (v + 0.044715f * v * v * v);
    return v * __builtin_amdgcn_rcpf(1.0f + __expf(-u));
  }
  return v;
}

__device__ __forceinline__ float act_bits(uint16_t b, int bf) { return bf ? bf2f(b) : h2f(b); }

// Output o of a row from its sums (u: the up projection's, where gated), before the residual.
__device__ __forceinline__ float finish(const ActArgs& a, int expert, int64_t o, float v, float u) {
  if (a.bias) {
    const uint16_t* b = a.bias + (int64_t)expert * a.nw;
    v += act_bits(b[o], a.bf);
    if (a.gated) u += act_bits(b[a.n + o], a.bf);
  }
  v = activate(v, a.act);
  return a.gated ? v * u : v;
}

// ---------------------------------------------------------------- copies to LDS

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// lane i copies 16 (4) bytes from sbase + voff to LDS bytes lds_base + 16 i (4 i)
__device__ __forceinline__ void lds_copy16(uint32_t voff, const void* sbase, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :
               : "v"(voff), "s"(sbase), "s"(lds_base)
               : "memory", "m0");
}
__device__ __forceinline__ void lds_copy4(uint32_t voff, const void* sbase, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
               :
               : "v"(voff), "s"(sbase), "s"(lds_base)
               : "memory", "m0");
}
#pragma clang diagnostic pop
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// a barrier without the fence of __syncthreads, which would wait for every copy in flight
__device__ __forceinline__ void tile_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// ---------------------------------------------------------------- few rows: weights streamed
//
// Up to TM rows of one expert times two blocks of 16 weight rows (gated: 16 outputs' gate rows
// and their up rows); the W <= 4 waves of a work-group share K in runs of four 128-channel
// blocks.  A lane reads 16 bytes (32 codes) of one weight row per block, straight into
// registers: every byte of the weights is read once and waits for nothing but memory, all of a
// run asked for before the first is used.  The rows of a run
// (512 channels; 256 where TM = 16) go through the wave's own LDS: scaled, rounded to fp16 and
// put in the order of the unpacked nibbles once, then read as operands.  An expert's rows times
// inv_s16, if there are four or fewer, enter as a pair: fp16 rounding loses 2^-11 of a product,
// and rows 4 .. 7 of the 8-row tile, else idle, hold what was lost (one token, gate and up of
// 2 x 14336 x 4096: 18.0 -> 18.3 us).
// v_mfma_f32_16x16x32_f16, rows as A, weights as B.  g = 128: a block is one group, its
// integers q - z enter exactly and the group's sum is scaled in fp32.  g = 32, 64: a lane's 32
// codes are of one group, but a product takes codes of four lanes and so of several groups; weights
// enter as fp16((q - z) D) and, in a second product, what that lost: at most 4 bits above the last
// bit of D, exact.  Against the first product alone: one token, gate and up of 2 x 14336 x 4096
// 23.4 -> 26.1 us (g = 64), 24.9 -> 27.1 (32); 64 tokens on 128 experts 104 -> 116, 110 -> 121.
// (Integers with the other groups' rows as zeros, two or four products a word: 26.2 and 31.9; 109
// and 153.)
// Bound by the weights' bytes: one token on two of 8 experts (122 MB) 28.0 us, 4.4 TB/s; dense
// gate and up of one token (61 MB) 14.4 us, 4.2; 64 tokens on 128 experts (256 MB) 69 us, 3.7:
// there 8000 work-groups of one run to a wave each pay for their plan, their rows and their
// first load (captured, weights cold: 77 us, without the plan 69, without rows too 54, the
// weight loads alone 52).
// Two blocks of 16 weight rows and up to 4 waves: four blocks or 8 waves leave too few work-
// groups or registers (experts of 1 token 36 to 46 us against 33, captured, weights cold).
constexpr int kRun = 4;                              // blocks of a run
constexpr int kCB = 2;                                // blocks of 16 weight rows
template <int TM>
struct StreamLds {
  static constexpr int SB = TM == 16 ? 2 : 4;        // blocks staged at a time
  static constexpr int STRIDE = SB * 256 + 16;       // bytes of a staged row: 16 rows on 64 banks
  static constexpr int WAVE = TM * STRIDE;
};

// What fp16 lost of hi = x s, element by element, times 2^kRest: at most half a unit of hi's last
// place, so within fp16's range, and above its subnormal numbers where hi is above 2^-14.  With it
// x s is within max(2^-22 |x s|, 2^-36).  Nothing where hi left fp16's range.
constexpr int kRest = 11;
__device__ __forceinline__ uint4 remainder8(const half8_t x, const half8_t s, const half8_t hi) {
  half8_t lo;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float h = (float)hi[i];
    const float r = __builtin_fmaf((float)x[i], (float)s[i], -h) * (float)(1 << kRest);
    lo[i] = (_Float16)(__builtin_fabsf(h) <= 65504.0f ? r : 0.0f);
  }
  return __builtin_bit_cast(uint4, lo);
}

// Scales and zero points of a lane's codes in the blocks of a run, as they are loaded.
// QUADS (g = 128, rows of a multiple of four groups): a run's scales are 8 aligned bytes.
template <int G, bool QUADS>
struct RunScales {
  uint32_t s[kCB][QUADS ? 2 : kRun];                  // fp16 bits, two to a word or one
  uint32_t z[kCB][G == 32 ? 2 : 1];                   // words of zero points
};

template <int G, int TM, bool QUADS>
__global__ __launch_bounds__(256, 2) void linear_act_stream_kernel(const ActArgs a) {
  static_assert((TM == 8 || TM == 16) && (G == 128 || !QUADS), "");
  constexpr int SB = StreamLds<TM>::SB, STRIDE = StreamLds<TM>::STRIDE;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int waves = blockDim.x >> 6;
  Place p;
  if (!find_place(a, lane, TM == 16 ? 4 : 3, p)) return;
  // rows 4 .. 7: what rounding rows 0 .. 3 lost; by the expert's rows, so that all of them are rounded alike
  const bool low = TM == 8 && a.inv && p.all <= 4;
  const int r = lane & 15, c = lane >> 4;
  const int k = (int)a.k;
  // outputs col0 .. of the gate and the same of the up projection, or two blocks of outputs
  const int half = a.gated ? kCB / 2 : kCB;
  const int col0 = p.col * half * 16;
  // lane i: the row of x that row i of the tile reads; asked for first, the rows wait for it
  const int row_i = p.row0 + (r < p.rows ? r : p.rows - 1);
  const int src = a.row_slot ? slot_token(a, a.row_slot[row_i]) : row_i;
  const char* qb = reinterpret_cast<const char*>(a.qw + (int64_t)p.expert * a.nw * (a.k / 8));
  const char* sb = reinterpret_cast<const char*>(a.sc + (int64_t)p.expert * a.nw * a.ng);
  const char* zb = reinterpret_cast<const char*>(a.qz + (int64_t)p.expert * a.nw * a.nzw);
  uint32_t row_w[kCB];
#pragma unroll
  for (int cb = 0; cb < kCB; ++cb) {
    const int up = cb >= half;
    const uint32_t o = (uint32_t)(col0 + (up ? cb - half : cb) * 16 + r), n = (uint32_t)a.n;
    row_w[cb] = (o < n ? o : n - 1) + (up ? n : 0);
  }
  const UnpackConsts uc = unpack_consts();
  const int nb = (k + 127) / 128;
  const int b0 = wave * a.per, b1 = b0 + a.per < nb ? b0 + a.per : nb;

  // the lane's 32 channels of block b: its first one, held within the row
  auto channel = [&](int b) {
    const int kk = b * 128 + 32 * c;
    return kk < k ? kk : k - 32;
  };
  auto load_w = [&](int b, uint4 (&w)[kRun][kCB], RunScales<G, QUADS>& rs) {
#pragma unroll
    for (int cb = 0; cb < kCB; ++cb) {                  // first: what returns in order is waited for in order
      const uint32_t so = row_w[cb] * (uint32_t)(a.ng * 2), zo = row_w[cb] * (uint32_t)(a.nzw * 4);
      if constexpr (QUADS) {
        const uint2 v = *reinterpret_cast<const uint2*>(sb + (so + (uint32_t)b * 2));
        rs.s[cb][0] = v.x;
        rs.s[cb][1] = v.y;
      } else {
#pragma unroll
        for (int i = 0; i < kRun; ++i)
          rs.s[cb][i] = *reinterpret_cast<const uint16_t*>(
              sb + (so + (uint32_t)(channel(b + i < b1 ? b + i : b1 - 1) / G) * 2));
      }
      // 8 zero points to a word: a run of four groups, eight or sixteen
      constexpr int ZW = G == 32 ? 2 : 1;
#pragma unroll
      for (int j = 0; j < ZW; ++j) {
        int w4 = b * (128 / G) / 8 + j;
        w4 = w4 < a.nzw ? w4 : a.nzw - 1;
        rs.z[cb][j] = *reinterpret_cast<const uint32_t*>(zb + (zo + (uint32_t)w4 * 4));
      }
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      const uint32_t off = (uint32_t)channel(b + i < b1 ? b + i : b1 - 1) / 2;
#pragma unroll
      for (int cb = 0; cb < kCB; ++cb)
        w[i][cb] = *reinterpret_cast<const uint4*>(qb + (row_w[cb] * (uint32_t)(k / 2) + off));
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // ---- the rows' channels of SB blocks: 16 bytes to a lane, 64 or 32 lanes to a row
  constexpr int XL = 8;                              // loads of a lane, all in flight
  unsigned char* stage = lds + wave * StreamLds<TM>::WAVE;
  const int xc = SB == 4 ? lane : lane & 31, xh = SB == 4 ? 0 : lane >> 5;
  auto load_x = [&](int b, uint4 (&x)[XL], uint4& iv) {
    const int ch = b * 128 + 8 * xc;
    const int cc = ch < k ? ch : k - 8;
#pragma unroll
    for (int i = 0; i < XL; ++i) {
      if (SB == 4) {
        if (i < p.rows)
          x[i] = *reinterpret_cast<const uint4*>(a.x + (int64_t)__builtin_amdgcn_readlane(src, i) * a.k + cc);
      } else if (2 * i < p.rows) {
        const int s0 = __builtin_amdgcn_readlane(src, 2 * i), s1 = __builtin_amdgcn_readlane(src, 2 * i + 1);
        x[i] = *reinterpret_cast<const uint4*>(a.x + (int64_t)(xh ? s1 : s0) * a.k + cc);
      }
    }
    if (a.inv) iv = *reinterpret_cast<const uint4*>(a.inv + cc);
  };
  auto store_x = [&](int b, const uint4 (&x)[XL], const uint4& iv) {
    const bool in = b * 128 + 8 * xc < k;            // the last block may be half a one (g < 128)
    auto store = [&](int i, const uint4& v, bool part) {
      // channels in the order of the unpacked nibbles: (0, 4), (1, 5), (2, 6), (3, 7)
      uint4 u = make_uint4(__builtin_amdgcn_perm(v.z, v.x, 0x05040100u), __builtin_amdgcn_perm(v.z, v.x, 0x07060302u),
                           __builtin_amdgcn_perm(v.w, v.y, 0x05040100u), __builtin_amdgcn_perm(v.w, v.y, 0x07060302u));
      if (!in) u = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(stage + ((SB == 4 ? i : 2 * i + xh) + (part ? 4 : 0)) * STRIDE + xc * 16) = u;
    };
#pragma unroll
    for (int i = 0; i < XL; ++i)
      if ((SB == 4 ? i : 2 * i) < p.rows) {
        uint4 v = act8_h(x[i], a.bf != 0);
        if (a.inv) {
          const half8_t xv = __builtin_bit_cast(half8_t, v), sv = __builtin_bit_cast(half8_t, iv);
          const half8_t hi = xv * sv;
          v = __builtin_bit_cast(uint4, hi);
          if (low) store(i, remainder8(xv, sv, hi), true);
        }
        store(i, v, false);
      }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  };

  floatx4_t acc[kCB];
#pragma unroll
  for (int cb = 0; cb < kCB; ++cb) acc[cb] = floatx4_t{};
  const unsigned char* frag = stage + (TM == 16 ? r : r & 7) * STRIDE + c * 64;
  auto block = [&](int b, int i, const uint4 (&w)[kCB], const RunScales<G, QUADS>& rs, auto rest) {
    half8_t af[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) af[s] = *reinterpret_cast<const half8_t*>(frag + (i % SB) * 256 + s * 16);
    const bool in = G == 128 || b * 128 + 32 * c < k;
#pragma unroll
    for (int cb = 0; cb < kCB; ++cb) {
      // fields of the zero word: the block's group within the eight of a word
      const int gr = G == 128 ? b & 7 : G == 64 ? (2 * i + (c >> 1)) : (4 * (i & 1) + c);
      const uint32_t z = (rs.z[cb][G == 32 ? i >> 1 : 0] >> (4 * gr)) & 0xFu;
      uint32_t d = QUADS ? (rs.s[cb][i >> 1] >> (16 * (i & 1))) & 0xFFFFu : rs.s[cb][QUADS ? 0 : i];
      if (!in) d = 0;
      const half2_t o1024 = __builtin_bit_cast(half2_t, (0xE400u + z) * 0x10001u);
      const half2_t o64 = __builtin_bit_cast(half2_t, (0xD400u + (z << 4)) * 0x10001u);
      const half2_t dd = __builtin_bit_cast(half2_t, d * 0x10001u);
      floatx4_t part = G == 128 ? floatx4_t{} : acc[cb];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const uint32_t word = s == 0 ? w[cb].x : s == 1 ? w[cb].y : s == 2 ? w[cb].z : w[cb].w;
        uint32_t u[4], lo[4];
        unpack_word(word, u, uc);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          half2_t q = __builtin_bit_cast(half2_t, u[j]) + (j & 1 ? o64 : o1024);
          if (G != 128) {
            const half2_t hi = q * dd;
            lo[j] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(q, dd, -hi));
            q = hi;
          }
          u[j] = __builtin_bit_cast(uint32_t, q);
        }
        if constexpr (G != 128 && rest)
          part = __builtin_amdgcn_mfma_f32_16x16x32_f16(
              af[s], __builtin_bit_cast(half8_t, make_uint4(lo[0], lo[1], lo[2], lo[3])), part, 0, 0, 0);
        part = __builtin_amdgcn_mfma_f32_16x16x32_f16(af[s], __builtin_bit_cast(half8_t, make_uint4(u[0], u[1], u[2], u[3])),
                                                      part, 0, 0, 0);
      }
      if (G == 128) {
        const float df = h2f((uint16_t)d);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[cb][j] = __builtin_fmaf(part[j], df, acc[cb][j]);
      } else {
        acc[cb] = part;
      }
    }
  };

  auto sweep = [&](auto rest) {
    for (int b = b0; b < b1; b += kRun) {
      uint4 w[kRun][kCB], x[XL], iv = make_uint4(0, 0, 0, 0);
      RunScales<G, QUADS> rs;
      load_x(b, x, iv);
      load_w(b, w, rs);
      store_x(b, x, iv);
      if (SB == 2 && b + 2 < b1) load_x(b + 2, x, iv);
      block(b, 0, w[0], rs, rest);
      if (b + 1 < b1) block(b + 1, 1, w[1], rs, rest);
      if (SB == 2 && b + 2 < b1) store_x(b + 2, x, iv);
      if (b + 2 < b1) block(b + 2, 2, w[2], rs, rest);
      if (b + 3 < b1) block(b + 3, 3, w[3], rs, rest);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
  };
  sweep(std::true_type{});
  if constexpr (G != 128) {
    // an infinity in x is NaN once multiplied with a rest of zero, a weight beyond fp16 with its rest:
    // such sums are taken once more, without the rests
    bool odd = false;
#pragma unroll
    for (int cb = 0; cb < kCB; ++cb)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = 4 * c + j;
        odd |= (row < p.rows || (low && row < p.rows + 4)) && acc[cb][j] != acc[cb][j];
      }
    if (__ballot(odd)) {
      floatx4_t first[kCB];
#pragma unroll
      for (int cb = 0; cb < kCB; ++cb) {
        first[cb] = acc[cb];
        acc[cb] = floatx4_t{};
      }
      sweep(std::false_type{});
#pragma unroll
      for (int cb = 0; cb < kCB; ++cb)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[cb][j] = first[cb][j] == first[cb][j] ? first[cb][j] : acc[cb][j];
    }
  }
  // ---- the waves' sums, added in wave order: [wave][block][4][lane]
  __syncthreads();
  float* red = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int cb = 0; cb < kCB; ++cb)
#pragma unroll
    for (int j = 0; j < 4; ++j) red[(wave * kCB + cb) * 256 + j * 64 + lane] = acc[cb][j];
  __syncthreads();
  const int outs = half * 256;
  for (int i = tid; i < outs; i += blockDim.x) {
    const int l = i & 63, j = (i >> 6) & 3, cb = i >> 8;
    const int row = (l >> 4) * 4 + j;
    const int64_t o = col0 + cb * 16 + (l & 15);
    if (row >= p.rows || o >= a.n) continue;
    float v = 0.0f, u = 0.0f;
    for (int w = 0; w < waves; ++w) {
      const float* s = red + w * kCB * 256 + i;
      v += s[0];
      if (a.gated) u += s[outs];
      if (low) {                                       // row + 4: lane + 16
        v += s[16] * (1.0f / (1 << kRest));
        if (a.gated) u += s[outs + 16] * (1.0f / (1 << kRest));
      }
    }
    const int64_t at = (int64_t)(p.row0 + row) * a.n + o;
    float f = finish(a, p.expert, o, v, u);
    if (a.res) f += act_bits(a.res[at], a.bf);
    a.y[at] = f2act(f, a.bf != 0);
  }
}

// ---------------------------------------------------------------- many rows: tiles
//
// BM rows x 256 weight rows of one expert, K-steps of BK, 4 waves side by side along the weight
// rows, each BM x 64 in 32 x 32 blocks of v_mfma_f32_32x32x16_f16; gated, a wave's two blocks
// are 32 outputs' gate rows and their up rows, so the product of the two needs no exchange.
// KG = 2: a second set of 4 waves takes every other K-step, where there are few tiles.
// Copies from global memory to LDS in a ring of three stages, two K-steps ahead, with explicit
// waits (the compiler sees neither).  Rows are read in channel order (gathered by the copies' own
// addresses), so nibbles are unpacked in pairs of neighbours: a byte permute and a mask per pair.
//
// The products take the integers q - z, exact in fp16, and the sums are kept in units of the
// group's scale: where a group ends they are multiplied by its scale over the next one's (fp32: a
// reciprocal and two products, 2^-22 a group), and at the end by the last one's.  A second set of
// sums, scaled and added per group, would take 128 registers that 128 rows do not have.  A scale
// of zero keeps the unit and takes the codes' bits instead (an infinity in x times it is NaN, as it
// should be).  What it costs against weights rounded to fp16((q - z) D), 1.7e-4 of a result: g = 128
// 4096 tokens on 8 experts 1975 -> 1993 us, down projection of 2048 rows 269 -> 277, 700 x 4096 x 4096
// (one wave to a SIMD, nothing to cover it) 46 -> 50, 8 experts of 16 rows 158 -> 145; g = 64, gate
// and up of 2048 rows 468 -> 482; g = 32 491 -> 570.
// 128-row tiles are bound by the matrix pipe and the card's power: 4096 tokens by twos on 8 experts
// (1924 GFLOP) 1.98 ms, 970 TFLOP/s where a large library product reaches 1054; 2048 rows of
// 4096 <- 14336 262 us, 21 of them the rows' conversion.  32-row tiles are
// bound by how the cache takes their copies: 64 weight rows a copy are 32 to 64 lines, and a
// K-step is there when the wave needs it only if enough work-groups share a CU (300 tokens on 60
// experts, 102 MB: 43 us; 333 rows of 4099 <- 1088: 18 us, a K-step of 64 1.2 us).  Fewer
// registers by a rolled ring (23.2 against 22.2 us), two stages and a third work-group (53
// against 48.6) or four and five stages brought nothing.
constexpr int kTileBN = 256;
constexpr int kTileStages = 3;
constexpr int tile_stage_bytes(int bm, int bk) { return bm * bk * 2 + kTileBN * bk / 2; }
// Per K group: two words of scales and two of zero points of every column, and a place for copies
// of nothing.
constexpr int kTileScales = 4 * kTileBN * 4 + 4 * 256;

// Masks and selectors of the unpack in channel order, opaque to constant folding: a VOP3
// instruction takes no literal and one scalar operand.
struct PairConsts {
  uint32_t sel[4], mask, magic;
};
__device__ __forceinline__ PairConsts pair_consts() {
  PairConsts p;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    p.sel[i] = 0x01040004u + 0x00010001u * i;        // bytes: code byte i, 0x64, code byte i, 0x54
    asm volatile("" : "+s"(p.sel[i]));
  }
  p.mask = 0xFFF0FF0Fu;
  asm volatile("" : "+s"(p.mask));
  p.magic = 0x00005464u;
  asm volatile("" : "+v"(p.magic));
  return p;
}

template <int G, int KG, int BM, int BK>
__global__ __launch_bounds__(256 * KG, KG == 1 ? 2 : 1) void linear_act_tile_kernel(const ActArgs a) {
  static_assert(BK == 64 || (BK == 128 && G >= 64), "a word of scales holds those of a K-step");
  constexpr int NG = BK > G ? BK / G : 1;             // groups of a K-step, one after the other
  constexpr int QS = NG > 1 && G == 32 ? 2 : 4;       // a lane's half of 16 QS channels: QS words, as many sub-steps
  constexpr int BN = kTileBN;
  constexpr int CH = BK / 8, BCH = BK / 32, NS = BK / 16;   // 16-byte chunks of a row and of a weight row, sub-steps
  constexpr int BMB = BM / 32, BNB = 2;
  constexpr int RPC = 64 / CH, AR = BM / 4 / RPC;     // rows of a copy, row copies of a wave and step
  constexpr int kCopies = AR + BCH + 2;               // + those of packed words, scale and zero words
  constexpr int kStage = tile_stage_bytes(BM, BK), ST = kTileStages;
  constexpr int kA = BM * BK * 2;
  __shared__ __attribute__((aligned(16))) unsigned char ring[KG * (ST * kStage + kTileScales)];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kgrp = wave >> 2, wv = wave & 3;
  Place p;
  if (!find_place(a, lane, BM == 32 ? 5 : BM == 64 ? 6 : 7, p)) return;
  const int k = (int)a.k;
  const int nk = k / BK;
  const int kt0 = (int)((int64_t)p.sl * nk / a.ks), kt1 = (int)((int64_t)(p.sl + 1) * nk / a.ks);
  const int nr = (kt1 - kt0 + KG - 1) / KG;           // round P: K group g takes K-step kt0 + KG P + g

  const uint32_t ring_lds = (uint32_t)(uintptr_t)(&ring[0]) + (uint32_t)(kgrp * kStage);
  const unsigned char* ring_g = ring + kgrp * kStage;
  const uint32_t words_lds = (uint32_t)(uintptr_t)(&ring[0]) + (uint32_t)(KG * ST * kStage + kgrp * kTileScales);
  const unsigned char* words_g = ring + KG * ST * kStage + kgrp * kTileScales;
  // ---- copy sources: a wave-uniform base and the lane's 32-bit byte offset
  const int a_lr = lane / CH, a_p = lane % CH;
  // chunks lie XOR-swizzled so that 16 rows' (columns') chunks fall on all banks
  auto a_swz = [](int row) { return BK == 64 ? (row >> 1) & 7 : row & 15; };
  auto b_swz = [](int col) { return (col >> 2) & (BCH - 1); };
  // rows: their own addresses when gathered (x below 4 GiB), else from the tile's first row
  const char* xb = reinterpret_cast<const char*>(a.x + (a.row_slot ? 0 : (int64_t)p.row0 * a.k));
  uint32_t a_voff[AR];
#pragma unroll
  for (int i = 0; i < AR; ++i) {
    const int lrow = wv * (BM / 4) + RPC * i + a_lr;
    const int row = lrow < p.rows ? lrow : p.rows - 1;
    const int src = a.row_slot ? slot_token(a, a.row_slot[p.row0 + row]) : row;
    a_voff[i] = (uint32_t)(((int64_t)src * a.k + (a_p ^ a_swz(lrow)) * 8) * 2);
  }
  // weight row of the tile's column lcol: gated, 32 gate rows and their 32 up rows per wave
  const int span = a.gated ? 128 : 256;
  const int64_t col0 = (int64_t)p.col * span;
  auto weight_row = [&](int lcol) -> int64_t {
    if (!a.gated) {
      const int64_t o = col0 + lcol;
      return o < a.n ? o : a.n - 1;
    }
    const int64_t o = col0 + (lcol >> 6) * 32 + (lcol & 31);
    return (o < a.n ? o : a.n - 1) + (lcol & 32 ? a.n : 0);
  };
  const char* qb = reinterpret_cast<const char*>(a.qw + (int64_t)p.expert * a.nw * (a.k / 8));
  const char* zb = reinterpret_cast<const char*>(a.qz + (int64_t)p.expert * a.nw * a.nzw);
  // scales in whole words: an expert may begin, and a row with an odd number of groups
  // does begin, in the middle of one
  const int64_t s_first = (int64_t)p.expert * a.nw * a.ng;
  const char* sb = reinterpret_cast<const char*>(a.sc + (s_first & ~1ll));
  const uint32_t s_odd = (uint32_t)(s_first & 1);
  uint32_t b_voff[BCH];
#pragma unroll
  for (int h = 0; h < BCH; ++h) {
    const int lcol = wv * 64 + 64 / BCH * h + lane / BCH;
    b_voff[h] = (uint32_t)(weight_row(lcol) * (k / 2) + (((lane % BCH) ^ b_swz(lcol)) * 16));
  }
  const int64_t sz_row = weight_row(wv * 64 + lane);
  const bool s_turn = (a.ng & 1) != 0;               // rows begin in either half of a word: new words every group
  // place of the scale word of group g: where a K group's rounds are two words apart, by pairs
  auto s_place = [&](int g) {
    const int word = s_turn ? g : g >> 1;
    return (KG * BK >= (s_turn ? 2 : 4) * G ? word >> 1 : word) & 1;
  };
  const uint32_t s_idx = (uint32_t)(sz_row * a.ng) + s_odd, z_voff = (uint32_t)(sz_row * a.nzw * 4);
  auto load = [&](int rnd, int st) {
    int kt = kt0 + KG * rnd + kgrp;
    kt = kt < kt1 ? kt : kt1 - 1;
    const uint32_t base = ring_lds + (uint32_t)(st * KG * kStage);
    const char* xk = xb + (int64_t)kt * BK * 2;
#pragma unroll
    for (int i = 0; i < AR; ++i) lds_copy16(a_voff[i], xk, base + (uint32_t)((wv * (BM / 4) + RPC * i) * BK * 2));
    const char* qk = qb + (int64_t)kt * (BK / 2);
#pragma unroll
    for (int h = 0; h < BCH; ++h) lds_copy16(b_voff[h], qk, base + (uint32_t)(kA + (wv * 64 + 64 / BCH * h) * (BK / 2)));
    // A word holds two groups' scales, or eight groups' zero points, and serves until the next:
    // 64 columns lie on 64 lines, so the copies between are of one line, to nowhere (the waits
    // count copies).  A word is read into registers a round ahead, so two places take turns.
    const int g0 = kt * BK / G, gp = rnd > 0 ? (kt0 + KG * (rnd - 1) + kgrp) * BK / G : -64;
    const bool past = kt0 + KG * rnd + kgrp >= kt1;
    const bool s_new = !past && (s_turn ? g0 != gp : g0 >> 1 != gp >> 1), z_new = !past && g0 >> 3 != gp >> 3;
    const uint32_t nowhere = words_lds + (uint32_t)(4 * BN * 4 + wv * 256);
    lds_copy4(s_new ? ((s_idx + (uint32_t)g0) >> 1) * 4 : 0u, sb,
              s_new ? words_lds + (uint32_t)(s_place(g0) * BN * 4 + wv * 256) : nowhere);
    lds_copy4(z_new ? z_voff + (uint32_t)(g0 >> 3) * 4 : 0u, zb,
              z_new ? words_lds + (uint32_t)((2 + ((g0 >> 3) & 1)) * BN * 4 + wv * 256) : nowhere);
  };

  floatx16_t acc[BMB][BNB];
#pragma unroll
  for (int i = 0; i < BMB; ++i)
#pragma unroll
    for (int j = 0; j < BNB; ++j) acc[i][j] = floatx16_t{};
  const PairConsts pc = pair_consts();
  // ---- fragments: sub-step s takes 8 channels of each half of the lanes, of one group:
  // from 16 QS (s / QS) + 8 QS (lane / 32) + 8 (s % QS) on, rows and words alike
  const int bj = lane & 31, bc = lane >> 5;
  uint32_t a_base[BMB];
#pragma unroll
  for (int bm = 0; bm < BMB; ++bm) {
    const int row = bm * 32 + bj;
    a_base[bm] = (uint32_t)(row * BK * 2 + ((QS * bc) ^ a_swz(row)) * 16);
  }
  uint32_t b_off[BNB], s_off[BNB], s_par[BNB];
#pragma unroll
  for (int bn = 0; bn < BNB; ++bn) {
    const int lcol = wv * 64 + bn * 32 + bj;
    b_off[bn] = (uint32_t)(kA + lcol * (BK / 2) + (QS == 4 ? (bc ^ b_swz(lcol)) * 16 : b_swz(lcol) * 16 + 8 * bc));
    s_off[bn] = (uint32_t)(lcol * 4);
    s_par[bn] = ((uint32_t)(weight_row(lcol) * a.ng) + s_odd) & 1;
  }
  struct BSet {
    uint4 wb[BNB][BCH / 2];
    half2_t off[NG][BNB];
    uint32_t d[BNB];                                  // scales of the K-step's groups, in halves
    uint32_t mask[BNB];                               // one group: no bits of the codes where its scale is zero
  };
  // what a wave copied itself needs only its own wait: the step's words, scale and zero
  auto prep = [&](int rnd, int st, BSet& r) {
    const unsigned char* s = ring_g + st * KG * kStage;
    const int g0 = (kt0 + KG * rnd + kgrp) * BK / G;
#pragma unroll
    for (int bn = 0; bn < BNB; ++bn) {
#pragma unroll
      for (int h = 0; h < BCH / 2; ++h) {
        if constexpr (QS == 4) {
          r.wb[bn][h] = *reinterpret_cast<const uint4*>(s + (b_off[bn] ^ (uint32_t)(32 * h)));
        } else {
          const uint2 l = *reinterpret_cast<const uint2*>(s + b_off[bn]);
          const uint2 u = *reinterpret_cast<const uint2*>(s + (b_off[bn] ^ 16u));
          r.wb[bn][h] = make_uint4(l.x, l.y, u.x, u.y);
        }
      }
      const uint32_t sw = *reinterpret_cast<const uint32_t*>(words_g + s_place(g0) * BN * 4 + s_off[bn]);
      const uint32_t zw = *reinterpret_cast<const uint32_t*>(words_g + (2 + ((g0 >> 3) & 1)) * BN * 4 + s_off[bn]);
#pragma unroll
      for (int e = 0; e < NG; ++e) {
        const int grp = g0 + e;
        const uint32_t d = (sw >> (16 * ((s_par[bn] + (uint32_t)grp) & 1))) & 0xFFFFu;
        const uint32_t z = (zw >> (4 * (grp & 7))) & 0xFu;
        r.off[e][bn] = __builtin_bit_cast(half2_t, 0xD400E400u + z + (z << 20));     // (-1024 - z, -64 - z)
        const bool none = (d & 0x7FFFu) == 0;         // a scale of zero: its weights are zeros
        r.d[bn] = e ? r.d[bn] | d << 16 : d;
        r.mask[bn] = none ? 0u : pc.mask;
        r.off[e][bn] = none ? half2_t{} : r.off[e][bn];
      }
    }
  };
  auto dequant = [&](const BSet& r, int s, half8_t (&out)[BNB]) {
#pragma unroll
    for (int bn = 0; bn < BNB; ++bn) {
      const uint4 wv4 = r.wb[bn][s >> 2];
      const uint32_t w = (s & 3) == 0 ? wv4.x : (s & 3) == 1 ? wv4.y : (s & 3) == 2 ? wv4.z : wv4.w;
      const int e = NG > 1 ? s / QS : 0;
      // two groups: by the offset, which is zero nowhere else (another mask would take registers that 128 rows lack)
      const uint32_t mask = NG == 1 ? r.mask[bn] : __builtin_bit_cast(uint32_t, r.off[e][bn]) == 0 ? 0u : pc.mask;
      uint32_t q[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t u = __builtin_amdgcn_perm(w, pc.magic, pc.sel[j]) & mask;
        q[j] = __builtin_bit_cast(uint32_t, (half2_t)(__builtin_bit_cast(half2_t, u) + r.off[e][bn]));
      }
      out[bn] = __builtin_bit_cast(half8_t, make_uint4(q[0], q[1], q[2], q[3]));
    }
  };
  BSet rs[2];
  half8_t bq[BNB];
  float unit[BNB];                                    // what a one in the sums stands for
#pragma unroll
  for (int bn = 0; bn < BNB; ++bn) unit[bn] = 1.0f;
  // the sums in units of the next group's scale
  auto rescale = [&](const BSet& r, int e) {
#pragma unroll
    for (int bn = 0; bn < BNB; ++bn) {
      const float d = h2f((uint16_t)(r.d[bn] >> (16 * e)));
      const float next = d == 0.0f ? unit[bn] : d;
      const float ratio = unit[bn] * __builtin_amdgcn_rcpf(next);
      unit[bn] = next;
#pragma unroll
      for (int bm = 0; bm < BMB; ++bm)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[bm][bn][i] *= ratio;
    }
  };
  // Round P in stage P % ST: meet, then sub-steps of 16 channels.  Each sub-step's products run
  // while the next one's weights are unpacked; the copies of round P + ST - 1 go out after the
  // first sub-step, into the stage round P - 1 used; the last sub-step waits for the wave's
  // own copies of round P + 1 and prepares its weights.
  auto step = [&](int rnd, int st, const BSet& r, BSet& rn) {
    const int stn = (st + ST - 1) % ST, stp = (st + 1) % ST;
    __builtin_amdgcn_sched_barrier(0);
    tile_barrier();
    if (KG == 1 || kt0 + KG * rnd + kgrp < kt1) {
      const unsigned char* cur = ring_g + st * KG * kStage;
      {
        const int kt = kt0 + KG * rnd + kgrp;
        if (NG > 1 || KG * BK >= G || rnd == 0 || kt * BK / G != (kt - KG) * BK / G) rescale(r, 0);
        if constexpr (G == 32 && KG == 1) __builtin_amdgcn_sched_barrier(0);   // else 128 rows lack 5 registers
      }
      half8_t af[BMB];
#pragma unroll
      for (int bm = 0; bm < BMB; ++bm) af[bm] = *reinterpret_cast<const half8_t*>(cur + a_base[bm]);
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        if (NG > 1 && s == QS) rescale(r, 1);
        half8_t bqn[BNB];
        if (s < NS - 1) {
          dequant(r, s + 1, bqn);
        } else {
          wait_copies<kCopies * (ST - 2)>();
          prep(rnd + 1, stp, rn);
          dequant(rn, 0, bqn);
        }
#pragma unroll
        for (int bm = 0; bm < BMB; ++bm) {
#pragma unroll
          for (int bn = 0; bn < BNB; ++bn)
            acc[bm][bn] = __builtin_amdgcn_mfma_f32_32x32x16_f16(af[bm], bq[bn], acc[bm][bn], 0, 0, 0);
          if (s < NS - 1) af[bm] = *reinterpret_cast<const half8_t*>(cur + (a_base[bm] ^ (uint32_t)(16 * ((s + 1) + ((s + 1) & QS)))));
        }
        if (s == 0) load(rnd + ST - 1, stn);
#pragma unroll
        for (int bn = 0; bn < BNB; ++bn) bq[bn] = bqn[bn];
      }
    } else {                                          // the second K group's share of an odd last round
      load(rnd + ST - 1, stn);
      wait_copies<kCopies * (ST - 2)>();
      prep(rnd + 1, stp, rn);
      dequant(rn, 0, bq);
    }
  };
#pragma unroll
  for (int i = 0; i < ST - 1; ++i) load(i, i);
  wait_copies<kCopies * (ST - 2)>();
  prep(0, 0, rs[0]);
  dequant(rs[0], 0, bq);
  int rp = 0;
  for (; rp + ST <= nr; rp += ST) {
#pragma unroll
    for (int i = 0; i < ST; ++i) step(rp + i, i, rs[i & 1], rs[1 - (i & 1)]);
    if (ST & 1) rs[0] = rs[1];
  }
#pragma unroll
  for (int i = 0; i < ST - 1; ++i)
    if (rp + i < nr) step(rp + i, i, rs[i & 1], rs[1 - (i & 1)]);
  wait_copies<0>();                                   // the look-ahead has landed before the LDS is used again
  tile_barrier();
#pragma unroll
  for (int bm = 0; bm < BMB; ++bm)
#pragma unroll
    for (int bn = 0; bn < BNB; ++bn)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[bm][bn][i] *= unit[bn];

  // ---- epilogue: value i of lane l in block (bm, bn) is row 8 (i / 4) + 4 (l / 32) + i % 4, column l % 32.
  const int outs = a.gated ? 32 : 64;                 // outputs of the wave
  const int64_t wcol = col0 + wv * outs;
  if (KG == 1 && a.ks > 1) {                          // a slice's sums, [slice][row][pitch]: columns in output order
    const int64_t np = (a.n + 3) & ~3ll, pitch = a.gated ? 2 * np : np;
    float* dst = a.part + ((int64_t)p.sl * a.rows + p.row0) * pitch;
#pragma unroll
    for (int bm = 0; bm < BMB; ++bm)
#pragma unroll
      for (int bn = 0; bn < BNB; ++bn)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int row = bm * 32 + 8 * (i / 4) + 4 * bc + (i % 4);
          const int64_t o = wcol + (a.gated ? bj : bn * 32 + bj);
          if (row < p.rows && o < a.n) dst[row * pitch + (a.gated && bn ? np : 0) + o] = acc[bm][bn][i];
        }
    return;
  }
  auto al = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; };
  const bool vec = a.n % 8 == 0 && al(a.y) && al(a.res);
  const uint16_t* bias = a.bias ? a.bias + (int64_t)p.expert * a.nw : nullptr;
  const int lsh = a.gated ? 2 : 3;                    // 4 or 8 lanes to a row
  const int c8 = (lane & ((1 << lsh) - 1)) * 8;
  const int64_t o = wcol + c8;
  float bv[8], bu[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int64_t oj = o + j < a.n ? o + j : a.n - 1;
    bv[j] = bias ? act_bits(bias[oj], a.bf) : 0.0f;
    bu[j] = bias && a.gated ? act_bits(bias[a.n + oj], a.bf) : 0.0f;
  }
  // ---- two K groups: each finishes 16 rows of every 32 and hands the sums of the others over
  // through LDS.  The staging below lies behind that area, or within the part that only the
  // wave itself reads.
  constexpr int ROWS = KG == 2 ? 16 : 32, NV = ROWS / 2;   // rows and values of a block that a wave finishes
  const int row_g = KG == 2 ? 16 * kgrp : 0;
  constexpr int kMine = BMB * BNB * 8 * 64;           // floats handed to a wave
  if constexpr (KG == 2) {
    float* hand = reinterpret_cast<float*>(ring) + (wv * 2 + (1 - kgrp)) * kMine;
#pragma unroll
    for (int bm = 0; bm < BMB; ++bm)
#pragma unroll
      for (int bn = 0; bn < BNB; ++bn)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float give[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float l = acc[bm][bn][4 * q + j], h = acc[bm][bn][8 + 4 * q + j];
            give[j] = kgrp ? l : h;
            acc[bm][bn][4 * q + j] = kgrp ? h : l;
          }
          *reinterpret_cast<float4*>(hand + (((bm * BNB + bn) * 2 + q) * 64 + lane) * 4) =
              make_float4(give[0], give[1], give[2], give[3]);
        }
    __syncthreads();
    hand = reinterpret_cast<float*>(ring) + (wv * 2 + kgrp) * kMine;
#pragma unroll
    for (int bm = 0; bm < BMB; ++bm)
#pragma unroll
      for (int bn = 0; bn < BNB; ++bn)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float4 v = *reinterpret_cast<const float4*>(hand + (((bm * BNB + bn) * 2 + q) * 64 + lane) * 4);
          acc[bm][bn][4 * q] += v.x;
          acc[bm][bn][4 * q + 1] += v.y;
          acc[bm][bn][4 * q + 2] += v.z;
          acc[bm][bn][4 * q + 3] += v.w;
        }
  }

  // ---- 32 rows at a time through the wave's own LDS: fp32, 8 neighbouring outputs to a lane
  constexpr int ER = 68;                              // floats of a staged row: two lane halves 16 banks apart
  constexpr int kHand = KG == 2 ? 8 * kMine : 0;
  constexpr bool kBehind = (kHand + 4 * KG * ROWS * ER) * 4 <= (int)sizeof(ring);
  static_assert(kCopies * (ST - 1) < 64, "the wait counter");
  static_assert(kBehind || ROWS * ER <= kMine, "else within the part that only the wave reads");
  float* ep = reinterpret_cast<float*>(ring) +
              (kBehind ? kHand + wave * ROWS * ER : (wv * 2 + kgrp) * kMine);
  constexpr int IT = ROWS / 8;                        // turns of a block, not gated
#pragma unroll
  for (int bm = 0; bm < BMB; ++bm) {
    const int first = bm * 32 + row_g;
    uint32_t rv[IT][4] = {};
    if (vec && a.res) {                               // a block's residual in flight together
#pragma unroll
      for (int t = 0; t < IT; ++t) {
        const int row = first + t * (64 >> lsh) + (lane >> lsh);
        if (t < ROWS >> (6 - lsh) && row < p.rows && o < a.n) {
          const uint4 r = *reinterpret_cast<const uint4*>(a.res + (int64_t)(p.row0 + row) * a.n + o);
          rv[t][0] = r.x; rv[t][1] = r.y; rv[t][2] = r.z; rv[t][3] = r.w;
        }
      }
    }
#pragma unroll
    for (int bn = 0; bn < BNB; ++bn)
#pragma unroll
      for (int i = 0; i < NV; ++i) ep[(8 * (i / 4) + 4 * bc + (i % 4)) * ER + bn * 32 + bj] = acc[bm][bn][i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll 1
    for (int t = 0; t < ROWS >> (6 - lsh); ++t) {
      const int row = t * (64 >> lsh) + (lane >> lsh);
      if (first + row < p.rows && o < a.n) {
        const float4 lo = *reinterpret_cast<const float4*>(ep + row * ER + c8);
        const float4 hi = *reinterpret_cast<const float4*>(ep + row * ER + c8 + 4);
        float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = activate(v[j] + bv[j], a.act);
        if (a.gated) {
          const float4 ul = *reinterpret_cast<const float4*>(ep + row * ER + 32 + c8);
          const float4 uh = *reinterpret_cast<const float4*>(ep + row * ER + 32 + c8 + 4);
          const float u[8] = {ul.x, ul.y, ul.z, ul.w, uh.x, uh.y, uh.z, uh.w};
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] *= u[j] + bu[j];
        }
        const int64_t at = (int64_t)(p.row0 + first + row) * a.n + o;
        if (vec) {
          if (a.res) {
            uint32_t ru[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              ru[q] = rv[0][q];
#pragma unroll
              for (int i = 1; i < IT; ++i) ru[q] = t == i ? rv[i][q] : ru[q];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += act_bits((uint16_t)(j & 1 ? ru[j / 2] >> 16 : ru[j / 2]), a.bf);
          }
          uint32_t u[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            u[j] = (uint32_t)f2act(v[2 * j], a.bf != 0) | (uint32_t)f2act(v[2 * j + 1], a.bf != 0) << 16;
          *reinterpret_cast<uint4*>(a.y + at) = make_uint4(u[0], u[1], u[2], u[3]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (o + j < a.n) {
              if (a.res) v[j] += act_bits(a.res[at + j], a.bf);
              a.y[at + j] = f2act(v[j], a.bf != 0);
            }
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

// Sums the K slices of one matrix in slice order and finishes the outputs: a thread takes 4 of a row.
__global__ __launch_bounds__(256) void linear_act_join_kernel(const ActArgs a) {
  const int64_t np = (a.n + 3) & ~3ll, pitch = a.gated ? 2 * np : np;
  const int64_t quads = np / 4;
  const int64_t unit = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = unit / quads;
  if (row >= a.rows) return;
  const int64_t o = (unit - row * quads) * 4;
  float v[4] = {0, 0, 0, 0}, u[4] = {0, 0, 0, 0};
  for (int s = 0; s < a.ks; ++s) {
    const float* src = a.part + ((int64_t)s * a.rows + row) * pitch + o;
    const float4 f = *reinterpret_cast<const float4*>(src);
    v[0] += f.x; v[1] += f.y; v[2] += f.z; v[3] += f.w;
    if (a.gated) {
      const float4 h = *reinterpret_cast<const float4*>(src + np);
      u[0] += h.x; u[1] += h.y; u[2] += h.z; u[3] += h.w;
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (o + j < a.n) {
      const int64_t at = row * a.n + o + j;
      float f = finish(a, 0, o + j, v[j], u[j]);
      if (a.res) f += act_bits(a.res[at], a.bf);
      a.y[at] = f2act(f, a.bf != 0);
    }
}

// x~ for the tile kernel: fp16(x), times inv_s rounded once, where x is bf16 or inv_s is given.
__global__ __launch_bounds__(256) void linear_act_prep_kernel(const ActArgs a, uint16_t* __restrict__ out) {
  const int64_t chunks = a.x_rows * (a.k / 8);
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= chunks) return;
  uint4 v = reinterpret_cast<const uint4*>(a.x)[i];
  v = act8_h(v, a.bf != 0);
  if (a.inv) {
    const uint4 iv = reinterpret_cast<const uint4*>(a.inv)[i % (a.k / 8)];
    v = __builtin_bit_cast(uint4, (half8_t)(__builtin_bit_cast(half8_t, v) * __builtin_bit_cast(half8_t, iv)));
  }
  reinterpret_cast<uint4*>(out)[i] = v;
}

// ---------------------------------------------------------------- plan
//
// Chosen by the sizes the host knows; the rows of an expert are taken as their mean.
// Microseconds of both sides near the borders (captured, weights cold):
//   streaming or tiles, one matrix: past 16 rows streaming reads and unpacks the weights again for every 16,
//     which pays up to 36 MiB of weights in all, unless short rows (k) make that many units: fewer than 2^16
//     weight rows in all.  4096 <- 4096, 17 / 64 / 96 / 128 rows (16 / 32 / 48 / 64 MiB) 11.2 / 15.4 / 19.7 / 25.3
//     against 16.4 / 18.8 / 20.5 / 21.5; 1024 <- 4096, 256 / 512 rows (32 / 64) 15.3 / 25.4 against 18.3 / 21.2;
//     512 <- 4096, 512 rows (32) 15.7 against 18.4; 1024 <- 2048, 512 rows (32) 16.1 against 17.7; 4096 <- 1024,
//     192 / 256 rows (24 / 32) 13.0 / 18.2 against 16.1 / 16.7; 4096 <- 512, 192 / 256 / 384 rows (12 / 16 / 24)
//     11.3 / 12.1 / 14.5 against 13.9 / 13.5 / 11.2.  28672 <- 4096 (56 MiB a time): 16 rows streamed 28, 17 rows
//     by tiles 28 (streamed 38).
//   streaming or tiles, experts, by their mean of rows: 8 of 14336 x 2 <- 4096, 6 / 7 rows 125 / 138 against 130;
//     8 of 4096 <- 14336, 6 / 7 rows 75 / 79 against 120; 128 of 1024 x 2 <- 2048, 3 / 5 / 7 rows 69 / 84 / 97
//     against 76 / 79 / 82; 128 of 2048 <- 1024, 5 / 7 rows 44 / 51 against 44 / 46; 60 of 2048 <- 1408 (g = 64),
//     3 / 6 rows 35 / 46 against 32 / 34: the border is at 6.
//   tiles of 32, 64, 128 rows, by the K-steps that 128-row tiles would take in all: 4096 x 4096, 96 rows (1024)
//     21 / 24 / 28, 256 rows (2048) 27 / 28 / 29; 4096 <- 14336, 96 rows (3584) 33 / 37 / 36; 4096 <- 4096,
//     520 rows (5120) 51 / 50 / 43, 1024 rows (8192) 59 / 55 / 56.
//   K-steps of 128 or 64 in 32-row tiles: 8 experts of 14336 x 2 <- 4096, 16 rows each 143 against 170.
//   K slices: a matrix of few tiles is split until 256 work-groups have one (a join follows, of 34 MB of
//     sums at most); two K groups in a work-group where that leaves at most one to a CU.  Split against not:
//     4096 <- 14336, 1024 rows (128 tiles) 150 against 228; 4096 <- 4096, 520 / 1024 rows 44 / 56 against
//     65 / 65; 1024 <- 4096, 2048 rows 37 against 64.
struct ActPlan {
  bool stream;
  int tm, waves, per;          // stream: rows of a tile, waves, blocks of a wave
  int bm, bk, kg, ks;          // tile: rows, K-step, K groups, K slices
  bool prep;
  int64_t ncol, units;         // column blocks; upper bound of the units
  size_t x_bytes, part_bytes;
};

static size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

static ActPlan act_plan(const ActArgs& a) {
  ActPlan p{};
  const int64_t active = a.offsets ? (a.e < a.rows ? a.e : a.rows) : 1;
  const int64_t avg = a.offsets ? (a.rows + a.e - 1) / a.e : a.rows;
  auto tiles = [&](int rows) { return a.offsets ? a.rows / rows + active : (a.rows + rows - 1) / rows; };
  const int64_t bytes = a.nw * (a.k / 2);              // packed weights of a matrix
  p.ks = 1;
  p.kg = 1;
  // streaming, unless that takes more units than a launch holds
  const int sm = avg <= 8 ? 8 : 16, s_outs = (a.gated ? kCB / 2 : kCB) * 16;
  const int64_t s_cols = (a.n + s_outs - 1) / s_outs, s_units = tiles(sm) * s_cols;
  const int64_t passes = (avg + 15) / 16;
  const bool again = avg <= 512 && passes * bytes <= (36 << 20) && passes * a.nw < (1 << 16);
  if ((a.offsets ? avg <= 6 : avg <= 16 || again) && s_units < kMaxUnits) {
    p.stream = true;
    p.tm = sm;
    const int nb = (int)((a.k + 127) / 128), runs = (nb + kRun - 1) / kRun;
    p.per = (runs + 3) / 4 * kRun;                     // whole runs, up to 4 waves
    p.waves = (nb + p.per - 1) / p.per;
    p.ncol = s_cols;
    p.units = s_units;
    return p;
  }
  const int outs = a.gated ? 128 : 256;
  p.ncol = (a.n + outs - 1) / outs;
  const int nk = (int)(a.k / 64);
  const int64_t steps = tiles(128) * p.ncol * nk;
  p.bm = avg <= 32 || steps <= 1024 ? 32 : avg <= 64 || steps <= 3000 ? 64 : 128;
  p.bk = p.bm == 32 && a.g >= 64 && a.k % 128 == 0 ? 128 : 64;
  const int64_t t = tiles(p.bm) * p.ncol;
  if (!a.offsets && t < 256) {
    int64_t ks = 256 / t;
    ks = ks > 16 ? 16 : ks;
    ks = ks > nk / 2 ? nk / 2 : ks;                    // two K-steps of 64 to a slice
    p.ks = ks < 1 ? 1 : (int)ks;
  }
  if (p.ks == 1 && t <= 256) p.kg = 2;
  p.units = t * p.ks;
  p.prep = a.bf || a.inv;
  if (p.prep) p.x_bytes = up256((size_t)a.x_rows * a.k * 2);
  if (p.ks > 1) {
    const int64_t np = (a.n + 3) & ~3ll;
    p.part_bytes = up256((size_t)p.ks * a.rows * (a.gated ? 2 * np : np) * 4);
  }
  return p;
}

size_t linear_act_scratch_bytes(const ActArgs& a) {
  const ActPlan p = act_plan(a);
  return p.x_bytes + p.part_bytes;
}

bool linear_act_fits(const ActArgs& a) {
  return act_plan(a).units < kMaxUnits && a.x_rows * (a.k / 8) <= (1ll << 31) && a.rows * ((a.n + 3) / 4) <= (1ll << 31);
}

template <int G, int TM>
static hipError_t run_stream(const ActArgs& a, const ActPlan& p, hipStream_t stream) {
  const size_t x = (size_t)p.waves * StreamLds<TM>::WAVE, red = (size_t)p.waves * kCB * 1024;
  const size_t lds = x > red ? x : red;                // 33 KB at most
  const dim3 grid((unsigned)((p.units + 7) / 8 * 8)), block(p.waves * 64);
  if constexpr (G == 128) {
    if (a.ng % 4 == 0) {
      hipLaunchKernelGGL((linear_act_stream_kernel<G, TM, true>), grid, block, lds, stream, a);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((linear_act_stream_kernel<G, TM, false>), grid, block, lds, stream, a);
  return hipGetLastError();
}

template <int G, int BM, int BK>
static hipError_t run_tile(const ActArgs& a, const ActPlan& p, hipStream_t stream) {
  const dim3 grid((unsigned)((p.units + 7) / 8 * 8));
  if (p.kg == 2) hipLaunchKernelGGL((linear_act_tile_kernel<G, 2, BM, BK>), grid, dim3(512), 0, stream, a);
  else hipLaunchKernelGGL((linear_act_tile_kernel<G, 1, BM, BK>), grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

template <int G>
static hipError_t run_act(const ActArgs& a, const ActPlan& p, hipStream_t stream) {
  if (p.stream) return p.tm == 8 ? run_stream<G, 8>(a, p, stream) : run_stream<G, 16>(a, p, stream);
  if constexpr (G >= 64) {
    if (p.bk == 128) return run_tile<G, 32, 128>(a, p, stream);
  }
  if (p.bm == 32) return run_tile<G, 32, 64>(a, p, stream);
  return p.bm == 64 ? run_tile<G, 64, 64>(a, p, stream) : run_tile<G, 128, 64>(a, p, stream);
}

hipError_t launch_linear_act(const ActArgs& args, void* scratch, hipStream_t stream) {
  ActArgs a = args;
  const ActPlan p = act_plan(a);
  a.ng = (int32_t)(a.k / a.g);
  a.nzw = (a.ng + 7) / 8;
  a.ncol = (int32_t)p.ncol;
  a.ks = p.ks;
  a.per = p.per;
  a.topk_inv = (uint32_t)(((1ull << 32) + a.topk - 1) / a.topk);   // (not read for 1)
  char* base = (char*)scratch;
  if (p.prep) {
    uint16_t* xt = (uint16_t*)base;
    const int64_t chunks = a.x_rows * (a.k / 8);
    hipLaunchKernelGGL(linear_act_prep_kernel, dim3((unsigned)((chunks + 255) / 256)), dim3(256), 0, stream, a, xt);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    a.x = xt;
  }
  a.part = (float*)(base + p.x_bytes);
  const hipError_t e = a.g == 128 ? run_act<128>(a, p, stream) : a.g == 64 ? run_act<64>(a, p, stream) : run_act<32>(a, p, stream);
  if (e != hipSuccess || p.ks == 1) return e;
  const int64_t quads = ((a.n + 3) / 4) * a.rows;
  hipLaunchKernelGGL(linear_act_join_kernel, dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace awq
