// Causal attention of new tokens over the 8-bit paged KV cache.
//
// Row i of a sequence's n new rows stands at position ctx - n + i and sees the
// positions 0 .. ctx - n + i.  For query head hq of key/value head h:
//   s_t = scale * ks(t) * (q . kcode_t),   o = sum_t softmax(s)_t vs(t) vcode_t,
//   lse = log sum_t exp(s_t).
//
// All kernels run the transposed products, S^T = K Q^T and O^T = V^T P^T, so a
// lane owns one (row, query head) pair ("column") throughout: its softmax
// statistics, its rescaling factor and its mask are per-lane scalars.  The
// group's query heads are further columns of the same key/value head: column
// c of a sequence is row c / G, query head h * G + c % G.
//
// One pass with a running maximum.  The page's value scale goes into the
// exponent: p' = exp2(s + log2 vs - m) <= 2^kLazy, O = sum p' vcode in units
// of 1, l = sum p' / vs.  So p' carries exactly the weight of its token's
// contribution to O whatever the scales are, and fp16 (11 bits) holds it with a
// relative rounding of 2^-12 to 2^-11; S, O, m and l are fp32.  m moves only when a
// score exceeds it by 2^kLazy (a wave-wide vote), so most steps neither
// exchange maxima between lanes nor rescale O.
#include "awq_internal.h"
#include "kv8_common.h"

namespace awq {
namespace {

constexpr int kStep = 64;            // tokens of one step (a page holds whole steps)
constexpr float kLazy = 8.0f;        // p' <= 2^8: far inside fp16
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kNone = -1e30f;      // running maximum before any visible token

struct AttnP {
  Kv8View v;
  const uint16_t* q;
  uint16_t* out;
  float* lse;                        // [rows][hq] or null
  int64_t q_stride, out_stride;
  int32_t hq, G;
  float scale2;                      // softmax scale * log2 e
  int32_t target;                    // units per head the plan aims at
  int32_t min_steps;                 // least steps of a unit
  int32_t slots;                     // partial slots per head in the workspace
  float* part;                       // partial O [slot][hkv][TC][D], then their (m, l)
  float* part_ml;
};

// The part of the work one work-group does: steps s of S of tile `tile` of
// sequence `b`.
struct Unit {
  int b, tile, s, S, slot;
  SeqRows r;
};

// The plan, computed by every wave from the device's own lengths (a captured
// graph replays with new ones): tiles of TC columns; a sequence's tiles are cut
// into S = ceil(steps / chunk) units, chunk = total steps over the target.
// Units of sequences with S > 1 have partial slots, numbered in the same
// order; there are fewer than 2 * target of them, as S > 1 needs
// steps > chunk and then ceil(steps / chunk) < 2 steps / chunk.
// TILE_ONLY: unit numbers count tiles (the pass that joins partials).
template <int TC, bool TILE_ONLY>
__device__ __forceinline__ bool find_unit(const AttnP& p, int u, int lane, Unit& w) {
  const Kv8View& v = p.v;
  const int cap = (int)(((int64_t)v.max_pages << v.shift) / kStep);
  auto load = [&](int i, SeqRows& r, int& tiles, int& steps) {
    r = SeqRows{0, 0, 0};
    tiles = steps = 0;
    if (i < v.b) {
      r = seq_rows(v, i);
      tiles = (int)(((int64_t)r.n * p.G + TC - 1) / TC);
      steps = r.ctx / kStep + (r.ctx % kStep ? 1 : 0);
      steps = steps < cap ? steps : cap;
    }
  };
  SeqRows r;
  int tiles, steps;
  uint64_t total = 0;
  for (int i0 = 0; i0 < v.b; i0 += 64) {
    load(i0 + lane, r, tiles, steps);
    total += (uint64_t)tiles * steps;
  }
  if (v.b > 1) {
#pragma unroll
    for (int o = 32; o; o >>= 1) total += __shfl_xor(total, o, 64);
  } else {
    total = __shfl(total, 0, 64);
  }
  const uint64_t per = (total + p.target - 1) / (uint64_t)p.target;
  const int chunk = per > (uint64_t)p.min_steps ? (per < 0x40000000u ? (int)per : 0x40000000) : p.min_steps;
  int before = 0, slots = 0;
  for (int i0 = 0; i0 < v.b; i0 += 64) {
    if (v.b > 64) load(i0 + lane, r, tiles, steps);
    int S = (steps + chunk - 1) / chunk;
    S = S < 1 ? 1 : S;
    const int mine = TILE_ONLY ? tiles : tiles * S;
    const int held = S > 1 ? tiles * S : 0;
    int incl = mine, hincl = held;
    if (v.b > 1) {
      incl = wave_scan(mine, lane);
      hincl = wave_scan(held, lane);
    }
    const int all = v.b > 1 ? __shfl(incl, 63, 64) : __shfl(incl, 0, 64);
    if (u - before < all) {
      const uint64_t past = __ballot(incl <= u - before);
      int l = v.b > 1 ? __popcll(past) : 0;
      l = l < 63 ? l : 63;
      const int at = u - before - __shfl(incl - mine, l, 64);
      w.b = i0 + l;
      w.S = __shfl(S, l, 64);
      w.r.r0 = __shfl(r.r0, l, 64);
      w.r.n = __shfl(r.n, l, 64);
      w.r.ctx = __shfl(r.ctx, l, 64);
      const int nt = __shfl(tiles, l, 64);
      const int order = TILE_ONLY ? at : at / w.S;
      w.s = TILE_ONLY ? 0 : at % w.S;
      w.tile = nt - 1 - order;               // later rows see more: the longest first
      w.slot = slots + __shfl(hincl - held, l, 64) + order * w.S + w.s;
      // always so for ascending cu; whatever else the array holds stays in bounds
      const int top = w.S > 1 ? (TILE_ONLY ? w.slot + w.S : w.slot + 1) : 0;
      return w.tile >= 0 && w.tile < nt && w.slot >= 0 && top <= p.slots;
    }
    before += all;
    slots += v.b > 1 ? __shfl(hincl, 63, 64) : 0;
  }
  return false;
}

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// One 16-column tile, four waves taking steps in turn, each wave on its own
// from cache to registers: no LDS and no barrier until the waves' results are
// joined.  MFMA 16x16x32: lane (c = l % 16, g = l / 16) holds column c and the
// 16 tokens 16 g .. 16 g + 15 of a step, so that its V operand is one 16-byte
// load per 16 channels and its K operand two, one per 64 channels:
//   score tile t, A row r   = token 16 (r / 4) + 4 t + r % 4 (the rows of an MFMA
//                             may be any tokens), so result i of lane group g
//                             is token 16 g + 4 t + i;
//   score k-step 2 x + e    = channels 64 x + 16 g + 8 e .. + 7;
//   output k-step e         = tokens 16 g + 8 e .. + 7.
template <int D, bool BF>
__global__ __launch_bounds__(256, 2) void attn_kv8_cols_kernel(AttnP p) {
  typedef Mma<BF> MQ;
  typedef Mma<false> MV;
  constexpr int TC = 16, NX = D / 64, ND = D / 16;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int h = blockIdx.x % p.v.hkv;
  Unit w;
  if (!find_unit<TC, false>(p, blockIdx.x / p.v.hkv, lane, w)) return;
  const Kv8View& v = p.v;
  const int b = uniform(w.b), S = uniform(w.S), sidx = uniform(w.s), tile = uniform(w.tile);
  const int n = uniform(w.r.n), r0 = uniform(w.r.r0), ctx = uniform(w.r.ctx);
  const int G = p.G, cols = n * G - tile * TC < TC ? n * G - tile * TC : TC;
  const int c = lane & 15, g = lane >> 4;
  const int col = tile * TC + c;
  // position of this lane's column (-1: sees nothing); of the tile's first and last
  const int pos = c < cols ? ctx - n + col / G : -1;
  const int first = ctx - n + (tile * TC) / G, last = ctx - n + (tile * TC + cols - 1) / G;
  const int64_t cap = (int64_t)v.max_pages << v.shift;
  const bool over = ctx > cap;               // longer than its row of the block table: NaN
  int steps = last < 0 ? 0 : last / kStep + 1;
  if (steps > (int)(cap / kStep)) steps = (int)(cap / kStep);
  const int st0 = (int)((int64_t)steps * sidx / S), st1 = (int)((int64_t)steps * (sidx + 1) / S);

  typename MQ::frag qf[NX][2];
  {
    const int cc = c < cols ? col : tile * TC;
    const uint16_t* qp = p.q + (int64_t)(r0 + cc / G) * p.q_stride + (int64_t)(h * G + cc % G) * D;
#pragma unroll
    for (int x = 0; x < NX; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        qf[x][e] = __builtin_bit_cast(typename MQ::frag, *(const uint4*)(qp + 64 * x + 16 * g + 8 * e));
  }
  floatx4_t o[ND];
#pragma unroll
  for (int i = 0; i < ND; ++i) o[i] = floatx4_t{0, 0, 0, 0};
  float m = kNone, l = 0.0f;

  const int krow = 16 * (c >> 2) + (c & 3);      // + 4 t
  for (int st = st0 + wave; st < st1; st += 4) {
    const int t0 = st * kStep;
    int pid = uniform(v.bt[(int64_t)b * v.max_pages + (t0 >> v.shift)]);
    const bool bad = over || (uint32_t)pid >= (uint64_t)v.pages;
    pid = bad ? 0 : pid;
    const int64_t ph = (int64_t)pid * v.hkv + h;
    const int slot0 = t0 & ((1 << v.shift) - 1);
    const uint8_t* kp = v.kc + ((ph << v.shift) + slot0) * D;
    const uint8_t* vp = v.vc + ((ph * D) << v.shift) + slot0;
    const float ks = bad ? __builtin_nanf("") : v.ks[ph] * p.scale2;
    const float vs = v.vs[ph];
    uint4 kr[4][NX], vr[ND];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int x = 0; x < NX; ++x) kr[t][x] = *(const uint4*)(kp + (krow + 4 * t) * D + 64 * x + 16 * g);
#pragma unroll
    for (int i = 0; i < ND; ++i) vr[i] = *(const uint4*)(vp + ((16 * i + c) << v.shift) + 16 * g);

    floatx4_t s[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      s[t] = floatx4_t{0, 0, 0, 0};
#pragma unroll
      for (int x = 0; x < NX; ++x) {
        s[t] = MQ::mma16(MQ::from_fp8(kr[t][x].x, kr[t][x].y), qf[x][0], s[t]);
        s[t] = MQ::mma16(MQ::from_fp8(kr[t][x].z, kr[t][x].w), qf[x][1], s[t]);
      }
    }
    const float lv = __builtin_amdgcn_logf(vs), rv = 1.0f / vs;
    const int tok = t0 + 16 * g;
    float mx = -__builtin_inff();
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[t][i] = __builtin_fmaf(s[t][i], ks, lv);
    if (t0 + kStep - 1 > first || cols < TC) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[t][i] = tok + 4 * t + i <= pos ? s[t][i] : -__builtin_inff();
    }
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) mx = __builtin_fmaxf(mx, s[t][i]);
    if (__ballot(mx > m + kLazy)) {
      mx = __builtin_fmaxf(mx, __shfl_xor(mx, 16, 64));
      mx = __builtin_fmaxf(mx, __shfl_xor(mx, 32, 64));
      const float mn = __builtin_fmaxf(m, mx);
      const float f = __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      l *= f;
#pragma unroll
      for (int i = 0; i < ND; ++i) o[i] *= f;
    }
    float sum = 0.0f;
    half8_t pf[2];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float e = __builtin_amdgcn_exp2f(s[t][i] - m);
        sum += e;
        pf[t >> 1][4 * (t & 1) + i] = (half_t)e;
      }
    l = __builtin_fmaf(sum, rv, l);
    // slots behind the sequence's end, and the page read in place of one that is
    // not in the cache, may hold anything, NaN codes too: 0 * NaN
    const int held = bad ? 0 : ctx;
    if (t0 + kStep > held) {
#pragma unroll
      for (int i = 0; i < ND; ++i) {
        uint32_t* x = (uint32_t*)&vr[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int left = held - (tok + 4 * j);
          x[j] &= left >= 4 ? ~0u : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < ND; ++i) {
      o[i] = MV::mma16(MV::from_fp8(vr[i].x, vr[i].y), pf[0], o[i]);
      o[i] = MV::mma16(MV::from_fp8(vr[i].z, vr[i].w), pf[1], o[i]);
    }
  }
  l += __shfl_xor(l, 16, 64);
  l += __shfl_xor(l, 32, 64);

  // join the waves: O [wave][channel][column], m and l per column
  __shared__ float so[4][D][TC + 1];
  __shared__ float sm[4][TC], sl[4][TC];
#pragma unroll
  for (int i = 0; i < ND; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) so[wave][16 * i + 4 * g + j][c] = o[i][j];
  if (g == 0) {
    sm[wave][c] = m;
    sl[wave][c] = l;
  }
  __syncthreads();
  // thread: column t / 16, channels (t % 16) + 16 x
  const int jc = threadIdx.x >> 4;
  if (jc >= cols) return;
  float top = kNone, sum = 0.0f, f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) top = __builtin_fmaxf(top, sm[i][jc]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = __builtin_amdgcn_exp2f(sm[i][jc] - top);
    sum += f[i] * sl[i][jc];
  }
  const int d0 = threadIdx.x & 15;
  const int jcol = tile * TC + jc;
  if (S == 1) {
    const int row = r0 + jcol / G, head = h * G + jcol % G;
    // no visible token: zeros and lse = -inf (a NaN sum is kept)
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint16_t* op = p.out + row * p.out_stride + (int64_t)head * D;
#pragma unroll
    for (int i = 0; i < ND; ++i) {
      const int d = d0 + 16 * i;
      float a = 0.0f;
#pragma unroll
      for (int x = 0; x < 4; ++x) a += f[x] * so[x][d][jc];
      op[d] = f2act(a * inv, BF);
    }
    if (p.lse && d0 == 0)
      p.lse[(int64_t)row * p.hq + head] =
          sum == 0.0f ? -__builtin_inff() : (top + __builtin_amdgcn_logf(sum)) * kLn2;
  } else {
    const int64_t at = ((int64_t)w.slot * v.hkv + h) * TC + jc;
    float* op = p.part + at * D;
#pragma unroll
    for (int i = 0; i < ND; ++i) {
      const int d = d0 + 16 * i;
      float a = 0.0f;
#pragma unroll
      for (int x = 0; x < 4; ++x) a += f[x] * so[x][d][jc];
      op[d] = a;
    }
    if (d0 == 0) {
      p.part_ml[2 * at] = top;
      p.part_ml[2 * at + 1] = sum;
    }
  }
}

// The state of one wave's 32 columns, and its steps st, st + stride, ... < st1:
// MFMA 32x32x16, lane (c = l % 32, half = l / 32) holds column c and, of each
// step's two 32-token tiles t, the tokens 32 t + 16 half .. + 15:
//   score tile t, A row r = token 32 t + 16 (r / 4 % 2) + 4 (r / 8) + r % 4, so result i
//                           of a half is token 32 t + 16 half + i;
//   score k-step 2 x + e  = channels 32 x + 16 half + 8 e .. + 7;
//   output k-step 2 t + e = tokens 32 t + 16 half + 8 e .. + 7.
// The next step's keys are asked for as soon as this step's scores have used
// theirs, and its values while those scores run, so a load has half a step to
// arrive.
template <int D, bool BF>
struct Wave32 {
  typedef Mma<BF> MQ;
  typedef Mma<false> MV;
  static constexpr int NX = D / 32, ND = D / 32;
  typename MQ::frag qf[NX][2];
  floatx16_t o[ND];
  float m, l;

  __device__ __forceinline__ void load_q(const uint16_t* qp, int half) {
#pragma unroll
    for (int x = 0; x < NX; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        qf[x][e] = __builtin_bit_cast(typename MQ::frag, *(const uint4*)(qp + 32 * x + 16 * half + 8 * e));
  }

  // pos: the last position this lane's column sees; first: the least of them in
  // the wave (-1: some column sees nothing at all).
  __device__ __forceinline__ void run(const Kv8View& v, float scale2, int h, int b, int ctx, bool over, int pos,
                                      int first, int st, int st1, int stride, int lane) {
    const int c = lane & 31, half = lane >> 5;
    const int krow = 16 * (c >> 2 & 1) + 4 * (c >> 3) + (c & 3);
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) o[i][j] = 0.0f;
    m = kNone;
    l = 0.0f;
    if (st >= st1) return;
    const int32_t* bt = v.bt + (int64_t)b * v.max_pages;
    const int smask = (1 << v.shift) - 1;
    uint4 kr[2][NX], vr[ND][2];
    float ks, vs;
    bool bad;
    const uint8_t* vp;
    auto locate = [&](int s) {
      const int t0 = s * kStep;
      int pid = uniform(bt[t0 >> v.shift]);
      bad = over || (uint32_t)pid >= (uint64_t)v.pages;
      pid = bad ? 0 : pid;
      const int64_t ph = (int64_t)pid * v.hkv + h;
      const uint8_t* kp = v.kc + ((ph << v.shift) + (t0 & smask)) * D;
      vp = v.vc + ((ph * D) << v.shift) + (t0 & smask);
      ks = bad ? __builtin_nanf("") : v.ks[ph] * scale2;
      vs = v.vs[ph];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int x = 0; x < NX; ++x) kr[t][x] = *(const uint4*)(kp + (32 * t + krow) * D + 32 * x + 16 * half);
    };
    locate(st);
    for (; st < st1; st += stride) {
      const int t0 = st * kStep;
#pragma unroll
      for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int t = 0; t < 2; ++t)
          vr[i][t] = *(const uint4*)(vp + ((32 * i + c) << v.shift) + 32 * t + 16 * half);
      floatx16_t s[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int j = 0; j < 16; ++j) s[t][j] = 0.0f;
#pragma unroll
        for (int x = 0; x < NX; ++x) {
          s[t] = MQ::mma32(MQ::from_fp8(kr[t][x].x, kr[t][x].y), qf[x][0], s[t]);
          s[t] = MQ::mma32(MQ::from_fp8(kr[t][x].z, kr[t][x].w), qf[x][1], s[t]);
        }
      }
      float a = ks, z = __builtin_amdgcn_logf(vs);
      const float rv = 1.0f / vs;
      const int held = bad ? 0 : ctx;
      if (st + stride < st1) locate(st + stride);
      if (t0 + kStep - 1 > first || held == 0) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int j = 0; j < 16; ++j)
            s[t][j] = t0 + 32 * t + 16 * half + j <= pos ? __builtin_fmaf(s[t][j], a, z) : -__builtin_inff();
        a = 1.0f;
        z = 0.0f;
      }
      float mx = s[0][0];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < 16; ++j) mx = __builtin_fmaxf(mx, s[t][j]);
      mx = __builtin_fmaf(mx, a, z);
      if (__ballot(mx > m + kLazy)) {
        mx = __builtin_fmaxf(mx, __shfl_xor(mx, 32, 64));
        const float mn = __builtin_fmaxf(m, mx);
        const float f = __builtin_amdgcn_exp2f(m - mn);
        m = mn;
        l *= f;
#pragma unroll
        for (int i = 0; i < ND; ++i) o[i] *= f;
      }
      z -= m;
      float sum = 0.0f;
      half8_t pf[4];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][j], a, z));
          sum += e;
          pf[2 * t + (j >> 3)][j & 7] = (half_t)e;
        }
      l = __builtin_fmaf(sum, rv, l);
      // slots behind the sequence's end, and the page read in place of one that is
      // not in the cache, may hold anything, NaN codes too: 0 * NaN
      if (t0 + kStep > held) {
#pragma unroll
        for (int i = 0; i < ND; ++i)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            uint32_t* x = (uint32_t*)&vr[i][t];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int left = held - (t0 + 32 * t + 16 * half + 4 * j);
              x[j] &= left >= 4 ? ~0u : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
            }
          }
      }
#pragma unroll
      for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          o[i] = MV::mma32(MV::from_fp8(vr[i][t].x, vr[i][t].y), pf[2 * t], o[i]);
          o[i] = MV::mma32(MV::from_fp8(vr[i][t].z, vr[i][t].w), pf[2 * t + 1], o[i]);
        }
    }
    l += __shfl_xor(l, 32, 64);
  }
};

// Tiles of 128 columns: each of the four waves has 32 of them and walks all of
// the unit's steps.  The waves read the same pages within a short time of each
// other, so all but the first of these reads come from the CU's own cache.
template <int D, bool BF>
__global__ __launch_bounds__(256, 2) void attn_kv8_tile_kernel(AttnP p) {
  constexpr int TC = 128, ND = D / 32;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int h = blockIdx.x % p.v.hkv;
  Unit w;
  if (!find_unit<TC, false>(p, blockIdx.x / p.v.hkv, lane, w)) return;
  const Kv8View& v = p.v;
  const int b = uniform(w.b), S = uniform(w.S), sidx = uniform(w.s), tile = uniform(w.tile);
  const int n = uniform(w.r.n), r0 = uniform(w.r.r0), ctx = uniform(w.r.ctx);
  const int G = p.G, c0 = tile * TC + 32 * wave;
  const int cols = n * G - c0 < 32 ? n * G - c0 : 32;
  if (cols <= 0) return;
  const int c = lane & 31, half = lane >> 5, col = c0 + c;
  const int pos = c < cols ? ctx - n + col / G : -1;
  const int first = cols < 32 ? -1 : ctx - n + c0 / G;
  // the unit's share of the tile's steps; this wave stops at what its own rows see
  const int tcols = n * G - tile * TC < TC ? n * G - tile * TC : TC;
  const int last = ctx - n + (tile * TC + tcols - 1) / G, wlast = ctx - n + (c0 + cols - 1) / G;
  const int cap = (int)(((int64_t)v.max_pages << v.shift) / kStep);
  int steps = last < 0 ? 0 : last / kStep + 1, wsteps = wlast < 0 ? 0 : wlast / kStep + 1;
  steps = steps < cap ? steps : cap;
  const int st0 = (int)((int64_t)steps * sidx / S);
  int st1 = (int)((int64_t)steps * (sidx + 1) / S);
  st1 = st1 < wsteps ? st1 : wsteps;

  Wave32<D, BF> a;
  const int cc = c < cols ? col : c0;
  a.load_q(p.q + (int64_t)(r0 + cc / G) * p.q_stride + (int64_t)(h * G + cc % G) * D, half);
  a.run(v, p.scale2, h, b, ctx, ctx > (int64_t)v.max_pages << v.shift, pos, first, st0, st1, 1, lane);
  if (c >= cols) return;
  if (S == 1) {
    const int row = r0 + col / G, head = h * G + col % G;
    const float inv = a.l == 0.0f ? 0.0f : 1.0f / a.l;
    uint16_t* op = p.out + row * p.out_stride + (int64_t)head * D + 4 * half;
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t x[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          x[e] = (uint32_t)f2act(a.o[i][4 * j + 2 * e] * inv, BF) |
                 (uint32_t)f2act(a.o[i][4 * j + 2 * e + 1] * inv, BF) << 16;
        *(uint2*)(op + 32 * i + 8 * j) = make_uint2(x[0], x[1]);
      }
    if (p.lse && half == 0)
      p.lse[(int64_t)row * p.hq + head] =
          a.l == 0.0f ? -__builtin_inff() : (a.m + __builtin_amdgcn_logf(a.l)) * kLn2;
  } else {
    const int64_t at = ((int64_t)w.slot * v.hkv + h) * TC + 32 * wave + c;
    float* op = p.part + at * D + 4 * half;
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *(float4*)(op + 32 * i + 8 * j) =
            make_float4(a.o[i][4 * j], a.o[i][4 * j + 1], a.o[i][4 * j + 2], a.o[i][4 * j + 3]);
    if (half == 0) {
      p.part_ml[2 * at] = a.m;
      p.part_ml[2 * at + 1] = a.l;
    }
  }
}

// Joins the S partial results of every column of the split sequences: one wave
// per column, the lanes' channels in the order of the units (a fixed order).
template <int D, int TC, bool BF>
__global__ __launch_bounds__(256) void attn_kv8_join_kernel(AttnP p) {
  constexpr int V = D / 64;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int part = blockIdx.x % (p.v.hkv * (TC / 4));
  const int h = part % p.v.hkv, jc = (part / p.v.hkv) * 4 + wave;
  Unit w;
  if (!find_unit<TC, true>(p, blockIdx.x / (p.v.hkv * (TC / 4)), lane, w)) return;
  const int S = uniform(w.S), G = p.G, col = uniform(w.tile) * TC + jc;
  if (S == 1 || col >= uniform(w.r.n) * G) return;
  const int64_t at0 = ((int64_t)uniform(w.slot) * p.v.hkv + h) * TC + jc, stride = (int64_t)p.v.hkv * TC;
  float top = kNone;
  for (int i = lane; i < S; i += 64) top = __builtin_fmaxf(top, p.part_ml[2 * (at0 + i * stride)]);
#pragma unroll
  for (int o = 32; o; o >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, o, 64));
  float acc[V] = {}, sum = 0.0f;
#pragma unroll 8
  for (int i = 0; i < S; ++i) {
    const int64_t at = at0 + i * stride;
    const float f = __builtin_amdgcn_exp2f(p.part_ml[2 * at] - top);
    sum = __builtin_fmaf(f, p.part_ml[2 * at + 1], sum);
#pragma unroll
    for (int x = 0; x < V; ++x) acc[x] = __builtin_fmaf(f, p.part[at * D + lane * V + x], acc[x]);
  }
  const int row = uniform(w.r.r0) + col / G, head = h * G + col % G;
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  uint16_t* op = p.out + row * p.out_stride + (int64_t)head * D + lane * V;
#pragma unroll
  for (int x = 0; x < V; ++x) op[x] = f2act(acc[x] * inv, BF);
  if (p.lse && lane == 0)
    p.lse[(int64_t)row * p.hq + head] =
        sum == 0.0f ? -__builtin_inff() : (top + __builtin_amdgcn_logf(sum)) * kLn2;
}

// The host's side of the plan: what the device's plan cannot exceed.
struct Plan {
  int tc, target, min_steps;
  int64_t tiles;                     // tiles per head, at most
  int64_t units;                     // units per head, at most
  int64_t slots;                     // partial slots per head, at most (0: nothing is split)
  size_t off_ml, bytes;
};

Plan plan_of(int64_t b, int64_t rows, int32_t hq, int32_t hkv, int32_t d, int32_t page, int64_t max_pages,
             int64_t max_q) {
  Plan p;
  const int64_t G = hq / hkv;
  p.tc = max_q * G > 64 ? 128 : 16;
  const int64_t by_rows = rows * ((G + p.tc - 1) / p.tc), by_cols = rows * G / p.tc + b;
  p.tiles = by_rows < by_cols ? by_rows : by_cols;
  const int64_t total = 512;
  p.target = (int)((total + hkv - 1) / hkv);
  p.min_steps = 8;
  const int64_t steps = max_pages * (page / kStep);
  const int64_t most = (steps + p.min_steps - 1) / p.min_steps;       // units of one tile, at most
  p.units = p.target + p.tiles;
  if (most <= p.units / (p.tiles ? p.tiles : 1)) p.units = p.tiles * (most > 0 ? most : 1);
  p.slots = most > 1 ? (2 * (int64_t)p.target < p.tiles * most ? 2 * (int64_t)p.target : p.tiles * most) : 0;
  const size_t cols = (size_t)p.slots * hkv * p.tc;
  p.off_ml = cols * d * sizeof(float);
  p.bytes = (p.off_ml + cols * 2 * sizeof(float) + 255) / 256 * 256;
  return p;
}

}  // namespace

size_t attn_kv8_scratch_bytes(int64_t b, int64_t rows, int32_t hq, int32_t hkv, int32_t d, int32_t page,
                              int64_t max_pages, int64_t max_q) {
  return plan_of(b, rows, hq, hkv, d, page, max_pages, max_q).bytes;
}

template <int D, bool BF>
static hipError_t launch(const AttnP& p, const Plan& pl, hipStream_t stream) {
  const unsigned grid = (unsigned)(pl.units * p.v.hkv), joins = (unsigned)(pl.tiles * p.v.hkv * (pl.tc / 4));
  if (pl.tc == 128) {
    attn_kv8_tile_kernel<D, BF><<<grid, 256, 0, stream>>>(p);
    if (pl.slots) attn_kv8_join_kernel<D, 128, BF><<<joins, 256, 0, stream>>>(p);
  } else {
    attn_kv8_cols_kernel<D, BF><<<grid, 256, 0, stream>>>(p);
    if (pl.slots) attn_kv8_join_kernel<D, 16, BF><<<joins, 256, 0, stream>>>(p);
  }
  return hipGetLastError();
}

hipError_t launch_attn_kv8(const Kv8Args& a, const uint16_t* q, int64_t q_stride, int32_t hq, int64_t max_q,
                           float scale, bool bf, uint16_t* out, int64_t out_stride, float* lse,
                           void* scratch, hipStream_t stream) {
  if (a.rows < 1 || a.b < 1) return hipSuccess;
  const Plan pl = plan_of(a.b, a.rows, hq, a.hkv, a.d, a.page, a.max_pages, max_q);
  AttnP p;
  p.v = Kv8View{a.k, a.v, a.k_scale, a.v_scale, a.block_table, a.cu_q, a.ctx, a.pages, a.rows,
                (int32_t)a.max_pages, __builtin_ctz((unsigned)a.page), a.hkv, (int32_t)a.b};
  p.q = q;
  p.out = out;
  p.lse = lse;
  p.q_stride = q_stride;
  p.out_stride = out_stride;
  p.hq = hq;
  p.G = hq / a.hkv;
  p.scale2 = scale * kLog2e;
  p.target = pl.target;
  p.min_steps = pl.min_steps;
  p.slots = (int32_t)pl.slots;
  p.part = (float*)scratch;
  p.part_ml = (float*)((char*)scratch + pl.off_ml);
  if (a.d == 64) return bf ? launch<64, true>(p, pl, stream) : launch<64, false>(p, pl, stream);
  return bf ? launch<128, true>(p, pl, stream) : launch<128, false>(p, pl, stream);
}

}  // namespace awq
