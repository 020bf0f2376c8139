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
// One pass with a running reference m.  The page's value scale goes into the
// exponent: p' = exp2(s + log2 vs - m), O = sum p' vcode, l = sum p' / vs.  So p'
// carries exactly the weight of its token's contribution to O whatever the scales
// are.  S, O, m and l are fp32; p' enters the value product in fp16, with a relative
// rounding of at most 2^-11: m lies 2^11 under the largest score it was set by, so
// weights down to 2^-25 of the largest are normal fp16 numbers (a first token
// that outweighs every other by 2^20 takes nothing from them).  m moves only when a
// score would leave fp16 (a wave-wide vote), so most steps exchange nothing
// between lanes and rescale nothing.
#include "awq_internal.h"
#include "kv8_common.h"

namespace awq {
namespace {

constexpr int kStep = 64;            // tokens of one step (a page holds whole steps)
constexpr float kRoom = 11.0f;       // m is set to the largest score less 11 ...
constexpr float kMost = 15.0f;       // ... and moves for scores that exceed it by 15: p' <= 2^15, inside fp16
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kNone = -1e30f;      // m before any visible token

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
  int32_t whole;                     // a context of so many steps is not split
  int32_t slots;                     // partial slots per head in the workspace
  float* part;                       // partial O [slot][hkv][TC][D], then their (m, l)
  float* part_ml;
  int4* rec;                         // line: what partial slot [k][first, last] of a head holds
};

// Results of one column's channels d .. d + 3: O / l, and the lse from channel 0.
// No visible token: zeros and -inf (a NaN sum is kept).
template <bool BF>
__device__ __forceinline__ void store4(const AttnP& p, int row, int head, int D, int d, float4 a, float top,
                                       float sum) {
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  *(uint2*)(p.out + row * p.out_stride + (int64_t)head * D + d) =
      make_uint2(pack2<BF>(a.x * inv, a.y * inv), pack2<BF>(a.z * inv, a.w * inv));
  if (p.lse && d == 0)
    p.lse[(int64_t)row * p.hq + head] = sum == 0.0f ? -__builtin_inff() : (top + __builtin_amdgcn_logf(sum)) * kLn2;
}

// The partial results of one tile: slots first, next, next + step, ...
struct Parts {
  int first, next, step, count, tile;
  SeqRows r;
};

// 16 bytes of the cache.  ONCE: nothing else of the launch reads them, so they
// are not kept in the caches (one sequence of 128 K tokens: 50.3 us against 56.1; 64 ragged
// of up to 8 K: 95.8 against 106.1).
template <bool ONCE>
__device__ __forceinline__ uint4 load16(const uint8_t* p) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  if (ONCE) return __builtin_bit_cast(uint4, __builtin_nontemporal_load((const u32x4*)p));
  return *(const uint4*)p;
}

// What a wave needs of the sequence whose columns it works on.
struct Seq {
  const int32_t* bt;       // its row of the block table
  int ctx, pos, first;     // pos: the last position that this lane's column sees (-1: none);
                           // first: the least pos of the wave's columns
};

// One wave's columns of one key/value head, a step at a time: keys and values go
// from the cache to registers, with no LDS and no barrier.  ask(st) asks for a
// step's keys; loop() runs the steps st, st + stride, ... < st1, the first of
// them asked for.  The next step's keys are asked for as soon as the scores have
// used this one's, and the values while the scores run.
//
// C = 16, MFMA 16x16x32: lane (c = l % 16, g = l / 16) holds column c and the 16 tokens
// 16 g .. 16 g + 15 of a step:
//   score tile t, A row r  = token 16 (r / 4) + 4 t + r % 4 (the rows of an MFMA may be
//                            any tokens), so result i of group g is token 16 g + 4 t + i;
//   score k-step 2 x + e   = channels 64 x + 16 g + 8 e .. + 7;
//   output k-step e        = tokens 16 g + 8 e .. + 7.
// C = 32, MFMA 32x32x16: lane (c = l % 32, g = l / 32) holds column c and, of each 32-token
// tile t, the tokens 32 t + 16 g .. + 15:
//   score tile t, A row r  = token 32 t + 16 (r / 4 % 2) + 4 (r / 8) + r % 4, so result i
//                            of group g is token 32 t + 16 g + i;
//   score k-step 2 x + e   = channels 32 x + 16 g + 8 e .. + 7;
//   output k-step 2 t + e  = tokens 32 t + 16 g + 8 e .. + 7.
// So every operand of the cache is a 16-byte load that feeds two MFMAs.
template <int D, bool BF, int C, bool ONCE>
struct Wave {
  typedef Mma<BF> MQ;
  typedef Mma<false> MV;
  static constexpr bool W = C == 32;
  static constexpr int GR = 64 / C;              // lane groups
  static constexpr int NT = W ? 2 : 4;           // score tiles of a step
  static constexpr int NJ = W ? 16 : 4;          // results of a lane in a tile
  static constexpr int NX = D / (16 * GR);       // key loads of a tile
  static constexpr int NV = W ? 2 : 1;           // value loads of C channels
  static constexpr int ND = D / C;
  typedef float acc_t __attribute__((ext_vector_type(W ? 16 : 4)));

  typename MQ::frag qf[NX][2];
  acc_t o[ND];
  float m, l;
  uint4 kr[NT][NX];
  float ks, vs;
  bool bad;
  const uint8_t* vp;

  static __device__ __forceinline__ acc_t mma_q(typename MQ::frag a, typename MQ::frag b, acc_t c) {
    if constexpr (W) return MQ::mma32(a, b, c);
    else return MQ::mma16(a, b, c);
  }
  static __device__ __forceinline__ acc_t mma_v(half8_t a, half8_t b, acc_t c) {
    if constexpr (W) return MV::mma32(a, b, c);
    else return MV::mma16(a, b, c);
  }
  // token of result j of score tile t in group g
  static __device__ __forceinline__ int token(int t, int j, int g) { return W ? 32 * t + 16 * g + j : 16 * g + 4 * t + j; }
  // channel of result j of output tile i in group g
  static __device__ __forceinline__ int channel(int i, int j, int g) {
    return W ? 32 * i + 8 * (j >> 2) + 4 * g + (j & 3) : 16 * i + 4 * g + j;
  }

  __device__ __forceinline__ void load_q(const uint16_t* qp, int lane) {
    const int g = lane / C;
#pragma unroll
    for (int x = 0; x < NX; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        qf[x][e] = __builtin_bit_cast(typename MQ::frag, *(const uint4*)(qp + 16 * GR * x + 16 * g + 8 * e));
  }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) o[i][j] = 0.0f;
    m = kNone;
    l = 0.0f;
  }

  __device__ __forceinline__ void ask(const Kv8View& v, float scale2, const Seq& q, int h, int st, int lane) {
    const int c = lane % C, g = lane / C, t0 = st * kStep;
    const int krow = W ? 16 * (c >> 2 & 1) + 4 * (c >> 3) + (c & 3) : 16 * (c >> 2) + (c & 3);
    int pid = scalar_load(q.bt + (t0 >> v.shift));
    bad = (uint32_t)pid >= (uint32_t)v.pages;
    pid = bad ? 0 : pid;
    const int64_t ph = (int64_t)pid * v.hkv + h;
    const int slot0 = t0 & ((1 << v.shift) - 1);
    const uint8_t* kp = v.kc + ((ph << v.shift) + slot0) * D;
    vp = v.vc + ((ph * D) << v.shift) + slot0;
    // not in the cache: the key scale makes NaN of what is seen; the value scale must be
    // one that leaves the sums of the columns that see none of it alone (0 / vs = 0)
    const float v1 = scalar_load(v.vs + ph);
    ks = bad ? __builtin_nanf("") : scalar_load(v.ks + ph) * scale2;
    vs = bad ? 1.0f : v1;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int x = 0; x < NX; ++x)
        kr[t][x] = load16<ONCE>(kp + ((W ? 32 : 4) * t + krow) * D + 16 * GR * x + 16 * g);
  }

  // Scores of one step to softmax weights.  level(): masks, moves m where it has to,
  // and leaves the scores' factor and addend in a and z; weights(): the weights in pf
  // as the value product's operand, their sum in l.
  __device__ __forceinline__ void level(acc_t* s, const Seq& q, int t0, float k1, float v1, bool out_of, int g,
                                        float& a, float& z) {
    a = k1;
    z = __builtin_amdgcn_logf(v1);
    if (t0 + kStep - 1 > q.first || out_of) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          s[t][j] = t0 + token(t, j, g) <= q.pos ? __builtin_fmaf(s[t][j], a, z) : -__builtin_inff();
      a = 1.0f;
      z = 0.0f;
    }
    float mx = s[0][0];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < NJ; ++j) mx = __builtin_fmaxf(mx, s[t][j]);
    mx = __builtin_fmaf(mx, a, z);
    if (__ballot(mx > m + kMost)) {
#pragma unroll
      for (int x = C; x < 64; x <<= 1) mx = __builtin_fmaxf(mx, __shfl_xor(mx, x, 64));
      const float mn = __builtin_fmaxf(m, mx - kRoom);
      const float f = __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      l *= f;
#pragma unroll
      for (int i = 0; i < ND; ++i) o[i] *= f;
    }
    z -= m;
  }
  __device__ __forceinline__ void weights(const acc_t* s, float a, float z, float v1, half8_t* pf) {
    float sum = 0.0f;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][j], a, z));
        sum += e;
        pf[(t * NJ + j) / 8][(t * NJ + j) % 8] = (half_t)e;
      }
    l = __builtin_fmaf(sum, __builtin_amdgcn_rcpf(v1), l);
  }

  // Codes of 16 tokens, `left` of them before the sequence's end: slots behind it, and
  // the page read in place of one that is not in the cache, may hold anything,
  // NaN codes too (0 * NaN).
  static __device__ __forceinline__ void trim(uint4& x, int left) {
    uint32_t* w = (uint32_t*)&x;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = left - 4 * j;
      w[j] &= n >= 4 ? ~0u : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
    }
  }

  __device__ __forceinline__ void loop(const Kv8View& v, float scale2, const Seq& q, int h, int st, int st1,
                                       int stride, int lane) {
    const int c = lane % C, g = lane / C;
    for (; st < st1; st += stride) {
      const int t0 = st * kStep;
      uint4 vr[ND][NV];
#pragma unroll
      for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int t = 0; t < NV; ++t)
          vr[i][t] = load16<ONCE>(vp + ((C * i + c) << v.shift) + 32 * t + 16 * g);
      acc_t s[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) s[t][j] = 0.0f;
#pragma unroll
        for (int x = 0; x < NX; ++x) {
          s[t] = mma_q(MQ::from_fp8(kr[t][x].x, kr[t][x].y), qf[x][0], s[t]);
          s[t] = mma_q(MQ::from_fp8(kr[t][x].z, kr[t][x].w), qf[x][1], s[t]);
        }
      }
      const float k1 = ks, v1 = vs;
      const bool out_of = bad;
      if (st + stride < st1) ask(v, scale2, q, h, st + stride, lane);
      half8_t pf[NT * NJ / 8];
      float a, z;
      level(s, q, t0, k1, v1, out_of, g, a, z);
      weights(s, a, z, v1, pf);
      if (t0 + kStep > (out_of ? 0 : q.ctx)) {
#pragma unroll
        for (int i = 0; i < ND; ++i)
#pragma unroll
          for (int t = 0; t < NV; ++t) trim(vr[i][t], (out_of ? 0 : q.ctx) - (t0 + 32 * t + 16 * g));
      }
#pragma unroll
      for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int t = 0; t < NV; ++t) {
          o[i] = mma_v(MV::from_fp8(vr[i][t].x, vr[i][t].y), pf[2 * t], o[i]);
          o[i] = mma_v(MV::from_fp8(vr[i][t].z, vr[i][t].w), pf[2 * t + 1], o[i]);
        }
    }
  }

  // l over the lane groups; NaN where the column sees positions behind the sequence's
  // row of the block table
  __device__ __forceinline__ void finish(const Kv8View& v, int pos) {
#pragma unroll
    for (int x = C; x < 64; x <<= 1) l += __shfl_xor(l, x, 64);
    if (pos >= (int64_t)v.max_pages << v.shift) l = __builtin_nanf("");
  }
};

// ---------------------------------------------------------------- few columns

// The work of a head lies on a line: the tiles of C columns one after another, each
// as long as its sequence has steps (at least one, so that rows that see nothing are
// written too).  Work-group k of the head takes the stretch from start(k) to
// start(k + 1): equal stretches whatever the lengths are, so all work-groups,
// one on each CU, end together.  A stretch's ends move off a tile that is too
// short to be worth sharing, and off a tile's last few steps.  (64 ragged sequences of
// up to 8 K tokens, 541 MB: 92 us, 5.9 TB/s.  When stretches came in the place of one unit
// for each share of a context: 101 us against 108 to 128, by the number of units.)
struct Line {
  uint32_t per;            // length of a stretch
  uint32_t all;            // length of the line
};
struct Place {             // a tile on the line
  uint32_t at;             // its first step
  int steps, b, tile;
  SeqRows r;
};

template <int C>
struct Stretch {
  const AttnP& p;
  const int lane, cap;
  // the sequences w0 + lane, a window that moves along the line; it begins at wat
  SeqRows r;
  int tiles, steps, w0;
  uint32_t wat;
  Line line;

  __device__ __forceinline__ void load(int i) {
    r = SeqRows{0, 0, 0};
    tiles = steps = 0;
    if (i < p.v.b) {
      r = seq_rows(p.v, i);
      tiles = (int)(((uint32_t)r.n * (uint32_t)p.G + C - 1) / C);      // rows * hq <= 2^30
      steps = r.ctx / kStep + (r.ctx % kStep ? 1 : 0);
      steps = steps < cap ? steps : cap;
      steps = steps < 1 ? 1 : steps;
    }
  }
  __device__ __forceinline__ void rewind() {
    w0 = 0;
    wat = 0;
    load(lane);
  }

  __device__ __forceinline__ Stretch(const AttnP& p, int lane)
      : p(p), lane(lane), cap((int)(((int64_t)p.v.max_pages << p.v.shift) / kStep)) {
    // below 2^31 for ascending cu (the host has seen to it)
    uint32_t sum = 0;
#pragma unroll 4
    for (int i0 = 0; i0 < p.v.b; i0 += 64) {
      load(i0 + lane);
      sum += (uint32_t)tiles * (uint32_t)steps;
    }
    line.all = __builtin_amdgcn_readlane(wave_scan((int)sum), 63);
    const uint32_t per = (uint32_t)(((uint64_t)line.all + p.target - 1) / (uint32_t)p.target);
    line.per = per > (uint32_t)p.min_steps ? per : p.min_steps;
    w0 = 0;
    wat = 0;
    if (p.v.b > 64) load(lane);
  }

  // the tile that holds x < line.all
  __device__ __forceinline__ Place place(uint32_t x) {
    Place w;
    w.b = -1;
    if (x < wat) rewind();
    for (;;) {
      const uint32_t mine = (uint32_t)tiles * (uint32_t)steps;
      const uint32_t incl = wave_scan((int)mine);
      const uint32_t sum = __builtin_amdgcn_readlane((int)incl, 63);
      if (x - wat < sum) {
        int l = __popcll(__ballot(incl <= x - wat));
        l = l < 63 ? l : 63;
        const uint32_t in = x - wat - __builtin_amdgcn_readlane((int)(incl - mine), l);
        // always so for ascending cu; whatever else the array holds ends here
        if (in >= (uint32_t)__builtin_amdgcn_readlane((int)mine, l)) return w;
        w.b = w0 + l;
        w.steps = __builtin_amdgcn_readlane(steps, l);
        w.r.r0 = __builtin_amdgcn_readlane(r.r0, l);
        w.r.n = __builtin_amdgcn_readlane(r.n, l);
        w.r.ctx = __builtin_amdgcn_readlane(r.ctx, l);
        w.tile = (int)(in / (uint32_t)w.steps);
        w.at = x - in + (uint32_t)w.tile * w.steps;
        return w;
      }
      if (w0 + 64 >= p.v.b) return w;
      w0 += 64;
      wat += sum;
      load(w0 + lane);
    }
  }

  // where work-group k begins
  __device__ __forceinline__ uint32_t start(int k) {
    const uint64_t x64 = (uint64_t)k * line.per;
    if (k == 0 || x64 >= line.all) return k == 0 ? 0 : line.all;
    const uint32_t x = (uint32_t)x64;
    const Place w = place(x);
    if (w.b < 0) return line.all;
    const uint32_t in = x - w.at, left = w.steps - in;
    if (in == 0) return x;
    if (w.steps <= p.whole || left < 4) return w.at + w.steps;
    return in < 4 ? w.at : x;
  }
};

// Tiles of C columns; the NW waves of a work-group take a tile's steps in turn and
// are joined in LDS at the tile's end, or at the stretch's: a tile that a stretch
// covers only in part leaves its O, m and l in the workspace, in slot 2 k of work-group k
// if the part begins the stretch, else in 2 k + 1; and a record of the slot (the same for
// every head, so head 0 writes it): row, rows, tile, and kBegins where the part has the
// tile's first steps, kEnds where it has the last, kHeld where the slot holds anything.
constexpr int kHeld = 1, kBegins = 2, kEnds = 4;

template <int D, bool BF, int C, int NW, bool ONCE>
__global__ __launch_bounds__(64 * NW, 2) void attn_kv8_line_kernel(AttnP p) {
  typedef Wave<D, BF, C, ONCE> E;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const Kv8View& v = p.v;
  const int h = blockIdx.x % v.hkv, k = blockIdx.x / v.hkv, G = p.G;
  const bool notes = p.rec && h == 0 && threadIdx.x == 0;
  if (notes) {
    p.rec[2 * k].w = 0;
    p.rec[2 * k + 1].w = 0;
  }
  Stretch<C> y(p, lane);
  const uint32_t x0 = y.start(k);
  Stretch<C> ahead = y;                          // leaves y's window where the stretch begins
  const uint32_t x1 = ahead.start(k + 1);
  if (x0 >= x1) return;
  const int c = lane % C, g = lane / C;
  __shared__ __attribute__((aligned(16))) float so[NW * C * (D + 4)];     // O [wave][column][channel]
  __shared__ float sm[NW * C], sl[NW * C];

  E e;
  Seq q;
  Place w = y.place(x0);
  uint32_t x = x0;
  int st, st1, cols;
  // the tile's columns and this stretch's steps of it
  auto begin = [&]() {
    w.b = uniform(w.b), w.steps = uniform(w.steps), w.tile = uniform(w.tile), w.at = uniform(w.at);
    w.r.n = uniform(w.r.n), w.r.ctx = uniform(w.r.ctx), w.r.r0 = uniform(w.r.r0);
    const int n = w.r.n, ctx = w.r.ctx, col = w.tile * C + c;
    cols = n * G - w.tile * C < C ? n * G - w.tile * C : C;
    q.bt = v.bt + (int64_t)w.b * v.max_pages;
    q.ctx = ctx;
    q.pos = c < cols ? ctx - n + col / G : -1;
    q.first = uniform(cols < C ? -1 : ctx - n + (w.tile * C) / G);
    const int held = ctx / kStep + (ctx % kStep ? 1 : 0), there = held < y.cap ? held : y.cap;
    const uint32_t z = w.at + w.steps < x1 ? w.at + w.steps : x1;
    st = (int)(x - w.at) + wave;
    st1 = (int)(z - w.at) < there ? (int)(z - w.at) : there;
    if (st < st1) e.ask(v, p.scale2, q, h, st, lane);
    const int cc = c < cols ? col : w.tile * C;
    e.load_q(p.q + (int64_t)(w.r.r0 + cc / G) * p.q_stride + (int64_t)(h * G + cc % G) * D, lane);
  };
  if (w.b < 0) return;
  begin();
  for (;;) {
    e.clear();
    e.loop(v, p.scale2, q, h, st, st1, NW, lane);
    e.finish(v, q.pos);
    const Place done = w;
    const int dcols = cols;
    const uint32_t from = x;
    x = w.at + w.steps;
    if (c < cols) {
#pragma unroll
      for (int i = 0; i < E::ND; ++i)
#pragma unroll
        for (int j = 0; j < E::NJ; j += 4)
          *(float4*)&so[(wave * C + c) * (D + 4) + E::channel(i, j, g)] =
              make_float4(e.o[i][j], e.o[i][j + 1], e.o[i][j + 2], e.o[i][j + 3]);
      if (g == 0) {
        sm[wave * C + c] = e.m;
        sl[wave * C + c] = e.l;
      }
    }
    // the next tile's first keys and queries travel while this one's waves are joined
    const bool more = x < x1 && x > from;
    if (more) {
      w = y.place(x);
      if (w.b < 0) return;
      begin();
    }
    __syncthreads();
    const bool begins = from == done.at, ends = x <= x1, whole = begins && ends;
    if (notes && !whole)
      p.rec[2 * k + (from == x0 ? 0 : 1)] =
          make_int4(done.r.r0, done.r.n, done.tile, kHeld | (begins ? kBegins : 0) | (ends ? kEnds : 0));
    // a thread: 4 channels of one column
    for (int it = threadIdx.x; it < dcols * (D / 4); it += 64 * NW) {
      const int jc = it / (D / 4), d = it % (D / 4) * 4;
      float top = kNone, sum = 0.0f;
#pragma unroll
      for (int i = 0; i < NW; ++i) top = __builtin_fmaxf(top, sm[i * C + jc]);
      float4 a = make_float4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        const float f = __builtin_amdgcn_exp2f(sm[i * C + jc] - top);
        const float4 b = *(const float4*)&so[(i * C + jc) * (D + 4) + d];
        sum = __builtin_fmaf(f, sl[i * C + jc], sum);
        a.x = __builtin_fmaf(f, b.x, a.x);
        a.y = __builtin_fmaf(f, b.y, a.y);
        a.z = __builtin_fmaf(f, b.z, a.z);
        a.w = __builtin_fmaf(f, b.w, a.w);
      }
      if (whole) {
        const int col = done.tile * C + jc, row = done.r.r0 + col / G, head = h * G + col % G;
        store4<BF>(p, row, head, D, d, a, top, sum);
      } else {
        const int64_t at = ((int64_t)(2 * k + (from == x0 ? 0 : 1)) * v.hkv + h) * C + jc;
        *(float4*)(p.part + at * D + d) = a;
        if (d == 0) {
          p.part_ml[2 * at] = top;
          p.part_ml[2 * at + 1] = sum;
        }
      }
    }
    if (!more) return;
    __syncthreads();
  }
}

// The parts of the tile that work-group k - 1 begins and work-group k goes on with:
// k - 1's last and the first ones of k, k + 1, ... up to the one that ends it.
__device__ __forceinline__ bool line_parts(const AttnP& p, int k, int lane, Parts& w) {
  const int4 a = p.rec[2 * k - 2], b = p.rec[2 * k - 1];
  // a lane for each of k, k + 1, ...
  int n = 0;
  for (int i0 = k; i0 < p.target; i0 += 64) {
    const int f = i0 + lane < p.target ? p.rec[2 * (i0 + lane)].w : kHeld | kBegins;
    const uint64_t stop = __ballot((f & kEnds) != 0 || (f & kBegins) != 0 || f == 0);
    if (stop) {
      const int l = __builtin_ctzll(stop);
      const int last = __builtin_amdgcn_readlane(f, l);
      if (!(last & kEnds) || last & kBegins) return false;      // k does not go on with anything
      n += l + 1;
      break;
    }
    n += 64;
  }
  const bool second = (b.w & (kBegins | kEnds)) == kBegins;
  if (!second && (a.w & (kBegins | kEnds)) != kBegins) return false;
  const int4 t = second ? b : a;
  w.first = 2 * (k - 1) + (second ? 1 : 0);
  w.next = 2 * k;
  w.step = 2;
  w.count = n + 1;
  w.tile = t.z;
  w.r = SeqRows{t.x, t.y, 0};
  return n > 0;
}

// ---------------------------------------------------------------- many columns

// The part of the work one work-group does: steps s of S of tile `tile` of
// sequence `b`.
struct Unit {
  int b, tile, s, S, slot;
  SeqRows r;
};

// The plan, computed by every wave from the device's own lengths (a captured
// graph replays with new ones): tiles of TC columns; a sequence's tiles are cut
// into S = ceil(steps / chunk) units, chunk = total steps over the target, and (of up
// to 64 sequences) those with longer units come first, so that the last
// work-groups to start are short.  The total counts what causal tiles see, never less than half of
// their steps, so there are at most 2 * target units and one for each tile.
// Units of sequences with S > 1 have partial slots, numbered in the same order;
// fewer than 4 * target, as S > 1 needs steps > chunk and then
// ceil(steps / chunk) < 2 steps / chunk.
// JOIN: u counts the tiles of the split sequences (fewer than 2 * target) instead.
// Everything returned is the same in all lanes.
template <int TC, bool JOIN>
__device__ __forceinline__ bool find_unit(const AttnP& p, int u, int lane, Unit& w) {
  const Kv8View& v = p.v;
  const int cap = (int)(((int64_t)v.max_pages << v.shift) / kStep);
  auto load = [&](int i, SeqRows& r, int& tiles, int& steps) {
    r = SeqRows{0, 0, 0};
    tiles = steps = 0;
    if (i < v.b) {
      r = seq_rows(v, i);
      tiles = (int)(((uint32_t)r.n * (uint32_t)p.G + TC - 1) / TC);   // rows * hq <= 2^30
      steps = r.ctx / kStep + (r.ctx % kStep ? 1 : 0);
      steps = steps < cap ? steps : cap;
    }
  };
  SeqRows r;
  int tiles, steps;
  uint64_t total = 0;
  for (int i0 = 0; i0 < v.b; i0 += 64) {
    load(i0 + lane, r, tiles, steps);
    // a causal tile sees on average what its sequence's middle row sees
    const int seen = steps - r.n / (2 * kStep), half = (steps + 1) / 2;
    total += (uint64_t)tiles * (seen > half ? seen : half);
  }
  // below 2^51 for ascending cu: two sums of 32 bits
  const uint32_t lo = __builtin_amdgcn_readlane(wave_scan((int)(total & 0x1FFFFFFu)), 63);
  const uint32_t hi = __builtin_amdgcn_readlane(wave_scan((int)(total >> 25)), 63);
  const double per = __builtin_ceil(((double)hi * 33554432.0 + (double)lo) / (double)p.target);
  const int chunk = per > (double)p.min_steps ? (per < 1e9 ? (int)per : 1000000000) : p.min_steps;
  int before = 0, slots = 0;
  for (int i0 = 0; i0 < v.b; i0 += 64) {
    if (v.b > 64) load(i0 + lane, r, tiles, steps);
    // a short context is not worth partial results and a second launch's work
    int S = steps <= p.whole ? 1 : (steps + chunk - 1) / chunk;
    S = S < 1 ? 1 : S;
    const int held = S > 1 ? tiles * S : 0;
    const int mine = JOIN ? (S > 1 ? tiles : 0) : tiles * S;
    const int incl = wave_scan(mine), hincl = wave_scan(held);
    const int all = __builtin_amdgcn_readlane(incl, 63);
    int from = incl - mine, sfrom = hincl - held;
    if (v.b <= 64) {
      // this lane's units and slots come behind those of the sequences with longer units
      const int len = steps / S;
      from = sfrom = 0;
      for (int j = 0; j < v.b; ++j) {
        const int other = __builtin_amdgcn_readlane(len, j);
        const int add = __builtin_amdgcn_readlane(mine, j), sadd = __builtin_amdgcn_readlane(held, j);
        const bool first = other > len || (other == len && j < lane);
        from += first ? add : 0;
        sfrom += first ? sadd : 0;
      }
    }
    if (u - before < all) {
      const int x = u - before;
      const uint64_t hit = __ballot(x >= from && x < from + mine);
      if (!hit) return false;                // cannot be for ascending cu
      const int l = __builtin_ctzll(hit);
      const int at = x - __builtin_amdgcn_readlane(from, l);
      w.b = i0 + l;
      w.S = __builtin_amdgcn_readlane(S, l);
      w.r.r0 = __builtin_amdgcn_readlane(r.r0, l);
      w.r.n = __builtin_amdgcn_readlane(r.n, l);
      w.r.ctx = __builtin_amdgcn_readlane(r.ctx, l);
      const int nt = __builtin_amdgcn_readlane(tiles, l);
      const int order = JOIN ? at : at / w.S;
      w.s = JOIN ? 0 : at % w.S;
      w.tile = nt - 1 - order;               // later rows see more: the longest first
      w.slot = slots + __builtin_amdgcn_readlane(sfrom, l) + order * w.S + w.s;
      // always so for ascending cu; whatever else the array holds stays in bounds
      const int top = w.S > 1 ? (JOIN ? w.slot + w.S : w.slot + 1) : 0;
      return w.tile >= 0 && w.tile < nt && w.slot >= 0 && top <= p.slots;
    }
    before += all;
    slots += __builtin_amdgcn_readlane(hincl, 63);
  }
  return false;
}

// Tiles of 128 columns: each of the four waves has 32 of them and walks all of the
// unit's steps.  A step's codes come to LDS once for the four waves, copied there
// straight from the cache two stages deep: 16-byte pieces, placed so that the 8
// lanes of an LDS cycle hit different banks.  (Read by each wave from the CU's
// vector cache instead, that cache was 92 % busy and the 8 K prompt took 740 us, against 607 at
// that step.)
//   keys    piece j of token r's D / 16 at j ^ key(r): the rows that an 8-lane cycle reads
//           are 4 neighbours of two blocks of 16;
//   values  piece j of channel d's four at j ^ (d / 2 % 4).
template <int D>
struct Stage {
  static constexpr int KP = D / 16;              // pieces of a token's keys
  uint4 k[kStep * KP];
  uint4 v[D * 4];
  static __device__ __forceinline__ int key(int r) { return KP == 8 ? (r & 3) | (r >> 2 & 4) : (r >> 1 & 1) | (r >> 3 & 2); }
  static __device__ __forceinline__ int kat(int r, int j) { return r * KP + (j ^ key(r)); }
  static __device__ __forceinline__ int vat(int d, int j) { return d * 4 + (j ^ (d >> 1 & 3)); }
};

// One 16-byte global -> LDS copy per lane, from src + off: lane i writes LDS bytes
// base + 16 i .. +15.
// From inline asm, so that the compiler leaves the waits to the caller: it would
// drain every outstanding copy before any read of the array.  M0 is the
// compiler's only to address LDS copies of its own; there are none here.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void lds_copy16(const void* src, uint32_t off, uint32_t base) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :
               : "v"(off), "s"(src), "s"(base)
               : "memory", "m0");
}
#pragma clang diagnostic pop

template <int D, bool BF>
__global__ __launch_bounds__(256, 2) void attn_kv8_tile_kernel(AttnP p) {
  constexpr int TC = 128, ND = D / 32, NW = 4;
  typedef Wave<D, BF, 32, false> E;
  typedef Stage<D> T;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int h = blockIdx.x % p.v.hkv;
  Unit w;
  if (!find_unit<TC, false>(p, blockIdx.x / p.v.hkv, lane, w)) return;
  const Kv8View& v = p.v;
  const int b = uniform(w.b), S = uniform(w.S), sidx = uniform(w.s), tile = uniform(w.tile);
  const int n = uniform(w.r.n), r0 = uniform(w.r.r0), ctx = uniform(w.r.ctx);
  const int G = p.G, c0 = tile * TC + 32 * wave;
  const int cols = n * G - c0 < 32 ? n * G - c0 : 32;           // may be none
  const int c = lane & 31, half = lane >> 5, col = c0 + c;
  const int pos = c < cols ? ctx - n + col / G : -1;
  const int first = uniform(cols < 32 ? -1 : ctx - n + c0 / G);
  // the unit's share of the tile's steps; this wave computes what its own rows see
  const int tcols = n * G - tile * TC < TC ? n * G - tile * TC : TC;
  const int last = ctx - n + (tile * TC + tcols - 1) / G, wlast = cols > 0 ? ctx - n + (c0 + cols - 1) / G : -1;
  const int cap = (int)(((int64_t)v.max_pages << v.shift) / kStep);
  int steps = last < 0 ? 0 : last / kStep + 1;
  steps = steps < cap ? steps : cap;
  // divisions leave wave-uniform values in vector registers: bring them back, so that
  // branches on them are scalar
  const int st0 = uniform((int)((int64_t)steps * sidx / S)), st1 = uniform((int)((int64_t)steps * (sidx + 1) / S));
  const int wst1 = uniform(wlast < 0 ? 0 : wlast / kStep + 1);

  __shared__ T stage[2];
  E a;
  const Seq q = {v.bt + (int64_t)b * v.max_pages, ctx, pos, first};
  {
    const int cc = c < cols ? col : tile * TC;
    a.load_q(p.q + (int64_t)(r0 + cc / G) * p.q_stride + (int64_t)(h * G + cc % G) * D, lane);
  }
  a.clear();

  // this wave's pieces of a step: chunks of 64 pieces, every fourth
  constexpr int CK = T::KP / NW, CV = D / 16 / NW;
  uint32_t koff[CK], voff[CV];
#pragma unroll
  for (int i = 0; i < CK; ++i) {
    const int at = (wave + NW * i) * 64 + lane, r = at / T::KP;
    koff[i] = r * D + 16 * (at % T::KP ^ T::key(r));
  }
#pragma unroll
  for (int i = 0; i < CV; ++i) {
    const int at = (wave + NW * i) * 64 + lane, d = at / 4;
    voff[i] = (d << v.shift) + 16 * (at % 4 ^ (d >> 1 & 3));
  }
  const int smask = (1 << v.shift) - 1;
  const uint32_t pages = (uint32_t)v.pages;                     // below 2^31
  // an LDS address is the low half of its flat one
  const uint32_t lds0 = uniform((int)(uint32_t)(uintptr_t)&stage[0]) + wave * 1024;
  auto page_of = [&](int st) { return st < st1 ? scalar_load(q.bt + ((st * kStep) >> v.shift)) : 0; };
  auto held = [&](int pid) { return (uint32_t)pid < pages; };
  auto head_of = [&](int pid) { return (int64_t)(held(pid) ? pid : 0) * v.hkv + h; };
  auto copy_k = [&](int st, int pid) {
    const uint8_t* kp = v.kc + ((head_of(pid) << v.shift) + ((st * kStep) & smask)) * D;
    const uint32_t base = lds0 + (st & 1) * (uint32_t)sizeof(T);
#pragma unroll
    for (int i = 0; i < CK; ++i) lds_copy16(kp, koff[i], base + NW * 1024 * i);
  };
  auto copy_v = [&](int st, int pid) {
    const uint8_t* vp = v.vc + ((head_of(pid) * D) << v.shift) + ((st * kStep) & smask);
    const uint32_t base = lds0 + (st & 1) * (uint32_t)sizeof(T) + (uint32_t)sizeof(stage[0].k);
#pragma unroll
    for (int i = 0; i < CV; ++i) lds_copy16(vp, voff[i], base + NW * 1024 * i);
  };
  // where this lane's operands lie in a stage, in bytes: tile t of the keys and tile i of
  // the values are a constant further on
  int kat[E::NX], vat[2];
  {
    const int r = 16 * (c >> 2 & 1) + 4 * (c >> 3) + (c & 3);
#pragma unroll
    for (int x = 0; x < E::NX; ++x) kat[x] = 16 * T::kat(r, 2 * x + half);
#pragma unroll
    for (int t = 0; t < 2; ++t) vat[t] = (int)sizeof(stage[0].k) + 16 * T::vat(c, 2 * t + half);
  }
  auto keys = [&](int st, uint4 (*kr)[E::NX]) {
    const char* sg = (const char*)&stage[st & 1];
#pragma unroll
    for (int x = 0; x < E::NX; ++x)
#pragma unroll
      for (int t = 0; t < 2; ++t) kr[t][x] = *(const uint4*)(sg + kat[x] + 32 * t * D);
  };
  // two chains of dependent products
  auto scores = [&](const uint4 (*kr)[E::NX], typename E::acc_t* s) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int j = 0; j < 16; ++j) s[t][j] = 0.0f;
#pragma unroll
    for (int x = 0; x < E::NX; ++x) {
#pragma unroll
      for (int t = 0; t < 2; ++t) s[t] = E::mma_q(E::MQ::from_fp8(kr[t][x].x, kr[t][x].y), a.qf[x][0], s[t]);
#pragma unroll
      for (int t = 0; t < 2; ++t) s[t] = E::mma_q(E::MQ::from_fp8(kr[t][x].z, kr[t][x].w), a.qf[x][1], s[t]);
    }
  };
  // behind it everyone's copies have landed, and nobody reads what was read before
  auto meet = [&]() {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
  };

  // The scores run a step ahead of the softmax and the value product, so that their
  // MFMAs have other work to hide behind: step st + 1's keys and step st's values
  // are in LDS at a time, step st + 2's keys and st + 1's values on their way.
  int pid = page_of(st0), pid1 = page_of(st0 + 1), pid2 = page_of(st0 + 2);
  typename E::acc_t s[2];
  // the queries have come: the compiler, which does not see the copies, would
  // otherwise wait for them inside the loop, and so for the copies asked for last
  __builtin_amdgcn_s_waitcnt(0);
  if (st0 < st1) {
    copy_k(st0, pid);
    meet();
    if (st0 + 1 < st1) copy_k(st0 + 1, pid1);
    copy_v(st0, pid);
    uint4 kr[2][E::NX];
    keys(st0, kr);
    scores(kr, s);
  }
  typename E::acc_t ahead[2];
  auto step = [&](int st, typename E::acc_t* now, typename E::acc_t* then) {
    const int t0 = st * kStep;
    const bool out_of = !held(pid);
    const float ks = out_of ? __builtin_nanf("") : scalar_load(v.ks + head_of(pid)) * p.scale2;
    const float v1 = scalar_load(v.vs + head_of(pid)), vs = out_of ? 1.0f : v1;   // as in Wave::ask
    meet();
    if (st + 1 < st1) copy_v(st + 1, pid1);
    if (st + 2 < st1) copy_k(st + 2, pid2);
    pid = pid1;
    pid1 = pid2;
    pid2 = page_of(st + 3);
    const int end = out_of ? 0 : ctx;
    if (t0 + kStep > end) {                    // once in a unit, at its end
      for (int i = threadIdx.x; i < D * 4; i += 64 * NW)
        E::trim(stage[st & 1].v[i], end - (t0 + 16 * (i % 4 ^ (i >> 3 & 3))));
      __syncthreads();
    }
    if (st >= wst1) return;
    half8_t pf[4];
    float f, z;
    // LDS reads are asked for well before their use: left to itself the compiler puts
    // them right in front of it
    uint4 kr[2][E::NX], vr[2][ND];
    keys(st + 1, kr);                          // of the last step: unused
    __builtin_amdgcn_sched_barrier(0);
    a.level(now, q, t0, ks, vs, out_of, half, f, z);
    const char* sg = (const char*)&stage[st & 1];
#pragma unroll
    for (int i = 0; i < ND; ++i) vr[0][i] = *(const uint4*)(sg + vat[0] + 32 * i * 64);
    scores(kr, then);
    a.weights(now, f, z, vs, pf);
#pragma unroll
    for (int i = 0; i < ND; ++i) vr[1][i] = *(const uint4*)(sg + vat[1] + 32 * i * 64);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int i = 0; i < ND; ++i) a.o[i] = E::mma_v(E::MV::from_fp8(vr[t][i].x, vr[t][i].y), pf[2 * t], a.o[i]);
#pragma unroll
      for (int i = 0; i < ND; ++i) a.o[i] = E::mma_v(E::MV::from_fp8(vr[t][i].z, vr[t][i].w), pf[2 * t + 1], a.o[i]);
    }
  };
  for (int st = st0; st < st1; st += 2) {
    step(st, s, ahead);
    if (st + 1 < st1) step(st + 1, ahead, s);
  }
  a.finish(v, pos);
  if (c >= cols) return;
  if (S == 1) {
    const int row = r0 + col / G, head = h * G + col % G;
    const float inv = a.l == 0.0f ? 0.0f : 1.0f / a.l;
    uint16_t* op = p.out + row * p.out_stride + (int64_t)head * D + 4 * half;
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t x[2] = {pack2<BF>(a.o[i][4 * j] * inv, a.o[i][4 * j + 1] * inv),
                               pack2<BF>(a.o[i][4 * j + 2] * inv, a.o[i][4 * j + 3] * inv)};
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

template <int TC>
__device__ __forceinline__ bool unit_parts(const AttnP& p, int u, int lane, Parts& w) {
  Unit t;
  if (!find_unit<TC, true>(p, u, lane, t)) return false;
  w = Parts{t.slot, t.slot + 1, 1, t.S, t.tile, t.r};
  return true;
}

// Joins the partial results of a split tile's columns in the order of their
// steps.  Work-group (tile, head, z of Z): a wave takes a column, or the four
// waves a quarter of its parts each where there are many; two parts' rows of D
// floats to a load (four for D = 64).
template <int D, int TC, bool BF>
__global__ __launch_bounds__(256) void attn_kv8_join_kernel(AttnP p, int Z) {
  constexpr int LPR = D / 4, RPL = 64 / LPR;       // lanes per row, rows per load
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int hkv = p.v.hkv, h = blockIdx.x % hkv, z = blockIdx.x / hkv % Z;
  Parts w;
  if (!(TC == 128 ? unit_parts<TC>(p, blockIdx.x / hkv / Z, lane, w)
                  : line_parts(p, blockIdx.x / hkv / Z + 1, lane, w)))
    return;
  const int S = w.count, G = p.G;
  auto slot = [&](int i) { return ((int64_t)(i ? w.next + (i - 1) * w.step : w.first) * hkv + h) * TC; };
  const int cols = w.r.n * G - w.tile * TC < TC ? w.r.n * G - w.tile * TC : TC;
  const bool shared = S > 16;
  const int per = shared ? (S + 3) / 4 : S, s0 = shared ? wave * per : 0;
  const int s1 = s0 + per < S ? s0 + per : S;
  __shared__ float so[4][D], sml[4][2];
  const int rowl = lane / LPR, d0 = (lane % LPR) * 4;
  // a column's parts s0 .. s1 - 1: the first rows are asked for with the statistics
  auto fold = [&](int jc, float& top, float& sum, float4& acc) {
    auto stats = [&](int i) {
      return i < s1 ? *(const float2*)(p.part_ml + 2 * (slot(i) + jc)) : make_float2(kNone, 0.0f);
    };
    auto row = [&](int i) { return *(const float4*)(p.part + (slot(i) + jc) * D + d0); };
    float2 ml = stats(s0 + lane);
    float4 ahead[2];
#pragma unroll
    for (int t = 0; t < 2; ++t)
      if (s0 + rowl + RPL * t < s1) ahead[t] = row(s0 + rowl + RPL * t);
    top = ml.x;
    for (int i0 = s0 + 64; i0 < s1; i0 += 64) top = __builtin_fmaxf(top, stats(i0 + lane).x);
    top = wave_fold(top, kNone, [](float x, float y) { return __builtin_fmaxf(x, y); });
    sum = 0.0f;
    acc = make_float4(0, 0, 0, 0);
    auto add = [&](float f, float4 x) {
      acc.x = __builtin_fmaf(f, x.x, acc.x);
      acc.y = __builtin_fmaf(f, x.y, acc.y);
      acc.z = __builtin_fmaf(f, x.z, acc.z);
      acc.w = __builtin_fmaf(f, x.w, acc.w);
    };
    for (int i0 = s0; i0 < s1; i0 += 64) {
      if (i0 > s0) ml = stats(i0 + lane);
      const float f = __builtin_amdgcn_exp2f(ml.x - top);
      sum = __builtin_fmaf(f, ml.y, sum);
      const int n = s1 - i0 < 64 ? s1 - i0 : 64;
#pragma unroll 4
      for (int t = 0; t * RPL < n; ++t) {
        const int i = t * RPL + rowl;
        const float g = __shfl(f, i, 64);
        if (i < n) add(g, i0 == s0 && t == 0 ? ahead[0] : i0 == s0 && t == 1 ? ahead[1] : row(i0 + i));
      }
    }
    sum = wave_fold(sum, 0.0f, [](float x, float y) { return x + y; });
#pragma unroll
    for (int o = LPR; o < 64; o <<= 1) {
      acc.x += __shfl_xor(acc.x, o, 64);
      acc.y += __shfl_xor(acc.y, o, 64);
      acc.z += __shfl_xor(acc.z, o, 64);
      acc.w += __shfl_xor(acc.w, o, 64);
    }
  };
  auto store = [&](int jc, float top, float sum, float4 acc) {
    const int col = w.tile * TC + jc;
    store4<BF>(p, w.r.r0 + col / G, h * G + col % G, D, d0, acc, top, sum);
  };
  float top, sum;
  float4 acc;
  if (!shared) {
    for (int jc = 4 * z + wave; jc < cols; jc += 4 * Z) {
      fold(jc, top, sum, acc);
      if (rowl == 0) store(jc, top, sum, acc);
    }
    return;
  }
  for (int jc = z; jc < cols; jc += Z) {
    fold(jc, top, sum, acc);
    if (rowl == 0) *(float4*)&so[wave][d0] = acc;
    if (lane == 0) {
      sml[wave][0] = top;
      sml[wave][1] = sum;
    }
    __syncthreads();
    if (wave == 0 && rowl == 0) {
      top = __builtin_fmaxf(__builtin_fmaxf(sml[0][0], sml[1][0]), __builtin_fmaxf(sml[2][0], sml[3][0]));
      sum = 0.0f;
      acc = make_float4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float f = __builtin_amdgcn_exp2f(sml[i][0] - top);
        const float4 x = *(const float4*)&so[i][d0];
        sum = __builtin_fmaf(f, sml[i][1], sum);
        acc.x = __builtin_fmaf(f, x.x, acc.x);
        acc.y = __builtin_fmaf(f, x.y, acc.y);
        acc.z = __builtin_fmaf(f, x.z, acc.z);
        acc.w = __builtin_fmaf(f, x.w, acc.w);
      }
      store(jc, top, sum, acc);
    }
    __syncthreads();
  }
}

// The host's side of the plan: what the device's plans cannot exceed.
struct Plan {
  int tc;                            // columns of a tile: 16 and 32 lie on a line, 128 in units
  int target, min_steps, whole;
  int waves;                         // of a work-group on the line
  bool once;                         // a sequence has one tile: its cache is read once
  int64_t groups;                    // work-groups per head
  int64_t slots;                     // partial slots per head (0: nothing can be split)
  int joins, z;                      // tiles per head to join, at most; work-groups for each
  size_t off_ml, off_rec, bytes;
};

Plan plan_of(int64_t b, int64_t rows, int32_t hq, int32_t hkv, int32_t d, int32_t page, int64_t max_pages,
             int64_t max_q) {
  Plan p;
  max_q = max_q < (1 << 24) ? max_q : 1 << 24;
  const int64_t G = hq / hkv, steps = max_pages * (page / kStep) > 1 ? max_pages * (page / kStep) : 1;
  auto tiles_of = [&](int tc) {
    const int64_t by_rows = rows * ((G + tc - 1) / tc), by_cols = rows * G / tc + b;
    return by_rows < by_cols ? by_rows : by_cols;
  };
  // `steps` is what the block table holds: the host does not know the lengths, so a table
  // far wider than its contexts is planned for as long ones are.  Microseconds of tables as
  // wide as their contexts, sequences x rows of 4 heads behind so many tokens:
  //   up to 64 columns of a sequence: 16 (8 x 16 behind 4000: 27, 29 with 32, 33 with 128;
  //   8 x 5: 18, 23, 44);
  //   more: 128, which share what they read among four waves (8 x 96 behind 4000, 160 tiles:
  //   61, 83 with 32; 40 x 48 behind 2000, 560 tiles: 54, 68; 20 x 20 behind 100: 10, 21);
  //   but 32 on the line, which shares its steps out evenly, where few such tiles stand
  //   under a table of more than 32 steps (8 x 24 behind 4000: 28, 53 with 128; 1 x 200
  //   behind 4000: 37, 44).
  const int64_t cols = max_q * G, t128 = tiles_of(128) * hkv;
  p.tc = cols <= 64 ? 16 : steps <= 32 ? 128 : t128 < 144 || (cols <= 128 && t128 < 400) ? 32 : 128;
  if (p.tc < 128 && tiles_of(p.tc) * steps >= (1ll << 31)) p.tc = 128;    // the line is 32 bits long
  const int64_t tiles = tiles_of(p.tc);
  if (p.tc < 128) {
    // Work-groups of eight waves: up to 8 steps a tile is one round of them, and
    // sharing it pays only for the launch that joins; up to 16 where nothing else
    // would need that launch (one sequence of 700 tokens: 8.5 us under a table of its own
    // width; 10.3 under one wider than 16 steps, whose launch finds nothing to join).
    p.whole = tiles * hkv < 64 ? 16 : 8;
    p.min_steps = 4;
    // One work-group of eight waves on each CU; four of two waves where there are so
    // many tiles that each CU has eight whatever their lengths (1024 sequences of 50
    // tokens: 48 us, 98 with eight waves; of 500: 124, 152; 512 tiles of up to 2000
    // tokens: 38, 34).  Tiles of 32 columns are never that many.
    p.waves = p.tc == 16 && tiles * hkv >= 2048 ? 2 : 8;
    const int total = p.waves == 8 ? 256 : 1024;
    p.target = hkv < total ? total / hkv : 1;
    p.groups = p.target;
    p.slots = steps > p.whole && p.target > 1 ? 2 * p.target : 0;
    p.joins = p.target - 1;                  // may be none
    p.z = (int)(max_q * G < 4 ? max_q * G : 4);
  } else {
    // a tile in parts writes and reads 64 KB for each, some 8 steps' time (a prompt of
    // 2048, 32 steps: 55 us whole, 74 in halves; chunks of prompts of up to 106
    // steps: 166 us in halves, 180 whole)
    p.whole = 32;
    p.min_steps = 8;
    // two work-groups on each CU
    const int64_t total = 512;
    p.target = hkv < total ? (int)(total / hkv) : 1;
    const int64_t most = steps <= p.whole ? 1 : (steps + p.min_steps - 1) / p.min_steps;
    p.groups = 2 * p.target + tiles;
    if (most <= p.groups / tiles) p.groups = tiles * most;
    p.slots = most > 1 ? (4 * (int64_t)p.target < tiles * most ? 4 * (int64_t)p.target : tiles * most) : 0;
    p.joins = (int)(tiles < p.slots / 2 ? tiles : p.slots / 2);
    p.z = 4;
  }
  p.once = max_q * G <= p.tc;
  const size_t kept = (size_t)p.slots * hkv * p.tc;
  p.off_ml = kept * d * sizeof(float);
  p.off_rec = (p.off_ml + kept * 2 * sizeof(float) + 255) / 256 * 256;
  p.bytes = p.tc < 128 && p.slots ? p.off_rec + ((size_t)p.slots * sizeof(int4) + 255) / 256 * 256 : p.off_rec;
  return p;
}

}  // namespace

size_t attn_kv8_scratch_bytes(int64_t b, int64_t rows, int32_t hq, int32_t hkv, int32_t d, int32_t page,
                              int64_t max_pages, int64_t max_q) {
  return plan_of(b, rows, hq, hkv, d, page, max_pages, max_q).bytes;
}

template <int D, bool BF, int C, int NW>
static void launch_line(const AttnP& p, const Plan& pl, unsigned grid, unsigned joins, hipStream_t stream) {
  auto kernel = attn_kv8_line_kernel<D, BF, C, NW, false>;
  if constexpr (C == 16) {       // a sequence in tiles of 32 has more than 64 columns: never one tile
    if (pl.once) kernel = attn_kv8_line_kernel<D, BF, C, NW, true>;
  }
  kernel<<<grid, 64 * NW, 0, stream>>>(p);
  if (pl.slots) attn_kv8_join_kernel<D, C, BF><<<joins, 256, 0, stream>>>(p, pl.z);
}

template <int D, bool BF>
static hipError_t launch(const AttnP& p, const Plan& pl, hipStream_t stream) {
  const unsigned grid = (unsigned)(pl.groups * p.v.hkv), joins = (unsigned)pl.joins * p.v.hkv * pl.z;
  if (pl.tc == 16) {
    if (pl.waves == 8) launch_line<D, BF, 16, 8>(p, pl, grid, joins, stream);
    else launch_line<D, BF, 16, 2>(p, pl, grid, joins, stream);
  } else if (pl.tc == 32) {
    launch_line<D, BF, 32, 8>(p, pl, grid, joins, stream);
  } else {
    attn_kv8_tile_kernel<D, BF><<<grid, 256, 0, stream>>>(p);
    if (pl.slots) attn_kv8_join_kernel<D, 128, BF><<<joins, 256, 0, stream>>>(p, pl.z);
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
  p.whole = pl.whole;
  p.slots = (int32_t)pl.slots;
  p.part = (float*)scratch;
  p.part_ml = (float*)((char*)scratch + pl.off_ml);
  p.rec = pl.tc < 128 && pl.slots ? (int4*)((char*)scratch + pl.off_rec) : nullptr;
  if (a.d == 64) return bf ? launch<64, true>(p, pl, stream) : launch<64, false>(p, pl, stream);
  return bf ? launch<128, true>(p, pl, stream) : launch<128, false>(p, pl, stream);
}

}  // namespace awq
