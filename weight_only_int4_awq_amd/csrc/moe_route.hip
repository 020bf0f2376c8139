// Routing of tokens to experts and the sum of the experts' results.
//
// Routing.  Token t has one logit per expert; its topk experts are those of the
// largest logits (ties to the lower index), closed ones (-inf or NaN) never
// among them.  Weights, in fp32:
//   softmax  p_j = exp(x_j - max) / sum over all experts, or over the chosen ones
//   sigmoid  p_j = 1 / (1 + exp(-x_j)), divided by the chosen ones' sum when renormalized
// The plan sorts the slots (token * topk + choice) by expert, slots of one expert in
// their order: a counting sort whose result does not depend on any timing.
//
// What bounds it: the logits are read once and 16 bytes a slot written; up to some
// thousand tokens that is nothing beside the launches and the chain of one token
// (topk times a maximum over the lanes).  One wave takes a token, or four; a work-group of 16
// waves takes a chunk of tokens and leaves the chunk's number of slots of each expert;
// the second launch adds the chunks before its own and places its slots.  Up to
// kRouteSmall tokens one work-group does both in one launch.  Measured on the GPU: one token
// of 8 experts 3.1 us; 8191 tokens, 8 of 128 experts 5.4 + 6.4 us (3.1 MB: 0.6 us of bytes).
// Chunks of 64 tokens: 13.0 us for both against 12.7, and 11.4 against 10.0 for 500 tokens.
#include "moe_common.h"

namespace awq {

constexpr int kRouteWaves = 16;

struct RouteArgs {
  const void* logits;
  int32_t type;                       // 0 fp32, 1 fp16, 2 bf16
  int32_t t, e, topk, scoring, renorm;
  float scale;
  int32_t* ids;
  float* weights;
  int32_t* offsets;
  int32_t* row_slot;
  int32_t* slot_row;
  int32_t* counts;                    // [chunks][e]
  int32_t chunk, chunks;              // tokens of a work-group, work-groups
  bool vec;                           // rows of logits are 16-byte chunks
};

// A float's bits in the order of the values; -0 as +0, NaN as the lowest.
__device__ __forceinline__ uint32_t order_key(float x) {
  x = x + 0.0f;
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  if (x != x) return 0u;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
constexpr uint32_t kClosedKey = 0x007FFFFFu;      // -inf

__device__ __forceinline__ float load_logit(const RouteArgs& a, int64_t i) {
  if (a.type == 0) return reinterpret_cast<const float*>(a.logits)[i];
  const uint16_t b = reinterpret_cast<const uint16_t*>(a.logits)[i];
  return a.type == 1 ? h2f(b) : bf2f(b);
}

__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += shfl_xor_f(v, m);
  return v;
}

// A token's logits: lane l holds experts l, l + 64, ...; -inf behind the last.
template <int NPL>
__device__ __forceinline__ void load_token(const RouteArgs& a, int64_t t, int lane, float (&v)[NPL]) {
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int x = lane + 64 * i;
    v[i] = x < a.e ? load_logit(a, t * a.e + x) : -__builtin_inff();
  }
}

// One token by one wave.  Lane j < topk ends with choice j; -1 and weight 0 where fewer
// experts are open; all weights NaN where a logit is NaN.
template <int NPL>
__device__ __forceinline__ void route_token(const RouteArgs& a, const float (&v)[NPL], int lane, int& id, float& w) {
  uint32_t key[NPL];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    key[i] = order_key(v[i]);
    bad |= v[i] != v[i];
  }
  auto value = [](uint32_t k) {
    return __builtin_bit_cast(float, k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
  };
  float sum = 0.0f, mine = 0.0f;
  id = -1;
  w = 0.0f;
  const uint32_t first = lanes_max([&] {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i) m = m > key[i] ? m : key[i];
    return m;
  }());
  const float top = value(first);
  const bool any = first > kClosedKey;
  if (any && a.scoring == 0 && !a.renorm) {       // over all experts; a closed one adds exp(-inf) = 0
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (key[i] > kClosedKey) s += expf(value(key[i]) - top);
    sum = lanes_sum(s);
  }
  uint32_t best = first;
  for (int j = 0; j < a.topk && best > kClosedKey; ++j) {
    // the lowest expert that holds the maximum
    int at = -1;
#pragma unroll
    for (int i = NPL - 1; i >= 0; --i) {
      const uint64_t here = __ballot(key[i] == best);
      at = here ? 64 * i + __builtin_ctzll(here) : at;
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (at == lane + 64 * i) key[i] = 0;
    if (lane == j) {
      id = at;
      mine = value(best);
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i) m = m > key[i] ? m : key[i];
    best = lanes_max(m);
  }
  if (id >= 0) w = a.scoring == 0 ? expf(mine - top) : 1.0f / (1.0f + expf(-mine));
  if (a.renorm) sum = lanes_sum(w);
  if (a.renorm || a.scoring == 0) w = sum > 0.0f || sum != sum ? w / sum : 0.0f;
  w = id >= 0 ? w * a.scale : 0.0f;
  if (__ballot(bad)) w = __builtin_nanf("");
}

// ---- four tokens to a wave, one to each row of 16 lanes: up to 512 experts and 16 choices.
// Lane q of a row holds experts K q .. K q + K - 1.  With K = 8 a choice takes some 50 vector
// instructions for four tokens, 40 for one in the form above, and it is their issue that bounds
// many tokens (both launches, 8 choices: 8191 tokens of 128 experts 12.7 us against 15.5, 30000
// 22.9 against 36.6; 8191 of 256 experts 17.6 against 22.1, of 512 27.0 against 33.3).

#define AWQ_ROW_ALL(NAME, TYPE, OP)                                                                  \
  __device__ __forceinline__ TYPE NAME(TYPE x) {                                                           \
    auto other = [](TYPE v, auto ctrl) {                                                                   \
      return __builtin_bit_cast(TYPE, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v),           \
                                                                  decltype(ctrl)::value, 0xf, 0xf, true)); \
    };                                                                                                     \
    TYPE o = other(x, std::integral_constant<int, 0x128>{});                                               \
    x = OP;                                                                                                \
    o = other(x, std::integral_constant<int, 0x124>{});                                                    \
    x = OP;                                                                                                \
    o = other(x, std::integral_constant<int, 0x122>{});                                                    \
    x = OP;                                                                                                \
    o = other(x, std::integral_constant<int, 0x121>{});                                                    \
    return OP;                                                                                             \
  }
// over the 16 lanes of a row (rotations by 8, 4, 2, 1), in every lane; sums alike in every lane
AWQ_ROW_ALL(row_max, uint32_t, x > o ? x : o)
AWQ_ROW_ALL(row_min, uint32_t, x < o ? x : o)
AWQ_ROW_ALL(row_sum, float, x + o)
#undef AWQ_ROW_ALL

// Experts K q .. K q + K - 1 of token t; -inf behind the last.
template <int K>
__device__ __forceinline__ void load_row(const RouteArgs& a, int64_t t, int q, float (&v)[K]) {
  const int64_t at = t * a.e + K * q;
#pragma unroll
  for (int i = 0; i < K; ++i) v[i] = -__builtin_inff();
  if (!a.vec) {
#pragma unroll
    for (int i = 0; i < K; ++i)
      if (K * q + i < a.e) v[i] = load_logit(a, at + i);
    return;
  }
#pragma unroll
  for (int c = 0; c < K; c += 8) {
    if (K * q + c >= a.e) continue;                   // experts are a multiple of 8 here
    if (a.type == 0) {
      const float* p = reinterpret_cast<const float*>(a.logits) + at + c;
      const float4 l = *reinterpret_cast<const float4*>(p), h = *reinterpret_cast<const float4*>(p + 4);
      v[c] = l.x; v[c + 1] = l.y; v[c + 2] = l.z; v[c + 3] = l.w;
      v[c + 4] = h.x; v[c + 5] = h.y; v[c + 6] = h.z; v[c + 7] = h.w;
    } else {
      const uint4 r = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.logits) + at + c);
      const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint16_t b = (uint16_t)(i & 1 ? u[i / 2] >> 16 : u[i / 2]);
        v[c + i] = a.type == 1 ? h2f(b) : bf2f(b);
      }
    }
  }
}

// The tokens of a wave's four rows, as route_token.  Lane q < topk of a row ends with choice q.
template <int K>
__device__ __forceinline__ void route_rows(const RouteArgs& a, const float (&v)[K], int lane, int& id, float& w) {
  const int q = lane & 15;
  uint32_t key[K];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < K; ++i) {
    key[i] = order_key(v[i]);
    bad |= v[i] != v[i];
  }
  auto value = [](uint32_t k) {
    return __builtin_bit_cast(float, k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
  };
  auto largest = [&] {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < K; ++i) m = m > key[i] ? m : key[i];
    return row_max(m);
  };
  float sum = 0.0f, mine = 0.0f;
  id = -1;
  w = 0.0f;
  uint32_t best = largest();
  const float top = value(best);
  if (a.scoring == 0 && !a.renorm) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < K; ++i)
      if (key[i] > kClosedKey) s += expf(value(key[i]) - top);
    sum = row_sum(s);
  }
  for (int j = 0; j < a.topk && __ballot(best > kClosedKey); ++j) {
    uint32_t at = 0xFFFFu;
#pragma unroll
    for (int i = K - 1; i >= 0; --i) at = key[i] == best ? (uint32_t)(K * q + i) : at;
    at = row_min(at);
#pragma unroll
    for (int i = 0; i < K; ++i) key[i] = at == (uint32_t)(K * q + i) ? 0u : key[i];
    if (q == j && best > kClosedKey) {
      id = (int)at;
      mine = value(best);
    }
    best = largest();
  }
  if (id >= 0) w = a.scoring == 0 ? expf(mine - top) : 1.0f / (1.0f + expf(-mine));
  if (a.renorm) sum = row_sum(w);
  if (a.renorm || a.scoring == 0) w = sum > 0.0f || sum != sum ? w / sum : 0.0f;
  w = id >= 0 ? w * a.scale : 0.0f;
  if ((__ballot(bad) >> (lane & 48)) & 0xFFFF) w = __builtin_nanf("");
}

// Slots [s0, s1) of the chunk, wave by wave in runs of 64: their ranks among the slots
// of the same expert.  `hist` [waves][e] in LDS, zeroed: afterwards the number of each
// wave's slots of every expert.  `ids` in LDS or global; calls put(slot, expert, rank).
template <class Ids, class Put>
__device__ __forceinline__ void rank_slots(int s0, int s1, int e, int wave, int lane, int bits, int* hist, Ids ids,
                                           Put put) {
  const int n = s1 - s0;
  const int per = ((n + kRouteWaves - 1) / kRouteWaves + 63) & ~63;
  const int a = s0 + wave * per;
  const int z = a + per < s1 ? a + per : s1;
  for (int s = a; s < z; s += 64) {
    const int slot = s + lane;
    const int id = slot < z ? ids(slot) : -1;
    uint64_t same = __ballot(id >= 0);
    for (int b = 0; b < bits; ++b) {
      const uint64_t m = __ballot((id >> b) & 1);
      same &= (id >> b) & 1 ? m : ~m;
    }
    if (id >= 0) {
      const uint64_t before = same & ((1ull << lane) - 1);
      volatile int* h = hist + wave * e + id;
      const int base = *h;
      put(slot, id, base + __builtin_popcountll(before));
      if ((same >> lane) == 1ull) *h = base + __builtin_popcountll(same);   // the last lane of the expert
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

// Tokens [t0, t1) by the work-group's waves, the next one's logits asked for ahead; choices to
// ids and weights, and each(token - t0, expert) in lane j for choice j.
template <int NPL, class Each>
__device__ __forceinline__ void route_chunk(const RouteArgs& a, int t0, int t1, int wave, int lane, Each each) {
  float next[NPL];
  if (t0 + wave < t1) load_token<NPL>(a, t0 + wave, lane, next);
  for (int t = t0 + wave; t < t1; t += kRouteWaves) {
    float v[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) v[i] = next[i];
    if (t + kRouteWaves < t1) load_token<NPL>(a, t + kRouteWaves, lane, next);
    int id;
    float w;
    route_token<NPL>(a, v, lane, id, w);
    if (lane < a.topk) {
      a.ids[(int64_t)t * a.topk + lane] = id;
      a.weights[(int64_t)t * a.topk + lane] = w;
      each(t - t0, id);
    }
  }
}

// Exclusive sums of tot[0 .. e) into start[0 .. e], by the first wave.
__device__ __forceinline__ void scan_experts(const int* tot, int* start, int e, int lane) {
  int carry = 0;
  for (int b = 0; b < e; b += 64) {
    const int x = b + lane < e ? tot[b + lane] : 0;
    const int inc = wave_scan(x);
    if (b + lane < e) start[b + lane] = carry + inc - x;
    carry += __builtin_amdgcn_readlane(inc, 63);
  }
  if (lane == 0) start[e] = carry;
}

// One work-group: choices, ranks and rows of up to kRouteSmall tokens.
// LDS: ids [t topk], rank [t topk], hist [waves][e], total [e], start [e + 1]
template <int NPL>
__global__ __launch_bounds__(kRouteWaves * 64) void moe_route_small_kernel(const RouteArgs a) {
  extern __shared__ int lds[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int slots = a.t * a.topk, e = a.e;
  int* ids = lds;
  int* rank = ids + slots;
  int* hist = rank + slots;
  int* tot = hist + kRouteWaves * e;
  int* start = tot + e;
  for (int i = tid; i < kRouteWaves * e; i += kRouteWaves * 64) hist[i] = 0;
  route_chunk<NPL>(a, 0, a.t, wave, lane, [&](int t, int id) { ids[t * a.topk + lane] = id; });
  __syncthreads();
  const int bits = 32 - __builtin_clz(e);
  rank_slots(0, slots, e, wave, lane, bits, hist, [&](int s) { return ids[s]; },
             [&](int s, int, int r) { rank[s] = r; });
  __syncthreads();
  for (int x = tid; x < e; x += kRouteWaves * 64) {     // before each wave's slots: those of the waves before it
    int sum = 0;
    for (int w = 0; w < kRouteWaves; ++w) {
      const int c = hist[w * e + x];
      hist[w * e + x] = sum;
      sum += c;
    }
    tot[x] = sum;
  }
  __syncthreads();
  if (wave == 0) scan_experts(tot, start, e, lane);
  __syncthreads();
  for (int x = tid; x <= e; x += kRouteWaves * 64) a.offsets[x] = start[x];
  const int per = ((slots + kRouteWaves - 1) / kRouteWaves + 63) & ~63;
  for (int s = tid; s < slots; s += kRouteWaves * 64) {
    const int id = ids[s];
    int row = -1;
    if (id >= 0) {
      row = start[id] + hist[(s / per) * e + id] + rank[s];
      a.row_slot[row] = s;
    }
    a.slot_row[s] = row;
  }
}

template <int NPL>
__global__ __launch_bounds__(kRouteWaves * 64) void moe_route_kernel(const RouteArgs a) {
  extern __shared__ int hist[];                       // [e]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int t0 = blockIdx.x * a.chunk, t1 = t0 + a.chunk < a.t ? t0 + a.chunk : a.t;
  for (int i = tid; i < a.e; i += kRouteWaves * 64) hist[i] = 0;
  __syncthreads();
  route_chunk<NPL>(a, t0, t1, wave, lane, [&](int, int id) {
    if (id >= 0) atomicAdd(&hist[id], 1);             // a count: the order of the additions does not show
  });
  __syncthreads();
  for (int i = tid; i < a.e; i += kRouteWaves * 64) a.counts[(int64_t)blockIdx.x * a.e + i] = hist[i];
}

// The same by rows of lanes.
template <int K>
__global__ __launch_bounds__(kRouteWaves * 64) void moe_route_rows_kernel(const RouteArgs a) {
  __shared__ int hist[16 * K];
  const int tid = threadIdx.x, lane = tid & 63, q = lane & 15;
  const int t0 = blockIdx.x * a.chunk, t1 = t0 + a.chunk < a.t ? t0 + a.chunk : a.t;
  if (tid < a.e) hist[tid] = 0;
  __syncthreads();
  for (int t = t0 + (tid >> 4); t - (lane >> 4) < t1; t += kRouteWaves * 4) {
    float v[K];
    load_row<K>(a, t < t1 ? t : t1 - 1, q, v);
    int id;
    float w;
    route_rows<K>(a, v, lane, id, w);
    if (t < t1 && q < a.topk) {
      a.ids[(int64_t)t * a.topk + q] = id;
      a.weights[(int64_t)t * a.topk + q] = w;
      if (id >= 0) atomicAdd(&hist[id], 1);
    }
  }
  __syncthreads();
  if (tid < a.e) a.counts[(int64_t)blockIdx.x * a.e + tid] = hist[tid];
}

// Places the slots of chunk blockIdx.x.  LDS: hist [waves][e], before [e], total [e], start [e + 1]
__global__ __launch_bounds__(kRouteWaves * 64) void moe_place_kernel(const RouteArgs a) {
  extern __shared__ int lds[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int e = a.e, c = blockIdx.x;
  int* hist = lds;
  int* before = hist + kRouteWaves * e;
  int* tot = before + e;
  int* start = tot + e;
  for (int i = tid; i < kRouteWaves * e; i += kRouteWaves * 64) hist[i] = 0;
  for (int i = tid; i < e; i += kRouteWaves * 64) before[i] = tot[i] = 0;
  __syncthreads();
  // slots of each expert in the chunks before this one, and in all: waves take runs of
  // chunks, lanes experts
  {
    const int per = (a.chunks + kRouteWaves - 1) / kRouteWaves;
    const int q0 = wave * per, q1 = q0 + per < a.chunks ? q0 + per : a.chunks;
    for (int x = lane; x < e; x += 64) {
      int b = 0, all = 0;
#pragma unroll 8
      for (int q = q0; q < q1; ++q) {
        const int n = a.counts[(int64_t)q * e + x];
        all += n;
        b += q < c ? n : 0;
      }
      if (b) atomicAdd(&before[x], b);
      if (all) atomicAdd(&tot[x], all);
    }
  }
  __syncthreads();
  if (wave == 0) scan_experts(tot, start, e, lane);
  const int bits = 32 - __builtin_clz(e);
  const int64_t t0 = (int64_t)c * a.chunk, t1 = t0 + a.chunk < a.t ? t0 + a.chunk : a.t;
  const int s0 = (int)(t0 * a.topk), s1 = (int)(t1 * a.topk);
  rank_slots(s0, s1, e, wave, lane, bits, hist, [&](int s) { return a.ids[s]; },
             [&](int s, int, int r) { a.slot_row[s] = r; });
  __syncthreads();
  for (int x = tid; x < e; x += kRouteWaves * 64) {
    int sum = start[x] + before[x];
    for (int w = 0; w < kRouteWaves; ++w) {
      const int n = hist[w * e + x];
      hist[w * e + x] = sum;
      sum += n;
    }
  }
  if (c == 0)
    for (int x = tid; x <= e; x += kRouteWaves * 64) a.offsets[x] = start[x];
  __syncthreads();
  // the same wave and lane as in rank_slots: a slot's rank is read by the lane that wrote it
  const int per = ((s1 - s0 + kRouteWaves - 1) / kRouteWaves + 63) & ~63;
  const int b0 = s0 + wave * per, b1 = b0 + per < s1 ? b0 + per : s1;
  for (int s = b0 + lane; s < b1; s += 64) {
    const int id = a.ids[s];
    int row = -1;
    if (id >= 0) {
      row = hist[wave * e + id] + a.slot_row[s];
      a.row_slot[row] = s;
    }
    a.slot_row[s] = row;
  }
}

// Tokens one work-group takes: all of up to kRouteSmall, else chunks of at least 32 in at
// most 256 work-groups.
constexpr int kRouteSmall = 48;
static int route_chunk_tokens(int64_t t) {
  int64_t c = (t + 255) / 256;
  c = (c + 15) / 16 * 16;
  return (int)(c < 32 ? 32 : c);
}
static bool route_small(int64_t t) { return t <= kRouteSmall; }

size_t moe_route_scratch_bytes(int64_t t, int32_t e) {
  if (route_small(t)) return 0;
  const int64_t c = route_chunk_tokens(t);
  return (size_t)((t + c - 1) / c) * e * 4;
}

template <int NPL>
static hipError_t route_npl(RouteArgs& a, hipStream_t stream) {
  const int threads = kRouteWaves * 64;
  if (route_small(a.t)) {
    const size_t lds = ((size_t)2 * a.t * a.topk + (size_t)(kRouteWaves + 2) * a.e + 1) * 4;
    if (lds > 65536) {
      const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(moe_route_small_kernel<NPL>),
                                               hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
      if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(moe_route_small_kernel<NPL>, dim3(1), dim3(threads), lds, stream, a);
    return hipGetLastError();
  }
  bool rows = false;
  if constexpr (NPL <= 8) {
    rows = a.topk <= 16;
    constexpr int K = NPL <= 2 ? 8 : 4 * NPL;         // experts of a lane
    if (rows) hipLaunchKernelGGL(moe_route_rows_kernel<K>, dim3(a.chunks), dim3(threads), 0, stream, a);
  }
  if (!rows) hipLaunchKernelGGL(moe_route_kernel<NPL>, dim3(a.chunks), dim3(threads), (size_t)a.e * 4, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const size_t lds = ((size_t)(kRouteWaves + 3) * a.e + 1) * 4;
  if (lds > 65536) {
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(moe_place_kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                            (int)lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(moe_place_kernel, dim3(a.chunks), dim3(threads), lds, stream, a);
  return hipGetLastError();
}

hipError_t launch_moe_route(const void* logits, int32_t type, int64_t t, int32_t e, int32_t topk, int32_t scoring,
                            bool renorm, float scale, int32_t* ids, float* weights, int32_t* offsets,
                            int32_t* row_slot, int32_t* slot_row, void* scratch, hipStream_t stream) {
  RouteArgs a{logits, type, (int32_t)t, e, topk, scoring, renorm ? 1 : 0, scale, ids, weights, offsets, row_slot,
              slot_row, (int32_t*)scratch, 0, 0, false};
  a.vec = e % 8 == 0 && (reinterpret_cast<uintptr_t>(logits) & 15) == 0;
  a.chunk = route_chunk_tokens(t);
  a.chunks = (int)((t + a.chunk - 1) / a.chunk);
  if (e <= 64) return route_npl<1>(a, stream);
  if (e <= 128) return route_npl<2>(a, stream);
  if (e <= 256) return route_npl<4>(a, stream);
  if (e <= 512) return route_npl<8>(a, stream);
  return route_npl<16>(a, stream);
}

// ---------------------------------------------------------------- combination
// y[t] = residual[t] + sum_j w[t][j] rows[slot_row[t][j]], in fp32 in the order of j, one
// rounding at the end.  A slot without a row adds its weight times zero: nothing, or NaN
// where the routing left NaN.  Bytes bound it: every row read once, y written once.  A
// thread takes 8 columns (16 bytes) of one token and asks for up to 8 rows at once.  8191 tokens
// with 8 rows of 4096 and a residual (665 MB) 130 us, 5.1 TB/s; 64 tokens of 8 x 2048 4.4 us
// (launch and latency).
template <bool BF>
__device__ __forceinline__ float load_act(uint32_t b) {
  return BF ? bf2f((uint16_t)b) : h2f((uint16_t)b);
}

template <bool BF, bool VEC>
__global__ __launch_bounds__(256) void moe_combine_kernel(const uint16_t* __restrict__ rows, int64_t cap,
                                                          const float* __restrict__ weights,
                                                          const int32_t* __restrict__ slot_row,
                                                          const uint16_t* __restrict__ residual, int64_t t, int64_t n,
                                                          int topk, int64_t per_token, uint16_t* __restrict__ y) {
  constexpr int C = VEC ? 8 : 1;
  const int64_t unit = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t tok = unit / per_token;
  if (tok >= t) return;
  const int64_t col = (unit - tok * per_token) * C;
  float acc[C];
  auto add = [&](const uint16_t* p, float w) {
    if constexpr (VEC) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[2 * i] = __builtin_fmaf(w, load_act<BF>(u[i] & 0xFFFFu), acc[2 * i]);
        acc[2 * i + 1] = __builtin_fmaf(w, load_act<BF>(u[i] >> 16), acc[2 * i + 1]);
      }
    } else {
      acc[0] = __builtin_fmaf(w, load_act<BF>(*p), acc[0]);
    }
  };
#pragma unroll
  for (int i = 0; i < C; ++i) acc[i] = 0.0f;
  if (residual) add(residual + tok * n + col, 1.0f);
  const int32_t* sr = slot_row + tok * topk;
  const float* wt = weights + tok * topk;
  for (int j0 = 0; j0 < topk; j0 += 8) {
    uint4 v[8];
    float w[8];
    bool on[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int jj = j0 + j < topk ? j0 + j : topk - 1;
      const int64_t r = sr[jj];
      w[j] = j0 + j < topk ? wt[jj] : 0.0f;
      on[j] = j0 + j < topk && r >= 0 && r < cap;
      const uint16_t* p = rows + (on[j] ? r : 0) * n + col;
      v[j] = make_uint4(0, 0, 0, 0);
      if (on[j]) {
        if constexpr (VEC) v[j] = *reinterpret_cast<const uint4*>(p);
        else v[j].x = *p;
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t u[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
      for (int i = 0; i < C; ++i)
        acc[i] = __builtin_fmaf(w[j], load_act<BF>(i & 1 ? u[i / 2] >> 16 : u[i / 2] & 0xFFFFu), acc[i]);
    }
  }
  if constexpr (VEC) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      u[i] = (uint32_t)f2act(acc[2 * i], BF) | (uint32_t)f2act(acc[2 * i + 1], BF) << 16;
    *reinterpret_cast<uint4*>(y + tok * n + col) = make_uint4(u[0], u[1], u[2], u[3]);
  } else {
    y[tok * n + col] = f2act(acc[0], BF);
  }
}

bool moe_combine_vec(const uint16_t* rows, const uint16_t* residual, const uint16_t* y, int64_t n) {
  auto al = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  return n % 8 == 0 && al(rows) && al(residual) && al(y);
}

hipError_t launch_moe_combine(const uint16_t* rows, int64_t cap, const float* weights, const int32_t* slot_row,
                              const uint16_t* residual, int64_t t, int64_t n, int32_t topk, bool bf, uint16_t* y,
                              hipStream_t stream) {
  const bool vec = moe_combine_vec(rows, residual, y, n);
  const int64_t per = vec ? n / 8 : n;
  const dim3 grid((unsigned)((t * per + 255) / 256));
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, rows, cap, weights, slot_row, residual, t, n, topk, per, y);
    return hipGetLastError();
  };
  if (bf) return vec ? go(moe_combine_kernel<true, true>) : go(moe_combine_kernel<true, false>);
  return vec ? go(moe_combine_kernel<false, true>) : go(moe_combine_kernel<false, false>);
}

}  // namespace awq
