// swiglu_route.hip -- the router of a mixture-of-experts block: which experts a
// token goes to and with what weight, and the order that puts the tokens of an
// expert next to each other.
//
// For token t with logits x (E of them, -inf or NaN: masked off), the chosen
// experts are the k largest logits, the lowest index first among equals, and
//   weight_i = exp(x_i - m) / S,  m = max x,
//   S = sum of exp(x_j - m) over the chosen ones (renormalize) or over all E.
// A token with fewer than k open experts has -1 and weight 0 in the places
// left over.  Slot t k + i then belongs to expert experts[t, i]; the slots
// sorted by (expert, slot) are `rows`, expert e's at [offsets[e],
// offsets[e + 1]), and -1 fills what follows offsets[E].
//
// The work is a few operations a logit: a call is bound by its launches and by
// the latency of its memory accesses.  Up to kRouteSmall slots one workgroup
// does all of it in one launch; beyond that one launch chooses and counts, a
// second one places.  The order comes from counts and ranks, never from the
// arrival of atomics, so it is the same in every run.  8191 tokens, 128 experts, 8
// choices of bf16 logits: 4.8 to 5.1 us to choose, 5.4 to 6.2 to place, 10.0 to
// 10.9 a call (fp32: 6.0 to 6.8 and 5.6 to 6.8, 10.9 to 12.2 a call); one token: 4.2 us.
#include "swiglu_internal.h"
#include "swiglu_ops_device.hpp"

#include <algorithm>
#include <type_traits>

namespace swiglu {

constexpr float kNegInf = -__builtin_inff();

__device__ __forceinline__ float logit_value(float x) { return x == x ? x : kNegInf; }

// C logits of the lane: indices [C gl, C gl + C) of a row of E.
template <int C>
__device__ __forceinline__ void load_logits(const float* row, int E, int i0, bool vec,
                                            float (&x)[C]) {
  if (vec) {
#pragma unroll
    for (int j = 0; j < C; j += 4) {
      const bool in = i0 + j < E;  // E % 4 == 0
      const f32x4 v = __builtin_bit_cast(f32x4, in ? load16(row + i0 + j) : u32x4{0, 0, 0, 0});
#pragma unroll
      for (int q = 0; q < 4; ++q) x[j + q] = in ? logit_value(v[q]) : kNegInf;
    }
  } else {
#pragma unroll
    for (int j = 0; j < C; ++j) x[j] = i0 + j < E ? logit_value(row[i0 + j]) : kNegInf;
  }
}
template <int C>
__device__ __forceinline__ void load_logits(const uint16_t* row, int E, int i0, bool vec,
                                            float (&x)[C]) {
  if (vec) {
#pragma unroll
    for (int j = 0; j < C; j += 8) {
      const bool in = i0 + j < E;  // E % 8 == 0
      const u32x4 v = in ? load16(row + i0 + j) : u32x4{0, 0, 0, 0};
#pragma unroll
      for (int q = 0; q < 8; ++q)
        x[j + q] = in ? logit_value(bf16_to_float((uint16_t)(v[q / 2] >> (16 * (q & 1))))) : kNegInf;
    }
  } else {
#pragma unroll
    for (int j = 0; j < C; ++j)
      x[j] = i0 + j < E ? logit_value(bf16_to_float(row[i0 + j])) : kNegInf;
  }
}

struct RouteArgs {
  const void* logits;
  float* weights;
  int32_t* experts;
  int32_t* offsets;
  int32_t* rows;
  int32_t* counts;  // workspace: [workgroups, E rounded up to 4]
  int T, E, k, renorm;
  int vec;          // rows are 16-byte aligned and a multiple of 16 bytes
  int tokens;       // tokens of a workgroup
};

// The experts of one token on G lanes (C logits each; lane order is index
// order, so the lowest of several equal maxima is in the lowest lane that has
// one).  Every lane takes part in the cross-lane steps; `in` says whether the
// token exists.  Lane gl < k ends up with choice gl, for k <= G.  The chain
// from one choice to the next is the bound of a call, so it holds only what it
// has to: the winner notes its index in `picked` (LDS, G places of this
// token), the exponentials wait until all choices are known.
template <typename In, int G, int C>
__device__ __forceinline__ void route_token(const RouteArgs& a, int t, bool in, int* picked,
                                            int32_t& expert, float& weight) {
  const int lane = threadIdx.x & 63, gl = lane & (G - 1);
  float x[C];
  load_logits<C>((const In*)a.logits + (size_t)(in ? t : 0) * a.E, in ? a.E : 0, gl * C, a.vec, x);
  float top = 0.0f, total = 0.0f, mine = kNegInf;
  for (int i = 0; i < a.k; ++i) {
    float v = x[0];
    int bj = 0;
#pragma unroll
    for (int j = 1; j < C; ++j)
      if (x[j] > v) v = x[j], bj = j;
    const float best = group_max<G>(v);
    if (i == 0) {
      // all E terms, before any is taken out; an infinite maximum (equal
      // shares of what is infinite) has no finite difference to itself
      top = best > kNegInf ? best : 0.0f;
      if (!a.renorm) {
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < C; ++j) s += x[j] == top ? 1.0f : expf(x[j] - top);
        total = group_sum<G>(s);
      }
    }
    if (gl == i) mine = best;
    const unsigned long long group = (G == 64 ? ~0ull : ((1ull << (G & 63)) - 1)) << (lane & ~(G - 1));
    if (lane == __ffsll(__ballot(v == best) & group) - 1) {
      picked[i] = gl * C + bj;
#pragma unroll
      for (int j = 0; j < C; ++j)
        if (j == bj) x[j] = kNegInf;
    }
  }
  __builtin_amdgcn_wave_barrier();  // other lanes' notes: no read moves above this
  const bool open = mine > kNegInf;
  const float p = !open ? 0.0f : (mine == top ? 1.0f : expf(mine - top));
  if (a.renorm) total = group_sum<G>(p);
  expert = open && gl < a.k ? picked[gl] : -1;  // written by this wave: in order
  weight = open ? p / total : 0.0f;
}

// The same for bf16 logits.  A logit and its index fit one whole number, the
// value's bits made monotone over 1023 - index, so the maximum alone names the
// winner: no vote, no note, about half the operations a choice (the launch that
// chooses, timed in turn: 5.7 us without, 4.6 us with them, at 8191 tokens, 128
// experts, 8 choices).
// 0 is a closed place; every open logit's number is above it.
__device__ __forceinline__ uint32_t route_key(float x, int index) {
  const uint32_t b = __builtin_bit_cast(uint32_t, x == 0.0f ? 0.0f : x);  // one zero
  const uint32_t m = (b ^ (uint32_t)((int)b >> 31 | (int)0x80000000)) & 0xffff0000u;
  return x > kNegInf ? m | (uint32_t)(kMaxExperts - 1 - index) : 0u;
}
__device__ __forceinline__ float route_key_value(uint32_t key) {
  const uint32_t m = key & 0xffff0000u;
  return __builtin_bit_cast(float, m & 0x80000000u ? m ^ 0x80000000u : ~m & 0xffff0000u);
}
template <int G, int C>
__device__ __forceinline__ void route_token_keys(const RouteArgs& a, int t, bool in,
                                                 int32_t& expert, float& weight) {
  const int gl = threadIdx.x & (G - 1);
  float x[C];
  load_logits<C>((const uint16_t*)a.logits + (size_t)(in ? t : 0) * a.E, in ? a.E : 0, gl * C,
                 a.vec, x);
  uint32_t key[C], mine = 0;
#pragma unroll
  for (int j = 0; j < C; ++j) key[j] = route_key(x[j], gl * C + j);
  float top = 0.0f, total = 0.0f;
  for (int i = 0; i < a.k; ++i) {
    uint32_t v = key[0];
#pragma unroll
    for (int j = 1; j < C; ++j) v = max(v, key[j]);
    const uint32_t best = group_max<G>(v);
    if (i == 0) {  // as in route_token
      top = best ? route_key_value(best) : 0.0f;
      if (!a.renorm) {
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < C; ++j) s += x[j] == top ? 1.0f : expf(x[j] - top);
        total = group_sum<G>(s);
      }
    }
    if (gl == i) mine = best;
#pragma unroll
    for (int j = 0; j < C; ++j)
      if (key[j] == best) key[j] = 0;
  }
  const float y = route_key_value(mine);
  const float p = !mine ? 0.0f : (y == top ? 1.0f : expf(y - top));
  if (a.renorm) total = group_sum<G>(p);
  expert = mine && gl < a.k ? (int32_t)(kMaxExperts - 1) - (int32_t)(mine & 0xffffu) : -1;
  weight = mine ? p / total : 0.0f;
}

// ---- scored choice -------------------------------------------------------------------
// swiglu_route_scored: with a score s of each logit (its sigmoid, or the softmax over the
// open ones) and c = s + bias, the k largest c of the kept groups are chosen, and s is
// the weight.  Scores, sums and comparisons are in 64 bits: neighbours among some hundred
// scores between 0 and 1 come as close as fp32 rounds exp, and the choice is to be that
// of the definition.
struct NoScore {};
template <int CTRL>
__device__ __forceinline__ double dpp_d(double v) {
  const uint64_t x = __builtin_bit_cast(uint64_t, v);
  const int lo = (int)(uint32_t)x, hi = (int)(uint32_t)(x >> 32);
  const uint32_t a = (uint32_t)__builtin_amdgcn_update_dpp(lo, lo, CTRL, 0xf, 0xf, false);
  const uint32_t b = (uint32_t)__builtin_amdgcn_update_dpp(hi, hi, CTRL, 0xf, 0xf, false);
  return __builtin_bit_cast(double, (uint64_t)b << 32 | a);
}
// over aligned groups of G lanes (16, 32 or 64); every lane receives the same bits
template <int G, typename F>
__device__ __forceinline__ double group_fold(double v, F f) {
  v = f(v, dpp_d<kDppXor1>(v));
  v = f(v, dpp_d<kDppXor2>(v));
  v = f(v, dpp_d<kDppHalfMirror>(v));
  v = f(v, dpp_d<kDppMirror>(v));
  if (G >= 32) v = f(v, __shfl_xor(v, 16));
  if (G >= 64) v = f(v, __shfl_xor(v, 32));
  return v;
}
constexpr double kNegInfD = -__builtin_inf();
__device__ __forceinline__ double larger(double a, double b) { return a > b ? a : b; }

// LDS of one token.
template <int N>
struct ScoreRoom {
  double c[N];             // of all experts
  double value[kMaxGroups];
  double picked[64];       // scores of the chosen ones
  int index[64];
};

// As route_token.
template <typename In, int G, int C>
__device__ __forceinline__ void route_token_scored(const RouteArgs& a, const RouteScore& sc, int t,
                                                   bool in, ScoreRoom<G * C>& room,
                                                   int32_t& expert, float& weight) {
  const int lane = threadIdx.x & 63, gl = lane & (G - 1);
  float x[C];
  load_logits<C>((const In*)a.logits + (size_t)(in ? t : 0) * a.E, in ? a.E : 0, gl * C, a.vec, x);
  double s[C], c[C];
  if (sc.sigmoid) {
#pragma unroll
    for (int j = 0; j < C; ++j) s[j] = 1.0 / (1.0 + exp(-(double)x[j]));
  } else {
    float m = x[0];
#pragma unroll
    for (int j = 1; j < C; ++j) m = fmaxf(m, x[j]);
    m = group_max<G>(m);
    m = m > kNegInf ? m : 0.0f;
    double total = 0.0;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      s[j] = x[j] == m ? 1.0 : exp((double)x[j] - (double)m);
      total += s[j];
    }
    total = group_fold<G>(total, [](double u, double v) { return u + v; });
#pragma unroll
    for (int j = 0; j < C; ++j) s[j] = total > 0.0 ? s[j] / total : 0.0;
  }
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int e = gl * C + j;
    const double v = s[j] + (sc.bias && e < a.E ? (double)sc.bias[e] : 0.0);
    c[j] = x[j] > kNegInf && v == v ? v : kNegInfD;
  }
  if (sc.groups > 1) {
    const int size = a.E / sc.groups;
#pragma unroll
    for (int j = 0; j < C; ++j) room.c[gl * C + j] = c[j];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    for (int g = gl; g < sc.groups; g += G) {
      double first = kNegInfD, second = kNegInfD;
      for (int i = 0; i < size; ++i) {
        const double v = room.c[g * size + i];
        second = larger(second, v < first ? v : first);
        first = larger(first, v);
      }
      room.value[g] = sc.group_best == 2 && second > kNegInfD ? first + second : first;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int e = gl * C + j;
      if (e >= a.E) continue;
      const int mine = e / size;
      const double value = room.value[mine];
      int before = 0;
      for (int g = 0; g < sc.groups; ++g) {
        const double v = room.value[g];
        before += v > value || (v == value && g < mine);
      }
      if (before >= sc.top_groups) c[j] = kNegInfD;
    }
  }
  bool open = false;
  for (int i = 0; i < a.k; ++i) {
    double v = c[0], p = s[0];
    int bj = 0;
#pragma unroll
    for (int j = 1; j < C; ++j)
      if (c[j] > v) v = c[j], p = s[j], bj = j;
    const double best = group_fold<G>(v, larger);
    if (gl == i) open = best > kNegInfD;
    const unsigned long long group = (G == 64 ? ~0ull : ((1ull << (G & 63)) - 1)) << (lane & ~(G - 1));
    if (lane == __ffsll(__ballot(v == best) & group) - 1) {
      room.index[i] = gl * C + bj;
      room.picked[i] = p;
#pragma unroll
      for (int j = 0; j < C; ++j)
        if (j == bj) c[j] = kNegInfD;
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  open = open && gl < a.k;
  double p = open ? room.picked[gl] : 0.0;
  expert = open ? room.index[gl] : -1;
  if (a.renorm) {
    const double total = group_fold<G>(p, [](double u, double v) { return u + v; });
    p = total > 0.0 ? p / total : 0.0;
  }
  weight = open ? (float)(p * (double)sc.scale) : 0.0f;
}

// Tokens [t0, t1) by the workgroup: results to memory, slots counted in hist,
// and with `slots` the choices kept in LDS too.
template <typename In, int G, int C, typename Score>
__device__ __forceinline__ void route_tokens(const RouteArgs& a, const Score& score, int t0, int t1,
                                             int* picked, ScoreRoom<G * C>* rooms, int* hist,
                                             int* slots) {
  const int per = blockDim.x / G, gl = threadIdx.x & (G - 1), first = (int)threadIdx.x / G;
  for (int t = t0 + first; t - first < t1; t += per) {
    const bool in = t < t1;
    int32_t e;
    float w;
    if constexpr (!std::is_same_v<Score, NoScore>)
      route_token_scored<In, G, C>(a, score, t, in, rooms[first], e, w);
    else if constexpr (std::is_same_v<In, uint16_t>)
      route_token_keys<G, C>(a, t, in, e, w);
    else
      route_token<In, G, C>(a, t, in, picked + (threadIdx.x & ~(G - 1)), e, w);
    if (in && gl < a.k) {
      const size_t s = (size_t)t * a.k + gl;
      a.experts[s] = e;
      a.weights[s] = w;
      if (slots) slots[s] = e;
      if (e >= 0) atomicAdd(hist + e, 1);
    }
  }
}

// Lanes of the wave with the same expert as this one.
__device__ __forceinline__ unsigned long long same_expert(int e, int E) {
  unsigned long long m = ~0ull;
  for (int b = 1; b <= E; b <<= 1) {  // -1 counts as E
    const unsigned long long one = __ballot((e < 0 ? E : e) & b);
    m &= ((e < 0 ? E : e) & b) ? one : ~one;
  }
  return m;
}

// The slots [begin, end) of this wave out of the workgroup's [s0, s1), and the
// expert of the lane's first one, which is fetched ahead.
struct RouteShare {
  int begin, end, first;
};
__device__ __forceinline__ RouteShare route_share(const int32_t* experts, int s0, int s1) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nw = blockDim.x >> 6;
  const int per = ((s1 - s0 + nw - 1) / nw + 63) / 64 * 64;
  RouteShare h{s0 + wave * per, 0, -1};
  h.end = min(h.begin + per, s1);
  if (h.begin + lane < h.end) h.first = experts[h.begin + lane];
  return h;
}

// Slots [s0, s1) into their places: `next` holds, for every wave and expert,
// the next free place (already advanced past the earlier slots).
__device__ __forceinline__ void route_place(const RouteArgs& a, const int32_t* experts,
                                            const RouteShare& h, int s0, int s1, int total,
                                            int* next) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int b = h.begin, e = h.end;
  const int n = a.T * a.k;
  int* mine = next + wave * a.E;
  for (int s = b + lane; s - lane < e; s += 64) {
    const int x = s - lane == b ? h.first : (s < e ? experts[s] : -1);
    const unsigned long long same = same_expert(x, a.E);
    if (x >= 0 && x < a.E) {
      const int rank = __popcll(same & ((1ull << lane) - 1));
      const int at = mine[x] + rank;
      if (at >= 0 && at < n) a.rows[at] = s;
      __builtin_amdgcn_wave_barrier();  // every lane has read its place
      if (rank == 0) mine[x] += __popcll(same);
    }
  }
  for (int s = s0 + (int)threadIdx.x; s < s1; s += blockDim.x)
    if (s >= total) a.rows[s] = -1;
}

// Counts of each wave's share into next[wave][expert].
__device__ __forceinline__ void route_count(const RouteArgs& a, const int32_t* experts,
                                            const RouteShare& h, int* next) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int s = h.begin + lane; s < h.end; s += 64) {
    const int x = s - lane == h.begin ? h.first : experts[s];
    if (x >= 0 && x < a.E) atomicAdd(next + wave * a.E + x, 1);
  }
}

// offset[e] = sum of count[0 .. e) for e <= E, by the first wave.
__device__ __forceinline__ void route_scan(const int* count, int* offset, int E) {
  const int lane = threadIdx.x;
  if (lane >= 64) return;
  int before = 0;
  for (int c = 0; c < E; c += 64) {
    const int n = c + lane < E ? count[c + lane] : 0;
    const int incl = wave_scan(n);
    if (c + lane < E) offset[c + lane] = before + incl - n;
    before += __builtin_amdgcn_readlane(incl, 63);
  }
  if (lane == 0) offset[E] = before;
}

// Turns counts per wave into places: expert x of wave w starts at offset[x] plus
// what earlier workgroups (`base`, if there are any) and earlier waves hold.
// The counts of all NW waves are read before the first one is written.
template <int NW>
__device__ __forceinline__ void route_bases(int* next, const int* offset, const int* base, int E) {
  const int nw = blockDim.x >> 6;
  for (int x = threadIdx.x; x < E; x += blockDim.x) {
    int n[NW];
#pragma unroll
    for (int w = 0; w < NW; ++w) n[w] = w < nw ? next[w * E + x] : 0;
    int at = offset[x] + (base ? base[x] : 0);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (w < nw) next[w * E + x] = at;
      at += n[w];
    }
  }
}

// Slots that one workgroup still takes by itself.  Measured (us of GPU time, one
// launch / two): bf16, 64 experts, 8 choices: 256 slots 4.6 / 6.8, 512 6.4 / 7.0,
// 768 8.8 / 7.0; fp32, whose choices take longer: 64 experts, 6 choices: 252 7.0 /
// 7.3, 510 9.1 / 7.4; 256 experts, 8 choices: 128 6.3 / 8.4, 256 9.3 / 8.6, 512
// 15.2 / 8.8.  So the bound is right for bf16, up to 512 slots late for fp32; a
// second launch also adds 1 to 2 us of the caller's time.
constexpr long long kRouteSmall = 512;

// ---- one workgroup does everything -------------------------------------------------
constexpr int kSmallThreads = 512;
template <typename In, int G, int C, typename Score>
__global__ __launch_bounds__(kSmallThreads) void route_small_kernel(RouteArgs a, Score score) {
  constexpr bool kScored = !std::is_same_v<Score, NoScore>;
  __shared__ __attribute__((aligned(16))) ScoreRoom<G * C> rooms[kScored ? kSmallThreads / G : 1];
  __shared__ __attribute__((aligned(16))) int next[kSmallThreads / 64 * G * C];
  __shared__ __attribute__((aligned(16))) int hist[G * C];
  __shared__ __attribute__((aligned(16))) int offset[G * C + 1];
  __shared__ __attribute__((aligned(16))) int picked[kSmallThreads];
  __shared__ __attribute__((aligned(16))) int slots[kRouteSmall];
  const int nw = blockDim.x >> 6, n = a.T * a.k;
  for (int i = threadIdx.x; i < nw * a.E; i += blockDim.x) next[i] = 0;
  for (int i = threadIdx.x; i < a.E; i += blockDim.x) hist[i] = 0;
  __syncthreads();
  route_tokens<In, G, C>(a, score, 0, a.T, picked, rooms, hist, slots);
  __syncthreads();
  const RouteShare share = route_share(slots, 0, n);
  route_count(a, slots, share, next);
  route_scan(hist, offset, a.E);
  __syncthreads();
  route_bases<kSmallThreads / 64>(next, offset, nullptr, a.E);
  for (int i = threadIdx.x; i <= a.E; i += blockDim.x) a.offsets[i] = offset[i];
  __syncthreads();
  route_place(a, slots, share, 0, n, offset[a.E], next);
}

// ---- many tokens: choose and count, then place ---------------------------------------
// The counts are [blocks, stride], stride = E rounded up to 4: a thread of the
// second launch adds up four experts' counts over every RP-th workgroup, eight
// 16-byte loads in flight, and LDS adds up the threads.  (One wave an expert
// with a scan over the workgroups took 1.1 us more at 128 experts and 8191
// tokens, 3.0 at 200 and 2000.)
constexpr int kSelectThreads = 512, kPlaceThreads = 1024;
constexpr int kMaxRouteBlocks = 256;  // one on every CU
template <typename In, int G, int C, typename Score>
__global__ __launch_bounds__(kSelectThreads) void route_select_kernel(RouteArgs a, Score score,
                                                                      int stride) {
  constexpr bool kScored = !std::is_same_v<Score, NoScore>;
  __shared__ __attribute__((aligned(16))) ScoreRoom<G * C> rooms[kScored ? kSelectThreads / G : 1];
  __shared__ __attribute__((aligned(16))) int hist[G * C];
  __shared__ __attribute__((aligned(16))) int picked[kSelectThreads];
  for (int i = threadIdx.x; i < a.E; i += blockDim.x) hist[i] = 0;
  __syncthreads();
  const int t0 = blockIdx.x * a.tokens;
  route_tokens<In, G, C>(a, score, t0, min(t0 + a.tokens, a.T), picked, rooms, hist, nullptr);
  __syncthreads();
  for (int i = threadIdx.x; i < a.E; i += blockDim.x)
    a.counts[(size_t)blockIdx.x * stride + i] = hist[i];
}

template <int EMAX>
__global__ __launch_bounds__(kPlaceThreads) void route_place_kernel(RouteArgs a, int stride) {
  constexpr int NW = kPlaceThreads / 64;
  constexpr int VP = EMAX / 4, RP = kPlaceThreads / VP;       // threads a row, rows at a time
  constexpr int RG = kPlaceThreads / (VP < 64 ? 64 : VP);     // sums left to LDS
  __shared__ __attribute__((aligned(16))) int next[NW * EMAX];
  __shared__ __attribute__((aligned(16))) u32x4 part[2 * RG * VP];
  __shared__ __attribute__((aligned(16))) int count[EMAX];
  __shared__ __attribute__((aligned(16))) int base[EMAX];
  __shared__ __attribute__((aligned(16))) int offset[EMAX + 1];
  static_assert(VP >= 32 && (VP & (VP - 1)) == 0 && RP >= 1, "rows of half a wave or more");
  const int nb = gridDim.x, me = blockIdx.x;
  const int s0 = me * a.tokens * a.k, s1 = min(s0 + a.tokens * a.k, a.T * a.k);
  const RouteShare share = route_share(a.experts, s0, s1);
  for (int i = threadIdx.x; i < NW * a.E; i += blockDim.x) next[i] = 0;
  // counts of all workgroups, and of those before this one
  const int v = threadIdx.x % VP, r0 = threadIdx.x / VP;
  u32x4 all{0, 0, 0, 0}, mine{0, 0, 0, 0};
  for (int r = r0; r < nb; r += RP * 8) {
    u32x4 n[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      n[j] = r + RP * j < nb && 4 * v < a.E
                 ? load16(a.counts + (size_t)(r + RP * j) * stride + 4 * v)
                 : u32x4{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        all[q] += n[j][q];
        mine[q] += r + RP * j < me ? n[j][q] : 0;
      }
  }
  if constexpr (VP == 32) {  // two rows a wave
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      all[q] += (uint32_t)__shfl_xor((int)all[q], 32);
      mine[q] += (uint32_t)__shfl_xor((int)mine[q], 32);
    }
  }
  const int group = threadIdx.x / (VP < 64 ? 64 : VP);
  if (VP >= 64 || (threadIdx.x & 63) < 32) {
    part[(2 * group) * VP + v] = all;
    part[(2 * group + 1) * VP + v] = mine;
  }
  __syncthreads();
  const int* sums = reinterpret_cast<const int*>(part);
  for (int x = threadIdx.x; x < 2 * EMAX; x += blockDim.x) {
    int n = 0;
#pragma unroll
    for (int g = 0; g < RG; ++g) n += sums[2 * g * EMAX + x];
    (x < EMAX ? count : base)[x % EMAX] = n;
  }
  route_count(a, a.experts, share, next);
  __syncthreads();
  route_scan(count, offset, a.E);
  __syncthreads();
  route_bases<NW>(next, offset, base, a.E);
  if (me == 0)
    for (int i = threadIdx.x; i <= a.E; i += blockDim.x) a.offsets[i] = offset[i];
  __syncthreads();
  route_place(a, a.experts, share, s0, s1, offset[a.E], next);
}

// ---- launches ---------------------------------------------------------------------------
// Lanes a token: the fewest that hold E logits at 8 a lane, and k choices.
static int route_lanes(long long E, long long k) {
  return E <= 128 && k <= 16 ? 16 : (E <= 256 && k <= 32 ? 32 : 64);
}
// At most kMaxRouteBlocks workgroups, of at least the tokens that one pass of
// their lanes takes.
static int route_blocks(long long T, long long E, long long k, long long* tokens) {
  const long long pass = kSelectThreads / route_lanes(E, k);
  long long per = (T + kMaxRouteBlocks - 1) / kMaxRouteBlocks;
  per = (per + pass - 1) / pass * pass;
  *tokens = per;
  return (int)((T + per - 1) / per);
}
long long route_workspace_bytes(long long T, long long E, long long k) {
  if (T * k <= kRouteSmall) return 0;
  long long tokens;
  return route_blocks(T, E, k, &tokens) * ((E + 3) / 4 * 4) * 4;
}

template <typename In, int G, int C, typename Score>
static hipError_t launch_route_as(RouteArgs a, const Score& score, hipStream_t stream) {
  if ((long long)a.T * a.k <= kRouteSmall) {
    // as many waves as the tokens fill: a token alone takes 4.2 us, with all 8 waves 4.8
    const int threads = std::max(64, std::min((a.T * G + 63) / 64 * 64, kSmallThreads));
    return launch_op(route_small_kernel<In, G, C, Score>, dim3(1), dim3(threads), stream, a, score);
  }
  long long tokens;
  const int blocks = route_blocks(a.T, a.E, a.k, &tokens), stride = (a.E + 3) / 4 * 4;
  a.tokens = (int)tokens;
  const hipError_t e = launch_op(route_select_kernel<In, G, C, Score>, dim3(blocks),
                                 dim3(kSelectThreads), stream, a, score, stride);
  if (e != hipSuccess) return e;
  return launch_op(route_place_kernel<G * C>, dim3(blocks), dim3(kPlaceThreads), stream, a, stride);
}
template <typename In, typename Score>
static hipError_t launch_route_in(const RouteArgs& a, const Score& score, hipStream_t stream) {
  const int lanes = route_lanes(a.E, a.k);
  if (lanes == 16) return launch_route_as<In, 16, 8>(a, score, stream);
  if (lanes == 32) return launch_route_as<In, 32, 8>(a, score, stream);
  if (a.E <= 512) return launch_route_as<In, 64, 8>(a, score, stream);
  return launch_route_as<In, 64, 16>(a, score, stream);
}
template <typename Score>
static hipError_t launch_route_with(const void* logits, bool f32, float* weights, int32_t* experts,
                                    int32_t* offsets, int32_t* rows, void* ws, int T, int E, int k,
                                    bool renorm, const Score& score, hipStream_t stream) {
  const int row = E * (f32 ? 4 : 2);
  const int vec = ((uintptr_t)logits % 16 == 0 && row % 16 == 0) ? 1 : 0;
  const RouteArgs a{logits, weights, experts, offsets, rows, (int32_t*)ws, T, E, k, renorm, vec, 0};
  return f32 ? launch_route_in<float>(a, score, stream) : launch_route_in<uint16_t>(a, score, stream);
}

hipError_t launch_route(const void* logits, bool f32, float* weights, int32_t* experts,
                        int32_t* offsets, int32_t* rows, void* ws, int T, int E, int k,
                        bool renorm, hipStream_t stream) {
  return launch_route_with(logits, f32, weights, experts, offsets, rows, ws, T, E, k, renorm,
                           NoScore{}, stream);
}
hipError_t launch_route_scored(const void* logits, bool f32, float* weights, int32_t* experts,
                               int32_t* offsets, int32_t* rows, void* ws, int T, int E, int k,
                               bool renorm, const RouteScore& score, hipStream_t stream) {
  return launch_route_with(logits, f32, weights, experts, offsets, rows, ws, T, E, k, renorm, score,
                           stream);
}

}  // namespace swiglu
