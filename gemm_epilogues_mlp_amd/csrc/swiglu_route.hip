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
// The scored form, with its own figures, is further down.
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
// the weight.  Scores, sums and comparisons are in 64 bits by definition: neighbours among
// some hundred scores between 0 and 1 come as close as fp32 rounds exp, and the choice is to
// be that of the definition.  Comparing 64-bit values lane by lane is slow (35.8 us for 8191
// tokens, 256 experts in 8 groups, against 20.0), so c is first compared as a
// whole number, its place between the least and the largest possible value in some 2^28
// steps.  Two numbers in different steps are in the right order; where two that meet at
// a choice are not told apart (equal logits, or chance: some 1e-7 a pair), the wave takes
// the 64-bit path.  Without a bias the logits themselves are in the order of the scores.
// What is left is instructions: some 950 vector ones of a wave for its two tokens of 256
// experts, a third of them the exponentials (13 to 15 us to choose in two passes, 5.6 to 7.2 to
// place; 1024 threads a workgroup, one pass: 15.6).  One token: 7.7 us a call, a chain of 1500
// instructions of one wave.
struct NoScore {};
template <bool SIGMOID_>
struct Scores : RouteScore {
  static constexpr bool SIGMOID = SIGMOID_;
};
constexpr double kNegInfD = -__builtin_inf();

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xf, 0xf, true);  // no lane is left out
}
template <int CTRL>
__device__ __forceinline__ double dpp_d(double v) {
  const uint64_t x = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)dpp_u<CTRL>((uint32_t)(x >> 32)) << 32 |
                                        dpp_u<CTRL>((uint32_t)x));
}
// v of the other row of 16 lanes of a pair, or of the other half wave: both are in a and b
__device__ __forceinline__ void both_rows(uint32_t v, uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ void both_halves(uint32_t v, uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  a = r[0];
  b = r[1];
}
// over aligned groups of G lanes (16, 32 or 64); every lane receives the same bits
template <int G>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  v = max(v, dpp_u<kDppXor1>(v));
  v = max(v, dpp_u<kDppXor2>(v));
  v = max(v, dpp_u<kDppHalfMirror>(v));
  v = max(v, dpp_u<kDppMirror>(v));
  uint32_t a, b;
  if (G >= 32) both_rows(v, a, b), v = max(a, b);
  if (G >= 64) both_halves(v, a, b), v = max(a, b);
  return v;
}
template <int G, typename F>
__device__ __forceinline__ double lanes_fold(double v, F f) {
  v = f(v, dpp_d<kDppXor1>(v));
  v = f(v, dpp_d<kDppXor2>(v));
  v = f(v, dpp_d<kDppHalfMirror>(v));
  v = f(v, dpp_d<kDppMirror>(v));
  auto pair = [&](auto split) __attribute__((always_inline)) {
    const uint64_t x = __builtin_bit_cast(uint64_t, v);
    uint32_t lo[2], hi[2];
    split((uint32_t)x, lo[0], lo[1]);
    split((uint32_t)(x >> 32), hi[0], hi[1]);
    v = f(__builtin_bit_cast(double, (uint64_t)hi[0] << 32 | lo[0]),
          __builtin_bit_cast(double, (uint64_t)hi[1] << 32 | lo[1]));
  };
  if (G >= 32) pair(both_rows);
  if (G >= 64) pair(both_halves);
  return v;
}
__device__ __forceinline__ double larger(double a, double b) { return a > b ? a : b; }
__device__ __forceinline__ double sum_of(double a, double b) { return a + b; }

// e^x, infinite past 2^1024, for x <= 760, within some 2^-52: x = n ln 2 + r with |r| <= ln(2) / 2,
// the Taylor polynomial of e^r to the 13th power (what is left out is below 2^-57), scaled by 2^n.
__device__ __forceinline__ double exp_d(double x) {
  x = x > -760.0 ? x : -760.0;  // 0 from there on
  const double n = __builtin_rint(x * 1.4426950408889634);
  // ln 2 as fp32, n times which is exact, and what that leaves of it
  double r = __builtin_fma(n, -(double)0.6931471805599453f, x);
  r = __builtin_fma(n, 1.904654299957768e-09, r);
  double p = 1.0 / 6227020800.0;
  constexpr double f[13] = {1.0 / 479001600.0, 1.0 / 39916800.0, 1.0 / 3628800.0, 1.0 / 362880.0,
                            1.0 / 40320.0,     1.0 / 5040.0,     1.0 / 720.0,     1.0 / 120.0,
                            1.0 / 24.0,        1.0 / 6.0,        0.5,             1.0,
                            1.0};
#pragma unroll
  for (int i = 0; i < 13; ++i) p = __builtin_fma(p, r, f[i]);
  return __builtin_ldexp(p, (int)n);
}
// 1 / d for a normal d: the hardware's estimate and two steps of Newton
__device__ __forceinline__ double reciprocal_d(double d) {
  double r = __builtin_amdgcn_rcp(d);
  r = __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
  return __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
}
// What logit x is below the largest one, m; an infinite m counts as 1e39, which is above all finite
// ones, and nothing is above m.
__device__ __forceinline__ double softmax_below(float x, float m) {
  const double top = m < __builtin_inff() ? (double)m : 1e39;
  return __builtin_fmin((double)x - top, 0.0);
}
// The score of logit x, but for the division by the sum in a softmax (m its largest logit; an
// infinite one shares the weight with its equals).  Next to where e^-x has no 64-bit value (from the
// fp32 logit -709.78271484375 on) the reciprocal of 1 + e^-x is too small for the steps of Newton:
// they are taken 2^64 away, and make a NaN of the infinite e^-x, which the sigmoid has as 0.
template <bool SIGMOID>
__device__ __forceinline__ double score_of(float x, float m) {
  if constexpr (SIGMOID) {
    const double d = __builtin_fma(exp_d(-(double)fmaxf(x, -760.0f)), 0x1p-64, 0x1p-64);
    return __builtin_fmax(reciprocal_d(d), 0.0) * 0x1p-64;
  }
  return exp_d(softmax_below(x, m));
}

// What stays the same from token to token: the biases of the lane's experts, and the
// step of a whole number.
template <int C>
struct ScoreLane {
  float bias[C];
  double steps, first;  // c is in step c steps + first
};
constexpr int kScoreBits = 28;
template <int G, int C>
__device__ __forceinline__ ScoreLane<C> score_lane(const RouteArgs& a, const RouteScore& sc) {
  const int gl = threadIdx.x & (G - 1);
  ScoreLane<C> o;
  uint32_t most = 0;  // the largest magnitude of a bias that leaves its expert open
#pragma unroll
  for (int j = 0; j < C; ++j) {
    o.bias[j] = sc.bias ? sc.bias[min(gl * C + j, a.E - 1)] : 0.0f;
    const uint32_t size = __builtin_bit_cast(uint32_t, o.bias[j]) & 0x7fffffffu;
    most = max(most, o.bias[j] > kNegInf ? size : 0u);
  }
  const double span = (double)__builtin_bit_cast(float, lanes_max<G>(most));
  // an infinite one tells nothing apart, and every token takes the 64-bit path
  o.steps = span < 3e38 ? (double)((1 << kScoreBits) - 3) * reciprocal_d(2.0 * span + 1.0) : 0.0;
  o.first = span * o.steps + 1.5;  // step 0 is that of a closed expert
  return o;
}

// LDS of one token.
template <int N>
struct ScoreRoom {
  double c[N];             // of all experts
  union {
    uint32_t key[N];       // what stands for c, while groups are compared
    float x[N];            // then their logits
  };
  union {
    double value[kMaxGroups];
    uint32_t number[kMaxGroups + 4];
  };
  int index[64];
};
__device__ __forceinline__ void room_written() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();  // other lanes' places: no read moves above this
}

// whether the groups of the lane's experts are kept, from `room`
template <int G, int C>
__device__ __forceinline__ void read_kept(const RouteArgs& a, int size, const ScoreRoom<G * C>& room,
                                          uint32_t& kept) {
  const int gl = threadIdx.x & (G - 1);
  const float by = 1.0f / (float)size;
  kept = 0;
#pragma unroll
  for (int j = 0; j < C; ++j) {
    // (e + 1/2) / size is 1 / (2 size) or more from a whole number
    const int e = min(gl * C + j, a.E - 1);
    kept |= (uint32_t)room.index[(int)(((float)e + 0.5f) * by)] << j;
  }
}

// Which of the lane's logits have a group that is kept; false where whole numbers do not tell
// (or none of the groups has two open experts, whose sum has another zero).
template <int G, int C>
__device__ __forceinline__ bool keep_groups(const RouteArgs& a, const RouteScore& sc,
                                            const uint32_t (&key)[C], bool exact,
                                            ScoreRoom<G * C>& room, uint32_t& kept) {
  const int gl = threadIdx.x & (G - 1), size = a.E / sc.groups, lanes = size / C;
  const bool two = sc.group_best == 2;
  bool sure = true;
  auto value = [&](uint32_t first, uint32_t second) __attribute__((always_inline)) {
    if (two && first != 0 && second == 0 && size > 1) sure = false;
    return first + (two ? second : 0u);
  };
  if (gl < 4) room.number[(sc.groups & ~3) + gl] = 0u;  // compared, as closed groups are
  // the rank of a value among the groups': exact ones go by index where they are equal,
  // others are two roundings of a step each from the sums
  auto keep = [&](uint32_t mine, int g) __attribute__((always_inline)) {
    int before = 0, near = 0;
    for (int i = 0; i < sc.groups; i += 4) {
      const u32x4 v = *reinterpret_cast<const u32x4*>(room.number + i);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        before += v[q] + (i + q < g ? 1u : 0u) > mine;
        near += v[q] - mine + 2u <= 4u;
      }
    }
    if (!exact && mine != 0 && near > 1) sure = false;
    return mine != 0 && before < sc.top_groups;
  };
  if (size % C == 0 && lanes <= 16 && (lanes & (lanes - 1)) == 0) {
    // a group is `lanes` lanes next to each other
    uint32_t first = 0, second = 0;
    auto merge = [&](uint32_t f, uint32_t s) __attribute__((always_inline)) {
      second = max(min(first, f), max(second, s));
      first = max(first, f);
    };
#pragma unroll
    for (int j = 0; j < C; ++j) merge(key[j], 0u);
    if (lanes >= 2) merge(dpp_u<kDppXor1>(first), dpp_u<kDppXor1>(second));
    if (lanes >= 4) merge(dpp_u<kDppXor2>(first), dpp_u<kDppXor2>(second));
    if (lanes >= 8) merge(dpp_u<kDppHalfMirror>(first), dpp_u<kDppHalfMirror>(second));
    if (lanes >= 16) merge(dpp_u<kDppMirror>(first), dpp_u<kDppMirror>(second));
    const int g = gl / lanes;
    const uint32_t mine = g < sc.groups ? value(first, second) : 0u;
    if (g < sc.groups) room.number[g] = mine;  // the group's lanes write the same
    room_written();
    kept = keep(mine, g) ? ~0u : 0u;
  } else {
    uint32_t* keys = room.key;
#pragma unroll
    for (int j = 0; j < C; ++j) keys[gl * C + j] = key[j];
    room_written();
    for (int g = gl; g < sc.groups; g += G) {
      uint32_t first = 0, second = 0;
      for (int i = 0; i < size; ++i) {
        const uint32_t v = keys[g * size + i];
        second = max(second, min(first, v));
        first = max(first, v);
      }
      room.number[g] = value(first, second);
    }
    room_written();
    for (int g = gl; g < sc.groups; g += G) room.index[g] = keep(room.number[g], g);
    room_written();
    read_kept<G, C>(a, size, room, kept);
  }
  return sure;
}

// The k largest of x, the lowest index first among equals: as route_token and
// route_token_keys choose.  Lane gl < k receives the index of choice gl, -1 if there is none.
template <typename In, int G, int C>
__device__ __forceinline__ int choose_logits(float (&x)[C], int k) {
  const int lane = threadIdx.x & 63, gl = lane & (G - 1);
  int choice = -1;
  if constexpr (std::is_same_v<In, uint16_t>) {
    uint32_t key[C];
#pragma unroll
    for (int j = 0; j < C; ++j) key[j] = route_key(x[j], gl * C + j);
    for (int i = 0; i < k; ++i) {
      uint32_t v = key[0];
#pragma unroll
      for (int j = 1; j < C; ++j) v = max(v, key[j]);
      const uint32_t best = lanes_max<G>(v);
      if (gl == i && best) choice = (int)(kMaxExperts - 1) - (int)(best & 0xffffu);
#pragma unroll
      for (int j = 0; j < C; ++j)
        if (key[j] == best) key[j] = 0;
    }
  } else {
    for (int i = 0; i < k; ++i) {
      float v = x[0];
      int bj = 0;
#pragma unroll
      for (int j = 1; j < C; ++j)
        if (x[j] > v) v = x[j], bj = j;
      const float best = group_max<G>(v);
      const unsigned long long group = (G == 64 ? ~0ull : ((1ull << (G & 63)) - 1)) << (lane & ~(G - 1));
      const int winner = __ffsll(__ballot(v == best) & group) - 1;
      const int index = __shfl(gl * C + bj, winner);
      if (gl == i && best > kNegInf) choice = index;
      if (lane == winner)
#pragma unroll
        for (int j = 0; j < C; ++j)
          if (j == bj) x[j] = kNegInf;
    }
  }
  return choice;
}

// The same of whole numbers, closed places 0; `sure` becomes false where two of them that meet
// are equal.  The lane's keys hold j in their last bits, so the largest names its place
// in the lane, and are sorted once: a choice then takes a lane's first one away.
template <int G, int C>
__device__ __forceinline__ int choose_numbers(const uint32_t (&number)[C], int k, bool& sure) {
  static_assert((C & (C - 1)) == 0 && (((uint64_t)C) << kScoreBits) <= (1ull << 32), "key");
  const int lane = threadIdx.x & 63, gl = lane & (G - 1);
  uint32_t key[C];
#pragma unroll
  for (int j = 0; j < C; ++j) key[j] = number[j] ? number[j] * C + (C - 1 - j) : 0u;
  // odd-even merge sort, largest first
#pragma unroll
  for (int p = 1; p < C; p *= 2)
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int i = q % p; i + q < C; i += 2 * q)
#pragma unroll
        for (int j = 0; j < q; ++j)
          if (i + j + q < C && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const uint32_t hi = max(key[i + j], key[i + j + q]), lo = min(key[i + j], key[i + j + q]);
            key[i + j] = hi;
            key[i + j + q] = lo;
          }
  int choice = -1;
  uint32_t last = 0;
  for (int i = 0;; ++i) {
    const uint32_t best = lanes_max<G>(key[0]);
    if (best != 0 && best / C == last / C) sure = false;
    if (i == k) break;
    last = best;
    const unsigned long long vote = __ballot(key[0] == best);
    const uint32_t mine = G == 64 ? 0u : (uint32_t)(vote >> (lane & 32)) >> (lane & 31 & ~(G - 1));
    const int winner = G == 64 ? __ffsll(vote) - 1 : __ffs(mine) - 1;  // lane of the token's
    if (gl == i && best) choice = winner * C + (int)(C - 1 - best % C);
    // (selected by bits: a choice between array elements becomes a chain of comparisons)
    const uint32_t take = gl == winner ? ~0u : 0u;
#pragma unroll
    for (int j = 0; j + 1 < C; ++j) key[j] = (key[j + 1] & take) | (key[j] & ~take);
    key[C - 1] &= ~take;
  }
  return choice;
}

// The definition in 64 bits, on the c in `room`: which of the lane's experts have a kept group, ...
template <int G, int C>
__device__ __forceinline__ void keep_scores(const RouteArgs& a, const RouteScore& sc,
                                            ScoreRoom<G * C>& room, uint32_t& kept) {
  const int gl = threadIdx.x & (G - 1), size = a.E / sc.groups;
  for (int g = gl; g < sc.groups; g += G) {
    double first = kNegInfD, second = kNegInfD;
    for (int i = 0; i < size; ++i) {
      const double v = room.c[g * size + i];
      second = larger(second, v < first ? v : first);
      first = larger(first, v);
    }
    room.value[g] = sc.group_best == 2 && second > kNegInfD ? first + second : first;
  }
  room_written();
  for (int g = gl; g < sc.groups; g += G) {
    const double value = room.value[g];
    int before = 0;
    for (int i = 0; i < sc.groups; ++i) {
      const double v = room.value[i];
      before += v > value || (v == value && i < g);
    }
    room.index[g] = before < sc.top_groups;
  }
  room_written();
  read_kept<G, C>(a, size, room, kept);
}
// ... and the k largest are chosen.
template <int G, int C>
__device__ __forceinline__ int choose_scores(double (&c)[C], int k) {
  const int lane = threadIdx.x & 63, gl = lane & (G - 1);
  int choice = -1;
  for (int i = 0; i < k; ++i) {
    double v = c[0];
    int bj = 0;
#pragma unroll
    for (int j = 1; j < C; ++j)
      if (c[j] > v) v = c[j], bj = j;
    const double best = lanes_fold<G>(v, larger);
    const unsigned long long group = (G == 64 ? ~0ull : ((1ull << (G & 63)) - 1)) << (lane & ~(G - 1));
    const int winner = __ffsll(__ballot(v == best) & group) - 1;
    const int index = __shfl(gl * C + bj, winner);
    if (gl == i && best > kNegInfD) choice = index;
    if (lane == winner)
#pragma unroll
      for (int j = 0; j < C; ++j)
        if (j == bj) c[j] = kNegInfD;
  }
  return choice;
}

// As route_token.
template <typename In, int G, int C, bool SIGMOID>
__device__ __forceinline__ void route_token_scored(const RouteArgs& a, const Scores<SIGMOID>& sc,
                                                   const ScoreLane<C>& sl, int t, bool in,
                                                   ScoreRoom<G * C>& room, int32_t& expert,
                                                   float& weight) {
  const int gl = threadIdx.x & (G - 1);
  float x[C];
  load_logits<C>((const In*)a.logits + (size_t)(in ? t : 0) * a.E, in ? a.E : 0, gl * C, a.vec, x);
  // softmax: the largest logit, and one over the sum where scores are compared or not divided by
  // their own sum
  const bool numbers = sc.bias || (sc.groups > 1 && sc.group_best == 2);
  float m = 0.0f;
  double over = 1.0;
  if constexpr (!SIGMOID) {
    m = x[0];
#pragma unroll
    for (int j = 1; j < C; ++j) m = fmaxf(m, x[j]);
    m = group_max<G>(m);
    m = m > kNegInf ? m : 0.0f;
  }
  uint32_t key[C];
  if (numbers || (!SIGMOID && !a.renorm)) {
    double s[C];
    double total = 0.0;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      s[j] = score_of<SIGMOID>(x[j], m);
      if constexpr (!SIGMOID) total += s[j];
    }
    if constexpr (!SIGMOID) {
      total = lanes_fold<G>(total, sum_of);
      over = total > 0.0 ? reciprocal_d(total) : 0.0;
    }
    if (numbers) {
#pragma unroll
      for (int j = 0; j < C; ++j) {
        const double c = s[j] * over + (double)sl.bias[j];
        const bool open = x[j] > kNegInf && c > kNegInfD;  // a NaN is not
        room.c[gl * C + j] = open ? c : kNegInfD;
        key[j] = open ? (uint32_t)__builtin_fma(c, sl.steps, sl.first) : 0u;
      }
    }
  }
  // logits, which tell all apart, for groups: whatever the sum above was needed for.  (Skipped where
  // there are none, one token's softmax takes 5.3 instead of 5.5 us, its sigmoid 7.8 instead of 7.5.)
  if (!numbers && (SIGMOID || sc.groups > 1)) {
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const uint32_t b = __builtin_bit_cast(uint32_t, x[j] == 0.0f ? 0.0f : x[j]);
      key[j] = x[j] > kNegInf ? b ^ (uint32_t)((int)b >> 31 | (int)0x80000000) : 0u;
    }
  }
  uint32_t kept = ~0u;  // by bits
  if (sc.groups > 1) {
    const bool sure = keep_groups<G, C>(a, sc, key, !numbers, room, kept);
    if (__ballot(!sure || (numbers && sl.steps == 0.0))) keep_scores<G, C>(a, sc, room, kept);
  }
#pragma unroll
  for (int j = 0; j < C; ++j) room.x[gl * C + j] = x[j];
  int choice;
  if (sc.bias) {
#pragma unroll
    for (int j = 0; j < C; ++j) key[j] &= (uint32_t)((int)(kept << (31 - j)) >> 31);
    bool sure = sl.steps != 0.0;
    choice = choose_numbers<G, C>(key, a.k, sure);
    if (__ballot(!sure)) {
      double c[C];
#pragma unroll
      for (int j = 0; j < C; ++j) c[j] = (kept >> j) & 1u ? room.c[gl * C + j] : kNegInfD;
      choice = choose_scores<G, C>(c, a.k);
    }
  } else {
#pragma unroll
    for (int j = 0; j < C; ++j) x[j] = (kept >> j) & 1u ? x[j] : kNegInf;
    choice = choose_logits<In, G, C>(x, a.k);
  }
  room_written();
  const bool open = gl < a.k && choice >= 0;
  const float y = open ? room.x[choice] : kNegInf;
  expert = open ? choice : -1;
  bool some = true;
  if constexpr (!SIGMOID) {
    // The largest logit may be of an expert that the bias or its group (by the sum of two) left out.
    // Weights that are divided by their sum are taken relative to the largest chosen one, whose share
    // is 1, unless all their scores are 0: e^-745.13 is the least that 64 bits round to something else.
    if (a.renorm && numbers) {
      const uint32_t b = __builtin_bit_cast(uint32_t, y);
      const uint32_t top = lanes_max<G>(b ^ (uint32_t)((int)b >> 31 | (int)0x80000000));
      const float most = __builtin_bit_cast(float, top ^ (uint32_t)(~((int)top >> 31) | (int)0x80000000));
      some = softmax_below(most, m) > -745.1332191019411;
      m = some ? most : m;
    }
  }
  double p = open && some ? score_of<SIGMOID>(y, m) : 0.0;
  if (a.renorm) {
    // a sum of sigmoids may be as small as one: moved to where its reciprocal has a value
    if constexpr (SIGMOID) p *= 0x1p512;
    const double total = lanes_fold<G>(p, sum_of);
    p = total > 0.0 ? p * reciprocal_d(total) : 0.0;
  } else {
    p *= over;
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
  constexpr bool kScored = !std::is_same_v<Score, NoScore>;
  [[maybe_unused]] std::conditional_t<kScored, ScoreLane<C>, NoScore> sl;
  if constexpr (kScored) sl = score_lane<G, C>(a, score);
  for (int t = t0 + first; t - first < t1; t += per) {
    const bool in = t < t1;
    int32_t e;
    float w;
    if constexpr (kScored)
      route_token_scored<In, G, C>(a, score, sl, t, in, rooms[first], e, w);
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
// Spans and sorted slots of the n choices in `slots`, by one workgroup of up to kSmallThreads;
// hist holds the experts' counts, next zeros.
__device__ __forceinline__ void route_sort(const RouteArgs& a, int* slots, int n, int* hist,
                                           int* offset, int* next) {
  const RouteShare share = route_share(slots, 0, n);
  route_count(a, slots, share, next);
  route_scan(hist, offset, a.E);
  __syncthreads();
  route_bases<kSmallThreads / 64>(next, offset, nullptr, a.E);
  for (int i = threadIdx.x; i <= a.E; i += blockDim.x) a.offsets[i] = offset[i];
  __syncthreads();
  route_place(a, slots, share, 0, n, offset[a.E], next);
}
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
  route_sort(a, slots, n, hist, offset, next);
}

// ---- few slots, many tokens for one workgroup: a wave's tokens a workgroup, then one sorts --
// The choices are read back from `experts`, so no workspace is needed.
template <int EMAX>
__global__ __launch_bounds__(kSmallThreads) void route_sort_kernel(RouteArgs a) {
  __shared__ __attribute__((aligned(16))) int next[kSmallThreads / 64 * EMAX];
  __shared__ __attribute__((aligned(16))) int hist[EMAX];
  __shared__ __attribute__((aligned(16))) int offset[EMAX + 1];
  __shared__ __attribute__((aligned(16))) int slots[kRouteSmall];
  const int nw = blockDim.x >> 6, n = a.T * a.k;
  for (int i = threadIdx.x; i < nw * a.E; i += blockDim.x) next[i] = 0;
  for (int i = threadIdx.x; i < a.E; i += blockDim.x) hist[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int x = a.experts[i];
    slots[i] = x;
    if (x >= 0) atomicAdd(&hist[x], 1);
  }
  __syncthreads();
  route_sort(a, slots, n, hist, offset, next);
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
  if (stride == 0) return;  // counted by the launch that sorts
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
  constexpr bool kScored = !std::is_same_v<Score, NoScore>;
  if ((long long)a.T * a.k <= kRouteSmall) {
    // as many waves as the tokens fill: a token alone takes 4.2 us, with all 8 waves 4.8
    const int threads = std::max(64, std::min((a.T * G + 63) / 64 * 64, kSmallThreads));
    // A scored choice takes that one compute unit 4 to 8 us a pass, so beyond one pass a wave's
    // tokens are a workgroup and a second launch sorts: 256 experts in 8 groups, 8 choices, 16
    // tokens 9.9 / 9.5 us (one launch / two), 24 13.9 / 9.5, 64 22.4 / 9.5, one choice of 512
    // tokens 89.4 / 8.3; 64 experts, 6 choices, 32 tokens 7.8 / 8.4, 48 10.8 / 8.2.
    if (kScored && a.T * G > kSmallThreads) {
      a.tokens = 64 / G;
      const hipError_t e = launch_op(route_select_kernel<In, G, C, Score>,
                                     dim3((a.T + a.tokens - 1) / a.tokens), dim3(64), stream, a,
                                     score, 0);
      if (e != hipSuccess) return e;
      const int n = a.T * a.k;
      return launch_op(route_sort_kernel<G * C>, dim3(1), dim3((n + 63) / 64 * 64), stream, a);
    }
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
  return score.sigmoid ? launch_route_with(logits, f32, weights, experts, offsets, rows, ws, T, E, k,
                                           renorm, Scores<true>{score}, stream)
                       : launch_route_with(logits, f32, weights, experts, offsets, rows, ws, T, E, k,
                                           renorm, Scores<false>{score}, stream);
}

}  // namespace swiglu
