// swiglu_checks.hpp -- argument checks of the mixture-of-experts and MXFP4 entry
// points: host code only, no device and no handle, so that they can be tried
// anywhere.  Each returns a swiglu_status_t value; *noop is set when there is
// nothing to compute.
#pragma once

#include <stdint.h>

#include <initializer_list>

#include "swiglu_internal.h"

namespace swiglu {
namespace checks {

constexpr int kOk = 0, kInvalid = 1, kUnsupported = 2;
constexpr long long kMaxInt = 0x7fffffffLL;
constexpr long long kMax2G = 1LL << 31;
constexpr long long kMaxSlots = 1LL << 30;
constexpr long long kMaxTotal = 1LL << 46;  // bytes of a tensor addressed with 64 bits
constexpr long long kMaxThreads = (1LL << 32) - 1;  // of a launch, along x

struct Span {
  const void* p;
  long long bytes;
};
inline bool overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  return x < y + (uintptr_t)b.bytes && y < x + (uintptr_t)a.bytes;
}
// no output overlaps an input or another output
inline bool clash(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (auto o = outs.begin(); o != outs.end(); ++o) {
    for (auto q = o + 1; q != outs.end(); ++q)
      if (overlap(*o, *q)) return true;
    for (const Span& i : ins)
      if (overlap(*o, i)) return true;
  }
  return false;
}
inline bool aligned(const void* p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }
inline bool aligned16(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!aligned(p, 16)) return false;
  return true;
}
// a * b with a, b >= 0, held at 2^62
inline long long mul(long long a, long long b) {
  const __int128 v = (__int128)a * b;
  return v > ((__int128)1 << 62) ? (1LL << 62) : (long long)v;
}

inline int route(const void* logits, const void* weights, const void* experts, const void* offsets,
                 const void* rows, const void* ws, long long ws_bytes, long long T, long long E,
                 long long k, int dtype) {
  if (T < 0 || E < 1 || k < 1 || k > E || (dtype != 0 && dtype != 1)) return kInvalid;
  if (!offsets) return kInvalid;
  if (T > 0 && (!logits || !weights || !experts || !rows)) return kInvalid;
  // 2^30 slots: the last workgroup's tokens are counted from past the last one
  if (E > kMaxExperts || k > kMaxChoices || mul(T, k) > kMaxSlots || mul(T, E) > kMaxTotal)
    return kUnsupported;
  const unsigned size = dtype ? 4 : 2;
  for (const void* p : {weights, experts, offsets, rows})
    if (!aligned(p, 4)) return kUnsupported;
  if (!aligned(ws, 16)) return kUnsupported;
  if (!aligned(logits, size)) return kUnsupported;
  const long long need = route_workspace_bytes(T, E, k);
  if (need > 0 && (!ws || ws_bytes < need)) return kInvalid;
  if (clash({{weights, 4 * T * k}, {experts, 4 * T * k}, {offsets, 4 * (E + 1)}, {rows, 4 * T * k},
             {ws, need}},
            {{logits, (long long)size * T * E}}))
    return kInvalid;
  return kOk;
}

inline int grouped(bool up, const void* A, const void* rows, const void* offsets, const void* W,
                   const void* Y, long long TA, long long R, long long N, long long K, long long E,
                   long long k, int variant, bool* noop) {
  *noop = false;
  if (TA < 0 || R < 0 || N < 0 || K < 0 || E < 1 || k < 1) return kInvalid;
  if (R == 0 || N == 0) {
    *noop = true;
    return kOk;
  }
  if (!rows || !offsets || !Y || (K > 0 && (!W || (TA > 0 && !A)))) return kInvalid;
  // N: a K step's 64 rows past a matrix of under 2 GiB end within 32-bit offsets
  if (E > kMaxExperts || TA > kMaxInt || R > kMaxInt || K > kMaxInt || N > (1LL << 23) ||
      k > kMaxInt || N % 8 != 0 || K % 8 != 0)
    return kUnsupported;
  if (!aligned16({A, W, Y}) || !aligned(rows, 4) || !aligned(offsets, 4)) return kUnsupported;
  // 32-bit byte offsets inside A and inside one expert's weights; the experts
  // and the rows of Y are addressed with 64 bits
  const long long abytes = 2 * mul(TA, K), wbytes = (up ? 4 : 2) * mul(K, N), ybytes = 2 * mul(R, N);
  if (abytes >= kMax2G || wbytes >= kMax2G || mul(E, wbytes) > kMaxTotal || ybytes > kMaxTotal)
    return kUnsupported;
  // workgroups: at most one tile of rows for every 16 rows and one more an
  // expert, times the column tiles of 128
  const long long some = R < E ? R : E;
  if (mul(R / 16 + some + 1, ((up ? 2 : 1) * N + 127) / 128) > kMaxInt) return kUnsupported;
  if (grouped_threads(up, R, N, E, variant) > kMaxThreads) return kUnsupported;
  if (clash({{Y, ybytes}},
            {{A, abytes}, {W, mul(E, wbytes)}, {rows, 4 * R}, {offsets, 4 * (E + 1)}}))
    return kInvalid;
  return kOk;
}

inline int combine_norm(const NormCall& c, int dtype, bool* noop) {
  *noop = false;
  if (c.T < 0 || c.D < 0 || c.k < 0 || c.gate_ld < 0 || (dtype != 0 && dtype != 1)) return kInvalid;
  if (c.T == 0 || c.D == 0) {
    *noop = true;
    return kOk;
  }
  if (!c.X || !c.pre || !c.X_out || !c.H || (c.k > 0 && (!c.B || !c.weights || !c.experts)))
    return kInvalid;
  if (c.gate && c.gate_ld != 0 && c.gate_ld < c.D) return kInvalid;
  if (c.D % 8 != 0 || c.D > kMaxNormWidth || c.T > kMaxInt / 4 || c.k > kMaxInt ||
      mul(mul(c.T, c.k), 2 * c.D) > kMaxTotal || mul(c.T, 4 * c.D) > kMaxTotal)
    return kUnsupported;
  if (norm_threads(c.T, c.D) > kMaxThreads) return kUnsupported;
  if (c.gate && (c.gate_ld % 8 != 0 || mul(c.T, mul(2, c.gate_ld)) > kMaxTotal)) return kUnsupported;
  if (!aligned16({c.B, c.S, c.X, c.post, c.gate, c.pre, c.X_out, c.H}) || !aligned(c.weights, 4) ||
      !aligned(c.experts, 4))
    return kUnsupported;
  const long long x = (dtype ? 4 : 2) * c.T * c.D;
  const Span B{c.B, 2 * c.T * c.k * c.D}, S{c.S, 2 * c.T * c.D}, w{c.weights, 4 * c.T * c.k},
      e{c.experts, 4 * c.T * c.k}, post{c.post, 2 * c.D}, pre{c.pre, 2 * c.D},
      gate{c.gate, 2 * ((c.T - 1) * c.gate_ld + c.D)}, X{c.X, x}, X_out{c.X_out, x}, H{c.H, 2 * c.T * c.D};
  // X may be updated in place; every other overlap of an output is refused
  if (c.X_out == c.X ? clash({X_out, H}, {B, S, w, e, post, pre, gate})
                     : clash({X_out, H}, {B, S, w, e, post, pre, gate, X}))
    return kInvalid;
  return kOk;
}

// bf16 X [rows, K] and its codes Q and scales S; `back`: X is the output
inline int convert_mxfp4(const void* X, const void* Q, const void* S, long long rows, long long K,
                         bool back, bool* noop) {
  *noop = false;
  if (rows < 0 || K < 0) return kInvalid;
  if (rows == 0 || K == 0) {
    *noop = true;
    return kOk;
  }
  if (!X || !Q || !S) return kInvalid;
  if (K % 32 != 0 || rows > kMaxInt || K > kMaxInt || mul(rows + 31, 2 * (K + 255)) > kMaxTotal)
    return kUnsupported;
  const long long q = fp4_code_bytes(rows, K), s = fp4_scale_bytes(rows, K);
  if (q / 1024 * 64 > kMaxThreads) return kUnsupported;  // one wave for each 1 KB of codes
  if (!aligned16({X, Q, S})) return kUnsupported;
  const Span x{X, 2 * rows * K}, cq{Q, q}, cs{S, s};
  if (back ? clash({x}, {cq, cs}) : clash({cq, cs}, {x})) return kInvalid;
  return kOk;
}

// 8 blocks of 32 rows past a tile's first stay within 32-bit offsets
constexpr long long kMaxFp4K = 1LL << 22;

inline int forward_mxfp4(const Fp4Call& c, bool* noop) {
  *noop = false;
  if (c.M < 0 || c.N < 0 || c.K < 0) return kInvalid;
  if (c.M == 0 || c.N == 0) {
    *noop = true;
    return kOk;
  }
  if (!c.Y || (c.K > 0 && (!c.A || !c.SA || !c.W || !c.SW))) return kInvalid;
  if (c.M > kMaxInt - 256 || c.K > kMaxFp4K || c.N > (kMaxInt >> 1) - 256 || c.N % 8 != 0 ||
      c.K % 32 != 0)
    return kUnsupported;
  if (!aligned16({c.Y, c.A, c.SA, c.W, c.SW})) return kUnsupported;
  const __int128 a128 = (__int128)((c.M + 31) / 32) * ((c.K + 255) / 256) * 4096;
  const __int128 w128 = (__int128)((2 * c.N + 31) / 32) * ((c.K + 255) / 256) * 4096;
  if (a128 >= kMax2G || w128 >= kMax2G || mul(c.M, 2 * c.N) > kMaxTotal) return kUnsupported;
  // eight waves for each block of 32 weight rows where they are streamed (with
  // K > 0 the weights' 2 GiB end sooner)
  if ((2 * c.N + 31) / 32 * 512 > kMaxThreads) return kUnsupported;
  // tiles of 128 x 64 outputs, the smallest
  if (mul((c.M + 127) / 128, (c.N + 63) / 64) > kMaxInt) return kUnsupported;
  if (clash({{c.Y, 2 * c.M * c.N}},
            {{c.A, (long long)a128}, {c.SA, (long long)a128 / 16}, {c.W, (long long)w128},
             {c.SW, (long long)w128 / 16}}))
    return kInvalid;
  return kOk;
}

}  // namespace checks
}  // namespace swiglu
