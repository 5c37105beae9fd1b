// swiglu_norm.hip -- the end of a block: the experts' outputs of a token summed
// with their weights, a norm behind the block, its gate and residual scale,
// and the norm in front of the next block, in one pass.
//
// For token t (experts[t, j] < 0: that row of B is not read into the sum,
// whatever it holds):
//   o = sum_j weights[t, j] B[t k + j] + S[t]
//   o = o / sqrt(mean(o^2) + eps) * post        (post given)
//   o = o * gate                                (a row [D], or one a token)
//   x = X[t] + scale o                          -> X_out
//   h = x / sqrt(mean(x^2) + eps) * pre         -> H (bf16)
// Everything between loads and stores is fp32 (the second norm takes x before
// its rounding); each input is read once, so the memory bounds it.
//
// A token's D values stay in registers: NW waves of it, VPL vectors of 8 a
// lane.  Many narrow tokens: one wave each (no barrier, k VPL 16-byte loads in
// flight a lane); else as many waves as D has (launch_norm_x has both sides).
// 8191 tokens, 8 slots, width 1536, fp32 stream: 66 us, 5.3 TB/s; one token, 6
// slots, width 3584: 3.5 us.
#include "swiglu_internal.h"
#include "swiglu_ops_device.hpp"

namespace swiglu {

struct NormArgs {
  const uint16_t* B;
  const float* weights;
  const int32_t* experts;
  const uint16_t* S;
  const void* X;
  const uint16_t* post;
  const uint16_t* gate;
  const uint16_t* pre;
  void* X_out;
  uint16_t* H;
  int T, D, k;
  float scale, eps;
  long long gate_ld;  // 0: one row for all tokens
};

__device__ __forceinline__ void unpack8(const u32x4& v, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __builtin_bit_cast(float, v[i] << 16);
    f[2 * i + 1] = __builtin_bit_cast(float, v[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ u32x4 pack8(const float (&f)[8]) {
  return u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
               pack_bf16x2(f[6], f[7])};
}

// Sum over the NW waves of a token; `part` is LDS of its own for this call.
template <int NW>
__device__ __forceinline__ float token_sum(float v, float* part) {
  v = group_sum<64>(v);
  if constexpr (NW > 1) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) v += part[w];
  }
  return v;
}

template <bool XF32, int NW, int VPL>
__global__ __launch_bounds__(NW == 1 ? 256 : 64 * NW) void combine_norm_kernel(NormArgs a) {
  __shared__ __attribute__((aligned(16))) float part[2 * NW];
  constexpr int kPer = NW == 1 ? 4 : 1;  // tokens of a workgroup
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = __builtin_amdgcn_readfirstlane((int)blockIdx.x * kPer + (NW == 1 ? wave : 0));
  if (t >= a.T) return;  // NW > 1: the whole workgroup
  const int l0 = NW == 1 ? lane : (int)threadIdx.x;
  const int nv = a.D / 8;

  bool in[VPL];
  size_t at[VPL];  // element offset in a row; past the row: the last vector, not stored
  float o[VPL][8];
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int c = l0 + v * 64 * NW;
    in[v] = c < nv;
    at[v] = (size_t)min(c, nv - 1) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[v][i] = 0.0f;
  }
  // With one vector a lane everything else is loaded here, ahead of the sums
  // that would make it wait; with more the registers go to rows of B.
  constexpr bool kEarly = VPL == 1;
  const uint16_t* none = a.pre;  // where an input is absent, any row that is there
  u32x4 vs[VPL], vpost[VPL], vgate[VPL], vpre[VPL], vx[VPL], vx2[VPL];
  auto load_s = [&](int v) __attribute__((always_inline)) {
    vs[v] = a.S ? load16(a.S + (size_t)t * a.D + at[v]) : u32x4{0, 0, 0, 0};
  };
  auto load_post = [&](int v) __attribute__((always_inline)) {
    vpost[v] = load16((a.post ? a.post : none) + at[v]);
  };
  auto load_gate = [&](int v) __attribute__((always_inline)) {
    vgate[v] = load16(a.gate ? a.gate + (size_t)t * a.gate_ld + at[v] : none + at[v]);
  };
  auto load_pre = [&](int v) __attribute__((always_inline)) { vpre[v] = load16(a.pre + at[v]); };
  auto load_x = [&](int v) __attribute__((always_inline)) {
    const size_t p = (size_t)t * a.D + at[v];
    if constexpr (XF32) {
      vx[v] = load16((const float*)a.X + p);
      vx2[v] = load16((const float*)a.X + p + 4);
    } else {
      vx[v] = load16((const uint16_t*)a.X + p);
    }
  };
  if constexpr (kEarly) load_s(0), load_post(0), load_gate(0), load_pre(0), load_x(0);
  const uint16_t* B = a.B + (size_t)t * a.k * a.D;
  auto add = [&](const u32x4 (&b)[VPL], int j) __attribute__((always_inline)) {
    const bool there = a.experts[(size_t)t * a.k + j] >= 0;
    const float w = there ? a.weights[(size_t)t * a.k + j] : 0.0f;
    const uint32_t keep = there ? 0xffffffffu : 0u;  // a row nobody wrote may hold NaN
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      float f[8];
      unpack8(b[v] & keep, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[v][i] = fmaf(w, f[i], o[v][i]);
    }
  };
  auto fetch = [&](u32x4 (&b)[VPL], int j) __attribute__((always_inline)) {
#pragma unroll
    for (int v = 0; v < VPL; ++v) b[v] = load16_stream(B + (size_t)j * a.D + at[v]);
  };
  constexpr int kAhead = VPL <= 2 ? 4 : 2;  // rows of B loaded together
  int j = 0;
  for (; j + kAhead <= a.k; j += kAhead) {
    u32x4 b[kAhead][VPL];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) fetch(b[q], j + q);
#pragma unroll
    for (int q = 0; q < kAhead; ++q) add(b[q], j + q);
  }
  for (; j < a.k; ++j) {
    u32x4 b[VPL];
    fetch(b, j);
    add(b, j);
  }
  if (a.S) {
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      float f[8];
      if constexpr (!kEarly) load_s(v);
      unpack8(vs[v], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[v][i] += f[i];
    }
  }
  if (a.post) {
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < VPL; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) s += in[v] ? o[v][i] * o[v][i] : 0.0f;
    const float r = rsqrtf(token_sum<NW>(s, part) / (float)a.D + a.eps);
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      float f[8];
      if constexpr (!kEarly) load_post(v);
      unpack8(vpost[v], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[v][i] *= r * f[i];
    }
  }
  if (a.gate) {
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      float f[8];
      if constexpr (!kEarly) load_gate(v);
      unpack8(vgate[v], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[v][i] *= f[i];
    }
  }
  float s = 0.0f;
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const size_t p = (size_t)t * a.D + at[v];
    float x[8];
    if constexpr (!kEarly) load_x(v);
    if constexpr (XF32) {
      const f32x4 lo = __builtin_bit_cast(f32x4, vx[v]), hi = __builtin_bit_cast(f32x4, vx2[v]);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = lo[i], x[4 + i] = hi[i];
    } else {
      unpack8(vx[v], x);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      o[v][i] = fmaf(a.scale, o[v][i], x[i]);
      s += in[v] ? o[v][i] * o[v][i] : 0.0f;
    }
    if (in[v]) {
      if constexpr (XF32) {
        float* out = (float*)a.X_out + p;
        *reinterpret_cast<f32x4*>(out) = f32x4{o[v][0], o[v][1], o[v][2], o[v][3]};
        *reinterpret_cast<f32x4*>(out + 4) = f32x4{o[v][4], o[v][5], o[v][6], o[v][7]};
      } else {
        *reinterpret_cast<u32x4*>((uint16_t*)a.X_out + p) = pack8(o[v]);
      }
    }
  }
  const float r = rsqrtf(token_sum<NW>(s, part + NW) / (float)a.D + a.eps);
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    float f[8];
    if constexpr (!kEarly) load_pre(v);
    unpack8(vpre[v], f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] *= r * o[v][i];
    if (in[v]) *reinterpret_cast<u32x4*>(a.H + (size_t)t * a.D + at[v]) = pack8(f);
  }
}

template <bool XF32, int NW, int VPL>
static hipError_t launch_norm_as(const NormArgs& a, hipStream_t stream) {
  const int per = NW == 1 ? 4 : 1;
  return launch_op(combine_norm_kernel<XF32, NW, VPL>, dim3((a.T + per - 1) / per),
                   dim3(NW == 1 ? 256 : 64 * NW), stream, a);
}

// One wave a token from 1024 tokens and up to 2048 wide.  Measured (us, one wave /
// several; 8 slots, shared row, bf16 stream): width 512: 256 tokens 4.4 / 4.6,
// 1024 5.5 / 6.9, 8191 20.0 / 25.7; 1024: 1024 tokens 8.3 / 8.3, 8191 38.4 / 37.5;
// 1536: 256 tokens 8.7 / 5.1, 1024 11.1 / 9.5, 8191 57.2 / 53.7; 2048: 256 tokens
// 10.1 / 5.4, 1024 13.7 / 11.1, 16384 142.2 / 141.9.  The bound on tokens is right,
// that on the width is late: from 1024 on one wave gains nothing, and at 1536 and
// 2048 it loses 3 to 7 % of a long call and a fifth of one of 1024 tokens.
template <bool XF32>
static hipError_t launch_norm_x(const NormArgs& a, hipStream_t stream) {
  const int nv = a.D / 8;  // at most 2048
  if (a.T >= 1024) {
    if (nv <= 64) return launch_norm_as<XF32, 1, 1>(a, stream);
    if (nv <= 128) return launch_norm_as<XF32, 1, 2>(a, stream);
    if (nv <= 192) return launch_norm_as<XF32, 1, 3>(a, stream);
    if (nv <= 256) return launch_norm_as<XF32, 1, 4>(a, stream);
  }
  if (nv <= 256) return launch_norm_as<XF32, 4, 1>(a, stream);
  if (nv <= 512) return launch_norm_as<XF32, 8, 1>(a, stream);
  if (nv <= 1024) return launch_norm_as<XF32, 8, 2>(a, stream);
  return launch_norm_as<XF32, 16, 2>(a, stream);
}

// Threads of the launch: a wave a token for many narrow ones, else the waves
// of launch_norm_x for each token.
long long norm_threads(long long T, long long D) {
  if (D <= 2048) return T >= 1024 ? (T + 3) / 4 * 256 : T * 256;
  return T * (D <= 8192 ? 512 : 1024);
}

hipError_t launch_combine_norm(const NormCall& c, hipStream_t stream) {
  const NormArgs a{(const uint16_t*)c.B,    c.weights, c.experts, (const uint16_t*)c.S,
                   c.X,                     (const uint16_t*)c.post, (const uint16_t*)c.gate,
                   (const uint16_t*)c.pre,  c.X_out,   (uint16_t*)c.H, (int)c.T, (int)c.D,
                   (int)c.k,                c.scale,   c.eps,     c.gate_ld};
  return c.f32 ? launch_norm_x<true>(a, stream) : launch_norm_x<false>(a, stream);
}

}  // namespace swiglu
