// swiglu_int8.hip -- 8-bit integers: quantisation of bf16 rows, weights into fragment
// order, and gated and plain products of such rows with such weights, for one
// weight set or grouped by expert.
//
// Codes are symmetric with one fp32 scale a row (a token of the activations, an
// output channel of the weights), so a product is exact in 32-bit integers and
//   p[m, c] = (SQ[m] sum_k Q[m, k] W[c, k]) SW[c],
// three roundings in all: the sum to fp32 and two products.
// Weights are stored in the order the 32x32x32 matrix instructions take them (rows
// in blocks of 32, K in groups of 128, G = ceil(K / 128)):
//   P[(((b G + g) 4 + s) 2 + h) 512 + 16 i + j] = W8[32 b + i][128 g + 32 s + 16 h + j]
// padded with zeros, so lane i + 32 h finds its 16 bytes next to its neighbours'
// (1 KB a load). Activations stay row-major, as a gather by row wants them; what is
// read past a row's end meets zeros of the weights.
#include "swiglu_internal.h"
#include "swiglu_ops_device.hpp"

#include <algorithm>
#include <type_traits>
#include <utility>

namespace swiglu {

enum Int8Op { I8_GATED = 0, I8_PLAIN = 1 };

// The tensors of a product, as its kernels take them.
struct Int8Args {
  const uint8_t* A;        // [TA, K]
  const float* SA;         // [TA]
  const int32_t* rows;     // grouped: [R] slot of each sorted row
  const int32_t* offsets;  // grouped: [E + 1]
  const uint8_t* W;        // E fragment-ordered matrices of C rows
  const float* SW;         // [E, C]
  uint16_t* Y;             // [R, N]
  int TA, R, N, K, E, k;   // not grouped: R = TA
  int C;                   // 2N (gated) or N (plain)
};

// Row of A of sorted row `pos`, -1 if the slot names no row of A.
template <int OP>
__device__ __forceinline__ int int8_a_row(const Int8Args& g, int pos) {
  if (OP == I8_PLAIN) return pos;
  const int slot = g.rows[pos];
  return slot >= 0 && slot / g.k < g.TA ? slot / g.k : -1;
}

// ============================================================================
// Quantisation
// ============================================================================
// The nearest integer to 127 x / a, the even one at a tie: c = 127 x is exact (15
// bits), t = c r with r the rounded 1 / a is within two steps of the quotient, and one
// step of Newton with the exact remainder c - t a makes a quotient that is a half
// exactly that half (all other quotients of two 8-bit significands times 127 are
// 2^-17 or more away from one, relative). Adding 1.5 2^23 rounds to an integer that
// then stands in the low bits.
__device__ __forceinline__ uint32_t int8_code(float c, float a, float r) {
  float t = c * r;
  t = __builtin_fmaf(__builtin_fmaf(-t, a, c), r, t);
  return __builtin_bit_cast(uint32_t, t + 12582912.0f);
}

// One row by W waves of a workgroup of 4 or more waves, a thread holding CH chunks of 8
// values from the load of the maximum to the store of the codes, so X is read once.
template <int W, int CH>
__global__ __launch_bounds__(64 * (W < 4 ? 4 : W)) void quantize_int8_kernel(
    const uint16_t* __restrict__ X, uint8_t* __restrict__ Q, float* __restrict__ S, int rows, int K) {
  constexpr int kThreads = 64 * (W < 4 ? 4 : W), T = 64 * W, RPW = kThreads / T;
  __shared__ __attribute__((aligned(16))) uint32_t top[W];
  const int tid = threadIdx.x % T;
  const int row = blockIdx.x * RPW + threadIdx.x / T;
  if (RPW > 1 && row >= rows) return;  // whole waves, and no barrier below
  const uint16_t* x = X + (size_t)row * K;
  u32x4 v[CH];
  uint32_t m = 0;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int k = (c * T + tid) * 8;
    v[c] = k < K ? load16_stream(x + k) : u32x4{0, 0, 0, 0};
  }
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int d = 0; d < 4; ++d) m = max(m, max(v[c][d] & 0x7fffu, (v[c][d] >> 16) & 0x7fffu));
  m = group_max<64>(m);
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) top[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W; ++w) m = max(m, top[w]);
  }
  // bf16 bits of the largest magnitude: from 0x7f80 on an infinity or a NaN. Very
  // large and very small rows are moved by a power of two, where the steps of
  // int8_code neither overflow nor lose bits.
  const bool bad = m >= 0x7f80u;
  const float a = bf16_to_float((uint16_t)m);
  const float move = a < 0x1p-60f ? 0x1p80f : (a > 0x1p60f ? 0x1p-80f : 1.0f);
  const float am = a * move, r = bad || m == 0 ? 0.0f : 1.0f / am;
  const float by = 127.0f * move;
  if (tid == 0) S[row] = bad ? __builtin_nanf("") : a / 127.0f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int k = (c * T + tid) * 8;
    if (k >= K) break;
    uint32_t q[8];
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      q[2 * d] = int8_code(bf16_to_float((uint16_t)v[c][d]) * by, am, r);
      q[2 * d + 1] = int8_code(__builtin_bit_cast(float, v[c][d] & 0xffff0000u) * by, am, r);
    }
    u32x2 o;
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      const uint32_t lo = __builtin_amdgcn_perm(q[4 * d + 1], q[4 * d], 0x0c0c0400u);
      const uint32_t hi = __builtin_amdgcn_perm(q[4 * d + 3], q[4 * d + 2], 0x04000c0cu);
      o[d] = bad ? 0u : lo | hi;
    }
    *reinterpret_cast<u32x2*>(Q + (size_t)row * K + k) = o;
  }
}

// Any K: the row is read twice, by one workgroup.
__global__ __launch_bounds__(1024) void quantize_int8_long_kernel(const uint16_t* __restrict__ X,
                                                                  uint8_t* __restrict__ Q,
                                                                  float* __restrict__ S, int K) {
  __shared__ __attribute__((aligned(16))) uint32_t top[16];
  const int row = blockIdx.x;
  const uint16_t* x = X + (size_t)row * K;
  uint32_t m = 0;
  for (int k = threadIdx.x * 8; k < K; k += 8192) {
    const u32x4 v = load16(x + k);
#pragma unroll
    for (int d = 0; d < 4; ++d) m = max(m, max(v[d] & 0x7fffu, (v[d] >> 16) & 0x7fffu));
  }
  m = group_max<64>(m);
  if ((threadIdx.x & 63) == 0) top[threadIdx.x >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 16; ++w) m = max(m, top[w]);
  const bool bad = m >= 0x7f80u;
  const float a = bf16_to_float((uint16_t)m);
  const float move = a < 0x1p-60f ? 0x1p80f : (a > 0x1p60f ? 0x1p-80f : 1.0f);
  const float am = a * move, r = bad || m == 0 ? 0.0f : 1.0f / am;
  const float by = 127.0f * move;
  if (threadIdx.x == 0) S[row] = bad ? __builtin_nanf("") : a / 127.0f;
  for (int k = threadIdx.x * 8; k < K; k += 8192) {
    const u32x4 v = load16(x + k);
    u32x2 o{0, 0};
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const uint32_t lo = int8_code(bf16_to_float((uint16_t)v[d]) * by, am, r) & 0xffu;
      const uint32_t hi = int8_code(__builtin_bit_cast(float, v[d] & 0xffff0000u) * by, am, r) & 0xffu;
      o[d / 2] |= (lo | hi << 8) << (16 * (d & 1));
    }
    *reinterpret_cast<u32x2*>(Q + (size_t)row * K + k) = bad ? u32x2{0, 0} : o;
  }
}

// ============================================================================
// Weights into fragment order
// ============================================================================
// A thread copies one run of 16 bytes at a time; once per weight set.
__global__ __launch_bounds__(256) void pack_int8_kernel(const uint8_t* __restrict__ W8,
                                                        uint8_t* __restrict__ P, int rows, int K,
                                                        long long chunks) {
  const int G = (K + 127) / 128, B = (rows + 31) / 32;
  for (long long c = (long long)blockIdx.x * 256 + threadIdx.x; c < chunks;
       c += (long long)gridDim.x * 256) {
    const int i = (int)(c & 31), h = (int)(c >> 5 & 1), s = (int)(c >> 6 & 3);
    const long long bg = c >> 8;
    const int g = (int)(bg % G);
    const long long eb = bg / G;
    const int b = (int)(eb % B);
    const int row = 32 * b + i, k = 128 * g + 32 * s + 16 * h;
    const u32x4 v = row < rows && k < K
                        ? load16(W8 + ((size_t)(eb / B) * rows + row) * K + k)
                        : u32x4{0, 0, 0, 0};
    *reinterpret_cast<u32x4*>(P + (size_t)c * 16) = v;
  }
}

// ============================================================================
// Few rows: weight streaming
// ============================================================================
// A workgroup takes NB blocks of 32 weight rows and MT blocks of 32 activation rows
// (D = W A^T, so that a Gate / Up pair is two adjacent registers of a lane); its NW
// waves take every NW-th group of 128 k, the next group's loads issued before
// this one's products. The waves' sums are added in LDS: integers, so their order does
// not matter.
template <int OP, bool GROUPED, int MT, int NB, int NW>
__global__ __launch_bounds__(64 * NW) void int8_stream_kernel(Int8Args g, int nblk) {
  constexpr int NQ = MT * NB * 4;
  __shared__ __attribute__((aligned(16))) i32x4 red[NW > 1 ? NW * NQ * 64 : 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = lane >> 5;
  const int K = g.K, G = (K + 127) / 128, B = (g.C + 31) / 32;
  int blk, pos0, nrows, expert = 0;
  if constexpr (GROUPED) {
    const GroupRange range = group_range<32 * MT, 1>(g.offsets, g.E, g.R, nblk, blockIdx.x % 8);
    const int t = range.begin + (int)blockIdx.x / 8;
    if (t >= range.end) return;
    const GroupUnit u = group_unit<32 * MT>(g.offsets, g.E, g.R, nblk, t);
    blk = u.local % nblk;
    pos0 = u.first + u.local / nblk * (32 * MT);
    nrows = min(u.first + u.rows - pos0, 32 * MT);
    expert = u.expert;
  } else {
    blk = xcd_remap(blockIdx.x, gridDim.x);
    pos0 = blockIdx.y * (32 * MT);
    nrows = min(g.R - pos0, 32 * MT);
  }
  const uint8_t* wp[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b)  // a block past the last repeats it; never stored
    wp[b] = g.W + ((size_t)expert * B + min(blk * NB + b, B - 1)) * G * 4096 + lane * 16;
  // this lane's rows of A; rows past the span repeat the last one and are never stored
  const uint8_t* ap[MT];
  int ar[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int pos = pos0 + min(32 * j + (lane & 31), nrows - 1);
    ar[j] = GROUPED ? int8_a_row<OP>(g, pos) : pos;
    ap[j] = g.A + (size_t)max(ar[j], 0) * K + 16 * h;
  }
  i32x16 acc[MT][NB];
#pragma unroll
  for (int j = 0; j < MT; ++j)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[j][b] = i32x16{};

  u32x4 w[2][NB][4], a[2][MT][4];
  auto load = [&](int p, int gi) __attribute__((always_inline)) {
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int s = 0; s < 4; ++s) w[p][b][s] = load16_stream(wp[b] + (size_t)gi * 4096 + s * 1024);
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int k = gi * 128 + s * 32;
        a[p][j][s] = k + 16 * h < K && ar[j] >= 0 ? load16(ap[j] + k) : u32x4{0, 0, 0, 0};
      }
  };
  auto multiply = [&](int p) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[j][b] = mfma32_i8(w[p][b][s], a[p][j][s], acc[j][b]);
  };
  int gi = wave;
  if (gi < G) load(0, gi);
  for (; gi < G; gi += 2 * NW) {
    if (gi + NW < G) load(1, gi + NW);
    multiply(0);
    if (gi + NW >= G) break;
    if (gi + 2 * NW < G) load(0, gi + 2 * NW);
    multiply(1);
  }

  // quarter q of a lane: weight rows 32 block + 8 q + 4 h + 0 .. 3 of A's row lane % 32
  auto store = [&](int j, int b, int q, const i32x4& v) __attribute__((always_inline)) {
    const int row = 32 * j + (lane & 31), c = (blk * NB + b) * 32 + 8 * q + 4 * h;
    if (row >= nrows || c >= g.C) return;
    const float sa = K > 0 && ar[j] >= 0 ? g.SA[ar[j]] : 0.0f;
    f32x4 sw{0, 0, 0, 0};
    if (K > 0) sw = __builtin_bit_cast(f32x4, load16(g.SW + (size_t)expert * g.C + c));
    float p[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) p[x] = (float)v[x] * sa * sw[x];
    const int out = GROUPED && OP == I8_PLAIN ? g.rows[pos0 + row] : pos0 + row;
    if (out < 0 || out >= g.R) return;
    uint16_t* y = g.Y + (size_t)out * g.N;
    if constexpr (OP == I8_GATED)
      *reinterpret_cast<uint32_t*>(y + c / 2) = pack_bf16x2(silu(p[0]) * p[1], silu(p[2]) * p[3]);
    else
      *reinterpret_cast<u32x2*>(y + c) = u32x2{pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3])};
  };
  if constexpr (NW == 1) {
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const i32x16& d = acc[j][b];
          store(j, b, q, i32x4{d[4 * q], d[4 * q + 1], d[4 * q + 2], d[4 * q + 3]});
        }
  } else {
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const i32x16& d = acc[j][b];
          red[(wave * NQ + (j * NB + b) * 4 + q) * 64 + lane] =
              i32x4{d[4 * q], d[4 * q + 1], d[4 * q + 2], d[4 * q + 3]};
        }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < NQ; ++x) {
      if (x % NW != wave) continue;
      i32x4 v = red[x * 64 + lane];
#pragma unroll
      for (int o = 1; o < NW; ++o) v += red[(o * NQ + x) * 64 + lane];
      store(x / 4 / NB, x / 4 % NB, x % 4, v);
    }
  }
}

// ============================================================================
// Launches
// ============================================================================
// At most this many tiles of bm rows, whatever the spans: one partial tile for
// each expert that has rows.
static long long int8_row_tiles(const Int8Call& c, long long bm) {
  if (!c.grouped) return (c.R + bm - 1) / bm;
  const long long some = std::min(c.R, c.E);
  return std::min(c.R, (c.R + some * (bm - 1)) / bm);
}
static long long int8_stream_units(const Int8Call& c, int mt, int nb) {
  return int8_row_tiles(c, 32 * mt) * ((c.C() + 32 * nb - 1) / (32 * nb));
}

template <int OP, bool GROUPED, int MT, int NB, int NW>
static hipError_t launch_int8_stream(const Int8Call& c, const Int8Args& g, hipStream_t stream) {
  const long long nblk = (c.C() + 32 * NB - 1) / (32 * NB);
  if (GROUPED) {
    const long long grid = (int8_stream_units(c, MT, NB) + 7) / 8 * 8;
    if (grid > 0x7fffffffLL) return hipErrorInvalidValue;
    return launch_op(int8_stream_kernel<OP, GROUPED, MT, NB, NW>, dim3((unsigned)grid),
                     dim3(64 * NW), stream, g, (int)nblk);
  }
  const long long nmb = (c.R + 32 * MT - 1) / (32 * MT);
  if (nblk > 0x7fffffffLL || nmb > 65535) return hipErrorInvalidValue;
  return launch_op(int8_stream_kernel<OP, GROUPED, MT, NB, NW>,
                   dim3((unsigned)nblk, (unsigned)nmb), dim3(64 * NW), stream, g, (int)nblk);
}

template <int OP, bool GROUPED>
static hipError_t launch_int8_as(const Int8Call& c, int variant, hipStream_t stream) {
  const Int8Args g{c.A,        c.SA,     c.rows,   c.offsets, c.W,      c.SW,     c.Y,       (int)c.TA,
                   (int)c.R,   (int)c.N, (int)c.K, (int)c.E,  (int)c.k, (int)c.C()};
  (void)variant;
  return launch_int8_stream<OP, GROUPED, 1, 1, 4>(c, g, stream);
}

hipError_t launch_int8(const Int8Call& c, int variant, hipStream_t stream) {
  if (c.grouped)
    return c.gated ? launch_int8_as<I8_GATED, true>(c, variant, stream)
                   : launch_int8_as<I8_PLAIN, true>(c, variant, stream);
  return c.gated ? launch_int8_as<I8_GATED, false>(c, variant, stream)
                 : launch_int8_as<I8_PLAIN, false>(c, variant, stream);
}

// Threads of the launch along x, and its workgroups along y.
void int8_launch_size(const Int8Call& c, int variant, long long* threads, long long* y) {
  (void)variant;
  *y = c.grouped ? 1 : (c.R + 31) / 32;
  *threads = 256 * (c.grouped ? (int8_stream_units(c, 1, 1) + 7) / 8 * 8 : (c.C() + 31) / 32);
}

// Waves of a row.
static int quantize_waves(long long K) {
  return K <= 1024 ? 1 : K <= 8192 ? 4 : K <= 16384 ? 8 : 16;
}
long long int8_quantize_threads(long long rows, long long K) {
  return quantize_waves(K) == 1 ? (rows + 3) / 4 * 256 : rows * 64 * quantize_waves(K);
}

template <int W, int CH>
static hipError_t launch_quantize_as(const uint16_t* X, uint8_t* Q, float* S, int rows, int K,
                                     hipStream_t stream) {
  constexpr int threads = 64 * (W < 4 ? 4 : W), per = threads / (64 * W);
  return launch_op(quantize_int8_kernel<W, CH>, dim3((unsigned)((rows + per - 1) / per)),
                   dim3(threads), stream, X, Q, S, rows, K);
}
hipError_t launch_quantize_int8(const uint16_t* X, uint8_t* Q, float* S, int rows, int K,
                                hipStream_t stream) {
  if (K <= 512) return launch_quantize_as<1, 1>(X, Q, S, rows, K, stream);
  if (K <= 1024) return launch_quantize_as<1, 2>(X, Q, S, rows, K, stream);
  if (K <= 2048) return launch_quantize_as<4, 1>(X, Q, S, rows, K, stream);
  if (K <= 4096) return launch_quantize_as<4, 2>(X, Q, S, rows, K, stream);
  if (K <= 8192) return launch_quantize_as<4, 4>(X, Q, S, rows, K, stream);
  if (K <= 16384) return launch_quantize_as<8, 4>(X, Q, S, rows, K, stream);
  if (K <= 32768) return launch_quantize_as<16, 4>(X, Q, S, rows, K, stream);
  return launch_op(quantize_int8_long_kernel, dim3((unsigned)rows), dim3(1024), stream, X, Q, S, K);
}

hipError_t launch_pack_int8(const uint8_t* W8, uint8_t* P, long long E, int rows, int K,
                            hipStream_t stream) {
  const long long chunks = E * int8_packed_bytes(rows, K) / 16;
  const long long blocks = std::min<long long>((chunks + 255) / 256, 1 << 16);
  return launch_op(pack_int8_kernel, dim3((unsigned)blocks), dim3(256), stream, W8, P, rows, K,
                   chunks);
}

}  // namespace swiglu
