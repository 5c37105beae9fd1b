// CPU bounds and LDS-ordering emulation of the grouped products and the MXFP4
// kernels (see emu_driver.cpp, whose model this is): one launch of a kernel
// variant, with as many workgroups as its launch function makes or, to have each
// of them walk over several units or tiles, with a few.
//
// usage: emu_ops_driver [--plant P] [--grid G] grouped UP VARIANT N K k DROP count,count,...
//        emu_ops_driver [--plant P] [--cus C]  fp4 VARIANT M N K
//        emu_ops_driver                        convert ROWS K
// UP 1: gated products, 0: down; DROP: slots behind the spans; --grid: workgroups
// of the tile kernel; --cus: compute units that the MXFP4 launch is told.  The
// products' values mean nothing here, but every element of Y that a launch has to
// write must have been written, and no other one.
#include <stdio.h>
#include <stdlib.h>

#include <string>
#include <vector>

#include "swiglu_fp4_emu.cpp"
#include "swiglu_grouped_emu.cpp"

dim3 threadIdx, blockIdx, gridDim, blockDim;
long g_emu_last_blocks = 0;
long g_emu_race_errors = 0;
long g_emu_race_blocks = 0;
int g_emu_plant = 0;

void emu_race_context(const char* ctx);
void emu_race_lds(const uint8_t* base, size_t n);
void emu_race_global(const void* p, size_t n);

namespace {
struct Alloc {
  const uint8_t* p;
  size_t n;
};
std::vector<Alloc> g_allocs;
uint8_t* g_lds = nullptr;
size_t g_lds_size = 0;
long g_errors = 0, g_lds_checks = 0, g_global_checks = 0;

void report(const char* what, const void* p, size_t n) {
  if (g_errors++ < 20)
    fprintf(stderr, "OUT OF BOUNDS: %s (%zu bytes at %p), block (%u,%u) thread %u\n", what, n, p,
            blockIdx.x, blockIdx.y, threadIdx.x);
}
}  // namespace

uint8_t* emu_lds(size_t bytes) {
  if (bytes != g_lds_size || !g_lds) {
    free(g_lds);
    g_lds = (uint8_t*)calloc(bytes ? bytes : 1, 1);
    g_lds_size = bytes;
    emu_race_lds(g_lds, bytes);
  }
  return g_lds;
}
uint8_t* emu_lds_base() { return g_lds; }
void emu_barrier() { emu_race_barrier(); }
void emu_check_lds(uint32_t off, size_t n, const char* what) {
  ++g_lds_checks;
  if (!g_lds || (size_t)off + n > g_lds_size) report(what, g_lds ? g_lds + off : nullptr, n);
}
void emu_check_global(const void* p, size_t n, const char* what) {
  ++g_global_checks;
  const uint8_t* b = (const uint8_t*)p;
  if (b)
    for (const Alloc& a : g_allocs)
      if (b >= a.p && b + n <= a.p + a.n) return;
  report(what, p, n);
}

namespace {
template <typename T>
T* alloc(size_t n) {
  T* p = (T*)calloc(n * sizeof(T) + (n == 0), 1);
  g_allocs.push_back({(const uint8_t*)p, n * sizeof(T)});
  emu_race_global(p, n * sizeof(T));
  return p;
}

constexpr uint16_t kUnwritten = 0xabab;
uint16_t* alloc_y(size_t n) {
  uint16_t* y = alloc<uint16_t>(n);
  for (size_t i = 0; i < n; ++i) y[i] = kUnwritten;
  return y;
}
void check_written(const uint16_t* y, size_t n, bool want) {
  size_t bad = 0, first = 0;
  for (size_t i = 0; i < n; ++i)
    if ((y[i] != kUnwritten) != want && bad++ == 0) first = i;
  if (!bad) return;
  ++g_errors;
  fprintf(stderr, "OUTPUT: %zu of %zu elements %s, the first is %zu\n", bad, n,
          want ? "not written" : "written past the spans", first);
}

// the tile kernels of launch_grouped_op, with a grid of the caller's
template <int OP, int BM, int BNW, int STAGES, int WGM, int WGN, int PARTS, int PWGM, int PWGN, int KG>
void run_tiles(const swiglu::GroupArgs& g, int grid) {
  swiglu::launch_op(swiglu::grouped_tile_kernel<OP, BM, BNW, STAGES, WGM, WGN, PARTS, PWGM, PWGN, KG>,
                    dim3(grid), dim3(64 * WGM * WGN * KG), nullptr, g, (g.ldw + BNW - 1) / BNW);
}
template <int OP>
void run_few(const swiglu::GroupArgs& g, int variant, int grid) {
  switch (variant) {
    case 1: return run_tiles<OP, 64, 128, 4, 2, 2, 1, 2, 2, 1>(g, grid);
    case 2: return run_tiles<OP, 128, 128, 4, 2, 2, 2, 2, 2, 1>(g, grid);
    case 4: return run_tiles<OP, 64, 64, 4, 2, 1, 1, 2, 1, 2>(g, grid);
    default: return run_tiles<OP, 256, 256, 4, 4, 2, 4, 2, 4, 1>(g, grid);
  }
}

void run_grouped(bool up, int variant, int N, int K, int k, int drop, const char* list, int grid) {
  std::vector<int> counts;
  for (const char* s = list; *s; s += *s == ',') counts.push_back((int)strtol(s, (char**)&s, 10));
  const int E = (int)counts.size();
  int32_t* offsets = alloc<int32_t>(E + 1);
  for (int e = 0; e < E; ++e) offsets[e + 1] = offsets[e] + counts[e];
  const int n = offsets[E], R = n + drop, T = up ? (R + k - 1) / k : R;
  int32_t* rows = alloc<int32_t>(R);
  for (int i = 0; i < R; ++i) rows[i] = i < n ? (int)((long long)i * 7919 % n) : -1;
  const uint16_t* A = alloc<uint16_t>((size_t)T * K);
  const uint16_t* W = alloc<uint16_t>((size_t)E * K * N * (up ? 2 : 1));
  uint16_t* Y = alloc_y((size_t)R * N);
  if (grid == 0) {
    swiglu::launch_grouped(up, A, rows, offsets, W, Y, T, R, N, K, E, up ? k : 1, variant, nullptr);
  } else {
    const swiglu::GroupArgs g{A, rows, offsets, W, Y, T, R, N, K, E, up ? k : 1, up ? 2 * N : N};
    if (up) run_few<swiglu::GROUP_UP>(g, variant, grid);
    else run_few<swiglu::GROUP_DOWN>(g, variant, grid);
  }
  check_written(Y, (size_t)n * N, true);
  check_written(Y + (size_t)n * N, (size_t)drop * N, false);
}

void run_fp4(int variant, int M, int N, int K, int cus) {
  using namespace swiglu;
  uint16_t* Y = alloc_y((size_t)M * N);
  const Fp4Call c{alloc<uint8_t>(fp4_code_bytes(M, K)),     alloc<uint8_t>(fp4_scale_bytes(M, K)),
                  alloc<uint8_t>(fp4_code_bytes(2 * N, K)), alloc<uint8_t>(fp4_scale_bytes(2 * N, K)),
                  Y, M, N, K, cus};
  launch_forward_mxfp4(c, variant, nullptr);
  check_written(Y, (size_t)M * N, true);
}

void run_convert(int rows, int K) {
  uint16_t* X = alloc<uint16_t>((size_t)rows * K);
  uint8_t* Q = alloc<uint8_t>(swiglu::fp4_code_bytes(rows, K));
  uint8_t* S = alloc<uint8_t>(swiglu::fp4_scale_bytes(rows, K));
  swiglu::launch_quantize_mxfp4(X, Q, S, rows, K, nullptr);
  swiglu::launch_dequantize_mxfp4(Q, S, X, rows, K, nullptr);
}
}  // namespace

int main(int argc, char** argv) {
  int grid = 0, cus = 256, i = 1;
  for (; i + 1 < argc && argv[i][0] == '-'; i += 2) {
    const std::string o = argv[i];
    (o == "--plant" ? g_emu_plant : o == "--grid" ? grid : cus) = atoi(argv[i + 1]);
  }
  const std::string what = i < argc ? argv[i] : "";
  auto n = [&](int j) { return atoi(argv[i + j]); };
  emu_race_context(what.c_str());
  emu_race_enable(true);
  if (what == "grouped" && argc == i + 8)
    run_grouped(n(1) != 0, n(2), n(3), n(4), n(5), n(6), argv[i + 7], grid);
  else if (what == "fp4" && argc == i + 5)
    run_fp4(n(1), n(2), n(3), n(4), cus);
  else if (what == "convert" && argc == i + 3)
    run_convert(n(1), n(2));
  else
    return 2;
  printf("%ld LDS accesses, %ld global reads checked\nerrors: %ld\n", g_lds_checks, g_global_checks,
         g_errors + g_emu_race_errors);
  return g_errors + g_emu_race_errors ? 1 : 0;
}
