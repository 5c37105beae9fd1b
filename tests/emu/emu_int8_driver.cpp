// CPU bounds and LDS-ordering emulation of the 8-bit integer kernels (see
// emu_driver.cpp and emu_ops_driver.cpp, whose models this is): one launch.
//
// usage: emu_int8_driver [--plant P] [--cus C] dense GATED VARIANT M N K
//        emu_int8_driver [--plant P] [--cus C] grouped GATED VARIANT N K k DROP count,count,...
//        emu_int8_driver quantize ROWS K
//        emu_int8_driver pack E ROWS K
// DROP: slots behind the spans; --cus: compute units that the launch is told.  The
// products' values mean nothing here, but every element of Y that a launch has to
// write must have been written, and no other one.
#include <stdio.h>
#include <stdlib.h>

#include <string>
#include <vector>

#include "swiglu_int8_emu.cpp"

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
template <typename T>
void check_written(const T* y, size_t n, bool want, T unwritten) {
  size_t bad = 0, first = 0;
  for (size_t i = 0; i < n; ++i)
    if ((y[i] != unwritten) != want && bad++ == 0) first = i;
  if (!bad) return;
  ++g_errors;
  fprintf(stderr, "OUTPUT: %zu of %zu elements %s, the first is %zu\n", bad, n,
          want ? "not written" : "written past the spans", first);
}

void launch(const swiglu::Int8Call& c, int variant) {
  if (swiglu::launch_int8(c, variant, nullptr) != hipSuccess) {
    ++g_errors;
    fprintf(stderr, "LAUNCH: refused\n");
  }
}

void run_dense(bool gated, int variant, int M, int N, int K, int cus) {
  const int C = gated ? 2 * N : N;
  uint16_t* Y = alloc_y((size_t)M * N);
  launch({gated, false, alloc<uint8_t>((size_t)M * K), alloc<float>(M), nullptr, nullptr,
          alloc<uint8_t>(swiglu::int8_packed_bytes(C, K)), alloc<float>(C), Y, M, M, N, K, 1, 1, cus},
         variant);
  check_written(Y, (size_t)M * N, true, kUnwritten);
}

void run_grouped(bool gated, int variant, int N, int K, int k, int drop, const char* list, int cus) {
  std::vector<int> counts;
  for (const char* s = list; *s; s += *s == ',') counts.push_back((int)strtol(s, (char**)&s, 10));
  const int E = (int)counts.size(), C = gated ? 2 * N : N;
  int32_t* offsets = alloc<int32_t>(E + 1);
  for (int e = 0; e < E; ++e) offsets[e + 1] = offsets[e] + counts[e];
  const int n = offsets[E], R = n + drop, T = gated ? (R + k - 1) / k : R;
  int32_t* rows = alloc<int32_t>(R);
  for (int i = 0; i < R; ++i) rows[i] = i < n ? (int)((long long)i * 7919 % n) : -1;
  uint16_t* Y = alloc_y((size_t)R * N);
  launch({gated, true, alloc<uint8_t>((size_t)T * K), alloc<float>(T), rows, offsets,
          alloc<uint8_t>(E * swiglu::int8_packed_bytes(C, K)), alloc<float>((size_t)E * C), Y, T, R, N,
          K, E, gated ? k : 1, cus},
         variant);
  check_written(Y, (size_t)n * N, true, kUnwritten);
  check_written(Y + (size_t)n * N, (size_t)drop * N, false, kUnwritten);
}

void run_quantize(int rows, int K) {
  uint16_t* X = alloc<uint16_t>((size_t)rows * K);
  uint8_t* Q = alloc<uint8_t>((size_t)rows * K);
  float* S = alloc<float>(rows);
  for (size_t i = 0; i < (size_t)rows * K; ++i) Q[i] = 0xab;
  for (int i = 0; i < rows; ++i) S[i] = -1.0f;
  swiglu::launch_quantize_int8(X, Q, S, rows, K, nullptr);
  check_written(Q, (size_t)rows * K, true, (uint8_t)0xab);
  check_written(S, rows, true, -1.0f);
}

void run_pack(int E, int rows, int K) {
  const size_t n = (size_t)E * swiglu::int8_packed_bytes(rows, K);
  const uint8_t* W8 = alloc<uint8_t>((size_t)E * rows * K);
  uint8_t* P = alloc<uint8_t>(n);
  for (size_t i = 0; i < n; ++i) P[i] = 0xab;
  swiglu::launch_pack_int8(W8, P, E, rows, K, nullptr);
  check_written(P, n, true, (uint8_t)0xab);
}
}  // namespace

int main(int argc, char** argv) {
  int cus = 256, i = 1;
  for (; i + 1 < argc && argv[i][0] == '-'; i += 2)
    (std::string(argv[i]) == "--plant" ? g_emu_plant : cus) = atoi(argv[i + 1]);
  const std::string what = i < argc ? argv[i] : "";
  auto n = [&](int j) { return atoi(argv[i + j]); };
  emu_race_context(what.c_str());
  emu_race_enable(true);
  if (what == "dense" && argc == i + 6)
    run_dense(n(1) != 0, n(2), n(3), n(4), n(5), cus);
  else if (what == "grouped" && argc == i + 8)
    run_grouped(n(1) != 0, n(2), n(3), n(4), n(5), n(6), argv[i + 7], cus);
  else if (what == "quantize" && argc == i + 3)
    run_quantize(n(1), n(2));
  else if (what == "pack" && argc == i + 4)
    run_pack(n(1), n(2), n(3));
  else
    return 2;
  printf("%ld LDS accesses, %ld global reads checked\nerrors: %ld\n", g_lds_checks, g_global_checks,
         g_errors + g_emu_race_errors);
  return g_errors + g_emu_race_errors ? 1 : 0;
}
