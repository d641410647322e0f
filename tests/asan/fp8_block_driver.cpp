// Host-side argument validation of the block-scaled FP8 entry points, run under
// AddressSanitizer (host code instrumented; no GPU is needed or touched).
//
// Every "device" pointer is the address of a freed heap block: the validation may look at
// the address (null, alignment, where outputs lie) but must never read through it.  The
// argument structs stand at the very end of heap blocks of their own, so that a read past
// one is reported too.  Calls whose arguments are valid stop at the device check.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "fp4moe.h"
#include "fp8block.h"

static int g_fail = 0;
static int g_calls = 0;

static void check(int line, const char* what, int st, bool want_bad) {
  ++g_calls;
  const char* msg = fp4moe_last_error();
  const size_t n = strlen(msg);                       // the whole message is read
  const bool bad = st == FP4MOE_ERR_INVALID_ARG;
  if (bad != want_bad || (bad && n == 0)) {
    fprintf(stderr, "line %d: %s -> %d (%s)\n", line, what, st, msg);
    ++g_fail;
  }
}
#define BAD(call) check(__LINE__, #call, (call), true)
#define VALID(call) check(__LINE__, #call, (call), false)

// `call` on a heap copy of args, changed by `change`.
template <class Args, class Change>
int with(int (*call)(const Args*, void*), const Args& args, Change change) {
  Args* a = static_cast<Args*>(malloc(sizeof(Args)));
  memcpy(a, &args, sizeof(Args));
  change(*a);
  const int st = call(a, nullptr);
  free(a);
  return st;
}

int main() {
  void* block = nullptr;
  if (posix_memalign(&block, 256, 1 << 16) != 0) return 2;
  free(block);
  char* D = static_cast<char*>(block);
  auto at = [&](int i) { return D + 8192 * i; };
  auto F = [&](int i) { return reinterpret_cast<float*>(at(i)); };
  auto I32 = [&](int i) { return reinterpret_cast<int32_t*>(at(i)); };
  auto U8 = [&](int i) { return reinterpret_cast<uint8_t*>(at(i)); };

  fp8block_norm_args n;
  memset(&n, 0, sizeof n);
  n.dtype = FP8BLOCK_BF16, n.M = 4, n.K = 300, n.eps = 1e-6f;
  n.x = at(0), n.ldx = 304, n.residual = at(1), n.ldr = 304, n.weight = at(2);
  n.residual_out = at(1), n.ldro = 304, n.y_out = at(3), n.ldy = 304;
  n.codes = U8(4), n.ldc = 304, n.scales = F(5), n.scale_row = 1, n.scale_blk = 4;
  using N = fp8block_norm_args;
  VALID(with(rms_norm_fp8, n, [](N&) {}));
  VALID(with(rms_norm_fp8, n, [](N& a) { a.dtype = FP8BLOCK_F32; }));
  VALID(with(rms_norm_fp8, n, [](N& a) { a.M = 0; a.x = nullptr; }));
  VALID(with(rms_norm_fp8, n, [](N& a) { a.codes = nullptr; a.scales = nullptr; }));
  BAD(rms_norm_fp8(nullptr, nullptr));
  BAD(with(rms_norm_fp8, n, [](N& a) { a.dtype = 7; }));
  BAD(with(rms_norm_fp8, n, [](N& a) { a.K = 65537; }));
  BAD(with(rms_norm_fp8, n, [](N& a) { a.weight = nullptr; }));
  BAD(with(rms_norm_fp8, n, [](N& a) { a.ldr = 299; }));
  BAD(with(rms_norm_fp8, n, [](N& a) { a.scale_row = 0; }));
  BAD(with(rms_norm_fp8, n, [](N& a) { a.scale_blk = INT64_MIN; }));
  BAD(with(rms_norm_fp8, n, [](N& a) { a.residual_out = const_cast<void*>(a.x); a.ldro = 300; }));
  BAD(with(rms_norm_fp8, n, [](N& a) { a.codes = static_cast<uint8_t*>(a.y_out) + 9; }));
  BAD(with(rms_norm_fp8, n, [](N& a) { a.x = static_cast<const char*>(a.x) + 1; }));

  VALID(swiglu_fp8(FP8BLOCK_F16, at(0), 4, 300, 600, I32(2), U8(3), 300, F(4), 1, 4, nullptr));
  VALID(swiglu_fp8(FP8BLOCK_F16, nullptr, 0, 300, 600, nullptr, nullptr, 300, nullptr, 1, 4, nullptr));
  BAD(swiglu_fp8(-1, at(0), 4, 300, 600, I32(2), U8(3), 300, F(4), 1, 4, nullptr));
  BAD(swiglu_fp8(FP8BLOCK_F16, at(0), 4, 300, 599, I32(2), U8(3), 300, F(4), 1, 4, nullptr));
  BAD(swiglu_fp8(FP8BLOCK_F16, at(0), 1 << 30, 300, 600, I32(2), U8(3), 300, F(4), 1, 1 << 30, nullptr));
  BAD(swiglu_fp8(FP8BLOCK_F16, at(0), 4, 300, 600, I32(2), U8(3), 300, F(4), 1, 1, nullptr));
  BAD(swiglu_fp8(FP8BLOCK_F16, at(0), 4, 300, 600, I32(2), nullptr, 300, F(4), 1, 4, nullptr));
  BAD(swiglu_fp8(FP8BLOCK_F32, at(0) + 2, 4, 300, 600, I32(2), U8(3), 300, F(4), 1, 4, nullptr));

  fp8block_gemm_args g;
  memset(&g, 0, sizeof g);
  g.M = 8, g.N = 40, g.K = 272, g.a_rows = 8;
  g.a = U8(0), g.lda = 272, g.a_scale = F(1), g.as_row = 1, g.as_blk = 8;
  g.w = U8(2), g.ldw = 272, g.w_scale = F(3), g.ld_ws = 3;
  g.out_dtype = FP8BLOCK_BF16, g.out = at(4), g.ldo = 40;
  g.n_experts = 2, g.block_m = 16, g.gather_div = 1, g.max_tiles = 3, g.w_expert = 40 * 272, g.ws_expert = 3;
  g.a_row_gather = I32(5), g.expert_offsets = I32(6), g.tiles = I32(7), g.n_tiles = I32(6);
  using G = fp8block_gemm_args;
  for (auto call : {fp8_block_linear, fp8_block_grouped_gemm}) {
    VALID(with(call, g, [](G&) {}));
    VALID(with(call, g, [](G& a) { a.M = 0; a.a = nullptr; }));
    VALID(with(call, g, [](G& a) { a.N = INT32_MAX; a.ldo = INT32_MAX; }));
    BAD(call(nullptr, nullptr));
    BAD(with(call, g, [](G& a) { a.K = 264; }));
    BAD(with(call, g, [](G& a) { a.lda = 280; }));
    BAD(with(call, g, [](G& a) { a.w += 8; }));
    BAD(with(call, g, [](G& a) { a.out_dtype = FP8BLOCK_F32; }));
    BAD(with(call, g, [](G& a) { a.ldo = 39; }));
    BAD(with(call, g, [](G& a) { a.as_blk = -1; }));
    BAD(with(call, g, [](G& a) { a.w_scale = nullptr; }));
  }
  VALID(with(fp8_block_linear, g, [](G& a) { a.tiles = nullptr; a.n_experts = -5; }));
  BAD(with(fp8_block_grouped_gemm, g, [](G& a) { a.tiles = nullptr; }));
  BAD(with(fp8_block_grouped_gemm, g, [](G& a) { a.block_m = 48; }));
  BAD(with(fp8_block_grouped_gemm, g, [](G& a) { a.gather_div = 0; }));
  BAD(with(fp8_block_grouped_gemm, g, [](G& a) { a.a_rows = 7; a.a_row_gather = nullptr; }));
  VALID(with(fp8_block_grouped_gemm, g, [](G& a) { a.max_tiles = 0; }));

  printf("%d calls, %d failures\n", g_calls, g_fail);
  return g_fail == 0 ? 0 : 1;
}
