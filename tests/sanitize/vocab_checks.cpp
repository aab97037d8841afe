// Host-side checks of the vocabulary-end entry points under AddressSanitizer and
// UndefinedBehaviorSanitizer (built with the sanitizers on the host code only; no
// GPU needed): workspace sizes over ordinary, extreme and drawn shapes, and the
// argument checks, which must return before any GPU work.  Prints "ok" and exits
// 0, or names the first failed checks and exits 1.
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include <random>

#include "ckl.h"

static int g_fail = 0;
#define CHECK(cond)                                                  \
  do {                                                               \
    if (!(cond)) {                                                   \
      if (g_fail < 20) fprintf(stderr, "check failed (line %d): %s\n", __LINE__, #cond); \
      ++g_fail;                                                      \
    }                                                                \
  } while (0)

static const int64_t kBig = (int64_t)1 << 26;

// The gradient's workspace: lists of 4-byte keys and positions, a bit per token
// and two partial rows per tile of 16 to 64 positions; 256-byte pieces.
static void check_embed_workspace(int64_t N, int64_t d, int64_t V) {
  uint64_t b = 1;
  const int st = ckl_embed_bwd_workspace(N, d, V, &b);
  if (N < 0 || d <= 0 || V <= 0) {
    CHECK(st == CKL_EINVAL);
  } else if (d % 8 != 0 || d > (int64_t)1 << 20 || V > kBig || N >= kBig) {
    CHECK(st == CKL_EUNSUPPORTED);
  } else {
    CHECK(st == CKL_OK);
    if (N == 0) {
      CHECK(b == 0);
    } else {
      const double tiles = ceil((double)N / (N <= 8192 ? 16 : N <= 16384 ? 32 : 64));
      const double part = tiles > 1 ? tiles * 2 * (double)d * 4 : 0;
      CHECK(b % 256 == 0);
      CHECK((double)b >= 8.0 * (double)N + (double)V / 8 + part);
      CHECK((double)b <= 16.0 * (double)N + (N > 8192 ? 2.0 * (double)N + 4096 : 0) + (double)V / 8 + part + 4096);
    }
  }
}

static void check_sample_workspace(int dt, int64_t N, int64_t V) {
  uint64_t b = 1;
  const int st = ckl_sample_workspace(dt, N, V, &b);
  if (N < 0 || V <= 0) {
    CHECK(st == CKL_EINVAL);
  } else if (V > kBig || N >= (int64_t)1 << 22) {
    CHECK(st == CKL_EUNSUPPORTED);
  } else {
    CHECK(st == CKL_OK);
    CHECK(b <= (uint64_t)256 * 8400 * 2);  // at most 256 slices' counts of 16 bits
    if (dt == CKL_DTYPE_F32 || N == 0 || N > 64 || V < 32768) CHECK(b == 0);
  }
}

int main() {
  const int64_t Ns[] = {INT64_MIN, -1, 0, 1, 15, 16, 17, 63, 64, 65, 256, 257, 8192, 8193, 16384, 16385, 262144,
                        kBig - 4, kBig - 3, kBig - 1, kBig, (int64_t)1 << 40, INT64_MAX};
  const int64_t ds[] = {INT64_MIN, -8, 0, 1, 8, 12, 64, 256, 264, 2880, (int64_t)1 << 20, ((int64_t)1 << 20) + 8,
                        INT64_MAX};
  const int64_t Vs[] = {INT64_MIN, 0, 1, 31, 32, 33, 32767, 32768, 201088, 262143, 262144, kBig - 1, kBig, kBig + 1,
                        INT64_MAX};
  for (int64_t N : Ns)
    for (int64_t V : Vs) {
      for (int64_t d : ds) check_embed_workspace(N, d, V);
      for (int dt = 0; dt < 2; ++dt) check_sample_workspace(dt, N, V);
    }
  std::mt19937_64 rng(1);
  auto draw = [&](int bits) { return (int64_t)(rng() >> (64 - 1 - rng() % bits)); };
  for (int i = 0; i < 200000; ++i) {
    check_embed_workspace(draw(27), 8 * draw(17), draw(27));
    check_sample_workspace(i & 1, draw(23), draw(27));
  }

  // argument checks: fake pointers that are never dereferenced
  void* g = (void*)(uintptr_t)(1 << 20);
  const int32_t* ids = (const int32_t*)g;
  float* f = (float*)g;
  uint8_t* q = (uint8_t*)g;
  uint64_t b = 0;
  CHECK(ckl_embed_bwd_workspace(1, 8, 1, nullptr) == CKL_EINVAL);
  CHECK(ckl_sample_workspace(2, 1, 1, &b) == CKL_EINVAL && ckl_sample_workspace(0, 1, 1, nullptr) == CKL_EINVAL);
  for (int64_t N : Ns)
    for (int64_t d : ds)
      for (int64_t V : Vs) {
        const bool wrong = N < 0 || d <= 0 || V <= 0;
        const bool large = d % 8 != 0 || d > (int64_t)1 << 20 || V > kBig || N >= kBig;
        const int want = wrong ? CKL_EINVAL : large ? CKL_EUNSUPPORTED : N == 0 ? CKL_OK : CKL_EINVAL;
        // null rows: the shape is judged first
        CHECK(ckl_embed(0, ids, nullptr, 1.f, N, d, V, g, nullptr) == want);
        CHECK(ckl_embed_bwd(1, ids, nullptr, 1.f, N, d, V, 1, f, g, 0, nullptr) == want);
        const bool wide = d % 16 != 0 || d > (int64_t)1 << 20 || V > kBig || N > kBig;
        const int m = ckl_matmul_fp8(0, q, f, nullptr, f, N, V, d, g, nullptr);
        if (wrong)
          CHECK(m == CKL_EINVAL);
        else if (wide)
          CHECK(m == CKL_EUNSUPPORTED);
        else
          CHECK(N == 0 ? m == CKL_OK || m == CKL_EUNSUPPORTED : m == CKL_EINVAL || m == CKL_EUNSUPPORTED);
        for (int64_t rows : {(int64_t)1, (int64_t)128, (int64_t)64}) {
          const int s = ckl_quantize_fp8(0, nullptr, N, d, rows, q, f, nullptr);
          if (N < 0 || d <= 0 || rows == 64)
            CHECK(s == CKL_EINVAL);
          else if (d % 16 != 0 || d > (int64_t)1 << 20 || N > kBig)
            CHECK(s == CKL_EUNSUPPORTED);
          else
            CHECK(N == 0 ? s == CKL_OK : s == CKL_EINVAL || s == CKL_EUNSUPPORTED);
        }
        const int s = ckl_sample(1, nullptr, N, V, d, f, nullptr, (int32_t*)g, f, nullptr, 0, nullptr);
        if (N < 0 || V <= 0 || d < 0)
          CHECK(s == CKL_EINVAL);
        else if (V > kBig || N >= (int64_t)1 << 22)
          CHECK(s == CKL_EUNSUPPORTED);
        else
          CHECK(s == (N == 0 ? CKL_OK : CKL_EINVAL));
      }
  // the last sizes that no launch takes, and a gradient whose tiles do not fit one
  CHECK(ckl_embed(0, ids, g, 1.f, kBig - 3, 264, 10, g, nullptr) == CKL_EUNSUPPORTED);
  CHECK(ckl_embed(1, ids, g, 1.f, kBig - 1, (int64_t)1 << 20, kBig, g, nullptr) == CKL_EUNSUPPORTED);
  CHECK(ckl_embed_bwd(0, ids, g, 1.f, kBig - 1, (int64_t)1 << 20, kBig, 0, f, g, UINT64_MAX, nullptr) ==
        CKL_EUNSUPPORTED);
  CHECK(ckl_embed_bwd(0, ids, g, 1.f, 4, 8, 10, 0, f, g, 255, nullptr) == CKL_EINVAL);
  CHECK(ckl_matmul_fp8(1, q, f, q, f, kBig, kBig, 16, g, nullptr) == CKL_EUNSUPPORTED);
  // settings
  const double nan = NAN;
  auto how = [](double T, int64_t k, double top_p, double min_p) {
    return ckl_sampling{T, k, top_p, min_p, nullptr, nullptr, nullptr, nullptr};
  };
  const ckl_sampling bad[] = {how(-1, 0, 1, 0),  how(nan, 0, 1, 0),  how(1, INT64_MIN, 1, 0), how(1, 0, 1.5, 0),
                              how(1, 0, nan, 0), how(1, 0, 1, -0.5), how(1, 0, 1, nan),       how(1, 0, 1, INFINITY)};
  for (const ckl_sampling& s : bad)
    CHECK(ckl_sample(0, g, 4, 10, 10, f, &s, (int32_t*)g, f, nullptr, 0, nullptr) == CKL_EINVAL);
  double ms = 0;
  int64_t n = 0;
  CHECK(ckl_timing_query(10, &ms, &n) == CKL_EINVAL);
  if (g_fail) return 1;
  printf("ok\n");
  return 0;
}
