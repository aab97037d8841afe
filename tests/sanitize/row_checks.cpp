// Host-side checks of the log-probabilities', the residual's and dropout's entry
// points under AddressSanitizer and UndefinedBehaviorSanitizer (built with the
// sanitizers on the host code only; no GPU needed): workspace sizes and the planner
// over ordinary, extreme and drawn shapes, and the argument checks, which must
// return before any GPU work.  Prints "ok" and exits 0, or names the first failed
// checks and exits 1.
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

static void check_logprobs_workspace(int64_t N, int64_t V, int64_t top) {
  uint64_t b = 1;
  const int st = ckl_logprobs_workspace(N, V, top, &b);
  if (N < 0 || V <= 0 || top < 0 || top > V) {
    CHECK(st == CKL_EINVAL);
  } else if (V > kBig || N >= (int64_t)1 << 22 || top > 512) {
    CHECK(st == CKL_EUNSUPPORTED);
  } else {
    CHECK(st == CKL_OK && b % 256 == 0);
    CHECK(b <= (uint64_t)1024 * 16 + (uint64_t)256 * 1024 * 8 + 256);  // 1,024 slices at most, 1,024 pairs a row
    if (N == 0 || N >= 256 || V < 8192) CHECK(b == 0);
  }
}

static void check_norm_workspace(int64_t N, int64_t d, int sums) {
  uint64_t b = 1;
  const int st = ckl_add_norm_bwd_workspace(N, d, sums, &b);
  if (sums < 0 || sums > 3 || N < 0 || d <= 0) {
    CHECK(st == CKL_EINVAL);
  } else if (d % 8 != 0 || d > 16384 || N > (int64_t)1 << 31) {
    CHECK(st == CKL_EUNSUPPORTED);
  } else {
    CHECK(st == CKL_OK && b % 256 == 0);
    CHECK((N == 0 || sums == 0) ? b == 0 : b >= (uint64_t)sums * d * 4);
    CHECK((double)b <= 1024.0 * 3 * 16384 * 4);  // four workgroups a compute unit at most
  }
}

static void check_plan(int back, int dt, int dw, int64_t N, int64_t d, int64_t V, int64_t chunk, uint64_t budget) {
  int64_t c = -1;
  uint64_t b = 0;
  const int st = ckl_head_logprobs_plan(back, dt, dw, N, d, V, chunk, budget, &c, &b);
  if (dt < 0 || dt > 1 || N < 0 || d <= 0 || V <= 0 || chunk < 0 || (back && (dw < 0 || dw > 1 || (dw == 0 && dt == 1)))) {
    CHECK(st == CKL_EINVAL);
  } else if (d % 8 != 0 || V > kBig || N > kBig || d > (int64_t)1 << 20) {
    CHECK(st == CKL_EUNSUPPORTED);
  } else {
    CHECK(st == CKL_OK || st == CKL_EBUDGET || (chunk > 0 && st == CKL_EUNSUPPORTED));
    if (st == CKL_OK && N > 0) {
      CHECK(c >= 1 && c <= N && c <= (int64_t)1 << 20);
      CHECK(budget == 0 || b <= budget);
      CHECK(chunk == 0 || c == (chunk < N ? chunk : N));
      CHECK((double)((V + 63) / 64) * (double)((c + 63) / 64) < 16777216.0 + 4.0 * ((V + 63) / 64));
    }
    if (st == CKL_OK && N == 0) CHECK(b == 0);
  }
}

int main() {
  const int64_t ns[] = {-1, 0, 1, 7, 255, 256, 4096, 32768, ((int64_t)1 << 22) - 1, (int64_t)1 << 22, kBig, kBig + 1,
                        (int64_t)1 << 31, ((int64_t)1 << 31) + 1, INT64_MAX};
  const int64_t vs[] = {-5, 0, 1, 127, 128, 8191, 8192, 32000, 201088, kBig, kBig + 1, INT64_MAX};
  const int64_t ds[] = {-8, 0, 4, 8, 64, 512, 520, 2880, 8192, 8200, 16384, 16392, (int64_t)1 << 20, ((int64_t)1 << 20) + 8,
                        INT64_MAX, INT64_MAX - 7};
  const int64_t tops[] = {-1, 0, 1, 20, 48, 128, 129, 512, 513, INT64_MAX};
  for (int64_t N : ns) {
    for (int64_t V : vs)
      for (int64_t top : tops) check_logprobs_workspace(N, V, top);
    for (int64_t d : ds) {
      for (int sums = -1; sums <= 4; ++sums) check_norm_workspace(N, d, sums);
      for (int64_t V : vs)
        for (int back = 0; back < 2; ++back)
          for (int dt = -1; dt < 3; ++dt)
            for (int dw = 0; dw < 2; ++dw)
              for (uint64_t budget : {(uint64_t)0, (uint64_t)1, (uint64_t)1 << 30, (uint64_t)1 << 40, UINT64_MAX}) {
                if (budget == UINT64_MAX && (d > 1 << 20 || d <= 0)) continue;
                check_plan(back, dt, dw, N, d, V, 0, budget);
                check_plan(back, dt, dw, N, d, V, 300, budget);
              }
    }
  }
  std::mt19937_64 rng(11);
  std::uniform_real_distribution<double> u(0.0, 1.0);
  for (int i = 0; i < 3000; ++i) {
    const auto draw = [&](double most) { return (int64_t)exp2(u(rng) * most); };
    check_logprobs_workspace(draw(23), draw(27), draw(11) - 1);
    check_norm_workspace(draw(33), 8 * draw(12), (int)(u(rng) * 4));
    check_plan(u(rng) < 0.5, u(rng) < 0.5, u(rng) < 0.5, draw(26.5), 8 * draw(13), draw(26.5), u(rng) < 0.5 ? 0 : draw(22),
               (uint64_t)draw(42));
  }
  // refusals, with addresses that are never used
  void* const G = (void*)((uintptr_t)1 << 20);
  float* const F = (float*)G;
  int32_t* const I = (int32_t*)G;
  ckl_drop half{0.5, 1, 2, nullptr}, nan{NAN, 1, 2, nullptr}, odd{0.5, 1, 2, (const int64_t*)((uintptr_t)G + 4)};
  CHECK(ckl_dropout(0, G, 8, nullptr, G, nullptr) == CKL_EINVAL);
  CHECK(ckl_dropout(0, G, 8, &nan, G, nullptr) == CKL_EINVAL);
  CHECK(ckl_dropout(0, G, 8, &odd, G, nullptr) == CKL_EINVAL);
  CHECK(ckl_dropout(0, G, INT64_MAX, &half, G, nullptr) == CKL_EUNSUPPORTED);
  CHECK(ckl_dropout(0, nullptr, 0, &half, nullptr, nullptr) == CKL_OK);
  ckl_norm how{G, G, G, 0, 1.f, 1e-6f, &nan};
  CHECK(ckl_add_norm(0, G, G, &how, 4, 64, G, G, F, nullptr) == CKL_EINVAL);
  how.drop = &half;
  CHECK(ckl_add_norm(0, G, G, &how, 4, 64, G, nullptr, F, nullptr) == CKL_EINVAL);
  CHECK(ckl_add_norm(0, G, G, &how, INT64_MAX, 64, G, G, F, nullptr) == CKL_EUNSUPPORTED);
  CHECK(ckl_add_norm(0, G, G, nullptr, 4, 64, G, G, F, nullptr) == CKL_EINVAL);
  CHECK(ckl_add_norm_bwd(0, G, G, &how, 4, 64, F, G, G, G, G, F, F, G, nullptr, 0, nullptr) == CKL_EINVAL);
  CHECK(ckl_logprobs(0, G, 4, 100, 100, I, 2049, nullptr, 0, F, F, F, nullptr, nullptr, nullptr, 0, nullptr) == CKL_EUNSUPPORTED);
  CHECK(ckl_logprobs(0, G, 4, 100, INT64_MIN, I, 1, nullptr, 0, F, F, F, nullptr, nullptr, nullptr, 0, nullptr) == CKL_EINVAL);
  CHECK(ckl_logprobs_bwd(0, G, (int64_t)1 << 21, kBig, kBig, I, 1, nullptr, F, F, F, F, G, kBig, nullptr) == CKL_EUNSUPPORTED);
  CHECK(ckl_head_logprobs(0, G, G, I, nullptr, kBig, 64, 100, 2048, 0, F, F, F, G, UINT64_MAX, nullptr) == CKL_EUNSUPPORTED);
  CHECK(ckl_head_logprobs(0, G, G, I, nullptr, 4, 64, 100, 1, 0, F, F, F, G, 0, nullptr) == CKL_EINVAL);
  CHECK(ckl_head_logprobs_bwd(1, G, G, I, nullptr, 4, 64, 100, 1, 0, F, F, F, F, F, G, 0, 0, G, G, UINT64_MAX, nullptr) ==
        CKL_EINVAL);
  if (g_fail) {
    fprintf(stderr, "%d checks failed\n", g_fail);
    return 1;
  }
  printf("ok\n");
  return 0;
}
