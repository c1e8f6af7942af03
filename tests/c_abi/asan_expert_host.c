/* Host-side checks of the expert block's C ABI under AddressSanitizer and
 * UndefinedBehaviorSanitizer.
 *
 * Built by tests/test_asan_expert_host.py with the sanitizers on the host code only; every
 * call below returns from its host-side argument checks before any HIP call, so no GPU is
 * needed and no device pointer is ever dereferenced (the "pointers" are small integers).
 * Covers: the host-only size and tile calls over a sweep of sizes, limits and extremes
 * included, checked against the rules moonep.h states; the argument-error and overlap paths
 * of every other call of the block. */
#include <limits.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "moonep.h"

static int g_checks = 0, g_fails = 0;
#define EXPECT(cond)                                                          \
  do {                                                                        \
    ++g_checks;                                                               \
    if (!(cond)) {                                                            \
      ++g_fails;                                                              \
      if (g_fails < 20) printf("FAIL line %d: %s\n", __LINE__, #cond);        \
    }                                                                         \
  } while (0)

/* the rules of the experts' sizes as moonep.h states them; the count of tiles, which is
 * bounded too, stays small for the plans here */
static int expected_ffn(int H, int I) {
  if (H <= 0 || H % 8 || I <= 0 || I % 8) return MOONEP_EINVAL;
  if (H > MOONEP_MAX_FFN || I > MOONEP_MAX_FFN) return MOONEP_ELIMIT;
  if (((long long)I + 256) * H >= 1ll << 30) return MOONEP_ELIMIT;
  return MOONEP_OK;
}
static int expected_rows(int64_t T, int H) {
  if (T < 0 || H <= 0 || H % 8) return MOONEP_EINVAL;
  if (H > MOONEP_MAX_NORM || T > INT32_MAX) return MOONEP_ELIMIT;
  return MOONEP_OK;
}

static void* at(int k) { return (void*)((uintptr_t)k << 40); }   /* never dereferenced */
static uint16_t* u(int k) { return (uint16_t*)at(k); }
static float* f(int k) { return (float*)at(k); }

int main(void) {
  const int sizes[] = {INT_MIN, -8, 0, 4, 8, 16, 32, 40, 64, 1000, 2048, 7168, 16384, 32640, 32760, 32768, 32776,
                       1 << 20, 1 << 30, INT_MAX - 7, INT_MAX};
  const int ns = (int)(sizeof(sizes) / sizeof(sizes[0]));
  const int64_t counts[] = {INT64_MIN, -1, 0, 1, 2, 1000, 1 << 20, INT32_MAX, (int64_t)INT32_MAX + 1, INT64_MAX};
  const int nc = (int)(sizeof(counts) / sizeof(counts[0]));
  const int shapes[][5] = {{4, 16, 2, 64, 4}, {1, 1, 1, 1, 0}, {64, 1024, 32, 64, 256}, {8, 64, 8, 4096, 3}};
  moonep_plan_desc d;

  /* 1. tiles and sizes */
  for (int k = 0; k < 4; ++k) {
    memset(&d, 0, sizeof(d));
    d.magic = 0x4D4F4E45u;
    d.dev = at(1);
    EXPECT(moonep_query(shapes[k][0], shapes[k][1], shapes[k][2], shapes[k][3], shapes[k][4], &d.sz) == MOONEP_OK);
    for (int a = 0; a < ns; ++a)
      for (int b = 0; b < ns; ++b)
        for (int p = -1; p <= 5; ++p) {
          int32_t t[3] = {-1, -1, -1};
          const int want = expected_ffn(sizes[a], sizes[b]);
          const int rc = moonep_expert_tile(&d, sizes[a], sizes[b], p, t);
          EXPECT(rc == (want != MOONEP_OK ? want : p < 0 || p > 4 ? MOONEP_EINVAL : MOONEP_OK));
          if (rc != MOONEP_OK) continue;
          EXPECT(t[0] == 128 || t[0] == 256);
          EXPECT(t[1] == 32 || t[1] == 64 || t[1] == 128 || t[1] == 256);
          EXPECT(t[2] == 0 || (t[2] == 1 && p == MOONEP_PRODUCT_G_WEIGHTS && t[0] == 256));
        }
    EXPECT(moonep_expert_tile(&d, 64, 32, 0, NULL) == MOONEP_EINVAL);
  }
  for (int a = 0; a < ns; ++a) {
    const int64_t b = moonep_q8_row_bytes(sizes[a]);
    if (sizes[a] <= 0 || sizes[a] % 32) EXPECT(b == MOONEP_EINVAL);
    else if (sizes[a] > MOONEP_MAX_NORM) EXPECT(b == MOONEP_ELIMIT);
    else EXPECT(b % 16 == 0 && b >= sizes[a] / 32 * 33 && b < sizes[a] / 32 * 33 + 16);
    for (int c = 0; c < nc; ++c) {
      const int64_t w = moonep_rmsnorm_bwd_workspace(counts[c], sizes[a]);
      const int want = expected_rows(counts[c], sizes[a]);
      if (want != MOONEP_OK) EXPECT(w == want);
      else EXPECT(w >= 0 && w % 4 == 0 && w <= counts[c] * sizes[a] * 4);
    }
  }

  /* 2. the experts' calls */
  memset(&d, 0, sizeof(d));
  EXPECT(moonep_expert_ffn(&d, u(2), 64, 32, 0, u(3), u(4), 6144, u(5), u(6), u(7), 0) == MOONEP_EPLAN);
  EXPECT(moonep_expert_ffn(NULL, u(2), 64, 32, 0, u(3), u(4), 6144, u(5), u(6), u(7), 0) == MOONEP_EPLAN);
  EXPECT(moonep_expert_ffn_bwd_data(&d, u(2), u(3), 64, 32, 0, u(4), u(5), 6144, u(6), u(7), 0) == MOONEP_EPLAN);
  EXPECT(moonep_expert_ffn_bwd_weight(&d, u(2), u(3), u(4), u(5), 64, 32, f(6), f(7), 6144, 0, 0) == MOONEP_EPLAN);
  EXPECT(moonep_expert_tile(&d, 64, 32, 0, (int32_t[3]){0}) == MOONEP_EPLAN);
  d.magic = 0x4D4F4E45u;
  d.dev = at(1);
  EXPECT(moonep_query(4, 16, 2, 4, 4, &d.sz) == MOONEP_OK);
  for (int a = 0; a < ns; ++a)
    for (int b = 0; b < ns; ++b) {
      const int H = sizes[a], I = sizes[b], want = expected_ffn(H, I);
      if (want == MOONEP_OK) {
        /* sizes that are taken: a pitch that is not, a missing buffer, one that is not aligned */
        const int64_t el = 3ll * H * I;
        const int64_t bad[] = {INT64_MIN, -8, 0, el - 8, el + 4, INT64_MAX};
        for (int k = 0; k < 6; ++k) {
          EXPECT(moonep_expert_ffn(&d, u(2), H, I, 0, u(3), u(4), bad[k], u(5), u(6), u(7), 0) == MOONEP_EINVAL);
          EXPECT(moonep_expert_ffn_bwd_data(&d, u(2), u(3), H, I, 0, u(4), u(5), bad[k], u(6), u(7), 0) == MOONEP_EINVAL);
        }
        EXPECT(moonep_expert_ffn_bwd_weight(&d, u(2), u(3), u(4), u(5), H, I, f(6), f(7), el - 4, 0, 0) == MOONEP_EINVAL);
        EXPECT(moonep_expert_ffn_bwd_weight(&d, u(2), u(3), u(4), u(5), H, I, f(6), f(7), el + 2, 0, 0) == MOONEP_EINVAL);
        EXPECT(moonep_expert_ffn_bwd_weight(&d, u(2), u(3), u(4), u(5), H, I, f(6), f(7), el, 2, 0) == MOONEP_EINVAL);
        EXPECT(moonep_expert_ffn(&d, u(2), H, I, 2, u(3), u(4), el, u(5), u(6), u(7), 0) == MOONEP_EINVAL);
        EXPECT(moonep_expert_ffn(&d, u(2), H, I, 0, u(3), NULL, el, u(5), u(6), u(7), 0) == MOONEP_EINVAL);
        EXPECT(moonep_expert_ffn(&d, u(2), H, I, 0, u(3), u(4), el, u(5), u(6), u(7) + 4, 0) == MOONEP_EALIGN);
        EXPECT(moonep_expert_ffn_bwd_data(&d, u(2), u(3) + 4, H, I, 1, u(4), u(5), el, u(6), u(7), 0) == MOONEP_EALIGN);
        EXPECT(moonep_expert_ffn_bwd_weight(&d, u(2), u(3), u(4), u(5), H, I, f(6), f(7) + 2, el, 0, 0) == MOONEP_EALIGN);
        /* overlaps: with another output, with an input, with the plan; pitches up to the largest */
        const int64_t big = INT64_MAX / 8 * 8;
        EXPECT(moonep_expert_ffn(&d, u(2), H, I, 0, u(3), u(4), el, u(5), u(6), u(6), 0) == MOONEP_EINVAL);
        EXPECT(moonep_expert_ffn(&d, u(2), H, I, 0, u(3), u(4), el, u(5), u(6), u(2) + 8, 0) == MOONEP_EINVAL);
        EXPECT(moonep_expert_ffn(&d, u(2), H, I, 0, u(3), u(4), el, u(1), u(6), u(7), 0) == MOONEP_EINVAL);
        EXPECT(moonep_expert_ffn(&d, u(2), H, I, 0, u(3), u(4), big, u(5), u(6), u(7), 0) == MOONEP_EINVAL);
        EXPECT(moonep_expert_ffn_bwd_data(&d, u(2), u(3), H, I, 0, u(4), u(5), el, u(3) + 8, u(7), 0) == MOONEP_EINVAL);
        EXPECT(moonep_expert_ffn_bwd_data(&d, u(2), u(3), H, I, 0, u(4), u(5), big, u(3), u(7), 0) == MOONEP_EINVAL);
        EXPECT(moonep_expert_ffn_bwd_weight(&d, u(2), u(3), u(4), u(5), H, I, f(6), f(6), el, 0, 0) == MOONEP_EINVAL);
        EXPECT(moonep_expert_ffn_bwd_weight(&d, u(2), u(3), u(4), u(5), H, I, f(6), f(7), big, 0, 0) == MOONEP_EINVAL);
        continue;
      }
      EXPECT(moonep_expert_ffn(&d, u(2), H, I, 0, u(3), u(4), INT64_MAX - 7, u(5), u(6), u(7), 0) == want);
      EXPECT(moonep_expert_ffn_bwd_data(&d, u(2), u(3), H, I, 0, u(4), u(5), INT64_MAX - 7, u(6), u(7), 0) == want);
      EXPECT(moonep_expert_ffn_bwd_weight(&d, u(2), u(3), u(4), u(5), H, I, f(6), f(7), INT64_MAX - 7, 0, 0) == want);
    }

  /* 3. the norm's */
  for (int a = 0; a < ns; ++a)
    for (int c = 0; c < nc; ++c) {
      const int H = sizes[a];
      const int64_t T = counts[c];
      int want = expected_rows(T, H);
      if (want != MOONEP_OK) {
        EXPECT(moonep_rmsnorm(u(2), u(3), u(4), 1e-6f, T, H, u(5), u(6), f(7), 0) == want);
        EXPECT(moonep_rmsnorm_q8(u(2), u(3), u(4), 1e-6f, T, H, at(5), u(6), f(7), 0) == want);
        EXPECT(moonep_rmsnorm_bwd(u(2), u(3), u(4), f(5), u(6), T, H, at(7), u(8), f(9), 0) == want);
      } else if (T > 0) {
        EXPECT(moonep_rmsnorm(u(2), u(3), u(4), -1.f, T, H, u(5), u(6), f(7), 0) == MOONEP_EINVAL);
        EXPECT(moonep_rmsnorm(u(2), u(3), u(4), 1e-6f, T, H, NULL, u(6), f(7), 0) == MOONEP_EINVAL);
        EXPECT(moonep_rmsnorm(u(2), u(3), u(4), 1e-6f, T, H, u(5) + 4, u(6), f(7), 0) == MOONEP_EALIGN);
        EXPECT(moonep_rmsnorm(u(2), u(3), u(4), 1e-6f, T, H, u(3), u(6), f(7), 0) == MOONEP_EINVAL);
        EXPECT(moonep_rmsnorm(u(2), u(3), u(4), 1e-6f, T, H, u(5), u(4), f(7), 0) == MOONEP_EINVAL);
        EXPECT(moonep_rmsnorm_bwd(u(2), u(3), u(4), f(5), u(6), T, H, NULL, u(8), f(9), 0) == MOONEP_EINVAL);
        EXPECT(moonep_rmsnorm_bwd(u(2), u(3), u(4), f(5), u(6), T, H, u(7) + 8, u(8), f(9), 0) == MOONEP_EALIGN);
        EXPECT(moonep_rmsnorm_bwd(u(2), u(3), u(4), f(5), u(6), T, H, at(8), u(8), f(9), 0) == MOONEP_EINVAL);
        EXPECT(moonep_rmsnorm_bwd(u(2), u(3), u(4), f(5), u(6), T, H, at(7), u(3), f(7), 0) == MOONEP_EINVAL);
      } else {
        EXPECT(moonep_rmsnorm(NULL, NULL, NULL, 1e-6f, 0, H, NULL, NULL, NULL, 0) == MOONEP_OK);
        EXPECT(moonep_rmsnorm_bwd(NULL, NULL, NULL, NULL, NULL, 0, H, NULL, NULL, NULL, 0) == MOONEP_EINVAL);
      }
      want = H <= 0 || H % 32 ? MOONEP_EINVAL : H > MOONEP_MAX_NORM ? MOONEP_ELIMIT : T < 0 ? MOONEP_EINVAL
             : T > INT32_MAX ? MOONEP_ELIMIT : T == 0 ? MOONEP_OK : MOONEP_EINVAL;
      EXPECT(moonep_q8_unpack(NULL, T, H, u(2), 0) == want);
      EXPECT(moonep_q8_unpack(at(3), T, H, u(3), 0) == want);
    }

  printf("asan expert host %s: %d checks, %d failed\n", g_fails ? "FAILED" : "ok", g_checks, g_fails);
  return g_fails ? 1 : 0;
}
