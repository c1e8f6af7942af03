/* Host-side checks of the experts in 4 bits and of the router under AddressSanitizer and
 * UndefinedBehaviorSanitizer.
 *
 * Built by tests/test_asan_w4_host.py with the sanitizers on the host code only; every call
 * below returns from its host-side argument checks before any HIP call, so no GPU is needed and no device
 * pointer is ever dereferenced (the "pointers" are small integers).  Covers: the host-only size and tile calls over a sweep
 * of sizes, limits and extremes included, checked against the rules moonep.h states; the
 * argument-error and overlap paths of the other calls. */
#include <limits.h>
#include <math.h>
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

static int expected_w4(int H, int I) {
  if (H <= 0 || H % 8 || I <= 0 || I % 8) return MOONEP_EINVAL;
  if (H > MOONEP_MAX_FFN || I > MOONEP_MAX_FFN) return MOONEP_ELIMIT;
  return MOONEP_OK;
}
static int expected_router(int64_t T, int E, int K) {
  if (T < 0 || E < 1 || K < 1 || K > E) return MOONEP_EINVAL;
  if (E > MOONEP_MAX_E || K > MOONEP_MAX_K || T > INT32_MAX) return MOONEP_ELIMIT;
  return MOONEP_OK;
}

static void* at(int k) { return (void*)((uintptr_t)k << 42); }   /* never dereferenced */
static uint16_t* u(int k) { return (uint16_t*)at(k); }
static uint8_t* b(int k) { return (uint8_t*)at(k); }
static float* f(int k) { return (float*)at(k); }
static int32_t* n(int k) { return (int32_t*)at(k); }

int main(void) {
  const int sizes[] = {INT_MIN, -8, 0, 4, 8, 16, 32, 40, 64, 1000, 2048, 7168, 16384, 32640, 32760, 32768, 32776,
                       1 << 20, 1 << 30, INT_MAX - 7, INT_MAX};
  const int ns = (int)(sizeof(sizes) / sizeof(sizes[0]));
  const int64_t counts[] = {INT64_MIN, -1, 0, 1, 2, 1000, 1 << 20, INT32_MAX, (int64_t)INT32_MAX + 1, INT64_MAX};
  const int nc = (int)(sizeof(counts) / sizeof(counts[0]));
  const int shapes[][5] = {{4, 16, 2, 64, 4}, {1, 1, 1, 1, 0}, {64, 1024, 32, 64, 256}, {8, 64, 8, 4096, 3}};
  moonep_plan_desc d;

  /* 1. sizes of slabs and tiles */
  for (int k = 0; k < 4; ++k) {
    memset(&d, 0, sizeof(d));
    EXPECT(moonep_expert_tile_w4(&d, 64, 32, 0, 0, n(2)) == MOONEP_EPLAN);
    d.magic = 0x4D4F4E45u;
    d.dev = at(1);
    EXPECT(moonep_query(shapes[k][0], shapes[k][1], shapes[k][2], shapes[k][3], shapes[k][4], &d.sz) == MOONEP_OK);
    for (int x = 0; x < ns; ++x)
      for (int y = 0; y < ns; ++y) {
        const int H = sizes[x], I = sizes[y], want = expected_w4(H, I);
        const int64_t bytes = moonep_w4_slab_bytes(H, I);
        if (want != MOONEP_OK) EXPECT(bytes == want);
        else EXPECT(bytes % 256 == 0 && bytes >= 3ll * H * I / 32 * 17);
        for (int q8 = -1; q8 <= 2; ++q8)
          for (int p = -1; p <= 2; ++p) {
            int32_t t[2] = {-1, -1};
            const int rc = moonep_expert_tile_w4(&d, H, I, q8, p, t);
            const int bad = q8 < 0 || q8 > 1 || p < 0 || p > 1 || (q8 == 1 && (H % 32 || I % 32));
            EXPECT(rc == (want != MOONEP_OK ? want : bad ? MOONEP_EINVAL : MOONEP_OK));
            if (rc == MOONEP_OK) EXPECT((t[0] == 128 || t[0] == 256) && t[1] >= 16 && t[1] <= 256);
          }
      }
  }

  /* 2. packing and the experts */
  EXPECT(moonep_query(4, 16, 2, 4, 4, &d.sz) == MOONEP_OK);
  for (int x = 0; x < ns; ++x)
    for (int y = 0; y < ns; ++y) {
      const int H = sizes[x], I = sizes[y], want = expected_w4(H, I);
      if (want != MOONEP_OK) {
        EXPECT(moonep_w4_pack(u(2), INT64_MAX - 7, 1, H, I, b(3), INT64_MAX - 15, 0) == want);
        EXPECT(moonep_w4_unpack(b(2), INT64_MAX - 15, 1, H, I, u(3), INT64_MAX - 7, 0) == want);
        EXPECT(moonep_expert_ffn_w4(&d, u(2), H, I, 0, b(3), b(4), INT64_MAX - 15, u(5), u(6), u(7), 0) == want);
        EXPECT(moonep_expert_ffn_w4q8(&d, b(2), H, I, 0, b(3), b(4), INT64_MAX - 15, b(6), u(7), 0) == want);
        continue;
      }
      const int64_t el = 3ll * H * I, by = moonep_w4_slab_bytes(H, I);
      for (int c = 0; c < nc; ++c) {
        const int64_t m = counts[c];
        const int rc = m < 0 ? MOONEP_EINVAL : m > INT32_MAX ? MOONEP_ELIMIT : m == 0 ? MOONEP_OK : MOONEP_EINVAL;
        EXPECT(moonep_w4_pack(NULL, el, m, H, I, b(3), by, 0) == rc);
        EXPECT(moonep_w4_unpack(b(3), by, m, H, I, u(3) + 8, el, 0) == rc);
      }
      EXPECT(moonep_w4_pack(u(2), el - 8, 1, H, I, b(3), by, 0) == MOONEP_EINVAL);
      EXPECT(moonep_w4_pack(u(2), el + 4, 1, H, I, b(3), by, 0) == MOONEP_EINVAL);
      EXPECT(moonep_w4_pack(u(2), INT64_MIN, 1, H, I, b(3), by, 0) == MOONEP_EINVAL);
      EXPECT(moonep_w4_pack(u(2), el, 1, H, I, b(3), by - 16, 0) == MOONEP_EINVAL);
      EXPECT(moonep_w4_pack(u(2), el, 1, H, I, b(3), by + 8, 0) == MOONEP_EINVAL);
      EXPECT(moonep_w4_pack(u(2) + 4, el, 1, H, I, b(3), by, 0) == MOONEP_EALIGN);
      EXPECT(moonep_w4_unpack(b(2), INT64_MAX - 15, INT32_MAX, H, I, u(3), el, 0) == MOONEP_EINVAL);  /* they overlap */
      const int64_t bad[] = {INT64_MIN, -16, 0, by - 16, by + 8, INT64_MAX};
      for (int k = 0; k < 6; ++k) {
        EXPECT(moonep_expert_ffn_w4(&d, u(2), H, I, 0, b(3), b(4), bad[k], u(5), u(6), u(7), 0) == MOONEP_EINVAL);
        EXPECT(moonep_expert_ffn_w4q8(&d, b(2), H, I, 0, b(3), b(4), bad[k], b(6), u(7), 0) == MOONEP_EINVAL);
      }
      EXPECT(moonep_expert_ffn_w4(&d, u(2), H, I, 2, b(3), b(4), by, u(5), u(6), u(7), 0) == MOONEP_EINVAL);
      EXPECT(moonep_expert_ffn_w4(&d, u(2), H, I, 0, b(3), NULL, by, u(5), u(6), u(7), 0) == MOONEP_EINVAL);
      EXPECT(moonep_expert_ffn_w4(&d, u(2), H, I, 0, b(3) + 8, b(4), by, u(5), u(6), u(7), 0) == MOONEP_EALIGN);
      EXPECT(moonep_expert_ffn_w4(&d, u(2), H, I, 0, b(3), b(4), by, u(6), u(6), u(7), 0) == MOONEP_EINVAL);
      EXPECT(moonep_expert_ffn_w4(&d, u(2), H, I, 0, b(3), b(4), by, u(5), u(6), u(2), 0) == MOONEP_EINVAL);
      EXPECT(moonep_expert_ffn_w4(&d, u(2), H, I, 0, b(3), b(4), INT64_MAX - 15, u(5), u(6), u(7), 0) == MOONEP_EINVAL);
      EXPECT(moonep_expert_ffn_w4q8(&d, b(2), H, I, 0, b(3), b(4), by, b(2), u(7), 0) == MOONEP_EINVAL);
    }

  /* 3. the router */
  const int experts[] = {INT_MIN, -1, 0, 1, 2, 8, 31, 64, 384, 1024, 1025, INT_MAX};
  const int ks[] = {INT_MIN, 0, 1, 2, 8, 32, 33, INT_MAX};
  for (int x = 0; x < 12; ++x)
    for (int k = 0; k < 8; ++k)
      for (int c = 0; c < nc; ++c) {
        const int E = experts[x], K = ks[k];
        const int64_t T = counts[c];
        int want = expected_router(T, E, K);
        if (want == MOONEP_OK && T > 0) want = MOONEP_EINVAL;              /* a missing output */
        for (int dt = 0; dt < 2; ++dt) {
          EXPECT(moonep_router(at(2), dt, f(3), T, E, K, 0, 1, 1, 1, 1.f, n(4), NULL, 0) == want);
          EXPECT(moonep_router_bwd(at(2), dt, n(3), f(4), T, E, K, 1, 0, 1.f, NULL, 0) == want);
        }
        if (want != MOONEP_EINVAL || T <= 0 || expected_router(T, E, K) != MOONEP_OK) continue;
        EXPECT(moonep_router(at(2), 2, f(3), T, E, K, 0, 1, 1, 1, 1.f, n(4), f(5), 0) == MOONEP_EINVAL);
        EXPECT(moonep_router(at(2), 0, f(3), T, E, K, 2, 1, 1, 1, 1.f, n(4), f(5), 0) == MOONEP_EINVAL);
        EXPECT(moonep_router(at(2), 0, f(3), T, E, K, 0, 1, 1, 2, 1.f, n(4), f(5), 0) == MOONEP_EINVAL);
        EXPECT(moonep_router(at(2), 0, f(3), T, E, K, 0, 1, 1, 1, NAN, n(4), f(5), 0) == MOONEP_EINVAL);
        EXPECT(moonep_router(at(2), 0, f(3), T, E, K, 0, 0, 0, 1, 1.f, n(4), f(5), 0) == MOONEP_EINVAL);
        EXPECT(moonep_router(at(2), 0, f(3), T, E, K, 0, 1, 2, 1, 1.f, n(4), f(5), 0) == MOONEP_EINVAL);
        EXPECT(moonep_router(at(2), 0, f(3), T, E, K, 0, INT_MAX, 1, 1, 1.f, n(4), f(5), 0) == MOONEP_EINVAL);
        EXPECT(moonep_router(at(2), 0, f(3), T, E, K, 0, 1, 1, 1, 1.f, n(4), f(4), 0) == MOONEP_EINVAL);
        EXPECT(moonep_router(at(2), 0, f(3), T, E, K, 0, 1, 1, 1, 1.f, n(2), f(5), 0) == MOONEP_EINVAL);
        EXPECT(moonep_router(b(2) + 2, 0, f(3), T, E, K, 0, 1, 1, 1, 1.f, n(4), f(5), 0) == MOONEP_EALIGN);
        EXPECT(moonep_router_bwd(at(2), 0, n(3), f(4), T, E, K, 0, 1, INFINITY, f(5), 0) == MOONEP_EINVAL);
        EXPECT(moonep_router_bwd(at(2), 0, n(3), f(4), T, E, K, 0, 1, 1.f, f(2), 0) == MOONEP_EINVAL);
        EXPECT(moonep_router_bwd(at(2), 1, n(3), f(4), T, E, K, 0, 1, 1.f, b(5) + 1, 0) == MOONEP_EALIGN);
      }

  printf("asan w4 host %s: %d checks, %d failed\n", g_fails ? "FAILED" : "ok", g_checks, g_fails);
  return g_fails ? 1 : 0;
}
