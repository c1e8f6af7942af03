// The root-mean-square norm in front of the experts: the residual's addition, an output in
// bf16 or in 8 bits with scales (rows that moonep_dispatch moves as they are), the
// expansion of such rows, and the backward pass.
#include "moonep_internal.h"

namespace moonep {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t bf2(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  bf16x2 v{(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d; d /= 2) v += __shfl_xor(v, d);
  return v;
}

// Sum over the workgroup, the same in every thread.  Two slots alternate between rows, so
// one barrier a row is enough.
__device__ __forceinline__ float block_sum(float v, float (*part)[8], int slot) {
  const int nw = blockDim.x >> 6;
  v = wave_sum(v);
  if (nw == 1) return v;
  if ((threadIdx.x & 63) == 0) part[slot][threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < nw; ++w) s += part[slot][w];
  return s;
}

constexpr int kOutBf16 = 0, kOutQ8 = 1;
constexpr int kThreads = 512;              // of a workgroup, at most

// A workgroup for each row; a thread holds U vectors of 8 elements, read once.  The kernel is
// an HBM stream: x and the residual in, their sum and the normed row out.  Measured on
// MI355X at 32768 rows of 7168 in 8 bits (1.65 GB): a workgroup a row, past the caches, 264 to
// 271 us (6.1 to 6.3 TB/s); through them 291 us; 8 workgroups a CU that take rows in turn 307
// and 337 us.  In bf16 (1.88 GB) 309 us a call.
// Where the rows fit in the last-level cache their readers find them there, and nothing
// passes it by.
template <int U, int OUT, bool NT>
__global__ __launch_bounds__(kThreads) void norm_kernel(const u32x4* x, const u32x4* res,
                                                        const u32x4* __restrict__ gamma, float eps,
                                                        int64_t T, int nvec, float inv_h, void* out,
                                                        int64_t out_row, u32x4* h_out, float* rstd_out) {
  __shared__ float part[2][8];
  const int tid = threadIdx.x, nt = blockDim.x;
  int slot = 0;
  // once, but for more rows than a grid can have workgroups
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x, slot ^= 1) {
    u32x4 v[U], r[U], gm[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = u * nt + tid;
      v[u] = i < nvec ? load<NT>(x + t * nvec + i) : u32x4{0, 0, 0, 0};
    }
    if (res) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = u * nt + tid;
        r[u] = i < nvec ? load<NT>(res + t * nvec + i) : u32x4{0, 0, 0, 0};
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      gm[u] = u * nt + tid < nvec ? gamma[u * nt + tid] : u32x4{0, 0, 0, 0};
    if (res) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[u][e] = bf2(lo(v[u][e]) + lo(r[u][e]), hi(v[u][e]) + hi(r[u][e]));
    }
    float ss = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        ss = __builtin_fmaf(lo(v[u][e]), lo(v[u][e]), __builtin_fmaf(hi(v[u][e]), hi(v[u][e]), ss));
    const float rstd = 1.f / sqrtf(block_sum(ss, part, slot) * inv_h + eps);
    if (rstd_out && tid == 0) rstd_out[t] = rstd;
    uint8_t* const row = static_cast<uint8_t*>(out) + t * out_row;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = u * nt + tid;
      if (h_out && i < nvec) store<NT>(v[u], h_out + t * nvec + i);
      float y[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y[2 * e] = lo(v[u][e]) * rstd * lo(gm[u][e]);
        y[2 * e + 1] = hi(v[u][e]) * rstd * hi(gm[u][e]);
      }
      if constexpr (OUT == kOutBf16) {
        u32x4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = bf2(y[2 * e], y[2 * e + 1]);
        if (i < nvec) store<NT>(o, reinterpret_cast<u32x4*>(row) + i);
      } else {
        // a block of 32 elements is 4 lanes (nvec is a multiple of 4).  Its scale is the
        // smallest power of two that brings the largest magnitude m * 2^E (1 <= m < 2) to
        // 448 = 1.75 * 2^8 or less.
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(y[e]));
        top = fmaxf(top, __shfl_xor(top, 1));
        top = fmaxf(top, __shfl_xor(top, 2));
        const uint32_t b = __float_as_uint(top);
        const int ex = max((int)(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u), 0);   // with e8m0's bias
        const float inv = __uint_as_float((uint32_t)(254 - ex) << 23);
        int c0 = 0, c1 = 0;
        c0 = __builtin_amdgcn_cvt_pk_fp8_f32(y[0] * inv, y[1] * inv, c0, false);
        c0 = __builtin_amdgcn_cvt_pk_fp8_f32(y[2] * inv, y[3] * inv, c0, true);
        c1 = __builtin_amdgcn_cvt_pk_fp8_f32(y[4] * inv, y[5] * inv, c1, false);
        c1 = __builtin_amdgcn_cvt_pk_fp8_f32(y[6] * inv, y[7] * inv, c1, true);
        if (i < nvec) {
          store<NT>(u32x2{(uint32_t)c0, (uint32_t)c1}, reinterpret_cast<u32x2*>(row) + i);
          if ((i & 3) == 0) row[nvec * 8 + (i >> 2)] = (uint8_t)ex;
        }
      }
    }
    if constexpr (OUT == kOutQ8) {
      const int end = nvec * 8 + (nvec >> 2);              // codes, scales, then zeros
      if (end + tid < out_row && tid < 16) row[end + tid] = 0;
    }
  }
}

// 8 elements a thread: the codes and the block's scale, expanded exactly.  A stream: 33
// bytes in for 64 out.  A grid as long as the rows, 113 to 116 us at 32768 rows of 7168 (6.2
// TB/s), against 131 us with 16 workgroups a CU that go on.
__global__ __launch_bounds__(256) void unpack_kernel(const uint8_t* __restrict__ rows, int64_t N,
                                                     int nvec, int64_t row_bytes,
                                                     u32x4* __restrict__ out) {
  for (int64_t first = (int64_t)blockIdx.x * 256; first < N * nvec; first += (int64_t)gridDim.x * 256) {
    const int64_t t0 = first / nvec;                       // uniform: one long division
    const uint32_t rem = (uint32_t)(first - t0 * nvec) + threadIdx.x, more = rem / (uint32_t)nvec;
    const int64_t t = t0 + more;
    const int v = (int)(rem - more * nvec);
    if (t >= N) return;
    const uint8_t* row = rows + t * row_bytes;
    const u32x2 c = reinterpret_cast<const u32x2*>(row)[v];
    const int ex = row[nvec * 8 + (v >> 2)];
    u32x4 o;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int w = (int)c[e >> 1];
      const f32x2 p = e & 1 ? __builtin_amdgcn_cvt_pk_f32_fp8(w, true) : __builtin_amdgcn_cvt_pk_f32_fp8(w, false);
      o[e] = bf2(ldexpf(p[0], ex - 127), ldexpf(p[1], ex - 127));
    }
    out[first + threadIdx.x] = o;
  }
}

// g_x = g_h + rstd (gg - xhat mean(gg xhat)), gg = g gamma, xhat = h rstd; the workgroup's
// sum of g xhat over its rows goes to its row of `partial`.  A stream of three rows in and
// one out; a workgroup takes rows in turn, holding gamma and its sums in registers, and (for
// U <= 2) reads the next row before it waits for the others of this one; for longer rows g_h
// is read when it is needed.
template <int U, bool NT>
__global__ __launch_bounds__(kThreads) void norm_bwd_kernel(const u32x4* g, const u32x4* h,
                                                            const u32x4* __restrict__ gamma,
                                                            const float* __restrict__ rstd,
                                                            const u32x4* g_h, int64_t T, int nvec,
                                                            float inv_h, u32x4* g_x, f32x4* partial) {
  __shared__ float part[2][8];
  constexpr bool kAhead = U <= 2;
  const int tid = threadIdx.x, nt = blockDim.x;
  u32x4 gm[U], a[U], b[U], c[U], a1[U], b1[U], c1[U];
  float rs = 0.f, rs1 = 0.f;
  float acc[U][8];
  auto fetch = [&](int64_t t, u32x4 (&a)[U], u32x4 (&b)[U], u32x4 (&c)[U], float& rs) {
    rs = rstd[t];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = u * nt + tid;
      const bool in = i < nvec;
      a[u] = in ? load<NT>(g + t * nvec + i) : u32x4{0, 0, 0, 0};
      b[u] = in ? load<NT>(h + t * nvec + i) : u32x4{0, 0, 0, 0};
      if (kAhead) c[u] = in && g_h ? load<NT>(g_h + t * nvec + i) : u32x4{0, 0, 0, 0};
    }
  };
#pragma unroll
  for (int u = 0; u < U; ++u) {
    gm[u] = u * nt + tid < nvec ? gamma[u * nt + tid] : u32x4{0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[u][e] = 0.f;
  }
  int slot = 0;
  if constexpr (kAhead) fetch(blockIdx.x, a, b, c, rs);
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x, slot ^= 1) {
    if constexpr (kAhead) {
      if (t + gridDim.x < T) fetch(t + gridDim.x, a1, b1, c1, rs1);
    } else {
      fetch(t, a, b, c, rs);
    }
    float dot = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float n0 = lo(b[u][e]) * rs, n1 = hi(b[u][e]) * rs;
        const float g0 = lo(a[u][e]), g1 = hi(a[u][e]);
        acc[u][2 * e] = __builtin_fmaf(g0, n0, acc[u][2 * e]);
        acc[u][2 * e + 1] = __builtin_fmaf(g1, n1, acc[u][2 * e + 1]);
        dot = __builtin_fmaf(g0 * lo(gm[u][e]), n0, dot);
        dot = __builtin_fmaf(g1 * hi(gm[u][e]), n1, dot);
      }
    const float m = block_sum(dot, part, slot) * inv_h;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = u * nt + tid;
      if (!kAhead) c[u] = i < nvec && g_h ? load<NT>(g_h + t * nvec + i) : u32x4{0, 0, 0, 0};
      u32x4 o;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float n0 = lo(b[u][e]) * rs, n1 = hi(b[u][e]) * rs;
        const float d0 = rs * (lo(a[u][e]) * lo(gm[u][e]) - n0 * m);
        const float d1 = rs * (hi(a[u][e]) * hi(gm[u][e]) - n1 * m);
        o[e] = bf2(d0 + lo(c[u][e]), d1 + hi(c[u][e]));
      }
      if (i < nvec) g_x[t * nvec + i] = o;
    }
    if constexpr (kAhead) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        a[u] = a1[u];
        b[u] = b1[u];
        c[u] = c1[u];
      }
      rs = rs1;
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = u * nt + tid;
    if (i < nvec) {
      f32x4* p = partial + ((int64_t)blockIdx.x * nvec + i) * 2;
      p[0] = f32x4{acc[u][0], acc[u][1], acc[u][2], acc[u][3]};
      p[1] = f32x4{acc[u][4], acc[u][5], acc[u][6], acc[u][7]};
    }
  }
}

// Column sums of the partial rows, in a fixed order: 64 threads to 4 columns, each a part of
// the rows.
constexpr int kGammaParts = 64;
__global__ __launch_bounds__(1024) void gamma_kernel(const f32x4* __restrict__ partial, int rows,
                                                     int ncol4, f32x4* __restrict__ g_gamma) {
  __shared__ f32x4 sums[kGammaParts][16];
  const int c = threadIdx.x & 15, part = threadIdx.x >> 4;
  const int col = blockIdx.x * 16 + c;
  f32x4 s{0.f, 0.f, 0.f, 0.f};
  if (col < ncol4) {
#pragma unroll 8
    for (int r = part; r < rows; r += kGammaParts) s = s + partial[(int64_t)r * ncol4 + col];
  }
  sums[part][c] = s;
  for (int half = kGammaParts / 2; half; half /= 2) {
    __syncthreads();
    if (part < half) sums[part][c] = s = s + sums[part + half][c];
  }
  if (part == 0 && col < ncol4) g_gamma[col] = s;
}

constexpr int kCus = 256;
constexpr int64_t kLastLevelCacheBytes = 256ll << 20;

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Vectors a thread (of those there are kernels for) and threads of a workgroup for rows of
// nvec vectors: the fewest vectors that fit.
void shape(int nvec, int* threads, int* u) {
  for (int k : {1, 2, 3, 4, 8}) {
    *u = k;
    *threads = ((nvec + k - 1) / k + 63) / 64 * 64;
    if (*threads <= kThreads) return;
  }
}

// Workgroups of the backward kernel: one for each CU, or as many short ones as take its place
// if they have four rows each (each costs a row of partial sums).
// At 16384 rows of 7168 (940 MB) one measured 142 us (6.6 TB/s) and 4 for the column sums; a call
// took 152 (165 on other boxes) with one, 162 with two, 190 with three without the rows ahead.
int bwd_blocks(int64_t T, int H) {
  int threads, u;
  shape(H / 8, &threads, &u);
  return (int)std::min<int64_t>(T, std::max<int64_t>(kCus, std::min<int64_t>(kCus * (kThreads / threads), T / 4)));
}

// A launch has fewer than 2^32 threads.
unsigned grid_of(int64_t blocks, int threads) {
  return (unsigned)std::min<int64_t>(blocks, UINT32_MAX / threads);
}

int check_rows(int64_t T, int H) {
  if (T < 0 || H <= 0 || H % 8 != 0) return MOONEP_EINVAL;
  if (H > MOONEP_MAX_NORM || T > INT32_MAX) return MOONEP_ELIMIT;
  return MOONEP_OK;
}

template <int OUT>
int norm(const uint16_t* x, const uint16_t* res, const uint16_t* gamma, float eps, int64_t T, int H,
         void* out, int64_t out_row, uint16_t* h_out, float* rstd, hipStream_t st) {
  if (T == 0) return MOONEP_OK;
  if (!x || !gamma || !out || !(eps >= 0.f)) return MOONEP_EINVAL;
  if (!aligned(x, 16) || !aligned(res, 16) || !aligned(gamma, 16) || !aligned(out, 16) ||
      !aligned(h_out, 16) || !aligned(rstd, 4))
    return MOONEP_EALIGN;
  // A workgroup has read its row when it writes it, so h may be x or res.  Anything else that
  // overlaps would be written before another workgroup reads it, or be lost to the backward pass.
  const Span xs = span(x, T, 2ll * H), rs = span(res, T, 2ll * H), gs = span(gamma, 1, 2ll * H);
  const Span os = span(out, T, out_row), hs = span(h_out, T, 2ll * H), ss = span(rstd, T, 4);
  if (overlap(os, {xs, rs, gs, hs, ss}) || overlap(ss, {xs, rs, gs, hs}) || overlap(hs, gs) ||
      (h_out != x && overlap(hs, xs)) || (h_out != res && overlap(hs, rs)))
    return MOONEP_EINVAL;
  int threads, u;
  shape(H / 8, &threads, &u);
  const bool nt = T * H * 8 > kLastLevelCacheBytes;     // of all rows
  const auto* xv = reinterpret_cast<const u32x4*>(x);
  const auto* rv = reinterpret_cast<const u32x4*>(res);
  const auto* gv = reinterpret_cast<const u32x4*>(gamma);
  auto* hv = reinterpret_cast<u32x4*>(h_out);
  (void)hipGetLastError();
  auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(grid_of(T, threads)), dim3(threads), 0, st, xv, rv, gv, eps, T, H / 8, 1.f / H, out,
                       out_row, hv, rstd);
  };
#define NORM(U) nt ? launch(norm_kernel<U, OUT, true>) : launch(norm_kernel<U, OUT, false>)
  if (u == 1) NORM(1); else if (u == 2) NORM(2); else if (u == 3) NORM(3); else if (u == 4) NORM(4); else NORM(8);
#undef NORM
  return hipGetLastError() == hipSuccess ? MOONEP_OK : MOONEP_EHIP;
}

}  // namespace
}  // namespace moonep

using namespace moonep;

extern "C" {

int64_t moonep_q8_row_bytes(int H) {
  if (H <= 0 || H % 32 != 0) return MOONEP_EINVAL;
  if (H > MOONEP_MAX_NORM) return MOONEP_ELIMIT;
  return ((int64_t)H + H / 32 + 15) / 16 * 16;
}

int moonep_rmsnorm(const uint16_t* x, const uint16_t* res, const uint16_t* gamma, float eps,
                   int64_t T, int H, uint16_t* out, uint16_t* h, float* rstd, hipStream_t stream) {
  const int rc = check_rows(T, H);
  if (rc != MOONEP_OK) return rc;
  return norm<kOutBf16>(x, res, gamma, eps, T, H, out, 2ll * H, h, rstd, stream);
}

int moonep_rmsnorm_q8(const uint16_t* x, const uint16_t* res, const uint16_t* gamma, float eps,
                      int64_t T, int H, uint8_t* rows, uint16_t* h, float* rstd, hipStream_t stream) {
  const int rc = check_rows(T, H);
  if (rc != MOONEP_OK) return rc;
  const int64_t rb = moonep_q8_row_bytes(H);
  if (rb < 0) return (int)rb;
  return norm<kOutQ8>(x, res, gamma, eps, T, H, rows, rb, h, rstd, stream);
}

int moonep_q8_unpack(const uint8_t* rows, int64_t N, int H, uint16_t* out, hipStream_t stream) {
  const int64_t rb = moonep_q8_row_bytes(H);
  if (rb < 0) return (int)rb;
  if (N < 0) return MOONEP_EINVAL;
  if (N > INT32_MAX) return MOONEP_ELIMIT;
  if (N == 0) return MOONEP_OK;
  if (!rows || !out) return MOONEP_EINVAL;
  if (!aligned(rows, 16) || !aligned(out, 16)) return MOONEP_EALIGN;
  if (overlap(span(rows, N, rb), span(out, N, 2ll * H))) return MOONEP_EINVAL;
  const int64_t blocks = (N * (H / 8) + 255) / 256;
  (void)hipGetLastError();
  hipLaunchKernelGGL(unpack_kernel, dim3(grid_of(blocks, 256)), dim3(256), 0, stream, rows, N, H / 8, rb, reinterpret_cast<u32x4*>(out));
  return hipGetLastError() == hipSuccess ? MOONEP_OK : MOONEP_EHIP;
}

int64_t moonep_rmsnorm_bwd_workspace(int64_t T, int H) {
  const int rc = check_rows(T, H);
  if (rc != MOONEP_OK) return rc;
  return (int64_t)bwd_blocks(T, H) * H * 4;
}

int moonep_rmsnorm_bwd(const uint16_t* g_out, const uint16_t* h, const uint16_t* gamma,
                       const float* rstd, const uint16_t* g_h, int64_t T, int H, void* workspace,
                       uint16_t* g_x, float* g_gamma, hipStream_t stream) {
  const int rc = check_rows(T, H);
  if (rc != MOONEP_OK) return rc;
  if (!gamma || !g_gamma || (T > 0 && (!g_out || !h || !rstd || !workspace || !g_x)))
    return MOONEP_EINVAL;
  if (!aligned(g_out, 16) || !aligned(h, 16) || !aligned(gamma, 16) || !aligned(rstd, 4) ||
      !aligned(g_h, 16) || !aligned(workspace, 256) || !aligned(g_x, 16) || !aligned(g_gamma, 16))
    return MOONEP_EALIGN;
  const Span gs = span(g_out, T, 2ll * H), hs = span(h, T, 2ll * H), ghs = span(g_h, T, 2ll * H);
  const Span gm = span(gamma, 1, 2ll * H), rs = span(rstd, T, 4);
  const Span xs = span(g_x, T, 2ll * H), ws = span(workspace, bwd_blocks(T, H), 4ll * H), os = span(g_gamma, 1, 4ll * H);
  if (overlap(xs, {gm, rs, ws, os}) || (g_x != g_out && overlap(xs, gs)) || (g_x != h && overlap(xs, hs)) ||
      (g_x != g_h && overlap(xs, ghs)) || overlap(ws, {gs, hs, ghs, gm, rs, os}) || overlap(os, {gs, hs, ghs, gm, rs}))
    return MOONEP_EINVAL;
  int threads, u;
  shape(H / 8, &threads, &u);
  const int grid = bwd_blocks(T, H);
  const bool nt = T * H * 8 > kLastLevelCacheBytes;     // of all rows
  (void)hipGetLastError();
  if (grid) {
    auto launch = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3(grid), dim3(threads), 0, stream, reinterpret_cast<const u32x4*>(g_out),
                         reinterpret_cast<const u32x4*>(h), reinterpret_cast<const u32x4*>(gamma), rstd,
                         reinterpret_cast<const u32x4*>(g_h), T, H / 8, 1.f / H, reinterpret_cast<u32x4*>(g_x),
                         static_cast<f32x4*>(workspace));
    };
#define BWD(U) nt ? launch(norm_bwd_kernel<U, true>) : launch(norm_bwd_kernel<U, false>)
    if (u == 1) BWD(1); else if (u == 2) BWD(2); else if (u == 3) BWD(3); else if (u == 4) BWD(4); else BWD(8);
#undef BWD
    if (hipGetLastError() != hipSuccess) return MOONEP_EHIP;
  }
  hipLaunchKernelGGL(gamma_kernel, dim3((H / 4 + 15) / 16), dim3(1024), 0, stream,
                     static_cast<const f32x4*>(workspace), grid, H / 4,
                     reinterpret_cast<f32x4*>(g_gamma));
  return hipGetLastError() == hipSuccess ? MOONEP_OK : MOONEP_EHIP;
}

}  // extern "C"
