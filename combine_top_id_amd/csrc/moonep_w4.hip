// The gated feed-forward experts with weights in 4 bits, and the packing of such weights.
//
//   value = code * 2^s: an e2m1 code (0, 0.5, 1, 1.5, 2, 3, 4, 6, with a sign) and a power of two
//   for 32 neighbours along k (e8m0: byte b is 2^(b-127)), which is the group that the scaled matrix
//   instructions take.  A value is a bf16 number exactly.
//
// Layout of a slab: what a wave needs for a step, in the order in which its lanes hold it.  A block is
// 64 rows of a matrix (a quad of four strips of 16) times 128 k: 4352 bytes,
//   strip t, lane (g, r) = g * 16 + r: 16 bytes at t * 1024 + lane * 16, the codes of row r of the
//     strip, k = 32 g ... 32 g + 31, two to a byte, the lower k in the lower bits;
//   scales: 4 bytes at 4096 + lane * 4, byte t that of strip t's row r and group g.
// A matrix is its quads in turn, each all its blocks along k; k and rows are filled up with zeros.
//   gate and up (one matrix of 2 I rows of H): row r of strips 0 and 1 of quad q is gate row 32 q + 2 r and
//     32 q + 2 r + 1, of strips 2 and 3 the same rows of up;
//   down (H rows of I): row r of strip t is row 64 q + 4 r + t:
// so that the results that a lane holds of the four strips are neighbours.
#include "moonep_expert.h"

namespace moonep {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kStepK = 128;                // k of a block
constexpr int kBlock = 4352;               // bytes of one
constexpr int kQuadI = 32, kQuadH = 64;    // columns of the products that a quad makes

__host__ __device__ inline int steps_of(int k) { return (k + kStepK - 1) / kStepK; }
__host__ __device__ inline int64_t gate_up_bytes(int H, int I) {
  return (int64_t)((I + kQuadI - 1) / kQuadI) * steps_of(H) * kBlock;
}
__host__ __device__ inline int64_t slab_bytes(int H, int I) {
  return gate_up_bytes(H, I) + (int64_t)((H + kQuadH - 1) / kQuadH) * steps_of(I) * kBlock;
}

// ---------------------------------------------------------------------------------------
// packing
// ---------------------------------------------------------------------------------------

// Block b of an expert's slab: which matrix row strip t's row r is (from the slab's first gate row on, in
// rows of `k` elements from element `at` on), or -1 past the end, and its first k.
struct BlockAt {
  int64_t at;                 // first element of the matrix in a bf16 slab
  int k, k0;
  int quad, H, I;
  bool down;
  __device__ __forceinline__ BlockAt(int64_t b, int H, int I) : H(H), I(I) {
    const int s1 = steps_of(H), s2 = steps_of(I);
    const int64_t n1 = (int64_t)((I + kQuadI - 1) / kQuadI) * s1;
    down = b >= n1;
    if (down) b -= n1;
    const int s = down ? s2 : s1;
    quad = (int)(b / s);
    k0 = (int)(b - (int64_t)quad * s) * kStepK;
    k = down ? I : H;
    at = down ? 2ll * I * H : 0;
  }
  __device__ __forceinline__ int64_t row(int t, int r) const {
    if (down) {
      const int h = quad * kQuadH + 4 * r + t;
      return h < H ? h : -1;
    }
    const int i = quad * kQuadI + 2 * r + (t & 1);
    return i < I ? i + (t >> 1) * (int64_t)I : -1;
  }
};

// A wave a block.  A stream: 64 bytes in for 17 out.
__global__ __launch_bounds__(256) void pack_kernel(const uint16_t* w, int64_t W_el, int64_t n, int H, int I,
                                                   uint8_t* out, int64_t pitch, int64_t per) {
#ifdef __HIP_DEVICE_COMPILE__   // gfx950 builtins: the host pass needs the kernel's name only
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int64_t all = n * per;
  for (int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); i < all; i += (int64_t)gridDim.x * 4) {
    const int64_t e = i / per, b = i - e * per;
    const BlockAt at(b, H, I);
    const int k = at.k0 + 32 * g;
    u32x4 v[4][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int64_t row = at.row(t, r);
      const uint16_t* p = w + e * W_el + at.at + row * at.k + k;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        v[t][c] = row >= 0 && k + 8 * c < at.k ? *reinterpret_cast<const u32x4*>(p + 8 * c) : u32x4{0, 0, 0, 0};
    }
    uint8_t* const to = out + e * pitch + b * kBlock;
    uint32_t scales = 0;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      uint32_t top = 0;                          // bf16 magnitudes compare as their bits do
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int d = 0; d < 4; ++d) top = max(top, max(v[t][c][d] & 0x7FFFu, v[t][c][d] >> 16 & 0x7FFFu));
      // largest = m * 2^E, 1 <= m < 2, and 6 = 1.5 * 2^2; infinities and NaN make the group NaN
      const int ex = top >= 0x7F80u ? 255 : max((int)(top >> 7) - 2 + ((top & 0x7Fu) > 0x40u), 1);
      const float scale = __uint_as_float((uint32_t)ex << 23);
      scales |= (uint32_t)ex << (8 * t);
      u32x4 codes;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t d = 0;
        d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, lo(v[t][c][0]), hi(v[t][c][0]), scale, 0);
        d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, lo(v[t][c][1]), hi(v[t][c][1]), scale, 1);
        d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, lo(v[t][c][2]), hi(v[t][c][2]), scale, 2);
        d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, lo(v[t][c][3]), hi(v[t][c][3]), scale, 3);
        codes[c] = d;
      }
      *reinterpret_cast<u32x4*>(to + t * 1024 + lane * 16) = codes;
    }
    *reinterpret_cast<uint32_t*>(to + 4096 + lane * 4) = scales;
  }
#endif
}

// The eight values of a word of codes, in bf16; scale is a float's exponent (255 makes NaN of them).
__device__ __forceinline__ u32x4 expand(uint32_t codes, float scale) {
#ifdef __HIP_DEVICE_COMPILE__
  return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3))};
#else
  return u32x4{codes, 0, 0, (uint32_t)scale};
#endif
}
__device__ __forceinline__ float strip_scale(uint32_t scales, int t) {
  return __uint_as_float(t < 3 ? scales << (23 - 8 * t) & 0x7F800000u : scales >> 1 & 0x7F800000u);
}

// pack_kernel's inverse, exact.
__global__ __launch_bounds__(256) void unpack_w4_kernel(const uint8_t* in, int64_t pitch, int64_t n, int H, int I,
                                                        uint16_t* w, int64_t W_el, int64_t per) {
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int64_t all = n * per;
  for (int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); i < all; i += (int64_t)gridDim.x * 4) {
    const int64_t e = i / per, b = i - e * per;
    const BlockAt at(b, H, I);
    const int k = at.k0 + 32 * g;
    const uint8_t* from = in + e * pitch + b * kBlock;
    u32x4 codes[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) codes[t] = *reinterpret_cast<const u32x4*>(from + t * 1024 + lane * 16);
    const uint32_t scales = *reinterpret_cast<const uint32_t*>(from + 4096 + lane * 4);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int64_t row = at.row(t, r);
      if (row < 0) continue;
      uint16_t* p = w + e * W_el + at.at + row * at.k + k;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (k + 8 * c < at.k) *reinterpret_cast<u32x4*>(p + 8 * c) = expand(codes[t][c], strip_scale(scales, t));
    }
  }
}

// ---------------------------------------------------------------------------------------
// the experts
// ---------------------------------------------------------------------------------------

enum W4Op { W4_FWD1, W4_FWD2 };

struct W4Args {
  const int32_t* plan;
  moonep_sizes s;
  int H, I, act;
  const uint8_t* in;           // the rows: recv or h
  int64_t in_row;              // bytes of one
  const uint8_t *home, *slot;
  int64_t pitch;
  uint8_t* out;                // h or y
  int64_t out_row;
  uint16_t* gu;                // gate and up rows, or null
  int tiles_bound;             // row tiles of any plan of these sizes, at most
};

// The largest of the 16 lanes of a row, in each of them.
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, quad_move<0xB1>(v));              // of lane ^ 1, of lane ^ 2, then mirrored in 8 and in 16
  v = fmaxf(v, quad_move<0x4E>(v));
  v = fmaxf(v, quad_move<0x141>(v));
  return fmaxf(v, quad_move<0x140>(v));
}

// A lane's results of a quad's four strips, of one buffer row: gate, gate, up, up, or four of y.  `c` is the
// lane's place among the quad's columns.
template <int OP, bool Q8>
__device__ __forceinline__ void put(const W4Args& a, const f32x4& d, int64_t row, bool in, int quad, int c) {
#ifdef __HIP_DEVICE_COMPILE__
  if constexpr (OP == W4_FWD2) {
    const int col = quad * kQuadH + 4 * c;
    if (in && col < a.H)
      *reinterpret_cast<u32x2*>(a.out + row * a.out_row + col * 2) = u32x2{bf2(d[0], d[1]), bf2(d[2], d[3])};
  } else {
    const int col = quad * kQuadI + 2 * c;
    float slope;
    const float h0 = act_of(d[0], a.act, &slope) * d[2], h1 = act_of(d[1], a.act, &slope) * d[3];
    if constexpr (!Q8) {
      if (in && col < a.I) {
        *reinterpret_cast<uint32_t*>(a.out + row * a.out_row + col * 2) = bf2(h0, h1);
        if (a.gu) {
          uint16_t* gu = a.gu + row * 2 * a.I + col;
          *reinterpret_cast<uint32_t*>(gu) = bf2(d[0], d[1]);
          *reinterpret_cast<uint32_t*>(gu + a.I) = bf2(d[2], d[3]);
        }
      }
    } else {
      // the rule of the 8-bit norm: the smallest power of two that brings the largest of the 32 to 448 =
      // 1.75 * 2^8 or less
      const uint32_t b = __float_as_uint(row_max(fmaxf(fabsf(h0), fabsf(h1))));
      const int ex = max((int)(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u), 0);
      const float inv = __uint_as_float((uint32_t)(254 - ex) << 23);
      const int codes = __builtin_amdgcn_cvt_pk_fp8_f32(h0 * inv, h1 * inv, 0, false);
      if (in) {
        uint8_t* p = a.out + row * a.out_row;
        *reinterpret_cast<uint16_t*>(p + col) = (uint16_t)codes;
        if (c == 0) p[a.I + quad] = (uint8_t)ex;
        const int end = a.I + a.I / 32;          // codes, scales, then zeros
        if (quad == a.I / 32 - 1 && end + c < a.out_row) p[end + c] = 0;
      }
    }
  }
#endif
}

// Few rows: the weights' stream.  A workgroup takes a quad of one row tile; its four waves take the steps
// along k in turn, each loading its blocks straight into the registers that the matrix instructions
// take, D steps ahead, and their sums meet in LDS.
template <int OP, bool Q8, int NQ>
__global__ __launch_bounds__(256) void stream_kernel(const W4Args a) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int BQ = 16 * NQ, D = 3;
  __shared__ float part[4][16 * NQ][64];
  const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  if (uni(a.plan[a.s.o_hdr + H_STATUS]) != 0) return;
  const int K = OP == W4_FWD1 ? a.H : a.I;
  const int nk = steps_of(K);
  const int nt = OP == W4_FWD1 ? (a.I + kQuadI - 1) / kQuadI : (a.H + kQuadH - 1) / kQuadH;
  RowTiles<BQ> queue(a.plan, a.s, lane, nt, a.tiles_bound);
  queue.look_up(0, true);
  for (int round = 0;; ++round) {
    const auto t = queue.tile(round);
    if (!t.rows) break;
    const uint8_t* W = t.w < a.s.E ? a.home + t.w * a.pitch : a.slot + (t.w - a.s.E) * a.pitch;
    if (OP == W4_FWD2) W += gate_up_bytes(a.H, a.I);
    const auto wr = __builtin_amdgcn_make_buffer_rsrc((void*)(W + (int64_t)t.tn * nk * kBlock), 0, nk * kBlock, kBufferFlags);
    const auto xr = __builtin_amdgcn_make_buffer_rsrc((void*)(a.in + t.row * a.in_row), 0, 0x7fffffff, kBufferFlags);
    u32x4 P[D][4], X[D][NQ][Q8 ? 2 : 4];
    uint32_t S[D], XS[D][NQ];
    auto load = [&](int d, int j) {               // past the end everything reads as zero
#pragma unroll
      for (int f = 0; f < 4; ++f)
        P[d][f] = __builtin_amdgcn_raw_buffer_load_b128(wr, j * kBlock + f * 1024 + lane * 16, 0, 0);
      S[d] = __builtin_amdgcn_raw_buffer_load_b32(wr, j * kBlock + 4096 + lane * 4, 0, 0);
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        const int r = q * 16 + c;
        const uint32_t row = r < t.rows ? (uint32_t)(r * a.in_row) : kOob;
        if constexpr (Q8) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int k = j * kStepK + i * 64 + g * 16;
            X[d][q][i] = __builtin_amdgcn_raw_buffer_load_b128(xr, k < K ? row + k : kOob, 0, 0);
          }
          const int b = j * 4 + g;
          XS[d][q] = __builtin_amdgcn_raw_buffer_load_b8(xr, b * 32 < K ? row + K + b : kOob, 0, 0);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int k = j * kStepK + g * 32 + i * 8;
            X[d][q][i] = __builtin_amdgcn_raw_buffer_load_b128(xr, k < K ? row + k * 2 : kOob, 0, 0);
          }
        }
      }
    };
    f32x4 acc[4][NQ];
    clear(acc);
#pragma unroll
    for (int d = 0; d < D; ++d) load(d, wave + 4 * d);
    for (int j0 = wave; j0 < nk; j0 += 4 * D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          if constexpr (Q8) {
            const i32x4 pv = __builtin_bit_cast(i32x4, P[d][f]);
            const i32x8 pw = __builtin_shufflevector(pv, pv, 0, 1, 2, 3, -1, -1, -1, -1);
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
              const i32x8 x = __builtin_shufflevector(__builtin_bit_cast(i32x4, X[d][q][0]),
                                                      __builtin_bit_cast(i32x4, X[d][q][1]), 0, 1, 2, 3, 4, 5, 6, 7);
              // the strip's byte of S
              if (f == 0) acc[f][q] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, pw, acc[f][q], 0, 4, 0, XS[d][q], 0, S[d]);
              if (f == 1) acc[f][q] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, pw, acc[f][q], 0, 4, 0, XS[d][q], 1, S[d]);
              if (f == 2) acc[f][q] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, pw, acc[f][q], 0, 4, 0, XS[d][q], 2, S[d]);
              if (f == 3) acc[f][q] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, pw, acc[f][q], 0, 4, 0, XS[d][q], 3, S[d]);
            }
          } else {
            const float scale = strip_scale(S[d], f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const bf16x8 p = __builtin_bit_cast(bf16x8, expand(P[d][f][i], scale));
#pragma unroll
              for (int q = 0; q < NQ; ++q)
                acc[f][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, X[d][q][i]), p, acc[f][q], 0, 0, 0);
            }
          }
        }
        load(d, j0 + 4 * (d + D));
      }
    }
    // wave w finishes the rows whose results are the lanes' elements w
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[wave][(q * 4 + i) * 4 + f][lane] = acc[f][q][i];
    __syncthreads();
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      f32x4 d{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < 4; ++w)
#pragma unroll
        for (int f = 0; f < 4; ++f) d[f] += part[w][(q * 4 + wave) * 4 + f][lane];
      const int r = q * 16 + g * 4 + wave;
      put<OP, Q8>(a, d, t.row + r, r < t.rows, t.tn, c);
    }
    __syncthreads();
  }
#endif
}

template <int OP, bool Q8>
hipError_t launch(W4Args a, hipStream_t st) {
  constexpr int NQ = 1, BQ = 16 * NQ;
  const int64_t segs = std::min<int64_t>(a.s.E + a.s.P_max, a.s.A);
  const int64_t mt = a.s.A / BQ + segs;
  const int nt = OP == W4_FWD1 ? (a.I + kQuadI - 1) / kQuadI : (a.H + kQuadH - 1) / kQuadH;
  a.tiles_bound = (int)mt;
  const int grid = (int)std::min<int64_t>((mt * nt + 7) / 8 * 8, 8 * kCus);
  hipLaunchKernelGGL((stream_kernel<OP, Q8, NQ>), dim3(grid), dim3(256), 0, st, a);
  return hipGetLastError();
}

int check_w4(int H, int I) {
  if (H <= 0 || H % 8 != 0 || I <= 0 || I % 8 != 0) return MOONEP_EINVAL;
  if (H > MOONEP_MAX_FFN || I > MOONEP_MAX_FFN) return MOONEP_ELIMIT;
  return MOONEP_OK;
}

int check_packing(const uint16_t* w, int64_t W_el, int64_t n, int H, int I, const uint8_t* w4, int64_t pitch) {
  const int rc = check_w4(H, I);
  if (rc != MOONEP_OK) return rc;
  if (n < 0 || W_el < 3ll * I * H || W_el % 8 != 0 || pitch < slab_bytes(H, I) || pitch % 16 != 0) return MOONEP_EINVAL;
  if (n > INT32_MAX) return MOONEP_ELIMIT;
  if (n == 0) return MOONEP_OK;
  if (!w || !w4) return MOONEP_EINVAL;
  if (!aligned(w, 16) || !aligned(w4, 16)) return MOONEP_EALIGN;
  if (overlap(slabs(w, n, W_el, 3ll * I * H, 2), slabs(w4, n, pitch, slab_bytes(H, I), 1))) return MOONEP_EINVAL;
  return MOONEP_OK;
}

// Workgroups of four waves, a block to each.
unsigned pack_grid(int64_t blocks) { return (unsigned)std::min<int64_t>((blocks + 3) / 4, 1 << 23); }

template <bool Q8>
int ffn_w4(const moonep_plan_desc* plan, const uint8_t* in, int64_t in_row, int H, int I, int act, const uint8_t* home,
           const uint8_t* slot, int64_t pitch, uint16_t* gu, uint8_t* h, int64_t h_row, uint16_t* y, hipStream_t st) {
  if (!in || !home || !h || !y || (plan->sz.slots > 0 && !slot)) return MOONEP_EINVAL;
  const int64_t bytes = slab_bytes(H, I), rows = plan->sz.recv_rows;
  if (pitch < bytes || pitch % 16 != 0 || (act != MOONEP_ACT_SILU && act != MOONEP_ACT_GELU)) return MOONEP_EINVAL;
  // tiles are counted in 32 bits, for the smallest tile
  const int64_t mt = plan->sz.A / 16 + plan->sz.E + plan->sz.P_max;
  if (mt * std::max((I + kQuadI - 1) / kQuadI, (H + kQuadH - 1) / kQuadH) > INT32_MAX) return MOONEP_ELIMIT;
  if (!aligned(in, 16) || !aligned(home, 16) || !aligned(slot, 16) || !aligned(gu, 16) || !aligned(h, 16) || !aligned(y, 16))
    return MOONEP_EALIGN;
  // other workgroups still read what an output that overlapped an input would change
  const Span pl = plan_span(plan), x = span(in, rows, in_row), hw = slabs(home, plan->sz.E, pitch, bytes, 1),
             sw = slabs(slot, (int64_t)plan->sz.R * plan->sz.slots, pitch, bytes, 1);
  const Span go = rows_span(plan, gu, 2 * I), ho = span(h, rows, h_row), yo = rows_span(plan, y, H);
  if (overlap(go, {pl, x, hw, sw, ho, yo}) || overlap(ho, {pl, x, hw, sw, yo}) || overlap(yo, {pl, x, hw, sw}))
    return MOONEP_EINVAL;
  W4Args a{};
  a.plan = static_cast<const int32_t*>(plan->dev);
  a.s = plan->sz;
  a.H = H; a.I = I; a.act = act;
  a.home = home; a.slot = slot; a.pitch = pitch;
  a.in = in; a.in_row = in_row; a.out = h; a.out_row = h_row; a.gu = gu;
  (void)hipGetLastError();
  if (launch<W4_FWD1, Q8>(a, st) != hipSuccess) return MOONEP_EHIP;
  a.in = h; a.in_row = h_row; a.out = reinterpret_cast<uint8_t*>(y); a.out_row = 2ll * H; a.gu = nullptr;
  return launch<W4_FWD2, Q8>(a, st) == hipSuccess ? MOONEP_OK : MOONEP_EHIP;
}

}  // namespace
}  // namespace moonep

using namespace moonep;

extern "C" {

int64_t moonep_w4_slab_bytes(int H, int I) {
  const int rc = check_w4(H, I);
  return rc != MOONEP_OK ? rc : slab_bytes(H, I);
}

int moonep_w4_pack(const uint16_t* w, int64_t W_el, int64_t n, int H, int I, uint8_t* w4, int64_t W_bytes,
                   hipStream_t stream) {
  const int rc = check_packing(w, W_el, n, H, I, w4, W_bytes);
  if (rc != MOONEP_OK || n == 0) return rc;
  const int64_t per = slab_bytes(H, I) / kBlock;
  (void)hipGetLastError();
  hipLaunchKernelGGL(pack_kernel, dim3(pack_grid(n * per)), dim3(256), 0, stream, w, W_el, n, H, I, w4, W_bytes, per);
  return hipGetLastError() == hipSuccess ? MOONEP_OK : MOONEP_EHIP;
}

int moonep_w4_unpack(const uint8_t* w4, int64_t W_bytes, int64_t n, int H, int I, uint16_t* w, int64_t W_el,
                     hipStream_t stream) {
  const int rc = check_packing(w, W_el, n, H, I, w4, W_bytes);
  if (rc != MOONEP_OK || n == 0) return rc;
  const int64_t per = slab_bytes(H, I) / kBlock;
  (void)hipGetLastError();
  hipLaunchKernelGGL(unpack_w4_kernel, dim3(pack_grid(n * per)), dim3(256), 0, stream, w4, W_bytes, n, H, I, w, W_el, per);
  return hipGetLastError() == hipSuccess ? MOONEP_OK : MOONEP_EHIP;
}

int moonep_expert_ffn_w4(const moonep_plan_desc* plan, const uint16_t* recv, int H, int I, int act,
                         const uint8_t* home_w4, const uint8_t* slot_w4, int64_t W_bytes, uint16_t* gu, uint16_t* h,
                         uint16_t* y, hipStream_t stream) {
  int rc = check_desc(plan);
  if (rc == MOONEP_OK) rc = check_w4(H, I);
  if (rc != MOONEP_OK) return rc;
  return ffn_w4<false>(plan, reinterpret_cast<const uint8_t*>(recv), 2ll * H, H, I, act, home_w4, slot_w4, W_bytes, gu,
                       reinterpret_cast<uint8_t*>(h), 2ll * I, y, stream);
}

int moonep_expert_ffn_w4q8(const moonep_plan_desc* plan, const uint8_t* rows, int H, int I, int act,
                           const uint8_t* home_w4, const uint8_t* slot_w4, int64_t W_bytes, uint8_t* h, uint16_t* y,
                           hipStream_t stream) {
  int rc = check_desc(plan);
  if (rc == MOONEP_OK) rc = check_w4(H, I);
  if (rc != MOONEP_OK) return rc;
  const int64_t rb = moonep_q8_row_bytes(H), hb = moonep_q8_row_bytes(I);
  if (rb < 0 || hb < 0) return (int)std::min(rb, hb);
  return ffn_w4<true>(plan, rows, rb, H, I, act, home_w4, slot_w4, W_bytes, nullptr, h, hb, y, stream);
}

}  // extern "C"
