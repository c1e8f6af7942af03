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

// A wave a block; in memory's order of the matrix, lane (i, j) of load u has chunk j (8 elements) of row 4 u + i of a
// strip, so that 16 lanes read 256 bytes that follow each other; the codes get into the slab's order in LDS.  Streams: 64
// bytes in for 17 out, and back.
// Measured on MI355X, 16 experts of H 7168, I 2048 (1.4 GB of bf16): with the lanes in the slab's order, whose 16-byte
// accesses are 64 bytes apart, 375 us and, back, 561; in memory's order 361 and 325, and, where more than the last-level
// cache holds passes it by, together 651 for 686 (0.2 GB: 39, and 56 if that passed it by).
template <bool NT>
__global__ __launch_bounds__(256) void pack_kernel(const uint16_t* w, int64_t W_el, int64_t n, int H, int I,
                                                   uint8_t* out, int64_t pitch, int64_t per) {
#ifdef __HIP_DEVICE_COMPILE__   // gfx950 builtins: the host pass needs the kernel's name only
  __shared__ __align__(16) uint8_t block[4][kBlock];
  const int lane = threadIdx.x & 63, j = lane & 15, sub = lane >> 4;
  uint8_t* const mine = block[threadIdx.x >> 6];
  const int64_t all = n * per;
  for (int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); i < all; i += (int64_t)gridDim.x * 4) {
    const int64_t e = i / per, b = i - e * per;
    const BlockAt at(b, H, I);
    const int k = at.k0 + 8 * j;
    u32x4 v[4][4];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t row = at.row(t, 4 * u + sub);
        v[t][u] = row >= 0 && k < at.k ? load<NT>(reinterpret_cast<const u32x4*>(w + e * W_el + at.at + row * at.k + k))
                                       : u32x4{0, 0, 0, 0};
      }
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        uint32_t top = 0;                        // bf16 magnitudes compare as their bits do
#pragma unroll
        for (int d = 0; d < 4; ++d) top = max(top, max(v[t][u][d] & 0x7FFFu, v[t][u][d] >> 16 & 0x7FFFu));
        top = max(top, __float_as_uint(quad_move<0xB1>(__uint_as_float(top))));      // four lanes are a group
        top = max(top, __float_as_uint(quad_move<0x4E>(__uint_as_float(top))));
        // largest = m * 2^E, 1 <= m < 2, and 6 = 1.5 * 2^2; infinities and NaN make the group NaN
        const int ex = top >= 0x7F80u ? 255 : max((int)(top >> 7) - 2 + ((top & 0x7Fu) > 0x40u), 1);
        const float scale = __uint_as_float((uint32_t)ex << 23);
        uint32_t d = 0;
        d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, lo(v[t][u][0]), hi(v[t][u][0]), scale, 0);
        d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, lo(v[t][u][1]), hi(v[t][u][1]), scale, 1);
        d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, lo(v[t][u][2]), hi(v[t][u][2]), scale, 2);
        d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, lo(v[t][u][3]), hi(v[t][u][3]), scale, 3);
        const int to = (j >> 2) * 16 + 4 * u + sub;                  // the lane of the slab's order
        *reinterpret_cast<uint32_t*>(mine + t * 1024 + to * 16 + (j & 3) * 4) = d;
        if ((j & 3) == 0) mine[4096 + to * 4 + t] = (uint8_t)ex;
      }
    wave_sync();
    uint8_t* const to = out + e * pitch + b * kBlock;
#pragma unroll
    for (int t = 0; t < 4; ++t)
      store<NT>(*reinterpret_cast<const u32x4*>(mine + t * 1024 + lane * 16), reinterpret_cast<u32x4*>(to + t * 1024 + lane * 16));
    *reinterpret_cast<uint32_t*>(to + 4096 + lane * 4) = *reinterpret_cast<const uint32_t*>(mine + 4096 + lane * 4);
    wave_sync();
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
// Strip t's scale of a word of four, as a float.
__device__ __forceinline__ float strip_scale(uint32_t scales, int t) {
  return __uint_as_float(t < 3 ? scales << (23 - 8 * t) & 0x7F800000u : scales >> 1 & 0x7F800000u);
}

// pack_kernel's inverse, exact.  A word of codes comes to the lane that writes its eight elements.
template <bool NT>
__global__ __launch_bounds__(256) void unpack_w4_kernel(const uint8_t* in, int64_t pitch, int64_t n, int H, int I,
                                                        uint16_t* w, int64_t W_el, int64_t per) {
  const int lane = threadIdx.x & 63, j = lane & 15, sub = lane >> 4;
  const int64_t all = n * per;
  for (int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); i < all; i += (int64_t)gridDim.x * 4) {
    const int64_t e = i / per, b = i - e * per;
    const BlockAt at(b, H, I);
    const int k = at.k0 + 8 * j;
    const uint8_t* from = in + e * pitch + b * kBlock;
    uint32_t codes[4][4], scales[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int l = (j >> 2) * 16 + 4 * u + sub;                     // the lane of the slab's order
      scales[u] = *reinterpret_cast<const uint32_t*>(from + 4096 + l * 4);
#pragma unroll
      for (int t = 0; t < 4; ++t) codes[t][u] = *reinterpret_cast<const uint32_t*>(from + t * 1024 + l * 16 + (j & 3) * 4);
    }
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t row = at.row(t, 4 * u + sub);
        if (row >= 0 && k < at.k)
          store<NT>(expand(codes[t][u], strip_scale(scales[u], t)), reinterpret_cast<u32x4*>(w + e * W_el + at.at + row * at.k + k));
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
// lane's place among the quad's columns; `out` and `gu` begin at the tile's first row, `r` is the row of the
// tile, and what is not `in` goes nowhere.  No branches: every store goes out (see Pipe).
template <int OP, bool Q8>
__device__ __forceinline__ void put(const W4Args& a, const Window& out, const Window& gu, const f32x4& d, int r, bool in,
                                    int quad, int c) {
#ifdef __HIP_DEVICE_COMPILE__
  const uint32_t at = r * (int)a.out_row;
  if constexpr (OP == W4_FWD2) {
    const int col = quad * kQuadH + 4 * c;
    out.store(u32x2{bf2(d[0], d[1]), bf2(d[2], d[3])}, in && col < a.H ? at + col * 2 : kOob);
  } else {
    // h in bf16 is rounded once, to 2^-8 of it: the second product's instructions take bf16
    const int col = quad * kQuadI + 2 * c;
    float slope;
    const float h0 = act_of(d[0], a.act, &slope) * d[2], h1 = act_of(d[1], a.act, &slope) * d[3];
    if constexpr (!Q8) {
      in = in && col < a.I;
      out.store(bf2(h0, h1), in ? at + col * 2 : kOob);
      if (a.gu) {
        const uint32_t to = (r * 2 * a.I + col) * 2;
        gu.store(bf2(d[0], d[1]), in ? to : kOob);
        gu.store(bf2(d[2], d[3]), in ? to + a.I * 2 : kOob);
      }
    } else {
      // the rule of the 8-bit norm: the smallest power of two that brings the largest of the 32 to 448 =
      // 1.75 * 2^8 or less.  h is rounded here once, to half a step of 2^-4 of it: half the bytes of bf16, and the second
      // product's instructions take no wider rows
      const uint32_t b = __float_as_uint(row_max(fmaxf(fabsf(h0), fabsf(h1))));
      const int ex = max((int)(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u), 0);
      const float inv = __uint_as_float((uint32_t)(254 - ex) << 23);
      const int codes = __builtin_amdgcn_cvt_pk_fp8_f32(h0 * inv, h1 * inv, 0, false);
      in = in && col < a.I;
      __builtin_amdgcn_raw_buffer_store_b16((uint16_t)codes, out.rs, in ? at + col : kOob, 0, 0);
      __builtin_amdgcn_raw_buffer_store_b8((uint8_t)ex, out.rs, in && c == 0 ? at + a.I + quad : kOob, 0, 0);
      const int end = a.I + a.I / 32;          // codes, scales, then zeros
      if (quad == a.I / 32 - 1 && end < a.out_row)
        __builtin_amdgcn_raw_buffer_store_b8(0, out.rs, in && end + c < a.out_row ? at + end + c : kOob, 0, 0);
    }
  }
#endif
}

// A tile of BP weight rows by BQ buffer rows, by WP x WQ waves: wave (p, q) has quad p of the weights and every WQ-th fragment
// of 16 rows from q on, so that a tile with few rows leaves work to all.  LDS holds NP steps of weights and NQ of rows.
template <int WP_, int BQ_, int WQ_, int NP_, int NQ_, int PER_CU_>
struct W4Geometry {
  static constexpr int WP = WP_, WQ = WQ_, NW = WP * WQ, BP = 64 * WP, BQ = BQ_, QF = BQ / WQ / 16, NP = NP_, NQ = NQ_;
  static constexpr int PER_CU = PER_CU_;         // workgroups, in LDS and in registers
};

// The products of one tile after another, without a break between them.  LDS holds NP steps of 128 k of weights, the
// blocks of the tile's quads as they are in memory (a wave's load fills 1024 bytes in the order in
// which its lanes read them back), and NQ steps of the buffer rows, in lines of 128 bytes, 16-byte chunk c of row r
// in the place of chunk c ^ (r & 7), so that the 16 lanes that read at once hit different banks.  A step's 256 bytes
// of a bf16 row are two lines: line L has, as chunks 4 j + g, k = 32 g + 16 L + 8 j ... + 7, since a
// matrix instruction's lanes take neighbours in g.
//
// The first half of the waves loads the weights, the other the rows: loads are waited for in their order, so a
// wave that loaded both could have no more weights on their way than rows.
//
// A step is cut into parts; in each, the operands of a later part are read from LDS into registers among its matrix
// instructions.  When all of a step has been read, every wave waits for the next step's loads and for the others, and
// starts the loads of the step NP (or NQ) further on over it.  One barrier a step.
//
// What bounds it, measured on MI355X (us of a gate and up launch with loads or matrix instructions left out, sums wrong):
//   32 experts of H 7168, I 2048, 1024 8-bit rows each, 256 x 256 tiles: 1023 (1.9 PFLOP/s, of 2.7 that a large 8-bit library
//     product reaches); 767 without matrix instructions, 790 without loads, 800 without those of rows, 931 without those of
//     weights: both sides take three quarters of the time and hide behind each other for half of it
//   64 experts, 64 rows each, both launches 389: 353 without loads of rows, 302 without those of weights, and no less
//     without matrix instructions: a step's latencies, which two waves a SIMD do not hide
//   64 experts, a row to most of them, both launches 190: the weights' stream, 0.98 GB at 5.2 TB/s; 182 without scales, which
//     are 6% of its bytes
template <bool Q8, class G>
struct W4Pipe {
  static constexpr int QF = G::QF, NW = G::NW, BQ = G::BQ, WP = G::WP, WQ = G::WQ, NP = G::NP, NQ = G::NQ;
  static constexpr int kLines = Q8 ? 1 : 2;                          // of 128 bytes of a row
  static constexpr int kHalf = NW / 2;                               // waves that load one side
  static constexpr int kP = WP * kBlock, kQ = kLines * BQ * 128, kQ0 = NP * kP;
  // the scales of rows in 8 bits: 16 bytes of each for four steps, NQ times four steps of a tile, or what there is
  static constexpr int kSW = Q8 ? (BQ + 63) / 64 : 0, kS = kSW * 1024, kS0 = kQ0 + NQ * kQ, kLds = kS0 + NQ * kS;
  static constexpr int kCP = WP * 4 / kHalf, kLP = kCP + 1;          // loads of a step: codes, and the first wave's scales
  // not counting the scales of rows: these are started before the others of a step, and so are waited for too early, if
  // at all
  static constexpr int kCQ = kQ / 1024 / kHalf, kLQ = kCQ;
  static_assert(kHalf >= 1 && kCP * kHalf == WP * 4 && WP <= 4 && kCQ * kHalf * 1024 == kQ && kSW <= kHalf &&
                NP >= 2 && NQ >= 2 && G::PER_CU * kLds <= 160 * 1024 && (NP - 1) * kLP < 48 && (NQ - 1) * kLQ < 48);
  static constexpr int kSteps = NP > NQ ? NP : NQ;                   // loads are that far ahead
  uint32_t lds;                   // LDS
  int wave, lane;
  bool rows;                      // this wave loads rows (uniform)
  int lane_p, lane_ps;            // this lane's first LDS byte of a fragment of weights, of their scales,
  int lane_q, lane_s;             // of a fragment of rows, of a row's scale
  int cp, cq, cs;                 // the current step's places in LDS
  int scaling;                    // where the next four steps' scales are loaded to
  uint32_t voff, voff_s;          // this lane's first load and its scale's
  uint32_t stride;                // bytes from a quad to the next, or of kHalf * 8 rows (uniform)
  const char *at, *at_s;          // the next step to load
  int range;                      // bytes from there to the tile's end: what is past it reads as zero
  int left, todo;                 // bytes of a row left from there, and steps of this tile
  int loading;                    // its place in LDS
  int first;                      // the byte of a row's step that this lane loads first

  __device__ __forceinline__ W4Pipe(char* smem, int wave, int lane)
      : lds((uint32_t)(uintptr_t)(LDS char*)smem), wave(wave), lane(lane), rows(wave >= kHalf), cp(0), cq(kQ0) {
    const int base = (int)lds, c = lane & 15, g = lane >> 4;
    loading = rows ? kQ0 : 0;
    const int chunk = (lane & 7) ^ (lane >> 3);
    first = Q8 ? chunk * 16 : (chunk & 3) * 64 + (chunk >> 2) * 16;
    lane_p = base + wave % WP * 4096 + lane * 16;
    lane_ps = base + WP * 4096 + wave % WP * 256 + lane * 4;
    const int row = wave / WP * 16 + c;
    lane_q = base + row * 128 + ((g ^ (row & 7)) << 4);
    lane_s = base + row * 16 + g;
    cs = scaling = kS0;
  }

  // One side of a tile: where it begins, and its bytes (0: there is none).
  struct Side {
    const char* at;
    int range;
  };
  Side ahead;                     // of the tile after the one that is loaded
  int kbytes, steps;              // of every tile: bytes of a row that are codes or elements, and steps

  // What all tiles have alike: `nk` blocks to a quad, rows of `row_bytes`.
  __device__ __forceinline__ void shape(int nk, int row_bytes, int kbytes_, int steps_) {
    kbytes = kbytes_;
    steps = steps_;
    if (!rows) {
      stride = nk * kBlock;
      voff = (wave >> 2) * stride + (wave & 3) * 1024 + lane * 16;
      voff_s = (lane >> 4) * stride + 4096 + (lane & 15) * 16;
    } else {
      stride = kHalf * 8 * row_bytes;
      const int r = (wave - kHalf) * 8 + (lane >> 3);
      voff = r * row_bytes + first;
      voff_s = (uint32_t)(((wave - kHalf) * 64 + lane) * row_bytes);
    }
  }
  // `w`: a tile's first quad's blocks, of `nquads` there are; `x`: its first row, of `n`.
  __device__ __forceinline__ Side side(const uint8_t* w, int nquads, const uint8_t* x, int n, int row_bytes) const {
    if (!rows) return Side{reinterpret_cast<const char*>(w), (nquads < WP ? nquads : WP) * (int)stride};
    return Side{reinterpret_cast<const char*>(x), n * row_bytes};
  }
  __device__ __forceinline__ void start(const Side& t) {
    at = t.at;
    at_s = at + kbytes;
    range = t.range;
    left = kbytes;
    todo = steps;
  }

  // The loads of the next step.  Past the end everything is out of range, and zeros are loaded.
  __device__ __forceinline__ void load() {
    if (todo == 0 && ahead.range) start(ahead);
    const uint64_t p = reinterpret_cast<uint64_t>(at);
    const i32x4 rs{(int)p, (int)(p >> 32) & 0xFFFF, left > 0 ? range : 0, kBufferFlags};
    if (!rows) {
      // chunk i * kHalf + wave of the step's, strip by strip; 16 lanes a quad's scales
      const uint32_t to = uni(lds + loading + wave * 1024);
      times<kCP>([&](auto i) {
        load_lds<i * kHalf * 1024>(rs, voff + (i * kHalf >> 2) * stride + (i * kHalf & 3) * 1024, to);
      });
      if (wave == 0 && (WP == 4 || lane < WP * 16)) load_lds<WP * 4096>(rs, voff_s, to);
      at += kBlock;
      range -= kBlock;
      loading = loading == (NP - 1) * kP ? 0 : loading + kP;
    } else {
      if constexpr (Q8) {
        const int step = steps - todo;
        if (step % 4 == 0) {
          if (wave - kHalf < kSW) {
            const uint64_t s = reinterpret_cast<uint64_t>(at_s);
            // to the end of the tile's last row
            const i32x4 r{(int)s, (int)(s >> 32) & 0xFFFF, left > 0 ? range - (int)(at_s - at) : 0, kBufferFlags};
            load_lds<0>(r, voff_s, uni(lds + scaling + (wave - kHalf) * 1024));
          }
          at_s += 16;
          scaling = scaling == kS0 + (NQ - 1) * kS ? kS0 : scaling + kS;
        }
      }
      const uint32_t to = uni(lds + loading + (wave - kHalf) * 1024);
      times<kCQ>([&](auto i) {                // eight rows of a line of 128 bytes
        constexpr int kLine = i * kHalf / (BQ / 8), kRow = i * kHalf % (BQ / 8) / kHalf;
        static_assert(BQ / 8 % kHalf == 0);
        constexpr int kSkip = kLine * (Q8 ? 128 : 32);
        const uint32_t v = voff + kRow * stride + kSkip;
        load_lds<i * kHalf * 1024>(rs, first + kSkip < left ? v : kOob, to);
      });
      at += kLines * 128;
      range -= kLines * 128;
      loading = loading == kQ0 + (NQ - 1) * kQ ? kQ0 : loading + kQ;
    }
    left -= kLines * 128;
    --todo;
  }
  // Waits until at most N - LESS steps of this wave's loads are on their way, and, where `younger` is set, the STORES
  // stores that went out after them.
  template <int LESS, int STORES>
  __device__ __forceinline__ void wait(bool younger) {
    asm volatile("" ::: "memory");
    auto until = [&](auto loads) {
      constexpr int kMore = loads + STORES;
      if (younger) __builtin_amdgcn_s_waitcnt(wait_vm_lds(kMore < 63 ? kMore : 63));
      else __builtin_amdgcn_s_waitcnt(wait_vm_lds(loads));
    };
    if (rows) until(std::integral_constant<int, (NQ - LESS) * kLQ>{});
    else if (wave == 0) until(std::integral_constant<int, (NP - LESS) * kLP>{});
    else until(std::integral_constant<int, (NP - LESS) * kCP>{});
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }

  __device__ __forceinline__ void begin() {
    for (int i = 0; i < (rows ? NQ : NP); ++i) load();
    wait<1, 0>(false);
  }

  struct Rows8 { i32x4 lo, hi; int scale; };
  __device__ __forceinline__ Rows8 rows8(int at, int scale, int q) const {
    const int x = lane_q + at, y = x ^ 64;
    return Rows8{*(const LDS i32x4*)(x + q * WQ * 2048), *(const LDS i32x4*)(y + q * WQ * 2048),
                 *(const LDS uint8_t*)(lane_s + scale + q * WQ * 256)};
  }
  __device__ __forceinline__ bf16x8 rows16(int at, int q, int i) const {
    return *(const LDS bf16x8*)(((lane_q + at) ^ (i & 1) << 6) + (i >> 1) * BQ * 128 + q * WQ * 2048);
  }
  __device__ __forceinline__ i32x4 codes(int at, int f) const { return *(const LDS i32x4*)(lane_p + at + f * 1024); }
  __device__ __forceinline__ uint32_t scales(int at) const { return *(const LDS uint32_t*)(lane_ps + at); }

  template <int F>
  static __device__ __forceinline__ void multiply8(f32x4& acc, const Rows8& x, const i32x4& p, uint32_t scales) {
    const i32x8 pw = __builtin_shufflevector(p, p, 0, 1, 2, 3, -1, -1, -1, -1);
    const i32x8 xw = __builtin_shufflevector(x.lo, x.hi, 0, 1, 2, 3, 4, 5, 6, 7);
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(xw, pw, acc, 0, 4, 0, x.scale, F, (int)scales);
  }

  // The next `nk` steps.  `live`: how many of the tile's rows there are from the wave's first on; where it has not ALL of its
  // fragments, the matrix instructions of the rest are left out.  `younger`: at least STORES stores went out since the last step.
  template <bool ALL, int STORES>
  __device__ __forceinline__ void run(int nk, int live, bool younger, f32x4 (&acc)[4][QF]) {
    // whether the wave has rows in fragment q; without any it takes part in the loads only
    auto there = [&](int q) { return ALL || q * WQ * 16 < live; };
    if constexpr (Q8) {
      constexpr int kRing = QF >= 4 ? 4 : 2, kRead = QF > 1 ? kRing / 2 : 1;        // fragments read ahead
      i32x4 p[4], pn[4];
      uint32_t ps = 0, psn = 0;
      Rows8 x[kRing];
      if (there(0)) {
        times<4>([&](auto f) { p[f] = codes(cp, f); });
        ps = scales(cp);
      }
      times<kRead>([&](auto q) {
        if (there(q)) x[q] = rows8(cq, cs, q);
      });
      for (int i = 0; i < nk; ++i) {
        const int np = cp == (NP - 1) * kP ? 0 : cp + kP, nq = cq == kQ0 + (NQ - 1) * kQ ? kQ0 : cq + kQ;
        const int four = cs - i % 4 * 4;         // these four steps' scales, then this tile's next, or another's first
        const int ns = i % 4 < 3 && i + 1 < nk ? cs + 4 : four == kS0 + (NQ - 1) * kS ? kS0 : four + kS;
        times<QF>([&](auto q) {
          if constexpr (q == QF - kRead) {
            wait<2, STORES>(younger && i == 0);
            load();
            if (there(0)) {
              times<4>([&](auto f) { pn[f] = codes(np, f); });
              psn = scales(np);
            }
          }
          // QF = 1: the one place is read anew after it has been multiplied
          if constexpr (QF > 1)
            if (there((q + kRead) % QF)) x[(q + kRead) % kRing] = rows8(q + kRead < QF ? cq : nq, q + kRead < QF ? cs : ns, (q + kRead) % QF);
          if (there(q))
            times<4>([&](auto f) { multiply8<f>(acc[f][q], x[q % kRing], p[f], ps); });
          if constexpr (QF == 1)
            if (there(0)) x[0] = rows8(nq, ns, 0);
          __builtin_amdgcn_sched_barrier(0);
        });
        times<4>([&](auto f) { p[f] = pn[f]; });
        ps = psn;
        cp = np;
        cq = nq;
        cs = ns;
      }
    } else {
      i32x4 p[4];
      uint32_t ps;
      bf16x8 x[2][QF], w[2][4];
      auto read = [&](int at) {
        times<4>([&](auto f) { p[f] = codes(at, f); });
        ps = scales(at);
      };
      auto widen = [&](auto k) {
        constexpr int kk = k;
        times<4>([&](auto f) { w[kk % 2][f] = __builtin_bit_cast(bf16x8, expand(p[f][kk], strip_scale(ps, f))); });
      };
      if (there(0)) {
        read(cp);
        widen(std::integral_constant<int, 0>{});
      }
      times<QF>([&](auto q) {
        if (there(q)) x[0][q] = rows16(cq, q, 0);
      });
      for (int i = 0; i < nk; ++i) {
        const int np = cp == (NP - 1) * kP ? 0 : cp + kP, nq = cq == kQ0 + (NQ - 1) * kQ ? kQ0 : cq + kQ;
        times<4>([&](auto k) {
          constexpr int kn = (k + 1) % 4;
          if constexpr (k == 3) {
            wait<2, STORES>(younger && i == 0);
            load();
            if (there(0)) read(np);
          }
          times<QF>([&](auto q) {
            if (there(q)) x[(k + 1) % 2][q] = rows16(k == 3 ? nq : cq, q, kn);
          });
          times<QF>([&](auto q) {
            if (there(q))
              times<4>([&](auto f) {
                acc[f][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[k % 2][q], w[k % 2][f], acc[f][q], 0, 0, 0);
              });
          });
          if (there(0)) widen(std::integral_constant<int, kn>{});
          __builtin_amdgcn_sched_barrier(0);
        });
        cp = np;
        cq = nq;
      }
    }
  }
};

template <int OP, bool Q8, class G>
__global__ __launch_bounds__(64 * G::NW, G::PER_CU * G::NW / 4 > 2 ? G::PER_CU * G::NW / 4 : 2) void tile_kernel(const W4Args a) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int BQ = G::BQ, WP = G::WP, QF = G::QF;
  constexpr int kQuads = G::BP / 64;
  using Tiles = W4Pipe<Q8, G>;
  __shared__ __align__(1024) char smem[Tiles::kLds];
  const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6);
  const int wp = wave % WP, wq = wave / WP;
  if (uni(a.plan[a.s.o_hdr + H_STATUS]) != 0) return;
  const int K = OP == W4_FWD1 ? a.H : a.I;
  const int steps = steps_of(K), nk = max(steps, Tiles::kSteps);      // loads are that far ahead, in one more tile only
  const int quads = OP == W4_FWD1 ? (a.I + kQuadI - 1) / kQuadI : (a.H + kQuadH - 1) / kQuadH;
  RowTiles<BQ> queue(a.plan, a.s, lane, (quads + kQuads - 1) / kQuads, a.tiles_bound);
  queue.look_up(0, true);
  Tiles pipe(smem, wave, lane);
  auto side = [&](const typename RowTiles<BQ>::Tile& t) {
    const uint8_t* W = t.w < a.s.E ? a.home + t.w * a.pitch : a.slot + (t.w - a.s.E) * a.pitch;
    if (OP == W4_FWD2) W += gate_up_bytes(a.H, a.I);
    const int q0 = t.tn * kQuads;
    return pipe.side(W + (int64_t)q0 * steps * kBlock, quads - q0, a.in + t.row * a.in_row, t.rows, (int)a.in_row);
  };
  auto cur = queue.tile(0), nxt = queue.tile(1);
  if (!cur.rows) return;
  pipe.shape(steps, (int)a.in_row, Q8 ? K : 2 * K, nk);
  pipe.start(side(cur));
  pipe.ahead = side(nxt);
  if (!nxt.rows) pipe.ahead.range = 0;
  pipe.begin();
  for (int round = 1;; ++round) {
    f32x4 acc[4][QF];
    clear(acc);
    const auto t = cur;
    const int quad = t.tn * kQuads + wp;
    const int live = quad < quads ? t.rows - wq * 16 : 0;
    constexpr int kStores = 4 * QF;
    if (live > (QF - 1) * G::WQ * 16) pipe.template run<true, kStores>(nk, live, round > 1, acc);
    else pipe.template run<false, kStores>(nk, live, round > 1, acc);
    // what the results' places are made of is worked out here, not kept during the products
    const int ln = here(lane);
    const Window out(a.out + t.row * a.out_row), gu(a.gu + (int64_t)t.row * 2 * a.I);
#pragma unroll
    for (int q = 0; q < QF; ++q) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = (q * G::WQ + wq) * 16 + (ln >> 4) * 4 + i;
        put<OP, Q8>(a, out, gu, f32x4{acc[0][q][i], acc[1][q][i], acc[2][q][i], acc[3][q][i]}, r,
                    r < t.rows && quad < quads, quad, ln & 15);
      }
      __builtin_amdgcn_sched_barrier(0);         // or all results are worked on at once, and spill
    }
    if (!nxt.rows) break;
    cur = nxt;
    nxt = queue.tile(round + 1);
    pipe.ahead = side(nxt);
    if (!nxt.rows) pipe.ahead.range = 0;
  }
  settled();                      // LDS is not given up while loads may still write to it
#endif
}

template <bool Q8>
struct W4Tiles {
  using Large = W4Geometry<4, 256, 2, 3, 3, 1>;                            // 8-bit rows only
  using Tall = W4Geometry<4, 128, 2, 3, 3, 1>;
  using Medium = std::conditional_t<Q8, W4Geometry<4, 64, 1, 2, 2, 3>, W4Geometry<4, 32, 1, 2, 2, 3>>;
  using Pair = W4Geometry<4, 64, 1, 2, 2, 2>;                              // bf16 rows only
  using Small = W4Geometry<2, 64, 2, 3, 3, 3>;                             // 8-bit rows only
  using Few = W4Geometry<2, 16, 1, 4, 2, Q8 ? 4 : 3>;
};
enum W4Tile { W4_LARGE, W4_TALL, W4_PAIR, W4_MEDIUM, W4_SMALL, W4_FEW };

template <int OP, bool Q8, class G>
hipError_t launch_tiles(W4Args a, hipStream_t st) {
  constexpr int kQuads = G::BP / 64;
  const int64_t mt = a.s.A / G::BQ + std::min<int64_t>(a.s.E + a.s.P_max, a.s.A);
  const int quads = OP == W4_FWD1 ? (a.I + kQuadI - 1) / kQuadI : (a.H + kQuadH - 1) / kQuadH;
  a.tiles_bound = (int)mt;
  const int grid = (int)std::min<int64_t>((mt * ((quads + kQuads - 1) / kQuads) + 7) / 8 * 8, G::PER_CU * kCus);
  hipLaunchKernelGGL((tile_kernel<OP, Q8, G>), dim3(grid), dim3(64 * G::NW), 0, st, a);
  return hipGetLastError();
}

// Which tile.  Where the weights' stream is everything, the smallest, of which the most are on their way; then the
// smallest that still is about one round over the CUs, as long as the few steps of a tile are no more than its start
// and its end, which other workgroups of the CU work beside; else the large ones, which read rows and weights
// the fewest times.  An expert's group and its replicas end inside a tile: half of one to each group.
// Measured on MI355X, us of each launch (Few, Medium, Pair, Tall; and with 8-bit rows Few, Small, Medium, Tall, Large; mean
// rows of an expert; R 8 for 64 experts, 4 for 16, 3 for 21):
//   64 experts, H 7168, I 2048, gate and up    1: 121, 126, 152, 154       140, 125, 128, 140, 167
//                                             16: 246, 259, 267, 298       231, 241, 256, 254, 305
//                                             64: 535, 365, 319, 427       430, 314, 287, 282, 369
//                                            128: 940, 647, 561, 581       691, 442, 398, 334, 434
//                                            256: 1723, 1126, 1028, 1014   1234, 749, 586, 654, 580
//                               down          16: 126, 123, 120, 141       126, 129, 123, 124, 140
//                                             64: 272, 169, 178, 206       204, 159, 150, 135, 166
//                                            256: 906, 555, 525, 489       627, 380, 317, 308, 318
//   64 experts, H 2048, I 1024, gate and up    1: 23, 30, 29, 38           27, 24, 32, 34, 48
//                                             32: 56, 35, 55, 68           39, 40, 40, 49, 71
//                                             64: 89, 54, 64, 85           61, 41, 39, 54, 81
//                                            256: 267, 151, 154, 166       194, 111, 95, 112, 111
//   16 experts, H 2048, I 1024, gate and up   32: 20, 22, 32, 28           17, 22, 23, 22, 30
//                                            128: 44, 30, 37, 37           34, 22, 29, 26, 38
//                                            256: 81, 53, 62, 63           54, 37, 31, 44, 42
//   21 experts, H 992, I 672,   gate and up   27: 14, 15, 20, 20           12, 14, 16, 16, 23
//                                            110: 27, 19, 22, 24           18, 16, 18, 19, 27
//   64 experts, H 2048, I 1408, gate and up  768: 1183, 736, 674, 647;   32 of H 7168, I 2048, 1024: 2320, 1359, 1063, 1067, 985
// The rule takes the best tile of these or one within 5%, but for 8-bit rows in the first product of 64 experts: with a row
// each it takes Few (140 for 125, 27 for 24), with 16 of H 7168 Tall (254 for 231), with 256 Tall (654 for 580; of H 2048 112 for
// 95).  Nothing was measured between 16 and 56 steps, where its limit of 32 lies.
template <int OP, bool Q8>
W4Tile w4_tile(const moonep_sizes& s, int H, int I) {
  const int quads = OP == W4_FWD1 ? (I + kQuadI - 1) / kQuadI : (H + kQuadH - 1) / kQuadH;
  const int steps = steps_of(OP == W4_FWD1 ? H : I);
  const double groups = (double)std::min<int64_t>(s.E + s.R - 1, s.A), mean = (double)s.A / std::min<int64_t>(s.E, s.A);
  auto tiles = [&](int bq, int wp) { return std::max(groups, (double)s.A / bq + groups / 2) * ((quads + wp - 1) / wp); };
  const bool few_steps = steps <= 32;
  if constexpr (Q8) {
    if (mean <= 12 || tiles(16, 2) <= 4 * kCus) return W4_FEW;
    if (few_steps && tiles(64, 2) <= 3 * kCus) return W4_SMALL;
    if (few_steps && tiles(64, 4) <= 3.3 * kCus) return W4_MEDIUM;
    return tiles(256, 4) >= 8 * kCus ? W4_LARGE : W4_TALL;
  } else {
    if (mean <= 20 || tiles(16, 2) <= 3 * kCus) return W4_FEW;
    if (!few_steps && mean >= 48) return mean < 160 ? W4_PAIR : W4_TALL;
    return tiles(128, 4) >= 10 * kCus ? W4_TALL : W4_MEDIUM;
  }
}

template <int OP, bool Q8>
hipError_t launch(const W4Args& a, hipStream_t st) {
  using T = W4Tiles<Q8>;
  const W4Tile t = w4_tile<OP, Q8>(a.s, a.H, a.I);
  if constexpr (Q8) {
    if (t == W4_LARGE) return launch_tiles<OP, Q8, typename T::Large>(a, st);
    if (t == W4_SMALL) return launch_tiles<OP, Q8, typename T::Small>(a, st);
  } else {
    if (t == W4_PAIR) return launch_tiles<OP, Q8, typename T::Pair>(a, st);
  }
  switch (t) {
    case W4_TALL: return launch_tiles<OP, Q8, typename T::Tall>(a, st);
    case W4_MEDIUM: return launch_tiles<OP, Q8, typename T::Medium>(a, st);
    default: return launch_tiles<OP, Q8, typename T::Few>(a, st);
  }
}

// Weight rows of a tile, half of them gate and half up in the first product, and buffer rows.
template <bool Q8, class G>
void tile_size(int32_t tile[2]) {
  tile[0] = G::BP;
  tile[1] = G::BQ;
}
template <int OP, bool Q8>
void tile_size(const moonep_sizes& s, int H, int I, int32_t tile[2]) {
  using T = W4Tiles<Q8>;
  switch (w4_tile<OP, Q8>(s, H, I)) {
    case W4_LARGE: return tile_size<Q8, typename T::Large>(tile);
    case W4_TALL: return tile_size<Q8, typename T::Tall>(tile);
    case W4_PAIR: return tile_size<Q8, typename T::Pair>(tile);
    case W4_MEDIUM: return tile_size<Q8, typename T::Medium>(tile);
    case W4_SMALL: return tile_size<Q8, typename T::Small>(tile);
    default: return tile_size<Q8, typename T::Few>(tile);
  }
}

int check_w4(int H, int I) {
  if (H <= 0 || H % 8 != 0 || I <= 0 || I % 8 != 0) return MOONEP_EINVAL;
  if (H > MOONEP_MAX_FFN || I > MOONEP_MAX_FFN) return MOONEP_ELIMIT;
  return MOONEP_OK;
}

// Tiles are counted in 32 bits, for the smallest tile.
int check_w4_tiles(const moonep_plan_desc* plan, int H, int I) {
  const int64_t mt = plan->sz.A / 16 + plan->sz.E + plan->sz.P_max;
  return mt * std::max((I + kQuadI - 1) / kQuadI, (H + kQuadH - 1) / kQuadH) > INT32_MAX ? MOONEP_ELIMIT : MOONEP_OK;
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
bool passes_cache(int64_t n, int H, int I) { return n > (int64_t)kLastLevelCacheBytes / (6ll * I * H); }

template <bool Q8>
int ffn_w4(const moonep_plan_desc* plan, const uint8_t* in, int64_t in_row, int H, int I, int act, const uint8_t* home,
           const uint8_t* slot, int64_t pitch, uint16_t* gu, uint8_t* h, int64_t h_row, uint16_t* y, hipStream_t st) {
  if (!in || !home || !h || !y || (plan->sz.slots > 0 && !slot)) return MOONEP_EINVAL;
  const int64_t bytes = slab_bytes(H, I), rows = plan->sz.recv_rows;
  if (pitch < bytes || pitch % 16 != 0 || (act != MOONEP_ACT_SILU && act != MOONEP_ACT_GELU)) return MOONEP_EINVAL;
  const int rc = check_w4_tiles(plan, H, I);
  if (rc != MOONEP_OK) return rc;
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

int moonep_expert_tile_w4(const moonep_plan_desc* plan, int H, int I, int rows_q8, int product, int32_t tile[2]) {
  int rc = check_desc(plan);
  if (rc == MOONEP_OK) rc = check_w4(H, I);
  if (rc == MOONEP_OK) rc = check_w4_tiles(plan, H, I);
  if (rc != MOONEP_OK) return rc;
  if (!tile || (rows_q8 != 0 && rows_q8 != 1) || (product != MOONEP_PRODUCT_GATE_UP && product != MOONEP_PRODUCT_DOWN) ||
      (rows_q8 && (H % 32 != 0 || I % 32 != 0)))
    return MOONEP_EINVAL;
  if (rows_q8) product == MOONEP_PRODUCT_DOWN ? tile_size<W4_FWD2, true>(plan->sz, H, I, tile) : tile_size<W4_FWD1, true>(plan->sz, H, I, tile);
  else product == MOONEP_PRODUCT_DOWN ? tile_size<W4_FWD2, false>(plan->sz, H, I, tile) : tile_size<W4_FWD1, false>(plan->sz, H, I, tile);
  return MOONEP_OK;
}

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
  const bool nt = passes_cache(n, H, I);
  hipLaunchKernelGGL((nt ? pack_kernel<true> : pack_kernel<false>), dim3(pack_grid(n * per)), dim3(256), 0, stream, w, W_el, n, H, I, w4,
                     W_bytes, per);
  return hipGetLastError() == hipSuccess ? MOONEP_OK : MOONEP_EHIP;
}

int moonep_w4_unpack(const uint8_t* w4, int64_t W_bytes, int64_t n, int H, int I, uint16_t* w, int64_t W_el,
                     hipStream_t stream) {
  const int rc = check_packing(w, W_el, n, H, I, w4, W_bytes);
  if (rc != MOONEP_OK || n == 0) return rc;
  const int64_t per = slab_bytes(H, I) / kBlock;
  (void)hipGetLastError();
  const bool nt = passes_cache(n, H, I);
  hipLaunchKernelGGL((nt ? unpack_w4_kernel<true> : unpack_w4_kernel<false>), dim3(pack_grid(n * per)), dim3(256), 0, stream, w4, W_bytes,
                     n, H, I, w, W_el, per);
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
