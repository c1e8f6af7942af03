// What the kernels of the experts' grouped matrix products share: the plan's segments, tiles of
// buffer rows in turn, operand tiles in LDS, activations and stores.
#pragma once

#include <cmath>
#include <type_traits>

#include "moonep_internal.h"

namespace moonep {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

#define LDS __attribute__((address_space(3)))

constexpr uint32_t kOob = 0x80000000u;     // a buffer offset past every range: reads as zero
constexpr int kBufferFlags = 0x00020000;   // raw buffer of 32-bit data
constexpr int kCus = 256;
constexpr int64_t kLastLevelCacheBytes = 256ll << 20;

constexpr int BK = 64;                     // k of a step

__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

// One group of buffer rows that shares its weights.
struct Seg {
  int row0, n;
  int w;                       // home expert, or E + rank * slots + slot
};

// Segment i of the plan: the E home groups, then the pieces.  Whatever the blob holds, the
// rows stay inside the buffer and the weights inside their tables.
template <class Load>
__device__ __forceinline__ Seg read_seg(const int32_t* plan, const moonep_sizes& s, int i, int np, Load load) {
  Seg g{0, 0, 0};
  if (i < s.E) {
    g.n = load(plan + s.o_keep + i);
    g.row0 = load(plan + s.o_home_row + i);
    g.w = i;
  } else if (i - s.E < np) {
    const int32_t* pc = plan + s.o_pieces + (int64_t)(i - s.E) * kPieceInts;
    const int e = load(pc + P_E), r = load(pc + P_R), slot = load(pc + P_SLOT);
    g.n = load(pc + P_CNT);
    g.row0 = load(pc + P_ROW0);
    if (slot >= 0) {
      g.w = s.E + r * s.slots + slot;
      if (slot >= s.slots || (unsigned)r >= (unsigned)s.R) g.n = 0;
    } else {
      g.w = e;
      if ((unsigned)e >= (unsigned)s.E) g.n = 0;
    }
  }
  const int rows = (int)s.recv_rows;
  if (g.n < 0 || g.n > rows || g.row0 < 0 || g.row0 > rows - g.n) g.n = 0;
  if (g.n == 0) g.row0 = g.w = 0;
  return g;
}

__device__ __forceinline__ Seg load_seg(const int32_t* plan, const moonep_sizes& s, int i, int np) {
  return read_seg(plan, s, i, np, [](const int32_t* p) { return *p; });
}

__device__ __forceinline__ int piece_count(const int32_t* plan, const moonep_sizes& s) {
  if (plan[s.o_hdr + H_STATUS] != 0) return 0;
  return min(max(plan[s.o_hdr + H_NPIECES], 0), s.P_max);
}

// A word of the plan through the scalar cache, at a uniform address: waited for apart from the
// loads into LDS.
__device__ __forceinline__ int scalar(const int32_t* p) {
  return *(const __attribute__((address_space(4))) int32_t*)(uintptr_t)p;
}

// load_seg for a uniform index.
__device__ __forceinline__ Seg scalar_seg(const int32_t* plan, const moonep_sizes& s, int i, int np) {
  return read_seg(plan, s, i, np, [](const int32_t* p) { return scalar(p); });
}

// 16 bytes a lane from the buffer straight into LDS, to `to` + OFF + lane * 16.  In assembly:
// for the builtin the compiler waits for every such load before any LDS read that it cannot
// tell apart from it, which here is each one, and the next steps' loads would never be in
// flight during this step's products.  No register is written, so there is none to wait
// for; arrive() is the wait.  m0 holds the LDS address.  gfx9 wants one instruction between
// writing it and the load, and five between a lane's value read into a scalar register,
// as which the compiler may bring back a spilled one, and a load that takes it.
// The compiler warns of m0 in the list because it keeps no value there across the statement:
// none is, it writes m0 itself right before each use (and these kernels' code has no other).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
template <int OFF>
__device__ __forceinline__ void load_lds(i32x4 rsrc, uint32_t voff, uint32_t to) {
  asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :: "s"(to), "v"(voff), "s"(rsrc), "i"(OFF) : "memory", "scc", "m0");
}
#pragma clang diagnostic pop

// ---------------------------------------------------------------------------------------
// operand tiles in LDS
// ---------------------------------------------------------------------------------------
// A step's tile holds BK k of R rows (of P or Q): 64 k are a cache line.  Two forms:
//   KC  memory is contiguous along k: LDS rows of 64 k, 16-byte chunk c of row r in the place
//       of chunk c ^ (r & 7): the 16 lanes that read at once hit different banks.
//   KS  memory is contiguous along the row index: LDS rows (one per k) of R elements, read
//       transposed.  A fragment of Q is 16 neighbours, and 32-byte unit u of row k is in the
//       place of u ^ (k & 3 | (k >> 3 & 1) << 2), or of u ^ (k & 3) where R is 64.  A
//       fragment f of P is every fourth run of four: runs f, f + 4, f + 8 and f + 12 of 64
//       elements; 16-byte chunk c is in the place of c ^ (k & 1 | (k & 2) << 2): two lanes
//       to a bank, the best that can be where only half of each 16 bytes is read.
// Both are filled by 16-byte loads straight into LDS; the swizzle is in each lane's
// global address, since a wave's load fills 1024 consecutive LDS bytes.

template <int R, bool KS, int NW, bool ISP>
struct Operand {
  static constexpr int kBytes = R * BK * 2;
  static constexpr int kLoads = kBytes / 1024 / NW;
  static_assert(kLoads >= 1 && kLoads * 1024 * NW == kBytes && (!KS || R >= (ISP ? 128 : 64)));
  static constexpr int kUnit4 = R >= 128;    // KS: a row of 64 has four units only
  uint32_t voff[kLoads];
  int kc;                        // KC: this lane's first k inside a step
  // the next step to load: its address, the k left from there, and the steps of this tile
  // from there on (uniform)
  const char* at;
  int left, todo;
  uint32_t ld;                   // bytes of a row in memory
  uint32_t skip;                 // KS: bytes of the row before `at`
  i32x4 rs;

  // KC: rowoff(r) is the byte offset of LDS row r in memory, or kOob
  template <class F>
  __device__ __forceinline__ void init_kc(int wave, int lane, F rowoff) {
    const int r = lane >> 3, c = (lane & 7) ^ r;
    kc = c * 8;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) voff[i] = rowoff((i * NW + wave) * 8 + r) + c * 16;
  }
  // KS: columns at or past ncols read as zero
  __device__ __forceinline__ void init_ks(int wave, int lane, int ncols) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int b = (i * NW + wave) * 1024 + lane * 16;
      const int k = b / (R * 2), cp = b % (R * 2) / 16;
      const int c = cp ^ (ISP ? (k & 1) | (k & 2) << 2 : ((k & 3) | (k >> 3 & kUnit4) << 2) << 1);
      voff[i] = c * 8 < ncols ? k * ld + c * 16 : kOob;
    }
  }
  // Makes the buffer descriptor of the next step and moves on.  Past the end everything is
  // out of range, and the tile is filled with zeros.
  __device__ __forceinline__ void next() {
    const uint64_t p = reinterpret_cast<uint64_t>(at);
    const int rows = max(min(left, BK), 0);
    const int range = !KS ? 0x7fffffff : rows ? rows * (int)ld - (int)skip : 0;
    rs = i32x4{(int)p, (int)(p >> 32) & 0xFFFF, range, kBufferFlags};
    if (!KS && left < BK) {     // the last k, or none
#pragma unroll
      for (int i = 0; i < kLoads; ++i) voff[i] |= kc >= left ? kOob : 0;
    }
    at += KS ? (uint64_t)ld * BK : BK * 2;
    left -= BK;
    --todo;
  }
  // load I of the step
  template <int I, int OFF>
  __device__ __forceinline__ void load(uint32_t to) const {
    load_lds<I * NW * 1024 + OFF>(rs, voff[I], to);
  }
};

// `v`, of which the compiler cannot know before: what is computed of it stays where it is
// used, and not in registers that the products need.
__device__ __forceinline__ int here(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// This lane's part of the LDS addresses of the fragments from row0 (a multiple of what the wave
// takes) on, and fragment f (16 rows), k from kk * 32 on, of the tile that `at` adds to it.
template <int R, bool KS, bool ISP>
__device__ __forceinline__ int fragment_lane(int row0, int lane) {
  if constexpr (!KS) return (row0 + (lane & 15)) * 128 + (((lane >> 4) ^ (lane & 7)) << 4);
  const int g = lane >> 4, j = (lane & 15) >> 2, k = (g * 8 + j) * (R * 2);
  if constexpr (ISP) return k + (((row0 / 8 + (lane & 3) * 2) ^ ((j & 1) | (j & 2) << 2)) << 4);
  return k + (((row0 / 16) ^ j ^ (R >= 128 ? (g & 1) << 2 : 0)) << 5) + (lane & 3) * 8;
}
template <int R, bool KS, bool ISP>
__device__ __forceinline__ bf16x8 fragment(int at, int f, int kk) {
  if constexpr (!KS) {
    return *(const LDS bf16x8*)((at ^ (kk << 6)) + f * 2048);
  } else {
    const int x = (ISP ? (at ^ (f >> 1) << 4) + (f & 1) * 8 : at ^ (f << 5)) + kk * 64 * R;
    union { s16x4 h[2]; bf16x8 v; } u;
    u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS s16x4*)x);
    u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS s16x4*)(x + 4 * R * 2));
    return u.v;
  }
}

// Row f * 16 + c of 64 LDS rows of a KC operand P holds row c * 4 + f of memory: lane c's
// results of the four fragments are neighbours.  With gate and up rows in turn, the first
// two fragments hold gate rows c * 2 + f, the others the same rows of up.
__device__ __forceinline__ int p_row(int r) { return (r & ~63) | (r & 15) << 2 | (r >> 4 & 3); }
__device__ __forceinline__ int p_row_pair(int r) { return (r >> 6) * 32 + ((r & 15) << 1 | (r >> 4 & 1)); }

template <int PF, int QF>
__device__ __forceinline__ void clear(f32x4 (&acc)[PF][QF]) {
#pragma unroll
  for (int p = 0; p < PF; ++p)
#pragma unroll
    for (int q = 0; q < QF; ++q) acc[p][q] = f32x4{0.f, 0.f, 0.f, 0.f};
}

// The tile of workgroup b in round `round` of a grid that is a multiple of 8: workgroups go
// to the 8 XCDs in turn, so each XCD takes a run of consecutive tiles, which share rows and
// weights in its L2.
__device__ __forceinline__ int tile_of(int round, int b, int grid) {
  return round * grid + (b & 7) * (grid >> 3) + (b >> 3);
}

// Tile `local` of an n x m grid of tiles: bands of kBand m, n by n within a band, so that 32
// consecutive tiles are about as many m as n.
constexpr int kBand = 4;
__device__ __forceinline__ void band(int local, int m, int n, int* tm, int* tn) {
  const int b = local / (kBand * n), r = local - b * kBand * n;
  const int cnt = min(kBand, m - b * kBand);
  *tm = b * kBand + r % cnt;
  *tn = r / cnt;
}

// s_waitcnt with the given vmcnt, and with lgkmcnt(0)
constexpr int wait_vm_lds(int vm) { return (vm & 15) | (vm >> 4) << 14 | 0x70; }

// Waits until at most VM of this wave's loads are on their way and its LDS reads are done,
// then for every wave of the workgroup.
template <int VM>
__device__ __forceinline__ void arrive() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(wait_vm_lds(VM));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The wave's own reads from memory have arrived: said here, the compiler does not wait for them
// later, when the next tile's loads would be waited for with them.
__device__ __forceinline__ void settled() { __builtin_amdgcn_s_waitcnt(wait_vm_lds(0)); }

template <int N, class F>
__device__ __forceinline__ void times(F f) {
  if constexpr (N > 0) {
    times<N - 1>(f);
    f(std::integral_constant<int, N - 1>{});
  }
}

// A tile's geometry: BP x BQ results by WP x WQ waves; LDS holds the tiles of NB steps of P and
// NB - 1 of Q.
template <int BP_, int BQ_, int WP_, int WQ_, int NB_>
struct Geometry {
  static constexpr int BP = BP_, BQ = BQ_, WP = WP_, WQ = WQ_, NB = NB_, NW = WP * WQ;
  static constexpr int PF = BP / WP / 16, QF = BQ / WQ / 16;
};

__device__ __forceinline__ uint32_t bf2(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  bf16x2 v{(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ float lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// act(z), and its slope.  SiLU: z s with s = 1 / (1 + e^-z), slope s + z s (1 - s).
// GELU in its tanh form: z p with p = (1 + tanh(u)) / 2 = 1 / (1 + e^-2u),
// u = c (z + 0.044715 z^3), slope p + 2 z p (1 - p) u'.  Beyond |z| = 16 p is exactly 0 or
// 1 in fp32 and u' would overflow, so u is taken of z cut to that range (a NaN stays one).
__device__ __forceinline__ float act_of(float z, int act, float* slope) {
  if (act == MOONEP_ACT_SILU) {
    const float s = 1.f / (1.f + __expf(-z));
    *slope = s + z * s * (1.f - s);
    return z * s;
  }
  const float c = 0.7978845608028654f;
  const float zc = z < -16.f ? -16.f : z > 16.f ? 16.f : z;
  const float z2 = zc * zc;
  const float p = 1.f / (1.f + __expf(-2.f * c * (zc + 0.044715f * zc * z2)));
  *slope = p + 2.f * zc * p * (1.f - p) * c * (1.f + 0.134145f * z2);
  return z * p;
}

// Memory from a tile's first element on, by byte offsets; kOob for what is not to be touched.
struct Window {
  __amdgpu_buffer_rsrc_t rs;
  template <class T>
  __device__ __forceinline__ explicit Window(T* p)
      : rs(__builtin_amdgcn_make_buffer_rsrc((void*)p, 0, 0x7fffffff, kBufferFlags)) {}
  __device__ __forceinline__ void store(uint32_t v, uint32_t at) const {
    __builtin_amdgcn_raw_buffer_store_b32(v, rs, at, 0, 0);
  }
  __device__ __forceinline__ void store(u32x2 v, uint32_t at) const {
    __builtin_amdgcn_raw_buffer_store_b64(v, rs, at, 0, 0);
  }
  template <bool NT>
  __device__ __forceinline__ void store(f32x4 v, uint32_t at) const {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rs, at, 0, NT ? 2 : 0);
  }
  __device__ __forceinline__ u32x2 load2(uint32_t at) const {
    return __builtin_amdgcn_raw_buffer_load_b64(rs, at, 0, 0);
  }
  __device__ __forceinline__ f32x4 load4(uint32_t at) const {
    return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, at, 0, 0));
  }
};

template <int CTRL>
__device__ __forceinline__ float quad_move(float v) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, 0xf, 0xf, true));
}

// Inclusive sum over the lanes of a wave.
__device__ __forceinline__ int wave_sums(int v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// The row tiles of the plan's segments, BQ rows each, times `nt` column tiles, dealt out to the
// workgroups round by round.  Each wave looks its workgroup's tiles up on its own, lane l that
// of round first + l: no LDS, no barrier, and 64 rounds without a wait for memory.
template <int BQ>
struct RowTiles {
  const int32_t* plan;
  const moonep_sizes& s;
  const int lane, np, nseg, nt;
  int per, sum, tiles;
  Seg mine;                                    // the lane's last
  int lane_row;                                // first row, or none
  uint32_t lane_rest;                          // rows - 1, column tile, weight
  // a weight is one of at most 1024 + 64 * 256: 15 bits
  static constexpr int kRowBits = BQ <= 16 ? 4 : BQ <= 32 ? 5 : BQ <= 64 ? 6 : BQ <= 128 ? 7 : 8;
  static constexpr uint32_t kMaxTn = 1u << (17 - kRowBits);

  struct Tile {
    int row, rows, tn, w;                      // rows 0: none
  };

  // Lane l sums the row tiles of segments [l * per, l * per + per).
  __device__ __forceinline__ RowTiles(const int32_t* plan, const moonep_sizes& s, int lane, int nt, int tiles_bound)
      : plan(plan), s(s), lane(lane), np(uni(piece_count(plan, s))), nseg(s.E + np), nt(nt), sum(0), mine{0, 0, 0},
        lane_row(-1), lane_rest(0) {
    per = (nseg + 63) / 64;
    for (int j = 0; j < per; ++j) {
      const int i = lane * per + j;
      if (i < nseg) mine = load_seg(plan, s, i, np);
      if (i < nseg) sum += (mine.n + BQ - 1) / BQ;
    }
    sum = wave_sums(sum, lane);
    tiles = min(__builtin_amdgcn_readlane(sum, 63), tiles_bound) * nt;
  }

  __device__ __forceinline__ void look_up(int first, bool held) {
    const int t = tile_of(first + lane, blockIdx.x, gridDim.x);
    const int want = t < 0 || t >= tiles ? 0 : t / nt;
    int l = 0;                                  // the sums that are at most `want`
#pragma unroll
    for (int d = 32; d; d /= 2)
      if (__shfl(sum, l + d - 1) <= want) l += d;
    int below = __shfl(sum, max(l - 1, 0));
    below = l ? below : 0;
    Seg g{0, 0, 0};
    int mt = 0;
    if (held && per == 1) {                     // the other lanes hold them all: no second read
      g = Seg{__shfl(mine.row0, l), __shfl(mine.n, l), __shfl(mine.w, l)};
      mt = (g.n + BQ - 1) / BQ;
    } else {
      for (int j = 0; j < per; ++j) {
        g = load_seg(plan, s, min(l * per + j, nseg - 1), np);
        mt = (g.n + BQ - 1) / BQ;
        if (below + mt > want) break;
        below += mt;
      }
    }
    lane_row = -1;
    const int local = t - below * nt;
    if (t >= 0 && t < tiles && local >= 0 && local < mt * nt) {
      int tm, tn;
      band(local, mt, nt, &tm, &tn);
      lane_row = g.row0 + tm * BQ;
      lane_rest = (uint32_t)(min(g.n - tm * BQ, BQ) - 1) | (uint32_t)tn << kRowBits | (uint32_t)g.w << 17;
    }
    settled();
  }

  __device__ __forceinline__ Tile tile(int round) {
    if (round && (round & 63) == 0) look_up(round, false);
    const int row = __builtin_amdgcn_readlane(lane_row, round & 63);
    const uint32_t rest = __builtin_amdgcn_readlane(lane_rest, round & 63);
    if (row < 0) return {0, 0, 0, 0};
    return {row, (int)(rest & ((1u << kRowBits) - 1)) + 1, (int)(rest >> kRowBits & (kMaxTn - 1)), (int)(rest >> 17)};
  }
};

// ---------------------------------------------------------------------------------------
// the host's side
// ---------------------------------------------------------------------------------------

inline bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Memory that the experts' calls are given.
inline Span plan_span(const moonep_plan_desc* d) { return span(d->dev, 1, d->sz.plan_bytes); }
inline Span rows_span(const moonep_plan_desc* d, const uint16_t* p, int n) { return span(p, d->sz.recv_rows, 2ll * n); }

}  // namespace
}  // namespace moonep
