// The gated feed-forward experts on the planned buffer: grouped matrix products over the
// plan's groups, forward and backward.
//
//   forward        gate = x Wg^T, up = x Wu^T, h = act(gate) * up     (one kernel)
//                  y = h Wd^T
//   rows' gradient g_h = g_y Wd, g_gate = g_h * up * act'(gate), g_up = g_h * act(gate)
//                  g_recv = g_gate Wg + g_up Wu
//   weights'       g_Wg = g_gate^T x, g_Wu = g_up^T x, g_Wd = g_y^T h
//
// Every product is D[q, p] = sum_k Q[q, k] * P[p, k] with v_mfma_f32_16x16x32_bf16, p being the
// index along the output's rows in memory: a lane holds four q of one p.  Which p belong
// to which of a wave's four fragments is chosen so that a lane's results of the four are
// neighbours, and those of lanes that follow each other are too.  A CU writes such runs
// four times as fast as 16-byte pieces of as many rows as it has lanes (141 and 35 GB/s),
// and all of an output is written at a tile's end.
//
// Roundings.  Sums, activations and their slopes are fp32, and each output is rounded once.  h,
// g_gate and g_up are outputs and the second products' operands, and so are rounded to bf16 in
// between: the matrix units multiply bf16 ten times as fast as fp32 (1530 and 153 TF in the
// library's products), and a second bf16 product of what the rounding leaves would cost
// its time once more.  y and g_recv are off by 0.0023 to 0.0024 of their size for it, against
// 0.0017 from one rounding at the end.  The weights' gradient is not rounded at all.
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

enum Op { FWD1, FWD2, BWD1, BWD2 };

struct FfnArgs {
  const int32_t* plan;
  moonep_sizes s;
  int H, I, act;
  const uint16_t* in;          // the rows: recv, h, g_y or g_gu
  const uint16_t* home_w;
  const uint16_t* slot_w;
  int64_t W_el;
  const uint16_t* gu_in;       // BWD1: the saved gate and up rows
  uint16_t* out;               // h, y, g_gu or g_recv
  uint16_t* gu_out;            // FWD1: gate and up rows, or null
  int tiles_bound;             // row tiles of any plan of these sizes, at most
};

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

// The products of one tile after another, without a break between them.  A step is two halves,
// each a matrix instruction (32 k) deep.  While a half is multiplied out of
// registers, the next is read from LDS into others.  When a step's last half is to be
// multiplied, every wave has read the whole tile: then the tiles of Q's step NB - 1 and P's
// step NB further on start to load over it, and the half that is read is the next step's
// first.  Past a tile's end these are the next tile's steps: more_p() and more_q() turn their
// side to it, or fill with zeros.  One barrier a step.  Each half is cut into parts that
// start a share of the loads, then spread a share of the LDS reads among their matrix
// instructions.
template <class G, bool KSP, bool KSQ>
struct Pipe {
  static constexpr int PF = G::PF, QF = G::QF, NB = G::NB;
  using OpP = Operand<G::BP, KSP, G::NW, true>;
  using OpQ = Operand<G::BQ, KSQ, G::NW, false>;
  static constexpr int kP = OpP::kBytes, kQ = OpQ::kBytes, kLP = OpP::kLoads, kLQ = OpQ::kLoads;
  static constexpr int kQ0 = NB * kP, kLds = NB * kP + (NB - 1) * kQ;
  static constexpr int kParts = QF >= 4 ? 4 : QF, kM = PF * QF / kParts, kF = PF + QF;
  static constexpr int kAhead = kLP + (NB - 3) * (kLP + kLQ);   // loads after the next step's
  static_assert(PF == 4 && QF % kParts == 0 && (NB - 1) * kLP + (NB - 2) * kLQ < 64 && kLds <= 160 * 1024);
  uint32_t lds;                   // this wave's first LDS byte of a load
  int lane_p, lane_q;             // this lane's first LDS byte of a fragment
  int cp, cq;                     // the current step's tiles
  OpP P;
  OpQ Q;

  __device__ __forceinline__ Pipe(char* smem, int wave, int lane) : cp(0), cq(kQ0) {
    const int at = (int)(uint32_t)(uintptr_t)(LDS char*)smem;
    lds = uni(at + wave * 1024);
    lane_p = at + fragment_lane<G::BP, KSP, true>(wave % G::WP * PF * 16, lane);
    lane_q = at + fragment_lane<G::BQ, KSQ, false>(wave / G::WP * QF * 16, lane);
  }

  // the first tile's first loads
  template <class FP, class FQ>
  __device__ __forceinline__ void begin(FP more_p, FQ more_q) {
    times<NB>([&](auto i) {
      more_p();
      P.next();
      times<kLP>([&](auto j) { P.template load<j, i * kP>(lds); });
      if constexpr (i < NB - 1) {
        more_q();
        Q.next();
        times<kLQ>([&](auto j) { Q.template load<j, kQ0 + i * kQ>(lds); });
      }
    });
    arrive<(NB - 1) * kLP + (NB - 2) * kLQ>();
  }

  // The next `nk` steps.  `live`: how many of the wave's rows of Q are there; where they are
  // not ALL, the matrix instructions of the rest are left out.  `younger`: at least STORES
  // stores went out since the last step, and need not have arrived for its loads to have
  // (memory operations are counted in order).
  template <bool ALL, int STORES, class FP, class FQ>
  __device__ __forceinline__ void run(int nk, int live, bool younger, f32x4 (&acc)[PF][QF], FP more_p,
                                      FQ more_q) {
    bf16x8 a[2][PF], b[2][QF];
    {
      const int tp = here(lane_p + cp), tq = here(lane_q + cq);
#pragma unroll
      for (int p = 0; p < PF; ++p) a[0][p] = fragment<G::BP, KSP, true>(tp, p, 0);
#pragma unroll
      for (int q = 0; q < QF; ++q) b[0][q] = fragment<G::BQ, KSQ, false>(tq, q, 0);
    }
    for (int i = 0; i < nk; ++i) {
      times<2>([&](auto h) {
        constexpr bool kLast = h == 1;
        const int np = cp == (NB - 1) * kP ? 0 : cp + kP, nq = cq == kQ0 + (NB - 2) * kQ ? kQ0 : cq + kQ;
        if constexpr (kLast) {
          more_q();
          Q.next();
          more_p();
          P.next();
          constexpr int kMore = kAhead + STORES < 63 ? kAhead + STORES : 63;
          if (younger && i == 0) arrive<kMore>();
          else arrive<kAhead>();
        }
        const uint32_t top = lds + cp, toq = lds + cq;
        const int tp = here(lane_p + (kLast ? np : cp)), tq = here(lane_q + (kLast ? nq : cq));
        times<kParts>([&](auto c) {
          times<kLP + kLQ>([&](auto j) {
            if constexpr (kLast && j * kParts / (kLP + kLQ) == c) {
              if constexpr (j < kLQ) Q.template load<j, 0>(toq);
              else P.template load<j - kLQ, 0>(top);
            }
          });
          times<kF>([&](auto f) {
            if constexpr (f * kParts / kF == c) {
              if constexpr (f < PF) a[h ^ 1][f] = fragment<G::BP, KSP, true>(tp, f, !kLast);
              else b[h ^ 1][f - PF] = fragment<G::BQ, KSQ, false>(tq, f - PF, !kLast);
            }
          });
          if (ALL || c * (QF / kParts) * 16 < live)
            times<kM>([&](auto m) {
              constexpr int p = m % PF, q = c * (QF / kParts) + m / PF;
              acc[p][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[h][q], a[h][p], acc[p][q], 0, 0, 0);
            });
          if constexpr (ALL)
            times<kM>([&](auto) {
              __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
              __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            });
          __builtin_amdgcn_sched_barrier(0);
        });
        if constexpr (kLast) {
          cp = np;
          cq = nq;
        }
      });
    }
  }
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

// This lane's results i of the four fragments, as four neighbours along p.  For KC that is
// what they are.  For KS lane (m, e) holds p = m * 16 + f * 4 + e for f = 0 ... 3, and the
// four lanes of a quad exchange theirs, for m * 16 + e * 4 + f.
template <bool KS, int QF>
__device__ __forceinline__ f32x4 neighbours(const f32x4 (&acc)[4][QF], int q, int i, int lane) {
  const float v0 = acc[0][q][i], v1 = acc[1][q][i], v2 = acc[2][q][i], v3 = acc[3][q][i];
  if constexpr (!KS) return f32x4{v0, v1, v2, v3};
  const bool odd = lane & 1, high = lane & 2;
  // every lane takes part in a move, so none is in a branch
  const float x0 = quad_move<0xB1>(v0), x1 = quad_move<0xB1>(v1);                          // of lane ^ 1
  const float x2 = quad_move<0xB1>(v2), x3 = quad_move<0xB1>(v3);
  const float n0 = odd ? x1 : v0, n1 = odd ? v1 : x0, n2 = odd ? x3 : v2, n3 = odd ? v3 : x2;
  const float y0 = quad_move<0x4E>(n0), y1 = quad_move<0x4E>(n1);                          // of lane ^ 2
  const float y2 = quad_move<0x4E>(n2), y3 = quad_move<0x4E>(n3);
  return f32x4{high ? y2 : n0, high ? y3 : n1, high ? n2 : y0, high ? n3 : y1};
}

// ---------------------------------------------------------------------------------------
// the row products: forward, and the rows' gradient
// ---------------------------------------------------------------------------------------

// Inclusive sum over the lanes of a wave.
__device__ __forceinline__ int wave_sums(int v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// What bounds it, on MI355X: with hundreds of rows to an expert, power.  1024 rows to each of
// 32 experts, H 7168, I 2048: 1.68 and 0.81 ms, 1160 TF of the formula's products, 1350 with
// the rows that fill up the groups' last tiles; the matrix units are busy 60% of the time at
// 1.7 GHz, where few rows run at 2.4 GHz.  (A 16384 x 8192 x 7168 library product: 88% at
// 1.48 GHz, 1360 TF.)  With few rows, the weights' stream: 64 rows in 64 experts at one
// token a rank, 4.0 GB of weights in 428 and 219 us, 6.1 TB/s.  The gradient g_gate, g_up:
// its epilogue, which reads two more arrays and writes two, and nothing else runs beside it on
// the CU.  49152 rows, H 2048, I 1408: 0.41 ms, 1340 to 1400 tiles in six rounds of 69 us, of
// which the 32 steps take 42.  g_recv of these: 0.51 ms, 1780 to 1860 tiles, of which the last
// tenth to third of a round is paid as a whole one, and power.
template <int OP, class G>
__global__ __launch_bounds__(64 * G::NW, 2) void rows_kernel(const FfnArgs a) {
#ifdef __HIP_DEVICE_COMPILE__   // gfx950 builtins: the host pass needs the kernel's name only
  constexpr int BP = G::BP, BQ = G::BQ, WP = G::WP, PF = G::PF, QF = G::QF;
  constexpr bool KSP = OP == BWD1 || OP == BWD2;
  constexpr bool PAIR = OP == FWD1;            // P's rows are gate and up rows in turn
  constexpr int BN = PAIR ? BP / 2 : BP;       // output columns of a tile
  using Tiles = Pipe<G, KSP, false>;
  __shared__ __align__(1024) char smem[Tiles::kLds];

  const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6);
  const int wp = wave % WP, wq = wave / WP;
  const int32_t* plan = a.plan;
  if (uni(plan[a.s.o_hdr + H_STATUS]) != 0) return;
  const int np = uni(piece_count(plan, a.s));
  const int nseg = a.s.E + np;
  const int K = OP == FWD1 || OP == BWD1 ? a.H : OP == FWD2 ? a.I : 2 * a.I;
  const int N = OP == FWD1 || OP == BWD1 ? a.I : a.H;
  const int nt = (N + BN - 1) / BN;
  const int nk = max((K + BK - 1) / BK, G::NB);      // P loads NB steps ahead, into one more tile only

  // Lane l sums the row tiles of segments [l * per, l * per + per).
  const int per = (nseg + 63) / 64;
  int sum = 0;
  Seg mine{0, 0, 0};                           // the lane's last
  for (int j = 0; j < per; ++j) {
    const int i = lane * per + j;
    if (i < nseg) mine = load_seg(plan, a.s, i, np);
    if (i < nseg) sum += (mine.n + BQ - 1) / BQ;
  }
  sum = wave_sums(sum, lane);
  const int tiles = min(__builtin_amdgcn_readlane(sum, 63), a.tiles_bound) * nt;

  // Lane l looks up the workgroup's tile of round first + l, each wave on its own: no LDS,
  // no barrier, and 64 rounds without a wait for memory.
  int lane_row = -1;                            // first row, or none
  uint32_t lane_rest = 0;                       // rows - 1, column tile, weight
  auto look_up = [&](int first, bool held) {
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
        g = load_seg(plan, a.s, min(l * per + j, nseg - 1), np);
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
      lane_rest = (uint32_t)(min(g.n - tm * BQ, BQ) - 1) | (uint32_t)tn << 8 | (uint32_t)g.w << 17;
    }
    settled();
  };
  struct Tile {
    int row, rows, n0, w;                       // rows 0: none
  };
  auto tile = [&](int round) -> Tile {
    if (round && (round & 63) == 0) look_up(round, false);
    const int row = __builtin_amdgcn_readlane(lane_row, round & 63);
    const uint32_t rest = __builtin_amdgcn_readlane(lane_rest, round & 63);
    if (row < 0) return {0, 0, 0, 0};
    return {row, (int)(rest & 255) + 1, (int)(rest >> 8 & 511) * BN, (int)(rest >> 17)};
  };
  look_up(0, true);

  Tiles pipe(smem, wave, lane);
  auto& P = pipe.P;
  auto& Q = pipe.Q;
  auto start_p = [&](const Tile& t) {
    const uint16_t* W = t.w < a.s.E ? a.home_w + t.w * a.W_el : a.slot_w + (t.w - a.s.E) * a.W_el;
    if (OP == FWD2 || OP == BWD1) W += 2ll * a.I * a.H;
    P.left = K;
    P.todo = nk;
    if constexpr (!KSP) {
      P.ld = K * 2;
      P.skip = 0;
      P.at = reinterpret_cast<const char*>(W) + (int64_t)t.n0 * P.ld;
      P.init_kc(wave, here(lane), [&](int r) -> uint32_t {
        const int c = PAIR ? p_row_pair(r) : p_row(r);
        return t.n0 + c < N ? (uint32_t)(c + (PAIR ? (r >> 5 & 1) * a.I : 0)) * P.ld : kOob;
      });
    } else {
      P.ld = N * 2;
      P.skip = t.n0 * 2;
      P.at = reinterpret_cast<const char*>(W) + P.skip;
      P.init_ks(wave, here(lane), N - t.n0);
    }
  };
  auto start_q = [&](const Tile& t) {
    Q.left = K;
    Q.todo = nk;
    Q.ld = K * 2;
    Q.skip = 0;
    Q.at = reinterpret_cast<const char*>(a.in) + (int64_t)t.row * Q.ld;
    Q.init_kc(wave, here(lane), [&](int r) -> uint32_t { return r < t.rows ? r * Q.ld : kOob; });
  };

  Tile cur = tile(0), nxt = tile(1);
  if (!cur.rows) return;
  auto more_p = [&] { if (P.todo == 0 && nxt.rows) start_p(nxt); };
  auto more_q = [&] { if (Q.todo == 0 && nxt.rows) start_q(nxt); };
  start_p(cur);
  start_q(cur);
  pipe.begin(more_p, more_q);
  for (int round = 1;; ++round) {
    f32x4 acc[PF][QF];
    clear(acc);
    const int trow = cur.row, tq = cur.rows, tn0 = cur.n0;
    const bool idle = tn0 + wp * (BN / WP) >= N;                    // no columns for this wave
    const int live = idle ? 0 : tq - wq * QF * 16;
    constexpr int kStores = 4 * QF;
    if (live >= QF * 16) pipe.template run<true, kStores>(nk, live, round > 1, acc, more_p, more_q);
    else pipe.template run<false, kStores>(nk, live, round > 1, acc, more_p, more_q);

    // what the results' places are made of is worked out here, not kept during the products
    const int ln = here(lane);
    const int ldo = OP == BWD1 ? 2 * N : N;                               // elements of an output row
    const int64_t o0 = (int64_t)trow * ldo + tn0;
    const Window out(a.out + o0), gu(OP == FWD1 ? a.gu_out + 2 * o0 - tn0 : a.gu_in + o0);
    const bool save = OP == FWD1 && a.gu_out;
    const int c = wp * (BN / WP) + (ln & 15) * (PAIR ? 2 : 4);
    const bool in = tn0 + c < N;
    auto place = [&](int q, int i, int ld) -> uint32_t {
      const int r = (wq * QF + q) * 16 + (ln >> 4) * 4 + i;
      return in && r < tq ? (uint32_t)(r * ld + c) * 2 : kOob;
    };
    // BWD1: the saved gate and up of the next two groups of rows are on their way while one is
    // worked on.  With none ahead each group waits for memory: 445 us against 404 at 49152
    // rows, H 2048, I 1408.
    constexpr int kSaved = OP == BWD1 ? (QF < 3 ? QF : 3) : 1;
    u32x2 vg[kSaved][4], vu[kSaved][4];
    auto fetch = [&](int q) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t at = place(q, i, ldo);
        vg[q % kSaved][i] = gu.load2(at);
        vu[q % kSaved][i] = gu.load2(at == kOob ? kOob : at + N * 2);
      }
    };
    if constexpr (OP == BWD1) {
#pragma unroll
      for (int q = 0; q < kSaved - 1; ++q) fetch(q);
      if constexpr (kSaved == 1) fetch(0);
    }
#pragma unroll
    for (int q = 0; q < QF; ++q) {
      if constexpr (OP == BWD1 && kSaved > 1) {
        if (q + kSaved - 1 < QF) fetch(q + kSaved - 1);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t at = place(q, i, ldo);
        if constexpr (OP == FWD1) {
          const float g0 = acc[0][q][i], g1 = acc[1][q][i], u0 = acc[2][q][i], u1 = acc[3][q][i];
          float s0, s1;
          out.store(bf2(act_of(g0, a.act, &s0) * u0, act_of(g1, a.act, &s1) * u1), at);
          if (save) {
            const uint32_t at2 = place(q, i, 2 * N);
            gu.store(bf2(g0, g1), at2);
            gu.store(bf2(u0, u1), at2 == kOob ? kOob : at2 + N * 2);
          }
        } else {
          const f32x4 d = neighbours<KSP>(acc, q, i, ln);
          if constexpr (OP == BWD1) {
            float gg[4], gv[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t wg = vg[q % kSaved][i][e >> 1], wu = vu[q % kSaved][i][e >> 1];
              const float z = e & 1 ? hi(wg) : lo(wg), u = e & 1 ? hi(wu) : lo(wu);
              float slope;
              gv[e] = d[e] * act_of(z, a.act, &slope);
              gg[e] = d[e] * u * slope;
            }
            out.store(u32x2{bf2(gg[0], gg[1]), bf2(gg[2], gg[3])}, at);
            out.store(u32x2{bf2(gv[0], gv[1]), bf2(gv[2], gv[3])}, at == kOob ? kOob : at + N * 2);
          } else {
            out.store(u32x2{bf2(d[0], d[1]), bf2(d[2], d[3])}, at);
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);         // or all results are worked on at once, and spill
    }
    if (!nxt.rows) break;
    cur = nxt;
    nxt = tile(round + 1);
  }
  settled();                      // LDS is not given up while loads may still write to it
#endif
}

// ---------------------------------------------------------------------------------------
// the weights' gradient
// ---------------------------------------------------------------------------------------
// Target i is home expert i (its home group, then its fallback pieces), or the slot of
// piece i - E.  A target's two products, [2I, H] and [H, I], are cut into tiles; k runs
// over the buffer rows of the target's segments.

struct GradArgs {
  const int32_t* plan;
  moonep_sizes s;
  int H, I, accumulate;
  const uint16_t *recv, *g_y, *h, *g_gu;
  float *home, *rep;
  int64_t G_el;
};

// What bounds it, on MI355X: its products and its writes, one after the other, a tile at a time on
// each CU, both slowed by power.  16384 rows of 16 experts, H 7168, I 2048: 1.58 ms, 914 TF,
// 50 rounds of 31.6 us, of which 14 steps take about 19 and 67 MB of gradients 10 at 6.5
// TB/s; the matrix units are busy 50% of the time at 1.6 GHz.
// Few rows: three steps at least to a tile (what LDS holds), then its writes, with
// nothing beside them; 21 experts of 73 rows, H 1000, I 680: 200 MB in 49 us.
// NT: gradients that the last-level cache cannot hold pass it by: 3-6% faster from 0.8 GB on, 10%
// slower at 0.2 GB.
template <class G, bool NT>
__global__ __launch_bounds__(64 * G::NW, 2) void grad_kernel(const GradArgs a) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int BP = G::BP, BQ = G::BQ, WP = G::WP, PF = G::PF, QF = G::QF;
  using Tiles = Pipe<G, true, true>;
  __shared__ __align__(1024) char smem[Tiles::kLds];
  const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6);
  const int wp = wave % WP, wq = wave / WP;
  const int32_t* plan = a.plan;
  const moonep_sizes& s = a.s;
  const int np = uni(piece_count(plan, s));
  const bool valid = uni(plan[s.o_hdr + H_STATUS]) == 0;
  const int p1 = (a.H + BP - 1) / BP, q1 = (2 * a.I + BQ - 1) / BQ;      // gate and up
  const int p2 = (a.I + BP - 1) / BP, q2 = (a.H + BQ - 1) / BQ;          // down
  const int per = p1 * q1 + p2 * q2;
  const int tiles = (s.E + np) * per;

  // A tile: the target's first segment and its fallback pieces [f0, f1), which product, where.
  struct Tile {
    int target, row, n, f0, f1, steps, down, p0, q0;        // steps 0: none
    float* out;
  };
  int round = 0;
  auto tile = [&]() -> Tile {
    for (;;) {
      const int first = tile_of(round, 0, gridDim.x);
      const int t = tile_of(round, blockIdx.x, gridDim.x);
      ++round;
      if (first >= tiles) return Tile{};
      if (t >= tiles) continue;
      Tile r{};
      r.target = t / per;
      int local = t - r.target * per;
      const Seg seg = scalar_seg(plan, s, r.target, np);
      r.row = seg.row0;
      r.n = valid ? seg.n : 0;
      if (r.target < s.E) {
        if (np) {
          r.f0 = min(max(scalar(plan + s.o_pfirst + r.target), 0), np);
          r.f1 = r.f0 + min(max(scalar(plan + s.o_pnum + r.target), 0), np - r.f0);
        }
        r.out = a.home + r.target * a.G_el;
      } else {
        if (seg.n == 0 || seg.w < s.E) continue;         // a fallback piece: in its home's sum
        r.out = a.rep + (seg.w - s.E) * a.G_el;
      }
      r.down = local >= p1 * q1;
      if (r.down) local -= p1 * q1;
      int tq, tp;
      band(local, r.down ? q2 : q1, r.down ? p2 : p1, &tq, &tp);
      r.p0 = tp * BP;
      r.q0 = tq * BQ;
      if (r.down) r.out += 2ll * a.I * a.H;
      r.steps = (r.n + BK - 1) / BK;
      for (int f = r.f0; f < r.f1; ++f) {
        const Seg fb = scalar_seg(plan, s, s.E + f, np);
        if (fb.w == r.target) r.steps += (fb.n + BK - 1) / BK;
      }
      if (r.steps == 0 && a.accumulate) continue;
      r.steps = max(r.steps, G::NB);             // P loads NB steps ahead, into one more tile only
      return r;
    }
  };

  Tiles pipe(smem, wave, lane);
  auto& P = pipe.P;
  auto& Q = pipe.Q;
  Tile cur = tile(), nxt = tile();
  if (!cur.steps) return;
  int tp = 0, fp = 0, ep = 0, tq = 0, fq = 0, eq = 0;      // each side's target, next piece and last
  auto start_p = [&](const Tile& t) {
    P.ld = (t.down ? a.I : a.H) * 2;
    P.skip = t.p0 * 2;
    P.at = reinterpret_cast<const char*>(t.down ? a.h : a.recv) + (int64_t)t.row * P.ld + P.skip;
    P.left = t.n;
    P.todo = t.steps;
    P.init_ks(wave, here(lane), (t.down ? a.I : a.H) - t.p0);
    tp = t.target;
    fp = t.f0;
    ep = t.f1;
  };
  auto start_q = [&](const Tile& t) {
    Q.ld = (t.down ? a.H : 2 * a.I) * 2;
    Q.skip = t.q0 * 2;
    Q.at = reinterpret_cast<const char*>(t.down ? a.g_y : a.g_gu) + (int64_t)t.row * Q.ld + Q.skip;
    Q.left = t.n;
    Q.todo = t.steps;
    Q.init_ks(wave, here(lane), (t.down ? a.H : 2 * a.I) - t.q0);
    tq = t.target;
    fq = t.f0;
    eq = t.f1;
  };
  // on to the next fallback piece with rows, where a side has done its segment
  auto walk = [&](auto& side, const char* src, int target, int& f, int end) {
    while (side.left <= 0 && f < end) {
      const Seg fb = scalar_seg(plan, s, s.E + f, np);
      ++f;
      if (fb.w == target && fb.n > 0) {
        side.at = src + (int64_t)fb.row0 * side.ld + side.skip;
        side.left = fb.n;
      }
    }
  };
  bool down_p = false, down_q = false;
  auto more_p = [&] {
    if (P.todo == 0 && nxt.steps) {
      start_p(nxt);
      down_p = nxt.down;
    }
    walk(P, reinterpret_cast<const char*>(down_p ? a.h : a.recv), tp, fp, ep);
  };
  auto more_q = [&] {
    if (Q.todo == 0 && nxt.steps) {
      start_q(nxt);
      down_q = nxt.down;
    }
    walk(Q, reinterpret_cast<const char*>(down_q ? a.g_y : a.g_gu), tq, fq, eq);
  };
  start_p(cur);
  start_q(cur);
  down_p = down_q = cur.down;
  pipe.begin(more_p, more_q);
  for (bool later = false;; later = true) {
    f32x4 acc[PF][QF];
    clear(acc);
    pipe.template run<true, 4 * QF>(cur.steps, 0, later, acc, more_p, more_q);
    const int tp0 = cur.p0, tq0 = cur.q0, tpc = cur.down ? a.I : a.H, tqc = cur.down ? a.H : 2 * a.I;
    const bool add = a.accumulate && cur.target < s.E;
    float* const tout = cur.out;
    const Window o(tout + (int64_t)tq0 * tpc + tp0);
    const int ln = here(lane), c = wp * 64 + (ln & 15) * 4;
    const bool in = tp0 + c < tpc;
#pragma unroll
    for (int f = 0; f < QF; ++f) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = (wq * QF + f) * 16 + (ln >> 4) * 4 + i;
        const uint32_t at = in && tq0 + r < tqc ? (uint32_t)(r * tpc + c) * 4 : kOob;
        f32x4 d = neighbours<true>(acc, f, i, ln);
        if (add) d = d + o.load4(at);
        o.template store<NT>(d, at);
      }
      __builtin_amdgcn_sched_barrier(0);         // or all results are worked on at once, and spill
    }
    if (!nxt.steps) break;
    cur = nxt;
    nxt = tile();
  }
  settled();                      // LDS is not given up while loads may still write to it
#endif
}

using Large = Geometry<256, 256, 4, 2, 3>;       // one workgroup of 8 waves to a CU
using Tall = Geometry<256, 128, 4, 2, 3>;
using Square = Geometry<128, 128, 2, 2, 3>;      // two of 4, as the next
using Medium = Geometry<128, 64, 2, 2, 3>;
using Small = Geometry<128, 32, 2, 2, 4>;
enum Tile { LARGE, TALL, SQUARE, MEDIUM, SMALL };

template <int OP, class G>
hipError_t launch_rows_as(FfnArgs a, int per_cu, hipStream_t st) {
  const int64_t segs = std::min<int64_t>(a.s.E + a.s.P_max, a.s.A);
  const int64_t mt = a.s.A / G::BQ + segs;
  const int N = OP == FWD1 || OP == BWD1 ? a.I : a.H;
  constexpr int BN = OP == FWD1 ? G::BP / 2 : G::BP;
  const int64_t tiles = mt * ((N + BN - 1) / BN);
  a.tiles_bound = (int)mt;
  const int grid = (int)std::min<int64_t>((tiles + 7) / 8 * 8, per_cu * kCus);
  hipLaunchKernelGGL((rows_kernel<OP, G>), dim3(grid), dim3(64 * G::NW), 0, st, a);
  return hipGetLastError();
}

// Which tile.  The large ones read the weights and the rows fewer times and multiply at the best
// rate, but fill up more rows with zeros and leave CUs without a tile.  So each launch takes
// the tile whose time is the least by a model: rounds of tiles over the CUs times a tile's
// time, which is its steps and about four more for its start and end.  Below the weights' own
// time at 6 TB/s, tiles differ only in what they leave of it, about a quarter of theirs.
// An expert's group and its replicas end inside a tile: half of one to each group.
// Measured on MI355X, us of each launch by itself (Large, Tall, Medium, Small; mean rows of an
// expert).  The model takes the best, or one within 2% of it, but for the two marked *, 6%
// and 8% behind; R is 8, and 4 for 4 experts.
//   64 experts, H 7168, I 2048, gate and up   16:  742,  709,  701,  699    64:  754,  734,  758, 1145
//                                            128:  811,  801, 1126, 1825   256: 1263, 1213, 1856, 3483
//                               down          16:  374,  372,  373,  366    64:  403,  403,  452,  533
//                                            128:  438, *466,  545,  810   256:  594,  597,  842, 1497
//   64 experts, H 2048, I 1024, g_gate, g_up  32:  109,   89,   82,   69    64:  113,   95,   81,   86
//                                            128:  125,  102,  108,  127   512:  207,  207,  261,  382
//                               g_recv        32:  134,  125, *135,  138    64:  136,  130,  128,  167
//                                            128:  147,  135,  173,  239   512:  291,  304,  426,  779
//   16 experts, H 2048, I 1024, gate and up  128:   51,   38,   49,   51   256:   54,   62,   61,   77
//                               down         128:   28,   22,   27,   29   256:   29,   33,   33,   43
//    4 experts, H 2048, I 512,  gate and up  128:   38,   31,   18,   15   256:   49,   30,   18,   20
//                               down         128: 14.5, 12.6, 10.0, 10.0   256: 17.7, 12.2, 10.4, 13.1
//   32 experts, H 1000, I 680,  g_gate, g_up 256:   47,   30,   36,   49    g_recv:  40,   44,   51,   70
//    4 experts, H 1024, I 512,  g_gate, g_up 1024:  44,   27,   19,   21    g_recv:  29,   19,   21,   24
// (128x128 tiles, two workgroups to a CU, were never the best.)
Tile rows_tile(int op, const moonep_sizes& s, int H, int I) {
  const int N = op == FWD1 ? 2 * I : op == BWD1 ? I : H;
  const int K = op == FWD1 || op == BWD1 ? H : op == FWD2 ? I : 2 * I;
  const double groups = (double)std::min<int64_t>(s.E + s.R - 1, s.A);
  const double weights_us = groups * N * K * 2 / 6e6;
  // us of a step where a workgroup has its CU alone, and where the CU, or the chip, is full
  auto us = [&](int bp, int bq, int wgs, double alone, double full) {
    const double tiles = std::max(groups, (double)s.A / bq + groups / 2) * ((N + bp - 1) / bp);
    const double r = tiles / wgs, rounds = r <= 1 ? 1 : r < 4 ? std::ceil(r) : r + 0.5;
    const double t = rounds * ((K + BK - 1) / BK + 4.3) * (tiles <= kCus ? alone : full);
    return std::max(t, weights_us) + 0.24 * t;
  };
  const double large = us(256, 256, kCus, 1.22, 1.31), tall = us(256, 128, kCus, 0.71, 0.81);
  const double medium = us(128, 64, 2 * kCus, 0.43, 0.62), small = us(128, 32, 2 * kCus, 0.37, 0.48);
  const double least = std::min(std::min(large, tall), std::min(medium, small));
  return large == least ? LARGE : tall == least ? TALL : medium == least ? MEDIUM : SMALL;
}

template <int OP>
hipError_t launch_rows(const FfnArgs& a, hipStream_t st) {
  switch (rows_tile(OP, a.s, a.H, a.I)) {
    case LARGE: return launch_rows_as<OP, Large>(a, 1, st);
    case TALL: return launch_rows_as<OP, Tall>(a, 1, st);
    case MEDIUM: return launch_rows_as<OP, Medium>(a, 2, st);
    default: return launch_rows_as<OP, Small>(a, 2, st);
  }
}

template <class G, bool NT>
hipError_t launch_grad_as(const GradArgs& a, int per_cu, hipStream_t st) {
  hipLaunchKernelGGL((grad_kernel<G, NT>), dim3(per_cu * kCus), dim3(64 * G::NW), 0, st, a);
  return hipGetLastError();
}

// Which tile: the largest that still gives the CUs work.  Measured on MI355X, us, by 256x256
// tiles of the targets (256x256, 128x128, 128x64, the latter two with two workgroups to a CU):
//    36: 51.7, 38.1, 30.1     66: 55.6, 37.4, 29.4     84: 23.2, 17.2, 16.9    144: 103.6, 64.2, 83.7
//   142: 18.4, 12.9, 14.7    228: 26.5, 28.6, 33.8    336: 44.3, 44.9, 50.6    912: 57.9, 62.7, 76.7
Tile grad_tile(const moonep_sizes& s, int H, int I) {
  auto of = [](int64_t n) { return (n + 255) / 256; };
  const int64_t targets = s.E + std::min<int64_t>(s.R - 1, (int64_t)s.R * s.slots);
  const int64_t tiles = targets * (of(H) * of(2 * I) + of(I) * of(H));
  return tiles <= kCus / 3 ? MEDIUM : tiles <= kCus * 5 / 8 ? SQUARE : LARGE;
}

// Whether the gradients pass the caches by: 256x256 tiles only (see grad_kernel).
bool grad_passes_caches(const moonep_sizes& s, int H, int I) {
  return grad_tile(s, H, I) == LARGE && (int64_t)s.E * 12 * I * H > kLastLevelCacheBytes;
}

hipError_t launch_grad(const GradArgs& a, hipStream_t st) {
  switch (grad_tile(a.s, a.H, a.I)) {
    case MEDIUM: return launch_grad_as<Medium, false>(a, 2, st);
    case SQUARE: return launch_grad_as<Square, false>(a, 2, st);
    default: break;
  }
  return grad_passes_caches(a.s, a.H, a.I) ? launch_grad_as<Large, true>(a, 1, st)
                                           : launch_grad_as<Large, false>(a, 1, st);
}

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

int check_ffn(const moonep_plan_desc* d, int H, int I) {
  const int rc = check_desc(d);
  if (rc != MOONEP_OK) return rc;
  if (H <= 0 || H % 8 != 0 || I <= 0 || I % 8 != 0) return MOONEP_EINVAL;
  if (H > MOONEP_MAX_FFN || I > MOONEP_MAX_FFN) return MOONEP_ELIMIT;
  // an expert's up rows are addressed from its gate rows, with a tile to spare, in 31 bits
  if ((int64_t)(I + 256) * H * 2 > INT32_MAX) return MOONEP_ELIMIT;
  // tiles are counted in 32 bits, for the smallest tile
  const int64_t mt = d->sz.A / 32 + d->sz.E + d->sz.P_max;
  if (mt * ((std::max(H, I) + 63) / 64) > INT32_MAX) return MOONEP_ELIMIT;
  return MOONEP_OK;
}

// Tiles of other columns still read the rows of one that is done, and other workgroups the weights:
// an output that overlapped either would change what they read.  All are known to be aligned.
Span plan_span(const moonep_plan_desc* d) { return span(d->dev, 1, d->sz.plan_bytes); }
Span rows_span(const moonep_plan_desc* d, const uint16_t* p, int n) { return span(p, d->sz.recv_rows, 2ll * n); }
Span home_span(const moonep_plan_desc* d, const void* p, int64_t pitch, int H, int I, int elem_bytes) {
  return slabs(p, d->sz.E, pitch, 3ll * I * H, elem_bytes);
}
Span slot_span(const moonep_plan_desc* d, const void* p, int64_t pitch, int H, int I, int elem_bytes) {
  return slabs(p, (int64_t)d->sz.R * d->sz.slots, pitch, 3ll * I * H, elem_bytes);
}

}  // namespace
}  // namespace moonep

using namespace moonep;

extern "C" {

int moonep_expert_tile(const moonep_plan_desc* plan, int H, int I, int product, int32_t tile[3]) {
  const int rc = check_ffn(plan, H, I);
  if (rc != MOONEP_OK) return rc;
  if (!tile || product < MOONEP_PRODUCT_GATE_UP || product > MOONEP_PRODUCT_G_WEIGHTS) return MOONEP_EINVAL;
  static_assert(FWD1 == MOONEP_PRODUCT_GATE_UP && FWD2 == MOONEP_PRODUCT_DOWN && BWD1 == MOONEP_PRODUCT_G_GATE_UP &&
                BWD2 == MOONEP_PRODUCT_G_ROWS);
  const bool grad = product == MOONEP_PRODUCT_G_WEIGHTS;
  const Tile t = grad ? grad_tile(plan->sz, H, I) : rows_tile(product, plan->sz, H, I);
  tile[0] = t == LARGE || t == TALL ? 256 : 128;
  tile[1] = t == LARGE ? 256 : t == MEDIUM ? 64 : t == SMALL ? 32 : 128;
  tile[2] = grad && grad_passes_caches(plan->sz, H, I);
  return MOONEP_OK;
}

int moonep_expert_ffn(const moonep_plan_desc* plan, const uint16_t* recv, int H, int I, int act,
                      const uint16_t* home_w, const uint16_t* slot_w, int64_t W_el, uint16_t* gu,
                      uint16_t* h, uint16_t* y, hipStream_t stream) {
  const int rc = check_ffn(plan, H, I);
  if (rc != MOONEP_OK) return rc;
  if (!recv || !home_w || !h || !y || (plan->sz.slots > 0 && !slot_w)) return MOONEP_EINVAL;
  if (W_el < 3ll * I * H || W_el % 8 != 0 || (act != MOONEP_ACT_SILU && act != MOONEP_ACT_GELU))
    return MOONEP_EINVAL;
  if (!aligned(recv, 16) || !aligned(home_w, 16) || !aligned(slot_w, 16) || !aligned(gu, 16) ||
      !aligned(h, 16) || !aligned(y, 16))
    return MOONEP_EALIGN;
  const Span pl = plan_span(plan), x = rows_span(plan, recv, H), hw = home_span(plan, home_w, W_el, H, I, 2),
             sw = slot_span(plan, slot_w, W_el, H, I, 2);
  const Span go = rows_span(plan, gu, 2 * I), ho = rows_span(plan, h, I), yo = rows_span(plan, y, H);
  if (overlap(go, {pl, x, hw, sw, ho, yo}) || overlap(ho, {pl, x, hw, sw, yo}) || overlap(yo, {pl, x, hw, sw}))
    return MOONEP_EINVAL;
  FfnArgs a{};
  a.plan = static_cast<const int32_t*>(plan->dev);
  a.s = plan->sz;
  a.H = H; a.I = I; a.act = act;
  a.home_w = home_w; a.slot_w = slot_w; a.W_el = W_el;
  a.in = recv; a.out = h; a.gu_out = gu;
  (void)hipGetLastError();
  if (launch_rows<FWD1>(a, stream) != hipSuccess) return MOONEP_EHIP;
  a.in = h; a.out = y; a.gu_out = nullptr;
  return launch_rows<FWD2>(a, stream) == hipSuccess ? MOONEP_OK : MOONEP_EHIP;
}

int moonep_expert_ffn_bwd_data(const moonep_plan_desc* plan, const uint16_t* g_y,
                               const uint16_t* gu, int H, int I, int act, const uint16_t* home_w,
                               const uint16_t* slot_w, int64_t W_el, uint16_t* g_gu,
                               uint16_t* g_recv, hipStream_t stream) {
  const int rc = check_ffn(plan, H, I);
  if (rc != MOONEP_OK) return rc;
  if (!g_y || !gu || !home_w || !g_gu || !g_recv || (plan->sz.slots > 0 && !slot_w))
    return MOONEP_EINVAL;
  if (W_el < 3ll * I * H || W_el % 8 != 0 || (act != MOONEP_ACT_SILU && act != MOONEP_ACT_GELU))
    return MOONEP_EINVAL;
  if (!aligned(g_y, 16) || !aligned(gu, 16) || !aligned(home_w, 16) || !aligned(slot_w, 16) ||
      !aligned(g_gu, 16) || !aligned(g_recv, 16))
    return MOONEP_EALIGN;
  const Span pl = plan_span(plan), gy = rows_span(plan, g_y, H), in = rows_span(plan, gu, 2 * I),
             hw = home_span(plan, home_w, W_el, H, I, 2), sw = slot_span(plan, slot_w, W_el, H, I, 2);
  const Span go = rows_span(plan, g_gu, 2 * I), ro = rows_span(plan, g_recv, H);
  if (overlap(go, {pl, gy, hw, sw, ro}) || (g_gu != gu && overlap(go, in)) || overlap(ro, {pl, gy, in, hw, sw}))
    return MOONEP_EINVAL;
  FfnArgs a{};
  a.plan = static_cast<const int32_t*>(plan->dev);
  a.s = plan->sz;
  a.H = H; a.I = I; a.act = act;
  a.home_w = home_w; a.slot_w = slot_w; a.W_el = W_el;
  a.in = g_y; a.gu_in = gu; a.out = g_gu;
  (void)hipGetLastError();
  if (launch_rows<BWD1>(a, stream) != hipSuccess) return MOONEP_EHIP;
  a.in = g_gu; a.gu_in = nullptr; a.out = g_recv;
  return launch_rows<BWD2>(a, stream) == hipSuccess ? MOONEP_OK : MOONEP_EHIP;
}

int moonep_expert_ffn_bwd_weight(const moonep_plan_desc* plan, const uint16_t* recv,
                                 const uint16_t* g_y, const uint16_t* h, const uint16_t* g_gu,
                                 int H, int I, float* home_grad, float* rep_grad, int64_t G_el,
                                 int accumulate, hipStream_t stream) {
  const int rc = check_ffn(plan, H, I);
  if (rc != MOONEP_OK) return rc;
  if (!recv || !g_y || !h || !g_gu || !home_grad || (plan->sz.slots > 0 && !rep_grad))
    return MOONEP_EINVAL;
  if (G_el < 3ll * I * H || G_el % 4 != 0 || (accumulate != 0 && accumulate != 1))
    return MOONEP_EINVAL;
  if (!aligned(recv, 16) || !aligned(g_y, 16) || !aligned(h, 16) || !aligned(g_gu, 16) ||
      !aligned(home_grad, 16) || !aligned(rep_grad, 16))
    return MOONEP_EALIGN;
  const Span pl = plan_span(plan), x = rows_span(plan, recv, H), gy = rows_span(plan, g_y, H),
             hh = rows_span(plan, h, I), gg = rows_span(plan, g_gu, 2 * I);
  const Span ho = home_span(plan, home_grad, G_el, H, I, 4), ro = slot_span(plan, rep_grad, G_el, H, I, 4);
  if (overlap(ho, {pl, x, gy, hh, gg, ro}) || overlap(ro, {pl, x, gy, hh, gg})) return MOONEP_EINVAL;
  GradArgs a{};
  a.plan = static_cast<const int32_t*>(plan->dev);
  a.s = plan->sz;
  a.H = H; a.I = I; a.accumulate = accumulate;
  a.recv = recv; a.g_y = g_y; a.h = h; a.g_gu = g_gu;
  a.home = home_grad; a.rep = rep_grad; a.G_el = G_el;
  (void)hipGetLastError();
  return launch_grad(a, stream) == hipSuccess ? MOONEP_OK : MOONEP_EHIP;
}

}  // extern "C"
