// The gated feed-forward experts on the planned buffer: grouped matrix products over the
// plan's groups, forward and backward.
//
//   forward        gate = x Wg^T, up = x Wu^T, h = act(gate) * up     (one kernel)
//                  y = h Wd^T
//   rows' gradient g_h = g_y Wd, g_gate = g_h * up * act'(gate), g_up = g_h * act(gate)
//                  g_recv = g_gate Wg + g_up Wu
//   weights'       g_Wg = g_gate^T x, g_Wu = g_up^T x, g_Wd = g_y^T h
//
// Every product is D[p, q] = sum_k P[p, k] * Q[q, k] with v_mfma_f32_16x16x32_bf16: P, the
// side whose index runs along the output's rows in memory, is the instruction's first
// operand, so a lane's four results are consecutive there.
#include <type_traits>

#include "moonep_internal.h"

namespace moonep {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

#define LDS __attribute__((address_space(3)))

constexpr int kBK = 64;                    // k elements of a step: 128 bytes, a cache line
constexpr int kMaxSegs = 2 * MOONEP_MAX_E + MOONEP_MAX_R;
constexpr uint32_t kOob = 0x80000000u;     // a buffer offset past every range: reads as zero
constexpr int kBufferFlags = 0x00020000;   // raw buffer of 32-bit data
constexpr int kCus = 256;

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
__device__ __forceinline__ Seg load_seg(const int32_t* plan, const moonep_sizes& s, int i, int np) {
  Seg g{0, 0, 0};
  if (i < s.E) {
    g.n = plan[s.o_keep + i];
    g.row0 = plan[s.o_home_row + i];
    g.w = i;
  } else if (i - s.E < np) {
    const int32_t* pc = plan + s.o_pieces + (int64_t)(i - s.E) * kPieceInts;
    const int e = pc[P_E], r = pc[P_R], slot = pc[P_SLOT];
    g.n = pc[P_CNT];
    g.row0 = pc[P_ROW0];
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

__device__ __forceinline__ int piece_count(const int32_t* plan, const moonep_sizes& s) {
  if (plan[s.o_hdr + H_STATUS] != 0) return 0;
  return min(max(plan[s.o_hdr + H_NPIECES], 0), s.P_max);
}

// 16 bytes a lane from the buffer straight into LDS, to `to` + OFF + lane * 16.  In assembly:
// for the builtin the compiler waits for every such load before any LDS read that it cannot
// tell apart from it, which here is each one, and the next steps' loads would never be in
// flight during this step's products.  No register is written, so there is none to wait
// for; arrive() is the wait.  (m0 holds the LDS address; gfx9 wants one instruction
// between writing it and the load.)
template <int OFF>
__device__ __forceinline__ void load_lds(i32x4 rsrc, uint32_t voff, uint32_t to) {
  asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :: "s"(to), "v"(voff), "s"(rsrc), "i"(OFF) : "memory", "scc");
}

// ---------------------------------------------------------------------------------------
// operand tiles in LDS
// ---------------------------------------------------------------------------------------
// A step's tile holds kBK k of R rows (of P or Q).  Two forms:
//   KC  memory is contiguous along k: LDS rows of 64 k (128 bytes), the 16-byte chunk c of
//       row r at chunk c ^ (r & 7): the 16 lanes that read at once hit different banks;
//   KS  memory is contiguous along the row index: LDS rows (one per k) of R elements, the
//       32-byte unit u of row k at u ^ (k & 3 | (k >> 3 & 1) << 2), read transposed.
// Both are filled by 16-byte loads straight into LDS; the swizzle is in each lane's
// global address, since a wave's load fills 1024 consecutive LDS bytes.

template <int R, bool KS, int NW>
struct Operand {
  static constexpr int kBytes = R * kBK * 2;
  static constexpr int kLoads = kBytes / 1024 / NW;
  static_assert(kLoads >= 1 && kLoads * 1024 * NW == kBytes);
  uint32_t voff[kLoads];
  int kc;                        // KC: this lane's first k inside a step
  // the next step to load: its address and the k left from there (uniform)
  const char* at;
  int left;
  uint32_t ld;                   // bytes of a row in memory
  uint32_t skip;                 // KS: bytes of the row before `at`
  i32x4 rs;

  // KC: rowoff(r) is the byte offset of LDS row r in memory, or kOob
  template <class F>
  __device__ __forceinline__ void init_kc(int wave, int lane, F rowoff) {
    const int c = (lane & 7) ^ (lane >> 3);
    kc = c * 8;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) voff[i] = rowoff((i * NW + wave) * 8 + (lane >> 3)) + c * 16;
  }
  // KS: columns at or past ncols read as zero
  __device__ __forceinline__ void init_ks(int wave, int lane, int ncols) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int b = (i * NW + wave) * 1024 + lane * 16;
      const int k = b / (R * 2), cp = b % (R * 2) / 16;
      const int u = (cp >> 1) ^ ((k & 3) | ((k >> 3 & 1) << 2));
      const int c = u * 2 + (cp & 1);
      voff[i] = c * 8 < ncols ? k * ld + c * 16 : kOob;
    }
  }
  // Makes the buffer descriptor of the next step and moves on.  Past the end everything is
  // out of range, and the tile is filled with zeros.
  __device__ __forceinline__ void next() {
    const uint64_t p = reinterpret_cast<uint64_t>(at);
    const int rows = max(min(left, kBK), 0);
    const int range = !KS ? 0x7fffffff : rows ? rows * (int)ld - (int)skip : 0;
    rs = i32x4{(int)p, (int)(p >> 32) & 0xFFFF, range, kBufferFlags};
    if (!KS && left < kBK) {     // the last k, or none
#pragma unroll
      for (int i = 0; i < kLoads; ++i) voff[i] |= kc >= left ? kOob : 0;
    }
    at += KS ? (uint64_t)ld * kBK : kBK * 2;
    left -= kBK;
  }
  // load I of the step
  template <int I, int OFF>
  __device__ __forceinline__ void load(uint32_t to) const {
    load_lds<I * NW * 1024 + OFF>(rs, voff[I], to);
  }
};

// Fragment f (16 rows from row0 on), k from kk * 32 on, of a tile.
template <int R, bool KS>
__device__ __forceinline__ bf16x8 fragment(const char* tile, int row0, int f, int kk, int lane) {
  if constexpr (!KS) {
    const int a = (lane & 15) * 128 + (((lane >> 4) ^ (lane & 7)) << 4);
    return *reinterpret_cast<const bf16x8*>(tile + row0 * 128 + (a ^ (kk << 6)) + f * 2048);
  } else {
    const int g = lane >> 4, j = (lane & 15) >> 2;
    const int sw = j | ((g & 1) << 2);
    const int a = (g * 8 + j) * (R * 2) + (((row0 / 16 + f) ^ sw) << 5) + (lane & 3) * 8 + kk * 64 * R;
    union { s16x4 h[2]; bf16x8 v; } u;
    u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS s16x4*)(tile + a));
    u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS s16x4*)(tile + a + 4 * R * 2));
    return u.v;
  }
}

// Inside a block of 32 rows of a KC operand P, LDS row f*16 + g*4 + i holds row
// g*8 + f*4 + i: a lane's results of two fragments are then 8 consecutive ones.
__device__ __forceinline__ int p_perm(int r) {
  return (r & ~31) | ((r >> 2 & 3) << 3) | ((r >> 4 & 1) << 2) | (r & 3);
}

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

template <int N, class F>
__device__ __forceinline__ void times(F f) {
  if constexpr (N > 0) {
    times<N - 1>(f);
    f(std::integral_constant<int, N - 1>{});
  }
}

// The products of a tile, `nk` steps; before_next() runs before a step's loads are made.
// Two steps' tiles are in LDS.  Each step is two matrix instructions deep: while its first
// half is multiplied out of registers, the second is read from LDS into others; then
// every wave has read the whole tile, and while the second half is multiplied, the first
// half of the next step, whose loads went out a step ago, is read, and the step after
// that starts to load over the tile just read.  One barrier a step.  Each half is cut into parts that
// start a share of the loads, then spread a share of the LDS reads among their matrix
// instructions.
template <int BP, int BQ, bool KSP, bool KSQ, int NW, int PF, int QF, class F>
__device__ __forceinline__ void products(char* smem, int nk, int wave, int p0, int q0, int lane,
                                         f32x4 (&acc)[PF][QF], Operand<BP, KSP, NW>& P,
                                         Operand<BQ, KSQ, NW>& Q, F before_next) {
  using OpP = Operand<BP, KSP, NW>;
  using OpQ = Operand<BQ, KSQ, NW>;
  constexpr int kStep = OpP::kBytes + OpQ::kBytes, kL = OpP::kLoads + OpQ::kLoads;
  constexpr int kParts = QF >= 4 ? 4 : QF, kM = PF * QF / kParts, kF = PF + QF;
  static_assert(kL < 64 && QF % kParts == 0);
  const uint32_t lds = uni((int)(uint32_t)(uintptr_t)(LDS char*)smem + wave * 1024);
  bf16x8 a[2][PF], b[2][QF];
  arrive<0>();                    // whatever an earlier tile still had in flight has landed
  times<2>([&](auto i) {
    before_next();
    P.next();
    Q.next();
    times<OpP::kLoads>([&](auto j) { P.template load<j, i * kStep>(lds); });
    times<OpQ::kLoads>([&](auto j) { Q.template load<j, i * kStep + OpP::kBytes>(lds); });
  });
  arrive<kL>();
#pragma unroll
  for (int p = 0; p < PF; ++p) a[0][p] = fragment<BP, KSP>(smem, p0, p, 0, lane);
#pragma unroll
  for (int q = 0; q < QF; ++q) b[0][q] = fragment<BQ, KSQ>(smem + OpP::kBytes, q0, q, 0, lane);
  int cur = 0;
  for (int i = 0; i < nk; ++i) {
    times<2>([&](auto h) {
      if constexpr (h == 1) {
        before_next();
        P.next();
        Q.next();
        arrive<0>();
      }
      const uint32_t to = lds + cur;
      const char* t = smem + (h ? cur ^ kStep : cur);
      times<kParts>([&](auto c) {
        times<kL>([&](auto j) {
          if constexpr (h == 1 && j * kParts / kL == c) {
            if constexpr (j < OpP::kLoads) P.template load<j, 0>(to);
            else Q.template load<j - OpP::kLoads, OpP::kBytes>(to);
          }
        });
        times<kF>([&](auto f) {
          if constexpr (f * kParts / kF == c) {
            if constexpr (f < PF) a[h ^ 1][f] = fragment<BP, KSP>(t, p0, f, h ^ 1, lane);
            else b[h ^ 1][f - PF] = fragment<BQ, KSQ>(t + OpP::kBytes, q0, f - PF, h ^ 1, lane);
          }
        });
        times<kM>([&](auto m) {
          constexpr int p = m % PF, q = c * (QF / kParts) + m / PF;
          acc[p][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[h][p], b[h][q], acc[p][q], 0, 0, 0);
        });
        times<kM>([&](auto) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        });
        __builtin_amdgcn_sched_barrier(0);
      });
    });
    cur ^= kStep;
  }
}

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
// 1 in fp32 and u' would overflow, so u is taken of z cut to that range.
__device__ __forceinline__ float act_of(float z, int act, float* slope) {
  if (act == MOONEP_ACT_SILU) {
    const float s = 1.f / (1.f + __expf(-z));
    *slope = s + z * s * (1.f - s);
    return z * s;
  }
  const float c = 0.7978845608028654f;
  const float zc = fminf(fmaxf(z, -16.f), 16.f);
  const float z2 = zc * zc;
  const float p = 1.f / (1.f + __expf(-2.f * c * (zc + 0.044715f * zc * z2)));
  *slope = p + 2.f * zc * p * (1.f - p) * c * (1.f + 0.134145f * z2);
  return z * p;
}

// ---------------------------------------------------------------------------------------
// the row products: forward, and the rows' gradient
// ---------------------------------------------------------------------------------------

template <int OP, int BP, int BQ, int WP, int WQ>
__global__ __launch_bounds__(64 * WP * WQ, 1) void rows_kernel(const FfnArgs a) {
#ifdef __HIP_DEVICE_COMPILE__   // gfx950 builtins: the host pass needs the kernel's name only
  constexpr int NW = WP * WQ, PF = BP / WP / 16, QF = BQ / WQ / 16;
  constexpr bool KSP = OP == BWD1 || OP == BWD2;
  constexpr bool PAIR = OP == FWD1;            // P's rows are gate and up rows in turn
  using OpP = Operand<BP, KSP, NW>;
  using OpQ = Operand<BQ, false, NW>;
  __shared__ __align__(1024) char smem[2 * (OpP::kBytes + OpQ::kBytes)];
  __shared__ int pre[kMaxSegs];
  __shared__ int wsum[NW];

  const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
  const int wp = wave % WP, wq = wave / WP;
  const int32_t* plan = a.plan;
  const int np = uni(piece_count(plan, a.s));
  const bool valid = uni(plan[a.s.o_hdr + H_STATUS]) == 0;
  const int nseg = valid ? a.s.E + np : 0;

  // inclusive sums of the segments' row tiles
  {
    constexpr int PER = (kMaxSegs + 64 * NW - 1) / (64 * NW);
    int cnt[PER], sum = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int i = tid * PER + j;
      cnt[j] = 0;
      if (i < nseg) cnt[j] = (load_seg(plan, a.s, i, np).n + BQ - 1) / BQ;
      sum += cnt[j];
    }
    int inc = sum;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int o = __shfl_up(inc, d);
      if (lane >= d) inc += o;
    }
    if (lane == 63) wsum[wave] = inc;
    __syncthreads();
    int before = inc - sum;
    for (int w = 0; w < wave; ++w) before += wsum[w];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int i = tid * PER + j;
      before += cnt[j];
      if (i < nseg) pre[i] = before;
    }
    __syncthreads();
  }
  const int K = OP == FWD1 || OP == BWD1 ? a.H : OP == FWD2 ? a.I : 2 * a.I;
  const int N = OP == FWD1 || OP == BWD1 ? a.I : a.H;          // output columns
  constexpr int BN = PAIR ? BP / 2 : BP;
  const int nt = (N + BN - 1) / BN;
  const int mt_all = nseg ? min(uni(pre[nseg - 1]), a.tiles_bound) : 0;
  const int tiles = mt_all * nt;
  const int nk = (K + kBK - 1) / kBK;

  for (int round = 0; round * (int)gridDim.x < tiles; ++round) {
    const int t = tile_of(round, blockIdx.x, gridDim.x);
    if (t >= tiles) continue;
    // the segment of tile t: the first whose sum of tiles exceeds t / nt
    int sl = 0, sh = nseg - 1;
    const int want = t / nt;
    while (sl < sh) {
      const int mid = (sl + sh) / 2;
      if (pre[mid] > want) sh = mid; else sl = mid + 1;
    }
    sl = uni(sl);
    const Seg g0 = load_seg(plan, a.s, sl, np);
    const int row0 = uni(g0.row0), n = uni(g0.n), w = uni(g0.w);
    const int mt = (n + BQ - 1) / BQ;
    const int local = t - (uni(pre[sl]) - mt) * nt;
    if (local < 0 || local >= mt * nt) continue;
    int tm, tn;
    band(local, mt, nt, &tm, &tn);
    const int q0 = tm * BQ, nq = n - q0;                        // rows of this tile
    const uint16_t* W = w < a.s.E ? a.home_w + w * a.W_el : a.slot_w + (w - a.s.E) * a.W_el;
    if (OP == FWD2 || OP == BWD1) W += 2ll * a.I * a.H;
    const int n0 = tn * BN;

    OpP P;
    OpQ Q;
    P.left = Q.left = K;
    if constexpr (!KSP) {
      P.ld = K * 2;
      P.skip = 0;
      P.at = reinterpret_cast<const char*>(W) + (int64_t)n0 * P.ld;
      P.init_kc(wave, lane, [&](int r) -> uint32_t {
        if (PAIR) {
          const int c = (r >> 6) * 32 + p_perm(r & 31);
          return n0 + c < N ? (uint32_t)(c + (r >> 5 & 1) * a.I) * P.ld : kOob;
        }
        const int c = p_perm(r);
        return n0 + c < N ? (uint32_t)c * P.ld : kOob;
      });
    } else {
      P.ld = N * 2;
      P.skip = n0 * 2;
      P.at = reinterpret_cast<const char*>(W) + P.skip;
      P.init_ks(wave, lane, N - n0);
    }
    Q.ld = K * 2;
    Q.skip = 0;
    Q.at = reinterpret_cast<const char*>(a.in) + (int64_t)(row0 + q0) * Q.ld;
    Q.init_kc(wave, lane, [&](int r) -> uint32_t { return r < nq ? r * Q.ld : kOob; });

    f32x4 acc[PF][QF];
    clear(acc);
    products<BP, BQ, KSP, false, NW>(smem, nk, wave, wp * PF * 16, wq * QF * 16, lane, acc, P, Q, [] {});

    const int g = lane >> 4;
#pragma unroll
    for (int q = 0; q < QF; ++q) {
      const int r = wq * QF * 16 + q * 16 + (lane & 15);
      if (r >= nq) continue;
      const int64_t row = row0 + q0 + r;
      if constexpr (OP == FWD1) {
#pragma unroll
        for (int pb4 = 0; pb4 < PF; pb4 += 4) {
          const int c = n0 + (wp * PF + pb4) * 8 + g * 8;       // 64 P rows give 32 columns
          if (c >= N) continue;
          u32x4 h, vg, vu;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int f = e >> 1, i = (e & 1) * 2;
            const float g0 = acc[pb4 + f][q][i], g1 = acc[pb4 + f][q][i + 1];
            const float u0 = acc[pb4 + 2 + f][q][i], u1 = acc[pb4 + 2 + f][q][i + 1];
            float sl0, sl1;
            h[e] = bf2(act_of(g0, a.act, &sl0) * u0, act_of(g1, a.act, &sl1) * u1);
            vg[e] = bf2(g0, g1);
            vu[e] = bf2(u0, u1);
          }
          *reinterpret_cast<u32x4*>(a.out + row * N + c) = h;
          if (a.gu_out) {
            *reinterpret_cast<u32x4*>(a.gu_out + row * 2 * N + c) = vg;
            *reinterpret_cast<u32x4*>(a.gu_out + row * 2 * N + N + c) = vu;
          }
        }
      } else if constexpr (OP == FWD2) {
#pragma unroll
        for (int p = 0; p < PF; p += 2) {
          const int c = n0 + (wp * PF + p) * 16 + g * 8;
          if (c >= N) continue;
          u32x4 v;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[e] = bf2(acc[p + (e >> 1)][q][(e & 1) * 2], acc[p + (e >> 1)][q][(e & 1) * 2 + 1]);
          *reinterpret_cast<u32x4*>(a.out + row * N + c) = v;
        }
      } else {
#pragma unroll
        for (int p = 0; p < PF; ++p) {
          const int c = n0 + (wp * PF + p) * 16 + g * 4;
          if (c >= N) continue;
          const f32x4 d = acc[p][q];
          if constexpr (OP == BWD2) {
            *reinterpret_cast<u32x2*>(a.out + row * N + c) = u32x2{bf2(d[0], d[1]), bf2(d[2], d[3])};
          } else {
            const u32x2 vg = *reinterpret_cast<const u32x2*>(a.gu_in + row * 2 * N + c);
            const u32x2 vu = *reinterpret_cast<const u32x2*>(a.gu_in + row * 2 * N + N + c);
            float gg[4], gu[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float z = i & 1 ? hi(vg[i >> 1]) : lo(vg[i >> 1]);
              const float u = i & 1 ? hi(vu[i >> 1]) : lo(vu[i >> 1]);
              float slope;
              gu[i] = d[i] * act_of(z, a.act, &slope);
              gg[i] = d[i] * u * slope;
            }
            *reinterpret_cast<u32x2*>(a.out + row * 2 * N + c) = u32x2{bf2(gg[0], gg[1]), bf2(gg[2], gg[3])};
            *reinterpret_cast<u32x2*>(a.out + row * 2 * N + N + c) = u32x2{bf2(gu[0], gu[1]), bf2(gu[2], gu[3])};
          }
        }
      }
    }
  }
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

template <int BP, int BQ, int WP, int WQ>
__global__ __launch_bounds__(64 * WP * WQ, 1) void grad_kernel(const GradArgs a) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int NW = WP * WQ, PF = BP / WP / 16, QF = BQ / WQ / 16;
  using OpP = Operand<BP, true, NW>;
  using OpQ = Operand<BQ, true, NW>;
  __shared__ __align__(1024) char smem[2 * (OpP::kBytes + OpQ::kBytes)];
  const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
  const int wp = wave % WP, wq = wave / WP;
  const int32_t* plan = a.plan;
  const moonep_sizes& s = a.s;
  const int np = uni(piece_count(plan, s));
  const bool valid = uni(plan[s.o_hdr + H_STATUS]) == 0;
  const int p1 = (a.H + BP - 1) / BP, q1 = (2 * a.I + BQ - 1) / BQ;      // gate and up
  const int p2 = (a.I + BP - 1) / BP, q2 = (a.H + BQ - 1) / BQ;          // down
  const int per = p1 * q1 + p2 * q2;
  const int tiles = (s.E + np) * per;

  for (int round = 0; round * (int)gridDim.x < tiles; ++round) {
    const int t = tile_of(round, blockIdx.x, gridDim.x);
    if (t >= tiles) continue;
    const int target = t / per;
    int local = t - target * per;
    Seg seg = load_seg(plan, s, target, np);
    int q = 0, qend = 0;                              // the fallback pieces of a home expert
    float* out;
    if (target < s.E) {
      if (!valid) seg.n = 0;
      if (np) {
        q = min(max(plan[s.o_pfirst + target], 0), np);
        qend = q + min(max(plan[s.o_pnum + target], 0), np - q);
      }
      out = a.home + target * a.G_el;
    } else {
      if (seg.n == 0 || seg.w < s.E) continue;        // a fallback piece: in its home's sum
      out = a.rep + (seg.w - s.E) * a.G_el;
    }
    const bool down = local >= p1 * q1;
    if (down) local -= p1 * q1;
    int tq, tp;
    band(local, down ? q2 : q1, down ? p2 : p1, &tq, &tp);
    const int p0 = tp * BP, q0 = tq * BQ;
    const int np_cols = down ? a.I : a.H, nq_cols = down ? a.H : 2 * a.I;
    const char* psrc = reinterpret_cast<const char*>(down ? a.h : a.recv);
    const char* qsrc = reinterpret_cast<const char*>(down ? a.g_y : a.g_gu);
    if (down) out += 2ll * a.I * a.H;

    OpP P;
    OpQ Q;
    P.ld = np_cols * 2;
    Q.ld = nq_cols * 2;
    P.skip = p0 * 2;
    Q.skip = q0 * 2;
    P.init_ks(wave, lane, np_cols - p0);
    Q.init_ks(wave, lane, nq_cols - q0);
    auto start = [&](int row, int n) {
      P.at = psrc + (int64_t)row * P.ld + P.skip;
      Q.at = qsrc + (int64_t)row * Q.ld + Q.skip;
      P.left = Q.left = n;
    };
    q = uni(q);
    qend = uni(qend);
    // the steps of the home group and of the fallback pieces
    start(uni(seg.row0), uni(seg.n));
    int steps = (P.left + kBK - 1) / kBK;
    for (int f = q; f < qend; ++f) {
      const Seg fb = load_seg(plan, s, s.E + f, np);
      if (uni(fb.w) == target) steps += (uni(fb.n) + kBK - 1) / kBK;
    }
    if (steps == 0 && a.accumulate) continue;
    f32x4 acc[PF][QF];
    clear(acc);
    if (steps)
      products<BP, BQ, true, true, NW>(smem, steps, wave, wp * PF * 16, wq * QF * 16, lane, acc, P, Q, [&] {
        while (P.left <= 0 && q < qend) {          // on to the next piece with rows
          const Seg fb = load_seg(plan, s, s.E + q, np);
          ++q;
          if (uni(fb.w) == target && uni(fb.n) > 0) start(uni(fb.row0), uni(fb.n));
          // here, and not at some later use on the common path, where it would drain the ring
          __builtin_amdgcn_s_waitcnt(wait_vm_lds(0));
        }
      });

#pragma unroll
    for (int f = 0; f < QF; ++f) {
      const int r = q0 + (wq * QF + f) * 16 + (lane & 15);
      if (r >= nq_cols) continue;
#pragma unroll
      for (int p = 0; p < PF; ++p) {
        const int c = p0 + (wp * PF + p) * 16 + (lane >> 4) * 4;
        if (c >= np_cols) continue;
        f32x4* o = reinterpret_cast<f32x4*>(out + (int64_t)r * np_cols + c);
        *o = a.accumulate && target < s.E ? *o + acc[p][f] : acc[p][f];
      }
    }
  }
#endif
}

template <int OP>
hipError_t launch_rows(FfnArgs a, hipStream_t st) {
  constexpr int BP = 256, BQ = 256;
  const int64_t segs = std::min<int64_t>(a.s.E + a.s.P_max, a.s.A);
  const int64_t mt = a.s.A / BQ + segs;
  const int N = OP == FWD1 || OP == BWD1 ? a.I : a.H;
  constexpr int BN = OP == FWD1 ? BP / 2 : BP;
  const int64_t tiles = mt * ((N + BN - 1) / BN);
  a.tiles_bound = (int)mt;
  const int grid = (int)std::min<int64_t>((tiles + 7) / 8 * 8, kCus);
  hipLaunchKernelGGL((rows_kernel<OP, BP, BQ, 4, 2>), dim3(grid), dim3(512), 0, st, a);
  return hipGetLastError();
}

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

int check_ffn(const moonep_plan_desc* d, int H, int I) {
  const int rc = check_desc(d);
  if (rc != MOONEP_OK) return rc;
  if (H <= 0 || H % 8 != 0 || I <= 0 || I % 8 != 0) return MOONEP_EINVAL;
  if (H > MOONEP_MAX_FFN || I > MOONEP_MAX_FFN) return MOONEP_ELIMIT;
  // tiles are counted in 32 bits, for the smallest tile
  const int64_t mt = d->sz.A / 32 + d->sz.E + d->sz.P_max;
  if (mt * ((std::max(H, I) + 63) / 64) > INT32_MAX) return MOONEP_ELIMIT;
  return MOONEP_OK;
}

}  // namespace
}  // namespace moonep

using namespace moonep;

extern "C" {

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
  GradArgs a{};
  a.plan = static_cast<const int32_t*>(plan->dev);
  a.s = plan->sz;
  a.H = H; a.I = I; a.accumulate = accumulate;
  a.recv = recv; a.g_y = g_y; a.h = h; a.g_gu = g_gu;
  a.home = home_grad; a.rep = rep_grad; a.G_el = G_el;
  (void)hipGetLastError();
  hipLaunchKernelGGL((grad_kernel<256, 256, 4, 2>), dim3(kCus), dim3(512), 0, stream, a);
  return hipGetLastError() == hipSuccess ? MOONEP_OK : MOONEP_EHIP;
}

}  // extern "C"
