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
#include "moonep_expert.h"

namespace moonep {
namespace {

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
  const int K = OP == FWD1 || OP == BWD1 ? a.H : OP == FWD2 ? a.I : 2 * a.I;
  const int N = OP == FWD1 || OP == BWD1 ? a.I : a.H;
  const int nk = max((K + BK - 1) / BK, G::NB);      // P loads NB steps ahead, into one more tile only
  RowTiles<BQ> queue(plan, a.s, lane, (N + BN - 1) / BN, a.tiles_bound);
  using Tile = typename RowTiles<BQ>::Tile;
  queue.look_up(0, true);

  Tiles pipe(smem, wave, lane);
  auto& P = pipe.P;
  auto& Q = pipe.Q;
  auto start_p = [&](const Tile& t) {
    const uint16_t* W = t.w < a.s.E ? a.home_w + t.w * a.W_el : a.slot_w + (t.w - a.s.E) * a.W_el;
    if (OP == FWD2 || OP == BWD1) W += 2ll * a.I * a.H;
    const int n0 = t.tn * BN;
    P.left = K;
    P.todo = nk;
    if constexpr (!KSP) {
      P.ld = K * 2;
      P.skip = 0;
      P.at = reinterpret_cast<const char*>(W) + (int64_t)n0 * P.ld;
      P.init_kc(wave, here(lane), [&](int r) -> uint32_t {
        const int c = PAIR ? p_row_pair(r) : p_row(r);
        return n0 + c < N ? (uint32_t)(c + (PAIR ? (r >> 5 & 1) * a.I : 0)) * P.ld : kOob;
      });
    } else {
      P.ld = N * 2;
      P.skip = n0 * 2;
      P.at = reinterpret_cast<const char*>(W) + P.skip;
      P.init_ks(wave, here(lane), N - n0);
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

  Tile cur = queue.tile(0), nxt = queue.tile(1);
  if (!cur.rows) return;
  auto more_p = [&] { if (P.todo == 0 && nxt.rows) start_p(nxt); };
  auto more_q = [&] { if (Q.todo == 0 && nxt.rows) start_q(nxt); };
  start_p(cur);
  start_q(cur);
  pipe.begin(more_p, more_q);
  for (int round = 1;; ++round) {
    f32x4 acc[PF][QF];
    clear(acc);
    const int trow = cur.row, tq = cur.rows, tn0 = cur.tn * BN;
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
    nxt = queue.tile(round + 1);
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
