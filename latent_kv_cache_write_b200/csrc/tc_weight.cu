// The attention weight every cached row received, on tcgen05 tensor cores (bf16, d_c = 512,
// d_R = 64 or 512): w(j) += sum over (node, head) rows r of g(r) exp(s(r, j) - lse(r)).
//
// With the log-sum-exps known this is a product S^T = K . Q^T whose epilogue is one exponential
// and one multiply-add per score, summed along the rows.  Keys are the M side (TMEM lanes), rows the
// N side (columns), so a thread owns a key and its sum never leaves the thread.  Nothing of S is
// stored; the sums of a key are joined in one place, without atomics, so the order is fixed.  The
// scores' sums are the tensor cores' float32, which cut what does not fit: of normal values weights come
// out some 1.5e-6 of themselves low (128 heads, 16 nodes, 3000 rows; 1e-7 where the sums are exact).
// Groups of 128 rows whose query weights are all 0 (rejected nodes) are left out.
//
// A CTA pair (cta_group::2) takes 256 keys at a time, 128 per CTA, and 256 rows per MMA, of which
// each CTA loads half: a lone CTA would need 128 rows x 64 dims for every 4 MMAs of M = N = 128,
// 64 B/clk, and an SM's TMA loads deliver about 44.
//   RES_K: the keys' tile (9 boxes of 128 rows x 64 dims, 144 KB) stays in shared memory while the
//          rows stream past it in 4 stages.  A tile of 256 x 256 x 576 takes 6600 to 7200 clk, the
//          rate that cuBLAS's bf16 GEMM reaches here; the rest of a call is the start (plan, first
//          loads) and clusters with fewer units than others.  A pass over 8 trees of up to 16
//          nodes, 128 heads, up to 8100 rows, its inputs new each time: 77 us against a floor of 48.
//   RES_Q: at most 128 rows per sequence (single tokens, small trees): the rows stay and the keys
//          stream, read once from HBM, which bounds it (64 sequences of 8191 rows, one token
//          each: a pass on new inputs 131 us, 110 over and over on the same ones, against a floor
//          of 94; a kernel that only streams them by TMA takes 102).
//   STREAM: d_R = 512 with more rows: 256 KB of keys do not fit, both operands stream.
//
// A cluster has one to four pairs.  It takes whole units (256 keys), and its pairs share the tiles of
// its units evenly: a unit that two or more of them share is summed by the first, which the others
// send their sums through distributed shared memory at the end.
//
// Warp roles (320 threads): warps 0-3 and 4-7 take alternate accumulators (256 columns each, the
// two fill tensor memory), warp 8 loads (each CTA its own halves; the bytes of both complete on
// the even CTA's barriers), warp 9 of the even CTA issues the MMAs.
#include "attend_common.cuh"
#include "launch.h"
#include "tc_ptx.cuh"
#include "tmap.h"

#include <mutex>

namespace mla {
namespace {

using namespace tc;
using namespace attn;

enum { RES_K = 0, RES_Q = 1, STREAM = 2 };

constexpr int WT = 320;                        // threads
constexpr int KEYS = 128;                      // keys per CTA
constexpr int KBOX = KEYS * 64 * 2;            // box of keys: 128 rows x 64 dims
constexpr int MAXCP = 4;                       // pairs per cluster
constexpr unsigned FULL = 0xffffffffu;

// NSL: 64-dim slices of a row (9 or 16).  NT: rows of a tile (N of the MMA), half from each CTA.
template <int NSL, int MODE>
struct WLay {
  static constexpr int NT = MODE == RES_Q ? 128 : 256;
  static constexpr int QBOX = NT / 2 * 64 * 2;
  static constexpr int RBOX = MODE == RES_K ? KBOX : (MODE == RES_Q ? QBOX : 0);
  static constexpr int NRES = MODE == STREAM ? 0 : NSL;               // resident boxes
  static constexpr int SBOX = MODE == RES_K ? QBOX : (MODE == RES_Q ? KBOX : KBOX + QBOX);
  // slices of a stage, stages.  A stage costs the loading and the MMA thread some 500 clk of waits
  // and arrivals whatever it holds: single slices bound RES_Q by that (64 x 8191 rows without other
  // work between the calls: 129 us where three take 115; with d_R = 512 two took as long as one).
  static constexpr int SPS = MODE == RES_Q && NSL == 9 ? 3 : 1;
  static constexpr int NST = MODE == RES_K ? 4 : (MODE == RES_Q ? (NSL == 9 ? 3 : 5) : 6);
  static constexpr int STAGE = SPS * SBOX;
  static_assert(NSL % SPS == 0, "whole stages");
  static constexpr int OFF_RES = 0;
  static constexpr int OFF_ST = NRES * RBOX;
  static constexpr int OFF_ROW = OFF_ST + NST * STAGE;     // (lse, weight) of rows [2][2][NT]
  static constexpr int OFF_SUM = OFF_ROW + 4 * NT * 8;    // sums handed between warpgroups [128]
  static constexpr int OFF_PART = OFF_SUM + 128 * 4;       // sums of the cluster's other pairs
  static constexpr int OFF_MASK = OFF_PART + MAXCP * 128 * 4;   // rows that add, bits [2][2][8]
  static constexpr int OFF_BAR = OFF_MASK + 4 * 8 * 4;
  static constexpr int B_SF = 0;                           // stage loaded, both CTAs   [NST]
  static constexpr int B_SE = B_SF + NST;                  // stage free                [NST]
  static constexpr int B_RF = B_SE + NST;                  // resident box loaded       [NRES]
  static constexpr int B_RE = B_RF + NRES;                 // resident box free         [NRES]
  static constexpr int B_AF = B_RE + NRES;                 // accumulator complete      [2]
  static constexpr int B_AE = B_AF + 2;                    // accumulator read, 8 warps [2]
  static constexpr int NBAR = B_AE + 2;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;      // TMEM slot, abort flag
  static constexpr int SMEM = OFF_MISC + 16 + 1024;
  static_assert(SMEM <= 227 * 1024, "dynamic shared memory of one CTA");
  static_assert(OFF_ST % 1024 == 0 && OFF_ROW % 1024 == 0 && RBOX % 1024 == 0 && SBOX % 1024 == 0,
                "swizzled boxes start on their alignment");
};

struct WeightArgs {
  AttnArgs a;                                  // g, n_q, q_abs, window, tree, bn, err
  float c2;                                    // softmax scale in log2 units
  const float* lse;
  const float* qw;
  const float* win;
  float* out;
};

// The row groups (128 rows) of a sequence that add to the weights, and the tiles they make.
struct Groups {
  uint64_t set;                                // bit g: group g (masked), else unused
  bool masked;                                 // up to 64 groups and query weights: listed in `set`
  int tiles;
};
__device__ __forceinline__ Groups row_groups(const WeightArgs& p, int64_t b, int64_t rows, int nt) {
  Groups r;
  r.masked = p.qw != nullptr && rows <= 64 * 128;
  r.set = 0;
  if (!r.masked) {
    r.tiles = (int)((rows + nt - 1) / nt);
    return r;
  }
  const float* qw = p.qw + b * p.a.n_q;
  const uint32_t H = (uint32_t)p.a.g.H, nodes = (uint32_t)rows / H;
#pragma unroll 8
  for (uint32_t i = 0; i < nodes; ++i)
    if (qw[i] != 0.f)                          // node i's rows lie in groups i H / 128 .. ((i + 1) H - 1) / 128
      r.set |= ((2ull << (((i + 1) * H - 1) >> 7)) - 1ull) & ~((1ull << (i * H >> 7)) - 1ull);
  r.tiles = (__popcll(r.set) + nt / 128 - 1) / (nt / 128);
  return r;
}

// The pieces of units (256 keys of a sequence) one pair walks, in order: tiles [qb, qe) of each.
struct UnitWalk {
  uint32_t pos, end;                           // position in the line of tiles, and its end
  int b, u, units, qb, qe, nt;
  TreeGeo s;
  Groups g;
  int64_t rows, qrow0;                         // (node, head) rows of the sequence, its first row

  __device__ void sequence(const WeightArgs& p, int seq) {
    b = seq;
    s = tree_geo<KEYS>(p.a, b);
    rows = (int64_t)(s.blk.L - s.ctx) * p.a.g.H;
    units = (s.blk.nblk + 1) / 2;
    g = row_groups(p, b, rows, nt);
    qrow0 = (int64_t)b * p.a.n_q * p.a.g.H;
  }
  __device__ void piece(int from) {
    qb = from;
    qe = (uint32_t)(g.tiles - from) < end - pos ? g.tiles : from + (int)(end - pos);
  }
  // from position `at`, offset `off` of sequence seq's
  __device__ void begin(const WeightArgs& p, int seq, uint32_t at, uint32_t off) {
    sequence(p, seq);
    pos = at;
    u = (int)(off / (uint32_t)g.tiles);
    piece((int)(off - (uint32_t)(u * g.tiles)));
  }
  __device__ bool valid() const { return pos < end; }
  __device__ void next(const WeightArgs& p) {
    pos += qe - qb;
    if (pos >= end) return;
    if (++u >= units) {
      u = 0;
      do {
        sequence(p, b + 1);                    // pos < end: a later sequence has tiles
      } while (g.tiles == 0);
    }
    piece(0);
  }
  // this CTA's key block of the unit: first slot, first logical row, keys (0: none)
  __device__ void keys(uint32_t side, int64_t S, int64_t& slot0, int64_t& j0, int& valid) const {
    const int j = 2 * u + (int)side;
    if (j < s.blk.nblk) {
      int sl, jl;
      s.blk.get<KEYS>(j, sl, jl, valid);
      slot0 = sl;
      j0 = jl;
    } else {
      slot0 = S;                               // outside the tensor: the box is filled with zeros
      j0 = 0;
      valid = 0;
    }
  }
};

// The groups of a tile, taken off in order.
struct GroupCursor {
  uint64_t left;
  int k;
  __device__ void begin(const Groups& g, int tile, int per_tile) {
    left = g.set;
    k = tile * per_tile;
    if (g.masked)
      for (int i = 0; i < k; ++i) left &= left - 1;
  }
  // the next group, or -1 (masked sets may end inside a tile)
  __device__ int take(const Groups& g) {
    if (!g.masked) return k++;
    if (left == 0) return -1;
    const int r = __ffsll((long long)left) - 1;
    left &= left - 1;
    return r;
  }
};

// Part k of CP of the positions [s0, s1).
__device__ __forceinline__ uint32_t line_part(uint32_t s0, uint32_t s1, int k, int CP) {
  const uint32_t n = s1 - s0, each = n / (uint32_t)CP, odd = n - each * (uint32_t)CP;
  return s0 + each * (uint32_t)k + odd * (uint32_t)k / (uint32_t)CP;
}

// The tiles of all units, sequence after sequence, make one line of W positions.  Cluster c of C
// takes the units that start in its equal share of it, [s0, s1); pair k of CP an equal part of
// those positions.  Warp-collective.
template <int NT>
__device__ __forceinline__ void plan_units(const WeightArgs& p, uint32_t C, uint32_t c, int k,
                                           int CP, UnitWalk& w, uint32_t& s0, uint32_t& s1) {
  const int lane = threadIdx.x & 31, B = p.a.g.B;
  w.nt = NT;
  w.pos = w.end = 0;
  auto span = [&](int b) {                     // tiles per unit, units
    const TreeGeo s = tree_geo<KEYS>(p.a, b);
    const int64_t rows = (int64_t)(s.blk.L - s.ctx) * p.a.g.H;
    return Span{(uint32_t)row_groups(p, b, rows, NT).tiles, (uint32_t)(s.blk.nblk + 1) / 2};
  };
  const Span mine = lane < B ? span(lane) : Span{0, 0};
  uint32_t W = 0;
  for (int b = lane; b - lane < B; b += 32) {
    const Span s = b == lane ? mine : (b < B ? span(b) : Span{0, 0});
    W += s.tiles * s.blocks;
  }
  W = __reduce_add_sync(FULL, W);
  s0 = s1 = 0;
  if (W == 0) return;
  // the shares' ends, moved up to where a unit starts; then where this pair's part lies
  const uint32_t each = W / C, odd = W - each * C;
  const uint32_t cut[2] = {each * c + odd * c / C, each * (c + 1) + odd * (c + 1) / C};
  if (cut[0] >= cut[1]) {                      // (a line shorter than the clusters are many)
    s0 = s1 = 0;
    return;
  }
  const uint32_t q[2] = {cut[0], cut[1] < W ? cut[1] : W - 1};
  Spot f[2];
  line_find(B, span, mine, q, f);
  auto up = [](const Spot& x) { return (x.off + x.s.tiles - 1) / x.s.tiles * x.s.tiles - x.off; };
  s0 = cut[0] + up(f[0]);
  s1 = cut[1] < W ? cut[1] + up(f[1]) : W;
  const uint32_t p0[1] = {line_part(s0, s1, k, CP)};
  const uint32_t p1 = line_part(s0, s1, k + 1, CP);
  if (p0[0] >= p1) return;                     // nothing for this pair
  Spot g[1];
  line_find(B, span, mine, p0, g);
  w.end = p1;
  w.begin(p, g[0].b, p0[0], g[0].off);
}

template <int NSL, int MODE>
__global__ void __launch_bounds__(WT, 1)
    attend_weight_kernel(const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmQ,
                         const __grid_constant__ WeightArgs p, int CP) {
  using LY = WLay<NSL, MODE>;
  constexpr int NT = LY::NT, SPS = LY::SPS, NST = LY::NST, NRES = LY::NRES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~uintptr_t(1023));
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + LY::OFF_BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + LY::OFF_MISC);
  volatile int* abort = reinterpret_cast<volatile int*>(sm + LY::OFF_MISC + 4);
  const uint32_t crank = cluster_ctarank(), rank = crank & 1u, leader = crank & ~1u;
  const int pair = (int)(crank >> 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const AttnArgs& a = p.a;

  if (tid == 0) {
    for (int q = 0; q < LY::B_AE; ++q) mbar_init(&bar[q], 1);
    for (int q = 0; q < 2; ++q) mbar_init(&bar[LY::B_AE + q], 8);
    *abort = 0;
    fence_mbar_init();
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmQ);
  }
  if (warp == 9) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                              // the pair's barriers exist before any remote use
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dep_wait();                             // the previous kernel's outputs are visible
  grid_dep_launch();

  UnitWalk w;
  uint32_t s0, s1;                             // the cluster's positions
  plan_units<NT>(p, gridDim.x / (2 * CP), blockIdx.x / (2 * CP), pair, CP, w, s0, s1);
  auto part = [&](int k) { return line_part(s0, s1, k, CP); };
  // (a pair's loads complete on the even CTA's barriers, but go to each CTA's own memory)
  float kept = 0.f, kept_base = 0.f;           // a unit this pair began and others went on with
  int64_t kept_at = -1;
  uint32_t kept_end = 0;

  if (warp == 8) {
    // ---------------------------------------------------------------- TMA producer
    if (lane == 0) {
      const uint32_t even = mapa(smem_u32(bar), leader);
      uint32_t it = 0, un = 0;                 // stages filled, resident tiles filled
      int res_b = -1;
      bool ok = true;
      for (; ok && w.valid(); w.next(p)) {
        int64_t slot0, j0;
        int valid;
        w.keys(rank, a.g.S, slot0, j0, valid);
        // resident boxes of the unit (RES_Q: of the sequence), each as soon as its last use is done
        const bool fill = MODE == RES_K || (MODE == RES_Q && w.b != res_b);
        auto resident = [&](int i) {
          if (!mbar_wait(&bar[LY::B_RE + i], (un & 1) ^ 1, abort, a.err, 0x31, i)) return false;
          if (rank == 0) mbar_expect_tx(&bar[LY::B_RF + i], 2 * LY::RBOX);
          const uint32_t full = even + (LY::B_RF + i) * 8;
          if (MODE == RES_K)
            tma_load_3d_pair(sm + LY::OFF_RES + i * LY::RBOX, &tmK, full, i * 64, (int32_t)slot0, w.b);
          else
            tma_load_2d_pair(sm + LY::OFF_RES + i * LY::RBOX, &tmQ, full, i * 64,
                             (int32_t)(w.qrow0 + rank * (NT / 2)));
          return true;
        };
        GroupCursor gc;
        gc.begin(w.g, w.qb, NT / 128);
        for (int q = w.qb; ok && q < w.qe; ++q) {
          // this CTA's half of the tile: a group of 128 rows (a missing second one loads any rows)
          int64_t row = w.qrow0;
          if (MODE != RES_Q) {
            const int g0 = gc.take(w.g), g1 = gc.take(w.g);
            const int g = rank == 0 ? g0 : g1;
            row += (int64_t)(g < 0 ? 0 : g) * 128;
          }
          for (int i = 0; ok && i < NSL; i += SPS, ++it) {
            if (fill && q == w.qb)
              for (int e = 0; ok && e < SPS; ++e) ok = resident(i + e);
            if (!ok) break;
            const int s = it % NST;
            ok = mbar_wait(&bar[LY::B_SE + s], ((it / NST) & 1) ^ 1, abort, a.err, 0x32, it);
            if (!ok) break;
            if (rank == 0) mbar_expect_tx(&bar[LY::B_SF + s], 2 * LY::STAGE);
            const uint32_t full = even + (LY::B_SF + s) * 8;
#pragma unroll
            for (int e = 0; e < SPS; ++e) {
              uint8_t* st = sm + LY::OFF_ST + s * LY::STAGE + e * LY::SBOX;
              if (MODE != RES_Q)
                tma_load_2d_pair(st, &tmQ, full, (i + e) * 64, (int32_t)row);
              if (MODE != RES_K)
                tma_load_3d_pair(st + (MODE == STREAM ? LY::QBOX : 0), &tmK, full, (i + e) * 64,
                                 (int32_t)slot0, w.b);
            }
          }
        }
        if (fill) {
          ++un;
          res_b = w.b;
        }
      }
      // the MMAs' last arrivals on this CTA's barriers land before it may exit
      for (uint32_t k = it > NST ? it - NST : 0; ok && k < it; ++k)
        ok = mbar_wait(&bar[LY::B_SE + k % NST], (k / NST) & 1, abort, a.err, 0x37, k);
      for (int i = 0; ok && un > 0 && i < NRES; ++i)
        ok = mbar_wait(&bar[LY::B_RE + i], (un - 1) & 1, abort, a.err, 0x38, i);
    }
  } else if (warp == 9 && rank == 1) {
    // ---------------------------------------------------------------- pass-through
    // sequences that add nothing have no tiles: their totals stay, a node's row gets 0
    for (int b = blockIdx.x >> 1; b < a.g.B; b += gridDim.x >> 1) {
      const Window v = load_window(a.window, b, a.g.S, a.n_q);
      if (v.len() == 0 || row_groups(p, b, (int64_t)v.nodes * a.g.H, NT).tiles > 0) continue;
      for (int j = lane; j < v.len(); j += 32) {
        const int64_t at = (int64_t)b * a.g.S + v.slot(j, a.g.S);
        p.out[at] = j < v.rows && p.win ? p.win[at] : 0.f;
      }
    }
  } else if (warp == 9) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      const uint32_t id = idesc_bf16(256, NT, false, false);
      const uint16_t both = (uint16_t)(3u << leader);
      uint32_t it = 0, un = 0, tc = 0;
      int res_b = -1;
      bool ok = true;
      while (ok && w.valid()) {
        const bool fill = MODE == RES_K || (MODE == RES_Q && w.b != res_b);
        const int b = w.b, tiles = w.qe - w.qb;
        w.next(p);                             // the next unit tells whether the boxes are done with
        const bool last = MODE == RES_K || !w.valid() || w.b != b;
        for (int q = 0; ok && q < tiles; ++q, ++tc) {
          const int acc = tc & 1;
          ok = mbar_wait_cluster(&bar[LY::B_AE + acc], ((tc >> 1) & 1) ^ 1, abort, a.err, 0x33, tc);
          if (!ok) break;
          tc_fence_after();
          for (int i = 0; i < NSL; i += SPS, ++it) {
            const int s = it % NST;
            if (fill && q == 0)
              for (int e = 0; ok && e < SPS; ++e)
                ok = mbar_wait_cluster(&bar[LY::B_RF + i + e], un & 1, abort, a.err, 0x34, i + e);
            if (ok)
              ok = mbar_wait_cluster(&bar[LY::B_SF + s], (it / NST) & 1, abort, a.err, 0x35, it);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int e = 0; e < SPS; ++e) {
              const uint32_t st = smem_u32(sm + LY::OFF_ST + s * LY::STAGE + e * LY::SBOX);
              const uint32_t rs = smem_u32(sm + LY::OFF_RES + (i + e) * LY::RBOX);
              const uint32_t kk = MODE == RES_K ? rs : (MODE == RES_Q ? st : st + LY::QBOX);
              const uint32_t qq = MODE == RES_Q ? rs : st;
              const uint64_t da = desc_sw128(kk, 16, 1024), db = desc_sw128(qq, 16, 1024);
#pragma unroll
              for (int k = 0; k < 4; ++k)      // 16-dim steps: +32 bytes inside the swizzle atom
                mma_ss_pair(tmem + acc * 256, da + 2 * k, db + 2 * k, id, (i | e | k) ? 1u : 0u);
            }
            mma_commit_pair(&bar[LY::B_SE + s], both);
            if (NRES > 0 && last && q == tiles - 1)
              for (int e = 0; e < SPS; ++e) mma_commit_pair(&bar[LY::B_RE + i + e], both);
          }
          if (ok) mma_commit_pair(&bar[LY::B_AF + acc], both);
        }
        if (fill) {
          ++un;
          res_b = b;
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- epilogue warpgroups
    const int wg = warp >> 2, t = tid & 127;   // accumulator, key = TMEM lane
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t drained = mapa(smem_u32(&bar[LY::B_AE + wg]), leader);
    float2* rowbuf = reinterpret_cast<float2*>(sm + LY::OFF_ROW) + wg * 2 * NT;
    uint32_t* rowmask = reinterpret_cast<uint32_t*>(sm + LY::OFF_MASK) + wg * 16;
    float* handed = reinterpret_cast<float*>(sm + LY::OFF_SUM);
    const uint32_t H = (uint32_t)a.g.H;
    uint32_t tc = 0, mine = 0;                 // tiles of the pair, tiles this warpgroup has taken
    // After an expired wait the warps still walk to the end (each further wait gives up at once):
    // the warpgroups meet at named barriers.
    bool ok = true;
    for (; w.valid(); w.next(p)) {
      int64_t slot0, j0;
      int valid;
      w.keys(rank, a.g.S, slot0, j0, valid);
      const bool nodes = j0 + valid > w.s.ctx;         // the block holds draft nodes
      const int64_t node = j0 + t - w.s.ctx;           // this key's node (negative: context)
      const uint8_t* tree =
          a.tree ? a.tree + (int64_t)w.b * a.n_q * a.n_q + (node > 0 ? node : 0) : nullptr;
      auto sees = [&](int64_t i) {                     // whether node i sees this key
        return node < 0 || t >= valid || (tree ? tree[i * a.n_q] != 0 : node <= i);
      };
      float total = 0.f;
      bool took = false;
      GroupCursor gc;
      gc.begin(w.g, w.qb, NT / 128);
      for (int q = w.qb; q < w.qe; ++q, ++tc) {
        // the tile's groups of 128 columns: first row and rows of each (0: nothing there)
        uint32_t row[NT / 128];
        int n[NT / 128];
#pragma unroll
        for (int h = 0; h < NT / 128; ++h) {
          const int g = gc.take(w.g);
          row[h] = (uint32_t)(g < 0 ? 0 : g) * 128u;
          const int64_t left = g < 0 ? 0 : w.rows - (int64_t)row[h];
          n[h] = left < 0 ? 0 : (left < 128 ? (int)left : 128);
        }
        if ((int)(tc & 1) != wg) continue;
        took = true;
        // log-sum-exps (log2 units) and weights of the tile's rows, and which of them add anything
        float2* rb = rowbuf + (mine & 1) * NT;
        uint32_t* rm = rowmask + (mine & 1) * 8;
#pragma unroll
        for (int h = 0; h < NT / 128; ++h) {
          float2 v = make_float2(INFINITY, 0.f);
          if (t < n[h]) {
            const float l = p.lse[w.qrow0 + row[h] + t];
            const float g = p.qw ? p.qw[(int64_t)w.b * a.n_q + (row[h] + t) / H] : 1.f;
            if (g != 0.f && l != -INFINITY) v = make_float2(l * 1.4426950408889634f, g);
          }
          rb[h * 128 + t] = v;
          const uint32_t adds = __ballot_sync(FULL, v.y != 0.f);
          if (lane == 0) rm[h * 4 + (warp & 3)] = adds;
        }
        named_bar(1 + wg, 128);
        ok = __all_sync(FULL, ok && mbar_wait_cluster(&bar[LY::B_AF + wg], mine & 1, abort, a.err,
                                                      0x36, (t << 16) | mine));
        ++mine;
        tc_fence_after();
        const uint32_t acc = tmem + lane_base + wg * 256;
#pragma unroll 1
        for (int c0 = 0; c0 < NT; c0 += 32) {
          uint32_t v[32];
          tmem_ld32(acc + c0, v);
          tmem_wait_ld();
          if (c0 + 32 == NT) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(drained);
          }
          // rows of these 32 columns that exist, the first one, and (where it matters) their nodes
          const bool second = NT > 128 && c0 >= 128;
          const uint32_t adds = rm[c0 / 32];             // (rows past the last have no weight)
          if (!ok || adds == 0) continue;
          const uint32_t r0 = (second ? row[NT / 128 - 1] : row[0]) + (c0 & 127);
          const uint32_t i0 = nodes ? r0 / H : 0, i1 = nodes ? (r0 + 31) / H : 0;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
          if (adds == ~0u && i0 == i1) {
            const float4* rv = reinterpret_cast<const float4*>(rb + c0);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float4 x = rv[e];                  // two rows' (lse, weight)
              const float p0 = ex2(fmaf(__uint_as_float(v[2 * e]), p.c2, -x.x));
              const float p1 = ex2(fmaf(__uint_as_float(v[2 * e + 1]), p.c2, -x.z));
              sum[(2 * e) & 3] = fmaf(p0, x.y, sum[(2 * e) & 3]);
              sum[(2 * e + 1) & 3] = fmaf(p1, x.w, sum[(2 * e + 1) & 3]);
            }
            const float s = (sum[0] + sum[1]) + (sum[2] + sum[3]);
            if (!nodes || sees(i0)) total += s;
          } else {
            // rows that add nothing, whatever their queries hold, or rows of several nodes next to draft
            // keys: a bit per row
            uint32_t in = adds;
            if (nodes) {
              const int live = 32 - __clz((int)adds);
              uint32_t seen = 0u;
              for (uint32_t i = i0; i <= i1; ++i) {
                const int lo = max((int)(i * H) - (int)r0, 0), hi = (int)((i + 1) * H) - (int)r0;
                const uint32_t run = (hi >= 32 ? ~0u : (1u << hi) - 1u) & ~((1u << lo) - 1u);
                if (lo < live && sees(i)) seen |= run;
              }
              in &= seen;
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float2 x = rb[c0 + e];
              const float pe = ex2(fmaf(__uint_as_float(v[e]), p.c2, -x.x));
              if (in >> e & 1) sum[e & 3] = fmaf(pe, x.y, sum[e & 3]);
            }
            total += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          }
        }
      }
      const int64_t at = (int64_t)w.b * a.g.S + slot0 + t;
      if (MODE == RES_Q) {
        // one warpgroup has the unit to itself
        if (took && ok && t < valid) p.out[at] = (p.win && node < 0 ? p.win[at] : 0.f) + total;
        continue;
      }
      // the sum of the even tiles plus that of the odd ones
      if (wg == 1) handed[t] = total;
      named_bar(3, 256);
      total += handed[t];
      named_bar(3, 256);
      if (wg == 0) {
        if (w.qb > 0) {
          // another pair started this unit: it is the last one whose part starts at or before it
          int k = pair - 1;
          while (k > 0 && part(k) > w.pos - w.qb) --k;
          st_cluster_f32(mapa(smem_u32(sm + LY::OFF_PART + (pair * 128 + t) * 4), 2 * k + rank), total);
        } else if (w.qe < w.g.tiles) {
          // other pairs go on with it: kept until their sums are here
          kept = total;
          kept_end = w.pos + w.g.tiles;
          kept_at = t < valid && ok ? at : -1;
          kept_base = p.win && node < 0 && t < valid ? p.win[at] : 0.f;
        } else if (ok && t < valid) {
          p.out[at] = (p.win && node < 0 ? p.win[at] : 0.f) + total;
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();                              // the pairs' sums are here; no remote access is pending
  if (kept_at >= 0) {
    const float* others = reinterpret_cast<const float*>(sm + LY::OFF_PART) + tid;
    for (int k = pair + 1; k < CP && part(k) < kept_end; ++k)
      if (part(k) < part(k + 1)) kept += others[k * 128];
    p.out[kept_at] = kept_base + kept;
  }
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// Clusters of cp pairs that can be resident at once on the current device (0: error).
template <int NSL, int MODE>
int weight_clusters(int cp) {
  using LY = WLay<NSL, MODE>;
  static std::mutex mu;
  static int cached[64][MAXCP + 1] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (dev < 64 && cached[dev][cp] > 0) return cached[dev][cp];
  // also opts the kernel in to its shared memory, once per device
  if (cudaFuncSetAttribute(attend_weight_kernel<NSL, MODE>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, LY::SMEM) != cudaSuccess)
    return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * MAXC);
  cfg.blockDim = dim3(WT);
  cfg.dynamicSmemBytes = LY::SMEM;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = 2 * cp;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, attend_weight_kernel<NSL, MODE>, &cfg) != cudaSuccess)
    return 0;
  n = n < 1 ? 1 : (n > MAXC ? MAXC : n);
  if (dev < 64) cached[dev][cp] = n;
  return n;
}

template <int NSL, int MODE>
cudaError_t launch_weight(const CUtensorMap& K, const CUtensorMap& Q, const WeightArgs& p, int cp,
                          cudaStream_t st) {
  const int n = weight_clusters<NSL, MODE>(cp);
  if (n == 0) return cudaErrorInvalidDevice;
  const cudaError_t e =
      launch_dependent(attend_weight_kernel<NSL, MODE>, (unsigned)(2 * cp * n), WT,
                       WLay<NSL, MODE>::SMEM, st, (unsigned)(2 * cp), K, Q, p, cp);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace

bool tc_attend_weight_supported(const Geo& g, int64_t n_nodes) {
  // the line of tiles (of at least 128 rows, 256 keys) is counted in 31 bits
  const int64_t tiles = (n_nodes * g.H + 127) / 128, units = g.S / 256 + 3;
  return g.Dc == 512 && (g.Dr == 64 || g.Dr == 512) &&
         (double)g.B * tiles * units < 2147483648.0;
}

cudaError_t tc_attend_weight(const Geo& g, const void* q_abs, int64_t n_nodes, const void* cache,
                             const int32_t* window, const uint8_t* tree, float scale,
                             const float* lse, const float* qw, const float* win, float* wout,
                             unsigned int* err, cudaStream_t st) {
  WeightArgs p{};
  p.a.g = g;
  p.a.n_q = n_nodes;
  p.a.bn = KEYS;
  p.a.window = window;
  p.a.tree = tree;
  p.a.err = err;
  p.c2 = scale * 1.4426950408889634f;
  p.lse = lse;
  p.qw = qw;
  p.win = win;
  p.out = wout;
  const bool few = n_nodes * g.H <= 128;       // one tile of 128 rows per sequence
  CUtensorMap K, Q;
  {
    uint64_t d[3] = {(uint64_t)g.row, (uint64_t)g.S, (uint64_t)g.B};
    uint64_t s[2] = {(uint64_t)g.row * 2, (uint64_t)g.S * g.row * 2};
    uint32_t b[3] = {64, KEYS, 1};
    if (!make_tmap_bf16(&K, cache, 3, d, s, b)) return cudaErrorInvalidValue;
  }
  {
    uint64_t d[2] = {(uint64_t)g.row, (uint64_t)g.B * n_nodes * g.H};
    uint64_t s[1] = {(uint64_t)g.row * 2};
    uint32_t b[2] = {64, few ? 64u : 128u};
    if (!make_tmap_bf16(&Q, q_abs, 2, d, s, b)) return cudaErrorInvalidValue;
  }
  // Pairs per cluster: with P clusters, units of up to T tiles take about ceil(units / P) turns of
  // T / cp tiles and a load of the keys each.  (Counted with full rings; 148 SMs give 74 clusters of
  // one pair, 37 of two, 17 of four.  Measured, us with 1 / 2 / 4 pairs: 1 sequence of 1000 rows
  // and 16 nodes, 128 heads 40 / 24 / 16; 1 of 8000 rows, 40 nodes 92 / 53 / 70; 32 of 4000 rows,
  // 32 nodes 529 / 588 / 636.)
  int cp = 1;
  if (!few) {
    const int64_t units = (int64_t)g.B * ((g.S + 255) / 256), tiles = (n_nodes * g.H + 255) / 256;
    double best = 1e300;
    for (int c = 1; c <= MAXCP; c *= 2) {
      const int n = g.Dr == 64 ? weight_clusters<9, RES_K>(c) : weight_clusters<16, STREAM>(c);
      if (n == 0) continue;
      const double turns = (double)((units + n - 1) / n) * (double)((tiles + c - 1) / c + 1);
      if (turns < best) {
        best = turns;
        cp = c;
      }
    }
  }
  if (g.Dr == 64)
    return few ? launch_weight<9, RES_Q>(K, Q, p, 1, st) : launch_weight<9, RES_K>(K, Q, p, cp, st);
  return few ? launch_weight<16, RES_Q>(K, Q, p, 1, st) : launch_weight<16, STREAM>(K, Q, p, cp, st);
}

}  // namespace mla
