// Tensor-core (tcgen05) GEMMs of the path, bf16 in, fp32 accumulation in TMEM:
//   cache write:  [h] x [W_DKV | W_KR]  -> RoPE on the W_KR columns -> bf16 -> ring slot
//   absorb:       q_nope[:, h] x W_UK[h] -> q_lat (plus RoPE of q_R in the same CTAs)
//   up-projection: o_lat[:, h] x W_UV[h]^T -> out
//   materialisation: c[slot] x W[h]^T -> per-head keys or values of every ring slot
// Persistent: one CTA per SM walks the 128 x 128 output tiles (M fastest, so CTAs that
// run together share the weight tile in L2).  Warp 0 lane 0 streams TMA loads through a
// 4-stage shared-memory ring, warp 1 lane 0 issues tcgen05.mma (M=128, N=128, K=16 steps)
// into one of two TMEM accumulators, and warps 2-5 drain the other accumulator (one row
// per thread) through the fused epilogue, so a tile's epilogue overlaps the next tile's
// main loop.
#include "launch.h"
#include "tc_ptx.cuh"
#include "tmap.h"
#include "window.cuh"

#include <mutex>

namespace mla {
namespace {

using namespace tc;

constexpr int GBM = 128, GBK = 64, GBN = 128;

constexpr int GTHREADS = 192;
constexpr int A_BYTES = GBM * GBK * 2;           // 16 KB
constexpr int B_BYTES = GBN * GBK * 2;           // 16 KB
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int MAX_PAIRS = 512;                   // RoPE pairs with a table entry (d_R <= 1024)
constexpr int STG_BYTES = 32 * 64;                // per epilogue warp: 32 rows x 32 cols bf16
constexpr int RB_BYTES = GBM * GBN * 4;          // split-K partials; KS - 1 of 128 / KS columns
// Shared memory: the stage ring, barriers, the RoPE frequency table, epilogue staging and,
// with split-K, the buffer the cluster's other CTAs send their fp32 partials of this one's columns
// into.
constexpr int OBOX_BYTES = GBM * 64 * 2;         // TMA-store box: 128 rows x 64 cols bf16
template <int ST, bool SK> struct GLay {
  static constexpr int OFF_TAB = ST * STAGE_BYTES + 256;
  static constexpr int OFF_STG = OFF_TAB + MAX_PAIRS * 8;
  static constexpr int OFF_RB = OFF_STG + 4 * STG_BYTES;
  // output boxes for the TMA stores of the absorption and the up-projection [2]
  static constexpr int OFF_OST = (OFF_RB + (SK ? RB_BYTES : 0) + 1023) & ~1023;
  static constexpr int SMEM = OFF_OST + (SK ? 0 : 2 * OBOX_BYTES) + 1024;
};

enum Mode { MODE_CACHE = 0, MODE_ABSORB = 1, MODE_UPV = 2, MODE_MAT = 3 };

struct TcGemm {
  int M, N, K, Z;
  int mode;
  int b_mn;                 // B is MN-major (N contiguous) instead of K-major
  int n_split;              // cache: tiles at n >= n_split read tmB2 at n - n_split
  bf16* out;
  int64_t rows_per_batch;   // cache: tokens per sequence in the call (n_tok)
  Geo geo;
  int64_t first_tok;        // cache: first token; absorb: first query token
  int32_t* slots;
  const bf16* q_rope;       // absorb: RoPE part input
  // draft nodes: positions per row (cache, absorb), and for the cache each sequence's window,
  // behind whose context its rows go, and the positions array to keep them in (may be null)
  const int32_t* token;
  const int32_t* window;
  int32_t* position;
  int ks;                   // split-K: CTAs per tile
  unsigned int* err;
};

// GSTAGES-deep TMA ring.  Four stages (one CTA per SM) suit long K loops; two stages let
// two CTAs share an SM, which hides the latency of short-K tiles (the absorption).
// SPLITK: launched in clusters of p.ks CTAs that share each tile, rank r taking the r-th part of
// the K blocks.  For few tiles with long K (the cache write: 65 tiles of K = 4096) that brings
// more SMs' load bandwidth to the same tiles.  Each rank finishes a part of the tile's columns, in
// chunks of 8: the others send it their fp32 sums of those through distributed shared memory
// (st.async, completion counted in bytes), and it adds them to its own, the lower ranks' first.
template <int GSTAGES, bool SPLITK>
__global__ void __launch_bounds__(GTHREADS, GSTAGES == 2 ? 2 : 1)
    tc_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmB2, const __grid_constant__ CUtensorMap tmO,
                   TcGemm p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + GSTAGES * STAGE_BYTES);
  uint64_t* empty = full + GSTAGES;
  uint64_t* accf = empty + GSTAGES;              // accumulator ready [2]
  uint64_t* acce = accf + 2;                     // accumulator drained [2]
  uint64_t* rbf = acce + 2;                      // split-K: partials landed (tx bytes)
  uint64_t* rbe = acce + 3;                      // split-K: the others have read this rank's
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acce + 4);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  using GL = GLay<GSTAGES, SPLITK>;
  double* inv_freq = reinterpret_cast<double*>(smem + GL::OFF_TAB);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nm = (p.M + GBM - 1) / GBM, nn = (p.N + GBN - 1) / GBN;
  const int ntiles = nm * nn * p.Z;
  const int nk = (p.K + GBK - 1) / GBK;
  // tiles this CTA (or cluster) walks, and its K blocks
  const uint32_t crank = SPLITK ? cluster_ctarank() : 0u;
  const int ks = SPLITK ? p.ks : 1;
  const int t_first = (int)blockIdx.x / ks;
  const int t_step = (int)gridDim.x / ks;
  const int kb0 = nk * (int)crank / ks;
  const int kb1 = nk * ((int)crank + 1) / ks;

  if (tid == 0) {
    for (int s = 0; s < GSTAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&accf[a], 1);
      mbar_init(&acce[a], 128);
    }
    mbar_init(rbf, 1);
    mbar_init(rbe, ks > 1 ? ks - 1 : 1);
    *abort = 0;
    fence_mbar_init();
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
    prefetch_tmap(&tmB2);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 2 * GBN);
    tmem_relinquish();
  }
  for (int q = tid; q < p.geo.Dr / 2 && q < MAX_PAIRS; q += GTHREADS)
    inv_freq[q] = rope_inv_freq(p.geo, q);
  tc_fence_before();
  __syncthreads();
  if constexpr (SPLITK) cluster_sync();        // the cluster's barriers exist before any remote use
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dep_wait();                               // the previous kernel's outputs are visible
  grid_dep_launch();

  auto tile_coords = [&](int t, int& m0, int& n0, int& z) {
    z = t / (nm * nn);
    const int r = t - z * nm * nn;
    m0 = (r % nm) * GBM;
    n0 = (r / nm) * GBN;
  };

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    if (lane == 0) {
      uint32_t it = 0;
      for (int t = t_first; t < ntiles; t += t_step) {
        int m0, n0, z;
        tile_coords(t, m0, n0, z);
        const bool second = p.mode == MODE_CACHE && n0 >= p.n_split;
        const CUtensorMap* mB = second ? &tmB2 : &tmB;
        const int nb = second ? n0 - p.n_split : n0;
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          const int s = it % GSTAGES;
          if (!mbar_wait(&empty[s], ((it / GSTAGES) & 1) ^ 1, abort, p.err, 0x11, kb)) break;
          uint8_t* a = smem + s * STAGE_BYTES;
          uint8_t* b = a + A_BYTES;
          mbar_expect_tx(&full[s], STAGE_BYTES);
          // the cache write's and the materialisation's A rows serve every head
          tma_load_3d(a, &tmA, &full[s], kb * GBK,
                      p.mode == MODE_CACHE || p.mode == MODE_MAT ? 0 : z, m0);
          if (p.b_mn) {
            tma_load_3d(b, mB, &full[s], nb, kb * GBK, z);
            tma_load_3d(b + B_BYTES / 2, mB, &full[s], nb + 64, kb * GBK, z);
          } else {
            tma_load_3d(b, mB, &full[s], kb * GBK, nb, z);
          }
        }
        if (*abort) break;
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16(GBM, GBN, false, p.b_mn != 0);
      uint32_t it = 0, tc = 0;
      for (int t = t_first; t < ntiles; t += t_step, ++tc) {
        const int acc = tc & 1;
        if (!mbar_wait(&acce[acc], ((tc >> 1) & 1) ^ 1, abort, p.err, 0x14, tc)) break;
        tc_fence_after();
        const uint32_t d = tmem + acc * GBN;
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          const int s = it % GSTAGES;
          if (!mbar_wait(&full[s], (it / GSTAGES) & 1, abort, p.err, 0x12, kb)) break;
          tc_fence_after();
          const uint32_t a = smem_u32(smem + s * STAGE_BYTES);
          const uint32_t b = a + A_BYTES;
          const uint64_t da = desc_sw128(a, 16, 1024);
          const uint64_t db = p.b_mn ? desc_sw128(b, B_BYTES / 2, 1024) : desc_sw128(b, 16, 1024);
#pragma unroll
          for (int k16 = 0; k16 < GBK / 16; ++k16) {
            // K-major operands advance 32 bytes per 16-element K step inside the swizzle
            // atom; the MN-major B advances 16 rows of 128 bytes.
            const uint64_t bstep = p.b_mn ? (uint64_t)(k16 * 2048 >> 4) : (uint64_t)(k16 * 32 >> 4);
            mma_ss(d, da + (uint64_t)(k16 * 32 >> 4), db + bstep, idesc,
                   (kb != kb0 || k16 != 0) ? 1u : 0u);
          }
          mma_commit(&empty[s]);
        }
        mma_commit(&accf[acc]);
        if (*abort) break;
      }
    }
  } else {
    // ---------------------------------------------------------------- epilogue warps
    // Thread r drains TMEM row r of its warp's lane quarter 32 columns at a time, into a
    // per-warp staging buffer (2 KB, 16-byte chunks XOR-swizzled by row so that neither
    // the row-wise writes nor the chunk-wise reads conflict); the warp then writes the
    // 32 rows as 64-byte segments, four lanes per row, instead of one scattered row per
    // lane.
    const int r = (warp & 3) * 32 + lane;       // TMEM lane quarter = warp id % 4
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const Geo& G = p.geo;
    uint8_t* stg = smem + GL::OFF_STG + (warp - 2) * STG_BYTES;
    // split-K partials, [rank][8-column chunk][2][128 rows] of 4 floats: conflict-free for both the
    // sending and the reading thread of a row
    const float4* rb = reinterpret_cast<const float4*>(smem + GL::OFF_RB) + r;
    const uint32_t rb_addr = smem_u32(rb), rbf_addr = smem_u32(rbf);
    uint32_t tc = 0, ost = 0;                   // ost: output boxes stored so far
    for (int t = t_first; t < ntiles; t += t_step, ++tc) {
      int m0, n0, z;
      tile_coords(t, m0, n0, z);
      const int acc = tc & 1;
      const uint32_t trow = tmem + lane_base + acc * GBN;
      // split-K: this rank finishes chunks [own0, own1) of the tile's nch
      const int nch = p.N - n0 < GBN ? (p.N - n0) / 8 : GBN / 8;
      const int own0 = nch * (int)crank / ks, own1 = nch * ((int)crank + 1) / ks;
      const int mrows = p.M - m0 < GBM ? p.M - m0 : GBM;
      bool ok = true;
      // (armed per tile)
      if (SPLITK && r == 0) mbar_expect_tx(rbf, (uint32_t)((ks - 1) * mrows * (own1 - own0) * 32));
      const int64_t m = m0 + r;
      const bool row_ok = m < p.M;
      // the absorption's share of RoPE(q_R) for this row: its loads are issued before the
      // wait for the accumulator, so that their latency overlaps it and the drain
      const bool rope_q = row_ok && p.mode == MODE_ABSORB && G.Dr > 0;
      int qa0 = 0, qa1 = 0;
      uint4 rin[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
      const uint4* rsrc = nullptr;
      if (rope_q) {
        // the row's rotation pairs are shared out over the tiles of its row block, a
        // multiple of 4 pairs (one 16-byte vector) each
        const int nn = (p.N + GBN - 1) / GBN, npairs = G.Dr / 2;
        const int ppt = ((npairs + nn - 1) / nn + 3) & ~3;
        qa0 = (n0 / GBN) * ppt;
        qa1 = qa0 + ppt < npairs ? qa0 + ppt : npairs;
        rsrc = reinterpret_cast<const uint4*>(p.q_rope + (m * G.H + z) * G.Dr);
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if (qa0 / 4 + u < qa1 / 4) rin[u] = rsrc[qa0 / 4 + u];
      }
      // this row's output base (element offset of column 0) and, for the cache, its token
      int64_t base = 0, g = 0;
      RopeAxes ax{0.0, 0.0, 0.0};
      if (p.mode == MODE_CACHE) {
        const int64_t b = m / p.rows_per_batch;
        g = p.first_tok + (m - b * p.rows_per_batch);
        if (p.window == nullptr) {
          base = (b * G.S + g % G.S) * G.row;
        } else {
          base = -1;                              // rows past a sequence's nodes are not stored
          if (row_ok) {
            const Window w = load_window(p.window, b, G.S, p.rows_per_batch);
            const int64_t i = m - b * p.rows_per_batch;
            if (i < w.nodes) {
              g = p.token[m];
              const int64_t at = b * G.S + w.slot(w.rows + i, G.S);
              base = at * G.row;
              if (p.position && n0 == 0 && crank == 0) p.position[at] = (int32_t)g;
            }
          }
        }
        if (row_ok && G.Dr > 0) ax = rope_axes(G, g);
      } else if (p.mode == MODE_ABSORB) {
        base = (m * G.H + z) * G.row;
      } else {
        base = (m * G.H + z) * G.Dn;
      }
      ok = __all_sync(0xffffffffu, mbar_wait(&accf[acc], (tc >> 1) & 1, abort, p.err, 0x13,
                                             (r << 16) | tc));
      // nq chunks of 8 columns from column n on: the rotation, bf16, the ring
      auto store_cols = [&](float (&f)[32], int n, int nq) {
        if (p.mode == MODE_CACHE && n >= p.n_split && row_ok) {
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            if (j >= 8 * nq) break;
            const int q = (n + j - p.n_split) / 2;
            rope_rotate_fast(f[j], f[j + 1], rope_axis_pos(G, ax, q), inv_freq[q]);
          }
        }
        uint4* srow = reinterpret_cast<uint4*>(stg + lane * 64);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          srow[q ^ ((lane >> 1) & 3)] = make_uint4(
              pack_bf16(f[8 * q + 0], f[8 * q + 1]), pack_bf16(f[8 * q + 2], f[8 * q + 3]),
              pack_bf16(f[8 * q + 4], f[8 * q + 5]), pack_bf16(f[8 * q + 6], f[8 * q + 7]));
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rr = 8 * i + (lane >> 2), j = lane & 3;        // row of the warp, chunk
          const int64_t rbase = __shfl_sync(0xffffffffu, base, rr);
          if (m0 + (warp & 3) * 32 + rr < p.M && rbase >= 0 && j < nq) {
            const uint4 w = reinterpret_cast<const uint4*>(stg + rr * 64)[j ^ ((rr >> 1) & 3)];
            *reinterpret_cast<uint4*>(p.out + rbase + n + 8 * j) = w;
          }
        }
        __syncwarp();
      };
      if constexpr (SPLITK) {
        // send the others' columns once they have read the previous tile's
        if (ok)
          ok = __all_sync(0xffffffffu, mbar_wait_cluster(rbe, (tc & 1) ^ 1, abort, p.err, 0x16,
                                                         (r << 16) | tc));
        tc_fence_after();
        for (int c0 = 0; c0 < GBN / 8; c0 += 4) {
          uint32_t v[32];
          tmem_ld32(trow + c0 * 8, v);
          tmem_wait_ld();
          if (!ok || !row_ok) continue;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int c = c0 + q;
            const int d = ((c + 1) * ks - 1) / nch;          // the rank that finishes chunk c
            if (c >= nch || d == (int)crank) continue;
            const int d0 = nch * d / ks, dn = nch * (d + 1) / ks - d0;
            const int from = (int)crank - ((int)crank > d);
            const uint32_t dst = mapa(rb_addr, d) + (uint32_t)((from * dn + c - d0) * 2 * GBM) * 16;
            const uint32_t dbar = mapa(rbf_addr, d);
            st_async_v4(dst, v[8 * q], v[8 * q + 1], v[8 * q + 2], v[8 * q + 3], dbar);
            st_async_v4(dst + GBM * 16, v[8 * q + 4], v[8 * q + 5], v[8 * q + 6], v[8 * q + 7],
                        dbar);
          }
        }
        if (ok)
          ok = __all_sync(0xffffffffu, mbar_wait_cluster(rbf, tc & 1, abort, p.err, 0x17,
                                                         (r << 16) | tc));
        if (!ok) break;
        for (int c0 = own0; c0 < own1; c0 += 4) {
          const int nq = own1 - c0 < 4 ? own1 - c0 : 4;
          uint32_t v[4][8];
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (q < nq) tmem_ld8(trow + (c0 + q) * 8, v[q]);
          tmem_wait_ld();
          if (c0 + 4 >= own1) {
            tc_fence_before();
            mbar_arrive(&acce[acc]);            // accumulator may be overwritten
          }
          float f[32];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[8 * q + j] = 0.f;
            if (q >= nq) continue;
            bool own = false;
            for (int k = 0; k < ks; ++k) {
              if (k == (int)crank) {
#pragma unroll
                for (int j = 0; j < 8; ++j) f[8 * q + j] += __uint_as_float(v[q][j]);
                own = true;
                continue;
              }
              const float4* o = rb + ((k - own) * (own1 - own0) + c0 - own0 + q) * 2 * GBM;
              const float4 lo = o[0], hi = o[GBM];
              f[8 * q] += lo.x;
              f[8 * q + 1] += lo.y;
              f[8 * q + 2] += lo.z;
              f[8 * q + 3] += lo.w;
              f[8 * q + 4] += hi.x;
              f[8 * q + 5] += hi.y;
              f[8 * q + 6] += hi.z;
              f[8 * q + 7] += hi.w;
            }
          }
          store_cols(f, n0 + c0 * 8, nq);
        }
        // every partial is read (its sums have been stored): the others may send the next tile's
        named_bar(1, 128);
        if (r < ks && r != (int)crank) mbar_arrive_cluster_relaxed(mapa(smem_u32(rbe), r));
        if (row_ok && n0 == 0 && crank == 0 && p.slots) p.slots[m] = (int32_t)(g % G.S);
        continue;
      }
      tc_fence_after();
      // two 32-column TMEM loads in flight per wait
      for (int c0 = 0; c0 < GBN; c0 += 64) {
        uint32_t v[2][32];
        tmem_ld32(trow + c0, v[0]);
        tmem_ld32(trow + c0 + 32, v[1]);
        tmem_wait_ld();
        if (c0 + 64 == GBN) {
          tc_fence_before();
          mbar_arrive(&acce[acc]);              // accumulator may be overwritten
        }
        if (p.mode != MODE_CACHE) {
          // The absorption's and the up-projection's outputs are plain 3-D tensors: the
          // warps fill one 128-row x 64-column box (128-byte swizzle) of a two-buffer
          // ring and one thread stores it with TMA, which writes the rows whole.
          uint8_t* ob = smem + GL::OFF_OST + (ost & 1) * OBOX_BYTES;
          ++ost;
          if (r == 0) bulk_wait_group_read<1>();   // the store that last read `ob` is done
          named_bar(1, 128);
          if (ok) {
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const uint32_t* w = &v[hh][8 * q];
                *reinterpret_cast<uint4*>(ob + r * 128 + (((4 * hh + q) ^ (r & 7)) * 16)) =
                    make_uint4(pack_bf16(__uint_as_float(w[0]), __uint_as_float(w[1])),
                               pack_bf16(__uint_as_float(w[2]), __uint_as_float(w[3])),
                               pack_bf16(__uint_as_float(w[4]), __uint_as_float(w[5])),
                               pack_bf16(__uint_as_float(w[6]), __uint_as_float(w[7])));
              }
          }
          fence_proxy_async_smem();
          named_bar(1, 128);
          if (ok && r == 0 && n0 + c0 < p.N) {
            tma_store_3d(&tmO, ob, n0 + c0, z, m0);
            bulk_commit_group();
          }
          continue;
        }
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const int n = n0 + c0 + 32 * hh;      // output column of v[hh][0] (warp-uniform)
          if (!ok || n >= p.N) continue;
          float f[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(v[hh][j]);
          store_cols(f, n, 4);
        }
      }
      if (ok && row_ok && n0 == 0 && p.mode == MODE_CACHE && p.slots)
        p.slots[m] = (int32_t)(g % G.S);
      if (rope_q && ok && qa0 < qa1) {
        // q_abs[.., Dc:] = RoPE(q_R) for the pairs [qa0, qa1) of this row
        const RopeAxes qa =
            rope_axes(G, p.token ? p.token[m] : p.first_tok + m % p.rows_per_batch);
        uint4* dst = reinterpret_cast<uint4*>(p.out + (m * G.H + z) * G.row + G.Dc);
        for (int c = qa0 / 4; c < qa1 / 4; c += 2) {
          uint4 in[2] = {rin[0], rin[1]};
          if (c > qa0 / 4) {
#pragma unroll
            for (int u = 0; u < 2; ++u) if (c + u < qa1 / 4) in[u] = rsrc[c + u];
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            if (c + u >= qa1 / 4) break;
            uint32_t w[4] = {in[u].x, in[u].y, in[u].z, in[u].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int q = (c + u) * 4 + e;
              const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[e]));
              float a = f.x, b = f.y;
              rope_rotate_fast(a, b, rope_axis_pos(G, qa, q), inv_freq[q]);
              w[e] = pack_bf16(a, b);
            }
            dst[c + u] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      if (!ok) break;
    }
    // the output boxes' stores have finished with shared memory and landed before exit
    if (r == 0) bulk_wait_group<0>();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if constexpr (SPLITK) cluster_sync();        // no remote access into this CTA is pending
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 2 * GBN);
  }
}

int sm_count() {
  static int n = 0;
  if (n == 0) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
      n = 148;
  }
  return n;
}

// Split-K clusters of ks CTAs that can be resident at once on the current device (0: error).
int split_clusters(int ks) {
  using GL = GLay<4, true>;
  static std::mutex mu;
  static int cached[64][9] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (dev < 64 && cached[dev][ks] > 0) return cached[dev][ks];
  if (cudaFuncSetAttribute(tc_gemm_kernel<4, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           GL::SMEM) != cudaSuccess)
    return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(ks * sm_count()));
  cfg.blockDim = dim3(GTHREADS);
  cfg.dynamicSmemBytes = GL::SMEM;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = ks;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, tc_gemm_kernel<4, true>, &cfg) != cudaSuccess) return 0;
  if (dev < 64) cached[dev][ks] = n;
  return n;
}

template <int ST, bool SK>
cudaError_t launch_st(const CUtensorMap& A, const CUtensorMap& B, const CUtensorMap& B2,
                      const CUtensorMap& O, const TcGemm& q, long long tiles, cudaStream_t st) {
  using GL = GLay<ST, SK>;
  {
    // the shared-memory opt-in is per device
    static std::mutex mu;
    static uint64_t done = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 64 || !(done >> dev & 1)) {
      e = cudaFuncSetAttribute(tc_gemm_kernel<ST, SK>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, GL::SMEM);
      if (e != cudaSuccess) return e;
      if (dev < 64) done |= 1ull << dev;
    }
  }
  if (!SK) {
    const long long slots = (long long)sm_count() * (ST == 2 ? 2 : 1);
    const int grid = (int)(tiles < slots ? tiles : slots);
    if (grid == 0) return cudaSuccess;
    cudaError_t e = launch_dependent(tc_gemm_kernel<ST, SK>, (unsigned)grid, GTHREADS, GL::SMEM, st,
                                     1u, A, B, B2, O, q);
    if (e != cudaSuccess) return e;
  } else {
    // one cluster per tile up to what the GPU holds
    const long long most = q.ks == 2 ? sm_count() / 2 : split_clusters(q.ks);
    const int nclu = (int)(tiles < most ? tiles : most);
    if (nclu == 0) return cudaSuccess;
    cudaError_t e = launch_dependent(tc_gemm_kernel<ST, SK>, (unsigned)(q.ks * nclu), GTHREADS,
                                     GL::SMEM, st, (unsigned)q.ks, A, B, B2, O, q);
    if (e != cudaSuccess) return e;
  }
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) count_launches(1);
  return e;
}

cudaError_t launch(const CUtensorMap& A, const CUtensorMap& B, const CUtensorMap& B2,
                   const CUtensorMap& O, const TcGemm& p, int zcount, cudaStream_t st) {
  TcGemm q = p;
  q.Z = zcount;
  const long long tiles =
      (long long)((p.M + GBM - 1) / GBM) * ((p.N + GBN - 1) / GBN) * zcount;
  const int nk = (p.K + GBK - 1) / GBK;
  // the absorption's tiles are two K-blocks long: two CTAs per SM hide their latency; so
  // do the materialisation's (eight K-blocks, but 1568 tiles; measured 2 % faster for the
  // whole non-absorbed call, while the up-projection measured slower that way)
  if (p.mode == MODE_ABSORB || p.mode == MODE_MAT)
    return launch_st<2, false>(A, B, B2, O, q, tiles, st);
  // Fewer tiles than SMs and a long K loop (the cache write): split K over CTA pairs; draft nodes'
  // rows, mostly a few tiles, over the number of CTAs with the shortest sequence of K blocks, a turn
  // after the first costing some 8 more, while each keeps a ring's worth.  Measured, us by 2 CTAs
  // / by the rule's, K = 4096, d_R = 64: 32 rows 16.0 / 8.6 (8 CTAs), 384 rows 16.3 / 11.0 (8), 1024
  // rows 17.6 / 14.7 (3).
  if (p.mode == MODE_CACHE && nk >= 2 && tiles < sm_count()) {
    q.ks = 2;
    if (p.window) {
      long long best = 0;
      for (int k : {2, 3, 4, 6, 8}) {
        if (k > 2 && nk < 4 * k) break;
        const long long at_once = k == 2 ? sm_count() / 2 : split_clusters(k);
        if (at_once == 0) continue;
        const long long turns = (tiles + at_once - 1) / at_once;
        const long long cost = turns * ((nk + k - 1) / k) + 8 * (turns - 1);
        if (best == 0 || cost < best) {
          best = cost;
          q.ks = k;
        }
      }
    }
    return launch_st<4, true>(A, B, B2, O, q, tiles, st);
  }
  return launch_st<4, false>(A, B, B2, O, q, tiles, st);
}

}  // namespace

bool tc_gemm_supported(const Geo& g, int d_model) {
  // every output width is a multiple of the epilogue's 32-column chunks
  return g.Dc % GBN == 0 && g.Dr % 64 == 0 && g.Dn % 64 == 0 && g.Dr / 2 <= MAX_PAIRS &&
         (d_model <= 0 || d_model % 64 == 0);
}

cudaError_t tc_cache_write(const Geo& g, const void* h, int d_model, int64_t n_tok,
                           int64_t first_tok, const void* w_dkv, const void* w_kr, void* cache,
                           int32_t* slots, const NodePlaces* at, unsigned int* err,
                           cudaStream_t st) {
  CUtensorMap A, B, B2;
  const uint64_t rows = (uint64_t)g.B * n_tok;
  {
    uint64_t d[3] = {(uint64_t)d_model, 1, rows};
    uint64_t s[2] = {(uint64_t)d_model * 2, (uint64_t)d_model * 2};
    uint32_t b[3] = {64, 1, 128};
    if (!make_tmap_bf16(&A, h, 3, d, s, b)) return cudaErrorInvalidValue;
  }
  {
    uint64_t d[3] = {(uint64_t)g.Dc, (uint64_t)d_model, 1};
    uint64_t s[2] = {(uint64_t)g.Dc * 2, (uint64_t)g.Dc * d_model * 2};
    uint32_t b[3] = {64, 64, 1};
    if (!make_tmap_bf16(&B, w_dkv, 3, d, s, b)) return cudaErrorInvalidValue;
  }
  if (g.Dr > 0) {
    uint64_t d[3] = {(uint64_t)g.Dr, (uint64_t)d_model, 1};
    uint64_t s[2] = {(uint64_t)g.Dr * 2, (uint64_t)g.Dr * d_model * 2};
    uint32_t b[3] = {64, 64, 1};
    if (!make_tmap_bf16(&B2, w_kr, 3, d, s, b)) return cudaErrorInvalidValue;
  } else {
    B2 = B;
  }
  TcGemm p{};
  p.M = (int)rows; p.N = g.row; p.K = d_model; p.mode = MODE_CACHE; p.b_mn = 1;
  p.n_split = g.Dc; p.out = (bf16*)cache; p.rows_per_batch = n_tok; p.geo = g;
  p.first_tok = first_tok; p.slots = slots; p.err = err;
  if (at) {
    p.window = at->window; p.token = at->token; p.position = at->position;
  }
  return launch(A, B, B2, B, p, 1, st);       // the cache write stores without TMA
}

cudaError_t tc_absorb_q(const Geo& g, const void* q_nope, const void* q_rope, int64_t n_q,
                        int64_t q_first, const int32_t* token, const void* w_uk, void* q_abs,
                        unsigned int* err, cudaStream_t st) {
  CUtensorMap A, B;
  const uint64_t rows = (uint64_t)g.B * n_q;
  {
    uint64_t d[3] = {(uint64_t)g.Dn, (uint64_t)g.H, rows};
    uint64_t s[2] = {(uint64_t)g.Dn * 2, (uint64_t)g.H * g.Dn * 2};
    uint32_t b[3] = {64, 1, 128};
    if (!make_tmap_bf16(&A, q_nope, 3, d, s, b)) return cudaErrorInvalidValue;
  }
  {
    uint64_t d[3] = {(uint64_t)g.Dc, (uint64_t)g.Dn, (uint64_t)g.H};
    uint64_t s[2] = {(uint64_t)g.Dc * 2, (uint64_t)g.Dc * g.Dn * 2};
    uint32_t b[3] = {64, 64, 1};
    if (!make_tmap_bf16(&B, w_uk, 3, d, s, b)) return cudaErrorInvalidValue;
  }
  TcGemm p{};
  p.M = (int)rows; p.N = g.Dc; p.K = g.Dn; p.mode = MODE_ABSORB; p.b_mn = 1;
  p.n_split = 1 << 30; p.out = (bf16*)q_abs; p.rows_per_batch = n_q; p.geo = g;
  p.first_tok = q_first; p.q_rope = (const bf16*)q_rope; p.token = token; p.err = err;
  CUtensorMap O;
  {
    // q_abs as (d_c + d_R, heads, rows): 64-column boxes of 128 rows of one head
    uint64_t d[3] = {(uint64_t)g.row, (uint64_t)g.H, rows};
    uint64_t s[2] = {(uint64_t)g.row * 2, (uint64_t)g.H * g.row * 2};
    uint32_t b[3] = {64, 1, (uint32_t)GBM};
    if (!make_tmap_bf16(&O, q_abs, 3, d, s, b)) return cudaErrorInvalidValue;
  }
  return launch(A, B, B, O, p, g.H, st);
}

cudaError_t tc_up_v(const Geo& g, const void* o_lat, int64_t n_q, const void* w_uv, void* out,
                    unsigned int* err, cudaStream_t st) {
  CUtensorMap A, B;
  const uint64_t rows = (uint64_t)g.B * n_q;
  {
    uint64_t d[3] = {(uint64_t)g.Dc, (uint64_t)g.H, rows};
    uint64_t s[2] = {(uint64_t)g.Dc * 2, (uint64_t)g.H * g.Dc * 2};
    uint32_t b[3] = {64, 1, 128};
    if (!make_tmap_bf16(&A, o_lat, 3, d, s, b)) return cudaErrorInvalidValue;
  }
  {
    uint64_t d[3] = {(uint64_t)g.Dc, (uint64_t)g.Dn, (uint64_t)g.H};
    uint64_t s[2] = {(uint64_t)g.Dc * 2, (uint64_t)g.Dc * g.Dn * 2};
    uint32_t b[3] = {64, (uint32_t)GBN, 1};
    if (!make_tmap_bf16(&B, w_uv, 3, d, s, b)) return cudaErrorInvalidValue;
  }
  TcGemm p{};
  p.M = (int)rows; p.N = g.Dn; p.K = g.Dc; p.mode = MODE_UPV; p.b_mn = 0;
  p.n_split = 1 << 30; p.out = (bf16*)out; p.rows_per_batch = n_q; p.geo = g; p.err = err;
  CUtensorMap O;
  {
    // out as (d_nope, heads, rows): 64-column boxes of 128 rows of one head
    uint64_t d[3] = {(uint64_t)g.Dn, (uint64_t)g.H, rows};
    uint64_t s[2] = {(uint64_t)g.Dn * 2, (uint64_t)g.H * g.Dn * 2};
    uint32_t b[3] = {64, 1, (uint32_t)GBM};
    if (!make_tmap_bf16(&O, out, 3, d, s, b)) return cudaErrorInvalidValue;
  }
  return launch(A, B, B, O, p, g.H, st);
}

cudaError_t tc_materialise(const Geo& g, const void* cache, const void* w, void* out,
                           unsigned int* err, cudaStream_t st) {
  CUtensorMap A, B;
  const uint64_t rows = (uint64_t)g.B * g.S;
  {
    // the latent columns of every cached row, as (d_latent, 1, slots)
    uint64_t d[3] = {(uint64_t)g.Dc, 1, rows};
    uint64_t s[2] = {(uint64_t)g.row * 2, (uint64_t)g.row * 2};
    uint32_t b[3] = {64, 1, 128};
    if (!make_tmap_bf16(&A, cache, 3, d, s, b)) return cudaErrorInvalidValue;
  }
  {
    uint64_t d[3] = {(uint64_t)g.Dc, (uint64_t)g.Dn, (uint64_t)g.H};
    uint64_t s[2] = {(uint64_t)g.Dc * 2, (uint64_t)g.Dc * g.Dn * 2};
    uint32_t b[3] = {64, (uint32_t)GBN, 1};
    if (!make_tmap_bf16(&B, w, 3, d, s, b)) return cudaErrorInvalidValue;
  }
  TcGemm p{};
  p.M = (int)rows; p.N = g.Dn; p.K = g.Dc; p.mode = MODE_MAT; p.b_mn = 0;
  p.n_split = 1 << 30; p.out = (bf16*)out; p.rows_per_batch = g.S; p.geo = g; p.err = err;
  CUtensorMap O;
  {
    // out as (d_nope, heads, slots): 64-column boxes of 128 slots of one head
    uint64_t d[3] = {(uint64_t)g.Dn, (uint64_t)g.H, rows};
    uint64_t s[2] = {(uint64_t)g.Dn * 2, (uint64_t)g.H * g.Dn * 2};
    uint32_t b[3] = {64, 1, (uint32_t)GBM};
    if (!make_tmap_bf16(&O, out, 3, d, s, b)) return cudaErrorInvalidValue;
  }
  return launch(A, B, B, O, p, g.H, st);
}

}  // namespace mla
