// Merge of the split-key partials of the tensor-core attention: a tile whose key blocks
// were cut between clusters left one normalised partial output (bf16; of draft trees float32)
// and one fp32 log-sum-exp per CTA half for each piece in the workspace.
#include "attend_common.cuh"
#include "launch.h"
#include "tc_ptx.cuh"

namespace mla {
namespace attn {
namespace {

using tc::pack_bf16;

// CSPLIT warps per row of a split tile, 8 / CSPLIT rows per CTA: warp k of a row merges
// pieces k, k + CSPLIT, ... (with several warps per row, the loads of four pieces, of float32 two, in
// flight at a time) and the row's warps add their sums in shared memory.  One warp per
// row suits tiles cut in a few pieces (the chunk shapes); more suit a tile cut across
// every cluster (decode of a few sequences).  A lane holds 16 latent dims (d_c = 512): of bf16
// pieces [16 l, 16 l + 16), of float32 ones 4 of each 128, so that a warp's access is one run of
// bytes either way.  The output is the partials weighted by exp(lse_p - lse),
// lse = log sum_p exp(lse_p), each half of the dims with the log-sum-exps of the CTA half
// that computed it.
//
// Row r of the tile (if row_ok) becomes row grow of the outputs; piece p of np is in workspace
// slot slot(p).  TREE: the pieces are float32, so that a row is rounded once however many pieces it
// came in, and a NaN piece makes the row NaN (a node that sees a NaN row); otherwise they are bf16, and
// a NaN piece counts as empty.
template <int CSPLIT, bool TREE, typename Slot>
__device__ __forceinline__ void combine_row(const AttnArgs& a, const float* ws_lse, float* red,
                                            int rr, int part, int lane, int r, bool row_ok,
                                            int64_t grow, int np, const Slot& slot) {
  // 16-byte vectors of a piece per lane, and the halves (of the CTAs that computed them) they are in
  constexpr int NV = TREE ? 4 : 2, NH = TREE ? 2 : 1;
  const int d = TREE ? lane * 4 : lane * 16, step = TREE ? 128 : 8;      // vector q: dims d + q step ..
  const int half = TREE ? 0 : d / HALF;      // (TREE: vectors 0, 1 are in half 0, 2 and 3 in half 1)
  // each half's largest log-sum-exp over the row's pieces, the lanes taking pieces in turn
  float m0 = -INFINITY, m1 = -INFINITY;
  bool nan = false;
  if (row_ok)
    for (int p = lane; p < np; p += 32) {
      const float l0 = ws_lse[((int64_t)slot(p) * 2) * TM + r];
      const float l1 = ws_lse[((int64_t)slot(p) * 2 + 1) * TM + r];
      m0 = fmaxf(m0, l0);
      m1 = fmaxf(m1, l1);
      if (TREE) nan = nan || l0 != l0 || l1 != l1;
    }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
    m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
  }
  float mx[NH], wsum[NH];
  mx[0] = half ? m1 : m0;
  if constexpr (TREE) {
    mx[1] = m1;
    if (__any_sync(0xffffffffu, nan))
      for (int h = 0; h < NH; ++h) mx[h] = mx[h] == -INFINITY ? 0.f : mx[h];
  }
#pragma unroll
  for (int h = 0; h < NH; ++h) wsum[h] = 0.f;
  const float* lse_h = ws_lse + half * TM + r;   // + slot * 2 * TM, + TM: the next half
  float acc[16];
#pragma unroll
  for (int q = 0; q < 16; ++q) acc[q] = 0.f;
  auto load = [&](int64_t ps, float (&lp)[NH], uint4 (&v)[NV]) {
#pragma unroll
    for (int h = 0; h < NH; ++h) lp[h] = lse_h[(ps * 2 + h) * TM];
    const int64_t at = (ps * TM + r) * a.g.Dc + d;
#pragma unroll
    for (int q = 0; q < NV; ++q)
      v[q] = TREE ? *reinterpret_cast<const uint4*>(a.ws_f + at + q * step)
                  : *reinterpret_cast<const uint4*>(a.ws_o + at + q * step);
  };
  auto add = [&](const float (&lp)[NH], const uint4 (&v)[NV]) {
    float wh[NH];
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      wh[h] = (TREE ? lp[h] != -INFINITY : lp[h] > -INFINITY) ? expf(lp[h] - mx[h]) : 0.f;
      wsum[h] += wh[h];
    }
#pragma unroll
    for (int q = 0; q < NV; ++q) {
      const uint32_t u[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
      const float w = wh[TREE ? q / 2 : 0];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (TREE) {
          acc[4 * q + e] += w * __uint_as_float(u[e]);
        } else {
          acc[8 * q + 2 * e] += w * __uint_as_float(u[e] << 16);
          acc[8 * q + 2 * e + 1] += w * __uint_as_float(u[e] & 0xffff0000u);
        }
      }
    }
  };
  if (row_ok && (TREE || mx[0] > -INFINITY)) {
    int p = part;
    if constexpr (CSPLIT > 1) {
      constexpr int U = TREE ? 2 : 4;                // pieces in flight: 128 bytes a lane
      for (; p + (U - 1) * CSPLIT < np; p += U * CSPLIT) {
        float lp[U][NH];
        uint4 v[U][NV];
#pragma unroll
        for (int u = 0; u < U; ++u) load(slot(p + u * CSPLIT), lp[u], v[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) add(lp[u], v[u]);
      }
    }
    for (; p < np; p += CSPLIT) {
      float lp[NH];
      uint4 v[NV];
      load(slot(p), lp, v);
      add(lp, v);
    }
  }
  if constexpr (CSPLIT > 1) {
    constexpr int RED = TREE ? 19 : 17;            // (odd: free of bank conflicts)
    float* mine = red + ((rr * CSPLIT + part) * 32 + lane) * RED;
#pragma unroll
    for (int q = 0; q < 16; ++q) mine[q] = acc[q];
#pragma unroll
    for (int h = 0; h < NH; ++h) mine[16 + h] = wsum[h];
    __syncthreads();
    if (part != 0 || !row_ok) return;
    for (int k = 1; k < CSPLIT; ++k) {
      const float* other = red + ((rr * CSPLIT + k) * 32 + lane) * RED;
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[q] += other[q];
#pragma unroll
      for (int h = 0; h < NH; ++h) wsum[h] += other[16 + h];
    }
  } else {
    if (!row_ok) return;
  }
  bool any[NH];
  float inv[NH];
#pragma unroll
  for (int h = 0; h < NH; ++h) {
    any[h] = TREE ? wsum[h] != 0.f : wsum[h] > 0.f;
    inv[h] = any[h] ? 1.f / wsum[h] : 0.f;
  }
  uint32_t w[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const float f = inv[TREE ? q / 4 : 0];
    w[q] = pack_bf16(acc[2 * q] * f, acc[2 * q + 1] * f);
  }
  bf16* dst = a.o_lat + grow * a.g.Dc + d;
#pragma unroll
  for (int q = 0; q < NV; ++q) {
    if constexpr (TREE)
      *reinterpret_cast<uint2*>(dst + q * step) = make_uint2(w[2 * q], w[2 * q + 1]);
    else
      *reinterpret_cast<uint4*>(dst + q * step) =
          make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
  }
  if (lane == 0 && a.lse) a.lse[grow] = any[0] ? mx[0] + logf(wsum[0]) : -INFINITY;
}

template <int CSPLIT>
__global__ void __launch_bounds__(256)
    combine_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CombineList cl) {
  constexpr int CROWS = 8 / CSPLIT;
  __shared__ float red[CSPLIT > 1 ? 8 * 32 * 17 : 1];     // [row][warp][lane][16 sums + w]
  tc::grid_dep_wait();                             // the attention's partials are visible
  tc::grid_dep_launch();
  const int i = blockIdx.x / (TM / CROWS);
  const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rr = wid / CSPLIT, part = wid % CSPLIT;
  const int r = (blockIdx.x % (TM / CROWS)) * CROWS + rr;
  const TileGeo tg =
      tile_geo(a.g, a.n_q, a.q_first, a.k_first, a.n_keys, a.tiles_per_batch, cl.tile[i], a.bn);
  const int p0 = cl.piece0[i];
  combine_row<CSPLIT, false>(a, a.ws_lse, red, rr, part, lane, r, tg.row0 + r < tg.rows_b, tg.grow0 + r,
                             cl.piece0[i + 1] - p0, [&](int p) { return p0 + p; });
}

// Draft trees: the clusters' cuts are known on the device only.  cut[i] is where the range of the
// i-th cluster that has one starts (sequence, tile, block, cluster).  It splits a tile when it lies
// inside it; the first such cut of a tile stands for the tile, whose pieces are the segment of the
// cluster before that reached the cut and the first segments of the clusters that start inside it.
// Every block lists the split tiles for itself (at most MAXC cuts) and the grid takes their rows in
// turn.
template <int CSPLIT>
__device__ __forceinline__ void combine_tiles(const AttnArgs& a, const float* ws_lse, float* red,
                                              const int4* cut, const int* first,
                                              const int* pieces, int n) {
  constexpr int CROWS = 8 / CSPLIT;
  const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rr = wid / CSPLIT, part = wid % CSPLIT;
  for (int it = blockIdx.x; it < n * (TM / CROWS); it += gridDim.x) {
    const int e = it / (TM / CROWS), i = first[e];
    const int r = (it % (TM / CROWS)) * CROWS + rr;
    const int4 c = cut[i], before = cut[i - 1];
    const Window w = load_window(a.window, c.x, a.g.S, a.n_q);
    const int64_t row = (int64_t)c.y * TM + r;
    // the segment before the cut is its cluster's first when that cluster starts this tile
    const int s0 = 2 * before.w + (before.x == c.x && before.y == c.y ? 0 : 1);
    combine_row<CSPLIT, true>(a, ws_lse, red, rr, part, lane, r, row < (int64_t)w.nodes * a.g.H,
                              (int64_t)c.x * a.n_q * a.g.H + row, pieces[e],
                              [&](int p) { return p == 0 ? s0 : 2 * cut[i + p - 1].w; });
    if (CSPLIT > 1) __syncthreads();               // `red` is the next row's
  }
}

__global__ void __launch_bounds__(256, 2)
    combine_tree_kernel(const __grid_constant__ AttnArgs a, int clusters) {
  __shared__ float red[8 * 32 * 19];
  __shared__ int4 cut[MAXC + 1];
  __shared__ int first[MAXC], pieces[MAXC];
  __shared__ int n_sh, most_sh;
  const int t = threadIdx.x;
  tc::grid_dep_wait();                             // the attention's partials are visible
  tc::grid_dep_launch();
  if (t < 32) {
    // the cuts of the clusters that have a range, four per lane
    int4 c[MAXC / 32];
#pragma unroll
    for (int q = 0; q < MAXC / 32; ++q)
      c[q] = 32 * q + t < clusters ? a.cuts[32 * q + t] : make_int4(-1, 0, 0, 0);
    unsigned split = 0;
#pragma unroll
    for (int q = 0; q < MAXC / 32; ++q) split |= (unsigned)(c[q].x >= 0 && c[q].z > 0);
    if (t == 0) n_sh = most_sh = 0;
    if (__any_sync(0xffffffffu, split)) {
      int ranges = 0;
#pragma unroll
      for (int q = 0; q < MAXC / 32; ++q) {
        const unsigned m = __ballot_sync(0xffffffffu, c[q].x >= 0);
        if (c[q].x >= 0) cut[ranges + __popc(m & ((1u << t) - 1u))] = c[q];
        ranges += __popc(m);
      }
      if (t == 0) cut[ranges] = make_int4(-1, 0, 0, 0);
      __syncwarp();
      int n = 0, most = 0;
      for (int i0 = 0; i0 < ranges; i0 += 32) {
        const int i = i0 + t;
        // a cut inside a tile has a block > 0; the tile's first one stands for it
        bool is = i > 0 && i < ranges && cut[i].z > 0;
        if (is) is = !(cut[i - 1].z > 0 && cut[i - 1].x == cut[i].x && cut[i - 1].y == cut[i].y);
        const unsigned m = __ballot_sync(0xffffffffu, is);
        if (is) {
          int k = i + 1;
          while (cut[k].z > 0 && cut[k].x == cut[i].x && cut[k].y == cut[i].y) ++k;
          const int e = n + __popc(m & ((1u << t) - 1u));
          first[e] = i;
          pieces[e] = k - i + 1;
          most = max(most, k - i + 1);
        }
        n += __popc(m);
      }
      most = __reduce_max_sync(0xffffffffu, most);
      if (t == 0) {
        n_sh = n;
        most_sh = most;
      }
    }
  }
  __syncthreads();
  if (most_sh >= 32)
    combine_tiles<8>(a, a.ws_lse, red, cut, first, pieces, n_sh);
  else if (most_sh >= 8)
    combine_tiles<4>(a, a.ws_lse, red, cut, first, pieces, n_sh);
  else
    combine_tiles<1>(a, a.ws_lse, red, cut, first, pieces, n_sh);
}

}  // namespace

cudaError_t launch_combine(const AttnArgs& a, const CombineList& cl, cudaStream_t st) {
  if (cl.n == 0) return cudaSuccess;
  int most = 0;                                    // the most pieces of one tile
  for (int k = 0; k < cl.n; ++k)
    most = cl.piece0[k + 1] - cl.piece0[k] > most ? cl.piece0[k + 1] - cl.piece0[k] : most;
  if (most >= 32)
    return launch_dependent(combine_kernel<8>, (unsigned)(cl.n * TM), 256, 0, st, 1u, a, cl);
  if (most >= 8)
    return launch_dependent(combine_kernel<4>, (unsigned)(cl.n * (TM / 2)), 256, 0, st, 1u, a, cl);
  return launch_dependent(combine_kernel<1>, (unsigned)(cl.n * (TM / 8)), 256, 0, st, 1u, a, cl);
}

cudaError_t launch_combine_tree(const AttnArgs& a, int clusters, cudaStream_t st) {
  // two blocks per SM: enough loads in flight, and few blocks to start when nothing was split
  return launch_dependent(combine_tree_kernel, 148u * 2u, 256, 0, st, 1u, a, clusters);
}

}  // namespace attn
}  // namespace mla
