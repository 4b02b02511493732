// Definitions shared by the tensor-core attention kernel (tc_attend.cu) and the merge of
// its split-key partials (attend_combine.cu).
#pragma once

#include "launch.h"
#include "window.cuh"

namespace mla {
namespace attn {

constexpr int TM = 128;                               // rows per tile
constexpr int HALF = 256;                             // latent dims per CTA of a cluster
constexpr int MAXC = 128;                             // clusters one launch can schedule

struct AttnArgs {
  Geo g;
  int64_t n_q, q_first, k_first, n_keys;
  float scale_log2;
  const bf16* q_abs;
  bf16* o_lat;
  float* lse;
  bf16* ws_o;               // partial outputs [slot][TM][Dc], bf16, normalised by their l
  float* ws_f;              // draft trees: the same in float32
  float* ws_lse;            // their natural log-sum-exps, one per CTA half [slot][2][TM]
  int tiles_per_batch;
  int bn;                   // keys per block of the launch
  int pf;                   // L2 look-ahead of the key loads in blocks (0: none)
  float xthr;               // largest raw partial score magnitude a row's 16-bit score
                            // exchange carries; a row with a larger one is sent exactly
  // the low-bit ring (packed variant only): codes of both paths, per-row float32 scales
  const uint8_t* pk_c;      // [B][S][d_c * cbits / 8]
  const uint8_t* pk_r;      // [B][S][d_R * rbits / 8]
  const float* sc_c;        // [B][S]
  const float* sc_r;        // [B][S]
  int cbits, rbits;
  // draft trees: ragged windows (null otherwise), and which node sees which
  const int32_t* window;    // [B][3]
  const uint8_t* tree;      // [B][n_q][n_q] bytes, or null (a chain)
  int4* cuts;               // where each cluster's range starts: (sequence or -1: none, tile,
                            // block, cluster), [MAXC]
  uint32_t zero;            // 0, which the compiler does not know
  unsigned int* err;
};

// Key blocks of one tile: its rows see the keys k_first .. k_first + L - 1 (frame-
// block-causal bound of its last row), stored in the ring as two contiguous slot runs.
struct Blocks {
  int64_t k_first, p1, n1, L;
  int bn;                   // keys per block
  int nb1, nblk;
  // block j: first ring slot, first global token, number of keys
  __device__ void get(int j, int64_t& slot0, int64_t& g0, int& valid) const {
    if (j < nb1) {
      slot0 = p1 + (int64_t)j * bn;
      g0 = k_first + (int64_t)j * bn;
      const int64_t v = n1 - (int64_t)j * bn;
      valid = v < bn ? (int)v : bn;
    } else {
      const int64_t jj = j - nb1;
      slot0 = jj * bn;
      g0 = k_first + n1 + jj * bn;
      const int64_t v = L - n1 - jj * bn;
      valid = v < bn ? (int)v : bn;
    }
  }
};

struct TileGeo {
  int b;
  int64_t rows_b, row0, grow0, i_last;
  Blocks blk;
};

// one past the last key query i sees (frame-block-causal, clipped to the key window)
__host__ __device__ inline int64_t key_end(const Geo& G, int64_t q_first, int64_t k_lim,
                                           int64_t i) {
  const int64_t e = ((q_first + i) / G.F + 1) * G.F;
  return e < k_lim ? e : k_lim;
}

__host__ __device__ inline TileGeo tile_geo(const Geo& G, int64_t n_q, int64_t q_first,
                                            int64_t k_first, int64_t n_keys,
                                            int tiles_per_batch, int tile, int bn) {
  TileGeo t;
  t.b = tile / tiles_per_batch;
  const int tb = tile - t.b * tiles_per_batch;
  t.rows_b = n_q * G.H;
  t.row0 = (int64_t)tb * TM;
  t.grow0 = (int64_t)t.b * t.rows_b + t.row0;
  const int64_t last_row = (t.row0 + TM < t.rows_b ? t.row0 + TM : t.rows_b) - 1;
  t.i_last = last_row / G.H;
  Blocks& k = t.blk;
  k.k_first = k_first;
  k.L = key_end(G, q_first, k_first + n_keys, t.i_last) - k_first;
  k.p1 = k_first % G.S;
  k.n1 = k.L < G.S - k.p1 ? k.L : G.S - k.p1;
  k.bn = bn;
  k.nb1 = (int)((k.n1 + bn - 1) / bn);
  k.nblk = k.nb1 + (int)((k.L - k.n1 + bn - 1) / bn);
  return t;
}

// Draft trees: a sequence's tiles of 128 (node, head) rows, and the key blocks (context, then
// nodes) that each of them walks.
struct TreeBlocks {          // as Blocks, from logical row 0, in 32 bits (registers are short)
  int32_t p1, n1, L;
  int nb1, nblk;
  template <int BN>
  __device__ void get(int j, int& slot0, int& g0, int& valid) const {
    const bool second = j >= nb1;
    const int r = (second ? j - nb1 : j) * BN;
    const int v = (second ? L - n1 : n1) - r;
    slot0 = second ? r : p1 + r;
    g0 = second ? n1 + r : r;
    valid = v < BN ? v : BN;
  }
  __device__ void get(int j, int64_t& slot0, int64_t& g0, int& valid) const {
    int s, g;
    get<64>(j, s, g, valid);
    slot0 = s;
    g0 = g;
  }
};
struct TreeGeo {
  int32_t ctx;              // context rows
  int tiles;
  TreeBlocks blk;
};
struct TreeTile {            // as TileGeo
  int b, rows_b, row0, grow0;
  TreeBlocks blk;
};

// BN keys per block (a power of two).  Everything fits 32 bits: rows and slots are below 2^31.
template <int BN>
__device__ __forceinline__ TreeGeo tree_geo(const AttnArgs& a, const Window& w) {
  TreeGeo t;
  t.ctx = w.rows;
  t.tiles = (int)(((uint32_t)w.nodes * (uint32_t)a.g.H + (TM - 1)) / TM);
  const uint32_t L = (uint32_t)w.len(), run = (uint32_t)a.g.S - (uint32_t)w.first;
  const uint32_t n1 = L < run ? L : run;
  t.blk.p1 = w.first;
  t.blk.L = (int32_t)L;
  t.blk.n1 = (int32_t)n1;
  t.blk.nb1 = (int)((n1 + (BN - 1)) / BN);
  t.blk.nblk = t.blk.nb1 + (int)((L - n1 + (BN - 1)) / BN);
  return t;
}
template <int BN>
__device__ __forceinline__ TreeGeo tree_geo(const AttnArgs& a, int64_t b) {
  return tree_geo<BN>(a, load_window(a.window, b, a.g.S, a.n_q));
}

// A line of work: every sequence takes tiles x blocks positions of it, one after the other (sizes
// are checked by the host: the line is shorter than 2^31).  The functions below are
// warp-collective and every warp of every CTA calls them for itself before its first load, so
// they keep to registers and to little code: lane l looks at sequence l, l + 32, ...
struct Span {
  uint32_t tiles, blocks;
};
struct Spot {
  int b;                    // the sequence
  uint32_t start, off;      // where its positions start, and the position inside them
  Span s;
};

__device__ __forceinline__ uint32_t warp_scan(uint32_t v) {     // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

// The sequences that hold positions p[0] .. p[N - 1], each below the line's length; span(b) gives a
// sequence's sizes and `mine` is span(lane) (B > 0; zero sizes past the last sequence).
template <int N, typename F>
__device__ __forceinline__ void line_find(int B, const F& span, Span mine, const uint32_t (&p)[N],
                                          Spot (&at)[N]) {
  const int lane = threadIdx.x & 31;
  uint32_t before = 0;
  unsigned found = 0;
  for (int b0 = 0;; b0 += 32) {
    const uint32_t n = mine.tiles * mine.blocks, end = before + warp_scan(n);
    bool all = true;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const unsigned past = __ballot_sync(0xffffffffu, end > p[k]);
      if (past && !(found >> k & 1)) {
        found |= 1u << k;
        const int l = __ffs(past) - 1;
        at[k].b = b0 + l;
        at[k].start = __shfl_sync(0xffffffffu, end - n, l);
        at[k].off = p[k] - at[k].start;
        at[k].s.tiles = __shfl_sync(0xffffffffu, mine.tiles, l);
        at[k].s.blocks = __shfl_sync(0xffffffffu, mine.blocks, l);
      }
      all = all && past;
    }
    if (all || b0 + 32 >= B) return;           // (the latter only as a bound)
    before = __shfl_sync(0xffffffffu, end, 31);
    mine = b0 + 32 + lane < B ? span(b0 + 32 + lane) : Span{0, 0};
  }
}

// Split tiles to merge: tile[i] has the partial segments in workspace slots
// [piece0[i], piece0[i + 1]).
struct CombineList {
  int32_t n;
  int32_t tile[MAXC];
  int32_t piece0[MAXC + 1];
};

// Merge the partials of the tiles that mla_attend_tree's clusters split: cluster c's first
// segment left its partial in workspace slot 2 c, its last in 2 c + 1 (cuts: a.cuts, `clusters`
// of them).
cudaError_t launch_combine_tree(const AttnArgs& a, int clusters, cudaStream_t st);

// Merge the partials of the split tiles listed in `cl` into o_lat (and lse).
cudaError_t launch_combine(const AttnArgs& a, const CombineList& cl, cudaStream_t st);

}  // namespace attn
}  // namespace mla
