// Moving rows up when others leave: the accepted nodes of a draft tree, and eviction of the
// context rows that attention has used least.
//
// Both come down to the same step.  Of the logical rows base .. base + n - 1 some stay, `count` of
// them; the ones that leave and lie below base + count are holes, and there are exactly as many
// staying rows at base + count and beyond.  The k-th such row moves into the k-th hole.  Every
// source lies at or past base + count and every hole below it, so the rows can move in place and
// in any order, and no more rows move than have to (a stable compaction would move every row behind
// the first hole).  The order of the rows does not matter to the attention: a cached key carries
// its rotation, and the position array moves along.
//
// Two launches: one block per sequence chooses the rows and lists the moves (latency-bound: a radix
// selection over the sequence's weights in shared memory, then two block scans), and the whole GPU
// copies the listed rows (bound by HBM: each moved row is read and written once).
#include "launch.h"
#include "window.cuh"

namespace mla {
namespace {

constexpr int NT = 1024;                    // threads of a planning block
constexpr unsigned FULL = 0xffffffffu;

// Workspace: counts [B] (padded to 4), then per sequence `cap` destination and `cap` source slots.
struct Plan {
  int32_t* count;
  int32_t* move;                            // [B][2][cap]
  int64_t cap;
};

__host__ __device__ inline int64_t plan_cap(int64_t S) { return S / 2 + 1; }

struct EvictArgs {
  int64_t S, n_nodes, n_keep;
  int32_t n_sink, n_recent;
  const uint8_t* accept;                    // accept: [B, n_nodes]; null for evict
  int32_t* window;
  const float* weight;
  const int32_t* position;
  Plan plan;
};

// Order of a weight as an unsigned number: larger weights larger, -0 as +0, NaN below all.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive sum over the block's threads of v, and the total.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* warp_sums, uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(FULL, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    uint32_t s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(FULL, s, o);
      if (lane >= o) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  const uint32_t before = warp ? warp_sums[warp - 1] : 0u;
  *total = warp_sums[31];
  __syncthreads();
  return before + x - v;
}

__global__ void __launch_bounds__(NT) evict_plan_kernel(EvictArgs a) {
  __shared__ uint32_t hist[2048];
  __shared__ uint32_t warp_sums[32];
  __shared__ uint32_t pick[2];              // chosen digit, rows still to take inside it
  __shared__ int newest_sh;
  const int b = blockIdx.x, t = threadIdx.x;
  const Window w = load_window(a.window, b, a.S, a.accept ? a.n_nodes : a.S);
  const int32_t* pos = a.position + (int64_t)b * a.S;
  const float* wt = a.weight + (int64_t)b * a.S;
  int32_t* dst = a.plan.move + (int64_t)b * 2 * a.plan.cap;
  int32_t* src = dst + a.plan.cap;

  int64_t base, n, count;                   // logical rows considered, and how many stay
  uint32_t thr = 0, ties = 0;
  int newest = 0;
  // evict: does logical row j outrank the threshold, or tie with it
  auto key = [&](int64_t j) -> uint32_t {
    const int64_t s = w.slot(j, a.S);
    const int32_t p = pos[s];
    if (p < a.n_sink || (int64_t)p > (int64_t)newest - a.n_recent) return 0xFFFFFFFFu;
    return weight_key(wt[s]);
  };

  if (a.accept) {
    base = w.rows;
    n = w.nodes;
    count = 0;
  } else {
    base = 0;
    n = w.rows;
    count = a.n_keep;
    if (n <= a.n_keep) {                    // the whole block agrees: nothing leaves
      __syncthreads();
      if (t == 0) {
        a.plan.count[b] = 0;
        a.window[3 * b] = w.first;
        a.window[3 * b + 1] = w.rows;
        a.window[3 * b + 2] = 0;
      }
      return;
    }
    if (t == 0) newest_sh = INT32_MIN;
    __syncthreads();
    int mx = INT32_MIN;
    for (int64_t j = t; j < n; j += NT) mx = max(mx, pos[w.slot(j, a.S)]);
    mx = __reduce_max_sync(FULL, mx);
    if ((t & 31) == 0) atomicMax(&newest_sh, mx);
    __syncthreads();
    newest = newest_sh;
    // the n_keep-th largest key, 11 + 11 + 10 bits at a time (11 bits take the exponent and two
    // mantissa bits at once: weights crowd in few exponents)
    uint32_t prefix = 0, take = (uint32_t)a.n_keep;
    const int shift[3] = {21, 10, 0}, bits[3] = {11, 11, 10};
    if (a.n_keep > 0) {
      for (int pass = 0; pass < 3; ++pass) {
        for (int q = t; q < 2048; q += NT) hist[q] = 0u;
        __syncthreads();
        const uint32_t mask = (1u << bits[pass]) - 1u;
        const int above = shift[pass] + bits[pass];
        for (int64_t j = t; j < n; j += NT) {
          const uint32_t k = key(j);
          if (above == 32 || (k >> above) == prefix) atomicAdd(&hist[(k >> shift[pass]) & mask], 1u);
        }
        __syncthreads();
        // thread t owns digits 2047 - 2t and 2046 - 2t: rows above them by an exclusive scan
        const uint32_t h0 = hist[2047 - 2 * t], h1 = hist[2046 - 2 * t];
        uint32_t total;
        const uint32_t before = block_scan(h0 + h1, warp_sums, &total);
        if (before < take && take <= before + h0 + h1) {
          const bool first = take <= before + h0;
          pick[0] = (uint32_t)(first ? 2047 - 2 * t : 2046 - 2 * t);
          pick[1] = take - before - (first ? 0u : h0);
        }
        __syncthreads();
        prefix = (prefix << bits[pass]) | pick[0];
        take = pick[1];
        __syncthreads();
      }
    }
    thr = prefix;
    ties = take;                            // rows at the threshold that stay: the lowest ones
  }

  // Each thread takes a run of consecutive rows, so that one scan orders them.
  const int64_t per = (n + NT - 1) / NT;
  const int64_t j0 = t * per < n ? t * per : n, j1 = j0 + per < n ? j0 + per : n;
  uint32_t tie0 = 0, total;
  if (a.accept) {
    const uint8_t* acc = a.accept + (int64_t)b * a.n_nodes;
    uint32_t c = 0;
    for (int64_t j = j0; j < j1; ++j) c += acc[j] != 0;
    block_scan(c, warp_sums, &total);
    count = total;
  } else if (a.n_keep > 0) {
    uint32_t c = 0;
    for (int64_t j = j0; j < j1; ++j) c += key(j) == thr;
    tie0 = block_scan(c, warp_sums, &total);
  }
  auto stays = [&](int64_t j, uint32_t& tie) -> bool {
    if (a.accept) return a.accept[(int64_t)b * a.n_nodes + j] != 0;
    if (a.n_keep == 0) return false;
    const uint32_t k = key(j);
    if (k == thr) return tie++ < ties;
    return k > thr;
  };
  // holes below count (low half) and staying rows past it (high half): at most 2^15 of each per
  // thread would be needed to mix them, but the block totals need 32 bits, so two scans
  uint32_t holes = 0, late = 0, tie = tie0;
  for (int64_t j = j0; j < j1; ++j) {
    const bool s = stays(j, tie);
    holes += j < count && !s;
    late += j >= count && s;
  }
  uint32_t n_move, n_late;
  uint32_t hole = block_scan(holes, warp_sums, &n_move);
  uint32_t lt = block_scan(late, warp_sums, &n_late);
  tie = tie0;
  for (int64_t j = j0; j < j1; ++j) {
    const bool s = stays(j, tie);
    if (j < count && !s) dst[hole++] = (int32_t)w.slot(base + j, a.S);
    if (j >= count && s) src[lt++] = (int32_t)w.slot(base + j, a.S);
  }
  if (t == 0) {
    a.plan.count[b] = (int32_t)n_move;
    a.window[3 * b] = w.first;
    a.window[3 * b + 1] = (int32_t)(base + count);
    a.window[3 * b + 2] = 0;
  }
}

// Copy the listed rows: blockIdx.y is the sequence; its blocks' threads take the rows' vectors
// in turn.
template <typename V>
__global__ void __launch_bounds__(256)
    evict_move_kernel(int64_t S, int per_row, V* cache, float* weight, int32_t* position,
                      Plan plan) {
  const int b = blockIdx.y;
  const int64_t n = plan.count[b];
  const int32_t* dst = plan.move + (int64_t)b * 2 * plan.cap;
  const int32_t* src = dst + plan.cap;
  V* rows = cache + (int64_t)b * S * per_row;
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  const int64_t t = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  for (int64_t k = t; k < n; k += step) {
    const int64_t d = b * S + dst[k], s = b * S + src[k];
    if (weight) weight[d] = weight[s];
    if (position) position[d] = position[s];
  }
  for (int64_t e = t; e < n * per_row; e += step) {
    const int64_t k = e / per_row;
    const int c = (int)(e - k * per_row);
    rows[(int64_t)dst[k] * per_row + c] = rows[(int64_t)src[k] * per_row + c];
  }
}

cudaError_t run(const Geo& g, bool bf, void* cache, float* weight, int32_t* position,
                const EvictArgs& a, cudaStream_t st) {
  evict_plan_kernel<<<g.B, NT, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  count_launches(1);
  const int bytes = g.row * (bf ? 2 : 4);
  const int x = (148 * 8 + g.B - 1) / g.B;
  const dim3 grid((unsigned)x, (unsigned)g.B);
  if (bytes % 16 == 0)
    evict_move_kernel<uint4><<<grid, 256, 0, st>>>(g.S, bytes / 16, (uint4*)cache, weight, position,
                                                   a.plan);
  else                                      // rows are an even number of 2- or 4-byte elements
    evict_move_kernel<uint32_t><<<grid, 256, 0, st>>>(g.S, bytes / 4, (uint32_t*)cache, weight,
                                                      position, a.plan);
  e = cudaGetLastError();
  if (e == cudaSuccess) count_launches(1);
  return e;
}

Plan make_plan(const Geo& g, void* workspace) {
  Plan p;
  p.count = static_cast<int32_t*>(workspace);
  p.move = p.count + ((g.B + 3) / 4) * 4;
  p.cap = plan_cap(g.S);
  return p;
}

}  // namespace

size_t evict_workspace(const Geo& g) {
  return (size_t)(((g.B + 3) / 4) * 4 + (int64_t)g.B * 2 * plan_cap(g.S)) * sizeof(int32_t);
}

cudaError_t tree_accept(const Geo& g, bool bf, void* cache, int64_t n_nodes, const uint8_t* accept,
                        int32_t* window, float* weight, int32_t* position, void* workspace,
                        cudaStream_t st) {
  EvictArgs a{};
  a.S = g.S; a.n_nodes = n_nodes; a.accept = accept; a.window = window;
  a.weight = weight; a.position = position; a.plan = make_plan(g, workspace);
  return run(g, bf, cache, weight, position, a, st);
}

cudaError_t cache_evict(const Geo& g, bool bf, void* cache, int64_t n_keep, int32_t n_sink,
                        int32_t n_recent, int32_t* window, float* weight, int32_t* position,
                        void* workspace, cudaStream_t st) {
  EvictArgs a{};
  a.S = g.S; a.n_keep = n_keep; a.n_sink = n_sink; a.n_recent = n_recent; a.window = window;
  a.weight = weight; a.position = position; a.plan = make_plan(g, workspace);
  return run(g, bf, cache, weight, position, a, st);
}

}  // namespace mla
