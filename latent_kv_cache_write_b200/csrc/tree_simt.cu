// Draft-tree attention and the attention weight of cached rows on CUDA cores: every dtype and
// shape (float32 storage uses it throughout, and bfloat16 shapes the tensor-core kernels do not
// take).  Accumulation is float32.  A block owns one row of the score matrix (attention) or one of
// its columns (weight); its warps share the keys (the queries), some at a time each, and join their
// sums in the order of the warps.  At the sizes float32 serves (a few heads, tens of rows) that is
// bound by the latency of one turn after the other (2 sequences of 57 rows, 7 nodes, 4 heads: 4.5
// us, weight 3.8; with one warp per row or column 15 and 12; 300 rows of 576, 16 heads: 26 against
// 184).
#include "launch.h"
#include "window.cuh"

namespace mla {
namespace {

constexpr int WIDE = 40, NARROW = 4;        // row width <= 32 * either
constexpr unsigned FULL = 0xffffffffu;

__device__ __forceinline__ float warp_sum(float s) {
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(FULL, s, o);
  return s;
}

// Elements lane, lane + 32, ... of a row of `width`; 0 past it.
template <typename T, int MAXR>
__device__ __forceinline__ void load_row(const T* row, int width, float (&v)[MAXR]) {
#pragma unroll
  for (int r = 0; r < MAXR; ++r) {
    const int d = (threadIdx.x & 31) + 32 * r;
    v[r] = d < width ? to_f32(row[d]) : 0.f;
  }
}

constexpr int NWARP = 8;

// One block per (sequence, node, head): online softmax over the visible rows, U at a time per warp.
// Hidden nodes are skipped, not masked, so nothing of their rows enters the sums.
template <typename T, int MAXR, int U>
__global__ void __launch_bounds__(32 * NWARP)
    attend_tree_simt_kernel(Geo g, const T* q_abs, int64_t n_nodes, const T* cache,
                            const int32_t* window, const uint8_t* tree, float scale, T* o_lat,
                            float* lse) {
  __shared__ float part[NWARP][32 * MAXR], ml[NWARP][2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.x;
  const int64_t i = blockIdx.y;
  const int b = blockIdx.z;
  const Window w = load_window(window, b, g.S, n_nodes);
  if (i >= w.nodes) return;
  const uint8_t* tb = tree ? tree + (int64_t)b * n_nodes * n_nodes : nullptr;
  const int64_t qrow = ((int64_t)b * n_nodes + i) * g.H + h;
  float qv[MAXR], acc[MAXR];
  load_row<T, MAXR>(q_abs + qrow * g.row, g.row, qv);
#pragma unroll
  for (int r = 0; r < MAXR; ++r) {
    qv[r] *= scale;
    acc[r] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const T* base = cache + (int64_t)b * g.S * g.row;
  for (int64_t j0 = warp * U; j0 < w.len(); j0 += NWARP * U) {
    float kv[U][MAXR], s[U];
    bool in[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t j = j0 + u;
      in[u] = j < w.rows || (j < w.len() && tree_sees(tb, n_nodes, i, j - w.rows));
      s[u] = 0.f;
      if (in[u]) {
        load_row<T, MAXR>(base + w.slot(j, g.S) * g.row, g.row, kv[u]);
      } else {
#pragma unroll
        for (int r = 0; r < MAXR; ++r) kv[u][r] = 0.f;
      }
#pragma unroll
      for (int r = 0; r < MAXR; ++r) s[u] = fmaf(qv[r], kv[u][r], s[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) s[u] = warp_sum(s[u]);
    float mn = m;
#pragma unroll
    for (int u = 0; u < U; ++u) mn = in[u] ? fmaxf(mn, s[u]) : mn;
    const float ref = mn == -INFINITY ? 0.f : mn;       // every score so far -inf
    const float corr = expf(m - ref);
    l *= corr;
#pragma unroll
    for (int r = 0; r < MAXR; ++r) acc[r] *= corr;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float p = in[u] ? expf(s[u] - ref) : 0.f;
      l += p;
#pragma unroll
      for (int r = 0; r < MAXR; ++r) acc[r] = fmaf(p, kv[u][r], acc[r]);
    }
    m = mn;
  }
  // join the warps' sums, each scaled from its own maximum to the common one
#pragma unroll
  for (int r = 0; r < MAXR; ++r)
    if (lane + 32 * r < g.Dc) part[warp][lane + 32 * r] = acc[r];
  if (lane == 0) {
    ml[warp][0] = m;
    ml[warp][1] = l;
  }
  __syncthreads();
  float top = -INFINITY, f[NWARP], sum = 0.f;
#pragma unroll
  for (int v = 0; v < NWARP; ++v) top = fmaxf(top, ml[v][0]);
  const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
  for (int v = 0; v < NWARP; ++v) {
    f[v] = expf(ml[v][0] - ref);
    sum = fmaf(f[v], ml[v][1], sum);
  }
  T* out = o_lat + qrow * g.Dc;
  const float inv = sum != 0.f ? 1.f / sum : 0.f;        // NaN stays NaN
  for (int d = threadIdx.x; d < g.Dc; d += 32 * NWARP) {
    float o = 0.f;
#pragma unroll
    for (int v = 0; v < NWARP; ++v) o = fmaf(f[v], part[v][d], o);
    out[d] = from_f32<T>(o * inv);
  }
  if (lse && threadIdx.x == 0) lse[qrow] = sum != 0.f ? top + logf(sum) : -INFINITY;
}

// One block per (sequence, row of the window), in turns: each warp keeps the row in registers while
// it walks its share of the queries, U at a time.
template <typename T, int MAXR, int U>
__global__ void __launch_bounds__(32 * NWARP)
    attend_weight_simt_kernel(Geo g, const T* q_abs, int64_t n_nodes, const T* cache,
                              const int32_t* window, const uint8_t* tree, float scale,
                              const float* lse, const float* qw, const float* win, float* wout) {
  __shared__ float part[2][NWARP];
  const int warp = threadIdx.x >> 5;
  const int b = blockIdx.y;
  const Window w = load_window(window, b, g.S, n_nodes);
  const uint8_t* tb = tree ? tree + (int64_t)b * n_nodes * n_nodes : nullptr;
  const int64_t q0 = (int64_t)b * n_nodes * g.H;
  const uint32_t queries = (uint32_t)w.nodes * g.H;       // below 2^31
  int turn = 0;
  for (int64_t j = blockIdx.x; j < w.len(); j += gridDim.x, turn ^= 1) {
    const int64_t at = (int64_t)b * g.S + w.slot(j, g.S);
    float kv[MAXR];
    load_row<T, MAXR>(cache + at * g.row, queries ? g.row : 0, kv);     // (not read for no one)
#pragma unroll
    for (int r = 0; r < MAXR; ++r) kv[r] *= scale;
    float total = 0.f;
    for (uint32_t x0 = warp * U; x0 < queries; x0 += NWARP * U) {
      float s[U], e[U], c[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t x = x0 + u, i = x / (uint32_t)g.H;
        s[u] = 0.f;
        c[u] = 0.f;
        e[u] = -INFINITY;
        if (x >= queries) continue;
        if (j < w.rows || tree_sees(tb, n_nodes, i, j - w.rows))
          c[u] = qw ? qw[(int64_t)b * n_nodes + i] : 1.f;
        e[u] = lse[q0 + x];
        float qv[MAXR];
        load_row<T, MAXR>(q_abs + (q0 + x) * g.row, g.row, qv);
#pragma unroll
        for (int r = 0; r < MAXR; ++r) s[u] = fmaf(qv[r], kv[r], s[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) s[u] = warp_sum(s[u]);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c[u] != 0.f && e[u] != -INFINITY) total = fmaf(c[u], expf(s[u] - e[u]), total);
    }
    if ((threadIdx.x & 31) == 0) part[turn][warp] = total;
    __syncthreads();                           // (the other half is the next turn's)
    if (threadIdx.x == 0) {
      total = 0.f;
#pragma unroll
      for (int v = 0; v < NWARP; ++v) total += part[turn][v];
      wout[at] = (j < w.rows && win ? win[at] : 0.f) + total;
    }
  }
}

template <typename T>
void launch_attend(const Geo& g, const void* q_abs, int64_t n_nodes, const void* cache,
                   const int32_t* window, const uint8_t* tree, float scale, void* o_lat, float* lse,
                   cudaStream_t st) {
  const dim3 grid(g.H, (unsigned)n_nodes, g.B);
  auto run = [&](auto kern) {
    kern<<<grid, 32 * NWARP, 0, st>>>(g, (const T*)q_abs, n_nodes, (const T*)cache, window, tree,
                                      scale, (T*)o_lat, lse);
  };
  // rows of up to 128 elements leave registers for eight keys at a time
  if (g.row <= 32 * NARROW)
    run(attend_tree_simt_kernel<T, NARROW, 8>);
  else
    run(attend_tree_simt_kernel<T, WIDE, 1>);
}

template <typename T>
void launch_weight(const Geo& g, const void* q_abs, int64_t n_nodes, const void* cache,
                   const int32_t* window, const uint8_t* tree, float scale, const float* lse,
                   const float* qw, const float* win, float* wout, cudaStream_t st) {
  const dim3 grid((unsigned)(g.S < 4096 ? g.S : 4096), g.B);
  auto run = [&](auto kern) {
    kern<<<grid, 32 * NWARP, 0, st>>>(g, (const T*)q_abs, n_nodes, (const T*)cache, window, tree,
                                      scale, lse, qw, win, wout);
  };
  if (g.row <= 32 * NARROW)
    run(attend_weight_simt_kernel<T, NARROW, 4>);
  else
    run(attend_weight_simt_kernel<T, WIDE, 2>);
}

}  // namespace

cudaError_t simt_attend_tree(const Geo& g, bool bf, const void* q_abs, int64_t n_nodes,
                             const void* cache, const int32_t* window, const uint8_t* tree,
                             float scale, void* o_lat, float* lse, cudaStream_t st) {
  if (bf)
    launch_attend<bf16>(g, q_abs, n_nodes, cache, window, tree, scale, o_lat, lse, st);
  else
    launch_attend<float>(g, q_abs, n_nodes, cache, window, tree, scale, o_lat, lse, st);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) count_launches(1);
  return e;
}

cudaError_t simt_attend_weight(const Geo& g, bool bf, const void* q_abs, int64_t n_nodes,
                               const void* cache, const int32_t* window, const uint8_t* tree,
                               float scale, const float* lse, const float* qw, const float* win,
                               float* wout, cudaStream_t st) {
  if (bf)
    launch_weight<bf16>(g, q_abs, n_nodes, cache, window, tree, scale, lse, qw, win, wout, st);
  else
    launch_weight<float>(g, q_abs, n_nodes, cache, window, tree, scale, lse, qw, win, wout, st);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace mla
