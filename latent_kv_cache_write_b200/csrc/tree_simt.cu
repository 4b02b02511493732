// Draft-tree attention and the attention weight of cached rows on CUDA cores: every dtype and
// shape (float32 storage uses it throughout, and bfloat16 shapes the tensor-core kernels do not
// take).  Accumulation is float32.  A warp owns one row of the score matrix (attention) or one of
// its columns (weight) and walks it in order.  At the sizes float32 serves (a few heads, tens of
// rows) that is bound by the latency of one dot product after the other, so rows of up to 128
// elements take eight at a time (57 rows, 4 heads: 32 -> 10 us); wider rows fill the registers
// one by one.
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

// One warp per (sequence, node, head): online softmax over the visible rows, U at a time.  Hidden
// nodes are skipped, not masked, so nothing of their rows enters the sums.
template <typename T, int MAXR, int U>
__global__ void __launch_bounds__(256)
    attend_tree_simt_kernel(Geo g, const T* q_abs, int64_t n_nodes, const T* cache,
                            const int32_t* window, const uint8_t* tree, float scale, T* o_lat,
                            float* lse) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.x * 8 + warp;
  const int64_t i = blockIdx.y;
  const int b = blockIdx.z;
  if (h >= g.H) return;
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
  for (int64_t j0 = 0; j0 < w.len(); j0 += U) {
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
  T* out = o_lat + qrow * g.Dc;
  const float inv = l != 0.f ? 1.f / l : 0.f;            // NaN stays NaN
#pragma unroll
  for (int r = 0; r < MAXR; ++r) {
    const int d = lane + 32 * r;
    if (d < g.Dc) out[d] = from_f32<T>(acc[r] * inv);
  }
  if (lse && lane == 0) lse[qrow] = l != 0.f ? m + logf(l) : -INFINITY;
}

// One warp per (sequence, row of the window): the row stays in registers while the warp walks
// the queries in order, U heads at a time.
template <typename T, int MAXR, int U>
__global__ void __launch_bounds__(256)
    attend_weight_simt_kernel(Geo g, const T* q_abs, int64_t n_nodes, const T* cache,
                              const int32_t* window, const uint8_t* tree, float scale,
                              const float* lse, const float* qw, const float* win, float* wout) {
  const int lane = threadIdx.x & 31;
  const int64_t j = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int b = blockIdx.y;
  const Window w = load_window(window, b, g.S, n_nodes);
  if (j >= w.len()) return;
  const uint8_t* tb = tree ? tree + (int64_t)b * n_nodes * n_nodes : nullptr;
  const int64_t at = (int64_t)b * g.S + w.slot(j, g.S);
  float kv[MAXR];
  load_row<T, MAXR>(cache + at * g.row, g.row, kv);
#pragma unroll
  for (int r = 0; r < MAXR; ++r) kv[r] *= scale;
  float total = 0.f;
  for (int64_t i = 0; i < w.nodes; ++i) {
    const float c = qw ? qw[(int64_t)b * n_nodes + i] : 1.f;
    if (c == 0.f || (j >= w.rows && !tree_sees(tb, n_nodes, i, j - w.rows))) continue;
    const int64_t q0 = ((int64_t)b * n_nodes + i) * g.H;
    for (int h0 = 0; h0 < g.H; h0 += U) {
      float s[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        s[u] = 0.f;
        if (h0 + u < g.H) {
          float qv[MAXR];
          load_row<T, MAXR>(q_abs + (q0 + h0 + u) * g.row, g.row, qv);
#pragma unroll
          for (int r = 0; r < MAXR; ++r) s[u] = fmaf(qv[r], kv[r], s[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) s[u] = warp_sum(s[u]);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (h0 + u >= g.H) break;
        const float e = lse[q0 + h0 + u];
        if (e != -INFINITY) total = fmaf(c, expf(s[u] - e), total);
      }
    }
  }
  if (lane == 0) wout[at] = (j < w.rows && win ? win[at] : 0.f) + total;
}

template <typename T>
void launch_attend(const Geo& g, const void* q_abs, int64_t n_nodes, const void* cache,
                   const int32_t* window, const uint8_t* tree, float scale, void* o_lat, float* lse,
                   cudaStream_t st) {
  const dim3 grid((g.H + 7) / 8, (unsigned)n_nodes, g.B);
  auto run = [&](auto kern) {
    kern<<<grid, 256, 0, st>>>(g, (const T*)q_abs, n_nodes, (const T*)cache, window, tree, scale,
                               (T*)o_lat, lse);
  };
  if (g.row <= 32 * NARROW)
    run(attend_tree_simt_kernel<T, NARROW, 8>);
  else
    run(attend_tree_simt_kernel<T, WIDE, 1>);
}

template <typename T>
void launch_weight(const Geo& g, const void* q_abs, int64_t n_nodes, const void* cache,
                   const int32_t* window, const uint8_t* tree, float scale, const float* lse,
                   const float* qw, const float* win, float* wout, cudaStream_t st) {
  const dim3 grid((unsigned)((g.S + 7) / 8), g.B);
  auto run = [&](auto kern) {
    kern<<<grid, 256, 0, st>>>(g, (const T*)q_abs, n_nodes, (const T*)cache, window, tree, scale,
                               lse, qw, win, wout);
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
