// Draft-tree attention and the attention weight of cached rows on CUDA cores: every dtype and
// shape (float32 storage uses it throughout, and bfloat16 shapes the tensor-core kernels do not
// take).  Accumulation is float32.  A warp owns one row of the score matrix (attention) or one of
// its columns (weight) and walks it in order; at the sizes float32 serves (a few heads, tens of
// rows) both are bound by the latency of one dot product after the other.
#include "launch.h"
#include "window.cuh"

namespace mla {
namespace {

constexpr int MAXR = 40;                    // row width <= 32 * MAXR
constexpr int U = 4;                        // scores in flight per warp
constexpr unsigned FULL = 0xffffffffu;

__device__ __forceinline__ float warp_sum(float s) {
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(FULL, s, o);
  return s;
}

// One warp per (sequence, node, head): online softmax over the visible rows.  Hidden nodes are
// skipped, not masked, so nothing of their rows enters the sums.
template <typename T>
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
  const T* q = q_abs + qrow * g.row;
  const int nr = (g.row + 31) / 32, nc = (g.Dc + 31) / 32;
  float qv[MAXR], acc[MAXR];
#pragma unroll
  for (int r = 0; r < MAXR; ++r) {
    const int d = lane + 32 * r;
    qv[r] = (r < nr && d < g.row) ? to_f32(q[d]) * scale : 0.f;
    acc[r] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const T* base = cache + (int64_t)b * g.S * g.row;
  for (int64_t j = 0; j < w.len(); ++j) {
    if (j >= w.rows && !tree_sees(tb, n_nodes, i, j - w.rows)) continue;
    const T* row = base + w.slot(j, g.S) * g.row;
    float kv[MAXR], s = 0.f;
#pragma unroll
    for (int r = 0; r < MAXR; ++r) {
      const int d = lane + 32 * r;
      kv[r] = (r < nr && d < g.row) ? to_f32(row[d]) : 0.f;
      s = fmaf(qv[r], kv[r], s);
    }
    s = warp_sum(s);
    const float mn = fmaxf(m, s);
    const float ref = mn == -INFINITY ? 0.f : mn;       // every score so far -inf
    const float corr = expf(m - ref), p = expf(s - ref);
    l = l * corr + p;
#pragma unroll
    for (int r = 0; r < MAXR; ++r) {
      const int d = lane + 32 * r;
      if (r < nc && d < g.Dc) acc[r] = fmaf(acc[r], corr, p * kv[r]);
    }
    m = mn;
  }
  T* out = o_lat + qrow * g.Dc;
  const float inv = l != 0.f ? 1.f / l : 0.f;            // NaN stays NaN
#pragma unroll
  for (int r = 0; r < MAXR; ++r) {
    const int d = lane + 32 * r;
    if (r < nc && d < g.Dc) out[d] = from_f32<T>(acc[r] * inv);
  }
  if (lse && lane == 0) lse[qrow] = l != 0.f ? m + logf(l) : -INFINITY;
}

// One warp per (sequence, row of the window): the row stays in registers while the warp walks
// the queries in order.
template <typename T>
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
  const T* row = cache + at * g.row;
  const int nr = (g.row + 31) / 32;
  float kv[MAXR];
#pragma unroll
  for (int r = 0; r < MAXR; ++r) {
    const int d = lane + 32 * r;
    kv[r] = (r < nr && d < g.row) ? to_f32(row[d]) * scale : 0.f;
  }
  float total = 0.f;
  for (int64_t i = 0; i < w.nodes; ++i) {
    const float c = qw ? qw[(int64_t)b * n_nodes + i] : 1.f;
    if (c == 0.f || (j >= w.rows && !tree_sees(tb, n_nodes, i, j - w.rows))) continue;
    const int64_t q0 = ((int64_t)b * n_nodes + i) * g.H;
    for (int h0 = 0; h0 < g.H; h0 += U) {
      float s[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const T* q = q_abs + (q0 + h0 + u) * g.row;
        s[u] = 0.f;
#pragma unroll
        for (int r = 0; r < MAXR; ++r) {
          const int d = lane + 32 * r;
          if (h0 + u < g.H && r < nr && d < g.row) s[u] = fmaf(to_f32(q[d]), kv[r], s[u]);
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

}  // namespace

cudaError_t simt_attend_tree(const Geo& g, bool bf, const void* q_abs, int64_t n_nodes,
                             const void* cache, const int32_t* window, const uint8_t* tree,
                             float scale, void* o_lat, float* lse, cudaStream_t st) {
  dim3 grid((g.H + 7) / 8, (unsigned)n_nodes, g.B);
  if (bf)
    attend_tree_simt_kernel<bf16><<<grid, 256, 0, st>>>(g, (const bf16*)q_abs, n_nodes,
                                                        (const bf16*)cache, window, tree, scale,
                                                        (bf16*)o_lat, lse);
  else
    attend_tree_simt_kernel<float><<<grid, 256, 0, st>>>(g, (const float*)q_abs, n_nodes,
                                                         (const float*)cache, window, tree, scale,
                                                         (float*)o_lat, lse);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) count_launches(1);
  return e;
}

cudaError_t simt_attend_weight(const Geo& g, bool bf, const void* q_abs, int64_t n_nodes,
                               const void* cache, const int32_t* window, const uint8_t* tree,
                               float scale, const float* lse, const float* qw, const float* win,
                               float* wout, cudaStream_t st) {
  dim3 grid((unsigned)((g.S + 7) / 8), g.B);
  if (bf)
    attend_weight_simt_kernel<bf16><<<grid, 256, 0, st>>>(g, (const bf16*)q_abs, n_nodes,
                                                          (const bf16*)cache, window, tree, scale,
                                                          lse, qw, win, wout);
  else
    attend_weight_simt_kernel<float><<<grid, 256, 0, st>>>(g, (const float*)q_abs, n_nodes,
                                                           (const float*)cache, window, tree,
                                                           scale, lse, qw, win, wout);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace mla
