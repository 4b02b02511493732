// Windows of ragged sequences: first slot, context rows and draft nodes of each, read from
// device memory and clipped to the ring, so that no value a caller leaves there can lead an
// access out of it.
#pragma once

#include "common.cuh"

namespace mla {

struct Window {
  int32_t first, rows, nodes;
  __device__ int32_t len() const { return rows + nodes; }
  // ring slot of logical row j (0 <= j <= S)
  __device__ int64_t slot(int64_t j, int64_t S) const {
    const int64_t r = first + j;
    return r >= S ? r - S : r;
  }
};

__device__ __forceinline__ Window load_window(const int32_t* window, int64_t b, int64_t S,
                                              int64_t n_nodes) {
  const int32_t* w = window + 3 * b;
  const int32_t f = w[0], r = w[1], n = w[2], s = (int32_t)S;   // S <= 2^31 - 1
  Window v;
  v.first = f < 0 ? 0 : (f >= s ? s - 1 : f);
  v.rows = r < 0 ? 0 : (r > s ? s : r);
  const int32_t most = (int64_t)(s - v.rows) < n_nodes ? s - v.rows : (int32_t)n_nodes;
  v.nodes = n < 0 ? 0 : (n > most ? most : n);
  return v;
}

// Whether node i sees node k (tree: [n_nodes, n_nodes] bytes of the sequence, or null: k <= i).
__device__ __forceinline__ bool tree_sees(const uint8_t* tree, int64_t n_nodes, int64_t i,
                                          int64_t k) {
  return tree ? tree[i * n_nodes + k] != 0 : k <= i;
}

}  // namespace mla
