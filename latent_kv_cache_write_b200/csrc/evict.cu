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
// A block per sequence chooses the rows and lists the moves: the rows' ranks as 32-bit keys (in
// registers up to 8192 rows, then in shared memory), a radix selection of the budget's threshold,
// then ballots and scans that keep the rows' order.  It is bound by its instructions (one SM per
// sequence) and the latency of its passes.  Where at most MOVE_HERE rows can move (accepted nodes, a full
// cache that drops a few rows per step) the block also moves them; otherwise a second launch lets the
// whole GPU copy the listed rows, each read and written once (bound by HBM).  A pass over 32 sequences
// of up to 8192 rows of 576 bf16, to 4096, with the copy that puts their state back: 44 us; alone and with
// cold caches the plan takes 14 and the move 28.  4 sequences that drop up to 16 rows each: 12 us.
#include "launch.h"
#include "tc_ptx.cuh"
#include "window.cuh"

#include <mutex>

namespace mla {
namespace {

constexpr int NT = 1024;                    // threads of a planning block
constexpr int NW = NT / 32;
constexpr int KEYS_SH = 48 * 1024;          // keys kept in shared memory
constexpr int HEAD = 8192 / NT;             // keys a thread holds in registers
constexpr int MOVE_HERE = 128;              // rows a planning block moves itself
constexpr unsigned FULL = 0xffffffffu;

// Workspace: counts [B] (padded to 4), then per sequence `cap` destination and `cap` source slots.
struct Plan {
  int32_t* count;
  int32_t* slots;                           // [B][2][cap]
  int64_t cap;
};

__host__ __device__ inline int64_t plan_cap(int64_t S) { return S / 2 + 1; }

struct EvictArgs {
  int64_t S, n_nodes, n_keep;
  int32_t n_sink, n_recent;
  const uint8_t* accept;                    // accept: [B, n_nodes]; null for evict
  int32_t* window;
  void* cache;
  float* weight;
  int32_t* position;
  int32_t per_row;                          // vectors of a cached row
  int32_t key_rows;                         // keys that fit this launch's shared memory
  Plan plan;
};

// Order of a weight as an unsigned number: larger weights larger, -0 as +0, NaN below all.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
constexpr uint32_t SAFE = 0xFFFFFFFFu;      // protected rows (+inf is 0xFF800000)

// Warp w's count -> the sum over the warps before it; *total: over all.  `sums`: one per warp, for
// this call alone.
template <typename T>
__device__ __forceinline__ T warp_offsets(T v, T* sums, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) sums[warp] = v;
  __syncthreads();
  T x = lane < NW ? sums[lane] : 0;
#pragma unroll
  for (int o = 1; o < NW; o <<= 1) {
    const T y = __shfl_up_sync(FULL, x, o);
    if (lane >= o) x += y;
  }
  *total = __shfl_sync(FULL, x, NW - 1);
  const T before = __shfl_sync(FULL, x, warp ? warp - 1 : 0);
  return warp ? before : 0;
}

// Rows listed in dst / src of one sequence, by `warps` warps of which this is number w: two rows at a
// time, all vectors of both loaded before the first is stored (up to 128 of a row; compilers do not
// move loads over stores, and one vector per row in flight left the copy waiting on latency).
template <typename V>
__device__ __forceinline__ void move_rows(V* rows, int per_row, float* weight, int32_t* position,
                                          const int32_t* dst, const int32_t* src, int n, int w,
                                          int warps) {
  const int lane = threadIdx.x & 31;
  for (int k0 = 2 * w; k0 < n; k0 += 2 * warps) {
    const int k1 = k0 + 1 < n ? k0 + 1 : k0;           // (an odd last row twice: the same values)
    const V* from[2] = {rows + (int64_t)src[k0] * per_row, rows + (int64_t)src[k1] * per_row};
    V* to[2] = {rows + (int64_t)dst[k0] * per_row, rows + (int64_t)dst[k1] * per_row};
    for (int c0 = lane; c0 < per_row; c0 += 128) {
      V v[2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (c0 + 32 * q < per_row) v[u][q] = from[u][c0 + 32 * q];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (c0 + 32 * q < per_row) to[u][c0 + 32 * q] = v[u][q];
    }
    if (lane < 2 && k0 + lane < n) {
      const int d = dst[k0 + lane], s = src[k0 + lane];
      if (weight) weight[d] = weight[s];
      if (position) position[d] = position[s];
    }
  }
}

template <typename V, bool MOVE>
__global__ void __launch_bounds__(NT) evict_plan_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ uint32_t keys_sh[];     // [key_rows]
  // of each pass: the digits' counts; chosen digit, rows still to take inside it, its rows
  __shared__ uint32_t hist[3][2048];
  __shared__ uint32_t pick[3][3];
  __shared__ uint32_t sums[4][NW];
  __shared__ uint64_t sums2[NW];
  __shared__ int newest_sh;
  __shared__ uint32_t safe_sh;
  __shared__ int32_t list[MOVE ? 2 * MOVE_HERE : 1];
  const int b = blockIdx.x, t = threadIdx.x, lane = t & 31, warp = t >> 5;
  if (!a.accept)
    for (int q = t; q < 3 * 2048; q += NT) hist[q / 2048][q % 2048] = 0u;
  if (t == 0) {
    newest_sh = INT32_MIN;
    safe_sh = 0u;
  }
  tc::grid_dep_wait();                      // the previous kernel's outputs are visible
  tc::grid_dep_launch();
  const Window w = load_window(a.window, b, a.S, a.accept ? a.n_nodes : a.S);
  int32_t* pos = a.position ? a.position + (int64_t)b * a.S : nullptr;
  float* wt = a.weight ? a.weight + (int64_t)b * a.S : nullptr;
  int32_t* dst = MOVE ? list : a.plan.slots + (int64_t)b * 2 * a.plan.cap;
  int32_t* src = dst + (MOVE ? MOVE_HERE : a.plan.cap);

  const int base = a.accept ? w.rows : 0;   // logical rows considered: base .. base + n - 1
  const int n = a.accept ? w.nodes : w.rows;
  int count = 0;                            // how many of them stay
  // the rows whose key is above thr stay, and `ties` of those at it, the lowest; or, if all_at, all
  // whose key is at least thr
  uint32_t thr = 0, ties = 0;
  bool all_at = false;
  const uint8_t* acc = a.accept ? a.accept + (int64_t)b * a.n_nodes : nullptr;
  // A warp owns consecutive rows, 32 at a time, so that ballots keep their order.  Of up to HEAD * NT
  // rows each thread holds the keys of its own in registers; more go through shared memory
  // (key_rows of them), and past that are worked out again at each pass.
  const bool small = n <= HEAD * NT, held = !acc && n <= a.key_rows;
  const int per = small ? HEAD * 32 : ((n + NT - 1) / NT) * 32;
  const int j0 = min(warp * per, n), j1 = min(j0 + per, n);
  uint32_t k8[HEAD];
  int64_t recent = INT64_MAX;               // positions past it are protected
  auto rank_key = [&](int32_t p, float x) -> uint32_t {
    return p < a.n_sink || p > recent ? SAFE : weight_key(x);
  };
  auto make_key = [&](int j) -> uint32_t {  // accept: the node's byte
    if (acc) return acc[j];
    const int64_t s = w.slot(j, a.S);
    return rank_key(pos[s], wt[s]);
  };
  // f(row, its key, whether it exists) for this lane's rows, the warp together; a row that does not
  // exist has key 0
  auto each = [&](auto&& f) {
    if (small) {
#pragma unroll
      for (int u = 0; u < HEAD; ++u)
        if (j0 + 32 * u < j1) f(j0 + 32 * u + lane, k8[u], j0 + 32 * u + lane < j1);
    } else {
#pragma unroll 2
      for (int j = j0 + lane; j - lane < j1; j += 32) {
        const bool in = j < j1;
        f(j, in ? (held ? keys_sh[j] : make_key(j)) : 0u, in);
      }
    }
  };
  auto finish = [&](int rows, int moves) {
    if (!MOVE) a.plan.count[b] = moves;
    a.window[3 * b] = w.first;
    a.window[3 * b + 1] = rows;
    a.window[3 * b + 2] = 0;
  };

  if (!a.accept) {
    if (n <= a.n_keep) {                    // the whole block agrees: nothing leaves
      __syncthreads();
      if (t == 0) finish(n, 0);
      return;
    }
    count = (int)a.n_keep;
    __syncthreads();
    // newest position, then the keys and the counts of their first digit
    int mx = INT32_MIN;
    uint32_t safe = 0;
    auto first_digit = [&](uint32_t k, bool in) {
      safe += in && k == SAFE;
      if (in && k != SAFE) atomicAdd(&hist[0][k >> 21], 1u);
    };
    if (small) {
      int32_t p8[HEAD];
      float x8[HEAD];
#pragma unroll
      for (int u = 0; u < HEAD; ++u) {                 // all loads in flight at once
        const int j = j0 + 32 * u + lane;
        const int64_t s = j < j1 ? w.slot(j, a.S) : 0;
        p8[u] = j < j1 ? pos[s] : INT32_MIN;
        x8[u] = j < j1 ? wt[s] : 0.f;
      }
#pragma unroll
      for (int u = 0; u < HEAD; ++u) mx = max(mx, p8[u]);
      mx = __reduce_max_sync(FULL, mx);
      if (lane == 0) atomicMax(&newest_sh, mx);
      __syncthreads();
      recent = (int64_t)newest_sh - a.n_recent;
#pragma unroll
      for (int u = 0; u < HEAD; ++u) {
        const bool in = j0 + 32 * u + lane < j1;
        k8[u] = in ? rank_key(p8[u], x8[u]) : 0u;
        first_digit(k8[u], in);
      }
    } else {
#pragma unroll 4
      for (int j = j0 + lane; j < j1; j += 32) mx = max(mx, pos[w.slot(j, a.S)]);
      mx = __reduce_max_sync(FULL, mx);
      if (lane == 0) atomicMax(&newest_sh, mx);
      __syncthreads();
      recent = (int64_t)newest_sh - a.n_recent;
#pragma unroll 4
      for (int j = j0 + lane; j < j1; j += 32) {
        const uint32_t k = make_key(j);
        if (held) keys_sh[j] = k;                      // (read by this thread only)
        first_digit(k, true);
      }
    }
    safe = __reduce_add_sync(FULL, safe);
    if (lane == 0 && safe) atomicAdd(&safe_sh, safe);
    __syncthreads();
    safe = safe_sh;
    if (count > 0 && safe >= (uint32_t)count) {
      thr = SAFE;                           // protected rows alone fill the budget
      ties = (uint32_t)count;
      all_at = safe == ties;
    } else if (count > 0) {
      // the largest key such that `take` rows below SAFE reach it, 11 + 11 + 10 bits at a time (11
      // bits take the exponent and two mantissa bits at once: weights crowd in few exponents);
      // done once all rows of the chosen digit stay, as a rule after two passes
      uint32_t prefix = 0, take = (uint32_t)count - safe;
#pragma unroll 1
      for (int pass = 0; pass < 3; ++pass) {
        const int bits = pass < 2 ? 11 : 10, sh = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
        const int above = sh + bits;
        const uint32_t mask = (1u << bits) - 1u;
        if (pass > 0) {
          each([&](int, uint32_t k, bool in) {
            if (in && k != SAFE && (k >> above) == prefix)
              atomicAdd(&hist[pass][(k >> sh) & mask], 1u);
          });
          __syncthreads();
        }
        // a thread owns PT digits from 2047 - PT t down: rows above each by a scan
        constexpr int PT = 2048 / NT;
        uint32_t h[PT], mine = 0;
#pragma unroll
        for (int q = 0; q < PT; ++q) {
          h[q] = hist[pass][2047 - PT * t - q];
          mine += h[q];
        }
        uint32_t x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(FULL, x, o);
          if (lane >= o) x += y;
        }
        uint32_t all;
        uint32_t before = warp_offsets(__shfl_sync(FULL, x, 31), sums[pass], &all) + x - mine;
#pragma unroll
        for (int q = 0; q < PT; ++q) {
          if (before < take && take <= before + h[q]) {
            pick[pass][0] = (uint32_t)(2047 - PT * t - q);
            pick[pass][1] = take - before;
            pick[pass][2] = h[q];
          }
          before += h[q];
        }
        __syncthreads();
        prefix = (prefix << bits) | pick[pass][0];
        take = pick[pass][1];
        thr = prefix << sh;
        all_at = take == pick[pass][2];
        if (all_at) break;
      }
      ties = take;                          // rows at the threshold that stay
    }
  }

  uint32_t tie0 = 0;
  if (a.accept) {
    if (small) {
#pragma unroll
      for (int u = 0; u < HEAD; ++u) {
        const int j = j0 + 32 * u + lane;
        k8[u] = j < j1 ? acc[j] : 0u;
      }
    }
    uint32_t c = 0, total;
    each([&](int, uint32_t k, bool) { c += __popc(__ballot_sync(FULL, k != 0u)); });
    warp_offsets(c, sums[3], &total);
    count = (int)total;
    thr = 1u;
    all_at = true;
  } else if (count == 0) {
    thr = SAFE;                             // nothing stays
  } else if (!all_at) {
    uint32_t c = 0, total;
    each([&](int, uint32_t k, bool in) { c += __popc(__ballot_sync(FULL, in && k == thr)); });
    tie0 = warp_offsets(c, sums[3], &total);
  }
  const unsigned below = (1u << lane) - 1u;
  // whether a row stays; `tie` counts the threshold's rows before the 32 at hand
  auto stays = [&](uint32_t k, bool in, uint32_t& tie) -> bool {
    if (all_at) return in && k >= thr;
    const unsigned m = __ballot_sync(FULL, in && k == thr);
    const bool s = in && (k > thr || (k == thr && tie + __popc(m & below) < ties));
    tie += __popc(m);
    return s;
  };
  uint32_t holes = 0, late = 0, tie = tie0;
  uint32_t mh[HEAD], ml[HEAD];              // (small) which of each 32 rows are holes, late rows
  if (small) {
#pragma unroll
    for (int u = 0; u < HEAD; ++u) {
      const int j = j0 + 32 * u + lane;
      const bool in = j < j1, s = stays(k8[u], in, tie);
      mh[u] = __ballot_sync(FULL, in && j < count && !s);
      ml[u] = __ballot_sync(FULL, j >= count && s);
      holes += __popc(mh[u]);
      late += __popc(ml[u]);
    }
  } else {
    each([&](int j, uint32_t k, bool in) {
      const bool s = stays(k, in, tie);
      holes += __popc(__ballot_sync(FULL, in && j < count && !s));
      late += __popc(__ballot_sync(FULL, j >= count && s));
    });
  }
  uint64_t moves;
  const uint64_t off = warp_offsets((uint64_t)late << 32 | holes, sums2, &moves);
  const int n_move = (int)(uint32_t)moves;
  uint32_t hole = (uint32_t)off, lt = (uint32_t)(off >> 32);
  const int32_t S = (int32_t)a.S, at0 = w.first + base;      // below 2^31: S <= 2^30
  auto list_row = [&](int j, unsigned h, unsigned l) {
    int32_t slot = at0 + j;                 // (base + j < S)
    if (slot >= S) slot -= S;
    if (h) {
      if (h >> lane & 1u) dst[hole + __popc(h & below)] = slot;
      hole += __popc(h);
    }
    if (l) {
      if (l >> lane & 1u) src[lt + __popc(l & below)] = slot;
      lt += __popc(l);
    }
  };
  if (small) {
#pragma unroll
    for (int u = 0; u < HEAD; ++u) list_row(j0 + 32 * u + lane, mh[u], ml[u]);
  } else {
    tie = tie0;
    each([&](int j, uint32_t k, bool in) {
      const bool s = stays(k, in, tie);
      const unsigned h = __ballot_sync(FULL, in && j < count && !s);
      list_row(j, h, __ballot_sync(FULL, j >= count && s));
    });
  }
  if (MOVE) {
    __syncthreads();                        // the list is complete
    move_rows(static_cast<V*>(a.cache) + (int64_t)b * a.S * a.per_row, a.per_row, wt, pos, dst, src,
              n_move, warp, NW);
  }
  if (t == 0) finish(base + count, n_move);
}

// Copy the listed rows; blockIdx.y is the sequence.
template <typename V>
__global__ void __launch_bounds__(256) evict_move_kernel(const __grid_constant__ EvictArgs a) {
  tc::grid_dep_wait();                      // the plan is visible
  tc::grid_dep_launch();
  const int b = blockIdx.y;
  const int32_t* dst = a.plan.slots + (int64_t)b * 2 * a.plan.cap;
  move_rows(static_cast<V*>(a.cache) + (int64_t)b * a.S * a.per_row, a.per_row,
            a.weight ? a.weight + (int64_t)b * a.S : nullptr,
            a.position ? a.position + (int64_t)b * a.S : nullptr, dst, dst + a.plan.cap,
            a.plan.count[b], (int)(blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32),
            (int)(gridDim.x * (blockDim.x / 32)));
}

template <typename V, bool MOVE>
cudaError_t launch_plan(const Geo& g, EvictArgs& a, cudaStream_t st) {
  {
    // the shared-memory opt-in is per device
    static std::mutex mu;
    static uint64_t done = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 64 || !(done >> dev & 1)) {
      e = cudaFuncSetAttribute(evict_plan_kernel<V, MOVE>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, KEYS_SH * 4);
      if (e != cudaSuccess) return e;
      if (dev < 64) done |= 1ull << dev;
    }
  }
  // keys go to shared memory where a sequence can have more rows than the registers hold
  a.key_rows = a.accept || g.S <= HEAD * NT ? 0 : (int)(g.S < KEYS_SH ? g.S : KEYS_SH);
  const cudaError_t e = launch_dependent(evict_plan_kernel<V, MOVE>, (unsigned)g.B, NT,
                                         (size_t)a.key_rows * 4, st, 1u, a);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

template <typename V>
cudaError_t run_as(const Geo& g, EvictArgs a, int64_t most, cudaStream_t st) {
  if (most <= MOVE_HERE) return launch_plan<V, true>(g, a, st);
  cudaError_t e = launch_plan<V, false>(g, a, st);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((148 * 8 + g.B - 1) / g.B), (unsigned)g.B);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, evict_move_kernel<V>, a);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

// most: how many rows of a sequence can move
cudaError_t run(const Geo& g, bool bf, EvictArgs a, int64_t most, cudaStream_t st) {
  const int bytes = g.row * (bf ? 2 : 4);
  if (bytes % 16 == 0) {
    a.per_row = bytes / 16;
    return run_as<uint4>(g, a, most, st);
  }
  a.per_row = bytes / 4;                    // rows are an even number of 2- or 4-byte elements
  return run_as<uint32_t>(g, a, most, st);
}

Plan make_plan(const Geo& g, void* workspace) {
  Plan p;
  p.count = static_cast<int32_t*>(workspace);
  p.slots = p.count + ((g.B + 3) / 4) * 4;
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
  a.S = g.S; a.n_nodes = n_nodes; a.window = window; a.cache = cache;
  // (null would mean eviction; without nodes no byte of it is read)
  a.accept = accept ? accept : reinterpret_cast<const uint8_t*>(window);
  a.weight = weight; a.position = position; a.plan = make_plan(g, workspace);
  return run(g, bf, a, n_nodes / 2, st);
}

cudaError_t cache_evict(const Geo& g, bool bf, void* cache, int64_t n_keep, int32_t n_sink,
                        int32_t n_recent, int32_t* window, float* weight, int32_t* position,
                        void* workspace, cudaStream_t st) {
  EvictArgs a{};
  a.S = g.S; a.n_keep = n_keep; a.n_sink = n_sink; a.n_recent = n_recent; a.window = window;
  a.cache = cache; a.weight = weight; a.position = position; a.plan = make_plan(g, workspace);
  return run(g, bf, a, n_keep < g.S - n_keep ? n_keep : g.S - n_keep, st);
}

}  // namespace mla
