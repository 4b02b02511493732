"""Inputs and tolerances of the draft-tree and eviction tests (CPU part; the GPU tests upload
them)."""

from __future__ import annotations

import numpy as np

from synth import configs as C
from synth import generate as G

# storage dtype, heads, latent, RoPE width, RoPE pairs, frame grid
TINY = dict(dtype="f32", n_heads=4, d_nope=32, d_latent=64, d_rope=16, rope_pairs=(2, 3, 3),
            grid_h=4, grid_w=4, d_model=128)
ODD = dict(dtype="bf16", n_heads=3, d_nope=32, d_latent=90, d_rope=6, rope_pairs=(1, 1, 1),
           grid_h=2, grid_w=3, d_model=40)
MAIN = dict(dtype="bf16", n_heads=8, d_nope=128, d_latent=512, d_rope=64, rope_pairs=(32, 0, 0),
            grid_h=1, grid_w=1, d_model=256)
HEADS = dict(MAIN, n_heads=128)
VIDEO = dict(MAIN, n_heads=32, rope_pairs=(8, 12, 12), grid_h=6, grid_w=11)
WIDE = dict(MAIN, d_rope=512, rope_pairs=(64, 96, 96), grid_h=5, grid_w=9)
DEEP = dict(VIDEO, n_heads=2, d_model=2304)          # a long K loop, split over several SMs
WIDE_DEEP = dict(WIDE, n_heads=2, d_model=2304)


def workload(cfg, batch, S) -> C.Workload:
    return C.Workload(name="tree", batch=batch, rope_theta=10000.0, window_frames=1,
                      chunk_frames=1, first_chunk_frame=1, ring_slots=S, **cfg)


def normal(rng, shape, dtype, std=1.0) -> G.Tensor:
    return G.to_storage(rng.standard_normal(shape) * std, dtype)


def random_tree(rng, B, n):
    """Parents before children; a node sees itself and its ancestors."""
    parent = np.full((B, n), -1)
    see = np.zeros((B, n, n), dtype=bool)
    for b in range(B):
        for i in range(n):
            p = int(rng.integers(-1, i)) if i else -1
            parent[b, i] = p
            if p >= 0:
                see[b, i] = see[b, p]
            see[b, i, i] = True
    return parent, see


BF16 = 2.0 ** -8        # half a step of bf16, relative
F32 = 2.0 ** -24


def score_error(q, k, scale):
    """Bound on a score's absolute error: float32 products and sums over the row's width (each of
    `width` additions rounds a partial sum of at most sum|q||k|; the tensor cores' adders may
    truncate, 2 F32 instead of F32)."""
    width = q.shape[-1]
    size = scale * float(np.linalg.norm(q, axis=-1).max() * np.linalg.norm(k, axis=-1).max())
    return width * 2 * F32 * size


def attend_tolerance(spread, o, n_keys, d_score, dtype):
    """|error| of o: each weight moves by a factor exp(+-2 d_score) (its own score, and the sum
    that normalises it) and by the exponential's 2^-21; sums of n_keys terms in float32; for
    bf16 storage P and a split piece round once each (2 x 2^-8 of the terms) and the output once."""
    per_term = 2 * d_score + 2.0 ** -21 + (n_keys + 8) * 2 * F32
    if dtype == "bf16":
        return (per_term + 2 * BF16) * spread + BF16 * np.abs(o) + 1e-30
    return per_term * spread + F32 * np.abs(o) + 1e-30


def check_within(got, ref, tol, what):
    got = np.asarray(got, dtype=np.float64)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], ref[bad][:4],
                           np.broadcast_to(tol, got.shape)[bad][:4])
