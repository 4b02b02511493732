"""Draft-tree calls and eviction on the GPU against the fp64 oracle."""

import numpy as np
import pytest
import torch

import latent_kv_cache_write_b200 as mla
from oracle import draft_tree as D
from oracle import mla_oracle as O
from tests import gpu_path as P
from tests import tree_cases as T

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = 0.07


def dev(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV, dtype)


def i32(x):
    return dev(np.asarray(x, dtype=np.int32), torch.int32)


def tree_dev(see):
    return None if see is None else torch.from_numpy(see).to(DEV)


def garbage_outside(cache, windows, n):
    """NaN in every slot outside the windows: no call may let one through."""
    S = cache.shape[1]
    dead = np.ones(cache.shape[:2], dtype=bool)
    for b, w in enumerate(windows):
        f, r, m = D.clip_window(w, S, n)
        dead[b, D.slots(f, r + m, S)] = False
    return dead


def attend(wl, q, cache_t, windows, see, n, split=True, fill=7.0):
    shape = mla.make_shape(wl)
    B = wl.batch
    o = torch.full((B, n, wl.n_heads, wl.d_latent), fill, device=DEV, dtype=q.dtype)
    lse = torch.full((B, n, wl.n_heads), fill, device=DEV)
    nws = mla.mla_attend_tree_workspace_size(shape, n) if split else 0
    ws = torch.empty(max(nws, 16), dtype=torch.uint8, device=DEV) if nws else None
    mla.mla_attend_tree(shape, q, n, cache_t, i32(windows), see, SCALE, o, lse, ws)
    assert mla.mla_device_error() == 0
    return o, lse


def check_attend(wl, qv, cv, windows, see, n, o, lse, fill=7.0):
    ref, rl, spread = D.attend_tree(qv, cv, windows, see, SCALE, wl.d_latent)
    got, gl = P.download(o), P.download(lse)
    for b in range(wl.batch):
        f, r, m = D.clip_window(windows[b], wl.ring_slots, n)
        assert (got[b, m:] == fill).all() and (gl[b, m:] == fill).all(), "rows past the nodes"
        if m == 0:
            continue
        ds = T.score_error(qv[b, :m], np.nan_to_num(cv[b, D.slots(f, r + m, wl.ring_slots)]),
                           SCALE)
        T.check_within(got[b, :m], ref[b, :m],
                       T.attend_tolerance(spread[b, :m], ref[b, :m], r + m, ds, wl.dtype), "o")
        empty = np.isneginf(rl[b, :m])
        assert (np.isneginf(gl[b, :m]) == empty).all()
        fin = ~empty
        T.check_within(gl[b, :m][fin], rl[b, :m][fin],
                       ds + 2.0 ** -20 * (1 + np.abs(rl[b, :m][fin])) + (r + m) * T.F32, "lse")


def weight_tolerance(q, rows, lse, n_heads):
    """Relative: every term moves by exp(+- its score's error) and carries the exponential's 2^-21,
    lse in log2 units rounds relative to itself, and the terms (all positive) add up in float32."""
    lse = np.where(np.isfinite(lse), np.abs(lse), 0.0).max(initial=0)
    return 2 * T.score_error(q, rows, SCALE) + 2.0 ** -20 + (len(q) * n_heads + 8) * T.F32 \
        + 2.0 ** -23 * lse


# configuration, nodes, ring, windows (first, rows, nodes) with lengths on and beside tile borders
CASES = [
    ("TINY", 7, 64, [(0, 20, 7), (60, 57, 3), (5, 0, 7), (9, 64, 0), (63, 1, 1)]),
    ("ODD", 5, 40, [(0, 3, 5), (38, 30, 2), (1, 0, 1)]),
    ("MAIN", 1, 70, [(0, 64, 1), (69, 63, 1), (3, 65, 1), (0, 0, 1), (0, 1, 1)]),
    ("MAIN", 16, 300, [(0, 200, 16), (290, 129, 9), (7, 0, 16), (299, 284, 16), (0, 48, 16)]),
    ("MAIN", 70, 200, [(190, 130, 70), (0, 0, 70), (4, 31, 65), (1, 5, 1), (0, 200, 9)]),
    ("HEADS", 3, 520, [(500, 517, 3), (0, 0, 2), (10, 447, 3)]),
    ("HEADS", 1, 700, [(600, 699, 1), (0, 2, 1), (0, 2, 0)]),
    # fewer key blocks than clusters, cut inside tiles
    ("HEADS", 1, 2700, [(2600, 2600, 1)]),
    ("HEADS", 2, 3000, [(5, 2990, 2), (0, 1500, 1)]),
    ("VIDEO", 20, 150, [(140, 97, 20), (2, 0, 13), (0, 128, 20)]),
    ("WIDE", 9, 150, [(140, 97, 9), (2, 0, 5), (0, 64, 9)]),
    ("WIDE", 40, 600, [(190, 530, 40), (0, 0, 33), (5, 64, 7)]),
]


@pytest.mark.parametrize("split", [True, False])
@pytest.mark.parametrize("cfg,n,S,windows", CASES)
def test_attend_tree(cuda_ok, cfg, n, S, windows, split):
    wl = T.workload(getattr(T, cfg), len(windows), S)
    rng = np.random.default_rng([n, S])
    q = T.normal(rng, (wl.batch, n, wl.n_heads, wl.row_width), wl.dtype)
    c = T.normal(rng, (wl.batch, S, wl.row_width), wl.dtype)
    _, see = T.random_tree(rng, wl.batch, n)
    dead = garbage_outside(c.values, windows, n)
    ct = P.upload(c)
    ct[torch.from_numpy(dead).to(DEV)] = float("nan")
    o, lse = attend(wl, P.upload(q), ct, windows, tree_dev(see), n, split)
    check_attend(wl, q.values, c.values, windows, see, n, o, lse)
    again, lse2 = attend(wl, P.upload(q), ct, windows, tree_dev(see), n, split)
    assert torch.equal(o, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("cfg", ["TINY", "MAIN", "WIDE"])
def test_attend_chain_and_hidden_nodes(cuda_ok, cfg):
    """No tree is a chain; a node that sees nothing; hidden rows that hold NaN and infinities."""
    n, S = 9, 90
    windows = [(80, 33, 9), (3, 0, 9), (0, 70, 9)]
    wl = T.workload(getattr(T, cfg), 3, S)
    rng = np.random.default_rng(5)
    q = T.normal(rng, (3, n, wl.n_heads, wl.row_width), wl.dtype)
    c = T.normal(rng, (3, S, wl.row_width), wl.dtype)
    ct = P.upload(c)
    o, lse = attend(wl, P.upload(q), ct, windows, None, n)
    check_attend(wl, q.values, c.values, windows, None, n, o, lse)

    see = np.tril(np.ones((3, n, n), dtype=bool))
    see[:, :, 4] = False                              # node 4 is seen by no one
    see[:, :, 6] = False
    see[1, 0] = False                                 # and this one sees nothing at all
    cv = c.values.copy()
    for b, (f, r, _) in enumerate(windows):
        for k, bad in ((4, np.nan), (6, np.inf)):
            s = (f + r + k) % S
            ct[b, s] = float(bad)
            ct[b, s, ::3] = float("-inf") if k == 6 else float("nan")
            cv[b, s] = 0.0
    o, lse = attend(wl, P.upload(q), ct, windows, tree_dev(see), n)
    check_attend(wl, q.values, cv, windows, see, n, o, lse)
    # the nodes that do see a NaN row are NaN, the others as before
    see[:, 5, 4] = True
    o2, lse2 = attend(wl, P.upload(q), ct, windows, tree_dev(see), n)
    assert torch.isnan(o2[:, 5]).all() and torch.isnan(lse2[:, 5]).all()
    rest = [i for i in range(n) if i != 5]
    assert torch.equal(o2[:, rest], o[:, rest])


@pytest.mark.parametrize("cfg", ["TINY", "MAIN"])
def test_attend_clips_windows(cuda_ok, cfg):
    """Values no ring has: clipped, not followed."""
    n, S = 4, 30
    windows = [(-7, 12, 4), (99, 1000, 3), (2, -5, 100), (5, 28, 4), (5, 7, -2)]
    wl = T.workload(getattr(T, cfg), 5, S)
    rng = np.random.default_rng(6)
    q = T.normal(rng, (5, n, wl.n_heads, wl.row_width), wl.dtype)
    c = T.normal(rng, (5, S, wl.row_width), wl.dtype)
    _, see = T.random_tree(rng, 5, n)
    o, lse = attend(wl, P.upload(q), P.upload(c), windows, tree_dev(see), n)
    check_attend(wl, q.values, c.values, windows, see, n, o, lse)


@pytest.mark.parametrize("cfg", ["MAIN", "WIDE"])
def test_attend_repeats(cuda_ok, cfg):
    """The same call gives the same bits every time, with scores that take the exact exchange (its
    buffers are handed between the two SMs three times per block)."""
    n, S, windows = 9, 90, [(0, 70, 9), (80, 64, 9), (5, 20, 3)]
    wl = T.workload(getattr(T, cfg), 3, S)
    rng = np.random.default_rng(5)
    q = T.normal(rng, (3, n, 8, wl.row_width), "bf16", 2.0)
    c = T.normal(rng, (3, S, wl.row_width), "bf16")
    qd, cd = P.upload(q), P.upload(c)
    o, lse = attend(wl, qd, cd, windows, None, n)
    check_attend(wl, q.values, c.values, windows, None, n, o, lse)
    for _ in range(200):
        o2, lse2 = attend(wl, qd, cd, windows, None, n)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("cfg,nodes", [("HEADS", (9, 3, 8, 1, 9, 5, 0, 7)),
                                       ("HEADS", (64, 60, 64, 33, 64, 1, 64, 64)),
                                       ("WIDE", (40, 64, 33, 64, 50, 3, 64, 64))])
def test_attend_in_rounds(cuda_ok, cfg, nodes):
    """Keys that crowd L2, so that tiles are handed out in rounds: whole tiles give the bits of one
    call per sequence (whose schedule has no rounds), split tiles one more bf16 rounding."""
    B, n, S = 8, max(nodes), 8192
    rows = [8000, 61, 7777, 8128, 5000, 8064, 8000, 6500]
    wl = T.workload(dict(getattr(T, cfg), n_heads=128), B, S)
    g = torch.Generator(device=DEV).manual_seed(4)
    q = torch.randn((B, n, 128, wl.row_width), device=DEV, generator=g).bfloat16()
    c = torch.randn((B, S, wl.row_width), device=DEV, generator=g).bfloat16()
    _, see = T.random_tree(np.random.default_rng(4), B, n)
    tree = tree_dev(see)
    windows = [(1000 * b, r, m) for b, (r, m) in enumerate(zip(rows, nodes))]
    o, lse = attend(wl, q, c, windows, tree, n, split=False)
    one = wl.scaled(batch=1)
    for b in range(B):
        ob, lb = attend(one, q[b:b + 1], c[b:b + 1], windows[b:b + 1], tree[b:b + 1], n, split=False)
        assert torch.equal(ob[0], o[b]) and torch.equal(lb[0], lse[b])
    os_, ls = attend(wl, q, c, windows, tree, n, split=True)
    # each piece and the merged row round once more; a merged row is a mean of its pieces
    scale = o.float().abs().amax(-1, keepdim=True)
    assert ((os_.float() - o.float()).abs() <= 4 * T.BF16 * scale).all()
    assert ((ls - lse).abs() <= 2.0 ** -12).all()


@pytest.mark.parametrize("cfg", ["MAIN", "WIDE"])
def test_attend_large_scores(cuda_ok, cfg):
    """Scores of hundreds and partial sums of 10^5 (the exact exchange), one key winning."""
    n, S = 6, 200
    windows = [(150, 140, 6), (0, 64, 6)]
    wl = T.workload(getattr(T, cfg), 2, S)
    rng = np.random.default_rng(8)
    q = T.normal(rng, (2, n, wl.n_heads, wl.row_width), wl.dtype, 64.0)
    c = T.normal(rng, (2, S, wl.row_width), wl.dtype, 16.0)
    _, see = T.random_tree(rng, 2, n)
    o, lse = attend(wl, P.upload(q), P.upload(c), windows, tree_dev(see), n)
    check_attend(wl, q.values, c.values, windows, see, n, o, lse)


@pytest.mark.parametrize("cfg,n,S,windows", CASES)
def test_attend_weight(cuda_ok, cfg, n, S, windows):
    wl = T.workload(getattr(T, cfg), len(windows), S)
    shape = mla.make_shape(wl)
    rng = np.random.default_rng([n, S, 3])
    q = T.normal(rng, (wl.batch, n, wl.n_heads, wl.row_width), wl.dtype)
    c = T.normal(rng, (wl.batch, S, wl.row_width), wl.dtype)
    _, see = T.random_tree(rng, wl.batch, n)
    _, lse, _ = D.attend_tree(q.values, c.values, windows, see, SCALE, wl.d_latent)
    lse32 = np.nan_to_num(lse, nan=np.nan).astype(np.float32)
    if n > 1:
        lse32[0, 1] = -np.inf                          # a query that saw nothing adds nothing
    qw = (rng.random((wl.batch, n)) < 0.7).astype(np.float32) * 1.5
    old = rng.random((wl.batch, S)).astype(np.float32)
    ct, qt = P.upload(c), P.upload(q)
    ct[torch.from_numpy(garbage_outside(c.values, windows, n)).to(DEV)] = float("nan")
    for b, w in enumerate(windows):                    # queries past the nodes hold anything
        qt[b, D.clip_window(w, S, n)[2]:] = float("nan")
    for weights_in, per_query in ((old, qw), (None, None)):
        wt = dev(old, torch.float32)
        win = None if weights_in is None else wt
        mla.mla_attend_weight(shape, qt, n, ct, i32(windows), tree_dev(see), SCALE,
                              dev(lse32, torch.float32),
                              None if per_query is None else dev(per_query, torch.float32), win, wt)
        assert mla.mla_device_error() == 0
        ref = D.attend_weight(q.values, c.values, windows, see, SCALE, lse32.astype(np.float64),
                              per_query, weights_in, old.astype(np.float64))
        for b, w in enumerate(windows):
            f, r, m = D.clip_window(w, S, n)
            at = D.slots(f, r + m, S)
            got = P.download(wt)[b]
            rest = np.setdiff1d(np.arange(S), at)
            assert (got[rest] == old[b, rest]).all(), "slots outside the window"
            if not at:
                continue
            rel = weight_tolerance(q.values[b], c.values[b, at], lse32[b, :m], wl.n_heads)
            T.check_within(got[at], ref[b, at], rel * np.abs(ref[b, at]) + 1e-30, "weight")


@pytest.mark.parametrize("cfg", ["TINY", "ODD", "MAIN", "VIDEO", "HEADS", "WIDE"])
@pytest.mark.parametrize("n", [5, 19])
def test_weight_ignores_rows_without_weight(cuda_ok, cfg, n):
    """Queries of weight 0 and queries that saw nothing may hold anything: the same bits come out."""
    S = 300
    windows = [(250, 200, n), (3, 0, n), (1, 9, n - 2)]
    wl = T.workload(getattr(T, cfg), 3, S)
    shape = mla.make_shape(wl)
    rng = np.random.default_rng([n, 8])
    q = P.upload(T.normal(rng, (3, n, wl.n_heads, wl.row_width), wl.dtype))
    ct = P.upload(T.normal(rng, (3, S, wl.row_width), wl.dtype))
    tree = tree_dev(T.random_tree(rng, 3, n)[1])
    _, lse = attend(wl, q, ct, windows, tree, n, fill=0.0)
    lse[1, 2] = float("-inf")
    lse[0, 3, ::2] = float("-inf")                        # some heads of a node
    qw = torch.ones((3, n), device=DEV)
    qw[:, 1] = 0.0
    qw[2, 0] = 0.0
    out = []
    for bad in (None, float("nan"), float("inf")):
        x = q.clone()
        if bad is not None:
            x[:, 1] = x[2, 0] = x[1, 2] = x[0, 3, ::2] = bad
        wt = torch.zeros((3, S), device=DEV)
        mla.mla_attend_weight(shape, x, n, ct, i32(windows), tree, SCALE, lse, qw, None, wt)
        out.append(wt)
    assert torch.isfinite(out[0]).all()
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])
    assert mla.mla_device_error() == 0


@pytest.mark.parametrize("B,n,S", [(700, 3, 150), (70, 20, 200), (33, 1, 1500)])
def test_many_sequences(cuda_ok, B, n, S):
    """More sequences than a warp has lanes, many of them empty or without nodes."""
    wl = T.workload(T.MAIN, B, S)
    shape = mla.make_shape(wl)
    rng = np.random.default_rng([B, n])
    windows = [(int(rng.integers(0, S)), int(rng.choice([0, rng.integers(0, S + 1)])),
                int(rng.integers(0, n + 1))) for _ in range(B)]
    windows = [(f, min(r, S - m), m) for f, r, m in windows]
    q = T.normal(rng, (B, n, wl.n_heads, wl.row_width), wl.dtype)
    c = T.normal(rng, (B, S, wl.row_width), wl.dtype)
    _, see = T.random_tree(rng, B, n)
    ct, qt = P.upload(c), P.upload(q)
    o, lse = attend(wl, qt, ct, windows, tree_dev(see), n)
    check_attend(wl, q.values, c.values, windows, see, n, o, lse)
    wt = torch.zeros((B, S), device=DEV)
    mla.mla_attend_weight(shape, qt, n, ct, i32(windows), tree_dev(see), SCALE, lse, None, None, wt)
    assert mla.mla_device_error() == 0
    l32 = P.download(lse)
    ref = D.attend_weight(q.values, c.values, windows, see, SCALE, l32, None, None,
                          np.zeros((B, S)))
    got = P.download(wt)
    for b, (f, r, m) in enumerate(windows):
        if r + m:
            rel = weight_tolerance(q.values[b], c.values[b, D.slots(f, r + m, S)], l32[b, :m],
                                   wl.n_heads)
            T.check_within(got[b], ref[b], rel * np.abs(ref[b]) + 1e-30, "weight")
        else:
            assert (got[b] == 0).all()


@pytest.mark.parametrize("split", [True, False])
@pytest.mark.parametrize("B,long", [
    (80, 1),         # more tiles than clusters, one of them far longer: cut inside tiles
    (80, 80),        # all long: whole tiles
    (40, 40),        # some tiles in pieces, others whole
    (30, 3),         # three in many pieces
    (2, 2),
])
def test_attend_plans(cuda_ok, B, long, split):
    """Ragged batches on both sides of each rule by which tiles are shared among the SMs."""
    n, S = 16, 2600
    wl = T.workload(T.MAIN, B, S)
    rng = np.random.default_rng([B, long])
    windows = [(int(rng.integers(0, S)), int(rng.integers(1000, S - n + 1)) if b < long
                else int(rng.integers(0, 60)), int(rng.integers(1, n + 1))) for b in range(B)]
    windows = [windows[b] for b in rng.permutation(B)]
    q = T.normal(rng, (B, n, wl.n_heads, wl.row_width), wl.dtype)
    one = T.normal(rng, (1, S, wl.row_width), wl.dtype)      # (every sequence's ring, at own windows)
    _, see = T.random_tree(rng, B, n)
    ct = P.upload(one).expand(B, -1, -1).contiguous()
    o, lse = attend(wl, P.upload(q), ct, windows, tree_dev(see), n, split)
    check_attend(wl, q.values, np.broadcast_to(one.values, (B,) + one.values.shape[1:]), windows, see,
                 n, o, lse)


def test_far_slots(cuda_ok):
    """A ring of more than 2^31 elements: a step at its end gives the bits of a step at the end of a
    short ring (neither splits a tile)."""
    n, rows, far, near = 6, 400, 3_800_000, 1000
    rng = np.random.default_rng(6)
    _, see = T.random_tree(rng, 1, n)
    acc = torch.tensor([[0, 1, 0, 0, 1, 1]], dtype=torch.uint8, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(6)
    rand = lambda *s: torch.randn(s, device=DEV, generator=g)
    h, wd, wr = (rand(1, n, 256).bfloat16(), rand(256, 512).bfloat16() / 16,
                 rand(256, 64).bfloat16() / 16)
    q, tok, context = rand(1, n, 8, 576).bfloat16(), i32([[9, 9, 9, 10, 10, 11]]), \
        rand(rows, 576).bfloat16()
    results = []
    for S in (far, near):
        wl = T.workload(T.MAIN, 1, S)
        shape = mla.make_shape(wl)
        window = [(S - 20, rows, n)]
        at = torch.tensor(D.slots(S - 20, rows + n, S), device=DEV)
        ct = torch.empty((1, S, 576), device=DEV, dtype=torch.bfloat16)
        ct[0, at[:rows]] = context
        pos = torch.zeros((1, S), device=DEV, dtype=torch.int32)
        pos[0, at[:rows]] = torch.arange(rows, device=DEV, dtype=torch.int32)
        wt, win = torch.zeros((1, S), device=DEV), i32(window)
        ws = torch.empty(mla.mla_cache_evict_workspace_size(shape), dtype=torch.uint8, device=DEV)
        mla.mla_tree_write(shape, h, 256, n, win, tok, wd, wr, ct, pos)
        o, lse = attend(wl, q, ct, window, tree_dev(see), n)
        mla.mla_attend_weight(shape, q, n, ct, win, tree_dev(see), SCALE, lse, None, wt, wt)
        one = [x[0, at].clone() for x in (ct, pos, wt)]
        mla.mla_tree_accept(shape, ct, n, acc, win, wt, pos, ws)
        mla.mla_cache_evict(shape, ct, 150, 4, 20, win, wt, pos, ws)
        assert mla.mla_device_error() == 0
        assert (win - i32([(S - 20, 150, 0)]) == 0).all()
        results.append([o, lse] + one + [x[0, at[:150]].clone() for x in (ct, pos, wt)])
    for x, y in zip(*results):
        assert torch.equal(x, y)
    check_attend(T.workload(T.MAIN, 1, rows + n), P.download(q), P.download(results[0][2])[None],
                 [(0, rows, n)], see, n, results[0][0], results[0][1])


@pytest.mark.parametrize("cfg,n,S,windows", [
    ("TINY", 5, 40, [(0, 10, 5), (38, 30, 2), (3, 0, 5), (0, 38, 5)]),
    ("ODD", 5, 40, [(0, 10, 5), (38, 30, 2), (3, 0, 0)]),
    ("MAIN", 1, 40, [(0, 10, 1), (38, 30, 1), (3, 40, 1)]),
    ("MAIN", 30, 100, [(95, 50, 30)] * 5 + [(1, 2, 17)] * 4 + [(0, 0, 0)]),
    ("VIDEO", 7, 100, [(95, 50, 7), (1, 2, 3)]),
    ("WIDE", 7, 100, [(95, 50, 7), (1, 2, 3)]),
    # K split 8, 3 and 4 ways (1, 8 and 20 tiles of rows; the last in several turns), and wide
    ("DEEP", 7, 100, [(95, 50, 7), (1, 2, 3)]),
    ("DEEP", 30, 100, [(95, 50, 30), (0, 80, 30), (7, 0, 11)] * 11 + [(1, 2, 30)]),
    ("DEEP", 32, 100, [(95, 50, 32), (0, 80, 30), (7, 0, 11), (1, 2, 31)] * 20),
    ("WIDE_DEEP", 7, 100, [(95, 50, 7), (1, 2, 3)]),
])
def test_place(cuda_ok, cfg, n, S, windows):
    """tree_write and tree_absorb_q: own positions, own slots, nothing past the nodes."""
    wl = T.workload(getattr(T, cfg), len(windows), S)
    shape = mla.make_shape(wl)
    B, d = wl.batch, wl.d_model
    rng = np.random.default_rng([n, S, 4])
    h = T.normal(rng, (B, n, d), wl.dtype)
    w_dkv = T.normal(rng, (d, wl.d_latent), wl.dtype, d ** -0.5)
    w_kr = T.normal(rng, (d, wl.d_rope), wl.dtype, d ** -0.5)
    w_uk = T.normal(rng, (wl.n_heads, wl.d_nope, wl.d_latent), wl.dtype, wl.d_latent ** -0.5)
    qn = T.normal(rng, (B, n, wl.n_heads, wl.d_nope), wl.dtype)
    qr = T.normal(rng, (B, n, wl.n_heads, wl.d_rope), wl.dtype)
    token = rng.integers(0, 200000, (B, n))
    c0 = T.normal(rng, (B, S, wl.row_width), wl.dtype)
    ct = P.upload(c0)
    pos = torch.full((B, S), -1, dtype=torch.int32, device=DEV)
    mla.mla_tree_write(shape, P.upload(h), d, n, i32(windows), i32(token), P.upload(w_dkv),
                       P.upload(w_kr), ct, pos)
    qa = P.empty(wl, (B, n, wl.n_heads, wl.row_width))
    mla.mla_tree_absorb_q(shape, P.upload(qn), P.upload(qr), n, i32(token), P.upload(w_uk), qa)
    assert mla.mla_device_error() == 0
    ref, rp = D.tree_write(c0.values, np.full((B, S), -1), h.values, w_dkv.values, w_kr.values,
                           windows, token, wl)
    assert (pos.cpu().numpy() == rp).all()
    got = P.download(ct)
    touched = rp >= 0
    assert (got[~touched] == c0.values[~touched]).all(), "rows outside the nodes"
    half = T.BF16 if wl.dtype == "bf16" else T.F32
    # a product of width d rounds d + 2 times in float32 at the size of sum |h||w|; the rotation
    # mixes a pair (factor 2) and its sine and cosine carry 2^-20; the result rounds once
    if touched.any():
        size = np.linalg.norm(h.values, axis=-1).max() * max(
            np.linalg.norm(w_dkv.values, axis=0).max(), np.linalg.norm(w_kr.values, axis=0).max())
        T.check_within(got[touched], ref[touched], half * np.abs(ref[touched])
                       + 2 * size * ((d + 2) * 2 * T.F32 + 2.0 ** -20), "cache")
    qref = D.tree_absorb_q(qn.values, qr.values, w_uk.values, token, wl)
    size = max(np.linalg.norm(qn.values, axis=-1).max() * np.linalg.norm(w_uk.values, axis=1).max(),
               np.abs(qr.values).max())
    T.check_within(P.download(qa), qref, half * np.abs(qref)
                   + 2 * size * ((wl.d_nope + 2) * 2 * T.F32 + 2.0 ** -20), "q_abs")


def test_write_matches_cache_write(cuda_ok):
    """One sequence whose nodes are the next tokens: the same bits as mla_cache_write."""
    wl = T.workload(T.MAIN, 2, 64)
    shape = mla.make_shape(wl)
    g = torch.Generator(device=DEV).manual_seed(1)
    h = torch.randn((2, 5, 256), device=DEV, generator=g).bfloat16()
    wd = torch.randn((256, 512), device=DEV, generator=g).bfloat16()
    wr = torch.randn((256, 64), device=DEV, generator=g).bfloat16()
    a = torch.zeros((2, 64, 576), device=DEV, dtype=torch.bfloat16)
    b = torch.zeros_like(a)
    mla.mla_cache_write(shape, h, 256, 5, 61, wd, wr, a)
    tok = i32(np.tile(np.arange(61, 66), (2, 1)))
    mla.mla_tree_write(shape, h, 256, 5, i32([(2, 59, 5)] * 2), tok, wd, wr, b)
    assert torch.equal(a, b)


def _state(wl, windows, n, seed):
    rng = np.random.default_rng(seed)
    S, B = wl.ring_slots, wl.batch
    c = T.normal(rng, (B, S, wl.row_width), wl.dtype)
    wt = rng.random((B, S)).astype(np.float32)
    pos = rng.permuted(np.tile(np.arange(S), (B, 1)), axis=1)
    return c, wt, pos


def _check_moved(ref, ct, win, wt, pos):
    c, w, wg, p = ref
    assert (win.cpu().numpy() == w).all()
    assert (P.download(ct) == c).all()
    if wt is not None:
        np.testing.assert_array_equal(wt.cpu().numpy(), wg.astype(np.float32))
    if pos is not None:
        assert (pos.cpu().numpy() == p).all()


@pytest.mark.parametrize("cfg", ["TINY", "ODD", "MAIN"])
@pytest.mark.parametrize("n,S,windows", [
    (1, 9, [(0, 3, 1), (8, 0, 1), (4, 8, 1), (3, 9, 0)]),
    (9000, 9100, [(9000, 80, 9000), (3, 100, 8192)]),
    (40, 101, [(90, 50, 40), (0, 0, 40), (7, 61, 40), (100, 1, 0), (-4, 500, 9), (3, 4, 99)]),
])
@pytest.mark.parametrize("extra", [True, False])
def test_accept(cuda_ok, cfg, n, S, windows, extra):
    wl = T.workload(getattr(T, cfg), len(windows), S)
    shape = mla.make_shape(wl)
    c, wt, pos = _state(wl, windows, n, [n, S])
    acc = np.random.default_rng(9).random((wl.batch, n)) < 0.4
    acc[0] = True
    acc[-1] = False
    win, ct = i32(windows), P.upload(c)
    wd, pd = (dev(wt, torch.float32), i32(pos)) if extra else (None, None)
    ws = torch.empty(mla.mla_cache_evict_workspace_size(shape), dtype=torch.uint8, device=DEV)
    mla.mla_tree_accept(shape, ct, n, torch.from_numpy(acc).to(DEV), win, wd, pd, ws)
    _check_moved(D.tree_accept(c.values, np.array(windows), wt, pos, acc), ct, win, wd, pd)


EVICT = [
    # S, windows, keep, sink, recent
    (9, [(0, 9, 0), (8, 5, 3), (2, 1, 0), (0, 0, 0)], 3, 1, 1),
    (9, [(0, 9, 0), (8, 5, 3)], 0, 1, 1),
    (9, [(0, 9, 0), (8, 9, 0)], 9, 0, 0),
    (300, [(290, 300, 0), (4, 77, 5), (-4, 999, 0), (100, 61, 0)], 60, 4, 20),
    (300, [(290, 300, 0), (4, 150, 0)], 60, 200, 500),          # more protected than kept
    (2600, [(2500, 2600, 0), (0, 2049, 0), (1, 1025, 0)], 1024, 0, 0),
    (5000, [(4000, 5000, 0), (0, 4999, 0)], 4990, 7, 100),
    (8193, [(4000, 8193, 0), (0, 8192, 0), (7, 8191, 0)], 8100, 7, 100),
    (20000, [(19000, 20000, 0), (0, 8193, 0)], 9000, 7, 5000),
    (60000, [(59000, 60000, 0), (0, 40000, 0)], 20000, 1, 3),
]


@pytest.mark.parametrize("cfg", ["TINY", "ODD"])
@pytest.mark.parametrize("S,windows,keep,sink,recent", EVICT)
@pytest.mark.parametrize("weights", ["random", "ties", "special"])
def test_evict(cuda_ok, cfg, S, windows, keep, sink, recent, weights):
    wl = T.workload(getattr(T, cfg), len(windows), S)
    shape = mla.make_shape(wl)
    c, wt, pos = _state(wl, windows, 1, [S, keep])
    rng = np.random.default_rng(S)
    if weights == "ties":
        wt = rng.integers(0, 3, wt.shape).astype(np.float32)
    elif weights == "special":
        wt = rng.choice(np.array([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-42, -1e-42, 3.4e38, 1.0,
                                  -1.0], dtype=np.float32), wt.shape)
    win, ct = i32(windows), P.upload(c)
    wd, pd = dev(wt, torch.float32), i32(pos)
    ws = torch.empty(mla.mla_cache_evict_workspace_size(shape), dtype=torch.uint8, device=DEV)
    mla.mla_cache_evict(shape, ct, keep, sink, recent, win, wd, pd, ws)
    _check_moved(D.cache_evict(c.values, np.array(windows), wt, pos, keep, sink, recent), ct, win,
                 wd, pd)


@pytest.mark.parametrize("cfg", ["TINY", "MAIN", "VIDEO"])
def test_serving_steps(cuda_ok, cfg):
    """Two steps as a server runs them (write, absorb, attend, project, weigh, accept, evict), each
    call checked against the oracle on the state the calls before it left."""
    wl = T.workload(getattr(T, cfg), 3, 96)
    shape = mla.make_shape(wl)
    B, n, d, S = 3, 6, wl.d_model, 96
    rng = np.random.default_rng(12)
    first = np.array([90, 0, 40])
    rows = np.array([60, 17, 3])
    c = T.normal(rng, (B, S, wl.row_width), wl.dtype)
    ct = P.upload(c)
    pos = np.zeros((B, S), dtype=np.int64)
    for b in range(B):
        pos[b, D.slots(first[b], rows[b], S)] = np.arange(rows[b])
    wt = rng.random((B, S)).astype(np.float32)
    win, pd, wd = i32(np.stack([first, rows, [n, n - 2, 1]], 1)), i32(pos), dev(wt, torch.float32)
    w = {k: T.normal(rng, s, wl.dtype, s[0 if k != "w_uk" and k != "w_uv" else 2] ** -0.5)
         for k, s in (("w_dkv", (d, wl.d_latent)), ("w_kr", (d, wl.d_rope)),
                      ("w_uk", (wl.n_heads, wl.d_nope, wl.d_latent)),
                      ("w_uv", (wl.n_heads, wl.d_nope, wl.d_latent)))}
    wdv = {k: P.upload(v) for k, v in w.items()}
    ews = torch.empty(mla.mla_cache_evict_workspace_size(shape), dtype=torch.uint8, device=DEV)
    nws = mla.mla_attend_tree_workspace_size(shape, n)
    ws = torch.empty(max(nws, 16), dtype=torch.uint8, device=DEV) if nws else None
    for step in range(2):
        if step:
            win[:, 2] = n
        parent, see = T.random_tree(rng, B, n)
        depth = see.sum(2) - 1
        token = 100 * (step + 1) + depth
        h = T.normal(rng, (B, n, d), wl.dtype)
        qn = T.normal(rng, (B, n, wl.n_heads, wl.d_nope), wl.dtype)
        qr = T.normal(rng, (B, n, wl.n_heads, wl.d_rope), wl.dtype)
        qa = P.empty(wl, (B, n, wl.n_heads, wl.row_width))
        o = torch.full((B, n, wl.n_heads, wl.d_latent), 7.0, device=DEV, dtype=qa.dtype)
        lse = torch.full((B, n, wl.n_heads), 7.0, device=DEV)
        out = P.empty(wl, (B, n, wl.n_heads, wl.d_nope))
        mla.mla_tree_write(shape, P.upload(h), d, n, win, i32(token), wdv["w_dkv"], wdv["w_kr"],
                           ct, pd)
        mla.mla_tree_absorb_q(shape, P.upload(qn), P.upload(qr), n, i32(token), wdv["w_uk"], qa)
        mla.mla_attend_tree(shape, qa, n, ct, win, tree_dev(see), SCALE, o, lse, ws)
        mla.mla_up_v(shape, o, n, wdv["w_uv"], out)
        windows = win.cpu().numpy()
        cv, qv = P.download(ct), P.download(qa)
        check_attend(wl, qv, cv, windows, see, n, o, lse)
        live = np.arange(n) < windows[:, 2:3]
        ref = O.up_v(P.download(o), w["w_uv"].values)
        P.tol_check(P.download(out)[live], ref[live], wl.dtype, "out")
        acc = np.zeros((B, n), dtype=bool)
        for b in range(B):
            i = int(rng.integers(0, windows[b, 2]))
            while i >= 0:
                acc[b, i] = True
                i = int(parent[b, i])
        at = torch.from_numpy(acc).to(DEV)
        w_before, l_now = P.download(wd), P.download(lse)
        mla.mla_attend_weight(shape, qa, n, ct, win, tree_dev(see), SCALE, lse, at.float(), wd, wd)
        ref = D.attend_weight(qv, cv, windows, see, SCALE, l_now, acc.astype(float), w_before,
                              w_before)
        for b in range(B):
            at_b = D.slots(windows[b, 0], windows[b, 1] + windows[b, 2], S)
            rel = weight_tolerance(qv[b], cv[b, at_b], l_now[b, :windows[b, 2]], wl.n_heads)
            T.check_within(P.download(wd)[b], ref[b], rel * np.abs(ref[b]) + 1e-30, "weight")
        w_now, p_now = P.download(wd), pd.cpu().numpy()
        mla.mla_tree_accept(shape, ct, n, at, win, wd, pd, ews)
        r1 = D.tree_accept(cv, windows, w_now, p_now, acc)
        _check_moved(r1, ct, win, wd, pd)
        mla.mla_cache_evict(shape, ct, 30, 2, 5, win, wd, pd, ews)
        _check_moved(D.cache_evict(r1[0], r1[1], r1[2], r1[3], 30, 2, 5), ct, win, wd, pd)
    assert mla.mla_device_error() == 0


def test_captured_loop_follows_its_windows(cuda_ok):
    """A captured attend + weight + accept + evict, replayed after the windows changed, equals the
    plain calls; two graphs with workspaces of their own, and a stream other than the default."""
    n, S = 6, 400
    wl = T.workload(T.MAIN, 3, S)
    shape = mla.make_shape(wl)
    rng = np.random.default_rng(2)
    q = P.upload(T.normal(rng, (3, n, 8, 576), "bf16"))
    c0 = P.upload(T.normal(rng, (3, S, 576), "bf16"))
    _, see = T.random_tree(rng, 3, n)
    tree = tree_dev(see)
    acc = torch.from_numpy(rng.random((3, n)) < 0.5).to(DEV)
    pos0 = i32(np.tile(np.arange(S), (3, 1)))
    nws = mla.mla_attend_tree_workspace_size(shape, n)

    class Loop:
        def __init__(self):
            self.ct, self.pos = c0.clone(), pos0.clone()
            self.win = i32([(0, 10, n)] * 3)
            self.wt = torch.zeros((3, S), device=DEV)
            self.o = torch.zeros((3, n, 8, 512), device=DEV, dtype=torch.bfloat16)
            self.lse = torch.zeros((3, n, 8), device=DEV)
            self.ws = torch.empty(max(nws, 16), dtype=torch.uint8, device=DEV) if nws else None
            self.ews = torch.empty(mla.mla_cache_evict_workspace_size(shape), dtype=torch.uint8,
                                   device=DEV)

        def run(self):
            mla.mla_attend_tree(shape, q, n, self.ct, self.win, tree, SCALE, self.o, self.lse,
                                self.ws)
            mla.mla_attend_weight(shape, q, n, self.ct, self.win, tree, SCALE, self.lse, None,
                                  self.wt, self.wt)
            mla.mla_tree_accept(shape, self.ct, n, acc, self.win, self.wt, self.pos, self.ews)
            mla.mla_cache_evict(shape, self.ct, 64, 2, 8, self.win, self.wt, self.pos, self.ews)

        def reset(self, windows):
            self.ct.copy_(c0)
            self.pos.copy_(pos0)
            for x in (self.wt, self.o, self.lse):      # rows past the nodes keep what was there
                x.zero_()
            self.win.copy_(i32(windows))

        def results(self):
            return [x.clone() for x in (self.ct, self.pos, self.win, self.wt, self.o, self.lse)]

    plain = Loop()
    plain.run()                                       # warm-up outside capture
    loops, graphs = [Loop(), Loop()], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for lp in loops:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                lp.run()
            graphs.append(g)
    torch.cuda.synchronize()
    for windows in ([(0, 300, n), (390, 64, 2), (5, 0, n)], [(7, 1, 1), (0, 390, n), (399, 65, n)]):
        plain.reset(windows)
        plain.run()
        torch.cuda.synchronize()
        for lp in loops:
            lp.reset(windows)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in loops]
        for g, s in zip(graphs, streams):             # both at once
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        want = plain.results()
        for lp in loops:
            for x, y in zip(want, lp.results()):
                assert torch.equal(x, y)
    assert mla.mla_device_error() == 0
