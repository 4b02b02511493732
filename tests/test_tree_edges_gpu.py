"""Draft-tree calls at the edges of their definitions, on the GPU: no nodes at all, rows that are NaN,
chains and trees of many nodes, the log-sum-exps of split tiles."""

import numpy as np
import pytest
import torch

import latent_kv_cache_write_b200 as mla
from oracle import draft_tree as D
from tests import gpu_path as P
from tests import tree_cases as T
from tests.test_tree_gpu import SCALE, attend, i32, tree_dev

pytestmark = pytest.mark.gpu
DEV = "cuda"

# sequences with and without context, one that wraps, values that are clipped; all with stale nodes
STALE = [(0, 20, 7), (35, 21, 3), (5, 0, 2), (9, 40, 1), (-4, 99, 5)]


@pytest.mark.parametrize("cfg", ["TINY", "ODD", "MAIN", "WIDE"])
@pytest.mark.parametrize("given", ["apart", "none", "in place"])
def test_weight_without_nodes(cuda_ok, cfg, given):
    """Every context row's total goes to weight_out (0 where none was given), and nothing else; also
    captured, with windows that change before the replay."""
    S, n = 40, 3
    wl = T.workload(getattr(T, cfg), len(STALE), S)
    shape = mla.make_shape(wl)
    rng = np.random.default_rng(3)
    q = P.upload(T.normal(rng, (wl.batch, n, wl.n_heads, wl.row_width), wl.dtype))
    c = torch.full((wl.batch, S, wl.row_width), float("nan"), device=DEV, dtype=q.dtype)
    lse = torch.zeros((wl.batch, n, wl.n_heads), device=DEV)
    old = rng.random((wl.batch, S)).astype(np.float32)
    before = rng.random((wl.batch, S)).astype(np.float32)
    win = i32(STALE)
    w_in = None if given == "none" else torch.from_numpy(old).to(DEV)
    w_out = w_in if given == "in place" else torch.from_numpy(before).to(DEV)

    def call():
        mla.mla_attend_weight(shape, q, 0, c, win, None, SCALE, lse, None, w_in, w_out)

    def check(windows):
        none = np.zeros((wl.batch, 0, wl.n_heads, 1))
        start = old if given == "in place" else before
        ref = D.attend_weight(none, np.zeros((wl.batch, S, 1)), windows, None, SCALE, none, None,
                              None if given == "none" else old, start)
        np.testing.assert_array_equal(w_out.cpu().numpy(), ref.astype(np.float32))

    call()
    check(STALE)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    other = [(3, 12, 7), (0, 0, 3), (39, 40, 2), (1, 1, 1), (0, 5, 0)]
    win.copy_(i32(other))
    w_out.copy_(torch.from_numpy(old if given == "in place" else before))
    graph.replay()
    check(other)
    assert mla.mla_device_error() == 0


@pytest.mark.parametrize("cfg", ["TINY", "MAIN"])
def test_accept_without_nodes(cuda_ok, cfg):
    """Windows keep their context and drop their nodes; rows, weights and positions stay."""
    S, n = 40, 3
    wl = T.workload(getattr(T, cfg), len(STALE), S)
    shape = mla.make_shape(wl)
    rng = np.random.default_rng(4)
    c = T.normal(rng, (wl.batch, S, wl.row_width), wl.dtype)
    wt = rng.random((wl.batch, S)).astype(np.float32)
    pos = rng.integers(0, 999, (wl.batch, S))
    ct, wd, pd, win = P.upload(c), torch.from_numpy(wt).to(DEV), i32(pos), i32(STALE)
    ws = torch.empty(mla.mla_cache_evict_workspace_size(shape), dtype=torch.uint8, device=DEV)
    acc = torch.ones((wl.batch, n), dtype=torch.uint8, device=DEV)
    mla.mla_tree_accept(shape, ct, 0, acc, win, wd, pd, ws)
    rc, rw, rwt, rp = D.tree_accept(c.values, np.array(STALE), wt, pos,
                                    np.zeros((wl.batch, 0), dtype=bool))
    np.testing.assert_array_equal(win.cpu().numpy(), rw)
    np.testing.assert_array_equal(P.download(ct), rc)
    np.testing.assert_array_equal(wd.cpu().numpy(), rwt)
    np.testing.assert_array_equal(pd.cpu().numpy(), rp)
    assert mla.mla_device_error() == 0


@pytest.mark.parametrize("cfg", ["TINY", "MAIN"])
def test_step_without_nodes(cuda_ok, cfg):
    """A whole step of a batch that drafts nothing, its per-node tensors empty: only the windows'
    nodes go."""
    S = 40
    wl = T.workload(getattr(T, cfg), len(STALE), S)
    shape = mla.make_shape(wl)
    B, d, H = wl.batch, wl.d_model, wl.n_heads
    rng = np.random.default_rng(4)
    c = P.upload(T.normal(rng, (B, S, wl.row_width), wl.dtype))
    empty = lambda *s: torch.empty(s, device=DEV, dtype=c.dtype)
    wt, pos, win = torch.rand((B, S), device=DEV), i32(rng.integers(0, 99, (B, S))), i32(STALE)
    before = [x.clone() for x in (c, wt, pos)]
    out = torch.full((B, S), 7.0, device=DEV)
    token, lse = i32(np.zeros((B, 0))), torch.empty((B, 0, H), device=DEV)
    q, o = empty(B, 0, H, wl.row_width), empty(B, 0, H, wl.d_latent)
    byte = torch.empty((B, 0), device=DEV, dtype=torch.uint8)
    ews = torch.empty(mla.mla_cache_evict_workspace_size(shape), dtype=torch.uint8, device=DEV)
    w_uk = empty(H, wl.d_nope, wl.d_latent)
    mla.mla_tree_write(shape, empty(B, 0, d), d, 0, win, token, empty(d, wl.d_latent),
                       empty(d, wl.d_rope), c, pos)
    mla.mla_tree_absorb_q(shape, empty(B, 0, H, wl.d_nope), empty(B, 0, H, wl.d_rope), 0, token, w_uk,
                          q)
    mla.mla_attend_tree(shape, q, 0, c, win, byte, SCALE, o, lse)
    mla.mla_attend_weight(shape, q, 0, c, win, byte, SCALE, lse, lse[:, :, 0], wt, out)
    mla.mla_tree_accept(shape, c, 0, byte, win, wt, pos, ews)
    for x, y in zip(before, (c, wt, pos)):
        assert torch.equal(x, y)
    for b, w in enumerate(STALE):
        first, rows, _ = D.clip_window(w, S, 0)
        assert win[b].tolist() == [first, rows, 0]
        at = torch.tensor(D.slots(first, rows, S), device=DEV, dtype=torch.long)
        assert torch.equal(out[b, at], wt[b, at])
        assert (out[b] == 7.0).sum() == S - rows
    assert mla.mla_device_error() == 0


# windows, rows (logical) that are NaN: a node that sees itself only, blocks of one warpgroup, blocks
# of both, the last piece of a split tile (contexts of whole blocks), its first
NANS = [
    ("TINY", 4, 64, [(0, 0, 4), (60, 8, 4), (3, 40, 2)], [[0], [9, 11], range(40)]),
    ("MAIN", 4, 300, [(290, 0, 4), (0, 64, 4), (5, 128, 4), (9, 128, 4), (2, 192, 4)],
     [[0], [64, 66], range(64), range(64, 128), range(128)]),
    ("HEADS", 1, 2700, [(7, 2624, 1)], [[2624]]),
    ("HEADS", 1, 2700, [(7, 2624, 1)], [range(64)]),
    ("WIDE", 4, 300, [(290, 0, 4), (0, 64, 4), (5, 128, 4), (9, 128, 4)],
     [[0], [64, 66], range(64), range(64, 128)]),
    ("WIDE", 2, 2700, [(7, 2624, 2)], [[2624]]),
]


@pytest.mark.parametrize("split", [True, False])
@pytest.mark.parametrize("cfg,n,S,windows,bad", NANS)
def test_nan_rows_reach_those_who_see_them(cuda_ok, cfg, n, S, windows, bad, split):
    """o_lat and lse are NaN for the nodes that see a NaN row, whatever else of the row's block they
    see, and for no others."""
    wl = T.workload(getattr(T, cfg), len(windows), S)
    rng = np.random.default_rng(S)
    q = T.normal(rng, (wl.batch, n, wl.n_heads, wl.row_width), wl.dtype)
    c = T.normal(rng, (wl.batch, S, wl.row_width), wl.dtype)
    see = np.tile(np.eye(n, dtype=bool), (wl.batch, 1, 1))         # every node sees itself only
    ct, cv = P.upload(c), c.values.copy()
    for b, (f, _, _) in enumerate(windows):
        at = [(f + j) % S for j in bad[b]]
        ct[b, at] = float("nan")
        cv[b, at] = np.nan
    o, lse = attend(wl, P.upload(q), ct, windows, tree_dev(see), n, split)
    ref, rl, spread = D.attend_tree(q.values, cv, windows, see, SCALE, wl.d_latent)
    got, gl = P.download(o), P.download(lse)
    for b, (f, r, m) in enumerate(windows):
        assert (np.isnan(gl[b, :m]) == np.isnan(rl[b, :m])).all()
        assert (np.isnan(got[b, :m]) == np.isnan(ref[b, :m])).all()
        ok = ~np.isnan(rl[b, :m])
        if ok.any():
            ds = T.score_error(q.values[b, :m], np.nan_to_num(cv[b]), SCALE)
            tol = T.attend_tolerance(spread[b, :m], ref[b, :m], r + m, ds, wl.dtype)
            T.check_within(got[b, :m][ok], ref[b, :m][ok], tol[ok], "o")


@pytest.mark.parametrize("cfg,n,S,windows", [
    ("HEADS", 1, 2700, [(7, 2690, 1)]),
    ("HEADS", 2, 3000, [(5, 2990, 2), (0, 1500, 1)]),
    ("WIDE", 4, 2700, [(2600, 2690, 4), (5, 2001, 4)]),
])
def test_split_tiles_round_once(cuda_ok, cfg, n, S, windows):
    """Queries of 0 over whole numbers: every weight is 1 and every sum exact, so that a row is off by
    its one rounding to bf16, however many pieces its tile came in."""
    wl = T.workload(getattr(T, cfg), len(windows), S)
    rng = np.random.default_rng(S)
    c = T.G.to_storage(rng.integers(-8, 9, (wl.batch, S, wl.row_width)).astype(float), "bf16")
    q = T.G.to_storage(np.zeros((wl.batch, n, wl.n_heads, wl.row_width)), "bf16")
    see = np.tril(np.ones((wl.batch, n, n), dtype=bool))
    o, lse = attend(wl, P.upload(q), P.upload(c), windows, tree_dev(see), n)
    ref, rl, spread = D.attend_tree(q.values, c.values, windows, see, SCALE, wl.d_latent)
    got, gl = P.download(o), P.download(lse)
    for b, (_, _, m) in enumerate(windows):
        half = 2.0 ** (np.frexp(ref[b, :m])[1] - 9)               # half a step of the value itself
        # a piece's lse (below 8) is off by 2^-20 at most, its exponential by 2^-22, above and below the
        # fraction line; at most 74 pieces add up in float32
        T.check_within(got[b, :m], ref[b, :m], half + 2.0 ** -17 * spread[b, :m], "o")
        T.check_within(gl[b, :m], rl[b, :m], 2.0 ** -19, "lse")
