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


# Whole numbers: q below 64 and c below 8 make every score's sum exact in float32 (below 2^24) but
# wider than 16 bits, and the scale is a power of two, so that what is left are the roundings of the
# softmax itself.
WHOLE = 2.0 ** -11


def whole_numbers(wl, n, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    draw = lambda top, *s: torch.randint(-top, top + 1, s, device=DEV, generator=g).bfloat16()  # noqa: E731
    return (draw(64, wl.batch, n, wl.n_heads, wl.row_width),
            draw(8, wl.batch, wl.ring_slots, wl.row_width))


def scores64(q, c, b, window, see, n):
    """Scores [nodes, heads, rows + nodes] of sequence b in 64 bits (-inf: hidden), and its rows."""
    f, r, m = D.clip_window(window, c.shape[1], n)
    at = torch.tensor(D.slots(f, r + m, c.shape[1]), device=DEV, dtype=torch.long)
    k = c[b, at].double()
    s = (q[b, :m].double().flatten(0, 1) @ k.T).view(m, q.shape[2], r + m) * WHOLE
    seen = torch.ones((n, n), device=DEV).tril().bool() if see is None else see[b]
    s[:, :, r:] = s[:, :, r:].masked_fill(~seen[:m, None, :m], float("-inf"))
    return s, k, at, r, m


def attend_whole(wl, q, c, windows, see, n, split=True):
    shape = mla.make_shape(wl)
    o = torch.zeros((wl.batch, n, wl.n_heads, wl.d_latent), device=DEV, dtype=q.dtype)
    lse = torch.zeros((wl.batch, n, wl.n_heads), device=DEV)
    ws = torch.empty(mla.mla_attend_tree_workspace_size(shape, n), dtype=torch.uint8,
                     device=DEV) if split else None
    mla.mla_attend_tree(shape, q, n, c, i32(windows), see, WHOLE, o, lse, ws)
    return o, lse


LONG = [
    # tiles in rounds and a tail that cuts them; few sequences, cut in pieces; chains without context
    ("HEADS", 128, 64, 8192, [(1000 * b, r, m) for b, (r, m) in enumerate(zip(
        (8000, 61, 7777, 8128, 5000, 8064, 8000, 6500), (64, 60, 64, 33, 64, 1, 64, 64)))], True),
    ("WIDE", 32, 40, 4000, [(3900, 3960, 40), (5, 1111, 9), (7, 0, 40)], True),
    ("MAIN", 8, 17, 6000, [(5990, 5983, 17), (1, 640, 5)], True),
    ("VIDEO", 32, 300, 1400, [(1300, 1100, 300), (0, 0, 300), (9, 64, 129)], False),
    ("HEADS", 128, 90, 300, [(250, 210, 90), (3, 0, 90)], False),
    ("WIDE", 16, 260, 700, [(650, 440, 260), (0, 0, 260), (1, 1, 65)], False),
]


@pytest.mark.parametrize("split", [True, False])
@pytest.mark.parametrize("cfg,heads,n,S,windows,tree", LONG)
def test_attend_exact_scores(cuda_ok, cfg, heads, n, S, windows, tree, split):
    """Long contexts, many nodes: lse to what float32 partial scores leave, and the same bits in every
    call while the two SMs hand their buffers back and forth over many blocks and tiles."""
    wl = T.workload(dict(getattr(T, cfg), n_heads=heads), len(windows), S)
    q, c = whole_numbers(wl, n, S)
    see = tree_dev(T.random_tree(np.random.default_rng(S), wl.batch, n)[1]) if tree else None
    o, lse = attend_whole(wl, q, c, windows, see, n, split)
    for b, w in enumerate(windows):
        s, k, _, r, m = scores64(q, c, b, w, see, n)
        rl = s.logsumexp(-1)
        # in log2 units: the scale 2^-23 of a score (below 16), the exponent's own rounding 2^-20, the
        # exponential 2^-22; sums some 230 additions deep (64 keys of a block in four chains, 64 blocks
        # and their rescaling, 74 pieces); lse, below 16, rounds by 2^-21
        assert rl.abs().max() < 16 and s[s > -1e30].abs().max() < 16
        assert (lse[b, :m] - rl).abs().max() <= 2.0 ** -15
        p = (s - rl[..., None]).exp().flatten(0, 1)
        ref, spread = p @ k[:, :512], p @ k[:, :512].abs()
        err = (o[b, :m].double().flatten(0, 1) - ref).abs()
        assert (err <= T.BF16 * ref.abs() + (T.BF16 + 2.0 ** -15) * spread).all()
        assert (o[b, m:] == 0).all() and (lse[b, m:] == 0).all()
    for _ in range(20):
        o2, lse2 = attend_whole(wl, q, c, windows, see, n, split)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert mla.mla_device_error() == 0


GROUPS = [
    # (node, head) rows in groups of 128: whole nodes, several nodes, parts of nodes; 64 groups, more
    ("HEADS", 128, 16, 3000, 2), ("HEADS", 128, 40, 2500, 24), ("HEADS", 128, 16, 700, 40),
    ("HEADS", 128, 64, 900, 2), ("HEADS", 128, 65, 900, 2), ("HEADS", 128, 80, 1500, 3),
    ("HEADS", 96, 30, 1200, 3), ("HEADS", 24, 100, 1200, 3), ("HEADS", 24, 350, 900, 2),
    ("MAIN", 5, 70, 1200, 3), ("MAIN", 8, 300, 1200, 2), ("HEADS", 300, 11, 600, 3),
    ("WIDE", 128, 20, 1500, 2), ("WIDE", 128, 70, 700, 2), ("WIDE", 32, 33, 900, 24),
    ("WIDE", 8, 16, 1500, 4), ("WIDE", 24, 100, 600, 3),
]


@pytest.mark.parametrize("chain", [False, True])
@pytest.mark.parametrize("cfg,heads,n,S,B", GROUPS)
def test_weight_row_groups(cuda_ok, cfg, heads, n, S, B, chain):
    """Query weights that leave half of the nodes out, at random, in runs and all but one."""
    wl = T.workload(dict(getattr(T, cfg), n_heads=heads), B, S)
    shape = mla.make_shape(wl)
    rng = np.random.default_rng([n, S, heads])
    nodes = [n] + [int(rng.integers(1, n + 1)) for _ in range(B - 1)]
    windows = [(int(rng.integers(0, S)), int(rng.integers(0, S - m + 1)), m) for m in nodes]
    q, c = whole_numbers(wl, n, S)
    see = None if chain else tree_dev(T.random_tree(rng, B, n)[1])
    qw = (rng.random((B, n)) < 0.5) * rng.uniform(0.5, 2.0, (B, n))
    qw[0, n // 4:n // 2] = 0.0
    if B > 2:
        qw[1] = 0.0
        qw[1, nodes[1] - 1] = 1.0
        qw[2] = 0.0
    qw = torch.from_numpy(qw.astype(np.float32)).to(DEV)
    old = torch.rand((B, S), device=DEV)
    win = i32(windows)
    lse = torch.full((B, n, heads), float("nan"), device=DEV)
    parts = [scores64(q, c, b, w, see, n) for b, w in enumerate(windows)]
    for b, (s, _, _, _, m) in enumerate(parts):
        lse[b, :m] = s.logsumexp(-1).float()
    lse[0, 0, ::3] = float("-inf")
    for weights in (qw, None):
        out = torch.full((B, S), 7.0, device=DEV)
        mla.mla_attend_weight(shape, q, n, c, win, see, WHOLE, lse, weights, old, out)
        assert mla.mla_device_error() == 0
        for b, (s, _, at, r, m) in enumerate(parts):
            p = (s - lse[b, :m, :, None].double()).exp()
            p = p.masked_fill(torch.isneginf(lse[b, :m])[..., None], 0.0).sum(1)
            if weights is not None:
                p = p * qw[b, :m, None].double()
            ref = p.sum(0)
            ref[:r] += old[b, at[:r]].double()
            # all terms are positive: the exponents (below 32 in log2 units, rounded four times) and the
            # exponential, then sums of 32 rows' columns, one after the other
            rel = 2.0 ** -16 + (n * heads / 32 + 24) * T.F32
            err = (out[b, at].double() - ref).abs()
            assert (err <= rel * ref).all(), (b, float((err / ref).max()), rel)
            rest = torch.ones(S, device=DEV, dtype=torch.bool)
            rest[at] = False
            assert (out[b, rest] == 7.0).all()


@pytest.mark.parametrize("cfg,B,n,S", [("MAIN", 40, 128, 300), ("WIDE", 24, 100, 200)])
def test_write_more_tiles_than_sms(cuda_ok, cfg, B, n, S):
    """Rows of as many tiles as no split of K is for, ragged: own slots and positions, nothing else."""
    wl = T.workload(getattr(T, cfg), B, S)
    shape = mla.make_shape(wl)
    rng = np.random.default_rng(B)
    windows = [(int(rng.integers(0, S)), int(rng.integers(0, S - n + 1)), int(rng.integers(0, n + 1)))
               for _ in range(B)]
    d = wl.d_model
    h = T.normal(rng, (B, n, d), wl.dtype)
    w_dkv = T.normal(rng, (d, wl.d_latent), wl.dtype, d ** -0.5)
    w_kr = T.normal(rng, (d, wl.d_rope), wl.dtype, d ** -0.5)
    token = rng.integers(0, 200000, (B, n))
    ct = torch.full((B, S, wl.row_width), 7.0, device=DEV, dtype=torch.bfloat16)
    pos = torch.full((B, S), -1, dtype=torch.int32, device=DEV)
    mla.mla_tree_write(shape, P.upload(h), d, n, i32(windows), i32(token), P.upload(w_dkv),
                       P.upload(w_kr), ct, pos)
    assert mla.mla_device_error() == 0
    ref, rp = D.tree_write(np.full((B, S, wl.row_width), 7.0), np.full((B, S), -1), h.values,
                           w_dkv.values, w_kr.values, windows, token, wl)
    assert (pos.cpu().numpy() == rp).all()
    got, at = P.download(ct), rp >= 0
    assert (got[~at] == 7.0).all()
    # as in test_place: d + 2 roundings of sums of sum |h||w|, the rotation, one rounding to bf16
    size = np.linalg.norm(h.values, axis=-1).max() * max(
        np.linalg.norm(w_dkv.values, axis=0).max(), np.linalg.norm(w_kr.values, axis=0).max())
    T.check_within(got[at], ref[at], T.BF16 * np.abs(ref[at])
                   + 2 * size * ((d + 2) * 2 * T.F32 + 2.0 ** -20), "cache")


@pytest.mark.parametrize("B", [8192, 8200])
def test_thousands_of_sequences(cuda_ok, B):
    """On both sides of the most sequences whose tiles go in rounds: whole tiles give the bits of calls
    of a few sequences, and so do the weights."""
    n, S, H, part = 40, 90, 7, 1100
    wl = T.workload(dict(T.MAIN, n_heads=H), B, S)
    rng = np.random.default_rng(B)
    windows = np.stack([rng.integers(0, S, B), rng.integers(0, S - n + 1, B), rng.integers(0, n + 1, B)], 1)
    q, c = whole_numbers(wl, n, B)
    win, w0 = i32(windows), torch.rand((B, S), device=DEV)
    o, lse = attend_whole(wl, q, c, windows, None, n, split=False)
    out = torch.zeros((B, S), device=DEV)
    mla.mla_attend_weight(mla.make_shape(wl), q, n, c, win, None, WHOLE, lse, None, w0, out)
    for b in range(0, B, part):
        few = wl.scaled(batch=min(part, B - b))
        e = b + few.batch
        ob, lb = attend_whole(few, q[b:e], c[b:e], windows[b:e], None, n, split=False)
        assert torch.equal(ob, o[b:e]) and torch.equal(lb, lse[b:e])
        wb = torch.zeros((few.batch, S), device=DEV)
        mla.mla_attend_weight(mla.make_shape(few), q[b:e], n, c[b:e], win[b:e], None, WHOLE, lb, None,
                              w0[b:e], wb)
        assert torch.allclose(wb, out[b:e], rtol=2.0 ** -18, atol=0)      # (pairs may share a unit)
    for b in range(0, B, 509):                               # and some of them in 64 bits
        s, k, at, r, m = scores64(q, c, b, windows[b], None, n)
        if m:
            assert (lse[b, :m] - s.logsumexp(-1)).abs().max() <= 2.0 ** -15
    assert mla.mla_device_error() == 0


@pytest.mark.parametrize("cfg", ["TINY", "MAIN", "WIDE"])
@pytest.mark.parametrize("split", [True, False])
def test_attend_without_lse(cuda_ok, cfg, split):
    """No lse asked for: the same o_lat."""
    n, S, windows = 5, 2700, [(2600, 2650, 5), (0, 3, 2)]
    wl = T.workload(getattr(T, cfg), 2, S)
    shape = mla.make_shape(wl)
    rng = np.random.default_rng(1)
    q = P.upload(T.normal(rng, (2, n, wl.n_heads, wl.row_width), wl.dtype))
    c = P.upload(T.normal(rng, (2, S, wl.row_width), wl.dtype))
    o, _ = attend(wl, q, c, windows, None, n, split)
    o2 = torch.full_like(o, 7.0)
    nws = mla.mla_attend_tree_workspace_size(shape, n) if split else 0
    ws = torch.empty(nws, dtype=torch.uint8, device=DEV) if nws else None
    mla.mla_attend_tree(shape, q, n, c, i32(windows), None, SCALE, o2, None, ws)
    assert torch.equal(o, o2)
    assert mla.mla_device_error() == 0
