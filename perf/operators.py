"""Cases that time and check the draft-tree and cache-eviction operators.

A serving loop over a latent KV ring drafts a small tree of tokens for every sequence, writes
the nodes behind the sequence's context, attends with each node seeing the context and its
ancestors, keeps the accepted path, and now and then drops the context rows that attention has
used least.  The operators of that loop, each with its plain form beside it:

  place    the nodes' latent rows and queries, each rotated at its own position
  attend   attention of the tree's nodes over the context and their ancestors
  weight   the attention weight every cached row received, added to a running total
  accept   the accepted nodes' rows moved up behind the context
  evict    the least used context rows dropped, the kept ones moved into their slots

`listed` and `draw` give the cases, `prepare` what a program holds before the call, `run` one
pass, `work` the bytes and operations a pass cannot do without, `exact` the result in 64 bits.
"""

import math

import numpy as np
import torch

own = False

THETA = 10000.0


# ---------------------------------------------------------------------------- cases


def _case(op, dtype, batch, heads, d_latent, d_rope, pairs, nodes, nodes_min, rows, rows_min,
          ring, **more):
    """`rows` / `nodes` are the largest context and tree of the batch, `*_min` the smallest."""
    c = {"op": op, "dtype": dtype, "batch": batch, "heads": heads, "d_nope": 128,
         "d_latent": d_latent, "d_rope": d_rope, "pairs_t": pairs[0], "pairs_y": pairs[1],
         "pairs_x": pairs[2], "nodes": nodes, "nodes_min": nodes_min, "rows": rows,
         "rows_min": rows_min, "ring": ring}
    c.update(more)
    return c


def _bf(op, batch, heads, nodes, nodes_min, rows, rows_min, ring, **more):
    return _case(op, "bf16", batch, heads, 512, 64, (32, 0, 0), nodes, nodes_min, rows, rows_min,
                 ring, **more)


def listed():
    cases = [
        # one user, a short prompt, a handful of drafted tokens: latency is all that counts
        dict(_bf("attend", 1, 128, 5, 5, 211, 211, 256), name="attend_one_short"),
        # a full serving batch with ragged contexts and trees: the bulk of a serving step
        dict(_bf("attend", 32, 128, 32, 16, 8192, 2048, 8256), name="attend_batch_ragged"),
        # the wide positional key of a video ring, 32 heads, windows that wrap
        dict(_case("attend", "bf16", 4, 32, 512, 512, (64, 96, 96), 16, 9, 15000, 4001, 15600),
             name="attend_wide_key"),
        # the float32 check configuration: small heads, small latent
        dict(_case("attend", "f32", 2, 4, 64, 16, (2, 3, 3), 7, 3, 57, 20, 64, d_nope=32),
             name="attend_tiny_f32"),
        # one new token for each of 64 long sequences: the cache is read once, bytes count
        dict(_bf("weight", 64, 128, 1, 1, 8191, 8191, 8192), name="weight_decode"),
        # trees of a medium batch: every cached row against all nodes and heads
        dict(_bf("weight", 8, 128, 16, 7, 8100, 1025, 8192), name="weight_tree_ragged"),
        # steady state of a full cache: a few rows over the budget leave at each step
        dict(_bf("evict", 4, 128, 16, 0, 4112, 4099, 4160, keep=4096, sink=4, recent=256),
             name="evict_step"),
        # a long prompt cut down to the budget once it has been read
        dict(_bf("evict", 32, 128, 1, 0, 8192, 6001, 8192, keep=4096, sink=16, recent=512),
             name="evict_prompt"),
        # the accepted path of a small and of a large batch
        dict(_bf("accept", 2, 128, 8, 8, 500, 300, 512), name="accept_small"),
        dict(_bf("accept", 64, 128, 48, 17, 1900, 64, 2048), name="accept_batch"),
        # the nodes of a few sequences (weights are most of the bytes), and of a full batch
        dict(_bf("place", 4, 32, 8, 5, 1000, 100, 1024, d_model=4096), name="place_small"),
        dict(_bf("place", 32, 128, 32, 16, 1900, 200, 2048, d_model=4096), name="place_batch"),
    ]
    return cases


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "weight", "evict", "accept", "place"])
    if op in ("attend", "weight") and rng.random() < 0.15:
        # the check configuration and its neighbours
        rows = _log_int(rng, 1, 60)
        nodes = rng.randint(1, 9)
        return _case(op, "f32", rng.randint(1, 4), rng.randint(1, 6), 64, 16, (2, 3, 3), nodes,
                     rng.randint(1, nodes), rows, rng.randint(0, rows),
                     rows + nodes + rng.randint(0, 9), d_nope=32)
    heads = rng.choice([8, 16, 32, 64, 128, 128])
    if op in ("attend", "weight"):
        wide = rng.random() < 0.2
        rows = _log_int(rng, 1, 8192)
        rows_min = rng.randint(0, rows)
        nodes = _log_int(rng, 1, 40)
        # no dearer than the listed batch: batch x rows x nodes x heads is bounded
        most = int(64e6 / (rows * nodes * heads)) + 1
        batch = _log_int(rng, 1, max(1, min(48, most)))
        ring = rows + nodes + rng.randint(0, 200)
        if wide:
            return _case(op, "bf16", batch, heads, 512, 512, (64, 96, 96), nodes,
                         rng.randint(1, nodes), rows, rows_min, ring)
        return _bf(op, batch, heads, nodes, rng.randint(1, nodes), rows, rows_min, ring)
    if op == "evict":
        rows = _log_int(rng, 64, 8192)
        batch = _log_int(rng, 1, 32)
        keep = rng.randint(rows // 8 + 1, rows)
        return _bf("evict", batch, heads, 1, 0, rows, rng.randint(1, rows), rows + rng.randint(0, 99),
                   keep=keep, sink=rng.randint(0, 8), recent=rng.randint(0, keep // 2))
    if op == "accept":
        rows = _log_int(rng, 1, 2000)
        nodes = _log_int(rng, 1, 64)
        return _bf("accept", _log_int(rng, 1, 64), heads, nodes, rng.randint(0, nodes), rows,
                   rng.randint(0, rows), rows + nodes + rng.randint(0, 50))
    rows = _log_int(rng, 1, 2000)
    nodes = _log_int(rng, 1, 32)
    return _bf("place", _log_int(rng, 1, 32), heads, nodes, rng.randint(1, nodes), rows,
               rng.randint(0, rows), rows + nodes + rng.randint(0, 50),
               d_model=rng.choice([512, 1024, 2048, 4096]))


def _spread(lo, hi, n):
    """n whole numbers spread over [lo, hi], the largest among them; the same for every seed."""
    out = []
    for b in range(n):
        f = math.fmod((b + 1) * 0.6180339887498949, 1.0)
        out.append(hi if b == 0 else lo + int(f * (hi - lo) + 0.5))
    return out


def _rows(case):
    return _spread(case["rows_min"], case["rows"], case["batch"])


def _nodes(case):
    return _spread(case["nodes_min"], case["nodes"], case["batch"])


def _width(case):
    return case["d_latent"] + case["d_rope"]


def work(case):
    B, H, dc, w = case["batch"], case["heads"], case["d_latent"], _width(case)
    el = 4 if case["dtype"] == "f32" else 2
    rows, nodes = _rows(case), _nodes(case)
    op = case["op"]
    if op == "attend":
        # pairs of a node and a row it may see: the whole context, and about half the tree
        pairs = sum(m * n + m * (m + 1) // 2 for n, m in zip(rows, nodes))
        byts = sum((n + m) * w * el + m * H * ((w + dc) * el + 4) + m * m
                   for n, m in zip(rows, nodes))
        return {"bytes": byts, "flops": 2 * pairs * H * (w + dc)}
    if op == "weight":
        pairs = sum(m * n + m * (m + 1) // 2 for n, m in zip(rows, nodes))
        byts = sum((n + m) * (w * el + 8) + m * H * (w * el + 4) + m * m + 4 * m
                   for n, m in zip(rows, nodes))
        return {"bytes": byts, "flops": 2 * pairs * H * w}
    if op == "evict":
        keep = case["keep"]
        # of the rows that leave, the share keep / n sits where kept rows have to go
        moved = sum(keep * (n - keep) / n for n in rows if n > keep)
        scan = sum(8 * n for n in rows if n > keep)
        return {"bytes": int(scan + moved * (2 * w * el + 8) + 24 * B), "flops": sum(rows)}
    if op == "accept":
        # a path of about a third of the tree's depth; its rows move up unless in place
        moved = sum(math.log2(m + 1) for m in nodes)
        return {"bytes": int(sum(nodes) + moved * (2 * w * el + 16) + 24 * B),
                "flops": sum(nodes)}
    d, dn = case["d_model"], case["d_nope"]
    M = sum(nodes)
    byts = el * (M * d + d * w + M * w + case["batch"] * case["nodes"] * H * (dn + case["d_rope"] + w)
                 + H * dn * dc) + 8 * M
    return {"bytes": byts, "flops": 2 * M * d * w + 2 * B * case["nodes"] * H * dn * dc}


# ---------------------------------------------------------------------------- inputs


def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed((seed * 1000003 + salt) & 0x7FFFFFFF)
    return g


def _normal(shape, g, dtype, std=1.0):
    x = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=g)
    return x.to(dtype)


def _trees(case, rnd):
    """Parents, visibility (a node sees itself and its ancestors) and depths, on the host."""
    B, n = case["batch"], case["nodes"]
    see = np.zeros((B, n, n), dtype=bool)
    depth = np.zeros((B, n), dtype=np.int64)
    parent = np.full((B, n), -1, dtype=np.int64)
    for b, m in enumerate(_nodes(case)):
        for i in range(m):
            p = int(rnd.integers(max(-1, i - 6), i)) if i else -1
            parent[b, i] = p
            if p >= 0:
                see[b, i] = see[b, p]
                depth[b, i] = depth[b, p] + 1
            see[b, i, i] = True
    return parent, see, depth


def prepare(case, seed):
    B, H, n, S, w = case["batch"], case["heads"], case["nodes"], case["ring"], _width(case)
    dc, dr, dn = case["d_latent"], case["d_rope"], case["d_nope"]
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    rnd = np.random.default_rng([seed, 11])
    g = _gen(seed, 17)
    rows, nodes = _rows(case), _nodes(case)
    op = case["op"]
    st = {"case": case, "dt": dt, "rows": rows, "nodes": nodes, "scale": (dn + dr) ** -0.5}
    first = rnd.integers(0, S, size=B)
    st["first"] = [int(f) for f in first]
    live = [0 if op == "evict" else m for m in nodes]
    win = np.stack([first, np.array(rows), np.array(live)], axis=1).astype(np.int32)
    st["window"] = torch.from_numpy(win).cuda()
    parent, see, depth = _trees(case, rnd)
    st["tree"] = torch.from_numpy(see).cuda()
    if op != "place":
        st["cache"] = _normal((B, S, w), g, dt)
    else:
        st["cache"] = torch.zeros((B, S, w), dtype=dt, device="cuda")
    if op in ("attend", "weight"):
        st["q_abs"] = _normal((B, n, H, w), g, dt)
    if op == "attend":
        st["o_lat"] = torch.zeros((B, n, H, dc), dtype=dt, device="cuda")
        st["lse"] = torch.zeros((B, n, H), dtype=torch.float32, device="cuda")
    if op == "weight":
        st["query_weight"] = torch.from_numpy((rnd.random((B, n)) < 0.7).astype(np.float32)).cuda()
        st["query_weight"][:, 0] = 1.0
        st["weight_in"] = torch.empty((B, S), device="cuda").uniform_(0.0, 2.0, generator=g)
        st["weight_out"] = torch.zeros((B, S), device="cuda")
        st["lse"] = _lse_of(st)
    if op in ("evict", "accept"):
        # weights as attention leaves them: a few rows take most of it
        wt = torch.empty((B, S), device="cuda").exponential_(1.0, generator=g) ** 3
        # the rows' positions: in order along the window, with gaps of earlier evictions
        pos = np.zeros((B, S), dtype=np.int32)
        for b in range(B):
            k = rows[b] + live[b]
            gaps = np.cumsum(rnd.integers(1, 3, size=k)) - 1
            pos[b, (first[b] + np.arange(k)) % S] = gaps
        # one buffer, so that a pass can start from the same state with one copy
        keep0 = torch.empty((2 * B * S + 3 * B,), dtype=torch.int32, device="cuda")
        keep0[:B * S] = wt.view(torch.int32).reshape(-1)
        keep0[B * S:2 * B * S] = torch.from_numpy(pos).cuda().reshape(-1)
        keep0[2 * B * S:] = st["window"].reshape(-1)
        now = keep0.clone()
        st["start"], st["now"] = keep0, now
        st["weight"] = now[:B * S].view(torch.float32).view(B, S)
        st["position"] = now[B * S:2 * B * S].view(B, S)
        st["window"] = now[2 * B * S:].view(B, 3)
    if op == "accept":
        acc = np.zeros((B, n), dtype=bool)
        for b, m in enumerate(nodes):
            if m == 0:
                continue
            i = int(rnd.integers(0, m))
            while i >= 0:
                acc[b, i] = True
                i = int(parent[b, i])
        st["accept"] = torch.from_numpy(acc).cuda()
    if op == "place":
        d = case["d_model"]
        st["h"] = _normal((B, n, d), g, dt)
        st["w_dkv"] = _normal((d, dc), g, dt, d ** -0.5)
        st["w_kr"] = _normal((d, dr), g, dt, d ** -0.5)
        st["w_uk"] = _normal((H, dn, dc), g, dt, dc ** -0.5)
        st["q_nope"] = _normal((B, n, H, dn), g, dt)
        st["q_rope"] = _normal((B, n, H, dr), g, dt)
        tok = np.array(rows)[:, None] + rnd.integers(0, 100000, size=(B, 1)) + depth
        st["token"] = torch.from_numpy(tok.astype(np.int32)).cuda()
        st["q_abs"] = torch.zeros((B, n, H, w), dtype=dt, device="cuda")
        st["position"] = torch.zeros((B, S), dtype=torch.int32, device="cuda")
    if own:
        _prepare_own(st)
    return st


def _prepare_own(st):
    import latent_kv_cache_write_b200 as mla
    c = st["case"]
    shape = mla.MlaShape(batch=c["batch"], n_heads=c["heads"], d_nope=c["d_nope"],
                         d_latent=c["d_latent"], d_rope=c["d_rope"],
                         rope_pairs=(c["pairs_t"], c["pairs_y"], c["pairs_x"]),
                         rope_theta=THETA, grid_h=1, grid_w=1, ring_slots=c["ring"],
                         dtype=mla.native.MLA_F32 if c["dtype"] == "f32" else mla.native.MLA_BF16)
    st["mla"], st["shape"] = mla, shape
    n = 0
    if c["op"] == "attend":
        n = mla.mla_attend_tree_workspace_size(shape, c["nodes"])
    elif c["op"] in ("evict", "accept"):
        n = mla.mla_cache_evict_workspace_size(shape)
    st["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda") if n else None


def _keys(st, b, count, cast):
    """The first `count` rows of sequence b's window, context then nodes, in order."""
    S = st["case"]["ring"]
    idx = (torch.arange(count, device="cuda") + st["first"][b]) % S
    return st["cache"][b].index_select(0, idx).to(cast), idx


def _lse_of(st):
    """The log-sum-exps that the attention of these nodes left, float32."""
    c = st["case"]
    B, H, n = c["batch"], c["heads"], c["nodes"]
    out = torch.zeros((B, n, H), dtype=torch.float32, device="cuda")
    for b in range(B):
        m, r = st["nodes"][b], st["rows"][b]
        k, _ = _keys(st, b, r + m, torch.float32)
        s = (st["q_abs"][b, :m].float().reshape(m * H, -1) @ k.t()).view(m, H, r + m) * st["scale"]
        s[:, :, r:] = s[:, :, r:].masked_fill(~st["tree"][b, :m, None, :m], float("-inf"))
        out[b, :m] = torch.logsumexp(s, -1)
    return out


# ---------------------------------------------------------------------------- the plain forms


def _plain_attend(st):
    c = st["case"]
    H, dc = c["heads"], c["d_latent"]
    for b in range(c["batch"]):
        m, r = st["nodes"][b], st["rows"][b]
        if m == 0:
            continue
        k, _ = _keys(st, b, r + m, torch.float32)
        q = st["q_abs"][b, :m].float().reshape(m * H, -1)
        s = (q @ k.t()).view(m, H, r + m) * st["scale"]
        s[:, :, r:] = s[:, :, r:].masked_fill(~st["tree"][b, :m, None, :m], float("-inf"))
        top = s.amax(-1, keepdim=True)
        p = torch.exp(s - top)
        total = p.sum(-1, keepdim=True)
        o = (p.view(m * H, -1) @ k[:, :dc]).view(m, H, dc) / total
        st["o_lat"][b, :m] = o.to(st["dt"])
        st["lse"][b, :m] = (top + torch.log(total)).squeeze(-1)
    return st["o_lat"], st["lse"]


def _plain_weight(st):
    c = st["case"]
    H = c["heads"]
    for b in range(c["batch"]):
        m, r = st["nodes"][b], st["rows"][b]
        k, idx = _keys(st, b, r + m, torch.float32)
        q = st["q_abs"][b, :m].float().reshape(m * H, -1)
        s = (q @ k.t()).view(m, H, r + m) * st["scale"]
        p = torch.exp(s - st["lse"][b, :m, :, None])
        p[:, :, r:] = p[:, :, r:] * st["tree"][b, :m, None, :m]
        new = (p * st["query_weight"][b, :m, None, None]).sum((0, 1))
        old = st["weight_in"][b].index_select(0, idx)
        old[r:] = 0.0
        st["weight_out"][b].index_copy_(0, idx, old + new)
    return st["weight_out"]


def _fill_holes(st, b, kept, base, slots):
    """Kept rows at or past index base + count move into the holes before it, in order."""
    count = int(kept.sum())
    dst = torch.nonzero(~kept[:count]).flatten()
    src = torch.nonzero(kept[count:]).flatten() + count
    d, s = slots[base + dst], slots[base + src]
    st["cache"][b].index_copy_(0, d, st["cache"][b].index_select(0, s))
    for x in (st["weight"][b], st["position"][b]):
        x.index_copy_(0, d, x.index_select(0, s))
    return count


def _plain_evict(st):
    c = st["case"]
    S, keep = c["ring"], c["keep"]
    for b in range(c["batch"]):
        n = st["rows"][b]
        slots = (torch.arange(n, device="cuda") + st["first"][b]) % S
        if n > keep:
            w, pos = st["weight"][b][slots], st["position"][b][slots]
            rank = torch.where((pos < c["sink"]) | (pos > pos.max() - c["recent"]),
                               torch.full_like(w, float("inf")), w)
            order = torch.sort(rank, descending=True, stable=True).indices
            kept = torch.zeros(n, dtype=torch.bool, device="cuda")
            kept[order[:keep]] = True
            _fill_holes(st, b, kept, 0, slots)
            st["window"][b, 1] = keep
    return st["cache"], st["weight"], st["position"], st["window"]


def _plain_accept(st):
    c = st["case"]
    for b in range(c["batch"]):
        n, m = st["rows"][b], st["nodes"][b]
        slots = (torch.arange(n + m, device="cuda") + st["first"][b]) % c["ring"]
        count = _fill_holes(st, b, st["accept"][b, :m], n, slots) if m else 0
        st["window"][b, 1] = n + count
        st["window"][b, 2] = 0
    return st["cache"], st["weight"], st["position"], st["window"]


def _angles(case, token):
    """Rotation angle of every pair for each token (a frame is one token): float64."""
    inv = []
    for a in ("pairs_t", "pairs_y", "pairs_x"):
        n = case[a]
        f = THETA ** (-torch.arange(n, dtype=torch.float64, device="cuda") / max(n, 1))
        inv.append(f if a == "pairs_t" else f * 0.0)
    return token.double()[..., None] * torch.cat(inv)


def _rotate(x, cos, sin):
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)


def _plain_place(st):
    c = st["case"]
    B, n, dc = c["batch"], c["nodes"], c["d_latent"]
    ang = _angles(c, st["token"])
    cos, sin = torch.cos(ang).float(), torch.sin(ang).float()
    h = st["h"].float().view(B * n, -1)
    lat = (h @ st["w_dkv"].float()).view(B, n, dc)
    key = _rotate((h @ st["w_kr"].float()).view(B, n, -1), cos, sin)
    row = torch.cat((lat, key), -1).to(st["dt"])
    for b in range(B):
        m = st["nodes"][b]
        idx = (torch.arange(m, device="cuda") + st["first"][b] + st["rows"][b]) % c["ring"]
        st["cache"][b].index_copy_(0, idx, row[b, :m])
        st["position"][b].index_copy_(0, idx, st["token"][b, :m])
    q = torch.einsum("bihd,hdc->bihc", st["q_nope"].float(), st["w_uk"].float())
    qr = _rotate(st["q_rope"].float(), cos[:, :, None], sin[:, :, None])
    st["q_abs"].copy_(torch.cat((q, qr), -1))
    return st["cache"], st["position"], st["q_abs"]


# ---------------------------------------------------------------------------- one pass


def run(st):
    c = st["case"]
    op, n = c["op"], c["nodes"]
    if op in ("evict", "accept"):
        st["now"].copy_(st["start"])       # every pass drops or accepts from the same state
    if not own:
        return {"attend": _plain_attend, "weight": _plain_weight, "evict": _plain_evict,
                "accept": _plain_accept, "place": _plain_place}[op](st)
    mla, shape, ws = st["mla"], st["shape"], st["workspace"]
    if op == "attend":
        mla.mla_attend_tree(shape, st["q_abs"], n, st["cache"], st["window"], st["tree"],
                            st["scale"], st["o_lat"], st["lse"], ws)
        return st["o_lat"], st["lse"]
    if op == "weight":
        mla.mla_attend_weight(shape, st["q_abs"], n, st["cache"], st["window"], st["tree"],
                              st["scale"], st["lse"], st["query_weight"], st["weight_in"],
                              st["weight_out"])
        return st["weight_out"]
    if op == "evict":
        mla.mla_cache_evict(shape, st["cache"], c["keep"], c["sink"], c["recent"], st["window"],
                            st["weight"], st["position"], ws)
        return st["cache"], st["weight"], st["position"], st["window"]
    if op == "accept":
        mla.mla_tree_accept(shape, st["cache"], n, st["accept"], st["window"], st["weight"],
                            st["position"], ws)
        return st["cache"], st["weight"], st["position"], st["window"]
    mla.mla_tree_write(shape, st["h"], c["d_model"], n, st["window"], st["token"], st["w_dkv"],
                       st["w_kr"], st["cache"], st["position"])
    mla.mla_tree_absorb_q(shape, st["q_nope"], st["q_rope"], n, st["token"], st["w_uk"],
                          st["q_abs"])
    return st["cache"], st["position"], st["q_abs"]


# ---------------------------------------------------------------------------- 64 bits


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    S, B, H, n = case["ring"], case["batch"], case["heads"], case["nodes"]
    dc = case["d_latent"]
    f64 = torch.float64

    def slot(b, j):
        return (st["first"][b] + j) % S

    if op in ("attend", "weight"):
        lat = torch.zeros((B, n, H, dc), dtype=f64, device="cuda")
        lse = torch.zeros((B, n, H), dtype=f64, device="cuda")
        tot = torch.zeros((B, S), dtype=f64, device="cuda")
        for b in range(B):
            r, m = st["rows"][b], st["nodes"][b]
            where = torch.tensor([slot(b, j) for j in range(r + m)], device="cuda")
            rows = st["cache"][b, where].double()
            if op == "weight":
                tot[b, where[:r]] = st["weight_in"][b, where[:r]].double()
            for i in range(m):
                # the rows node i sees, gathered: nothing else enters its sums
                vis = torch.cat((torch.ones(r, dtype=torch.bool, device="cuda"),
                                 st["tree"][b, i, :m]))
                sc = st["q_abs"][b, i].double() @ rows[vis].t() * st["scale"]
                if op == "attend":
                    lse[b, i] = torch.logsumexp(sc, 1)
                    lat[b, i] = torch.softmax(sc, 1) @ rows[vis, :dc]
                else:
                    p = torch.exp(sc - st["lse"][b, i].double()[:, None]).sum(0)
                    tot[b].index_add_(0, where[vis], p * st["query_weight"][b, i].double())
        return (lat, lse) if op == "attend" else tot
    if op in ("evict", "accept"):
        cache = st["cache"].double()
        wt, pos = st["weight"].double(), st["position"].double()
        win = st["window"].double()
        hw, hp = st["weight"].cpu().numpy(), st["position"].cpu().numpy()
        for b in range(B):
            r, m = st["rows"][b], st["nodes"][b]
            if op == "evict":
                if r <= case["keep"]:
                    continue
                sl = [slot(b, j) for j in range(r)]
                newest = max(hp[b, s] for s in sl)
                safe = [hp[b, s] < case["sink"] or hp[b, s] > newest - case["recent"] for s in sl]
                ranked = sorted(range(r), key=lambda j: (not safe[j], 0.0 if safe[j]
                                                         else -float(hw[b, sl[j]]), j))
                kept, lo, cnt = set(ranked[:case["keep"]]), 0, case["keep"]
                hi = r
                win[b, 1] = cnt
            else:
                acc = st["accept"][b, :m].cpu().numpy()
                kept, lo, hi = {r + i for i in range(m) if acc[i]}, r, r + m
                cnt = len(kept)
                win[b, 1], win[b, 2] = r + cnt, 0
            holes = [slot(b, j) for j in range(lo, lo + cnt) if j not in kept]
            late = [slot(b, j) for j in range(lo + cnt, hi) if j in kept]
            if holes:
                cache[b, holes] = cache[b, late]
                wt[b, holes] = wt[b, late]
                pos[b, holes] = pos[b, late]
        return cache, wt, pos.to(torch.int32), win.to(torch.int32)

    # place: the rotation as a product of complex numbers
    def turned(x, tok):
        k = x.shape[-1] // 2
        z = torch.view_as_complex(x.reshape(*x.shape[:-1], k, 2).contiguous())
        ang = torch.zeros((*tok.shape, k), dtype=f64, device="cuda")
        for j in range(case["pairs_t"]):
            ang[..., j] = tok.double() * THETA ** (-j / case["pairs_t"])
        while ang.dim() < z.dim():
            ang = ang.unsqueeze(-2)
        return torch.view_as_real(z * torch.polar(torch.ones_like(ang), ang)).flatten(-2)

    cache = st["cache"].double()
    position = st["position"].clone()
    q_abs = torch.zeros((B, n, H, _width(case)), dtype=f64, device="cuda")
    for b in range(B):
        tok, hb = st["token"][b], st["h"][b].double()
        rows = torch.cat((hb @ st["w_dkv"].double(), turned(hb @ st["w_kr"].double(), tok)), 1)
        for i in range(st["nodes"][b]):
            cache[b, slot(b, st["rows"][b] + i)] = rows[i]
            position[b, slot(b, st["rows"][b] + i)] = tok[i]
        for i in range(n):
            q_abs[b, i, :, :dc] = torch.bmm(st["q_nope"][b, i].double()[:, None],
                                            st["w_uk"].double())[:, 0]
        q_abs[b, :, :, dc:] = turned(st["q_rope"][b].double(), tok)
    return cache, position, q_abs
