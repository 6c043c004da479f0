"""Block-sparse chunk attention and the paged K/V store: the operators, their plain forms and cases.

Keys lie in segments: a latent frame of T = frame_w * frame_h rows in a store,
the whole sequence in explicit buffers.  A segment is cut into blocks of 128
keys, its last block ragged; queries are cut into groups of 256.

* summarize: the mean of every block's keys;
* select: per (head, query group), the `keep` blocks whose mean key has the
  largest product with the group's mean query, ties to the lowest index;
* attend: softmax attention of each group over the blocks of its list;
* paged: chunk attention of streams that share pages of a paged store;
* fork, compact: page copies of the paged store.

Where `own` is false, `run` computes them with elementary torch operations;
where it is true, through `same_step_kv_b200.pv`.
"""
import math

import torch

own = False

BLOCK = 128   # keys of a block
GROUP = 256   # queries of a group
FIRST = 3     # latent frames of the first chunk


# ------------------------------------------------------------------ cases
def listed():
    return [
        # after the append of one steady chunk: the new frame's 7 blocks per head
        dict(name="summarize_chunk", op="summarize_store", heads=24, head_dim=128, frame_w=40,
             frame_h=22, ring=18, chunks="28"),
        # a whole clip at once, before sparse whole-video attention
        dict(name="summarize_clip", op="summarize_dense", heads=24, head_dim=128, n_k=18480),
        # one query (a probe token, a register token) against a long key set
        dict(name="select_token", op="select_dense", heads=24, head_dim=128, n_q=1, n_k=40007,
             keep=32, front=4),
        # one layer of the steady chunk: a quarter of 147 blocks, sink and own frame always
        dict(name="select_chunk", op="select_store", heads=24, head_dim=128, frame_w=40, frame_h=22,
             ring=18, chunks="28", keep=37, force=3),
        # whole clip: 73 query groups of every head
        dict(name="select_clip", op="select_dense", heads=24, head_dim=128, n_q=18480, n_k=18480,
             keep=36, front=0),
        # one query over its 32 blocks: few rows, work split along the keys
        dict(name="attend_token", op="attend_dense", heads=24, head_dim=128, n_q=1, n_k=40007, keep=32),
        # one layer of the steady chunk
        dict(name="attend_chunk", op="attend_store", heads=24, head_dim=128, frame_w=40, frame_h=22,
             ring=18, chunks="28", keep=37),
        # several streams at ragged ring fills, 64-wide heads, frames that end inside a block
        dict(name="attend_streams", op="attend_store", heads=12, head_dim=64, frame_w=37, frame_h=21,
             ring=18, chunks="1,4,9,23", keep=33),
        # whole clip
        dict(name="attend_clip", op="attend_dense", heads=24, head_dim=128, n_q=18480, n_k=18480, keep=36),
        # four branches of one video that share every page but their own frame
        dict(name="paged_branches", op="paged", heads=24, head_dim=128, frame_w=40, frame_h=22, ring=18,
             chunk=12, branches=4),
        # branching while a chunk is being denoised: its page is copied for each branch
        dict(name="fork_chunk", op="fork", heads=24, head_dim=128, frame_w=40, frame_h=22, ring=6,
             layers=4, steps=4, chunk=5, branches=3),
        # a stream ended and the other one's pages move down
        dict(name="compact_stream", op="compact", heads=24, head_dim=128, frame_w=40, frame_h=22, ring=18,
             layers=1, steps=4, chunk=18),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _store(rng, op, most):
    """A store of random geometry whose keys over all streams stay below `most` values."""
    while True:
        c = dict(op=op, heads=rng.randint(1, 24), head_dim=rng.choice([64, 128]), frame_w=_log(rng, 2, 48),
                 frame_h=_log(rng, 2, 27), ring=rng.randint(1, 18))
        n = rng.choice([1, 1, 2, 3, 4])
        c["chunks"] = ",".join(str(rng.randint(1, 30)) for _ in range(n))
        if n * c["heads"] * c["head_dim"] * c["frame_w"] * c["frame_h"] * (FIRST + c["ring"]) <= most:
            return c


def draw(rng):
    op = rng.choice(["summarize_store", "summarize_dense", "select_store", "select_dense", "attend_store",
                     "attend_store", "attend_dense", "attend_dense", "paged", "fork", "compact"])
    if op == "summarize_dense":
        return dict(op=op, heads=rng.randint(1, 24), head_dim=rng.choice([64, 128]), n_k=_log(rng, 1, 18480))
    if op in ("select_dense", "attend_dense"):
        heads, dim, n_q = rng.randint(1, 24), rng.choice([64, 128]), _log(rng, 1, 18480)
        n_k = _log(rng, 1, min(60000, 18480 * 18480 // n_q))
        nb = -(-n_k // BLOCK)
        keep = _log(rng, 1, max(1, min(nb, 64)))
        while op == "attend_dense" and n_q * keep > 18480 * 36:
            keep //= 2
        c = dict(op=op, heads=heads, head_dim=dim, n_q=n_q, n_k=n_k, keep=keep)
        if op == "select_dense":
            c["front"] = rng.randint(0, min(keep, 4))
        return c
    if op in ("summarize_store", "select_store", "attend_store"):
        c = _store(rng, op, 24 * 128 * 18480 * 2)
        bps = -(-(c["frame_w"] * c["frame_h"]) // BLOCK)
        if op != "summarize_store":
            c["keep"] = (FIRST + 1) * bps + rng.randint(0, 2 * c["ring"])
        if op == "select_store":
            c["force"] = rng.choice([0, 1, 2, 3])
        return c
    if op == "paged":
        while True:
            c = _store(rng, op, 24 * 128 * 18480)
            c["chunk"], c["branches"] = int(c.pop("chunks").split(",")[0]), rng.randint(1, 5)
            q = c["branches"] * c["heads"] * c["head_dim"] * c["frame_w"] * c["frame_h"]
            if q <= 3 * 24 * 128 * 880:
                return c
    while True:
        c = dict(op=op, heads=rng.randint(1, 24), head_dim=rng.choice([64, 128]), frame_w=_log(rng, 4, 48),
                 frame_h=_log(rng, 4, 27), ring=rng.randint(2, 18), layers=rng.randint(1, 4),
                 steps=rng.randint(1, 4), chunk=rng.randint(1, 24))
        if op == "fork":
            c["branches"] = rng.randint(2, 6)
        page = c["heads"] * c["head_dim"] * c["frame_w"] * c["frame_h"] * c["layers"] * c["steps"]
        pages = c["branches"] if op == "fork" else FIRST + min(c["chunk"], c["ring"])
        room = FIRST + min(c["chunk"], c["ring"]) + 6 if op == "fork" else 2 * pages
        if 10 ** 5 < page * pages <= 24 * 128 * 880 * 4 * 21 and page * room * 4 <= 8e9:
            return c


# ------------------------------------------------------------------ geometry
def _blocks(n):
    return -(-n // BLOCK)


def _geom(c):
    """(tokens per frame, blocks per frame, [(chunk, fill, slot)] per stream) of a store case."""
    t = c["frame_w"] * c["frame_h"]
    js = [int(x) for x in c["chunks"].split(",")]
    return t, _blocks(t), [(j, min(j, c["ring"]), (j - 1) % c["ring"]) for j in js]


def _branch_pages(c):
    """Page of every segment for each branch of a `paged` case: the history of `chunk` chunks is
    stream 0's, pages taken lowest first; then each branch in turn starts its own next chunk."""
    j, r, n = c["chunk"], c["ring"], c["branches"]
    fill, slot = min(j, r), j % r
    hist = list(range(FIRST + fill))
    tables = []
    for i in range(n):
        p = list(hist)
        if j < r:
            p.append(FIRST + fill + i)
        elif i < n - 1:
            p[FIRST + slot] = FIRST + r + i
        tables.append(p)      # the last holder of a full ring's page writes in place
    return tables


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _tokens(g, heads, n, dim):
    """bf16 [heads][n][dim] of unit variance: noise, an offset shared by runs of 64 neighbouring
    tokens (a region of the picture) and a bias of the channel (the projection's)."""
    x = torch.randn(heads, n, dim, generator=g, device="cuda")
    x += 0.5 * torch.randn(heads, -(-n // 64), dim, generator=g, device="cuda").repeat_interleave(64, 1)[:, :n]
    x += 0.25 * torch.randn(heads, 1, dim, generator=g, device="cuda")
    return (x / 1.146).to(torch.bfloat16)


def _inputs(c, seed):
    """The operands of a case that does not move pages, without this repository's code."""
    g = _gen(seed)
    h, d, op = c["heads"], c["head_dim"], c["op"]
    x = {}
    if op in ("summarize_dense", "select_dense", "attend_dense"):
        x["k"] = _tokens(g, h, c["n_k"], d)
        if op != "summarize_dense":
            x["q"] = _tokens(g, h, c["n_q"], d)
        if op == "attend_dense":
            x["v"] = _tokens(g, h, c["n_k"], d)
        return x
    t = c["frame_w"] * c["frame_h"]
    if op == "paged":
        tables = _branch_pages(c)
        rows = (max(max(p) for p in tables) + 1) * t
        x["k"], x["v"] = _tokens(g, h, rows, d), _tokens(g, h, rows, d)
        x["q"] = torch.cat([_tokens(g, h, t, d).reshape(-1, d) for _ in tables])
        return x
    _, _, streams = _geom(c)
    rows = (FIRST + c["ring"]) * t
    x["k"] = torch.stack([_tokens(g, h, rows, d) for _ in streams])
    if op != "summarize_store":
        x["q"] = torch.cat([_tokens(g, h, t, d).reshape(-1, d) for _ in streams])
    if op == "attend_store":
        x["v"] = torch.stack([_tokens(g, h, rows, d) for _ in streams])
    return x


# ------------------------------------------------------------------ plain forms
def _means(x, size):
    """f32 [heads][ceil(n / size)][dim]: the means of runs of `size` rows, sums in 64 bits."""
    h, n, d = x.shape
    m = -(-n // size)
    pad = torch.zeros(h, m * size, d, dtype=torch.float64, device=x.device)
    pad[:, :n] = x
    rows = torch.full((m,), size, dtype=torch.float64, device=x.device)
    rows[-1] = n - (m - 1) * size
    return (pad.view(h, m, size, d).sum(2) / rows[None, :, None]).float()


def _frame_means(k, t):
    """The block means of every frame of k [heads][frames * t][dim]: [heads][frames * bps][dim]."""
    h, n, d = k.shape
    return _means(k.reshape(h * (n // t), t, d), BLOCK).reshape(h, -1, d)


def _select(q, means, keep, forced):
    """int32 [heads][groups][keep]: the best blocks of each query group, ascending, -1 behind them."""
    s = torch.matmul(_means(q, GROUP).double(), means.double().transpose(1, 2))
    s[:, :, forced] = math.inf
    n = min(keep, s.shape[2])
    best = torch.sort(s, dim=2, descending=True, stable=True).indices[:, :, :n].sort(2).values
    out = torch.full((*s.shape[:2], keep), -1, dtype=torch.int32, device=q.device)
    out[:, :, :n] = best
    return out


def _forced(c, fill, slot, bps):
    """The block indices that `force` takes always: 1 the sink's, 2 the current frame's."""
    b = torch.zeros((FIRST + fill) * bps, dtype=torch.bool, device="cuda")
    if c.get("force", 0) & 1:
        b[:FIRST * bps] = True
    if c.get("force", 0) & 2:
        b[(FIRST + slot) * bps:(FIRST + slot + 1) * bps] = True
    return b


def _rows_of(blocks, seg, bps):
    """(rows, valid) of the listed blocks: [..., n * 128]."""
    off = torch.arange(BLOCK, device=blocks.device)
    b = blocks.long()
    inside = (b % bps * BLOCK)[..., None] + off
    ok = (inside < seg) & (b >= 0)[..., None]
    rows = torch.where(ok, (b // bps * seg)[..., None] + inside, 0)
    return rows.flatten(-2), ok.flatten(-2)


def _attend(q, k, v, blocks, seg, bps):
    """Attention of q [heads][n][dim] over each group's blocks: out [n][heads][dim], lse [n][heads]."""
    h, n, d = q.shape
    out = torch.empty(n, h, d, dtype=torch.bfloat16, device=q.device)
    lse = torch.empty(n, h, dtype=torch.float32, device=q.device)
    groups = blocks.shape[1]
    step = max(1, 100_000_000 // (GROUP * blocks.shape[2] * BLOCK))
    for i in range(h):
        kf, vf = k[i].float(), v[i].float()
        for a in range(0, groups, step):
            e = min(groups, a + step)
            rows, ok = _rows_of(blocks[i, a:e], seg, bps)
            qg = torch.zeros((e - a) * GROUP, d, device=q.device)
            part = q[i, a * GROUP:e * GROUP]
            qg[:part.shape[0]] = part
            s = torch.matmul(qg.view(e - a, GROUP, d), kf[rows].transpose(1, 2)) / math.sqrt(d)
            s.masked_fill_(~ok[:, None, :], -math.inf)
            m = s.amax(2, keepdim=True)
            p = torch.exp(s - m)
            total = p.sum(2, keepdim=True)
            o = (torch.matmul(p, vf[rows]) / total).view(-1, d)[:part.shape[0]]
            out[a * GROUP:a * GROUP + part.shape[0], i] = o.to(torch.bfloat16)
            lse[a * GROUP:a * GROUP + part.shape[0], i] = (m + total.log()).view(-1)[:part.shape[0]]
    return out, lse


def _lists(c, x):
    """The lists that an attention case reads, chosen as `select` chooses them."""
    if c["op"] == "attend_dense":
        forced = torch.zeros(_blocks(c["n_k"]), dtype=torch.bool, device="cuda")
        return _select(x["q"], _means(x["k"], BLOCK), c["keep"], forced)
    t, bps, streams = _geom(c)
    h, d = c["heads"], c["head_dim"]
    lists = []
    for i, (_, fill, slot) in enumerate(streams):
        m = _frame_means(x["k"][i][:, :(FIRST + fill) * t], t)
        q = x["q"][i * h * t:(i + 1) * h * t].view(h, t, d)
        lists.append(_select(q, m, c["keep"], _forced(dict(force=3), fill, slot, bps)).reshape(-1, c["keep"]))
    return torch.cat(lists)


# ------------------------------------------------------------------ states
def _steady(pv, chunk):
    st = pv.pv_kv_state()
    st.phase, st.chunk = pv.PV_PHASE_STEADY, chunk
    return st


def _own_store(c, x):
    from same_step_kv_b200 import pv
    _, _, streams = _geom(c)
    cfg = pv.make_config(1, c["heads"], c["head_dim"], c["frame_w"], c["frame_h"], ring_slots=c["ring"],
                         steps=1, max_streams=len(streams))
    store = pv.KVStore(cfg, summaries=c["op"] != "attend_store")
    for i, (j, _, _) in enumerate(streams):
        pv.pv_kv_set_state(store.handle, i, _steady(pv, j))
        store.k_region()[0, 0, i] = x["k"][i]
        if "v" in x:
            store.v_region()[0, 0, i] = x["v"][i]
    return store


def _prepare_pages(c, seed, through):
    """K and V regions [layers][steps][heads][pages * T][dim] and what moves between their pages."""
    t = c["frame_w"] * c["frame_h"]
    live = FIRST + min(c["chunk"], c["ring"])
    pages = live + c["branches"] - 1 if c["op"] == "fork" else 2 * live
    s = dict(case=c, live=live)
    shape = (c["layers"], c["steps"], c["heads"], pages * t, c["head_dim"])
    if through:
        from same_step_kv_b200 import pv
        cfg = pv.make_config(c["layers"], c["heads"], c["head_dim"], c["frame_w"], c["frame_h"],
                             ring_slots=c["ring"], steps=c["steps"], max_streams=c.get("branches", 2))
        store = pv.KVStore(cfg, pages=pages)
        for i in range(1 if c["op"] == "fork" else 2):
            pv.pv_kv_set_state(store.handle, i, _steady(pv, c["chunk"]))
        s |= dict(store=store, ends=0)
        s["k"], s["v"] = store.k_region(), store.v_region()
    else:
        s["k"], s["v"] = (torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert tuple(s["k"].shape) == shape
    g = _gen(seed)
    for r in (s["k"], s["v"]):
        for i in range(c["layers"]):
            for j in range(c["steps"]):
                r[i, j] = torch.randn(shape[2:], generator=g, device="cuda", dtype=torch.bfloat16)
    return s


def prepare(case, seed):
    c = dict(case)
    if c["op"] in ("fork", "compact"):
        return _prepare_pages(c, seed, own)
    x = _inputs(c, seed)
    s = dict(case=c, **x)
    h, d, op = c["heads"], c["head_dim"], c["op"]
    if op in ("select_dense", "select_store"):
        if op == "select_dense":
            s["means"] = _means(x["k"], BLOCK)
        else:
            t, bps, streams = _geom(c)
            s["means"] = [_frame_means(x["k"][i], t) for i in range(len(streams))]
    if op in ("attend_dense", "attend_store"):
        s["blocks"] = _lists(c, x)
    if not own:
        return s
    from same_step_kv_b200 import pv
    new = lambda *shape, dtype=torch.bfloat16: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    if op == "summarize_dense":
        s["out"] = new(h, _blocks(c["n_k"]), d, dtype=torch.float32)
    elif op == "select_dense":
        s["out"] = new(h, -(-c["n_q"] // GROUP), c["keep"], dtype=torch.int32)
    elif op == "attend_dense":
        s["ws_bytes"] = pv.pv_block_attn_dense_ws_bytes(c["n_q"], c["n_k"], h, d, c["keep"])
        s["ws"] = torch.zeros(s["ws_bytes"], dtype=torch.uint8, device="cuda")
        s["out"], s["lse"] = new(c["n_q"], h, d), new(c["n_q"], h, dtype=torch.float32)
    elif op == "paged":
        t, n = c["frame_w"] * c["frame_h"], c["branches"]
        cfg = pv.make_config(1, h, d, c["frame_w"], c["frame_h"], ring_slots=c["ring"], steps=1, max_streams=n)
        s["store"] = store = pv.KVStore(cfg, pages=x["k"].shape[1] // t)
        pv.pv_kv_set_state(store.handle, 0, _steady(pv, c["chunk"]))
        if n > 1:
            pv.pv_kv_fork(store.handle, 0, range(1, n), 0)
        for i in range(n):
            pv.pv_kv_begin_chunk(store.handle, i, 1)
        store.k_region()[0, 0], store.v_region()[0, 0] = x["k"], x["v"]
        s["out"], s["lse"] = new(n * t, h, d), new(n * t, h, dtype=torch.float32)
    else:
        t, bps, streams = _geom(c)
        s["store"] = store = _own_store(c, x)
        n = len(streams)
        s["ids"] = list(range(n))
        if op == "select_store":
            s["out"] = new(n * h * -(-t // GROUP), c["keep"], dtype=torch.int32)
            region = store.summary_region()
            for i in range(n):
                region[0, 0, i] = s["means"][i]
        elif op == "attend_store":
            s["out"], s["lse"] = new(n * t, h, d), new(n * t, h, dtype=torch.float32)
    return s


# ------------------------------------------------------------------ one pass
def _run_own(s):
    from same_step_kv_b200 import pv
    c = s["case"]
    h, d, op = c["heads"], c["head_dim"], c["op"]
    if op == "summarize_dense":
        pv.pv_block_summarize_dense(s["k"], c["n_k"], h, d, s["out"])
        return s["out"]
    if op == "summarize_store":
        pv.pv_block_summarize(s["store"].handle, s["ids"], 0, 0)
        _, bps, streams = _geom(c)
        region = s["store"].summary_region()
        return [region[0, 0, i, :, (FIRST + slot) * bps:(FIRST + slot + 1) * bps]
                for i, (_, _, slot) in enumerate(streams)]
    if op == "select_dense":
        pv.pv_block_select_dense(s["q"], s["means"], c["n_q"], c["n_k"], h, d, c["keep"], c["front"], s["out"])
        return s["out"]
    if op == "select_store":
        pv.pv_block_select(s["store"].handle, s["ids"], 0, 0, s["q"], c["keep"], c["force"], s["out"])
        return s["out"]
    if op == "attend_dense":
        pv.pv_block_attn_dense(s["q"], s["k"], s["v"], c["n_q"], c["n_k"], h, d, s["blocks"], c["keep"],
                               s["out"], s["lse"], s["ws"], s["ws_bytes"])
        return s["out"], s["lse"]
    if op == "attend_store":
        pv.pv_block_attn(s["store"].handle, s["ids"], 0, 0, s["q"], s["blocks"], c["keep"], s["out"], s["lse"])
        return s["out"], s["lse"]
    if op == "paged":
        pv.pv_chunk_attn(s["store"].handle, range(c["branches"]), 0, 0, s["q"], s["out"], s["lse"])
        return s["out"], s["lse"]
    kv = s["store"].handle
    if op == "fork":
        pv.pv_kv_fork(kv, 0, range(1, c["branches"]), 1)
        for i in range(1, c["branches"]):
            pv.pv_kv_release(kv, i)
    else:  # the stream in the low pages ends, the other one moves down, a new one starts behind it
        pv.pv_kv_release(kv, s["ends"])
        pv.pv_kv_compact(kv)
        pv.pv_kv_set_state(kv, s["ends"], _steady(pv, c["chunk"]))
        s["ends"] = 1 - s["ends"]
    return _moved(s)


def _moved(s):
    """The pages that a fork or a compaction wrote."""
    c = s["case"]
    t = c["frame_w"] * c["frame_h"]
    a, b = (s["live"], s["live"] + c["branches"] - 1) if c["op"] == "fork" else (0, s["live"])
    return s["k"][:, :, :, a * t:b * t], s["v"][:, :, :, a * t:b * t]


def run(state):
    s = state
    if own:
        return _run_own(s)
    c = s["case"]
    h, d, op = c["heads"], c["head_dim"], c["op"]
    if op == "summarize_dense":
        return _means(s["k"], BLOCK)
    if op == "select_dense":
        forced = torch.arange(_blocks(c["n_k"]), device="cuda") < c["front"]
        return _select(s["q"], s["means"], c["keep"], forced)
    if op == "attend_dense":
        return _attend(s["q"], s["k"], s["v"], s["blocks"], c["n_k"], _blocks(c["n_k"]))
    t = c["frame_w"] * c["frame_h"]
    if op == "paged":
        outs = []
        for i, pages in enumerate(_branch_pages(c)):
            rows = (torch.tensor(pages, device="cuda")[:, None] * t + torch.arange(t, device="cuda")).flatten()
            q = s["q"][i * h * t:(i + 1) * h * t].view(h, t, d)
            bps = _blocks(t)
            every = torch.arange(len(pages) * bps, device="cuda").expand(h, -(-t // GROUP), -1)
            outs.append(_attend(q, s["k"][:, rows], s["v"][:, rows], every, t, bps))
        return torch.cat([o for o, _ in outs]), torch.cat([e for _, e in outs])
    if op in ("fork", "compact"):
        n = s["live"] * t
        for r in (s["k"], s["v"]):
            if op == "fork":
                src = FIRST + (c["chunk"] - 1) % c["ring"]
                for i in range(c["branches"] - 1):
                    r[:, :, :, n + i * t:n + (i + 1) * t] = r[:, :, :, src * t:(src + 1) * t]
            else:
                r[:, :, :, :n] = r[:, :, :, n:]
        return _moved(s)
    t, bps, streams = _geom(c)
    if op == "summarize_store":
        return [_means(s["k"][i][:, (FIRST + slot) * t:(FIRST + slot + 1) * t], BLOCK)
                for i, (_, _, slot) in enumerate(streams)]
    outs = []
    for i, (_, fill, slot) in enumerate(streams):
        q = s["q"][i * h * t:(i + 1) * h * t].view(h, t, d)
        if op == "select_store":
            m = s["means"][i][:, :(FIRST + fill) * bps]
            outs.append(_select(q, m, c["keep"], _forced(c, fill, slot, bps)).reshape(-1, c["keep"]))
        else:
            g = -(-t // GROUP)
            lists = s["blocks"][i * h * g:(i + 1) * h * g].view(h, g, -1)
            outs.append(_attend(q, s["k"][i], s["v"][i], lists, t, bps))
    if op == "select_store":
        return torch.cat(outs)
    return torch.cat([o for o, _ in outs]), torch.cat([e for _, e in outs])


# ------------------------------------------------------------------ work of one pass
def work(case):
    c = case
    h, d, op = c["heads"], c["head_dim"], c["op"]
    if op == "summarize_dense":
        return dict(bytes=h * d * (2 * c["n_k"] + 4 * _blocks(c["n_k"])), flops=h * d * c["n_k"])
    if op == "select_dense":
        g, nb = -(-c["n_q"] // GROUP), _blocks(c["n_k"])
        return dict(bytes=h * (2 * d * c["n_q"] + 4 * d * nb + 4 * g * c["keep"]),
                    flops=h * d * (c["n_q"] + 2 * g * nb))
    if op == "attend_dense":
        # keys: at the least the blocks of one group's list, at the most all of them
        nb, g = _blocks(c["n_k"]), -(-c["n_q"] // GROUP)
        n = min(c["keep"], nb)
        rows = min(c["n_k"], n * BLOCK)
        keys = min(c["n_k"], rows * (1 if g == 1 else min(g, 4)))
        return dict(bytes=h * d * (4 * c["n_q"] + 4 * keys) + 4 * h * (c["n_q"] + g * n),
                    flops=4 * h * d * c["n_q"] * rows)
    t = c["frame_w"] * c["frame_h"]
    bps, g = _blocks(t), -(-t // GROUP)
    if op == "paged":
        tables = _branch_pages(c)
        pages = len(set(p for x in tables for p in x))
        n = sum(len(x) for x in tables)
        return dict(bytes=4 * h * d * t * (len(tables) + pages) + 4 * h * t * len(tables),
                    flops=4 * h * d * t * t * n)
    if op in ("fork", "compact"):
        pages = c["branches"] - 1 if op == "fork" else FIRST + min(c["chunk"], c["ring"])
        read = 1 if op == "fork" else pages
        return dict(bytes=4 * h * d * t * c["layers"] * c["steps"] * (read + pages), flops=0)
    n = b = f = 0
    for _, fill, _ in _geom(c)[2]:
        nb = (FIRST + fill) * bps
        if op == "summarize_store":
            b += h * d * (2 * t + 4 * bps)
            f += h * d * t
        elif op == "select_store":
            b += h * (2 * d * t + 4 * d * nb + 4 * g * c["keep"])
            f += h * d * (t + 2 * g * nb)
        else:
            n = min(c["keep"], nb)
            rows = min((FIRST + fill) * t, n * BLOCK)
            keys = min((FIRST + fill) * t, rows * (1 if g == 1 else 2))
            b += h * d * (4 * t + 4 * keys) + 4 * h * (t + g * n)
            f += 4 * h * d * t * rows
    return dict(bytes=b, flops=f)


# ------------------------------------------------------------------ in 64 bits
def _exact_means(x, size):
    parts = [p.double().mean(1) for p in torch.split(x, size, dim=1)]
    return torch.stack(parts, 1)


def _exact_select(q, means, keep, forced):
    """By threshold: everything above the keep-th largest score, then the first ones equal to it."""
    qm = _exact_means(q, GROUP).float().double()
    s = (qm[:, :, None, :] * means.double()[:, None]).sum(-1)
    s[:, :, forced] = math.inf
    nb = s.shape[2]
    n = min(keep, nb)
    edge = s.topk(n, dim=2).values[:, :, -1:]
    above, equal = s > edge, s == edge
    chosen = above | (equal & (equal.cumsum(2) <= n - above.sum(2, keepdim=True)))
    out = torch.full((*s.shape[:2], keep), -1, dtype=torch.int32, device=q.device)
    out[:, :, :n] = chosen.nonzero()[:, 2].view(*s.shape[:2], n)
    return out


def _exact_attend(q, keys, values, lists):
    """lists(head, group): the key rows that the group reads.  f64 out [n][heads][dim], lse."""
    h, n, d = q.shape
    out = torch.empty(n, h, d, dtype=torch.float64, device=q.device)
    lse = torch.empty(n, h, dtype=torch.float64, device=q.device)
    for i in range(h):
        for g, part in enumerate(torch.split(q[i].double(), GROUP)):
            at = lists(i, g)
            s = part @ keys[i][at].double().T * d ** -0.5
            at_q = slice(g * GROUP, g * GROUP + part.shape[0])
            lse[at_q, i] = torch.logsumexp(s, 1)
            out[at_q, i] = torch.softmax(s, 1) @ values[i][at].double()
    return out, lse


def _listed_rows(blocks, seg, bps):
    """The key rows of one list, block by block on the host."""
    rows = []
    for b in blocks:
        if b >= 0:
            s, o = b // bps * seg, b % bps * BLOCK
            rows += range(s + o, s + min(seg, o + BLOCK))
    return torch.tensor(rows, device="cuda")


def exact(case, seed):
    c = dict(case)
    h, d, op = c["heads"], c["head_dim"], c["op"]
    if op in ("fork", "compact"):
        s = _prepare_pages(c, seed, False)
        t = c["frame_w"] * c["frame_h"]
        if op == "compact":
            return tuple(r[:, :, :, s["live"] * t:] for r in (s["k"], s["v"]))
        src = FIRST + (c["chunk"] - 1) % c["ring"]
        return tuple(r[:, :, :, src * t:(src + 1) * t].repeat(1, 1, 1, c["branches"] - 1, 1)
                     for r in (s["k"], s["v"]))
    x = _inputs(c, seed)
    if op == "summarize_dense":
        return _exact_means(x["k"], BLOCK)
    if op == "select_dense":
        forced = torch.arange(_blocks(c["n_k"]), device="cuda") < c["front"]
        return _exact_select(x["q"], _exact_means(x["k"], BLOCK).float(), c["keep"], forced)
    if op == "attend_dense":
        lists = _lists(c, x).tolist()
        return _exact_attend(x["q"], x["k"], x["v"],
                             lambda i, g: _listed_rows(lists[i][g], c["n_k"], _blocks(c["n_k"])))
    t = c["frame_w"] * c["frame_h"]
    if op == "paged":
        outs = []
        for i, pages in enumerate(_branch_pages(c)):
            rows = torch.cat([torch.arange(p * t, (p + 1) * t, device="cuda") for p in pages])
            q = x["q"][i * h * t:(i + 1) * h * t].view(h, t, d)
            outs.append(_exact_attend(q, x["k"], x["v"], lambda i, g, rows=rows: rows))
        return torch.cat([o for o, _ in outs]), torch.cat([e for _, e in outs])
    t, bps, streams = _geom(c)
    if op == "summarize_store":
        return [_exact_means(x["k"][i][:, (FIRST + slot) * t:(FIRST + slot + 1) * t], BLOCK)
                for i, (_, _, slot) in enumerate(streams)]
    outs = []
    if op == "attend_store":
        every = _lists(c, x).tolist()
        groups = -(-t // GROUP)
    for i, (_, fill, slot) in enumerate(streams):
        q = x["q"][i * h * t:(i + 1) * h * t].view(h, t, d)
        if op == "select_store":
            k = x["k"][i][:, :(FIRST + fill) * t].reshape(h * (FIRST + fill), t, d)
            m = _exact_means(k, BLOCK).float().reshape(h, -1, d)
            outs.append(_exact_select(q, m, c["keep"], _forced(c, fill, slot, bps)).reshape(-1, c["keep"]))
        else:
            mine = every[i * h * groups:(i + 1) * h * groups]
            outs.append(_exact_attend(q, x["k"][i], x["v"][i],
                                      lambda a, g, mine=mine: _listed_rows(mine[a * groups + g], t, bps)))
    if op == "select_store":
        return torch.cat(outs)
    return torch.cat([o for o, _ in outs]), torch.cat([e for _, e in outs])
