"""The paged store and the block calls of a store on the GPU: the same
schedule on fixed rows and on scattered, shared and moved pages gives the same
bits, which are held to the plain f64 forms (block_common) once."""
import pytest
import torch

from block_common import attend64, blocks_of, check_attention, means64, rows_of, select64
from same_step_kv_b200 import synth

pytestmark = pytest.mark.gpu
F0 = 3


@pytest.fixture(scope="module")
def pv():
    from same_step_kv_b200 import pv as m
    return m


class Run:
    """One stream's calls on a store; keeps nothing but the store."""

    def __init__(self, pv, store, stream, layers, steps):
        self.pv, self.store, self.h, self.stream = pv, store, store.handle, stream
        self.layers, self.steps = layers, steps

    def layer(self, tag, layer, step, n, keep=None):
        """Append, means, selection, attention over the list and over everything."""
        pv, c, h = self.pv, self.store.cfg, self.h
        q, k, v = synth.chunk_qkv(tag, step, layer, 7, n, c.heads, c.head_dim, "cuda")
        q_rot = torch.empty(c.heads, n, c.head_dim, dtype=torch.bfloat16, device="cuda")
        pv.pv_rope_append(h, [self.stream], layer, step, q, k, v, q_rot)
        pv.pv_block_summarize(h, [self.stream], layer, step)
        return self.read(q_rot, layer, step, keep)

    def read(self, q_rot, layer, step, keep=None):
        pv, c, h = self.pv, self.store.cfg, self.h
        n = q_rot.shape[1]
        out = torch.empty(2, n, c.heads, c.head_dim, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(2, n, c.heads, device="cuda")
        st = pv.pv_kv_get_state(h, self.stream)
        nb = st.n_keys // self.store.T * blocks_of(self.store.T)
        keep = keep or nb
        blocks = torch.empty(c.heads, -(-n // 256), keep, dtype=torch.int32, device="cuda")
        pv.pv_block_select(h, [self.stream], layer, step, q_rot, keep, 0, blocks)
        pv.pv_block_attn(h, [self.stream], layer, step, q_rot, blocks, keep, out[0], lse[0])
        pv.pv_chunk_attn(h, [self.stream], layer, step, q_rot, out[1], lse[1])
        return q_rot, blocks, out, lse

    def chunk(self, tag, keep=None):
        st = self.pv.pv_kv_get_state(self.h, self.stream)
        res = []
        for step in range(self.steps):
            for layer in range(self.layers):
                res.append(self.layer(tag, layer, step, st.n_queries, keep))
        return res

    def first(self, tag, keep=None):
        self.pv.pv_kv_begin_chunk(self.h, self.stream, F0)
        res = self.chunk(tag, keep)
        self.pv.pv_kv_begin_sink(self.h, self.stream)
        for layer in range(self.layers):
            res.append(self.layer(tag, layer, self.pv.PV_STEP_SINK, F0 * self.store.T, keep))
        return res

    def next(self, tag, keep=None):
        self.pv.pv_kv_begin_chunk(self.h, self.stream, 1)
        return self.chunk(tag, keep)


def stores(pv, W, Hh, H, D, R, pages, streams=3, layers=2, steps=2):
    cfg = pv.make_config(layers, H, D, W, Hh, ring_slots=R, steps=steps, max_streams=streams,
                         max_frames=64)
    return pv.KVStore(cfg, summaries=True), pv.KVStore(cfg, pages=pages, summaries=True)


def same(a, b, dense_bits=False):
    """Lists and block attention alike to the bit; chunk attention over contiguous rows and over
    pages differ in the rounding of P only."""
    for (qa, ba, oa, la), (qb, bb, ob, lb) in zip(a, b, strict=True):
        assert torch.equal(qa, qb) and torch.equal(ba, bb)
        assert torch.equal(oa[0], ob[0]) and torch.equal(la[0], lb[0])
        if dense_bits:
            assert torch.equal(oa[1], ob[1]) and torch.equal(la[1], lb[1])
        else:
            assert (oa[1].float() - ob[1].float()).abs().max() < 2e-2
            assert (la[1] - lb[1]).abs().max() < 2e-2


GEOMS = [dict(W=8, Hh=4, H=2, D=64, R=2), dict(W=12, Hh=11, H=3, D=128, R=3),
         dict(W=20, Hh=15, H=2, D=64, R=2), dict(W=1, Hh=1, H=1, D=128, R=1)]


@pytest.mark.parametrize("g", GEOMS, ids=str)
def test_scattered_pages_give_the_bits_of_fixed_rows(pv, g):
    fixed, paged = stores(pv, **g, pages=3 * (F0 + g["R"]))
    other = Run(pv, paged, 2, 2, 2)
    a, b = Run(pv, fixed, 0, 2, 2), Run(pv, paged, 0, 2, 2)
    other.first(90)
    ra, rb = a.first(5), b.first(5)
    same(ra, rb)
    for j in range(1, g["R"] + 3):
        other.next(90 + j)            # takes pages in between
        same(a.next(5 + j, keep=2), b.next(5 + j, keep=2))
        if j == 2:
            pv.pv_kv_release(paged.handle, 2)
            assert pv.pv_kv_compact(paged.handle) > 0
            other = Run(pv, paged, 1, 2, 2)
            other.first(80)
    assert pv.pv_kv_poll_device_error(paged.handle) == 0
    fixed.close(), paged.close()


@pytest.mark.parametrize("g", GEOMS, ids=str)
def test_store_calls_against_the_plain_forms(pv, g):
    fixed, _ = stores(pv, **g, pages=9)
    T, H, D, R = fixed.T, g["H"], g["D"], g["R"]
    bps = blocks_of(T)
    run = Run(pv, fixed, 1, 2, 2)
    run.first(3)
    for j in range(1, R + 2):
        res = run.next(3 + j, keep=bps + 1)
        st = pv.pv_kv_get_state(fixed.handle, 1)
        n = st.n_keys
        for i, (q_rot, blocks, out, lse) in enumerate(res):
            step, layer = divmod(i, 2)
            k, v = (r[layer, step, 1, :, :n] for r in (fixed.k_region(), fixed.v_region()))
            m = means64(k.reshape(H * n // T, T, D), 128).float().reshape(H, -1, D)
            assert torch.equal(fixed.summary_region()[layer, step, 1, :, :m.shape[1]], m)
            assert torch.equal(blocks.cpu(), select64(q_rot, m, bps + 1))
            t = blocks.tolist()
            check_attention(out[0], lse[0], attend64(q_rot, k, v, lambda h, a: rows_of(
                t[h][a], T, m.shape[1])))
    fixed.close()


def test_forced_blocks(pv):
    W, Hh, H, D, R = 20, 15, 2, 64, 3          # 3 blocks a frame
    fixed, paged = stores(pv, W, Hh, H, D, R, pages=9)
    T, bps = W * Hh, 3
    want = {}
    for store in (fixed, paged):
        run = Run(pv, store, 0, 1, 1)
        run.first(1)
        for j in range(5):
            q_rot = run.next(2 + j)[-1][0]
        st = pv.pv_kv_get_state(store.handle, 0)
        assert (st.fill, st.slot) == (3, 1)
        sink, cur = set(range(9)), set(range(4 * bps, 5 * bps))
        for force, must in ((1, sink), (2, cur), (3, sink | cur)):
            keep = len(must) + 2
            blocks = torch.empty(H, 2, keep, dtype=torch.int32, device="cuda")
            pv.pv_block_select(store.handle, [0], 0, 0, q_rot, keep, force, blocks)
            if store is fixed:
                k = fixed.k_region()[0, 0, 0, :, :6 * T]
                m = means64(k.reshape(H * 6, T, D), 128).float().reshape(H, -1, D)
                want[force] = select64(q_rot, m, keep, sorted(must))
            assert torch.equal(blocks.cpu(), want[force])
            assert all(must <= set(r) for r in blocks.flatten(0, 1).tolist())
            with pytest.raises(pv.PVError) as e:
                pv.pv_block_select(store.handle, [0], 0, 0, q_rot, len(must) - 1, force, blocks)
            assert e.value.status == pv.PV_ERR_SHAPE
        with pytest.raises(pv.PVError) as e:
            pv.pv_block_select(store.handle, [0], 0, 0, q_rot, 20, 4, blocks)
        assert e.value.status == pv.PV_ERR_INVALID_ARG
        store.close()


@pytest.mark.parametrize("g", GEOMS[:3], ids=str)
@pytest.mark.parametrize("when", ["first", "sink", "steady", "full"])
def test_branches_are_streams_of_their_own(pv, g, when):
    """A branch taken in mid-chunk (its page copied) or after a chunk (everything shared) goes on as
    a stream that ran the whole history itself."""
    fixed, paged = stores(pv, **g, pages=3 * (F0 + g["R"]))
    a = [Run(pv, fixed, i, 2, 2) for i in range(3)]
    b = [Run(pv, paged, i, 2, 2) for i in range(3)]
    chunks = {"first": 0, "sink": 0, "steady": 1, "full": g["R"] + 1}[when]
    # fixed rows: three streams with the same history
    for r in a + b[:1]:
        if when == "first":
            pv.pv_kv_begin_chunk(r.h, r.stream, F0)
            r.layer(40, 0, 0, F0 * r.store.T)
            continue
        r.first(40)
        for j in range(chunks):
            r.next(41 + j)
    pv.pv_kv_fork(paged.handle, 0, [2, 1], 1)
    # every one of them writes its current chunk again, with its own data
    for i in (1, 0, 2):
        if when == "sink":
            n = F0 * fixed.T
            same([a[i].layer(50 + i, 0, pv.PV_STEP_SINK, n)], [b[i].layer(50 + i, 0, pv.PV_STEP_SINK, n)])
        else:
            same(a[i].chunk(50 + i), b[i].chunk(50 + i))
    if when == "first":
        for r in a + b:
            pv.pv_kv_begin_sink(r.h, r.stream)
            r.layer(60 + r.stream, 0, pv.PV_STEP_SINK, F0 * r.store.T)
            r.layer(70 + r.stream, 1, pv.PV_STEP_SINK, F0 * r.store.T)
    for j in range(3):
        for i in (2, 0, 1):
            same(a[i].next(100 + 10 * i + j, keep=2), b[i].next(100 + 10 * i + j, keep=2))
        pv.pv_kv_compact(paged.handle)
    fixed.close(), paged.close()


def test_shared_history_and_the_page_that_may_not_be_written(pv):
    fixed, paged = stores(pv, 12, 11, 2, 64, 2, pages=9)
    a, b = Run(pv, fixed, 0, 2, 2), Run(pv, paged, 0, 2, 2)
    a.first(1), b.first(1)
    a.next(2), b.next(2)
    pv.pv_kv_fork(paged.handle, 0, [1], 0)
    k0 = paged.k_region().clone()
    q = torch.zeros(132, 2, 64, dtype=torch.bfloat16, device="cuda")
    for stream in (0, 1):
        for call in (lambda: pv.pv_rope_append(paged.handle, [stream], 0, 0, q, q, q, torch.empty_like(q)),
                     lambda: pv.pv_block_summarize(paged.handle, [stream], 0, 0)):
            with pytest.raises(pv.PVError) as e:
                call()
            assert e.value.status == pv.PV_ERR_STATE
    assert torch.equal(paged.k_region(), k0)
    # both read the shared page; each goes on by itself
    c = Run(pv, paged, 1, 2, 2)
    pv.pv_kv_fork(fixed.handle, 0, [1], 0)
    d = Run(pv, fixed, 1, 2, 2)
    same(d.next(30), c.next(30))
    same(a.next(31), b.next(31))
    pv.pv_kv_release(paged.handle, 0)
    pv.pv_kv_compact(paged.handle)
    same(d.next(32), c.next(32))
    fixed.close(), paged.close()


@pytest.mark.parametrize("D,T", [(64, 1), (128, 5), (64, 333)])
def test_compaction_moves_every_plane_and_nothing_else(pv, D, T):
    L, S, H, R, n = 3, 2, 5, 4, 30
    cfg = pv.make_config(L, H, D, T, 1, ring_slots=R, steps=S, max_streams=8, max_frames=64)
    store = pv.KVStore(cfg, pages=n, summaries=True)
    h = store.handle
    st = pv.pv_kv_state()
    st.phase, st.chunk = pv.PV_PHASE_STEADY, 2
    for i in range(6):
        pv.pv_kv_set_state(h, i, st)          # five pages each
    for r in (store.k_region(), store.v_region(), store.summary_region()):
        r.copy_(torch.randn(r.shape, device="cuda"))
    for i in (0, 3, 5):
        pv.pv_kv_release(h, i)
    pv.pv_kv_fork(h, 1, [0, 3], 1)            # copies at pages 0 and 1, the rest shared
    kv = [r.clone() for r in (store.k_region(), store.v_region(), store.summary_region())]
    before = {i: pv.pv_kv_page_table(h, i) for i in range(6)}
    moved = pv.pv_kv_compact(h)
    after = {i: pv.pv_kv_page_table(h, i) for i in range(6)}
    flat = lambda t: [t[0] + i for i in range(F0)] + t[1][:2] if t[0] >= 0 else []  # noqa: E731
    held = sorted(set(p for t in before.values() for p in flat(t)))
    to = {p: i for i, p in enumerate(held)}
    assert moved == sum(to[p] != p for p in held)
    for i in before:
        assert flat(after[i]) == [to[p] for p in flat(before[i])]
    for was, now in zip(kv, (store.k_region(), store.v_region(), store.summary_region())):
        rows = was.shape[3] // n
        want = was.clone()
        for p in held:
            want[:, :, :, to[p] * rows:(to[p] + 1) * rows] = was[:, :, :, p * rows:(p + 1) * rows]
        assert torch.equal(want, now)
    assert pv.pv_kv_free_pages(h) == (n - len(held), n - len(held))
    store.close()


def test_fork_of_fixed_rows_copies_the_history(pv):
    fixed, _ = stores(pv, 12, 11, 2, 64, 3, pages=3)
    a = Run(pv, fixed, 1, 2, 2)
    a.first(1)
    a.next(2)
    before = [r.clone() for r in (fixed.k_region(), fixed.v_region(), fixed.summary_region())]
    pv.pv_kv_fork(fixed.handle, 1, [0], 0)
    for was, now in zip(before, (fixed.k_region(), fixed.v_region(), fixed.summary_region())):
        rows = was.shape[4] // 6 * 4          # sink and one slot of the ring of three
        want = was.clone()
        want[:, :, 0, :, :rows] = was[:, :, 1, :, :rows]
        assert torch.equal(want, now)
    fixed.close()


def test_many_streams_in_one_call(pv):
    """64 streams, each with a page table of its own, fills from 1 to 5, against one call each."""
    H, D, R, S = 2, 64, 5, 64
    cfg = pv.make_config(1, H, D, 10, 13, ring_slots=R, steps=1, max_streams=S, max_frames=64)
    store = pv.KVStore(cfg, pages=S * (F0 + R), summaries=True)
    h, T = store.handle, 130
    st = pv.pv_kv_state()
    st.phase = pv.PV_PHASE_STEADY
    for i in range(S):
        st.chunk = 1 + i % 9
        pv.pv_kv_set_state(h, i, st)
    for r in (store.k_region(), store.v_region()):
        r.copy_(torch.randn(r.shape, device="cuda"))
    store.summary_region().copy_(torch.randn(store.summary_region().shape, device="cuda"))
    ids = list(range(S))[::-1]
    q = torch.randn(S, H, T, D, device="cuda").to(torch.bfloat16)
    new = lambda n: (torch.empty(n * T, H, D, dtype=torch.bfloat16, device="cuda"),  # noqa: E731
                     torch.empty(n * T, H, device="cuda"),
                     torch.empty(n, H, 1, 7, dtype=torch.int32, device="cuda"))
    out, lse, blocks = new(S)
    pv.pv_block_summarize(h, ids, 0, 0)
    pv.pv_block_select(h, ids, 0, 0, q, 7, 2, blocks)
    pv.pv_block_attn(h, ids, 0, 0, q, blocks, 7, out, lse)
    full = torch.empty_like(out)
    pv.pv_chunk_attn(h, ids, 0, 0, q, full)
    for a, i in enumerate(ids):
        o, e, b = new(1)
        pv.pv_block_select(h, [i], 0, 0, q[a], 7, 2, b)
        assert torch.equal(b[0], blocks[a]), i
        pv.pv_block_attn(h, [i], 0, 0, q[a], b, 7, o, e)
        # another plan splits the keys elsewhere: equal up to the roundings
        assert (o.float() - out[a * T:(a + 1) * T].float()).abs().max() < 2e-2
        assert (e - lse[a * T:(a + 1) * T]).abs().max() < 1e-4
        pv.pv_chunk_attn(h, [i], 0, 0, q[a], o)
        assert (o.float() - full[a * T:(a + 1) * T].float()).abs().max() < 2e-2
    store.close()


@pytest.mark.parametrize("D,heads", [(128, 2), (64, 5)])
def test_projection_appends_to_pages(pv, D, heads):
    """pv_qkv_rope_append on scattered pages writes what it writes to fixed rows."""
    W, Hh, R, T = 12, 11, 2, 132
    fixed, paged = stores(pv, W, Hh, heads, D, R, pages=12, layers=1)
    pv.pv_kv_begin_chunk(paged.handle, 1, F0)       # pages 0 .. 2
    dim = heads * D
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    w, bias = (rnd(3 * dim, dim) / dim ** 0.5).bfloat16(), rnd(3 * dim)
    gq, gk = rnd(dim), rnd(dim)
    for h in (fixed.handle, paged.handle):
        pv.pv_kv_begin_chunk(h, 0, F0)
    for chunk in range(4):
        n = F0 * T if chunk == 0 else T
        ws = torch.empty(pv.pv_qkv_ws_bytes(n, dim), dtype=torch.uint8, device="cuda")
        for step in (0, 1, pv.PV_STEP_SINK) if chunk == 0 else (0, 1):
            if step == pv.PV_STEP_SINK:
                for h in (fixed.handle, paged.handle):
                    pv.pv_kv_begin_sink(h, 0)
            x = rnd(n, dim).bfloat16()
            q = [torch.empty(heads, n, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            for h, o in zip((fixed.handle, paged.handle), q):
                pv.pv_qkv_rope_append(h, [0], 0, step, x, w, bias, gq, gk, 1e-6, o, ws, ws.numel())
            assert torch.equal(*q)
        sink, ring = pv.pv_kv_page_table(paged.handle, 0)
        pages = list(range(sink, sink + F0)) + [p for p in ring if p >= 0]
        for a, b in ((fixed.k_region(), paged.k_region()), (fixed.v_region(), paged.v_region())):
            for seg, page in enumerate(pages):
                assert torch.equal(a[0, :, 0, :, seg * T:(seg + 1) * T], b[0, :, :, page * T:(page + 1) * T])
        for h in (fixed.handle, paged.handle):
            pv.pv_kv_begin_chunk(h, 0, 1)
        if chunk == 1:
            pv.pv_kv_begin_sink(paged.handle, 1)
            pv.pv_kv_begin_chunk(paged.handle, 1, 1)    # a page between the stream's own
    assert pv.pv_kv_poll_device_error(paged.handle) == 0
    fixed.close(), paged.close()


def test_a_store_beyond_32_bit_offsets(pv):
    """100 pages of 880 x 24 x 128 in 16 planes: 4.3e9 values of K and of V; the last plane is used."""
    H, D, R, L, S, T, n = 24, 128, 18, 4, 4, 880, 100
    cfg = pv.make_config(L, H, D, 40, 22, ring_slots=R, steps=S, max_streams=4)
    store = pv.KVStore(cfg, pages=n, summaries=True)
    h = store.handle
    st = pv.pv_kv_state()
    st.phase, st.chunk = pv.PV_PHASE_STEADY, 18
    for i in range(4):
        pv.pv_kv_set_state(h, i, st)          # 21 pages each: stream 3 in 63 .. 83
    K, V = store.k_region()[3, 3], store.v_region()[3, 3]
    K.copy_(torch.randn(K.shape, device="cuda")), V.copy_(torch.randn(V.shape, device="cuda"))
    k, v = K[:, 63 * T:84 * T].clone(), V[:, 63 * T:84 * T].clone()
    q = torch.randn(H, T, D, device="cuda").bfloat16()
    out, lse = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda"), torch.empty(T, H, device="cuda")
    lists = torch.randint(0, 147, (H, 4, 5), dtype=torch.int32, device="cuda")
    t = lists.tolist()
    ref = attend64(q, k, v, lambda a, g: rows_of(t[a][g], T, 147))
    pv.pv_block_attn(h, [3], 3, 3, q, lists, 5, out, lse)
    check_attention(out, lse, ref)
    pv.pv_block_summarize(h, [3], 3, 3)
    assert torch.equal(store.summary_region()[3, 3][:, 83 * 7:84 * 7],
                       means64(k[:, 20 * T:], 128).float())
    # the page in hand copied beyond the others, then everything moved down
    pv.pv_kv_release(h, 0)
    pv.pv_kv_fork(h, 3, [0], 1)               # page 0
    assert torch.equal(K[:, :T], k[:, 20 * T:])
    assert pv.pv_kv_compact(h) == 63
    assert pv.pv_kv_page_table(h, 3)[0] == 43
    assert torch.equal(K[:, 43 * T:64 * T], k) and torch.equal(V[:, 43 * T:64 * T], v)
    for i in (3, 0):
        out.zero_()
        pv.pv_block_attn(h, [i], 3, 3, q, lists, 5, out, lse)
        check_attention(out, lse, ref)
    store.close()


@pytest.mark.parametrize("paged", [False, True])
def test_streams_in_different_phases_in_one_call(pv, paged):
    """A first chunk (3 frames of queries) and two steady ones at different fills: one call against one each."""
    H, D, R, W, Hh = 3, 128, 4, 17, 13
    T = W * Hh
    cfg = pv.make_config(1, H, D, W, Hh, ring_slots=R, steps=2, max_streams=4, max_frames=64)
    store = pv.KVStore(cfg, pages=24 if paged else None, summaries=True)
    h = store.handle
    st = pv.pv_kv_state()
    for i, (phase, chunk) in enumerate([(pv.PV_PHASE_STEADY, 2), (pv.PV_PHASE_FIRST, 0),
                                        (pv.PV_PHASE_STEADY, 9)]):
        st.phase, st.chunk = phase, chunk
        pv.pv_kv_set_state(h, i, st)
    for r in (store.k_region(), store.v_region()):
        r.copy_(torch.randn(r.shape, device="cuda"))
    ids, n = [2, 1, 0], [T, F0 * T, T]
    fill = {0: 2, 1: 0, 2: 4}
    for i in range(3):          # means of every frame: the current chunk's by the call, others plain
        bps = blocks_of(T)
        k, m = store.k_region(), store.summary_region()
        if paged:
            sink, ring = pv.pv_kv_page_table(h, i)
            pages = list(range(sink, sink + F0)) + ring[:fill[i]]
            for p in pages:
                m[0, 1, :, p * bps:(p + 1) * bps] = means64(k[0, 1, :, p * T:(p + 1) * T], 128).float()
        else:
            for s in range(F0 + R):
                m[0, 1, i, :, s * bps:(s + 1) * bps] = means64(k[0, 1, i, :, s * T:(s + 1) * T], 128).float()
    before = store.summary_region().clone()
    pv.pv_block_summarize(h, ids, 0, 1)
    assert torch.equal(before, store.summary_region())
    tok = sum(n)
    q = torch.randn(H * tok, D, device="cuda").bfloat16()
    keep = 9
    rows = [H * -(-x // 256) for x in n]
    blocks = torch.empty(sum(rows), keep, dtype=torch.int32, device="cuda")
    out = torch.empty(tok, H, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(tok, H, device="cuda")
    pv.pv_block_select(h, ids, 0, 1, q, keep, pv.PV_FORCE_CURRENT, blocks)
    pv.pv_block_attn(h, ids, 0, 1, q, blocks, keep, out, lse)
    t0 = r0 = 0
    for i, x, r in zip(ids, n, rows):
        nb = (F0 + fill[i]) * blocks_of(T)
        one = torch.empty(r, keep, dtype=torch.int32, device="cuda")
        qi = q[H * t0:H * (t0 + x)].view(H, x, D)
        pv.pv_block_select(h, [i], 0, 1, qi, keep, pv.PV_FORCE_CURRENT, one)
        assert torch.equal(one, blocks[r0:r0 + r])
        if paged:
            sink, ring = pv.pv_kv_page_table(h, i)
            at = torch.cat([torch.arange(p * T, (p + 1) * T) for p in
                            list(range(sink, sink + F0)) + ring[:fill[i]]]).cuda()
            k, v = store.k_region()[0, 1][:, at], store.v_region()[0, 1][:, at]
        else:
            k, v = store.k_region()[0, 1, i], store.v_region()[0, 1, i]
        lists = one.view(H, -1, keep).tolist()
        check_attention(out[t0:t0 + x], lse[t0:t0 + x],
                        attend64(qi, k, v, lambda a, g: rows_of(lists[a][g], T, nb)), f"stream {i}")
        t0, r0 = t0 + x, r0 + r
    store.close()


def test_missing_means_and_other_refusals(pv):
    cfg = pv.make_config(1, 2, 64, 8, 4, ring_slots=2, steps=1, max_streams=2, max_frames=64)
    store = pv.KVStore(cfg, pages=8)
    h = store.handle
    pv.pv_kv_begin_chunk(h, 0, F0)
    t = torch.zeros(F0 * 32, 2, 64, dtype=torch.bfloat16, device="cuda")
    blocks = torch.zeros(2, 1, 3, dtype=torch.int32, device="cuda")

    def refused(status, call):
        with pytest.raises(pv.PVError) as e:
            call()
        assert e.value.status == status

    refused(pv.PV_ERR_STATE, lambda: pv.pv_block_summarize(h, [0], 0, 0))
    refused(pv.PV_ERR_STATE, lambda: pv.pv_block_select(h, [0], 0, 0, t, 3, 0, blocks))
    n = pv.pv_kv_summary_bytes(h)
    buf = torch.empty(n + 256, dtype=torch.uint8, device="cuda")
    refused(pv.PV_ERR_CAPACITY, lambda: pv.pv_kv_set_summaries(h, buf, n - 1))
    refused(pv.PV_ERR_INVALID_ARG, lambda: pv.pv_kv_set_summaries(h, buf.data_ptr() + 16, n))
    pv.pv_kv_set_summaries(h, buf, n)
    assert (buf[:n] == 0).all()
    for kw in (dict(layer=1), dict(layer=-1), dict(step=1), dict(step=-2), dict(streams=[2]),
               dict(streams=[0, 0]), dict(streams=[])):
        a = dict(streams=[0], layer=0, step=0) | kw
        for call in (lambda: pv.pv_block_summarize(h, a["streams"], a["layer"], a["step"]),
                     lambda: pv.pv_block_select(h, a["streams"], a["layer"], a["step"], t, 3, 0, blocks),
                     lambda: pv.pv_block_attn(h, a["streams"], a["layer"], a["step"], t, blocks, 3, t)):
            refused(pv.PV_ERR_INVALID_ARG, call)
    refused(pv.PV_ERR_STATE, lambda: pv.pv_block_select(h, [0], 0, -1, t, 3, 0, blocks))
    refused(pv.PV_ERR_STATE, lambda: pv.pv_block_attn(h, [1], 0, 0, t, blocks, 3, t))
    refused(pv.PV_ERR_SHAPE, lambda: pv.pv_block_select(h, [0], 0, 0, t, 0, 0, blocks))
    refused(pv.PV_ERR_SHAPE, lambda: pv.pv_block_attn(h, [0], 0, 0, t, blocks, 0, t))
    refused(pv.PV_ERR_INVALID_ARG, lambda: pv.pv_block_attn(h, [0], 0, 0, t, None, 3, t))
    refused(pv.PV_ERR_INVALID_ARG, lambda: pv.pv_block_attn(h, [0], 0, 0, t.data_ptr() + 2, blocks, 3, t))
    pv.pv_kv_set_summaries(h, None)
    refused(pv.PV_ERR_STATE, lambda: pv.pv_block_summarize(h, [0], 0, 0))
    store.close()
