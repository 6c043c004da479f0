"""Page bookkeeping of the paged store on the host (bookkeeping-only handles,
no device): page tables after begin / fork / release / compact / set_state
against a plain model, capacity failures that change nothing, and the argument
checks of the page and block calls."""
import random

import pytest

from same_step_kv_b200 import pv

F0 = 3


def cfg_of(R=3, streams=4, D=64, W=8, Hh=4, max_frames=64, first=F0):
    return pv.make_config(2, 2, D, W, Hh, first_frames=first, ring_slots=R, max_streams=streams,
                          max_frames=max_frames)


class Model:
    """Who holds which page, straight from the documented rules."""

    def __init__(self, n_pages, R, streams):
        self.n, self.R = n_pages, R
        self.st = [self.new() for _ in range(streams)]

    def new(self):
        return dict(phase="NEW", chunk=-1, sink=-1, ring=[-1] * self.R)

    def held(self):
        count = [0] * self.n
        for s in self.st:
            if s["sink"] >= 0:
                for i in range(F0):
                    count[s["sink"] + i] += 1
            for p in s["ring"]:
                if p >= 0:
                    count[p] += 1
        return count

    def find(self, n, held=None):
        held = held or self.held()
        for i in range(self.n - n + 1):
            if not any(held[i:i + n]):
                return i
        return -1

    def begin(self, i):
        s = self.st[i]
        if s["phase"] == "NEW":
            p = self.find(F0)
            if p < 0:
                return False
            s.update(phase="FIRST", chunk=0, sink=p)
            return True
        slot = s["chunk"] % self.R
        held = self.held()
        if s["ring"][slot] < 0 or held[s["ring"][slot]] > 1:
            p = self.find(1, held)
            if p < 0:
                return False
            s["ring"][slot] = p
        s.update(phase="STEADY", chunk=s["chunk"] + 1)
        return True

    def fork(self, src, dst, copy):
        s = self.st[src]
        steady = s["phase"] == "STEADY"
        fresh, held = [], self.held()
        for _ in dst if copy else []:
            p = self.find(1 if steady else F0, held)
            if p < 0:
                return False
            for k in range(1 if steady else F0):
                held[p + k] = 1
            fresh.append(p)
        for k, d in enumerate(dst):
            self.st[d] = dict(s, ring=list(s["ring"]))
            if copy and steady:
                self.st[d]["ring"][(s["chunk"] - 1) % self.R] = fresh[k]
            elif copy:
                self.st[d]["sink"] = fresh[k]
        return True

    def compact(self):
        held = self.held()
        to, n, moved = {}, 0, 0
        for i, c in enumerate(held):
            if c:
                to[i] = n
                moved += n != i
                n += 1
        for s in self.st:
            s["sink"] = to.get(s["sink"], -1)
            s["ring"] = [to.get(p, -1) for p in s["ring"]]
        return moved


def check(h, m):
    for i, s in enumerate(m.st):
        sink, pages = pv.pv_kv_page_table(h, i)
        assert (sink, pages[:m.R]) == (s["sink"], s["ring"]), i
        assert all(p == -1 for p in pages[m.R:])
        assert pv.pv_kv_get_state(h, i).chunk == s["chunk"]
    held = m.held()
    run = best = 0
    for c in held:
        run = run + 1 if c == 0 else 0
        best = max(best, run)
    assert pv.pv_kv_free_pages(h) == (held.count(0), best)


@pytest.mark.parametrize("seed", range(8))
def test_random_schedules_against_the_model(seed):
    rng = random.Random(seed)
    R, streams = rng.randint(1, 5), rng.randint(2, 6)
    n = rng.randint(F0 + 1, streams * (F0 + R))
    h = pv.pv_kv_init_paged(cfg_of(R, streams, max_frames=1000), n)
    m = Model(n, R, streams)
    refused = 0
    for _ in range(400):
        i = rng.randrange(streams)
        s = m.st[i]
        op = rng.random()
        try:
            if op < 0.6:
                if s["phase"] == "FIRST":
                    pv.pv_kv_begin_sink(h, i)
                    s["phase"] = "BOOT"
                else:
                    ok = m.begin(i)
                    pv.pv_kv_begin_chunk(h, i, F0 if pv.pv_kv_get_state(h, i).chunk < 0 else 1)
                    assert ok
            elif op < 0.8:
                free = [j for j in range(streams) if m.st[j]["phase"] == "NEW"]
                if s["phase"] != "NEW" and free:
                    dst = rng.sample(free, rng.randint(1, len(free)))
                    copy = rng.random() < 0.5
                    ok = m.fork(i, dst, copy)
                    pv.pv_kv_fork(h, i, dst, copy)
                    assert ok
            elif op < 0.92:
                pv.pv_kv_release(h, i)
                m.st[i] = m.new()
            else:
                assert pv.pv_kv_compact(h) == m.compact()
        except pv.PVError as e:
            assert e.status == pv.PV_ERR_CAPACITY and not ok
            refused += 1
        check(h, m)
    assert refused or n >= streams * (F0 + R) - 2
    pv.pv_kv_destroy(h)


def grow(h, stream, chunk):
    pv.pv_kv_begin_chunk(h, stream, F0)
    if chunk:
        pv.pv_kv_begin_sink(h, stream)
    for _ in range(chunk):
        pv.pv_kv_begin_chunk(h, stream, 1)


def test_full_ring_writes_its_own_page_again_and_leaves_a_shared_one():
    h = pv.pv_kv_init_paged(cfg_of(2), 8)
    grow(h, 0, 2)
    assert pv.pv_kv_page_table(h, 0)[1][:2] == [3, 4]
    pv.pv_kv_begin_chunk(h, 0, 1)
    assert pv.pv_kv_page_table(h, 0)[1][:2] == [3, 4]
    pv.pv_kv_fork(h, 0, [1], 0)
    pv.pv_kv_begin_chunk(h, 0, 1)           # slot 1's page is shared: a fresh one
    assert pv.pv_kv_page_table(h, 0)[1][:2] == [3, 5]
    pv.pv_kv_begin_chunk(h, 1, 1)           # the last holder keeps it
    assert pv.pv_kv_page_table(h, 1)[1][:2] == [3, 4]
    pv.pv_kv_destroy(h)


def test_fragmented_store_takes_a_first_chunk_after_compaction():
    h = pv.pv_kv_init_paged(cfg_of(2, streams=4), 9)
    grow(h, 0, 1)          # pages 0-2, 3
    grow(h, 1, 2)          # pages 4-6, 7, 8
    pv.pv_kv_release(h, 0)
    pv.pv_kv_begin_chunk(h, 0, F0)          # 0-2 again
    pv.pv_kv_release(h, 1)
    pv.pv_kv_begin_sink(h, 0)
    for _ in range(2):
        pv.pv_kv_begin_chunk(h, 0, 1)       # 3, 4
    pv.pv_kv_fork(h, 0, [1], 1)             # 5
    pv.pv_kv_begin_chunk(h, 0, 1)           # slot 0 shared: 6
    pv.pv_kv_release(h, 0)                  # holes at 4 and 6 .. 8: the fork holds 0-3, 5
    assert pv.pv_kv_free_pages(h) == (4, 3)
    pv.pv_kv_begin_chunk(h, 2, F0)
    pv.pv_kv_release(h, 1)
    assert pv.pv_kv_page_table(h, 2)[0] == 6
    assert pv.pv_kv_compact(h) == 3
    assert pv.pv_kv_page_table(h, 2)[0] == 0
    assert pv.pv_kv_free_pages(h) == (6, 6)
    pv.pv_kv_destroy(h)


def test_set_state_keeps_takes_and_gives_back_pages():
    h = pv.pv_kv_init_paged(cfg_of(3), 8)
    grow(h, 0, 2)
    before = pv.pv_kv_page_table(h, 0)
    pv.pv_kv_set_state(h, 0, pv.pv_kv_get_state(h, 0))
    assert pv.pv_kv_page_table(h, 0) == before
    st = pv.pv_kv_get_state(h, 0)
    st.chunk = 7
    pv.pv_kv_set_state(h, 0, st)
    assert pv.pv_kv_page_table(h, 0)[1][:3] == [3, 4, 5]
    with pytest.raises(pv.PVError) as e:    # 2 pages left, 6 wanted: nothing changes
        pv.pv_kv_set_state(h, 1, st)
    assert e.value.status == pv.PV_ERR_CAPACITY
    assert pv.pv_kv_free_pages(h) == (2, 2)
    assert pv.pv_kv_page_table(h, 1) == (-1, [-1] * pv.PV_MAX_RING)
    st.phase, st.chunk = pv.PV_PHASE_FIRST, 0
    pv.pv_kv_set_state(h, 0, st)
    assert pv.pv_kv_page_table(h, 0) == (0, [-1] * pv.PV_MAX_RING)
    st.phase, st.chunk = pv.PV_PHASE_NEW, -1
    pv.pv_kv_set_state(h, 0, st)
    assert pv.pv_kv_free_pages(h) == (8, 8)
    pv.pv_kv_destroy(h)


def test_row_offsets_follow_the_page_table():
    c = cfg_of(2)
    h = pv.pv_kv_init_paged(c, 9)
    T, D = 32, 64
    grow(h, 1, 0)          # takes 0-2
    grow(h, 0, 2)          # 3-5, 6, 7
    pv.pv_kv_release(h, 1)
    pv.pv_kv_compact(h)    # 0-2, 3, 4
    region = 2 * 4 * 2 * 9 * T
    k, v = pv.pv_kv_row_offset(h, 1, 2, 0, 1, 4 * T + 5)   # ring slot 1, token 5
    row = ((1 * 4 + 2) * 2 + 1) * 9 * T + 4 * T + 5
    assert (k, v) == (row * D, (region + row) * D)
    with pytest.raises(pv.PVError) as e:
        pv.pv_kv_row_offset(h, 0, 0, 1, 0, 0)
    assert e.value.status == pv.PV_ERR_STATE
    with pytest.raises(pv.PVError) as e:
        pv.pv_kv_row_offset(h, 0, 0, 0, 0, 5 * T)
    assert e.value.status == pv.PV_ERR_INVALID_ARG
    pv.pv_kv_destroy(h)


def test_paged_sizes():
    c = pv.make_config(30, 24, 128, 40, 22, ring_slots=18, max_streams=16)
    kv, ws = pv.pv_kv_paged_required_bytes(c, 40)
    assert kv == 2 * 30 * 4 * 24 * 40 * 880 * 128 * 2
    assert ws == pv.pv_kv_required_bytes(pv.make_config(30, 24, 128, 40, 22, ring_slots=18,
                                                        max_streams=16))[1]
    for n in (0, -1, 2, 1 << 30):
        with pytest.raises(pv.PVError) as e:
            pv.pv_kv_paged_required_bytes(c, n)
        assert e.value.status == pv.PV_ERR_SHAPE
    # 16 streams of fixed rows would pass 2^31 rows; 800 pages do not
    big = pv.make_config(30, 24, 128, 40, 22, ring_slots=64, max_streams=64)
    with pytest.raises(pv.PVError):
        pv.pv_kv_required_bytes(big)
    pv.pv_kv_paged_required_bytes(big, 800)


def test_fork_release_and_compact_of_fixed_rows():
    h = pv.pv_kv_init(cfg_of(3))
    grow(h, 0, 4)
    pv.pv_kv_fork(h, 0, [2, 1], 1)
    a, b = pv.pv_kv_get_state(h, 0), pv.pv_kv_get_state(h, 2)
    assert (a.chunk, a.slot, list(a.slot_frame)) == (b.chunk, b.slot, list(b.slot_frame))
    assert pv.pv_kv_compact(h) == 0 and pv.pv_kv_free_pages(h) == (0, 0)
    pv.pv_kv_release(h, 2)
    assert pv.pv_kv_get_state(h, 2).phase == pv.PV_PHASE_NEW
    with pytest.raises(pv.PVError) as e:
        pv.pv_kv_page_table(h, 0)
    assert e.value.status == pv.PV_ERR_STATE
    pv.pv_kv_destroy(h)


@pytest.mark.parametrize("paged", [False, True])
def test_fork_refusals_change_nothing(paged):
    h = pv.pv_kv_init_paged(cfg_of(3), 12) if paged else pv.pv_kv_init(cfg_of(3))
    grow(h, 0, 1)
    grow(h, 3, 0)
    for src, dst, status in [(1, [2], pv.PV_ERR_STATE), (0, [0], pv.PV_ERR_STATE),
                             (0, [1, 3], pv.PV_ERR_STATE), (0, [1, 1], pv.PV_ERR_INVALID_ARG),
                             (0, [4], pv.PV_ERR_INVALID_ARG), (0, [], pv.PV_ERR_INVALID_ARG),
                             (4, [1], pv.PV_ERR_INVALID_ARG), (-1, [1], pv.PV_ERR_INVALID_ARG)]:
        with pytest.raises(pv.PVError) as e:
            pv.pv_kv_fork(h, src, dst, 1)
        assert e.value.status == status, (src, dst)
        assert pv.pv_kv_get_state(h, 1).phase == pv.PV_PHASE_NEW
    for bad in (-1, 4):
        with pytest.raises(pv.PVError):
            pv.pv_kv_release(h, bad)
    pv.pv_kv_destroy(h)


def test_null_handles_and_outputs():
    for call in (lambda: pv.pv_kv_fork(None, 0, [1], 0), lambda: pv.pv_kv_release(None, 0),
                 lambda: pv.pv_kv_compact(None), lambda: pv.pv_kv_page_table(None, 0),
                 lambda: pv.pv_kv_free_pages(None), lambda: pv.pv_kv_summary_bytes(None),
                 lambda: pv.pv_kv_set_summaries(None, 256, 1 << 30),
                 lambda: pv.pv_block_summarize(None, [0], 0, 0),
                 lambda: pv.pv_block_select(None, [0], 0, 0, 16, 1, 0, 16),
                 lambda: pv.pv_block_attn(None, [0], 0, 0, 16, 16, 1, 16)):
        with pytest.raises(pv.PVError) as e:
            call()
        assert e.value.status == pv.PV_ERR_INVALID_ARG


def test_block_calls_need_device_buffers():
    h = pv.pv_kv_init_paged(cfg_of(2), 6)
    grow(h, 0, 1)
    for call in (lambda: pv.pv_kv_set_summaries(h, 256, 1 << 30),
                 lambda: pv.pv_block_summarize(h, [0], 0, 0),
                 lambda: pv.pv_block_select(h, [0], 0, 0, 16, 4, 0, 16),
                 lambda: pv.pv_block_attn(h, [0], 0, 0, 16, 16, 4, 16),
                 lambda: pv.pv_chunk_attn(h, [0], 0, 0, 16, 16)):
        with pytest.raises(pv.PVError) as e:
            call()
        assert e.value.status == pv.PV_ERR_STATE
    # one block of T = 32 keys per frame
    assert pv.pv_kv_summary_bytes(h) == 2 * 4 * 2 * 6 * 1 * 64 * 4
    pv.pv_kv_destroy(h)


SHAPE, ARG, CAP = pv.PV_ERR_SHAPE, pv.PV_ERR_INVALID_ARG, pv.PV_ERR_CAPACITY


@pytest.mark.parametrize("args,status", [
    ((None, 5, 1, 64, 16), ARG), ((16, 5, 1, 64, None), ARG), ((8, 5, 1, 64, 16), ARG),
    ((16, 5, 1, 64, 8), ARG), ((16, 0, 1, 64, 16), SHAPE), ((16, 5, 0, 64, 16), SHAPE),
    ((16, 5, 1, 96, 16), SHAPE), ((16, (1 << 30) + 1, 1, 64, 16), SHAPE),
    ((16, 1 << 20, 2048, 64, 16), SHAPE)])
def test_summarize_dense_refusals(args, status):
    with pytest.raises(pv.PVError) as e:
        pv.pv_block_summarize_dense(*args, cuda_stream=0)
    assert e.value.status == status


def select(q=16, means=16, n_q=5, n_k=300, heads=2, head_dim=128, keep=2, n_front=0, blocks=16):
    pv.pv_block_select_dense(q, means, n_q, n_k, heads, head_dim, keep, n_front, blocks, 0)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), ARG), (dict(means=None), ARG), (dict(blocks=None), ARG), (dict(q=24), ARG),
    (dict(means=8), ARG), (dict(blocks=2), ARG), (dict(n_q=0), SHAPE), (dict(n_k=0), SHAPE),
    (dict(heads=0), SHAPE), (dict(head_dim=32), SHAPE), (dict(keep=0), SHAPE),
    (dict(keep=(1 << 24) + 1), SHAPE),
    (dict(n_front=-1), SHAPE), (dict(n_front=3), SHAPE), (dict(n_k=16384 * 128 + 1), SHAPE)])
def test_select_dense_refusals(kw, status):
    with pytest.raises(pv.PVError) as e:
        select(**kw)
    assert e.value.status == status


def attend(q=16, k=16, v=16, n_q=5, n_k=300, heads=2, head_dim=128, blocks=16, keep=2, out=16,
           lse=None, ws=256, ws_bytes=1 << 30):
    pv.pv_block_attn_dense(q, k, v, n_q, n_k, heads, head_dim, blocks, keep, out, lse, ws, ws_bytes, 0)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), ARG), (dict(k=None), ARG), (dict(v=None), ARG), (dict(out=None), ARG),
    (dict(blocks=None), ARG), (dict(q=8), ARG), (dict(k=8), ARG), (dict(v=8), ARG),
    (dict(out=8), ARG), (dict(lse=2), ARG), (dict(blocks=2), ARG), (dict(n_q=0), SHAPE),
    (dict(n_k=0), SHAPE), (dict(heads=0), SHAPE), (dict(head_dim=256), SHAPE),
    (dict(keep=0), SHAPE), (dict(keep=-4), SHAPE), (dict(keep=1 << 30), SHAPE), (dict(ws=None), CAP), (dict(ws=128), CAP),
    (dict(ws_bytes=1000), CAP), (dict(n_q=1 << 30, heads=2), SHAPE)])
def test_attn_dense_refusals(kw, status):
    with pytest.raises(pv.PVError) as e:
        attend(**kw)
    assert e.value.status == status


def test_attn_dense_workspace_counts_listed_blocks():
    size = lambda *a: pv.pv_block_attn_dense_ws_bytes(*a)  # noqa: E731
    slot = (128 * 128 + 2 * 128) * 4
    assert size(100, 5000, 2, 128, 3) - size(100, 5000, 1, 128, 1) == 4 * (6 - 1) * slot
    assert size(100, 300, 2, 128, 1 << 24) == size(100, 300, 2, 128, 3)
    assert size(5000, 5000, 24, 128, 30) == size(900, 5000, 24, 128, 30)     # every SM has its slots


def test_contiguous_tensors_are_asked_for():
    torch = pytest.importorskip("torch")
    q = torch.zeros(2, 128, 5, dtype=torch.bfloat16).transpose(1, 2)
    with pytest.raises(pv.PVError) as e:
        select(q=q)
    assert e.value.status == ARG
