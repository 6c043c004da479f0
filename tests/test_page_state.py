"""pv_kv_set_state of a paged store whose streams share pages (bookkeeping-only handles, no device):
a stream that is set to other frames leaves the pages that others hold to them."""
import pytest

from same_step_kv_b200 import pv

F0, R = 3, 3


def store(pages, streams=3):
    return pv.pv_kv_init_paged(pv.make_config(2, 2, 64, 8, 4, first_frames=F0, ring_slots=R, max_streams=streams,
                                              max_frames=64), pages)


def grow(h, stream, chunk):
    pv.pv_kv_begin_chunk(h, stream, F0)
    pv.pv_kv_begin_sink(h, stream)
    for _ in range(chunk):
        pv.pv_kv_begin_chunk(h, stream, 1)


def set_chunk(h, stream, chunk, phase=pv.PV_PHASE_STEADY):
    st = pv.pv_kv_state()
    st.phase, st.chunk = phase, chunk
    pv.pv_kv_set_state(h, stream, st)


def ring(h, stream):
    sink, pages = pv.pv_kv_page_table(h, stream)
    return sink, pages[:R]


def frames(chunk):
    """Frame of each slot at `chunk`, from the schedule: slot i holds the latest chunk j with (j - 1) % R == i."""
    return [max([j for j in range(1, chunk + 1) if (j - 1) % R == i], default=None) for i in range(R)]


@pytest.mark.parametrize("src", range(1, 8))
@pytest.mark.parametrize("to", range(1, 10))
def test_no_page_of_another_frame_stays_shared(src, to):
    h = store(20)
    grow(h, 0, src)
    pv.pv_kv_fork(h, 0, [1], 0)
    before = ring(h, 0)
    set_chunk(h, 1, to)
    assert ring(h, 0) == before
    sink, mine = ring(h, 1)
    assert sink == before[0]                     # the same F0 frames
    for i, (was, now) in enumerate(zip(frames(src), frames(to))):
        if now is None:
            assert mine[i] == -1
        elif was == now:
            assert mine[i] == before[1][i]       # a frame that stays
        else:
            assert mine[i] >= 0 and mine[i] not in before[1] and mine[i] not in range(sink, sink + F0)
    held = set(range(sink, sink + F0)) | set(p for p in before[1] + mine if p >= 0)
    assert pv.pv_kv_free_pages(h)[0] == 20 - len(held)
    # what stream 1 took it gives back, what stream 0 holds stays
    pv.pv_kv_release(h, 1)
    assert pv.pv_kv_free_pages(h)[0] == 20 - F0 - min(src, R)
    assert ring(h, 0) == before
    pv.pv_kv_destroy(h)


def test_pages_of_its_own_are_kept_for_other_frames():
    h = store(12)
    grow(h, 0, 5)
    before = ring(h, 0)
    set_chunk(h, 0, 9)
    assert ring(h, 0) == before and pv.pv_kv_free_pages(h) == (6, 6)
    pv.pv_kv_destroy(h)


def test_too_few_free_pages_change_nothing():
    h = store(F0 + R + 2)
    grow(h, 0, 4)
    pv.pv_kv_fork(h, 0, [1, 2], 0)
    before = [ring(h, i) for i in range(3)]
    with pytest.raises(pv.PVError) as e:
        set_chunk(h, 1, 4 + R)                   # three other frames, two free pages
    assert e.value.status == pv.PV_ERR_CAPACITY
    assert [ring(h, i) for i in range(3)] == before
    assert pv.pv_kv_free_pages(h) == (2, 2)
    assert pv.pv_kv_get_state(h, 1).chunk == 4
    set_chunk(h, 1, 4 + 2)                       # two other frames: slots 1 and 2
    assert ring(h, 1)[1][0] == before[0][1][0]
    assert sorted(ring(h, 1)[1][1:]) == [F0 + R, F0 + R + 1]
    pv.pv_kv_destroy(h)


def test_a_stream_with_no_history_takes_pages_of_its_own():
    h = store(16)
    grow(h, 0, 3)
    set_chunk(h, 1, 3)
    assert not set(ring(h, 1)[1]) & set(ring(h, 0)[1])
    set_chunk(h, 1, 0, pv.PV_PHASE_FIRST)
    assert ring(h, 1)[1] == [-1] * R
    set_chunk(h, 1, -1, pv.PV_PHASE_NEW)
    assert pv.pv_kv_free_pages(h)[0] == 10
    pv.pv_kv_destroy(h)


@pytest.mark.parametrize("heads,fits", [((1 << 24) - 1, True), (1 << 24, False), (1 << 25, False),
                                        ((1 << 25) + (1 << 18), False)])
def test_arrival_counters_beyond_32_bits_are_refused(heads, fits):
    """The streams of a paged store are not bounded by its rows: 64 streams of 2^24 heads would need
    2^31 counters."""
    c = pv.make_config(1, heads, 64, 1, 1, first_frames=1, ring_slots=1, steps=1, max_streams=64)
    if fits:
        kv, ws = pv.pv_kv_paged_required_bytes(c, 2)
        assert kv == 2 * heads * 2 * 64 * 2 and ws > 64 * heads * 2 * 4
        return
    for call in (lambda: pv.pv_kv_paged_required_bytes(c, 2), lambda: pv.pv_kv_init_paged(c, 2)):
        with pytest.raises(pv.PVError) as e:
            call()
        assert e.value.status == pv.PV_ERR_SHAPE
