"""Chunk attention through the page table against the f64 form (block_common) over the rows that the
table names: frames that end inside a 128-key tile, streams at mixed ring fills whose pages lie
between one another's, few queries (one mma.sync tile) and many.  Every row that the streams do not
hold is NaN."""
import pytest
import torch

from block_common import attend64, check_attention

pytestmark = pytest.mark.gpu
F0 = 3


@pytest.fixture(scope="module")
def pv():
    from same_step_kv_b200 import pv as m
    return m


def pages_of(pv, h, stream, fill):
    sink, ring = pv.pv_kv_page_table(h, stream)
    return list(range(sink, sink + F0)) + ring[:fill]


# frames of 1, 8 and 20 tokens: at most 32 queries a stream; the others go in 256-query items
@pytest.mark.parametrize("W,Hh", [(1, 1), (4, 2), (5, 4), (12, 11), (16, 8), (20, 15), (37, 9)])
@pytest.mark.parametrize("D,H", [(64, 3), (128, 2)])
def test_paged_chunk_attention(pv, W, Hh, D, H):
    T, R, chunks = W * Hh, 5, [7, 2, 4]
    cfg = pv.make_config(2, H, D, W, Hh, ring_slots=R, steps=2, max_streams=4, max_frames=64)
    store = pv.KVStore(cfg, pages=4 * (F0 + R))
    h = store.handle
    st = pv.pv_kv_state()
    st.phase = pv.PV_PHASE_STEADY
    for up_to in range(1, max(chunks) + 1):      # in turn, so that the pages interleave
        for i, c in enumerate(chunks):
            st.chunk = min(c, up_to)
            pv.pv_kv_set_state(h, i, st)
    pv.pv_kv_fork(h, 1, [3], 0)                  # stream 3 reads stream 1's pages
    fills = [min(c, R) for c in chunks] + [2]
    layer, step = 1, 0
    K, V = store.k_region(), store.v_region()
    K.fill_(float("nan")), V.fill_(float("nan"))
    g = torch.Generator(device="cuda")
    g.manual_seed(T + D)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    tables = [pages_of(pv, h, i, f) for i, f in enumerate(fills)]
    assert tables[3] == tables[1] and tables[0] != sorted(range(len(tables[0])))
    for p in sorted(set(sum(tables, []))):
        for r in (K, V):
            r[layer, step, :, p * T:(p + 1) * T] = rnd(H, T, D)
    for ids in ([0], [2, 0], [3, 0, 2, 1]):
        q = rnd(len(ids), H, T, D)
        out = torch.full((len(ids) * T + 1, H, D), 3.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((len(ids) * T + 1, H), 3.0, device="cuda")
        pv.pv_chunk_attn(h, ids, layer, step, q, out, lse)
        for a, i in enumerate(ids):
            at = torch.cat([torch.arange(p * T, (p + 1) * T) for p in tables[i]]).cuda()
            k, v = K[layer, step][:, at], V[layer, step][:, at]
            ref = attend64(q[a], k, v, lambda head, group, n=len(at): range(n))
            check_attention(out[a * T:(a + 1) * T], lse[a * T:(a + 1) * T], ref, f"stream {i} of {ids}")
        assert (out[-1] == 3).all() and (lse[-1] == 3).all()
    assert pv.pv_kv_poll_device_error(h) == 0
    store.close()


def test_paged_first_chunk_and_sink_pass(pv):
    """The first chunk's queries over its own F0 pages, in mid-store."""
    W, Hh, D, H, R = 20, 15, 64, 2, 2
    T = W * Hh
    cfg = pv.make_config(1, H, D, W, Hh, ring_slots=R, steps=2, max_streams=2, max_frames=64)
    store = pv.KVStore(cfg, pages=12)
    h = store.handle
    pv.pv_kv_begin_chunk(h, 0, F0)
    pv.pv_kv_begin_chunk(h, 1, F0)
    K, V = store.k_region(), store.v_region()
    K.fill_(float("nan")), V.fill_(float("nan"))
    at = slice(F0 * T, 2 * F0 * T)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    for s in range(2):
        K[0, s, :, at], V[0, s, :, at] = rnd(H, F0 * T, D), rnd(H, F0 * T, D)
    q = rnd(H, F0 * T, D)
    out = torch.empty(F0 * T, H, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(F0 * T, H, device="cuda")
    for step in (1, pv.PV_STEP_SINK):
        if step == pv.PV_STEP_SINK:
            pv.pv_kv_begin_sink(h, 1)
        s = max(step, 0)
        pv.pv_chunk_attn(h, [1], 0, step, q, out, lse)
        ref = attend64(q, K[0, s, :, at], V[0, s, :, at], lambda head, group: range(F0 * T))
        check_attention(out, lse, ref, f"step {step}")
    store.close()
