"""Attaching block means on the GPU: the zero fill is complete when the call returns, whatever the
default stream still has to do, so that calls on other streams may follow at once."""
import pytest
import torch

from block_common import blocks_of, means64
from same_step_kv_b200 import synth

pytestmark = pytest.mark.gpu
F0 = 3


@pytest.fixture(scope="module")
def pv():
    from same_step_kv_b200 import pv as m
    return m


@pytest.mark.parametrize("pages", [None, 6])
def test_means_written_right_after_attaching_stay(pv, pages):
    H, D, W, Hh, R = 4, 128, 20, 15, 2
    cfg = pv.make_config(1, H, D, W, Hh, ring_slots=R, steps=1, max_streams=1, max_frames=64)
    store = pv.KVStore(cfg, pages=pages)
    h, T = store.handle, W * Hh
    pv.pv_kv_begin_chunk(h, 0, F0)
    n = F0 * T
    q, k, v = synth.chunk_qkv(1, 0, 0, 7, n, H, D, "cuda")
    pv.pv_rope_append(h, [0], 0, 0, q, k, v, torch.empty(H, n, D, dtype=torch.bfloat16, device="cuda"))
    size = pv.pv_kv_summary_bytes(h)
    buf = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    a = torch.randn(8192, 8192, device="cuda").bfloat16()
    side = torch.cuda.Stream()
    rows = F0 * blocks_of(T)
    kr = store.k_region().view(H, -1, D)[:, :n]
    want = means64(kr.reshape(H * F0, T, D), 128).float().reshape(H, rows, D)
    for _ in range(3):
        torch.cuda.synchronize()
        for _ in range(30):                      # the default stream is busy for some 20 ms
            torch.matmul(a, a)
        pv.pv_kv_set_summaries(h, buf, size)
        pv.pv_block_summarize(h, [0], 0, 0, side)
        torch.cuda.synchronize()
        got = buf.view(torch.float32).view(H, -1, D)
        assert torch.equal(got[:, :rows], want)
        assert (got[:, rows:] == 0).all()
        pv.pv_kv_set_summaries(h, None)
        buf.fill_(255)
    store.close()


def test_a_store_made_on_a_busy_stream(pv):
    """Memory that the allocator hands out again while work of the current stream still writes it."""
    side = torch.cuda.Stream()
    cfg = pv.make_config(1, 4, 128, 20, 15, ring_slots=2, steps=1, max_streams=1, max_frames=64)
    a = torch.randn(8192, 8192, device="cuda").bfloat16()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        first = pv.KVStore(cfg, summaries=True)
        sizes = first.kv_bytes, first.ws_bytes, first.summ_buf.numel()
        b = torch.empty_like(a)
        for _ in range(30):
            torch.matmul(a, a, out=b)
        junk = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
        for t in junk:
            t.fill_(255)
        del junk, t
        made = pv.KVStore(cfg, summaries=True)
        torch.cuda.synchronize()
        assert (made.summary_region() == 0).all()
        assert (made.k_region() == 0).all() and (made.v_region() == 0).all()
    first.close(), made.close()
