"""Block means, block selection and attention over listed blocks on the GPU, on
explicit buffers, against plain f64 forms (block_common)."""
import pytest
import torch

from block_common import (attend64, blocks_of, check_attention, means64, rows_of, select64)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pv():
    from same_step_kv_b200 import pv as m
    return m


def randn(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g, device="cuda")).to(torch.bfloat16)


# ------------------------------------------------------------------ means
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,n", [(1, 1), (3, 127), (2, 128), (2, 129), (1, 255), (5, 1000), (24, 2640)])
def test_means(pv, H, n, D):
    k = randn(n + D, H, n, D)
    out = torch.full((H + 1, blocks_of(n), D), 7.0, device="cuda")
    pv.pv_block_summarize_dense(k, n, H, D, out)
    assert torch.equal(out[:H], means64(k, 128).float())
    assert (out[H] == 7).all()


def test_means_of_large_small_and_negative_values(pv):
    k = torch.zeros(1, 256, 64, dtype=torch.bfloat16, device="cuda")
    k[0, 0], k[0, 1], k[0, 2] = 2.0 ** 100, -(2.0 ** 100), 2.0 ** 64
    k[0, 128], k[0, 129] = 2.0 ** -120, -(2.0 ** -127)
    out = torch.empty(1, 2, 64, device="cuda")
    pv.pv_block_summarize_dense(k, 256, 1, 64, out)
    assert (out[0, 0] == 2.0 ** 57).all()
    assert torch.equal(out[0, 1].double(), torch.full((64,), (2.0 ** -120 - 2.0 ** -127) / 128,
                                                      dtype=torch.float64, device="cuda").float().double())


@pytest.mark.parametrize("D,n", [(64, 700), (128, 700), (128, 90000)])
def test_means_of_infinities_nan_and_subnormals(pv, D, n):
    k = randn(n, 2, n, D)
    inf, nan = float("inf"), float("nan")
    for c, value in ((0, inf), (1, inf), (2, -inf), (3, nan), (4, nan), (5, 2.0 ** 127), (6, 2.0 ** 127),
                     (7, -inf), (9, 2.0 ** -133), (10, 2.0 ** -130)):
        k[:, 5, c] = value
        k[1, n - 1, c] = value
    k[0, 200, 7] = inf
    k[0, 300:400, 9:11] = 0
    k[0, 300, 9:11] = 2.0 ** -133
    out = torch.empty(2, blocks_of(n), D, device="cuda")
    pv.pv_block_summarize_dense(k, n, 2, D, out)
    assert torch.equal(out.nan_to_num(7.0, 8.0, 9.0), means64(k, 128).float().nan_to_num(7.0, 8.0, 9.0))
    assert out[0, 0, 1] == inf and out[0, 0, 3].isnan() and out[0, 0, 7] == -inf


# ------------------------------------------------------------------ selection
@pytest.mark.parametrize("H,D,n_q,n_k,keep,front", [
    (1, 64, 1, 1, 1, 0), (1, 128, 1, 1, 5, 1), (2, 128, 5, 129, 1, 0), (3, 64, 256, 2000, 4, 2),
    (2, 128, 257, 4096, 32, 0), (24, 128, 880, 18480, 37, 3), (1, 64, 700, 256 * 128, 100, 0),
    (1, 128, 3, 257 * 128 + 1, 17, 17), (2, 64, 300, 40007, 313, 0), (2, 64, 300, 40007, 312, 1),
    (40, 64, 1100, 3000, 9, 0)])
def test_select(pv, H, D, n_q, n_k, keep, front):
    q = randn(n_q, H, n_q, D)
    m = randn(n_k, H, blocks_of(n_k), D).float()
    out = torch.full((H, -(-n_q // 256), keep), 99, dtype=torch.int32, device="cuda")
    pv.pv_block_select_dense(q, m, n_q, n_k, H, D, keep, front, out)
    assert torch.equal(out.cpu(), select64(q, m, keep, range(min(front, m.shape[1]))))


@pytest.mark.parametrize("nb", [9, 256, 300, 1000, 5000])
@pytest.mark.parametrize("n_q", [1, 256])
def test_select_ties_go_to_the_lowest_index(pv, nb, n_q):
    # whole-number scores of few values: exact in any order, many of them equal
    g = torch.Generator().manual_seed(nb)
    m = torch.zeros(2, nb, 64)
    m[:, :, 0] = torch.randint(-2, 3, (2, nb), generator=g).float()
    m[1, :, 0] = 0.0
    m[1, ::3, 0] = -0.0
    q = torch.zeros(2, n_q, 64, dtype=torch.bfloat16)
    q[:, :, 0] = 1.0
    q, m = q.cuda(), m.cuda()
    for keep in (1, nb // 3, nb // 2, nb - 1, nb, nb + 3):
        out = torch.empty(2, 1, keep, dtype=torch.int32, device="cuda")
        pv.pv_block_select_dense(q, m, n_q, nb * 128, 2, 64, keep, 0, out)
        assert torch.equal(out.cpu(), select64(q, m, keep)), keep
        assert out[1, 0, :min(keep, nb)].tolist() == list(range(min(keep, nb)))


@pytest.mark.parametrize("nb,close", [(40, 7), (200, 60), (900, 300), (900, 700), (3000, 600)])
def test_select_tells_scores_apart_that_f32_cannot(pv, nb, close):
    # `close` blocks whose scores differ in the 30th bit and later, spread over the list, the
    # border among them: f64 decides
    g = torch.Generator().manual_seed(nb + close)
    m = torch.randn(1, nb, 64, generator=g) * 0.1
    at = torch.randperm(nb, generator=g)[:close]
    m[0, at] = torch.randn(64, generator=g)
    m[0, at, 0] = 1.0
    m[0, at, 1] = torch.randint(-40, 40, (close,), generator=g).float() * 2.0 ** -33
    q = torch.randn(1, 1, 64, generator=g).to(torch.bfloat16)
    q[0, 0, 0], q[0, 0, 1] = 4.0, 1.5
    q, m = q.cuda(), m.cuda()
    for keep in (1, close // 2, close - 1, min(nb, close + 3)):
        out = torch.empty(1, 1, keep, dtype=torch.int32, device="cuda")
        pv.pv_block_select_dense(q, m, 1, nb * 128, 1, 64, keep, 0, out)
        assert torch.equal(out.cpu(), select64(q, m, keep)), keep


@pytest.mark.parametrize("scale", [2.0 ** -70, 2.0 ** -40, 2.0 ** 60, 2.0 ** 100])
def test_select_of_very_small_and_very_large_values(pv, scale):
    # products and squares outside f32's range
    q = (randn(1, 2, 3, 64).float() * scale).to(torch.bfloat16)
    m = randn(2, 2, 300, 64).float() * scale
    out = torch.empty(2, 1, 50, dtype=torch.int32, device="cuda")
    pv.pv_block_select_dense(q, m, 3, 300 * 128, 2, 64, 50, 1, out)
    assert torch.equal(out.cpu(), select64(q, m, 50, [0]))


def test_select_of_the_most_blocks(pv):
    nb = 16384
    q = randn(1, 2, 1, 64)
    m = randn(2, 2, nb, 64).float()
    out = torch.empty(2, 1, 700, dtype=torch.int32, device="cuda")
    pv.pv_block_select_dense(q, m, 1, nb * 128, 2, 64, 700, 5, out)
    assert torch.equal(out.cpu(), select64(q, m, 700, range(5)))


def test_select_puts_nan_last_and_stays_in_range(pv):
    q = randn(1, 1, 1, 64)
    m = randn(2, 1, 40, 64).float()
    m[0, ::2] = float("nan")
    m[0, 1] = float("inf") * torch.sign(q[0, 0].float())
    m[0, 3] = -m[0, 1]
    out = torch.empty(1, 1, 22, dtype=torch.int32, device="cuda")
    pv.pv_block_select_dense(q, m, 1, 40 * 128, 1, 64, 22, 0, out)
    got = out[0, 0].tolist()
    assert got == sorted(set(range(1, 40, 2)) | {0, 2})


# ------------------------------------------------------------------ attention
def lists_of(seed, H, n_q, nb, keep):
    g = torch.Generator().manual_seed(seed)
    rows = [[sorted(torch.randperm(nb, generator=g)[:keep].tolist()) for _ in range(-(-n_q // 256))]
            for _ in range(H)]
    t = torch.full((H, -(-n_q // 256), keep), -1, dtype=torch.int32)
    for h in range(H):
        for i, r in enumerate(rows[h]):
            t[h, i, :len(r)] = torch.tensor(r, dtype=torch.int32)
    return t


def attend(pv, q, k, v, lists, lse=True):
    (H, n_q, D), n_k, keep = q.shape, k.shape[1], lists.shape[2]
    n = pv.pv_block_attn_dense_ws_bytes(n_q, n_k, H, D, keep)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    out = torch.full((n_q + 1, H, D), 3.0, dtype=torch.bfloat16, device="cuda")
    e = torch.full((n_q + 1, H), 3.0, device="cuda")
    pv.pv_block_attn_dense(q, k, v, n_q, n_k, H, D, lists.cuda(), keep, out, e if lse else None, ws, n)
    assert pv.pv_attn_poll_device_error(ws, n) == 0
    assert (out[n_q:] == 3).all() and (e[n_q:] == 3).all(), "rows behind the sequence were written"
    return out[:n_q], e[:n_q] if lse else None


def reference(q, k, v, lists):
    n_k = k.shape[1]
    t = lists.tolist()
    return attend64(q, k, v, lambda h, g: rows_of(t[h][g], n_k, blocks_of(n_k)))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,n_q,n_k,keep", [
    (1, 1, 1, 1), (2, 1, 130, 2), (3, 7, 127, 3), (1, 128, 128, 1), (2, 129, 1000, 3),
    (2, 256, 1024, 8), (3, 257, 1300, 5), (1, 300, 129, 4), (24, 1, 40007, 32), (5, 600, 5000, 17),
    # either side of each kernel's row counts, few and many parts to an item
    (3, 8, 3000, 9), (3, 9, 3000, 9), (1, 16, 9000, 70), (1, 17, 9000, 70), (2, 31, 300, 3),
    (20, 32, 2000, 15), (20, 33, 2000, 15), (1, 64, 9000, 70), (1, 100, 9000, 71), (150, 3, 500, 2),
    (2, 1000, 777, 1)])
def test_attention(pv, H, n_q, n_k, keep, D):
    q, k, v = randn(1, H, n_q, D), randn(2, H, n_k, D), randn(3, H, n_k, D)
    lists = lists_of(n_q + n_k, H, n_q, blocks_of(n_k), keep)
    out, lse = attend(pv, q, k, v, lists)
    check_attention(out, lse, reference(q, k, v, lists), f"{H} {n_q} {n_k} {keep} {D}")


@pytest.mark.parametrize("D", [64, 128])
def test_attention_at_chunk_size(pv, D):
    H, n_q, n_k, keep = 24, 880, 18480, 37
    q, k, v = randn(1, H, n_q, D), randn(2, H, n_k, D), randn(3, H, n_k, D)
    lists = lists_of(5, H, n_q, blocks_of(n_k), keep)
    out, lse = attend(pv, q, k, v, lists)
    check_attention(out, lse, reference(q, k, v, lists))
    again, _ = attend(pv, q, k, v, lists, lse=False)
    assert torch.equal(out, again)


def test_sharp_and_flat_rows(pv):
    # scores of +-100 (one key takes all), equal scores, and a maximum that grows tile by tile
    H, n_q, n_k, D = 3, 200, 1500, 128
    q, k, v = randn(1, H, n_q, D), randn(2, H, n_k, D), randn(3, H, n_k, D)
    q[0] *= 16
    q[1] = 0
    k[2] = (k[2].float() * torch.linspace(0, 8, n_k, device="cuda")[:, None]).to(torch.bfloat16)
    lists = lists_of(5, H, n_q, blocks_of(n_k), 12)
    out, lse = attend(pv, q, k, v, lists)
    check_attention(out, lse, reference(q, k, v, lists))


def test_empty_blocks_repeated_blocks_and_empty_rows(pv):
    H, n_q, n_k, D = 2, 700, 900, 64
    nb, keep = blocks_of(n_k), 6
    q, k, v = randn(1, H, n_q, D), randn(2, H, n_k, D), randn(3, H, n_k, D)
    lists = torch.tensor([[[-1] * 6, [7, -1, -1, -1, -1, -1], [-1, -1, 3, -5, 2 ** 31 - 1, 0]],
                          [[nb, nb + 1, -1, -1, -1, -1], [2, 2, 7, 7, 7, 1], [5, 4, 3, 2, 1, 0]]],
                         dtype=torch.int32)
    out, lse = attend(pv, q, k, v, lists)
    check_attention(out, lse, reference(q, k, v, lists))
    assert (out[:256] == 0).all() and torch.isinf(lse[:256]).all()


@pytest.mark.parametrize("n_q", [1, 520])
def test_nothing_outside_the_listed_blocks_is_read(pv, n_q):
    # NaN and infinities in every unlisted block, and behind the last key of a head's last block
    H, n_k, D, keep = 3, 1000, 128, 3
    q, k, v = randn(1, H, n_q, D), randn(2, H, n_k, D), randn(3, H, n_k, D)
    lists = torch.tensor([[0, 3, 7], [1, 2, 7], [7, -1, -1]], dtype=torch.int32)
    lists = lists[:, None].expand(H, -(-n_q // 256), keep).contiguous()
    ref = reference(q, k, v, lists)
    for h in range(H):
        for b in set(range(8)) - set(lists[h, 0].tolist()):
            k[h, b * 128:(b + 1) * 128] = float("nan")
            v[h, b * 128:(b + 1) * 128] = float("inf") if b % 2 else float("nan")
    out, lse = attend(pv, q, k, v, lists)
    check_attention(out, lse, ref)


def test_every_block_listed_is_dense_attention(pv):
    H, n_q, n_k, D = 4, 500, 3001, 128
    q, k, v = randn(1, H, n_q, D), randn(2, H, n_k, D), randn(3, H, n_k, D)
    nb = blocks_of(n_k)
    lists = torch.arange(nb, dtype=torch.int32).expand(H, 2, nb).contiguous()
    out, lse = attend(pv, q, k, v, lists)
    check_attention(out, lse, reference(q, k, v, lists))
    n = pv.pv_attn_dense_ws_bytes(n_q, n_k, H, D)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    dense = torch.empty_like(out)
    pv.pv_attn_dense(q, k, v, n_q, n_k, H, D, dense, None, ws, n)
    assert (dense.float() - out.float()).abs().max() < 2e-2


# ------------------------------------------------------------------ together
def pipeline(pv, q, k, v, keep, front, bufs, stream=None):
    (H, n_q, D), n_k = q.shape, k.shape[1]
    pv.pv_block_summarize_dense(k, n_k, H, D, bufs["means"], stream)
    pv.pv_block_select_dense(q, bufs["means"], n_q, n_k, H, D, keep, front, bufs["blocks"], stream)
    pv.pv_block_attn_dense(q, k, v, n_q, n_k, H, D, bufs["blocks"], keep, bufs["out"], bufs["lse"],
                           bufs["ws"], bufs["n"], stream)


def buffers(pv, H, n_q, n_k, D, keep):
    n = pv.pv_block_attn_dense_ws_bytes(n_q, n_k, H, D, keep)
    return dict(means=torch.empty(H, blocks_of(n_k), D, device="cuda"),
                blocks=torch.empty(H, -(-n_q // 256), keep, dtype=torch.int32, device="cuda"),
                out=torch.empty(n_q, H, D, dtype=torch.bfloat16, device="cuda"),
                lse=torch.empty(n_q, H, device="cuda"),
                ws=torch.zeros(n, dtype=torch.uint8, device="cuda"), n=n)


@pytest.mark.parametrize("H,D,n_q,n_k,keep,front", [(4, 128, 900, 5000, 11, 2), (2, 64, 1, 3000, 4, 0)])
def test_summarize_select_attend(pv, H, D, n_q, n_k, keep, front):
    q, k, v = randn(1, H, n_q, D), randn(2, H, n_k, D), randn(3, H, n_k, D)
    b = buffers(pv, H, n_q, n_k, D, keep)
    pipeline(pv, q, k, v, keep, front, b)
    m = means64(k, 128).float()
    want = select64(q, m, keep, range(front))
    assert torch.equal(b["means"], m) and torch.equal(b["blocks"].cpu(), want)
    check_attention(b["out"], b["lse"], reference(q, k, v, want))


def test_one_workspace_for_calls_of_any_shape(pv):
    """Heads, queries, keys, lists and head dimensions change from call to call, and with them the
    kernel and the way the work is shared out."""
    shapes = [(3, 128, 30, 5000, 20), (3, 128, 200, 900, 3), (40, 64, 700, 3000, 24), (3, 128, 5, 3000, 24),
              (2, 64, 1100, 6000, 40), (24, 128, 1, 9000, 60), (50, 64, 2000, 200, 2), (3, 128, 30, 200, 2),
              (24, 64, 20, 4000, 7)] * 2
    n = max(pv.pv_block_attn_dense_ws_bytes(a, b, h, d, c) for h, d, a, b, c in shapes)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    for i, (H, D, n_q, n_k, keep) in enumerate(shapes):
        q, k, v = randn(i, H, n_q, D), randn(40 + i, H, n_k, D), randn(80 + i, H, n_k, D)
        lists = lists_of(i, H, n_q, blocks_of(n_k), keep)
        out = torch.zeros(n_q, H, D, dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros(n_q, H, device="cuda")
        pv.pv_block_attn_dense(q, k, v, n_q, n_k, H, D, lists.cuda(), keep, out, lse, ws, n)
        check_attention(out, lse, reference(q, k, v, lists), str(i))
    assert pv.pv_attn_poll_device_error(ws, n) == 0


def test_tensors_of_another_kind_are_refused(pv):
    q, m = randn(1, 2, 5, 64), torch.zeros(2, 3, 64, device="cuda")
    out = torch.empty(2, 1, 2, dtype=torch.int32, device="cuda")
    for a, b, c in ((q.float(), m, out), (q, m.bfloat16(), out), (q, m, out.long()), (q.cpu(), m, out),
                    (q.transpose(0, 1), m, out)):
        with pytest.raises(pv.PVError) as e:
            pv.pv_block_select_dense(a, b, 5, 300, 2, 64, 2, 0, c)
        assert e.value.status == pv.PV_ERR_INVALID_ARG


def test_captured_replayed_and_on_other_streams(pv):
    H, D, n_q, n_k, keep = 3, 128, 300, 2500, 5
    sets = []
    for i in range(2):
        q, k, v = randn(10 + i, H, n_q, D), randn(20 + i, H, n_k, D), randn(30 + i, H, n_k, D)
        sets.append((q, k, v, buffers(pv, H, n_q, n_k, D, keep)))
    want = []
    for q, k, v, b in sets:
        pipeline(pv, q, k, v, keep, 1, b)
        want.append([b[x].clone() for x in ("blocks", "out", "lse")])
    torch.cuda.synchronize()
    # two streams at once, each with its own workspace
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        for s, (q, k, v, b) in zip(streams, sets):
            pipeline(pv, q, k, v, keep, 1, b, s)
    torch.cuda.synchronize()
    for (_, _, _, b), w in zip(sets, want):
        assert all(torch.equal(b[x], y) for x, y in zip(("blocks", "out", "lse"), w))
    # one graph, new inputs in the captured buffers
    q, k, v, b = sets[0]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pipeline(pv, q, k, v, keep, 1, b)
    for src, w in ((1, want[1]), (0, want[0])):
        fresh = [randn(a + src, *t.shape) for a, t in ((10, q), (20, k), (30, v))]
        for t, f in zip((q, k, v), fresh):
            t.copy_(f)
        for x in ("blocks", "out", "lse"):
            b[x].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(b[x], y) for x, y in zip(("blocks", "out", "lse"), w))


@pytest.mark.parametrize("captured", [False, True])
def test_inputs_from_copies_memsets_and_other_streams(pv, captured):
    """The calls wait for whatever came before them in the stream: a copy, a memset, a kernel, work of
    another stream; and what comes after waits for them."""
    H, D, n_q, n_k, keep = 3, 128, 300, 2500, 5
    q, k, v = randn(1, H, n_q, D), randn(2, H, n_k, D), randn(3, H, n_k, D)
    b = buffers(pv, H, n_q, n_k, D, keep)
    big = torch.randn(40_000_000, device="cuda")
    pipeline(pv, q, k, v, keep, 1, b)
    want = [b[x].clone() for x in ("means", "blocks", "out", "lse")]
    qc, kc, vc = (torch.empty_like(t) for t in (q, k, v))
    side = torch.cuda.Stream()
    got = [torch.empty_like(w) for w in want]

    def body():
        here = torch.cuda.current_stream()
        for t in (qc, kc, vc, *(b[x] for x in ("means", "blocks", "out", "lse"))):
            t.zero_()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            big.mul_(1.0)
            kc.copy_(k)
        big.add_(0.0)
        qc.copy_(q)
        vc.copy_(v)
        here.wait_stream(side)
        pipeline(pv, qc, kc, vc, keep, 1, b)
        for g, x in zip(got, ("means", "blocks", "out", "lse")):
            g.copy_(b[x])
            b[x].zero_()

    if captured:
        body()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            body()
        for _ in range(5):
            graph.replay()
    else:
        for _ in range(5):
            body()
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))


@pytest.mark.parametrize("n_q", [20, 300])
def test_offsets_beyond_32_bits(pv, n_q):
    """12 heads of 2,000,077 keys: 3.1e9 values of K and of V; the last head is checked."""
    H, n_k, D, keep, h = 12, 2_000_077, 128, 6, 11
    nb = blocks_of(n_k)
    k, v = (torch.empty(H, n_k, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for i in range(H):
        k[i], v[i] = randn(i, n_k, D), randn(100 + i, n_k, D)
    q = randn(7, H, n_q, D)
    b = buffers(pv, H, n_q, n_k, D, keep)
    pipeline(pv, q, k, v, keep, 1, b)
    m = means64(k[h:], 128).float()
    assert torch.equal(b["means"][h:], m)
    assert torch.equal(b["blocks"][h:].cpu(), select64(q[h:], m, keep, [0]))
    lists = b["blocks"]
    lists[:, :, -1] = nb - 1       # the ragged last block
    pv.pv_block_attn_dense(q, k, v, n_q, n_k, H, D, lists, keep, b["out"], b["lse"], b["ws"], b["n"])
    t = lists[h:].tolist()
    check_attention(b["out"][:, h:], b["lse"][:, h:],
                    attend64(q[h:], k[h:], v[h:], lambda a, g: rows_of(t[a][g], n_k, nb)))
