"""Block selection where f32 products overflow: the scores are defined in f64, so a block whose
f32 score is infinite or NaN has its place by its f64 one, beside blocks of ordinary size."""
import pytest
import torch

from block_common import select64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pv():
    from same_step_kv_b200 import pv as m
    return m


def select(pv, q, m, keep, front=0):
    (H, n_q, D), nb = q.shape, m.shape[1]
    out = torch.full((H, 1, keep), 99, dtype=torch.int32, device="cuda")
    pv.pv_block_select_dense(q, m, n_q, nb * 128, H, D, keep, front, out)
    return out.cpu()


def test_products_that_cancel_in_f64_and_not_in_f32(pv):
    # f64 scores -2^180 < 2^180 < 2^181; in f32 -inf, NaN, NaN
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    q[0, 0, :2] = 2.0 ** 90
    m = torch.zeros(1, 3, 64, device="cuda")
    m[0, 0, 0] = -(2.0 ** 90)
    m[0, 1, 0], m[0, 1, 1] = 2.0 ** 91, -(2.0 ** 90)
    m[0, 2, 0], m[0, 2, 1] = 1.5 * 2.0 ** 91, -(2.0 ** 90)
    for keep, want in ((1, [2]), (2, [1, 2]), (3, [0, 1, 2])):
        assert select(pv, q, m, keep)[0, 0].tolist() == want, keep


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("nb", [5, 40, 256, 300, 900])
@pytest.mark.parametrize("n_q", [1, 200])
def test_small_blocks_among_overflowing_ones(pv, nb, n_q, D):
    g = torch.Generator(device="cuda")
    g.manual_seed(nb + D)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    q = (rnd(2, n_q, D) * 2.0 ** 90).to(torch.bfloat16)
    m = rnd(2, nb, D) * 2.0 ** 90
    small = torch.rand(2, nb, generator=g, device="cuda") < 0.4
    m[small] *= 2.0 ** -100          # finite f32 scores of either sign
    m[0, nb // 2] = 0.0
    for keep in sorted({1, 2, nb // 4 + 1, nb // 2, nb - 1, nb, nb + 2}):
        for front in (0, min(keep, 2)):
            got = select(pv, q, m, keep, front)
            assert torch.equal(got, select64(q, m, keep, range(front))), (keep, front)
