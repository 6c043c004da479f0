"""The binding's look at the tensors of the block calls: each argument has one type, and a tensor of
another one, of the same size in bytes or not, is refused before its address is asked for."""
import pytest
import torch

from same_step_kv_b200 import pv


class Tensor:
    """A CUDA tensor as far as the binding looks; its address is never to be asked for."""

    def __init__(self, dtype, contiguous=True, cuda=True):
        self.dtype, self.is_cuda, self.shape, self.device = dtype, cuda, (2, 5, 64), "cuda:0"
        self.contiguous = contiguous

    def is_contiguous(self):
        return self.contiguous

    def element_size(self):
        return torch.empty(0, dtype=self.dtype).element_size()

    def data_ptr(self):
        raise AssertionError(f"the address of a {self.dtype} tensor was taken")


BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
OTHERS = [torch.float16, torch.bfloat16, torch.int16, torch.float32, torch.int32, torch.int64, torch.float64,
          torch.uint8]
# call, its tensor arguments by position and their types (the other arguments are never reached)
CALLS = {
    "pv_block_summarize_dense": (lambda t: pv.pv_block_summarize_dense(t[0], 5, 2, 64, t[1], 0), [BF, F32]),
    "pv_block_select_dense": (lambda t: pv.pv_block_select_dense(t[0], t[1], 5, 300, 2, 64, 2, 0, t[2], 0),
                              [BF, F32, I32]),
    "pv_block_attn_dense": (lambda t: pv.pv_block_attn_dense(t[0], t[1], t[2], 5, 300, 2, 64, t[3], 2, t[4], t[5],
                                                             t[6], 1 << 30, 0),
                            [BF, BF, BF, I32, BF, F32, torch.uint8]),
    "pv_block_select": (lambda t: pv.pv_block_select(None, [0], 0, 0, t[0], 2, 0, t[1], 0), [BF, I32]),
    "pv_block_attn": (lambda t: pv.pv_block_attn(None, [0], 0, 0, t[0], t[1], 2, t[2], t[3], 0),
                      [BF, I32, BF, F32]),
}


@pytest.mark.parametrize("name,at", [(n, i) for n, (_, types) in CALLS.items() for i in range(len(types))])
def test_tensors_of_another_type_are_refused(name, at):
    call, types = CALLS[name]
    wrong = [Tensor(d) for d in OTHERS if d != types[at]]
    wrong += [Tensor(types[at], contiguous=False), Tensor(types[at], cuda=False)]
    for w in wrong:
        t = [256] * len(types)          # an address stands for any tensor
        t[at] = w
        with pytest.raises(pv.PVError) as e:
            call(t)
        assert e.value.status == pv.PV_ERR_INVALID_ARG
        assert str(types[at]) in str(e.value)


@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_the_right_type_are_passed_on(name):
    call, types = CALLS[name]
    for at in range(len(types)):
        t = [256] * len(types)
        t[at] = Tensor(types[at])
        with pytest.raises(AssertionError, match="address"):
            call(t)
