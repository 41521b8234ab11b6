"""What block.py refuses before the library is called, on the CPU."""
import pytest
import torch

from communication_overlap_gb300 import block, fo

ROWS, INTER = 3, 40
CODES, SCALES = fo.fo_checkpoint_sizes(ROWS, INTER)


def codes(n=CODES, dtype=torch.int8):
    return torch.zeros(n, dtype=dtype)


def scales(n=SCALES, dtype=torch.uint8):
    return torch.zeros(n, dtype=dtype)


def test_a_checkpoint_holds_what_its_sizes_say():
    kept = block.Checkpoint(codes(), scales(), ROWS, INTER, "silu")
    assert kept.values().shape == (ROWS, 2 * INTER)
    for bad in ((codes(CODES - 1), scales(), ROWS, INTER, "silu"),
                (codes(), scales(SCALES - 1), ROWS, INTER, "silu"),
                (codes(), scales(), ROWS + 1, INTER, "silu"),
                (codes(), scales(), ROWS, 2 * INTER, "silu"),
                (codes(dtype=torch.uint8), scales(), ROWS, INTER, "silu"),
                (codes(), scales(dtype=torch.int8), ROWS, INTER, "silu"),
                (codes(2 * CODES)[::2], scales(), ROWS, INTER, "silu"),
                (codes(), scales(2 * SCALES)[::2], ROWS, INTER, "silu"),
                (codes(), scales(), ROWS, INTER, "tanh")):
        with pytest.raises(ValueError):
            block.Checkpoint(*bad)


def test_a_sum_into_a_tensor_that_requires_a_gradient():
    index = torch.zeros((2, 1), dtype=torch.int32)
    with pytest.raises(ValueError, match="gradient"):
        block.combine(torch.zeros((4, 8)), index, out=torch.zeros((2, 8), requires_grad=True))
    with pytest.raises(ValueError, match="one CUDA device"), torch.no_grad():
        block.combine(torch.zeros((4, 8)), index, out=torch.zeros((2, 8), requires_grad=True))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float64])
def test_norms_of_another_type(dtype):
    x = torch.ones((4, 8), device="cuda")
    g = torch.ones(8, device="cuda")
    n = block.norm(x, pre_gain=g)
    n.rstd = n.rstd.to(dtype)
    with pytest.raises(ValueError):
        block.norm_backward(x, None, n, dy=x, pre_gain=g)
