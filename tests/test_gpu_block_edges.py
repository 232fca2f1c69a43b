"""GPU tests of the edges of blocks.py, against oracle/block_oracle.py or dense forms in 64 bits."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as bo
from tests.test_gpu_blocks import BF, _lib, bf, check_rows, f64, i32, rope_inputs, tokens, within  # noqa: F401

pytestmark = pytest.mark.gpu

svg = pytest.importorskip("sparse_attention_long_svg_b200")


# ----------------------------------------------------------------------- selection
@pytest.mark.parametrize("Nq", [3, 70])
@pytest.mark.parametrize("nblk,topk", [(100, 9), (400, 60), (1100, 12)])
def test_selection_of_scores_beyond_fp32(Nq, nblk, topk):
    """Finite queries and means whose products overflow: the list is still the one of exact scores, and whole."""
    D, Nk = 64, nblk * 64
    q = bf(200, 8, Nq, D)
    mean = torch.randn(4, nblk, D, generator=torch.Generator().manual_seed(201)).cuda()
    q[0:2, :, 0] = 1e20                              # every score overflows, to either side
    mean[0, :, 0] *= 1e20
    q[2:4, :, 5] = 1e20                              # a few blocks do
    mean[1, :, 5] = 0
    mean[1, 3:7, 5] = torch.tensor([2e20, 1e20, -1e20, 3e20], device="cuda")
    q[4, ::2, 9] = 1e30                              # some queries, by norm alone
    q[5, 1::2, 9] = -1e30
    mean[2, :, 9] *= 1e-3
    q[6, 1, 3] = float("inf")                        # a query with an infinity, one with a NaN
    q[7, 2, 3] = float("nan")
    sel = torch.full((4, Nq, topk), -7, dtype=torch.int32, device="cuda")
    svg.block_select(q, mean, 64, topk, Nk, 1, 1, True, sel=sel)
    want = bo.select_blocks(f64(q), f64(mean), 64, topk, 1, 1, True, [Nk] * 4)
    assert np.array_equal(sel.cpu().numpy(), want), np.argwhere(sel.cpu().numpy() != want)[:5]
