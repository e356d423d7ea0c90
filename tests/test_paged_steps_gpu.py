"""A serving step on the paged FP8 cache where its parts meet: block tables, slots, the write and attention."""
import pytest
import torch

import bit_quantized_linear_quantizers_gb300 as qz

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_pages_whose_slots_do_not_fit_an_int():
    """Entries so large that page * page_size wraps are no pages: their slots are -1, not another page's."""
    for P in (16, 128):
        wrap = (1 << 32) // P                                 # times P: 0 in 32 bits
        top = ((1 << 31) - 1) // P                            # the last page whose slots fit
        table = i32([[3, wrap, -1, -1], [wrap // 2, -1, -1, -1], [top, -1, -1, -1]])
        got = qz.qz_block_tables(i32([P + 2, 1, P - 1]), i32([P, 1, 2]), table, i32([wrap, top, 5]), i32([0]), P, P + 4)
        slots = [-1] * P + [-1] + [top * P + P - 1, top * P, -1]
        assert got[0].tolist() == slots
