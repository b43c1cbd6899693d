"""Grouped products at the borders between their tiles, against 64 bits: lengths of the sum on either side of where tiles of
256 x 256 begin, routing in which one expert has most rows."""
import pytest
import torch

import bit_gathered_quantized_amd as bgq
from grouped_util import check, offsets_of, product
from test_grouped_use import FORMS, gen, operands

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


# 504 and more tiles of 256 x 256, 512 rows an expert and more
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("form,K", [("bf16", 632), ("bf16", 640), ("bf16", 1000), ("transposed", 248), ("transposed", 256),
                                    ("transposed", 520), ("mx", 32), ("mx", 256), ("mx", 544)])
@pytest.mark.parametrize("sizes,N", [([9001, 0, 6970], 2040), ([257, 14001, 1, 256], 2056)])
def test_many_rows_by_length(sizes, N, form, K, out):
    g = gen(N + K)
    args, kw, x, w = operands(form, g, sum(sizes), len(sizes), N, K)
    offsets = offsets_of(sizes)
    check(bgq.grouped_matmul(*args, offsets, out_dtype=out, **kw), *product(x, w, offsets), K)


# the variant is that of the average: few rows an expert but one with most of them, and the other way round
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("sizes,N,K", [
    ([1, 0, 900, 2] + [1] * 124, 328, 1056), ([2000] + [0, 1, 3] * 40, 264, 544), ([5, 8191, 0, 0], 520, 672),
    ([33] + [0] * 31, 1000, 1312), ([0] * 60 + [130, 1, 1, 1], 2056, 1024),
])
def test_one_expert_with_most_rows(sizes, N, K, form, out):
    g = gen(N + K)
    args, kw, x, w = operands(form, g, sum(sizes), len(sizes), N, K)
    offsets = offsets_of(sizes)
    check(bgq.grouped_matmul(*args, offsets, out_dtype=out, **kw), *product(x, w, offsets), K)
