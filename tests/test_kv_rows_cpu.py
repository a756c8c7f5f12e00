"""Which layouts of output rows kv8_read takes (include/kvcache.h), by its checks
alone: without sequences a call is checked and does nothing."""
import itertools

import pytest

from dit_quantization_amd import int4, kvcache
from dit_quantization_amd import nvfp4 as nv

A = 0x10000


def status(tokens, heads, dim, token_stride, head_stride):
    t = dict(codes=A, scales=A, code_stride=4 * heads * dim, scale_stride=4 * heads, rows=A, token_stride=token_stride, head_stride=head_stride,
             dim=dim)
    p = dict(page_table=A, cu=A, starts=None, seqs=0, table_width=3, tokens=tokens, heads=heads, pages=9, page_size=4)
    return kvcache.lib().kv8_read(kvcache.Tensor(**t), kvcache.Tensor(**t), kvcache.Places(**p), int4.BF16, int4.I8, None)


def test_rows_behind_one_another_are_taken():
    """The last row of a token may end where the next token starts, also where rows have room between them."""
    assert status(2, 2, 16, 40, 24) == nv.OK          # [0, 16), [24, 40), [40, 56), [64, 80)
    assert status(5, 3, 32, 112, 40) == nv.OK
    assert status(5, 3, 32, 104, 40) == nv.ERR_SHAPE  # 8 elements of the next token's first row
    assert status(3, 5, 32, 40, 112) == nv.OK         # heads before tokens
    assert status(3, 5, 32, 40, 104) == nv.ERR_SHAPE


@pytest.mark.parametrize("dim", [16, 32])
def test_no_overlapping_rows_are_taken(dim):
    for tokens, heads in itertools.product((1, 2, 3, 5), (1, 2, 3, 4)):
        for s, h in itertools.product(range(0, 168, 8), range(0, 168, 8)):
            starts = sorted(t * s + i * h for t in range(tokens) for i in range(heads))
            apart = all(b - a >= dim for a, b in zip(starts, starts[1:]))
            spans = s >= (heads - 1) * h + dim or h >= (tokens - 1) * s + dim or tokens == 1 or heads == 1
            assert status(tokens, heads, dim, s, h) == (nv.OK if apart and spans else nv.ERR_SHAPE), (tokens, heads, s, h)
