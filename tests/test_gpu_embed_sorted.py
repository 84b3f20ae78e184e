"""The sorted embedding gradient over several column blocks: partial sums, arrival counts and units of work lie a
block apart there.  Definitions and tolerances are those of test_gpu_train_ops.py."""

from __future__ import annotations

import pytest

from test_gpu_train_ops import check_embed_grad, torch  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("n,vocab,dim,kind,dtype,idt,ld,shift", [
    (5000, 600, 2051, "zipf", "bf16", "int64", 0, 0),   # three column blocks, the last of three columns
    (5000, 600, 2051, "zipf", "bf16", "int32", 5, 3),
    (3000, 300, 1030, "any", "fp32", "int32", 3, 1),    # three column blocks of two vectors a lane
    (3000, 7, 1100, "one", "fp32", "int64", 0, 0),      # one row: 94 chunks in three groups, in each column block
    (2100, 40, 4096, "zipf", "bf16", "int64", 8, 0),    # whole column blocks
    (1025, 2000, 513, "pad", "bf16", "int64", 0, 0)])   # nothing to add, in the second block's one column too
def test_sorted_embedding_gradient_of_several_column_blocks(torch, n, vocab, dim, kind, dtype, idt, ld, shift, first):
    check_embed_grad(torch, n, vocab, dim, kind, dtype, idt, first, ld, shift)
