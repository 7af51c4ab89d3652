"""What the embedding gradient asks for: parts of runs in float32, one for each 32 tokens and one more for
every second of them, next to what sorting takes.  No GPU."""

import pytest

import fsdp_sharded_optimizer_layout_amd as F


@pytest.mark.parametrize("tokens,vocab,dim", [(65536, 32000, 8192), (65536, 32000, 64),
                                              (131072, 32000, 1024)])
def test_workspace_is_three_halves_of_the_parts(tokens, vocab, dim):
    parts = tokens // 32
    need = F.embedding_grad_workspace_bytes(tokens, vocab, dim)
    sums = 4 * dim * (parts + parts // 2)
    assert sums < need <= sums + 8 * tokens + vocab + 4 * parts + 200
