"""The binding of a drafting step's operators on the CPU: what is refused before the library is called."""
import pytest
import torch

import tensor_core_matrix_amd as tcm


def test_a_tree_without_words_is_not_a_chain():
    """A tree of no words has no address, which would stand for a chain."""
    q, kc = torch.zeros((6, 8, 64), dtype=torch.bfloat16), torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    for words, nodes in ((0, 3), (0, 1), (1, 65), (2, 129)):
        with pytest.raises(ValueError, match="tree"):
            tcm.paged_tree_attention(q, kc, kc, i(2, 2), i(2), i(3), nodes,
                                     tree=torch.zeros((6, words), dtype=torch.int64))
    # no tokens, no words needed; and what fits goes on to the next check (the tensors are not on a GPU)
    for words, nodes in ((0, 0), (1, 64), (2, 65)):
        with pytest.raises(ValueError, match="GPU"):
            tcm.paged_tree_attention(q, kc, kc, i(2, 2), i(2), i(3), nodes,
                                     tree=torch.zeros((6, words), dtype=torch.int64))
