"""The binding refuses a type that contradicts the tensor it is given (no GPU)."""
import pytest
import torch

import moe_expert_routing_sqrt_amd as M


def test_embedding_refuses_a_type_that_is_not_its_outputs():
    ids, table = torch.zeros(4, dtype=torch.int32), torch.zeros(9, 8)
    with pytest.raises(TypeError, match="out_dtype"):
        M.embedding(ids, table, out=torch.zeros(4, 8), out_dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="dtype"):
        M.embedding_backward(torch.zeros(4, 8), ids, 9, d_table=table, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):  # the tensor's own type is no contradiction, nor is none
        M.embedding_backward(torch.zeros(4, 8), ids, 9, d_table=table.bfloat16(), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        M.embedding_backward(torch.zeros(4, 8), ids, 9, d_table=table.bfloat16())
