"""A workspace whose bytes are not there (a view of stride 0) is refused by the binding."""

import pytest
import torch

from head_latent_attention_absorb_b200 import api


@pytest.mark.parametrize("workspace", [torch.zeros(1, dtype=torch.uint8).expand(1 << 24), torch.zeros(1 << 12, dtype=torch.uint8)[::2]])
def test_a_workspace_with_gaps_is_refused(workspace):
    q, qp = torch.zeros((1, 4, 64)), torch.zeros((1, 4, 16))
    c4, sc, kr = torch.zeros((1, 8, 32), dtype=torch.uint8), torch.zeros((1, 8, 4), dtype=torch.uint8), torch.zeros((1, 8, 16))
    with pytest.raises(ValueError, match="workspace"):
        api.mla_decode_absorb_fp4kv((4, 64, 16, 32, 32), q, qp, c4, sc, kr, torch.full((1,), 8, dtype=torch.int32), 0.1, workspace=workspace)
