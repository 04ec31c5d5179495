"""Refusals of the MXFP4 wrappers that need no device."""
import pytest
import torch

import fp4_routed_expert_amd as moe


def test_glu_weights_need_both_projections():
    """Without the up projection there is no SwiGLU form (and no silent plain one)."""
    q, s = torch.zeros(32, 64, dtype=torch.uint8), torch.zeros(32, 4, dtype=torch.uint8)
    for uq, us in ((None, None), (None, s), (q, None)):
        with pytest.raises(ValueError, match="up projection"):
            moe.mxfp4_prepack_glu(q, s, uq, us)
