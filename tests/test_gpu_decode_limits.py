"""The decode-step calls at their limits: sizes that take other paths than the
usual ones, calls from several streams and threads, and what they refuse."""
import pytest
import torch

import serving_moe_route_gb300 as moe
from serving_moe_route_gb300 import _binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("kv,step", [(B.MOE_KV_F32, 8), (B.MOE_KV_BF16, 8), (B.MOE_KV_E4M3, 16)])
def test_workspace_is_0_for_what_attention_refuses(kv, step):
    for dim in range(-1, 273):
        fits = 0 < dim <= 256 and dim % step == 0
        assert (B.moe_attn_workspace(kv, dim) > 0) == fits, dim
    assert moe.attn_workspace(torch.float8_e4m3fn, 72) == 0
