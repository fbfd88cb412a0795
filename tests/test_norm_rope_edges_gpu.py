"""Norm, rotation and write at the ends of what the calls take."""

import pytest
import torch

import paged_kv_cache_111_gb300 as pkv
from latent_ref import angles

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
def test_errors_name_the_call(fp8):
    x = torch.zeros(2, 1, 64, dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros(1, 1, 2, 16, 64, dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    at = torch.arange(2, device="cuda")
    call = pkv.qk_norm_rope_kv_write_fp8 if fp8 else pkv.qk_norm_rope_kv_write
    with pytest.raises(pkv.PagedKVError, match="^pkv_qk_norm_rope_kv_write" + ("_fp8:" if fp8 else ":")):
        call(x, cache, x, x, x, None, None, 1e-6, angles(24, 4).cuda(), at, at, *((1.0, 1.0) if fp8 else ()))
