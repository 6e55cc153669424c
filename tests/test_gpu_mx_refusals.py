"""What the binding of the microscaled operators refuses on a GPU, before
anything is launched."""

import numpy as np
import pytest

from gpu_util import announce

pytestmark = pytest.mark.gpu


def test_a_closed_plan_is_not_no_plan():
    import butterfly_rotation_quantization_amd as brq
    import torch
    announce("closed plans")
    plan = brq.Plan(64, (2,) * 6, "hadamard", signs=np.ones(64, np.int8))
    x = torch.randn((4, 64), device="cuda")
    codes, scales = brq.mx_quantize(plan, x)
    cache, slots = brq.kv_cache(2, 1, 64, 16), torch.arange(4, device="cuda")
    kv = x.view(4, 1, 64)
    table, lens = torch.zeros((4, 1), dtype=torch.int32, device="cuda"), torch.ones(4, dtype=torch.int32, device="cuda")
    plan.close()
    for call in (lambda: brq.mx_quantize(plan, x), lambda: brq.mx_dequantize(plan, codes, scales),
                 lambda: brq.kv_append(plan, kv, kv, slots, cache, 16), lambda: brq.kv_read(plan, cache, slots, 64, 16),
                 lambda: brq.paged_attention(plan, kv, cache, table, lens, 16),
                 lambda: brq.rotate_quantize_pack(plan, None, x.t().contiguous(), 4, 4)):
        with pytest.raises(ValueError, match="closed"):
            call()
    assert not cache.any()
