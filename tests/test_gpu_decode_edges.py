"""The decode step's operators where their numbers and sizes end: rows past
2^31 values.  Tolerances as in test_gpu_decode_ops."""

import numpy as np
import pytest
import torch

from test_gpu_decode_ops import DEV, cache_of, check_attention, dev, filled, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bl():
    import ternary_weight_linear_token_b200 as bl
    return bl


# ---------------------------------------------------------------- attention
def test_attention_joined_rows_past_2_31_values(bl):
    """Two pieces joined by the second kernel, for the last of so many rows that their values pass 2^31;
    the rows before belong to no sequence."""
    H, P, D, T = 300, 128, 128, 56000
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of free device memory")
    assert T * H * D > 1 << 31
    rng = np.random.default_rng(1)
    parts = filled(rng, 2, H, P, D)
    table = np.array([[1, 0]], dtype=np.int32)
    Q = torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV)
    O = torch.empty_like(Q)
    Q[-1] = dev(rng.standard_normal((H, D)).astype(np.float32))
    O[[0, T // 2, T - 2]] = 7.0
    assert bl.bitnet_kv_attention_workspace_size(bl.KVCache(2, P, H, D), torch.bfloat16, T, H, 1, 2) >= 2 * 4 * T * H * D
    bl.bitnet_kv_attention(cache_of(bl, parts), Q, i32(table), i32([200]), offsets=i32([T - 1, T]), max_new=1, O=O)
    check_attention(Q[-1:], O[-1:], parts, table, [200], [1])
    assert (O[[0, T // 2, T - 2]] == 7).all() and bl.bitnet_get_device_status() == bl.OK
