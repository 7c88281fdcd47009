"""The decode step's operators where their numbers and sizes end: rows past
2^31 values, the largest queries.  Tolerances as in test_gpu_decode_ops."""

import numpy as np
import pytest
import torch

from test_gpu_decode_ops import DEV, cache_of, check_attention, dev, filled, i32, offsets_of, table_of

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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [1, 60])
def test_attention_of_the_largest_queries(bl, dtype, n):
    """Queries up to 0.99 * 2^128, with keys and a scale that make ordinary scores of them."""
    rng = np.random.default_rng(n)
    H, P, D, Hq = 2, 16, 64, 8
    lens, new = [150, 97], [n, 1]
    table, pages = table_of(rng, lens, P)
    parts = filled(rng, pages, H, P, D)
    parts[1] *= np.float32(2.0 ** -40)
    q = np.clip(rng.standard_normal((sum(new), Hq, D)), -3.9, 3.9) / 4
    q[:, :, 0] = 0.99
    for e in (125, 126, 127, 128):
        x = dev(np.ldexp(q, e).astype(np.float32)).to(dtype)
        assert x.isfinite().all()
        scale = 2.0 ** (40 - e)
        o = bl.bitnet_kv_attention(cache_of(bl, parts), x, i32(table), i32(lens), offsets=i32(offsets_of(new)),
                                   max_new=n, scale=scale)
        check_attention(x, o, parts, table, lens, new, scale=scale)
