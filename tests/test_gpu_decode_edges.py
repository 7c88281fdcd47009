"""The decode step's operators where their numbers and sizes end: rows past
2^31 values, the largest queries and activations, value scales far apart or no
numbers, the low bits of fp32.  Tolerances as in test_gpu_decode_ops where none
is given."""

import numpy as np
import pytest
import torch

import decode_ref as ref
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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,new,P", [([150], [1], 16), ([150], [60], 16), ([5000], [1], 128),
                                        ([300] * 24, [1] * 24, 32), ([700], [200], 64)])
@pytest.mark.parametrize("large", [20, 40, 61, 100, 119])
def test_attention_value_scales_far_apart(bl, dtype, lens, new, P, large):
    """Pages of zeros, of values near 2^-59 and of huge ones side by side, in any order: the small ones count
    in the row sum as they should."""
    rng = np.random.default_rng(large + sum(lens))
    H, D, Hq = 2, 64, 8
    table, pages = table_of(rng, lens, P)
    parts = filled(rng, pages, H, P, D)
    for b in range(len(lens)):
        held = -(-lens[b] // P)
        kind = rng.integers(0, 4, held)
        kind[:3] = rng.permutation(3)
        for k, p in zip(kind, table[b, :held]):
            if k == 0:
                parts[2][p], parts[3][p] = 0, 0
            elif k == 1:
                parts[3][p] = 2.0 ** large
            elif k == 2:
                parts[3][p] = 2.0 ** -59
    q = dev(rng.standard_normal((sum(new), Hq, D)).astype(np.float32)).to(dtype)
    o = bl.bitnet_kv_attention(cache_of(bl, parts), q, i32(table), i32(lens), offsets=i32(offsets_of(new)),
                               max_new=max(new))
    check_attention(q, o, parts, table, lens, new)
    assert bl.bitnet_get_device_status() == bl.OK


@pytest.mark.parametrize("new", [[1, 1, 1], [40, 1, 25]])
def test_attention_scales_of_unseen_pages(bl, new):
    """Huge and tiny value scales of pages before every row's window change nothing."""
    rng = np.random.default_rng(8)
    H, P, D, Hq, window = 1, 16, 128, 4, 40
    lens = [100, 85, 77]
    table, pages = table_of(rng, lens, P)
    parts = filled(rng, pages, H, P, D)
    q = dev(rng.standard_normal((sum(new), Hq, D)).astype(np.float32))
    args = dict(offsets=i32(offsets_of(new)), max_new=max(new), window=window)
    used = set()
    for b, (n, t) in enumerate(zip(lens, new)):
        used |= set(table[b, max(0, n - t - window + 1) // P: (n - 1) // P + 1].tolist())
    unseen = sorted(set(range(pages)) - used)
    assert len(unseen) > 2
    other = parts[:3] + [parts[3].copy()]
    other[3][unseen[::2]], other[3][unseen[1::2]] = 2.0 ** 100, 2.0 ** -59
    for x in (q, q.bfloat16()):
        a, b = (bl.bitnet_kv_attention(cache_of(bl, p), x, i32(table), i32(lens), **args) for p in (parts, other))
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("new", [[3, 1, 4], [40, 1, 25]])
def test_attention_scales_that_are_no_numbers(bl, dtype, new):
    """A NaN or infinite scale of the last page: rows before that page, in the same tiles as rows that see
    it, stay as they were; with NaN the others are NaN."""
    rng = np.random.default_rng(8)
    H, P, D, Hq = 1, 16, 128, 4
    lens = [99, 45, 35]
    table, pages = table_of(rng, lens, P)
    parts = filled(rng, pages, H, P, D)
    q = dev(rng.standard_normal((sum(new), Hq, D)).astype(np.float32)).to(dtype)
    args = dict(offsets=i32(offsets_of(new)), max_new=max(new))
    first = bl.bitnet_kv_attention(cache_of(bl, parts), q, i32(table), i32(lens), **args)
    pos = np.concatenate([np.arange(n - t, n) for n, t in zip(lens, new)])
    edge = np.repeat([(n - 1) // P * P for n in lens], new)
    before = torch.from_numpy(pos < edge).to(DEV)
    assert before.any() and not before.all()
    for bad in (np.nan, np.inf):
        for i in (1, 3):
            other = [a.copy() for a in parts]
            for b, n in enumerate(lens):
                other[i][table[b, (n - 1) // P]] = bad
            o = bl.bitnet_kv_attention(cache_of(bl, other), q, i32(table), i32(lens), **args)
            assert torch.equal(o[before], first[before])
            if np.isnan(bad):
                assert o[~before].isnan().all()


@pytest.mark.parametrize("Hq,H,P,D,lens,new", [
    (8, 2, 16, 64, [20, 3], [1, 1]),
    (4, 1, 32, 128, [31], [5]),
    (3, 3, 128, 64, [9, 24, 2], [2, 7, 1]),
])
def test_attention_low_bits_of_fp32(bl, Hq, H, P, D, lens, new):
    """fp32 queries and weights keep 22 bits.  Each query has one element, so that a score is one product:
    |log2 score| <= 4 is off by 4 (2^-22 + 2^-23 + 2 * 2^-24) + 2^-22 and by two roundings of 2^-21 next to
    the maximum (up to 16), with ex2 below 2^-18.8; a weight by that times ln 2, twice (its own and the
    normaliser's), 2^-22 for its two halves, a sum of 32 by 2^-20: below 2^-17 in all.  Weights or queries of
    one half are off by more."""
    rng = np.random.default_rng(D + P)
    table, pages = table_of(rng, lens, P)
    parts = filled(rng, pages, H, P, D)
    parts[1][:], parts[3][:] = 2.0 ** -5, 1.0
    T = sum(new)
    q = np.zeros((T, Hq, D), dtype=np.float32)
    at = rng.integers(0, D, (T, Hq))
    size = rng.uniform(0.5, 1, (T, Hq)) * rng.choice([-1, 1], (T, Hq))
    np.put_along_axis(q, at[..., None], size[..., None].astype(np.float32), -1)
    args = (*parts, table, lens, new, 0.6)
    want, mass, score, _ = ref.attention(q, *args)
    assert score.max() * np.log2(np.e) <= 4
    o = bl.bitnet_kv_attention(cache_of(bl, parts), dev(q), i32(table), i32(lens), offsets=i32(offsets_of(new)),
                               max_new=max(new), scale=0.6)
    tol = 2.0 ** -17 * mass
    assert (np.abs(o.cpu().numpy() - want) <= tol).all()
    one_half = ref.attention(q.astype(np.float16).astype(np.float32), *args)[0]
    assert (np.abs(one_half - want) > tol).any()
    assert (np.abs(one_half_weights(q, *args) - want) > tol).any()


def one_half_weights(q, kc, ks, vc, vs, table, lens, new, scale):
    """What weights rounded once to fp16, their sum exact, would give."""
    o = np.zeros(q.shape)
    H, P = kc.shape[1:3]
    for b, (r0, t, n) in enumerate(ref.rows_of(lens, new)):
        k, v = (np.concatenate([c[p] * s[p][:, None, None].astype(np.float64) for p in table[b, :-(-n // P)]], 1)
                for c, s in ((kc, ks), (vc, vs)))
        for i in range(t):
            for h in range(q.shape[1]):
                g, seen = h // (q.shape[1] // H), n - t + i + 1
                s = scale * (k[g, :seen] @ q[r0 + i, h].astype(np.float64))
                w = np.exp(s - s.max()) * 128
                o[r0 + i, h] = w.astype(np.float16).astype(np.float64) @ v[g, :seen] / w.sum()
    return o


# ---------------------------------------------------------------- 4-bit weights
@pytest.mark.parametrize("M", [1, 4, 9, 23])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_w4_matmul_low_bits_of_fp32(bl, M, group):
    """fp32 activations keep 24 bits.  Rows of one code: its product's three terms add up with one rounding to
    24 bits, which may truncate: 2^-23 of it.  Rows of two codes that cancel but for the low bits: three
    roundings more, at the size of one product.  Two terms of 16 bits would be off by more."""
    rng = np.random.default_rng(M + group)
    N, K = 48, 384
    codes = np.zeros((N, K), dtype=np.int64)
    size = np.zeros(N)
    for n in range(N):
        a, b = rng.choice(K, 2, replace=False)
        codes[n, a] = c = rng.choice([-7, -5, -3, -1, 1, 2, 3, 5, 6, 7])
        if n % 2:
            codes[n, b] = -c
        size[n] = abs(c) * (4 if n % 2 else 1)
    x = (1 + rng.integers(0, 1 << 22, (M, K)) * 2.0 ** -22 + 2.0 ** -23).astype(np.float32)
    s = torch.ones(N, K // group, dtype=torch.bfloat16, device=DEV)
    y = bl.bitnet_w4a16_matmul(dev(x), dev(ref.pack_w4(codes)), s, out_dtype=torch.float32).cpu().numpy()
    want = x.astype(np.float64) @ codes.T
    tol = 2.0 ** -23 * 2 * size  # |x| < 2
    assert (np.abs(y - want) <= tol).all()
    high = (x.view(np.uint32) & 0xFFFFFF00).view(np.float32)
    assert (np.abs(high.astype(np.float64) @ codes.T - want) > tol).any()


@pytest.mark.parametrize("M", [1, 8, 9])
def test_w4_matmul_largest_activations(bl, M):
    """Finite activations up to the largest of their type: a row of one code each, exact but for one rounding.
    A group's sum of x * code is fp32 and comes before the scale: from 2^128 on it is infinite."""
    N, K, group = 14, 256, 64
    codes = np.zeros((N, K), dtype=np.int64)
    codes[np.arange(N), 17 * np.arange(N)] = [c for c in range(-7, 8) if c != 0]
    s = torch.full((N, K // group), 2.0 ** -10, dtype=torch.bfloat16, device=DEV)
    packed = dev(ref.pack_w4(codes))
    for dtype in (torch.float32, torch.bfloat16):
        for value in (torch.finfo(dtype).max, 3.39e38, 2.6e36, -torch.finfo(dtype).max):
            x = torch.full((M, K), value, device=DEV).to(dtype)
            y = bl.bitnet_w4a16_matmul(x, packed, s, out_dtype=torch.float32).double().cpu().numpy()
            want = x.double().cpu().numpy() @ codes.T * 2.0 ** -10
            fits = np.abs(want) < 2.0 ** 118
            assert (np.abs(y - want)[fits] <= 2.0 ** -23 * np.abs(want)[fits]).all() and fits.any()
            assert (y[~fits] == np.inf * np.sign(want[~fits])).all()
