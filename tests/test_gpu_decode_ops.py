"""The decode step's operators on the GPU against their plain definitions in
64 bits.  Tolerances are worked out from the number formats:

* cache and 4-bit quantisers: equal, code by code (the definition fixes every
  fp32 rounding).
* attention: with A = sum p |v| and m = the largest sum |q k| scale of the row,
  a score is off by at most m (2^-22 for fp32 q in two fp16 terms + 2^-18 for
  sums of 2 x 128 products on the tensor core, whose additions may truncate)
  + 2^-21 (|log2 vs|, |score| rounded in fp32 and ex2), a weight by twice that
  (its own score and the normaliser) + 2^-12 (bf16 q: fp16 weights) or 2^-22,
  the sums over at most 4096 tokens in sequence by 256 steps of 2^-23 = 2^-15;
  the output rounding adds half a step of its type.  Where A is far below the
  row's largest value (that token's code is 0 in this column) one more term
  counts: fp16 holds a weight p vs below its normal numbers to 2^-25, with the
  row's largest p vs at 2^7 or more, so each token adds |code| vs* 2^-32 at
  most, vs* the value scale of the token with the largest p vs (the row sum
  is at least that token's weight).
* 4-bit products: sums of K products of exact factors (fp32 x: three bf16
  terms, 2^-24) in K / 16 steps that may truncate, then K / group scaled sums:
  (K / 16 + K / group + 8) 2^-23 of sum |x w|, plus half a step of the output.
* log probabilities: sums of V positive terms, at most V / 4096 + 32 in
  sequence per thread and join, each term off by 2^-21 + |x - m| 2^-23: its
  logarithm by that; the difference x - m and the two subtractions by 2^-23
  of their size.
"""

import numpy as np
import pytest
import torch

import decode_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def bl():
    import ternary_weight_linear_token_b200 as bl
    return bl


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def i32(a):
    return dev(np.asarray(a, dtype=np.int32))


def table_of(rng, lens, P, spare=2):
    """Pages in random order: (table [B, W], number of pages)."""
    held = [-(-n // P) for n in lens]
    order = rng.permutation(sum(held) + spare)
    table = np.full((len(lens), max(max(held), 1)), -7, dtype=np.int32)  # unused entries are not read
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = order[at:at + h]
        at += h
    return table, len(order)


def offsets_of(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


def filled(rng, pages, H, P, D, spread=1.0):
    """A cache whose pages differ in size: (k codes, k scales, v codes, v scales)."""
    out = []
    for _ in range(2):
        c = rng.integers(-127, 128, (pages, H, P, D)).astype(np.int8)
        s = (0.02 * np.exp(spread * rng.standard_normal((pages, H)))).astype(np.float32)
        out += [c, s]
    return out


def cache_of(bl, parts):
    kc, ks, vc, vs = (dev(a) for a in parts)
    return bl.KVCache.from_tensors(kc, vc, ks, vs)


# ---------------------------------------------------------------- append
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,P,D,lens,new", [
    (5, 64, 128, [1, 64, 65, 700], [1, 1, 1, 1]),
    (1, 16, 64, [3, 16, 33], [3, 16, 20]),
    (2, 128, 64, [300, 1, 129, 40], [300, 0, 2, 17]),
    (3, 32, 128, [97, 31], [66, 31]),
    (8, 128, 128, [513], [400]),
])
def test_append(bl, dtype, H, P, D, lens, new):
    rng = np.random.default_rng(len(lens) * P + D + H)
    table, pages = table_of(rng, lens, P)
    parts = filled(rng, pages, H, P, D)
    T = sum(new)
    # keys and values are columns of a wider row; sizes from row to row by factors of up to 100
    wide = rng.standard_normal((T, 2 * H + 1, D)) * np.exp(2 * rng.standard_normal((T, 2 * H + 1, 1)))
    x = dev(wide.astype(np.float32)).to(dtype)
    if T > 2:
        x[1] = 0
    cache = cache_of(bl, parts)
    want = [a.copy() for a in parts]
    ref.append(want[0], want[1], x[:, :H].float().cpu().numpy(), table, lens, new)
    ref.append(want[2], want[3], x[:, H:2 * H].float().cpu().numpy(), table, lens, new)
    one = all(t == 1 for t in new)
    for again in range(2):  # the same rows once more change nothing
        bl.bitnet_kv_append(cache, x[:, :H], x[:, H:2 * H], i32(table), i32(lens),
                            offsets=None if one else i32(offsets_of(new)),
                            max_new=None if again else max(new))
        for got, w in zip((cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales), want):
            assert np.array_equal(got.cpu().numpy(), w)
    assert bl.bitnet_get_device_status() == bl.OK


def test_append_sizes_at_the_edge(bl):
    """Zeros, values below the smallest scale, the largest finite ones, exact halves."""
    H, P, D = 1, 16, 64
    x = np.zeros((5, H, D), dtype=np.float32)
    x[1] = 1e-30
    x[2] = np.finfo(np.float32).max
    x[3, 0, :5] = [127, 0.5, -1.5, 2.5, -126.5]
    x[4] = 127 * 2.0 ** -60
    lens, new = [1] * 5, [1] * 5
    table = np.arange(5, dtype=np.int32)[:, None]
    parts = [np.full((5, H, P, D), 9, np.int8), np.full((5, H), 3.0, np.float32)] * 2
    want = [a.copy() for a in parts]
    for i in (0, 2):
        ref.append(want[i], want[i + 1], x, table, lens, new)
    cache = cache_of(bl, parts)
    bl.bitnet_kv_append(cache, dev(x), dev(x), i32(table), i32(lens))
    assert np.array_equal(cache.k_codes.cpu().numpy(), want[0])
    assert np.array_equal(cache.v_scales.cpu().numpy(), want[3])
    assert cache.k_codes[3, 0, 0, :5].tolist() == [127, 1, -2, 3, -127]
    assert cache.k_scales[:2].abs().sum() == 0 and cache.k_scales[4, 0] == 2.0 ** -60


def test_append_leaves_alone_what_is_not_there(bl):
    """Lengths, offsets and pages that do not exist: nothing is written for them, the others are, and the
    status word says so."""
    rng = np.random.default_rng(3)
    H, P, D = 2, 16, 64
    parts = filled(rng, 6, H, P, D)
    x = rng.standard_normal((6, H, D)).astype(np.float32)
    lens = [1, 16 * 2 + 1, 5, 1, 1, 0]        # 1: above the table; 5: below its new rows
    table = np.array([[0, 9], [1, 2], [6, 0], [-1, 0], [3, 0], [4, 0]], dtype=np.int32)
    cache = cache_of(bl, parts)
    bl.bitnet_kv_append(cache, dev(x), dev(x), i32(table), i32(lens))
    assert bl.bitnet_get_device_status() == bl.ERR_RANGE
    assert bl.bitnet_get_device_status() == bl.OK
    want = [a.copy() for a in parts]
    for i in (0, 2):
        for b in (0, 4):
            ref.append(want[i], want[i + 1], x[b:b + 1], table[b:b + 1], [lens[b]], [1])
    for got, w in zip((cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales), want):
        assert np.array_equal(got.cpu().numpy(), w)
    # offsets outside the rows
    for offs in ([0, 7], [-1, 3], [4, 2]):
        cache = cache_of(bl, parts)
        bl.bitnet_kv_append(cache, dev(x), dev(x), i32(table[:1]), i32([9]), offsets=i32(offs))
        assert bl.bitnet_get_device_status() == bl.ERR_RANGE
        assert np.array_equal(cache.k_codes.cpu().numpy(), parts[0])


# ---------------------------------------------------------------- attention
def check_attention(q, o, parts, table, lens, new, scale=None, window=0):
    want, size, mass, floor = ref.attention(q.float().cpu().numpy(), *parts, table, lens, new, scale, window)
    two = q.dtype == torch.float32
    score = mass * (2.0 ** -18 + (2.0 ** -22 if two else 0)) + 2.0 ** -21 * (64 + mass)
    rel = 2 * score + (2.0 ** -22 if two else 2.0 ** -12) + 2.0 ** -15
    tol = rel * size + HALF[q.dtype] * np.abs(want) + 2.0 ** -32 * floor
    err = np.abs(o.float().cpu().numpy().astype(np.float64) - want)
    assert not np.isnan(err).any()
    bad = err > tol
    assert not bad.any(), f"{bad.sum()} of {bad.size}, worst {np.max(err / np.maximum(tol, 1e-300)):.3g} of the tolerance"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("Hq,H,P,D,lens,new,window", [
    (20, 5, 64, 128, [1], [1], 0),
    (20, 5, 64, 128, [700], [1], 0),
    (4, 1, 16, 64, [1, 15, 16, 17, 33, 200], [1] * 6, 0),
    (7, 1, 32, 128, [129, 0, 40], [1, 1, 1], 0),          # an empty sequence
    (8, 8, 128, 64, [500, 3], [1, 1], 0),
    (16, 2, 16, 128, [300, 37], [1, 1], 33),
    (3, 3, 64, 64, [90, 5], [1, 1], 1),                    # sees itself only
    (8, 4, 16, 64, [50, 6, 200], [5, 6, 3], 0),
    (12, 2, 32, 128, [70, 100], [9, 0], 20),
    (10, 5, 128, 128, [260, 131], [37, 131], 0),
    (24, 1, 64, 128, [333], [40], 100),
    (6, 2, 16, 64, [2500], [2], 0),
    (4, 1, 64, 128, [150, 40], [200, 3], 0),               # more rows than tokens: zeros before the first
])
def test_attention(bl, dtype, Hq, H, P, D, lens, new, window):
    rng = np.random.default_rng(Hq * 1000 + P + D + sum(lens))
    table, pages = table_of(rng, lens, P)
    parts = filled(rng, pages, H, P, D)
    q = dev(rng.standard_normal((sum(new), Hq, D)).astype(np.float32)).to(dtype)
    one = all(t == 1 for t in new)
    o = bl.bitnet_kv_attention(cache_of(bl, parts), q, i32(table), i32(lens),
                               offsets=None if one else i32(offsets_of(new)), max_new=max(new), window=window)
    check_attention(q, o, parts, table, lens, new, window=window)
    assert bl.bitnet_get_device_status() == bl.OK
    if not one:  # the hint sizes the launch, not the result
        for hint in (1, None):
            o2 = bl.bitnet_kv_attention(cache_of(bl, parts), q, i32(table), i32(lens),
                                        offsets=i32(offsets_of(new)), max_new=hint, window=window)
            check_attention(q, o2, parts, table, lens, new, window=window)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [1, 60])
def test_attention_values_of_all_sizes(bl, dtype, n):
    """Pages of zeros (keys, values), scales from 2^-59 to 1e5, queries from 1e-6 to 1e4, a large scale."""
    rng = np.random.default_rng(n)
    H, P, D, Hq = 2, 16, 64, 8
    lens, new = [150, 97], [n, 1]
    table, pages = table_of(rng, lens, P)
    parts = filled(rng, pages, H, P, D, spread=2.0)
    for c, s in (parts[:2], parts[2:]):
        s[table[0, 2]] = 0
        c[table[0, 2]] = 0
    parts[3][table[0, 3]] = 2.0 ** -59
    parts[3][table[1, 0]] = 1e5
    q = rng.standard_normal((sum(new), Hq, D)).astype(np.float32) * 0.2
    q[:, 1] *= 1e-6
    q[:, 2] *= 20
    q[:, 3] = 0
    q = dev(q).to(dtype)
    for scale in (None, 3.0, -0.5, 0.0):
        o = bl.bitnet_kv_attention(cache_of(bl, parts), q, i32(table), i32(lens), offsets=i32(offsets_of(new)),
                                   max_new=n, scale=scale)
        check_attention(q, o, parts, table, lens, new, scale=scale)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attention_all_pages_of_zeros(bl, dtype):
    cache = bl.KVCache(4, 32, 2, 64, device=DEV)
    q = torch.randn(3, 4, 64, device=DEV).to(dtype)
    o = bl.bitnet_kv_attention(cache, q, i32([[0, 1], [2, 3], [1, 0]]), i32([33, 64, 0]))
    assert torch.equal(o, torch.zeros_like(q))


@pytest.mark.parametrize("new", [[1, 1, 1], [40, 1, 25]])
def test_attention_what_is_masked_does_not_count(bl, new):
    """Codes behind the last position and scales of pages that no row sees change nothing, NaN among them."""
    rng = np.random.default_rng(8)
    H, P, D, Hq, window = 1, 16, 128, 4, 40
    lens = [100, 45, 37]
    table, pages = table_of(rng, lens, P)
    parts = filled(rng, pages, H, P, D)
    q = dev(rng.standard_normal((sum(new), Hq, D)).astype(np.float32)).to(torch.bfloat16)
    args = dict(offsets=i32(offsets_of(new)), max_new=max(new), window=window)
    first = bl.bitnet_kv_attention(cache_of(bl, parts), q, i32(table), i32(lens), **args)
    other = [a.copy() for a in parts]
    for i in (0, 2):
        for b, n in enumerate(lens):
            other[i][table[b, (n - 1) // P], :, (n - 1) % P + 1:] = 127
    used = set()
    for b, (n, t) in enumerate(zip(lens, new)):
        used |= set(table[b, max(0, n - t - window + 1) // P: (n - 1) // P + 1].tolist())
    for p in set(range(pages)) - used:
        other[1][p] = np.nan
        other[3][p] = np.inf
    again = bl.bitnet_kv_attention(cache_of(bl, other), q, i32(table), i32(lens), **args)
    assert torch.equal(first, again)


@pytest.mark.parametrize("Hq,H,P,D,lens,new,window,hint", [
    (2, 1, 64, 128, [700, 10], [700, 4], 0, 130),          # more row blocks than the hint tells of
    (4, 2, 16, 64, [900, 300], [600, 290], 150, 70),
    (3, 1, 32, 64, [1300], [500], 0, 500),                 # a long prefix
    (5, 1, 128, 128, [400, 0, 1], [90, 0, 1], 1, 90),
])
def test_attention_of_long_prompts(bl, Hq, H, P, D, lens, new, window, hint):
    rng = np.random.default_rng(Hq + P + D + sum(lens))
    table, pages = table_of(rng, lens, P)
    parts = filled(rng, pages, H, P, D)
    q = dev(rng.standard_normal((sum(new), Hq, D)).astype(np.float32)).bfloat16()
    for most in (hint, max(new)):
        o = bl.bitnet_kv_attention(cache_of(bl, parts), q, i32(table), i32(lens), offsets=i32(offsets_of(new)),
                                   max_new=most, window=window)
        check_attention(q, o, parts, table, lens, new, window=window)
    assert bl.bitnet_get_device_status() == bl.OK


def test_attention_nan_query_stays_in_its_row(bl):
    rng = np.random.default_rng(9)
    lens, new = [70, 200], [3, 20]
    table, pages = table_of(rng, lens, 16)
    parts = filled(rng, pages, 1, 16, 64)
    q = rng.standard_normal((23, 4, 64)).astype(np.float32)
    clean = bl.bitnet_kv_attention(cache_of(bl, parts), dev(q).bfloat16(), i32(table), i32(lens),
                                   offsets=i32(offsets_of(new)), max_new=20)
    q[1, 2, 5] = np.nan
    q[9, 0, 63] = np.nan
    o = bl.bitnet_kv_attention(cache_of(bl, parts), dev(q).bfloat16(), i32(table), i32(lens),
                               offsets=i32(offsets_of(new)), max_new=20)
    assert o[1, 2].isnan().all() and o[9, 0].isnan().all()
    o[1, 2], o[9, 0] = clean[1, 2], clean[9, 0]
    assert torch.equal(o, clean)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("new", [[1, 1, 1, 1], [30, 1, 2, 1]])
def test_attention_of_what_is_not_there(bl, dtype, new):
    """A page number that does not exist is not followed (its tokens are not seen); a sequence whose length
    the table cannot hold keeps its rows, as do rows of no sequence; both are recorded."""
    rng = np.random.default_rng(4)
    H, P, D, Hq = 2, 16, 64, 4
    lens = [48, 30, 49, 20]
    parts = filled(rng, 8, H, P, D)
    table = np.array([[0, 1, 2], [3, 4, 0], [0, 1, 2], [6, 7, 0]], dtype=np.int32)
    T = sum(new) + 3
    q = dev(rng.standard_normal((T, Hq, D)).astype(np.float32)).to(dtype)
    o = torch.full_like(q, 7.0)
    bad = table.copy()
    bad[0, 1] = 8
    bl.bitnet_kv_attention(cache_of(bl, parts), q, i32(bad), i32(lens), offsets=i32(offsets_of(new)),
                           max_new=max(new), O=o)
    assert bl.bitnet_get_device_status() == bl.ERR_RANGE
    r = offsets_of(new)
    assert (o[r[2]:r[3]] == 7).all() and (o[r[4]:] == 7).all()
    # the others are as they should be (sequence 0 without its middle page: the same as a shorter one
    # where that page is skipped, for its last row)
    sub = np.array([[0, 2, 0]], dtype=np.int32)
    check_attention(q[r[1] - 1:r[1]], o[r[1] - 1:r[1]], parts, sub, [32], [1])
    for b in (1, 3):
        check_attention(q[r[b]:r[b + 1]], o[r[b]:r[b + 1]], parts, table[b:b + 1], [lens[b]], [new[b]])


def test_attention_long_cache_offsets(bl):
    """Codes past 2^31 bytes: pages at the end of a cache of more than 2 GiB."""
    H, P, D, Hq = 5, 128, 128, 20
    pages = (1 << 31) // (H * P * D) + 40
    kc = torch.zeros((pages, H, P, D), dtype=torch.int8, device=DEV)
    vc = torch.zeros((pages, H, P, D), dtype=torch.int8, device=DEV)
    ks = torch.zeros((pages, H), device=DEV)
    vs = torch.zeros((pages, H), device=DEV)
    cache = bl.KVCache.from_tensors(kc, vc, ks, vs)
    rng = np.random.default_rng(0)
    lens, new = [300], [300]
    table = np.array([[pages - 1, pages - 30, pages - 2]], dtype=np.int32)
    x = dev(rng.standard_normal((300, 2 * H, D)).astype(np.float32)).bfloat16()
    bl.bitnet_kv_append(cache, x[:, :H], x[:, H:], i32(table), i32(lens), offsets=i32([0, 300]))
    parts = [a[table[0].tolist()].cpu().numpy() for a in (kc, ks, vc, vs)]
    want = [np.zeros_like(a) for a in parts]
    here = np.array([[0, 1, 2]])
    ref.append(want[0], want[1], x[:, :H].float().cpu().numpy(), here, lens, new)
    ref.append(want[2], want[3], x[:, H:].float().cpu().numpy(), here, lens, new)
    for a, b in zip(parts, want):
        assert np.array_equal(a, b)
    q = dev(rng.standard_normal((300, Hq, D)).astype(np.float32)).bfloat16()
    o = bl.bitnet_kv_attention(cache, q, i32(table), i32(lens), offsets=i32([0, 300]))
    check_attention(q, o, parts, here, lens, new)
    o1 = bl.bitnet_kv_attention(cache, q[-1:], i32(table), i32(lens))
    check_attention(q[-1:], o1, parts, here, lens, [1])


# ---------------------------------------------------------------- 4-bit weights
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,K,group", [(1, 32, 32), (3, 64, 64), (17, 384, 128), (5, 96, 32), (130, 2560, 128)])
def test_quantize_w4(bl, dtype, N, K, group):
    rng = np.random.default_rng(N + K)
    w = rng.standard_normal((N, K)).astype(np.float32) * np.exp(rng.standard_normal((N, 1)) * 3).astype(np.float32)
    w[0, :group] = 0
    if N > 1:
        w[1, :group] = 1e-30
        w[1, :7] = [0, 0, 0, 0, 0, 0, 0]
    if N > 2:  # exact halves at scale 1
        w[2, :8] = [7, 0.5, -0.5, 1.5, -6.5, 6.5, 2.5, -7]
        w[2, 8:group] = 0
    W = dev(w).to(dtype)
    packed, scales = bl.bitnet_quantize_weights_w4(W, group)
    codes, s = ref.quantize_w4(W.float().cpu().numpy(), group)
    assert np.array_equal(scales.float().cpu().numpy(), s)
    assert np.array_equal(packed.cpu().numpy(), ref.pack_w4(codes))


def check_w4(x, y, codes, s, group):
    w = codes.reshape(*s.shape, group) * s.astype(np.float64)[..., None]
    w = w.reshape(codes.shape)
    xd = x.float().cpu().numpy().astype(np.float64)
    want, size = xd @ w.T, np.abs(xd) @ np.abs(w).T
    K = codes.shape[1]
    steps = (K / 16 * (3 if x.dtype == torch.float32 else 1) + K / group + 8) * 2.0 ** -23
    tol = steps * size + HALF[y.dtype] * np.abs(want)
    err = np.abs(y.float().cpu().numpy().astype(np.float64) - want)
    assert not (err > tol).any() and not np.isnan(err).any(), np.max(err / np.maximum(tol, 1e-300))


@pytest.mark.parametrize("x_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K,group", [
    (1, 1, 32, 32), (1, 16, 128, 128), (1, 2560, 2560, 128), (1, 515, 96, 32), (2, 33, 192, 64),
    (7, 100, 640, 128), (8, 31, 256, 64), (9, 64, 1280, 64), (16, 17, 512, 128), (17, 40, 160, 32),
    (23, 200, 6912, 64), (33, 48, 384, 128), (70, 50, 256, 32), (129, 17, 128, 128), (4, 4000, 3456, 128),
])
def test_w4_matmul(bl, x_dtype, M, N, K, group):
    rng = np.random.default_rng(M * N + K)
    codes = rng.integers(-8, 8, (N, K))
    s = torch.from_numpy((0.01 * np.exp(rng.standard_normal((N, K // group)))).astype(np.float32)).bfloat16()
    x = dev(rng.standard_normal((M, K)).astype(np.float32) * np.exp(rng.standard_normal((M, 1))).astype(np.float32))
    x = x.to(x_dtype)
    packed = dev(ref.pack_w4(codes))
    for out in (torch.bfloat16, torch.float32):
        y = bl.bitnet_w4a16_matmul(x, packed, s.to(DEV), out_dtype=out, weights_static=out == torch.float32)
        assert y.shape == (M, N) and y.dtype == out
        check_w4(x, y, codes, s.float().numpy(), group)


@pytest.mark.parametrize("x_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M", [1, 8, 9])
def test_w4_matmul_outliers(bl, x_dtype, M):
    """Large activations on codes of 0, single ones and a group of them under a scale that is not 0, add
    nothing: the tolerance goes by sum |x w|."""
    rng = np.random.default_rng(M)
    N, K, group = 40, 1280, 128
    codes = rng.integers(-8, 8, (N, K))
    s = np.full((N, K // group), 0.25, dtype=np.float32)
    codes[:, [3 * group + 5, 9 * group + 64]] = 0
    codes[:, 4 * group:5 * group] = 0
    for size in (1e3, 1e4, 1e5, 1e6, 3e38):
        x = rng.standard_normal((M, K)).astype(np.float32)
        x[:, 3 * group + 5] = size
        x[:, 9 * group + 64] = -size
        x[:, 4 * group:5 * group] *= size / 8
        x = dev(x).to(x_dtype)
        y = bl.bitnet_w4a16_matmul(x, dev(ref.pack_w4(codes)), dev(s).bfloat16(), out_dtype=torch.float32)
        check_w4(x, y, codes, s, group)


def test_w4_matmul_rows_are_their_own(bl):
    """A NaN in one token or an infinity in one scale stays in its row or column; a scale of 0 is 0."""
    rng = np.random.default_rng(5)
    M, N, K, group = 11, 40, 256, 64
    codes = rng.integers(-8, 8, (N, K))
    s = np.full((N, K // group), 0.5, dtype=np.float32)
    s[7] = 0
    s[20, 1] = np.inf
    x = rng.standard_normal((M, K)).astype(np.float32)
    x[4, 9] = np.nan
    for dtype in (torch.bfloat16, torch.float32):
        y = bl.bitnet_w4a16_matmul(dev(x).to(dtype), dev(ref.pack_w4(codes)), dev(s).bfloat16(),
                                   out_dtype=torch.float32)
        assert y[4].isnan().all()
        ok = [m for m in range(M) if m != 4]
        assert (y[ok][:, 7] == 0).all() and not y[ok][:, 20].isfinite().any()
        cols = [n for n in range(N) if n != 20]
        check_w4(dev(x[ok]).to(dtype), y[ok][:, cols], codes[cols], s[cols], group)


# ---------------------------------------------------------------- log probabilities
def check_logprobs(logits, tokens, top, got):
    x = logits.float().cpu().numpy().astype(np.float64)
    lp, h, ids, tl = ref.logprobs(x, tokens.cpu().numpy(), top)
    glp, gh, gids, gtl = (t.cpu().numpy() for t in got)
    assert glp.dtype == gh.dtype == gtl.dtype == np.float32 and gids.dtype == np.int64
    assert np.array_equal(gids, ids)
    steps = (x.shape[1] / 4096 + 32 + 40) * 2.0 ** -23

    def close(a, b, size):
        same = (a == b) | (np.isnan(a) & np.isnan(b))
        with np.errstate(invalid="ignore"):
            bad = ~same & ~(np.abs(a - b) <= steps + size * 2.0 ** -21)
        assert not bad.any(), (a[bad][:4], b[bad][:4])
    # a term's share of the sums is e^d <= 2^-20 where |d| > 14: |d| 2^-23 counts up to there
    close(glp, lp, np.abs(lp) + 14)
    close(gtl, tl, np.abs(tl) + 14)
    close(gh, h, np.abs(h) * 4 + 14)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,V,top", [(1, 1, 1), (1, 5, 5), (2, 31, 20), (3, 1000, 0), (1, 128256, 20), (5, 4097, 32),
                                     (160, 9001, 3), (2, 262147, 32), (700, 300, 7), (1, 32768, 1), (40, 50257, 10)])
def test_logprobs(bl, dtype, M, V, top):
    rng = np.random.default_rng(M + V)
    x = dev(3 * rng.standard_normal((M, V)).astype(np.float32)).to(dtype)
    tokens = dev(rng.integers(-1, V, M))
    check_logprobs(x, tokens, top, bl.bitnet_token_logprobs(x, tokens, top=top))
    assert bl.bitnet_get_device_status() == bl.OK


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_logprobs_of_difficult_rows(bl, dtype):
    """Ties over a whole row, rows of nothing but -infinity or the type's lowest value, rising rows, one
    thread's chunks holding all the large values, zeros of both signs, rows part of wider ones at odd
    addresses."""
    V, top = 70001, 32
    low = torch.finfo(dtype).min
    wide = torch.zeros(10, V + 12, device=DEV, dtype=dtype)
    x = wide[:, 5:5 + V]
    x[1] = -torch.inf
    x[2] = low
    x[3] = torch.linspace(-20, 20, V, device=DEV)
    x[4] = -torch.inf
    x[4, 12345] = 3.0
    x[5] = low
    x[5, 100::512 * 8] = 5.0
    x[6, ::2] = -0.0
    x[7] = torch.randn(V, device=DEV) * 100
    x[8] = torch.linspace(80, -80, V, device=DEV)
    x[9] = -torch.inf
    x[9, :7] = torch.tensor([1.0, 2, 2, 1, 0, -0.0, 1])
    tokens = dev(np.array([3, 7, 11, V - 1, 12345, 100, 0, 5, V - 1, 6]))
    check_logprobs(x, tokens, top, bl.bitnet_token_logprobs(x, tokens, top=top))
    # two CTAs to eight of them for one row
    for m in range(10):
        check_logprobs(x[m:m + 1], tokens[m:m + 1], top, bl.bitnet_token_logprobs(x[m:m + 1], tokens[m:m + 1], top=top))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_logprobs_of_values_far_apart(bl, dtype):
    """Finite values whose distance to the row's maximum is no fp32 number, before and after the maximum."""
    low = torch.finfo(dtype).min
    x = torch.randn(6, 9000, device=DEV).to(dtype)
    x[0, 7], x[0, 8000] = 2e32, low
    x[1], x[1, 8999] = low, 3e38
    x[2], x[2, ::3] = -3e38, 3e38
    x[3], x[3, 5] = low, 1e31
    x[4, ::7] = low          # an ordinary row, some of it masked by the lowest value
    x[5], x[5, 1] = 1e38, low
    tokens = dev(np.array([7, 0, 1, 5, 3, 1]))
    lp, h, ids, tl = ref.logprobs(x.double().cpu().numpy(), tokens.cpu().numpy(), 5)
    with np.errstate(over="ignore"):  # below fp32's lowest number: rounded to -infinity
        lp, tl = lp.astype(np.float32), tl.astype(np.float32)
    steps = (9000 / 4096 + 32 + 40) * 2.0 ** -23  # as in check_logprobs
    for rows in [slice(0, 6)] + [slice(m, m + 1) for m in range(6)]:
        glp, gh, gids, gtl = (t.cpu().numpy() for t in bl.bitnet_token_logprobs(x[rows], tokens[rows], top=5))
        assert np.array_equal(gids, ids[rows])
        for got, want in ((glp, lp[rows]), (gtl, tl[rows])):
            assert np.array_equal(got == -np.inf, want == -np.inf)
            fine = want != -np.inf
            assert (np.abs(got[fine] - want[fine]) <= steps + (np.abs(want[fine]) + 14) * 2.0 ** -21).all()
        assert (np.abs(gh - h[rows]) <= steps + (np.abs(h[rows]) * 4 + 14) * 2.0 ** -21).all()


def test_logprobs_nan_and_tokens_that_are_not_there(bl):
    x = torch.randn(4, 5000, device=DEV)
    x[1, 77] = torch.nan
    x[2, 4999] = torch.inf
    lp, h, ids, tl = bl.bitnet_token_logprobs(x, dev(np.array([5000, 3, 4, -5])), top=2)
    assert bl.bitnet_get_device_status() == bl.ERR_RANGE
    assert lp[:3].isnan().all() and lp[3] == 0
    assert h.isnan().tolist() == [False, True, True, False]
    assert tl.isnan().any(1).tolist() == [False, True, True, False]
    assert ((ids >= 0) & (ids < 5000)).all()
