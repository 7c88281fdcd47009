"""Refusals of the decode step's operators, without a GPU: bad arguments get
the documented status before the device would be touched."""

import ctypes as C

import pytest
import torch

A, B, D = 0x10000000, 0x20000000, 0x30000000
PAGES, LENS, OFFS, WS = 0x40000000, 0x50000000, 0x60000000, 0x70000000


@pytest.fixture(scope="module")
def tw():
    from __graft_entry__ import load_builder
    load_builder().build()
    import ternary_weight_linear_token_b200 as tw
    return tw


def cache(tw, kc=A, vc=B, ks=D, vs=D + 4096, pages=10, heads=5, P=64, dim=128):
    return tw.KVCacheStruct(kc, vc, ks, vs, pages, heads, P, dim)


def append(tw, K=A, kst=640, V=B, vst=640, dt=1, T=2, table=PAGES, W=4, lens=LENS, offs=None, n=2, new=1, **kw):
    c = cache(tw, **kw)
    return tw.lib.bitnet_kv_append(C.addressof(c), K, kst, V, vst, dt, T, table, W, lens, offs, n, new, None)


def attend(tw, Q=A, O=B, dt=1, T=2, q_heads=20, table=PAGES, W=4, lens=LENS, offs=None, n=2, new=1, scale=0.1,
           window=0, ws=WS, wsb=1 << 40, **kw):
    c = cache(tw, **kw)
    return tw.lib.bitnet_kv_attention(C.addressof(c), Q, O, dt, T, q_heads, table, W, lens, offs, n, new, scale, window,
                                      ws, wsb, None)


BAD_CACHES = [dict(kc=None), dict(vs=None), dict(pages=0), dict(heads=0), dict(heads=40000), dict(pages=1 << 31)]
BAD_SHAPES = [dict(P=48), dict(P=256), dict(dim=96), dict(dim=256)]
BAD_PLACES = [dict(kc=A + 8), dict(ks=D + 2)]


@pytest.mark.parametrize("call", [append, attend])
def test_cache_and_batch(tw, call):
    for bad in BAD_CACHES:
        assert call(tw, **bad) == tw.ERR_INVALID_ARG, bad
    for bad in BAD_SHAPES:
        assert call(tw, **bad) == tw.ERR_UNSUPPORTED_SHAPE, bad
    for bad in BAD_PLACES:
        assert call(tw, **bad) == tw.ERR_MISALIGNED, bad
    for bad in (dict(dt=2), dict(dt=3), dict(dt=9), dict(T=-1), dict(n=-1), dict(W=-1), dict(new=-1),
                dict(T=3), dict(W=1 << 30), dict(table=None), dict(lens=None)):
        assert call(tw, **bad) == tw.ERR_INVALID_ARG, bad
    assert call(tw, lens=LENS + 2) == tw.ERR_MISALIGNED
    assert call(tw, offs=OFFS + 1) == tw.ERR_MISALIGNED
    # empty calls succeed without touching the device
    assert call(tw, T=0, n=0) == tw.OK
    assert call(tw, T=0, n=3, offs=OFFS) == tw.OK


def test_no_cache(tw):
    assert tw.lib.bitnet_kv_append(None, A, 640, B, 640, 1, 2, PAGES, 4, LENS, None, 2, 1, None) == tw.ERR_INVALID_ARG
    assert tw.lib.bitnet_kv_attention_workspace_size(None, 1, 2, 20, 2, 1000, 1, 0) == 0


def test_append(tw):
    assert append(tw, K=None) == tw.ERR_INVALID_ARG
    assert append(tw, V=None) == tw.ERR_INVALID_ARG
    assert append(tw, kst=639) == tw.ERR_INVALID_ARG        # rows overlap
    assert append(tw, vst=-640) == tw.ERR_INVALID_ARG
    assert append(tw, kst=644) == tw.ERR_MISALIGNED         # rows not on 16 bytes
    assert append(tw, V=B + 8) == tw.ERR_MISALIGNED
    assert append(tw, T=1 << 30, n=1 << 30, offs=OFFS, new=1 << 30) == tw.ERR_UNSUPPORTED_SHAPE


def test_attention(tw):
    assert attend(tw, Q=None) == tw.ERR_INVALID_ARG
    assert attend(tw, O=None) == tw.ERR_INVALID_ARG
    assert attend(tw, q_heads=18) == tw.ERR_INVALID_ARG      # not a multiple of the key heads
    assert attend(tw, q_heads=0) == tw.ERR_INVALID_ARG
    assert attend(tw, q_heads=32770) == tw.ERR_UNSUPPORTED_SHAPE
    assert attend(tw, window=-1) == tw.ERR_INVALID_ARG
    assert attend(tw, scale=float("nan")) == tw.ERR_INVALID_ARG
    assert attend(tw, scale=float("inf")) == tw.ERR_INVALID_ARG
    assert attend(tw, Q=A + 8) == tw.ERR_MISALIGNED
    assert attend(tw, O=B + 4) == tw.ERR_MISALIGNED
    assert attend(tw, O=A + 256) == tw.ERR_INVALID_ARG     # on top of Q
    # a long cache for few rows is cut into pieces, which need a workspace
    size = tw.lib.bitnet_kv_attention_workspace_size
    c = cache(tw)
    need = size(C.addressof(c), 1, 2, 20, 2, 1000, 1, 0)
    assert need > 0 and need % 256 == 0
    assert attend(tw, W=1000, ws=None) == tw.ERR_WORKSPACE
    assert attend(tw, W=1000, wsb=need - 1) == tw.ERR_WORKSPACE
    assert attend(tw, W=1000, ws=WS + 16) == tw.ERR_MISALIGNED
    assert size(C.addressof(c), 1, 2, 20, 2, 1, 1, 0) == 0          # one page: one piece
    assert size(C.addressof(c), 1, 2, 18, 2, 1000, 1, 0) == 0       # refused arguments
    assert size(C.addressof(c), 1, 0, 20, 0, 1000, 1, 0) == 0


def test_attention_largest_windows(tw):
    """Windows past every position, the largest there are among them, cut a call as no window does."""
    c = cache(tw)
    size = tw.lib.bitnet_kv_attention_workspace_size
    for n in (1, 2, 8):
        none = size(C.addressof(c), 1, n, 20, n, 1000, 1, 0)
        assert none > 0
        for window in (64000, 1 << 30, (1 << 31) - 1, 1 << 31, 1 << 62, (1 << 63) - 1):
            assert size(C.addressof(c), 1, n, 20, n, 1000, 1, window) == none


def test_w4(tw):
    q = tw.lib.bitnet_quantize_weights_w4
    ok = dict(W=A, dt=0, N=4, K=256, g=128, P=B, s=D)

    def quant(**kw):
        a = ok | kw
        return q(a["W"], a["dt"], a["N"], a["K"], a["g"], a["P"], a["s"], None)
    for bad in (dict(W=None), dict(P=None), dict(s=None), dict(dt=2), dict(N=-1), dict(K=0), dict(P=A + 16),
                dict(s=A)):
        assert quant(**bad) == tw.ERR_INVALID_ARG, bad
    for bad in (dict(g=16), dict(g=256), dict(K=192), dict(K=(1 << 24) + 128), dict(g=0)):
        assert quant(**bad) == tw.ERR_UNSUPPORTED_SHAPE, bad
    for bad in (dict(W=A + 4), dict(P=B + 8), dict(s=D + 4)):
        assert quant(**bad) == tw.ERR_MISALIGNED, bad
    assert quant(N=0) == tw.OK

    def mm(X=A, xd=1, P=B, s=D, M=1, N=8, K=256, g=128, Y=OFFS, yd=1, flags=0):
        return tw.lib.bitnet_w4a16_matmul(X, xd, P, s, M, N, K, g, Y, yd, flags, None)
    for bad in (dict(X=None), dict(P=None), dict(s=None), dict(Y=None), dict(xd=2), dict(yd=3), dict(M=-1),
                dict(N=1 << 31), dict(K=-128), dict(flags=2), dict(Y=A)):
        assert mm(**bad) == tw.ERR_INVALID_ARG, bad
    for bad in (dict(g=96), dict(K=192), dict(K=1 << 25)):
        assert mm(**bad) == tw.ERR_UNSUPPORTED_SHAPE, bad
    for bad in (dict(X=A + 2), dict(P=B + 4), dict(Y=OFFS + 2), dict(s=D + 8)):
        assert mm(**bad) == tw.ERR_MISALIGNED, bad
    assert mm(M=0) == tw.OK and mm(N=0) == tw.OK
    assert mm(M=1 << 20) == tw.ERR_UNSUPPORTED_SHAPE


def test_logprobs(tw):
    def lp(x=A, dt=1, M=2, V=100, stride=100, tok=B, top=3, a=D, b=D + 64, ids=OFFS, tl=LENS):
        return tw.lib.bitnet_token_logprobs(x, dt, M, V, stride, tok, top, a, b, ids, tl, None)
    for bad in (dict(x=None), dict(tok=None), dict(a=None), dict(b=None), dict(ids=None), dict(tl=None), dict(dt=2),
                dict(M=-1), dict(V=0), dict(V=1 << 31), dict(top=-1), dict(top=101), dict(V=2), dict(stride=99)):
        assert lp(**bad) == tw.ERR_INVALID_ARG, bad
    assert lp(top=33) == tw.ERR_UNSUPPORTED_SHAPE
    for bad in (dict(x=A + 1), dict(tok=B + 4), dict(a=D + 2), dict(ids=OFFS + 4), dict(tl=LENS + 1)):
        assert lp(**bad) == tw.ERR_MISALIGNED, bad
    assert lp(M=0, x=None) == tw.OK


def test_binding_refuses(tw):
    """The binding's own checks: CPU tensors, types, shapes, layouts."""
    cpu = torch.zeros(2, 20, 128)
    with pytest.raises(ValueError, match="CUDA"):
        tw.KVCache(4, 64, 5, 128, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        tw.bitnet_quantize_weights_w4(torch.zeros(4, 128))
    with pytest.raises(TypeError):
        tw.bitnet_quantize_weights_w4(torch.zeros(4, 128, dtype=torch.float16))
    with pytest.raises(ValueError, match="group"):
        tw.bitnet_quantize_weights_w4(torch.zeros(4, 128, device="meta"), group=100)
    with pytest.raises(ValueError, match="CUDA"):
        tw.bitnet_w4a16_matmul(torch.zeros(1, 128), torch.zeros(4, 64, dtype=torch.uint8),
                               torch.zeros(4, 1, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="K/2"):
        tw.bitnet_w4a16_matmul(torch.zeros(1, 256), torch.zeros(4, 64, dtype=torch.uint8),
                               torch.zeros(4, 1, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="scales"):
        tw.bitnet_w4a16_matmul(torch.zeros(1, 128), torch.zeros(4, 64, dtype=torch.uint8),
                               torch.zeros(3, 1, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="CUDA"):
        tw.bitnet_token_logprobs(torch.zeros(2, 8), torch.zeros(2, dtype=torch.int64))
    with pytest.raises(TypeError):
        tw.bitnet_token_logprobs(torch.zeros(2, 8), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="row of logits"):
        tw.bitnet_token_logprobs(torch.zeros(8, 2).t(), torch.zeros(2, dtype=torch.int64))

    class FakeCache:  # a cache's shape without its memory
        heads, head_dim, page_tokens, num_pages = 5, 128, 64, 4
        k_codes = torch.zeros(1)
        _ref = 0
    pages, lens = torch.zeros(2, 3, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    kv = torch.zeros(2, 5, 128)
    with pytest.raises(ValueError, match="CUDA"):
        tw.bitnet_kv_append(FakeCache, kv, kv, pages, lens)
    with pytest.raises(ValueError, match=r"K and V must be"):
        tw.bitnet_kv_append(FakeCache, kv[:, :4], kv[:, :4], pages, lens)
    with pytest.raises(TypeError):
        tw.bitnet_kv_append(FakeCache, kv, kv.bfloat16(), pages, lens)
    with pytest.raises(ValueError, match="one after the other"):
        wide = torch.zeros(2, 5, 256)[..., ::2]
        tw.bitnet_kv_append(FakeCache, wide, wide, pages, lens)
    with pytest.raises(TypeError):
        tw.bitnet_kv_append(FakeCache, kv, kv, pages.long(), lens)
    with pytest.raises(ValueError, match="without offsets"):
        tw.bitnet_kv_append(FakeCache, kv[:1], kv[:1], pages, lens)
    with pytest.raises(ValueError, match="offsets"):
        tw.bitnet_kv_append(FakeCache, kv, kv, pages, lens, offsets=lens)
    with pytest.raises(ValueError, match="Q must be"):
        tw.bitnet_kv_attention(FakeCache, cpu[..., :64].contiguous(), pages, lens)
    with pytest.raises(ValueError, match="contiguous"):
        tw.bitnet_kv_attention(FakeCache, cpu[..., ::2], pages, lens)
    with pytest.raises(ValueError, match="CUDA"):
        tw.bitnet_kv_attention(FakeCache, cpu, pages, lens)
