"""A decode step of all the operators together: the chain with a cache per
layer and an output head, token by token, every link against its definition
on the link's own inputs; captured and replayed; two at once."""

import numpy as np
import pytest
import torch

import decode_ref as dref
from test_gpu_decode_ops import check_attention, check_logprobs, check_w4

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
D, HEADS, Q_HEADS, FFN, VOCAB = 64, 2, 6, 512, 1003
WIDTH = D * Q_HEADS


@pytest.fixture(scope="module")
def bl():
    import ternary_weight_linear_token_b200 as bl
    return bl


def chain_of(bl, layers=2, pages=3, page_tokens=16, seed=0, **kw):
    from ternary_weight_linear_token_b200.chain import DecodeChain
    g = torch.Generator().manual_seed(seed)

    def w(n, k):
        return torch.randn(n, k, generator=g) * 0.02
    weights = [[(w(WIDTH + 2 * HEADS * D, WIDTH), False), (w(WIDTH, WIDTH), False), (w(FFN, WIDTH), True),
                (w(WIDTH, FFN), False)] for _ in range(layers)]
    caches = [bl.KVCache(pages, page_tokens, HEADS, D, device=DEV) for _ in range(layers)]
    return DecodeChain(weights, caches=caches, head=w(VOCAB, WIDTH), **kw)


def tokens_of(n, seed=1):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(1, WIDTH, generator=g).bfloat16().to(DEV) for _ in range(n)]


def test_every_link(bl):
    from oracle import ref
    chain = chain_of(bl)
    shape = (3, HEADS, 16, D)
    parts = [[np.zeros(shape, np.int8), np.zeros(shape[:2], np.float32), np.zeros(shape, np.int8),
              np.zeros(shape[:2], np.float32)] for _ in chain.layers]
    table = np.arange(3, dtype=np.int32)[None]
    weights = [[(p["packed"].cpu().numpy(), float(p["gamma"].item())) for p in proj] for proj in chain.layers]

    def linear(x, w, n, relu2=False):
        y = ref.bitlinear(x.float().cpu().numpy(), w[0], w[1], n, relu2=relu2)["y"]
        return torch.from_numpy(np.ascontiguousarray(y)).bfloat16()
    for pos, x in enumerate(tokens_of(35)):  # past two page borders
        out = chain.run(x)
        for li, (proj, bufs) in enumerate(zip(chain.layers, chain.outs)):
            kv = bufs[0].view(1, -1, D).float().cpu().numpy()
            for i, at in ((0, Q_HEADS), (2, Q_HEADS + HEADS)):
                dref.append(parts[li][i], parts[li][i + 1], kv[:, at:at + HEADS], table, [pos + 1], [1])
            c = chain.caches[li]
            for got, want in zip((c.k_codes, c.k_scales, c.v_codes, c.v_scales), parts[li]):
                assert np.array_equal(got.cpu().numpy(), want)
            q = bufs[0].view(1, -1, D)[:, :Q_HEADS]
            check_attention(q, chain.attended[li], parts[li], table, [pos + 1], [1])
            assert torch.equal(linear(chain.attended[li].view(1, WIDTH), weights[li][1], WIDTH), bufs[1].cpu())
            assert torch.equal(linear(bufs[1], weights[li][2], FFN, relu2=True), bufs[2].cpu())
        if pos % 10 == 0:
            packed, scales = chain.head
            s = scales.float().cpu().numpy()
            words = packed.cpu().numpy().view(np.uint32)
            codes = np.stack([(words >> np.uint32(16 * (e % 2) + 4 * (e // 2))) & 15 for e in range(8)], -1)
            check_w4(out, chain.logits, codes.reshape(VOCAB, WIDTH).astype(np.int64) - 8, s, 128)
            tok = torch.tensor([pos * 7], device=DEV)
            check_logprobs(chain.logits, tok, 5, chain.score(tok, top=5))
    assert chain.lens.item() == 35 and bl.bitnet_get_device_status() == bl.OK
    # a new sequence in the old one's cache
    first = tokens_of(1)[0]
    again = chain_of(bl)
    want = again.run(first).clone(), again.logits.clone()
    chain.reset()
    assert torch.equal(chain.run(first), want[0]) and torch.equal(chain.logits, want[1])


def test_captured_and_replayed(bl):
    eager, replayed = chain_of(bl), chain_of(bl)
    xs = tokens_of(20)
    graph = replayed.capture()
    assert replayed.lens.item() == 0
    for x in xs:
        want = eager.run(x)
        replayed.x_in.copy_(x)
        graph.replay()
        assert torch.equal(replayed.outs[-1][4], want) and torch.equal(replayed.logits, eager.logits)
        for a, b in zip(replayed.caches, eager.caches):
            assert torch.equal(a.k_codes, b.k_codes) and torch.equal(a.v_scales, b.v_scales)
    assert eager.launches_per_token() == 2 * (4 + 2) + 2 and bl.bitnet_get_device_status() == bl.OK


@pytest.mark.parametrize("ran,page_tokens,pages", [(21, 16, 3), (16, 16, 3), (32, 16, 2)])
def test_capture_leaves_no_trace(bl, ran, page_tokens, pages):
    """Captured after some tokens, in the middle of a page, at its end and on a full cache, with a large
    token left in x_in: caches, links, logits, length and status stay as they were, and what follows is
    what an eager chain gives."""
    eager, chain = (chain_of(bl, pages=pages, page_tokens=page_tokens) for _ in range(2))
    xs = tokens_of(ran + 6)
    for x in xs[:ran]:
        eager.run(x)
        chain.run(x)
    chain.x_in.copy_(xs[0] * 1000)

    def state(c):
        return ([t for k in c.caches for t in (k.k_codes, k.k_scales, k.v_codes, k.v_scales)]
                + [t for bufs in c.outs for t in bufs] + c.attended + [c.logits, c.lens])
    before = [t.clone() for t in state(chain)]
    graph = chain.capture()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(state(chain), before))
    assert bl.bitnet_get_device_status() == bl.OK
    for x in xs[ran:min(ran + 6, pages * page_tokens)]:
        eager.run(x)
        chain.x_in.copy_(x)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(state(chain), state(eager)))
    assert bl.bitnet_get_device_status() == bl.OK


def test_two_chains_at_once(bl):
    """Two sequences on two streams, graphs of both in flight together, give what each gives alone."""
    alone = [chain_of(bl, seed=s) for s in (0, 1)]
    xs = [tokens_of(6, seed=s) for s in (5, 6)]
    want = [[c.run(x).clone() for x in t] for c, t in zip(alone, xs)]
    both = [chain_of(bl, seed=s) for s in (0, 1)]
    graphs = [c.capture() for c in both]
    streams = [torch.cuda.Stream() for _ in both]
    torch.cuda.synchronize()
    got = [[], []]
    for i in range(6):
        for c, g, s, t, out in zip(both, graphs, streams, xs, got):
            with torch.cuda.stream(s):
                c.x_in.copy_(t[i])
                g.replay()
                out.append(c.outs[-1][4].clone())
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_prompt_then_tokens(bl):
    """A prompt appended and attended to at once, then single tokens: each row as if it had come alone."""
    rng = np.random.default_rng(2)
    H, P, Dm, Hq, n = 2, 32, 128, 8, 150
    cache = bl.KVCache(8, P, H, Dm, device=DEV)
    i32 = lambda v: torch.tensor(np.asarray(v, dtype=np.int32), device=DEV)  # noqa: E731
    pages = i32([[7, 0, 3, 1, 5, 2, 4, 6]])
    kv = torch.from_numpy(rng.standard_normal((n + 5, 2 * H, Dm)).astype(np.float32)).to(DEV).bfloat16()
    q = torch.from_numpy(rng.standard_normal((n + 5, Hq, Dm)).astype(np.float32)).to(DEV).bfloat16()
    host = lambda: [a.cpu().numpy() for a in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]  # noqa: E731
    bl.bitnet_kv_append(cache, kv[:n, :H], kv[:n, H:], pages, i32([n]), offsets=i32([0, n]))
    o = bl.bitnet_kv_attention(cache, q[:n], pages, i32([n]), offsets=i32([0, n]))
    check_attention(q[:n], o, host(), pages.cpu().numpy(), [n], [n])
    for i in range(n, n + 5):
        bl.bitnet_kv_append(cache, kv[i:i + 1, :H], kv[i:i + 1, H:], pages, i32([i + 1]))
        o = bl.bitnet_kv_attention(cache, q[i:i + 1], pages, i32([i + 1]))
        check_attention(q[i:i + 1], o, host(), pages.cpu().numpy(), [i + 1], [1])


def test_on_another_stream(bl):
    """The stream argument: work and what is allocated for it are the stream's."""
    s = torch.cuda.Stream()
    x = torch.randn(3, 2560, device=DEV).bfloat16()
    packed, scales = bl.bitnet_quantize_weights_w4(torch.randn(640, 2560, device=DEV), 128)
    want = bl.bitnet_w4a16_matmul(x, packed, scales)
    lp = bl.bitnet_token_logprobs(want, torch.tensor([1, 2, 3], device=DEV), top=4)
    torch.cuda.synchronize()
    s.wait_stream(torch.cuda.current_stream())
    y = bl.bitnet_w4a16_matmul(x, packed, scales, stream=s)
    lp2 = bl.bitnet_token_logprobs(y, torch.tensor([1, 2, 3], device=DEV), top=4, stream=s)
    s.synchronize()
    assert torch.equal(y, want) and all(torch.equal(a, b) for a, b in zip(lp, lp2))


def test_chain_refuses(bl):
    with pytest.raises(ValueError, match="persistent"):
        chain_of(bl, persistent=True)
    from ternary_weight_linear_token_b200.chain import DecodeChain
    plain = DecodeChain([], quantized=chain_of(bl).layers)
    with pytest.raises(ValueError, match="no head"):
        plain.score(torch.zeros(1, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError, match="caches for"):
        DecodeChain([], quantized=plain.layers, caches=[])
    with pytest.raises(ValueError, match="QKV columns"):
        DecodeChain([], quantized=plain.layers, caches=[bl.KVCache(1, 16, 1, 64, device=DEV)] * 2)
    with pytest.raises(ValueError, match="head must be"):
        DecodeChain([], quantized=plain.layers, head=torch.zeros(10, 128))
    # a token past the last page: refused on the device, the status word says so
    chain = chain_of(bl, pages=1)
    for x in tokens_of(17):
        chain.run(x)
    assert bl.bitnet_get_device_status() == bl.ERR_RANGE
