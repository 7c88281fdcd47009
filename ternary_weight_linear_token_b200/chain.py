"""Decode chain: a stack of decoder layers' BitLinear projections run for one
token (M = 1), each projection re-quantising its own input per token.

Per layer: q = BitLinear_qkv(x)[:, :d]; o = BitLinear_o(q);
u = ReLU^2(BitLinear_up(o)); d = BitLinear_down(u); x <- rms_norm(d).

Attention, RoPE and the KV cache are not part of the BitLinear path; the first
d columns of the fused QKV output stand in for the attention output.  The
model card (BitNet b1.58 2B4T, 模型详情 -> 架构) names ReLU^2 in the FFN and a
"subln" normalisation without giving its formula; the weightless RMS
normalisation between layers is the plain stand-in (without it the squared
activations vanish within a few layers).

Two ways to run it, both through the C-ABI library on one stream and both
capturable in a CUDA graph (``capture``):
  * per launch (default): ``run`` makes one call per projection, 4 kernels
    per layer (each layer's QKV call normalises its input itself,
    ``bitnet_rms_norm_w158a8_matmul``) plus one normalisation at the end;
  * persistent (``persistent=True``): ``run`` makes one call of
    ``bitnet_decode_chain``, one kernel for the whole stack, with the
    normalisation folded into the next layer's QKV projection.
Both fill the same buffers (``outs``), so every link can be checked.

The per-launch form can also run what stands around the projections:
  * ``caches``, a ``KVCache`` per layer: attention over the tokens that have
    run takes the place of the stand-in.  The fused QKV output holds the query
    heads (the first d columns), then the key heads, then the value heads; the
    token's keys and values are appended to the layer's cache and its queries
    attend to it.  No position encoding: queries and keys are used as the
    projection gives them, and a model that rotates them calls the entry points
    itself.  One sequence, token by token; prompts, batches and drafts by the
    entry points too.
  * ``head`` [vocabulary, d]: the output head, kept in 4 bits with a scale per
    128 weights; ``run`` leaves the token's logits in ``logits`` (fp32) and
    ``score`` gives log probabilities, entropy and top alternatives of them.
"""

from __future__ import annotations

import torch

from . import (KVCache, bitnet_decode_chain, bitnet_decode_chain_steps, bitnet_decode_chain_workspace_size,
               bitnet_kv_append, bitnet_kv_attention, bitnet_kv_attention_workspace_size,
               bitnet_quantize_weights, bitnet_quantize_weights_w4, bitnet_rms_norm,
               bitnet_rms_norm_w158a8_matmul, bitnet_token_logprobs, bitnet_w158a8_matmul,
               bitnet_w4a16_matmul)


class DecodeChain:
    def __init__(self, weights, device="cuda:0", weights_static: bool = True,
                 persistent: bool = False, quantized=None, caches=None,
                 head: torch.Tensor | None = None):
        """weights: list over layers of a list of 4 (W [N, K] float tensor,
        relu2) pairs in the order qkv, o, up, down (any iterable: a
        generator keeps only one layer's latent weights alive at a time).
        Weights are quantised on the device once, here.
        quantized: instead of weights, the ``layers`` of another DecodeChain
        (packed weights shared, nothing quantised again).
        caches: a KVCache per layer (per-launch form only): one sequence, whose
        token p lies in page p // page_tokens of each; ``lens`` counts its
        tokens, ``reset`` starts over, and a token past the last page is
        refused on the device (bitnet_get_device_status).
        head: the output head's weights [vocabulary, d], fp32 or bf16."""
        self.device = torch.device(device)
        self.weights_static = weights_static
        if quantized is not None:
            self.layers = quantized
        else:
            self.layers = []
            for layer in weights:
                proj = []
                for W, relu2 in layer:
                    W = W.to(self.device).contiguous()
                    packed, gamma = bitnet_quantize_weights(W)
                    proj.append(dict(packed=packed, gamma=gamma, N=W.shape[0], K=W.shape[1],
                                     relu2=relu2))
                    del W
                self.layers.append(proj)
        d = self.layers[0][1]["K"]
        self.d = d
        # activation buffers, one per step, kept so every link can be checked
        self.x_in = torch.zeros((1, d), dtype=torch.bfloat16, device=self.device)
        self.outs = []
        for proj in self.layers:
            bufs = [torch.empty((1, p["N"]), dtype=torch.bfloat16, device=self.device) for p in proj]
            bufs.append(torch.empty((1, d), dtype=torch.bfloat16, device=self.device))  # norm out
            self.outs.append(bufs)
        self.graph = None
        self.persistent = persistent
        self.caches = None
        if caches is not None:
            self._take_caches(list(caches))
        self.head = None
        if head is not None:
            if head.dim() != 2 or head.shape[1] != d:
                raise ValueError(f"head must be [vocabulary, {d}]")
            self.head = bitnet_quantize_weights_w4(head.to(self.device).contiguous(), group=128)
            self.logits = torch.empty((1, head.shape[0]), dtype=torch.float32, device=self.device)
        if persistent:
            steps = []
            for li, (proj, bufs) in enumerate(zip(self.layers, self.outs)):
                for pi, p in enumerate(proj):
                    step = dict(packed=p["packed"], gamma=p["gamma"], Y=bufs[pi], relu2=p["relu2"])
                    if pi == 0 and li > 0:  # the previous layer's normalisation, folded in
                        step.update(norm_in=True, X_normed=self.outs[li - 1][4])
                    steps.append(step)
            self._steps = bitnet_decode_chain_steps(steps)
            self._keep = steps
            self.workspace = torch.zeros(bitnet_decode_chain_workspace_size(self._steps),
                                         dtype=torch.uint8, device=self.device)

    def _take_caches(self, caches):
        if self.persistent:
            raise ValueError("the persistent chain runs projections only: caches need the per-launch form")
        if len(caches) != len(self.layers):
            raise ValueError(f"{len(caches)} caches for {len(self.layers)} layers")
        first = caches[0]
        shape = (first.num_pages, first.heads, first.page_tokens, first.head_dim)
        heads, rest = divmod(self.d, first.head_dim)
        for li, (c, proj) in enumerate(zip(caches, self.layers)):
            if (c.num_pages, c.heads, c.page_tokens, c.head_dim) != shape:
                raise ValueError("the layers' caches must have the same shape")
            if rest or heads % c.heads or proj[0]["N"] != (heads + 2 * c.heads) * c.head_dim:
                raise ValueError(f"layer {li}: {proj[0]['N']} QKV columns are not {self.d} of queries and "
                                 f"2 x {c.heads} heads of {c.head_dim}")
        self.caches, self.q_heads = caches, heads
        self.pages = torch.arange(first.num_pages, dtype=torch.int32, device=self.device)[None]
        self.lens = torch.zeros(1, dtype=torch.int32, device=self.device)
        # attention output of each layer, kept like the other links
        self.attended = [torch.empty((1, heads, first.head_dim), dtype=torch.bfloat16, device=self.device)
                         for _ in caches]
        size = bitnet_kv_attention_workspace_size(first, torch.bfloat16, 1, heads, 1, first.num_pages)
        self._kv_workspace = torch.empty(max(size, 1), dtype=torch.uint8, device=self.device)
        self._kv_launches = 3 if size > 0 else 2

    def reset(self) -> None:
        """Starts a new sequence: the next token is its first."""
        if self.caches is not None:
            self.lens.zero_()

    def _attend(self, li: int, qkv: torch.Tensor) -> torch.Tensor:
        """The token's keys and values into layer li's cache, its queries over it."""
        c = self.caches[li]
        q, k, v = qkv.view(1, -1, c.head_dim).split((self.q_heads, c.heads, c.heads), dim=1)
        bitnet_kv_append(c, k, v, self.pages, self.lens)
        out = self.attended[li]
        bitnet_kv_attention(c, q, self.pages, self.lens, O=out, workspace=self._kv_workspace)
        return out.view(1, self.d)

    def score(self, tokens: torch.Tensor, top: int = 0):
        """(logprob, entropy, top_ids, top_logprobs) of the last token's logits
        (bitnet_token_logprobs); tokens [1] int64."""
        if self.head is None:
            raise ValueError("the chain has no head")
        return bitnet_token_logprobs(self.logits, tokens, top=top)

    @property
    def packed_bytes(self) -> int:
        return sum(p["packed"].numel() for layer in self.layers for p in layer)

    def _bl(self, x, p, y):
        bitnet_w158a8_matmul(x, p["packed"], p["gamma"], relu2=p["relu2"], Y=y,
                             weights_static=self.weights_static)

    def run(self, x0: torch.Tensor | None = None) -> torch.Tensor:
        if x0 is not None:
            self.x_in.copy_(x0)
        if self.persistent:
            bitnet_decode_chain(self._steps, self.x_in, self.workspace, y_norm=self.outs[-1][4])
            return self._finish()
        if self.caches is not None:
            self.lens.add_(1)
        for li, (proj, bufs) in enumerate(zip(self.layers, self.outs)):
            qkv, o, up, down = proj
            if li == 0:
                self._bl(self.x_in, qkv, bufs[0])
            else:  # the previous layer's normalisation, inside this call
                prev = self.outs[li - 1]
                bitnet_rms_norm_w158a8_matmul(prev[3], qkv["packed"], qkv["gamma"],
                                              X_normed=prev[4], relu2=qkv["relu2"], Y=bufs[0],
                                              weights_static=self.weights_static)
            if self.caches is not None:
                q = self._attend(li, bufs[0])
            else:
                q = bufs[0][:, : self.d]      # contiguous for one token
            self._bl(q, o, bufs[1])
            self._bl(bufs[1], up, bufs[2])
            self._bl(bufs[2], down, bufs[3])
        last = self.outs[-1]
        bitnet_rms_norm(last[3], Y=last[4])
        return self._finish()

    def _finish(self) -> torch.Tensor:
        x = self.outs[-1][4]
        if self.head is not None:
            bitnet_w4a16_matmul(x, *self.head, Y=self.logits, weights_static=self.weights_static)
        return x

    def capture(self) -> torch.cuda.CUDAGraph:
        """Capture one token through the whole stack in a CUDA graph.  (With
        caches the warm-up is the first token of a cache of its own, into
        buffers of its own: nothing of the sequence changes.)"""
        s = torch.cuda.Stream(self.device)
        s.wait_stream(torch.cuda.current_stream(self.device))
        with torch.cuda.stream(s):
            self._warm_up()
        torch.cuda.current_stream(self.device).wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self.run()
        self.graph = g
        return g

    def _warm_up(self) -> None:
        """Runs a token outside capture.  An append would leave its mark on the
        caches that taking the length back does not remove: a page's scale that
        grew, and its older tokens' codes rounded to it."""
        if self.caches is None:
            self.run()
            return
        c = self.caches[0]
        kept = dict(vars(self))
        try:
            self.caches = [KVCache(1, c.page_tokens, c.heads, c.head_dim, device=self.device)] * len(self.caches)
            self.pages = torch.zeros_like(self.pages)  # as wide as the sequence's: the same kernels
            self.lens = torch.zeros_like(self.lens)
            self.outs = [[torch.empty_like(t) for t in bufs] for bufs in self.outs]
            self.attended = [torch.empty_like(t) for t in self.attended]
            if self.head is not None:
                self.logits = torch.empty_like(self.logits)
            self.run()
        finally:
            vars(self).update(kept)

    def launches_per_token(self) -> int:
        """Kernels of the library per token (with caches, torch's addition to
        ``lens`` comes on top)."""
        head = 0 if self.head is None else 1
        if self.persistent:
            return 1 + head
        return (4 + (0 if self.caches is None else self._kv_launches)) * len(self.layers) + 1 + head
