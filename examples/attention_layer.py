"""One attention layer of a decoder, served from a paged cache.

    python examples/attention_layer.py

Every projection runs on int8 codes of rotated activations and weights; the
queries and keys pass a per-head norm and a rotary embedding; keys and values
live in a paged cache, of which the first pages (a prompt that all sequences
share) are read once for all of them.  The script fills the prompt, captures a
decode step as a graph, replays it, compares the last outputs with a float64
layer and prints the time of a step."""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import rotated_bit_quantized_amd as oq  # noqa: E402


class AttentionLayer:
    """Weights are float32 [out][in]: qkv has (heads + 2 kv_heads) d rows, out has hidden rows."""

    def __init__(self, qkv, out, w_q, w_k, heads, kv_heads, d, rope, block, seed=0):
        self.heads, self.kv_heads, self.d, self.rope = heads, kv_heads, d, rope
        self.w_q, self.w_k = w_q, w_k
        g = torch.Generator().manual_seed(seed)
        self.rot_in, self.rot_out = (self._rotation(w.shape[1], block, g, w.device) for w in (qkv, out))
        self.qkv = oq.oq_quant_weight_w8(qkv, self.rot_in)
        self.out = oq.oq_quant_weight_w8(out, self.rot_out)

    @staticmethod
    def _rotation(K, block, g, dev):
        perm = torch.randperm(K, generator=g)[None]
        signs = torch.randint(0, 2, (1, K), generator=g) * 2 - 1
        return oq.Rotation.rpbh(perm.to(dev), signs.to(dev), block)

    def _linear(self, x, rot, w):
        a = oq.oq_quant_act(x, rot, oq.OQ_A8)
        return oq.oq_gemm_w8a8(a["codes"], a["scale"], w["codes"], w["scales"])

    def forward(self, x, n_q, kv, pos, slot, prefix_table, prefix_len, tables, lens):
        """x bfloat16 [B n_q][hidden], the last n_q tokens of each sequence; lens count them."""
        T = x.shape[0]
        y = self._linear(x, self.rot_in, self.qkv).view(T, self.heads + 2 * self.kv_heads, self.d)
        q, k, v = y.split((self.heads, self.kv_heads, self.kv_heads), 1)
        q, _ = oq.oq_qk_norm_rope(q, None, self.w_q, None, rope=self.rope, pos=pos, q_out=q)
        oq.oq_kv_append(k, v, slot, kv, self.w_k, rope=self.rope, pos=pos)
        o, _ = oq.oq_attn_prefix(q, n_q, kv, prefix_table, prefix_len, tables, lens, 1 / math.sqrt(self.d))
        return self._linear(o.view(T, self.heads * self.d), self.rot_out, self.out)


class Decoder:
    """B sequences behind one shared prompt, a token each at a time."""

    def __init__(self, layer, prompt, B, max_new, page=64):
        dev, self.layer, self.page, self.P = prompt.device, layer, page, prompt.shape[0]
        shared, own = -(-self.P // page), -(-max_new // page)
        pages = shared + B * own
        k = torch.zeros(pages, layer.kv_heads, page, layer.d, dtype=torch.bfloat16, device=dev)
        self.kv = oq.PagedKV(k, torch.zeros_like(k))
        self.prefix_table = torch.arange(shared, dtype=torch.int32, device=dev)
        self.tables = torch.arange(shared, pages, dtype=torch.int32, device=dev).view(B, own)
        self.lens = torch.zeros(B, dtype=torch.int32, device=dev)
        self.x = torch.zeros(B, prompt.shape[1], dtype=torch.bfloat16, device=dev)
        # the prompt is its own sequence: nothing shared before it, causal inside
        at = torch.arange(self.P, device=dev)
        self.prompt_y = layer.forward(prompt, self.P, self.kv, at.int(), at, None, 0, self.prefix_table[None],
                                      torch.full((1,), self.P, dtype=torch.int32, device=dev))

    def step(self):
        """The next token of every sequence, whose input stands in self.x."""
        at = self.lens.long()
        slot = self.tables.gather(1, (at // self.page)[:, None])[:, 0].long() * self.page + at % self.page
        pos = self.lens + self.P
        self.lens += 1
        self.y = self.layer.forward(self.x, 1, self.kv, pos, slot, self.prefix_table, self.P, self.tables, self.lens)
        return self.y

    def capture(self):
        """A graph of step(): self.x in, self.y out.  lens is as before afterwards."""
        lens = self.lens.clone()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            self.step()
        torch.cuda.current_stream().wait_stream(s)
        self.lens.copy_(lens)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self.step()
        return g


def random_layer(hidden, heads, kv_heads, d, rows, block=128, seed=0, dev="cuda"):
    """A layer of random weights and its weights (qkv, out, w_q, w_k, cos, sin)."""
    g = torch.Generator(device=dev).manual_seed(seed)
    qkv = torch.randn((heads + 2 * kv_heads) * d, hidden, generator=g, device=dev) / math.sqrt(hidden)
    out = torch.randn(hidden, heads * d, generator=g, device=dev) / math.sqrt(heads * d)
    w_q, w_k = (1 + 0.1 * torch.randn(d, generator=g, device=dev) for _ in range(2))
    angle = torch.arange(rows, device=dev)[:, None] * 10000.0 ** (-torch.arange(0, d, 2, device=dev) / d)
    cos, sin = angle.cos(), angle.sin()
    layer = AttentionLayer(qkv, out, w_q, w_k, heads, kv_heads, d, oq.Rope(cos, sin), block, seed)
    return layer, (qkv, out, w_q, w_k, cos, sin)


def reference(weights, heads, kv_heads, d, tokens, eps=1e-6):
    """The layer's last output in float64 for one whole sequence, tokens [n][hidden]."""
    qkv, out, w_q, w_k, cos, sin = (w.double() for w in weights)
    y = (tokens.double() @ qkv.T).view(-1, heads + 2 * kv_heads, d)
    q, k, v = y.split((heads, kv_heads, kv_heads), 1)

    def turn(x, w):
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w
        a, b = x.chunk(2, -1)
        c, s = cos[: len(x), None], sin[: len(x), None]
        return torch.cat((a * c - b * s, b * c + a * s), -1)

    q, k = turn(q, w_q)[-1].view(kv_heads, heads // kv_heads, d), turn(k, w_k)
    p = torch.softmax((q[:, :, None] * k.transpose(0, 1)[:, None]).sum(-1) / math.sqrt(d), -1)
    o = (p[..., None] * v.transpose(0, 1)[:, None]).sum(2)
    return o.reshape(heads * d) @ out.T


def main(hidden=4096, heads=32, kv_heads=8, d=128, B=16, prompt_len=4096, steps=32):
    layer, weights = random_layer(hidden, heads, kv_heads, d, prompt_len + steps + 1)
    g = torch.Generator(device="cuda").manual_seed(1)
    prompt = torch.randn(prompt_len, hidden, generator=g, device="cuda").bfloat16()
    xs = torch.randn(steps, B, hidden, generator=g, device="cuda").bfloat16()
    dec = Decoder(layer, prompt, B, steps + 1)
    graph = dec.capture()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for x in xs:
        dec.x.copy_(x)
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    off = 0.0
    for b in (0, B - 1):
        want = reference(weights, heads, kv_heads, d, torch.cat((prompt, xs[:, b])))
        off = max(off, float((dec.y[b].double() - want).norm() / want.norm()))
    print(f"{B} sequences behind {prompt_len} shared tokens: {start.elapsed_time(end) / steps * 1e3:.1f} us a step, "
          f"{off:.4f} of the float64 layer's norm off")


if __name__ == "__main__":
    main()
