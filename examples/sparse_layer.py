"""The feed-forward half of a mixture-of-experts decoder layer, and the answer
behind it.

    python examples/sparse_layer.py

The output of the block before (attention, say) joins the residual stream and is
normed in one pass; a router chooses each token's experts; their gate and up
projections run on int8 codes of rotated activations with the SwiGLU as epilogue,
their down projections on codes of its result; the weighted sum over the experts
joins the residual stream with the norm before the head; the head's logits give
the drawn tokens' log probabilities and the best alternatives.  The script
captures a step as a graph, replays it, compares the last results with a float64
layer and prints the time of a step."""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import rotated_bit_quantized_amd as oq  # noqa: E402


class SparseLayer:
    """Weights are float32: router [E][hidden], gate_up [E][2 f][hidden], down [E][hidden][f], head [V][hidden], norms [hidden]."""

    def __init__(self, router, gate_up, down, head, w_pre, w_post, w_out, k, block, score="softmax", bias=None, seed=0):
        E, hidden = router.shape
        g = torch.Generator().manual_seed(seed)
        self.rot_in, self.rot_mid, self.rot_out = (self._rotation(n, block, g, router.device) for n in (hidden, down.shape[2], hidden))
        self.router_w, self.k = router, k
        self.router = oq.Router(E, k, score=score, bias=bias)
        self.up, self.down = (self._experts(w, rot) for w, rot in ((gate_up, self.rot_in), (down, self.rot_mid)))
        self.head = oq.oq_quant_weight_w8(head, self.rot_out)
        self.pre, self.post, self.out = (oq.Norm(oq.OQ_NORM_RMS, hidden, w=w) for w in (w_pre, w_post, w_out))

    @staticmethod
    def _rotation(K, block, g, dev):
        perm = torch.randperm(K, generator=g)[None]
        signs = torch.randint(0, 2, (1, K), generator=g) * 2 - 1
        return oq.Rotation.rpbh(perm.to(dev), signs.to(dev), block)

    @staticmethod
    def _experts(w, rot):
        E, N, K = w.shape
        q = oq.oq_quant_weight_w8(w.reshape(E * N, K), rot)
        return q["codes"].view(E, N, K), q["scales"].view(E, N)

    def forward(self, y, r, mask=None):
        """y, r bfloat16 [T][hidden]: the last block's output and the residual stream;
        mask (uint8, nullable): padding is 0.  Returns (r, h, ids, weights): the stream
        behind the layer, its normed form, the experts and their weights."""
        r, h = oq.oq_residual_norm(y, r, pre=self.pre)
        ids, weights, offsets, order = oq.oq_route(h.float() @ self.router_w.t(), self.router, mask=mask)
        a = oq.oq_quant_act(h, self.rot_in, oq.OQ_A8)
        u = oq.oq_gemm_w8a8_experts(a["codes"], a["scale"], *self.up, offsets, order, per=self.k, act=oq.OQ_ACT_SWIGLU)
        b = oq.oq_quant_act(u, self.rot_mid, oq.OQ_A8)
        d = oq.oq_gemm_w8a8_experts(b["codes"], b["scale"], *self.down, offsets, order, per=1)
        # rows of entries without an expert were not written; their weights are 0
        r, h = oq.oq_residual_norm(d, r, weights=weights, post=self.post, pre=self.out)
        return r, h, ids, weights

    def answer(self, h, tokens, top):
        """Logits of normed rows, and what oq_logprobs says of them."""
        a = oq.oq_quant_act(h, self.rot_out, oq.OQ_A8)
        logits = oq.oq_gemm_w8a8(a["codes"], a["scale"], self.head["codes"], self.head["scales"])
        return logits, oq.oq_logprobs(logits, tokens, top=top)


def random_layer(hidden, f, E, k, V, block=128, seed=0, dev="cuda", **how):
    """A layer of random weights and its weights."""
    g = torch.Generator(device=dev).manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    router = rand(E, hidden) / math.sqrt(hidden)
    gate_up, down = rand(E, 2 * f, hidden) / math.sqrt(hidden), rand(E, hidden, f) * 2 / math.sqrt(f)
    head = rand(V, hidden) * 2 / math.sqrt(hidden)
    norms = [1 + 0.1 * rand(hidden) for _ in range(3)]
    weights = (router, gate_up, down, head, *norms)
    return SparseLayer(*weights, k, block, seed=seed, **how), weights


def reference(weights, y, r, ids, score="softmax", bias=None, eps=1e-6):
    """The layer in float64 with the experts `ids` [T][k] (-1: none): (r, h, router scores, logits of the head)."""
    router, gate_up, down, head, w_pre, w_post, w_out = weights

    def norm(x, w):
        return x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()

    r = r.double() + y.double()
    h = norm(r, w_pre)
    x = h @ router.double().t()
    s = torch.softmax(x, 1) if score == "softmax" else torch.sigmoid(x)
    out = torch.zeros_like(r)
    for t in range(len(r)):
        mine = [e for e in ids[t].tolist() if e >= 0]
        if not mine:
            continue
        p = s[t, mine] / s[t, mine].sum()
        for w, e in zip(p, mine):
            g, u = (gate_up[e].double() @ h[t]).chunk(2)
            out[t] += w * (down[e].double() @ (g * torch.sigmoid(g) * u))
    r = r + norm(out, w_post)
    h = norm(r, w_out)
    return r, h, s if bias is None else s + bias.double(), h @ head.double().t()


def main(hidden=2048, f=768, E=128, k=8, V=32000, T=64, steps=32):
    layer, weights = random_layer(hidden, f, E, k, V)
    g = torch.Generator(device="cuda").manual_seed(1)
    ys, rs = (torch.randn(steps, T, hidden, generator=g, device="cuda").bfloat16() for _ in range(2))
    tokens = torch.randint(0, V, (T, 1), generator=g, device="cuda", dtype=torch.int32)
    y, r = torch.empty_like(ys[0]), torch.empty_like(rs[0])

    def step():
        out = layer.forward(y, r)
        return out, layer.answer(out[1], tokens, 5)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y.copy_(ys[0]), r.copy_(rs[0])
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        (r_out, h, ids, _), (logits, answer) = step()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for i in range(steps):
        y.copy_(ys[i]), r.copy_(rs[i])
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    some = slice(0, 4)
    want = reference(weights, y[some], r[some], ids[some])
    off = max(float((a[some].double() - b).norm() / b.norm()) for a, b in ((r_out, want[0]), (logits, want[3])))
    print(f"{T} tokens, {k} of {E} experts: {start.elapsed_time(end) / steps * 1e3:.1f} us a step, {off:.4f} of the float64 layer's norm off, "
          f"mean entropy {float(answer[2].mean()):.2f}")


if __name__ == "__main__":
    main()
