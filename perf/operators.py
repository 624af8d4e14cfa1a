"""Workloads of the serving operators around the quantized linear layer.

Four operators of one attention layer of a quantized transformer, in the order
in which a serving step runs them:

- ``gemm_w8a8``: int8 activations (one scale a token) times int8 weights (one
  scale an output channel), bfloat16 out, with the layer's rank-1 mean
  restore and bias;
- ``qk_norm_rope``: RMS norm of every query and key head and the rotary
  position embedding, one pass;
- ``kv_append``: keys (normed and rotated on the way) and values written to
  the slots of a paged cache;
- ``attn_prefix``: attention of a batch of sequences that share a long prefix
  of the cache, each with a paged suffix of its own.

``own`` selects between the plain form of an operator (elementary torch
operations in float32, rounded once) and this repository's entry points.
"""
import math

import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one new token through the fused query/key/value projection of a 4096-wide LLM layer
        # (32 + 8 + 8 heads of 128): the latency of a single weight pass
        dict(name="w8a8 one token", op="gemm_w8a8", M=1, K=4096, N=6144, bias=False, center=False),
        # a ragged batch of tokens through the up projection of a 1920-wide transformer, centred and biased
        dict(name="w8a8 333 tokens", op="gemm_w8a8", M=333, K=1920, N=7680, bias=True, center=True),
        # a full prefill through the up projection of a 4096-wide LLM layer
        dict(name="w8a8 prefill 8192", op="gemm_w8a8", M=8192, K=4096, N=14336, bias=False, center=False),
        # one decode step of 64 sequences, grouped query heads
        dict(name="qk decode 64", op="qk_norm_rope", T=64, Hq=32, Hk=8, D=128, R=128, interleaved=False, gather=True),
        # one image's tokens in a 3072-wide diffusion transformer: rotary pairs interleaved, a table row per token
        dict(name="qk image 4096", op="qk_norm_rope", T=4096, Hq=24, Hk=24, D=128, R=128, interleaved=True, gather=False),
        # a long prefill of a 4096-wide LLM layer
        dict(name="qk prefill 32768", op="qk_norm_rope", T=32768, Hq=32, Hk=8, D=128, R=128, interleaved=False, gather=True),
        # the new token of each of 64 sequences
        dict(name="append decode 64", op="kv_append", T=64, H=8, D=128, R=128, page=64, norm=True, interleaved=False),
        # an odd prompt in a model of 30 heads of 64, half of each head rotated, no key norm, small pages
        dict(name="append prompt 4099", op="kv_append", T=4099, H=30, D=64, R=32, page=16, norm=False, interleaved=True),
        # a long prefill of a 4096-wide LLM layer
        dict(name="append prefill 32768", op="kv_append", T=32768, H=8, D=128, R=128, page=64, norm=True, interleaved=False),
        # three requests over a short shared system prompt
        dict(name="prefix 3 x 777", op="attn_prefix", B=3, n_q=1, Hk=8, G=4, D=128, page=16, prefix=777, suffix=60),
        # draft verification: four query tokens a sequence, heads of 64, few sequences over a document
        dict(name="prefix 24 x 4 x 5000", op="attn_prefix", B=24, n_q=4, Hk=6, G=5, D=64, page=32, prefix=5000, suffix=333),
        # a large batch over one long shared document
        dict(name="prefix 256 x 32768", op="attn_prefix", B=256, n_q=1, Hk=8, G=4, D=128, page=64, prefix=32768, suffix=512),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gemm_w8a8", "qk_norm_rope", "kv_append", "attn_prefix"])
    while True:
        if op == "gemm_w8a8":
            c = dict(op=op, M=_log(rng, 1, 8192), K=16 * _log(rng, 16, 896), N=_log(rng, 64, 14336), bias=rng.random() < 0.5,
                     center=rng.random() < 0.3)
            if c["M"] * c["K"] * c["N"] <= 8192 * 4096 * 14336:
                return c
        elif op == "qk_norm_rope":
            D = rng.choice([64, 80, 128, 256])
            Hk = rng.choice([1, 2, 4, 8, 24])
            c = dict(op=op, T=_log(rng, 1, 32768), Hq=Hk * rng.choice([1, 2, 4, 5]), Hk=Hk, D=D, R=rng.choice([D, D // 2]),
                     interleaved=rng.random() < 0.5, gather=rng.random() < 0.7)
            if c["T"] * (c["Hq"] + c["Hk"]) * D <= 32768 * 40 * 128:
                return c
        elif op == "kv_append":
            D = rng.choice([64, 80, 128, 256])
            c = dict(op=op, T=_log(rng, 1, 32768), H=rng.choice([1, 2, 4, 8, 30]), D=D, R=rng.choice([D, D // 2]),
                     page=rng.choice([16, 32, 64, 128]), norm=rng.random() < 0.5, interleaved=rng.random() < 0.5)
            if c["T"] * c["H"] * D <= 32768 * 8 * 128:
                return c
        else:
            c = dict(op=op, B=_log(rng, 1, 256), n_q=rng.choice([1, 1, 1, 2, 4]), Hk=rng.choice([1, 2, 4, 8]),
                     G=rng.choice([1, 2, 4, 5, 8]), D=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]),
                     prefix=_log(rng, 16, 32768), suffix=_log(rng, 8, 1024))
            if c["B"] * c["n_q"] * c["Hk"] * c["G"] * c["D"] * (c["prefix"] + c["suffix"]) <= 256 * 32 * 128 * 32768:
                return c


# ----------------------------------------------------------------- inputs --
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _codes8(g, rows, cols, std):
    """Rows of N(0, std^2) as absmax int8 codes and their scales."""
    v = torch.randn(rows, cols, generator=g, device="cuda") * std
    scale = v.abs().amax(1).clamp_min(1e-10) / 127
    return torch.round(v / scale[:, None]).clamp_(-127, 127).to(torch.int8), scale


def _rotary(rows, R):
    """cos and sin of position / 10000^(2 i / R), float32 [rows][R / 2]."""
    freq = 10000.0 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
    a = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * freq
    return a.cos().float(), a.sin().float()


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    op = case["op"]
    bf = torch.bfloat16
    if op == "gemm_w8a8":
        M, K, N = case["M"], case["K"], case["N"]
        st["qa"], st["a_scale"] = _codes8(g, M, K, 1.0)
        st["w"], st["w_scale"] = _codes8(g, N, K, 0.02)
        st["bias_v"] = torch.randn(N, generator=g, device="cuda") if case["bias"] else None
        st["mean"] = 3 * torch.randn(M, generator=g, device="cuda") if case["center"] else None
        st["w1"] = torch.randn(N, generator=g, device="cuda") if case["center"] else None
        st["y"] = torch.empty(M, N, dtype=bf, device="cuda")
        return st
    if op == "qk_norm_rope":
        T, Hq, Hk, D = case["T"], case["Hq"], case["Hk"], case["D"]
        # the fused projection's output, one row a token: query heads, key heads, value heads
        x = (1.5 * torch.randn(T, (Hq + 2 * Hk) * D, generator=g, device="cuda")).to(bf)
        st["q"] = x[:, : Hq * D].view(T, Hq, D)
        st["k"] = x[:, Hq * D : (Hq + Hk) * D].view(T, Hk, D)
        st["w_q"] = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
        st["w_k"] = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
        rows = max(T, 8192)
        st["cos"], st["sin"] = _rotary(rows, case["R"])
        st["pos"] = None
        if case["gather"]:  # decode: unrelated positions; prefill: sequences of ordered ones
            start = torch.randint(0, rows, (max(1, T // 4096 if T >= 4096 else T),), generator=g, device="cuda")
            st["pos"] = ((start.repeat_interleave(-(-T // start.numel()))[:T] + torch.arange(T, device="cuda")) % rows).int()
        st["q_out"] = torch.empty(T, Hq, D, dtype=bf, device="cuda")
        st["k_out"] = torch.empty(T, Hk, D, dtype=bf, device="cuda")
        return st
    if op == "kv_append":
        T, H, D, page = case["T"], case["H"], case["D"], case["page"]
        x = (1.5 * torch.randn(T, 2 * H * D, generator=g, device="cuda")).to(bf)
        st["k"] = x[:, : H * D].view(T, H, D)
        st["v"] = x[:, H * D :].view(T, H, D)
        st["w_k"] = 1 + 0.1 * torch.randn(D, generator=g, device="cuda") if case["norm"] else None
        rows = max(T, 8192)
        st["cos"], st["sin"] = _rotary(rows, case["R"])
        pages = -(-max(T + T // 4, 2048) // page)
        st["k_cache"] = torch.randn(pages, H, page, D, generator=g, device="cuda").to(bf)
        st["v_cache"] = torch.randn(pages, H, page, D, generator=g, device="cuda").to(bf)
        order = torch.randperm(pages, generator=g, device="cuda")
        if T >= 1024:  # a prompt: consecutive places of shuffled pages
            i = torch.arange(T, device="cuda")
            st["slot"] = order[i // page] * page + i % page
            st["pos"] = i.int()
        else:  # one token of each sequence: a place of a page of its own where there are enough
            i = torch.randperm(pages * page, generator=g, device="cuda")[:T]
            st["slot"] = order[i // page] * page + i % page
            st["pos"] = torch.randint(0, rows, (T,), generator=g, device="cuda").int()
        return st
    B, n_q, Hk, G, D, page = (case[n] for n in ("B", "n_q", "Hk", "G", "D", "page"))
    prefix_pages = -(-case["prefix"] // page)
    suffix_pages = -(-case["suffix"] // page)
    pages = prefix_pages + B * suffix_pages
    st["q"] = torch.randn(B * n_q, Hk * G, D, generator=g, device="cuda").to(bf)
    st["k_cache"] = torch.empty(pages, Hk, page, D, dtype=bf, device="cuda").normal_(generator=g)
    st["v_cache"] = torch.empty(pages, Hk, page, D, dtype=bf, device="cuda").normal_(generator=g)
    order = torch.randperm(pages, generator=g, device="cuda").int()
    st["prefix_table"] = order[:prefix_pages].contiguous()
    st["tables"] = order[prefix_pages:].view(B, suffix_pages).contiguous()
    # the suffix holds the query tokens themselves; its length differs from sequence to sequence
    st["lens"] = torch.randint(min(n_q, case["suffix"]), case["suffix"] + 1, (B,), generator=g, device="cuda").int()
    st["scale"] = 1 / math.sqrt(D)
    st["o"] = torch.empty(B * n_q, Hk * G, D, dtype=bf, device="cuda")
    st["lse"] = torch.empty(B * n_q, Hk * G, device="cuda")
    return st


# ------------------------------------------------------------ plain forms --
def _norm_plain(x, w):
    if w is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def _rope_plain(x, cos, sin, interleaved):
    half = cos.shape[-1]
    c, s = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0 : 2 * half : 2], x[..., 1 : 2 * half : 2]
        y = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half : 2 * half]
        y = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((y, x[..., 2 * half :]), -1)


def _run_plain(st):
    op = st["op"]
    bf = torch.bfloat16
    if op == "gemm_w8a8":
        y = torch.matmul(st["qa"].float(), st["w"].float().t()) * st["a_scale"][:, None] * st["w_scale"]
        if st["mean"] is not None:
            y = y + st["mean"][:, None] * st["w1"]
        if st["bias_v"] is not None:
            y = y + st["bias_v"]
        return y.to(bf)
    if op == "qk_norm_rope":
        T = st["T"]
        cos, sin = (t[:T] if st["pos"] is None else t[st["pos"]] for t in (st["cos"], st["sin"]))
        q = _rope_plain(_norm_plain(st["q"].float(), st["w_q"]), cos, sin, st["interleaved"]).to(bf)
        k = _rope_plain(_norm_plain(st["k"].float(), st["w_k"]), cos, sin, st["interleaved"]).to(bf)
        return q, k
    if op == "kv_append":
        k = _rope_plain(_norm_plain(st["k"].float(), st["w_k"]), st["cos"][st["pos"]], st["sin"][st["pos"]], st["interleaved"])
        at, off = st["slot"] // st["page"], st["slot"] % st["page"]
        st["k_cache"][at, :, off] = k.to(bf)
        st["v_cache"][at, :, off] = st["v"]
        return st["k_cache"], st["v_cache"]
    B, n_q, Hk, G, D, P = (st[n] for n in ("B", "n_q", "Hk", "G", "D", "prefix"))
    q = st["q"].float().view(B, n_q, Hk, G, D) * st["scale"]
    # the prefix: all rows of a key head against the one copy of its keys
    kp = st["k_cache"][st["prefix_table"]].float().transpose(0, 1).reshape(Hk, -1, D)[:, :P]
    vp = st["v_cache"][st["prefix_table"]].float().transpose(0, 1).reshape(Hk, -1, D)[:, :P]
    sp = torch.matmul(q.permute(2, 0, 1, 3, 4).reshape(Hk, B * n_q * G, D), kp.transpose(1, 2))
    # the suffixes: each sequence's own pages, up to each query token's own place
    ks = st["k_cache"][st["tables"]].float().transpose(1, 2).reshape(B, Hk, -1, D)
    vs = st["v_cache"][st["tables"]].float().transpose(1, 2).reshape(B, Hk, -1, D)
    ss = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(B, Hk, n_q * G, D), ks.transpose(2, 3))
    L = ss.shape[-1]
    seen = st["lens"][:, None] - n_q + 1 + torch.arange(n_q, device="cuda")  # [B][n_q]
    hidden = torch.arange(L, device="cuda") >= seen[:, :, None]
    ss = ss.view(B, Hk, n_q, G, L).masked_fill_(hidden[:, None, :, None], float("-inf")).view(B, Hk, n_q * G, L)
    sp = sp.view(Hk, B, n_q * G, P).transpose(0, 1)
    m = torch.maximum(sp.amax(-1), ss.amax(-1))[..., None]
    sp = torch.exp(sp - m)
    ss = torch.exp(ss - m)
    total = (sp.sum(-1) + ss.sum(-1))[..., None]
    o = torch.matmul(sp.transpose(0, 1).reshape(Hk, B * n_q * G, P), vp).view(Hk, B, n_q * G, D).transpose(0, 1)
    o = (o + torch.matmul(ss, vs)) / total
    lse = m + torch.log(total)
    back = lambda t: t.view(B, Hk, n_q, G, -1).transpose(1, 2).reshape(B * n_q, Hk * G, -1)  # noqa: E731
    return back(o).to(bf), back(lse)[..., 0]


# ------------------------------------------------------- this repository's --
def _run_own(st):
    import rotated_bit_quantized_amd as oq

    op = st["op"]
    if op == "gemm_w8a8":
        return oq.oq_gemm_w8a8(st["qa"], st["a_scale"], st["w"], st["w_scale"], mean=st["mean"], w1=st["w1"], bias=st["bias_v"],
                               y=st["y"])
    if op == "attn_prefix":
        if "cache" not in st:  # the handle and the workspace that a serving loop keeps
            st["cache"] = oq.PagedKV(st["k_cache"], st["v_cache"])
            st["ws"] = torch.empty(oq.oq_attn_prefix_ws_bytes(st["B"], st["n_q"], st["Hk"] * st["G"], st["cache"], st["prefix"],
                                                              st["tables"].shape[1]), dtype=torch.uint8, device="cuda")
        return oq.oq_attn_prefix(st["q"], st["n_q"], st["cache"], st["prefix_table"], st["prefix"], st["tables"], st["lens"],
                                 st["scale"], o=st["o"], lse=st["lse"], ws=st["ws"])
    if "rope" not in st:
        st["rope"] = oq.Rope(st["cos"], st["sin"], st["interleaved"])
    if op == "qk_norm_rope":
        return oq.oq_qk_norm_rope(st["q"], st["k"], st["w_q"], st["w_k"], EPS, st["rope"], st["pos"], q_out=st["q_out"],
                                  k_out=st["k_out"])
    if "cache" not in st:
        st["cache"] = oq.PagedKV(st["k_cache"], st["v_cache"])
    oq.oq_kv_append(st["k"], st["v"], st["slot"], st["cache"], w_k=st["w_k"], eps=EPS, rope=st["rope"], pos=st["pos"])
    return st["k_cache"], st["v_cache"]


def run(st):
    return _run_own(st) if own else _run_plain(st)


# ------------------------------------------------------------------- work --
def work(case):
    op = case["op"]
    if op == "gemm_w8a8":
        M, K, N = case["M"], case["K"], case["N"]
        vectors = M + N + (M + N if case["center"] else 0) + (N if case["bias"] else 0)
        return {"bytes": M * K + N * K + 2 * M * N + 4 * vectors, "flops": 2 * M * N * K}
    if op == "qk_norm_rope":
        T, D, R = case["T"], case["D"], case["R"]
        n = T * (case["Hq"] + case["Hk"]) * D
        return {"bytes": 4 * n + 4 * T * R + (4 * T if case["gather"] else 0) + 8 * D, "flops": 8 * n}
    if op == "kv_append":
        T, D, R = case["T"], case["D"], case["R"]
        n = T * case["H"] * D
        return {"bytes": 8 * n + 4 * T * R + 12 * T + (4 * D if case["norm"] else 0), "flops": (8 if case["norm"] else 4) * n}
    B, n_q, Hk, G, D = (case[n] for n in ("B", "n_q", "Hk", "G", "D"))
    mean_len = (min(n_q, case["suffix"]) + case["suffix"]) / 2
    rows = B * n_q * Hk * G
    kv = 4 * Hk * D * (case["prefix"] + B * mean_len)
    return {"bytes": kv + 4 * rows * D + 4 * rows, "flops": 4 * rows * D * (case["prefix"] + mean_len - (n_q - 1) / 2)}


# ------------------------------------------------------------------ exact --
def _turned(x, w, cos, sin, R, interleaved):
    """float64 norm and rotation of x [T][H][D]; a rotary pair is a complex number that the position turns."""
    x = x.double()
    if w is not None:
        x = w.double() * x / ((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()
    turn = torch.complex(cos.double(), sin.double())[:, None, :]
    if interleaved:
        z = torch.view_as_complex(x[..., :R].unflatten(-1, (R // 2, 2)).contiguous()) * turn
        y = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(x[..., : R // 2], x[..., R // 2 : R]) * turn
        y = torch.cat((z.real, z.imag), -1)
    out = x.clone()
    out[..., :R] = y
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "gemm_w8a8":
        wt = st["w"].double().t()
        out = torch.empty(case["M"], case["N"], dtype=torch.float64, device="cuda")
        for r in range(0, case["M"], 2048):  # int8 products and their sums are whole numbers below 2^53
            rows = slice(r, r + 2048)
            y = st["a_scale"][rows].double()[:, None] * ((st["qa"][rows].double() @ wt) * st["w_scale"].double())
            if case["center"]:
                y += torch.outer(st["mean"][rows].double(), st["w1"].double())
            if case["bias"]:
                y += st["bias_v"].double()
            out[rows] = y
        return out
    if op == "qk_norm_rope":
        at = torch.arange(case["T"], device="cuda") if st["pos"] is None else st["pos"].long()
        cos, sin = st["cos"][at], st["sin"][at]
        return (_turned(st["q"], st["w_q"], cos, sin, case["R"], case["interleaved"]),
                _turned(st["k"], st["w_k"], cos, sin, case["R"], case["interleaved"]))
    if op == "kv_append":
        at = st["pos"].long()
        k = _turned(st["k"], st["w_k"], st["cos"][at], st["sin"][at], case["R"], case["interleaved"])
        got = []
        for cache, new in ((st["k_cache"], k), (st["v_cache"], st["v"].double())):
            pages, H, page, D = cache.shape
            flat = cache.double().transpose(1, 2).reshape(pages * page, H, D)  # one row a slot
            flat[st["slot"]] = new
            got.append(flat.view(pages, page, H, D).transpose(1, 2).contiguous())
        return tuple(got)
    B, n_q, Hk, G, D, P, page = (case[n] for n in ("B", "n_q", "Hk", "G", "D", "prefix", "page"))
    o = torch.empty(B * n_q, Hk * G, D, dtype=torch.float64, device="cuda")
    lse = torch.empty(B * n_q, Hk * G, dtype=torch.float64, device="cuda")
    lens, width = st["lens"].tolist(), st["tables"].shape[1] * page
    for h in range(Hk):
        heads = slice(h * G, (h + 1) * G)
        shared = [c[st["prefix_table"].long(), h].reshape(-1, D)[:P].double() for c in (st["k_cache"], st["v_cache"])]
        for b0 in range(0, B, 32):  # one softmax over prefix and suffix together, some sequences at a time
            nb = min(32, B - b0)
            q = st["q"].view(B, n_q, Hk * G, D)[b0 : b0 + nb, :, heads].double().reshape(nb, n_q * G, D)
            mine = [c[st["tables"][b0 : b0 + nb].long(), h].reshape(nb, width, D).double() for c in (st["k_cache"], st["v_cache"])]
            s = torch.empty(nb, n_q * G, P + width, dtype=torch.float64, device="cuda")
            s[:, :, :P] = (q.reshape(-1, D) @ shared[0].t()).view(nb, n_q * G, P)
            s[:, :, P:] = torch.bmm(q, mine[0].transpose(1, 2).contiguous())
            s *= st["scale"]
            for b in range(nb):
                for i in range(n_q):
                    s[b, i * G : (i + 1) * G, P + max(0, lens[b0 + b] - n_q + 1 + i) :] = -math.inf
            z = torch.logsumexp(s, -1)
            p = torch.exp(s - z[..., None])
            y = (p[:, :, :P].reshape(-1, P) @ shared[1]).view(nb, n_q * G, D) + torch.bmm(p[:, :, P:].contiguous(), mine[1])
            o.view(B, n_q, Hk * G, D)[b0 : b0 + nb, :, heads] = y.view(nb, n_q, G, D)
            lse.view(B, n_q, Hk * G)[b0 : b0 + nb, :, heads] = z.view(nb, n_q, G)
    return o, lse
