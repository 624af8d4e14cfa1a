"""Workloads of the operators that complete a quantized sparse layer and answer with it.

Four operators, in the order in which a serving step of a mixture-of-experts
transformer runs them:

- ``route``: scores of every token for every expert (softmax or sigmoid, with
  a balance bias and groups), its best experts, their weights, and the lists
  of entries by expert that the products read;
- ``experts``: the experts' int8 products, each entry with its own expert's
  weights, with the SwiGLU of an up projection as epilogue;
- ``residual_norm``: the weighted sum over a token's experts (or the plain
  output of a block), norms after and before a block, gate, residual and
  modulation in one pass;
- ``logprobs``: log probabilities of given tokens, their ranks, the entropy
  and the best alternatives of a row of logits.

``own`` selects between the plain form of an operator (elementary torch
operations in float32, in float64 where neighbouring scores decide a choice)
and this repository's entry points.
"""
import math

import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one new token through a softmax router, eight of 128 experts: latency
        dict(name="route one token", op="route", T=1, E=128, k=8, score="softmax", bias=False, groups=1, top_groups=1, best=1, renorm=True,
             factor=1.0, dtype="f32"),
        # a ragged batch through a sigmoid router with a balance bias, eight groups of which four are open
        dict(name="route 333 tokens in groups", op="route", T=333, E=256, k=8, score="sigmoid", bias=True, groups=8, top_groups=4, best=2,
             renorm=True, factor=2.5, dtype="f32"),
        # a long prefill, bfloat16 logits as a projection leaves them
        dict(name="route prefill 32768", op="route", T=32768, E=128, k=8, score="softmax", bias=False, groups=1, top_groups=1, best=1,
             renorm=True, factor=1.0, dtype="bf16"),
        # one decode step of 16 sequences: gate and up projection of the few experts that they reach
        dict(name="experts decode 16", op="experts", T=16, E=128, k=8, K=2048, N=1536, act=True, down=False, bias=False, center=False),
        # an odd batch through the down projections of a smaller layer, centred and biased
        dict(name="experts down 1003", op="experts", T=1003, E=60, k=4, K=1408, N=2048, act=False, down=True, bias=True, center=True),
        # a full prefill through the gate and up projections
        dict(name="experts prefill 8192", op="experts", T=8192, E=128, k=8, K=2048, N=1536, act=True, down=False, bias=False, center=False),
        # one decode step of 64 sequences: the sum over eight experts, residual and the next norm
        dict(name="norm decode 64", op="residual_norm", T=64, d=2048, k=8, post="none", pre="rms", gate=False, mod=False, tokens=1, res="bf16"),
        # a diffusion transformer's images, 1920 wide: gated block output, layer norm and modulation, a row of both per image
        dict(name="norm images 4100", op="residual_norm", T=4100, d=1920, k=1, post="none", pre="layer", gate=True, mod=True, tokens=1025,
             res="f32"),
        # a long prefill of a 4096-wide LLM layer, norms on both sides of the block
        dict(name="norm prefill 32768", op="residual_norm", T=32768, d=4096, k=1, post="rms", pre="rms", gate=False, mod=False, tokens=1,
             res="bf16"),
        # the token that a single sequence has just drawn, twenty alternatives
        dict(name="logprobs one token", op="logprobs", T=1, V=32000, n=1, top=20, scale=1.0, dtype="f32"),
        # a ragged batch of draft tokens, two candidates each, odd vocabulary, a temperature
        dict(name="logprobs 77 x 2", op="logprobs", T=77, V=100003, n=2, top=5, scale=1.25, dtype="bf16"),
        # prompts scored token by token
        dict(name="logprobs 2048 prompt", op="logprobs", T=2048, V=131072, n=1, top=5, scale=1.0, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "experts", "residual_norm", "logprobs"])
    while True:
        if op == "route":
            groups = rng.choice([1, 1, 2, 4, 8])
            best = rng.choice([1, 2])
            each = _log(rng, max(best, -(-8 // groups)), 512 // groups)
            top_groups = rng.randint(1, groups)
            c = dict(op=op, T=_log(rng, 1, 32768), E=groups * each, k=rng.randint(1, min(10, top_groups * each)),
                     score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups, top_groups=top_groups, best=best,
                     renorm=rng.random() < 0.7, factor=rng.choice([1.0, 2.5]), dtype=rng.choice(["f32", "bf16"]))
            if c["T"] * c["E"] * (4 if c["dtype"] == "f32" else 2) <= 32768 * 128 * 2 and c["T"] * c["k"] <= 32768 * 8:
                return c
        elif op == "experts":
            E = rng.choice([8, 16, 60, 64, 128])
            act = rng.random() < 0.5
            c = dict(op=op, T=_log(rng, 1, 8192), E=E, k=rng.randint(1, 8), K=16 * _log(rng, 16, 256), N=2 * _log(rng, 32, 2048), act=act,
                     down=not act and rng.random() < 0.7, bias=rng.random() < 0.3, center=rng.random() < 0.3)
            if c["T"] * c["k"] * c["K"] * c["N"] <= 65536 * 2048 * 1536 and E * c["K"] * c["N"] <= 128 * 2048 * 1536:
                return c
        elif op == "residual_norm":
            c = dict(op=op, T=_log(rng, 1, 32768), d=8 * _log(rng, 8, 2048), k=rng.choice([1, 1, 1, 2, 4, 6, 8]),
                     post=rng.choice(["none", "none", "rms", "layer"]), pre=rng.choice(["none", "rms", "rms", "layer"]),
                     gate=rng.random() < 0.4, mod=rng.random() < 0.4, tokens=_log(rng, 1, 4096), res=rng.choice(["bf16", "f32"]))
            if c["T"] * (c["k"] + (3 if c["res"] == "bf16" else 5)) * c["d"] <= 32768 * 4 * 4096:
                return c
        else:
            c = dict(op=op, T=_log(rng, 1, 4096), V=_log(rng, 500, 262144), n=rng.choice([1, 1, 2, 5]), top=rng.choice([0, 1, 5, 20]),
                     scale=rng.choice([1.0, 1.25, 0.7]), dtype=rng.choice(["f32", "bf16"]))
            if c["T"] * c["V"] * (4 if c["dtype"] == "f32" else 2) <= 2048 * 131072 * 2:
                return c


# ----------------------------------------------------------------- inputs --
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _codes8(v):
    """Rows as absmax int8 codes and their scales."""
    scale = v.abs().amax(-1).clamp_min(1e-10) / 127
    return torch.round(v / scale[..., None]).clamp_(-127, 127).to(torch.int8), scale


def _type(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _lists(ids, E):
    """Entries (token times k plus choice) by expert, and where each expert's begin."""
    flat = ids.flatten().long()
    order = torch.sort(flat, dim=0, stable=True).indices
    count = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    count[1:] = torch.bincount(flat, minlength=E)
    return torch.cumsum(count, 0).int(), order.int()


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    op = case["op"]
    bf = torch.bfloat16
    T = case["T"]
    if op == "route":
        E, k = case["E"], case["k"]
        # some experts are liked by all tokens, as in a model whose balance the bias has to hold
        liked = 0.5 * _randn(g, E)
        st["logits"] = (1.5 * _randn(g, T, E) + liked).to(_type(case["dtype"]))
        st["bias_v"] = -0.1 * liked + 0.02 * _randn(g, E) if case["bias"] else None
        st["ids"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
        st["weights"] = torch.empty(T, k, device="cuda")
        st["offsets"] = torch.empty(E + 1, dtype=torch.int32, device="cuda")
        st["order"] = torch.empty(T * k, dtype=torch.int32, device="cuda")
        return st
    if op == "experts":
        E, k, K, N = (case[n] for n in ("E", "k", "K", "N"))
        ids = torch.topk(_randn(g, T, E) + 0.5 * _randn(g, E), k, dim=1).indices
        st["offsets"], st["order_v"] = _lists(ids, E)
        rows = T * k if case["down"] else T  # an up projection's entries share their token's row
        st["qa"], st["a_scale"] = _codes8(_randn(g, rows, K))
        st["w"] = torch.empty(E, N, K, dtype=torch.int8, device="cuda")
        st["w_scale"] = torch.empty(E, N, device="cuda")
        for e in range(E):
            st["w"][e], st["w_scale"][e] = _codes8(0.02 * _randn(g, N, K))
        st["bias_v"] = 0.5 * _randn(g, E, N) if case["bias"] else None
        st["mean"] = 0.3 * _randn(g, rows) if case["center"] else None
        st["w1"] = _randn(g, E, N) if case["center"] else None
        st["y"] = torch.empty(T * k, N // 2 if case["act"] else N, dtype=bf, device="cuda")
        return st
    if op == "residual_norm":
        d, k = case["d"], case["k"]
        st["y"] = (1.5 * _randn(g, T * k, d)).to(bf)
        st["mix"] = torch.softmax(_randn(g, T, k), 1) if k > 1 else None
        st["r"] = (3 * _randn(g, T, d) + 0.2).to(_type(case["res"]))
        st["w_post"] = 1 + 0.1 * _randn(g, d) if case["post"] != "none" else None
        st["w_pre"] = 1 + 0.1 * _randn(g, d) if case["pre"] != "none" and not case["mod"] else None
        images = -(-T // case["tokens"])
        # one projection gives shift, scale and gate of an image side by side
        table = (0.3 * _randn(g, images, 3 * d)).to(bf)
        st["shift"], st["scale"] = (table[:, :d], table[:, d : 2 * d]) if case["mod"] else (None, None)
        st["gate_v"] = table[:, 2 * d :] if case["gate"] else None
        st["row"] = (torch.arange(T, device="cuda") // case["tokens"]).int()
        st["r_out"] = torch.empty_like(st["r"])
        st["h"] = torch.empty(T, d, dtype=bf, device="cuda")
        return st
    V, n = case["V"], case["n"]
    logits = 2 * _randn(g, T, V)
    st["tokens"] = torch.randint(0, V, (T, n), generator=g, device="cuda", dtype=torch.int32)
    # what a model finds likely, from hardly to nearly certain
    logits.scatter_add_(1, st["tokens"].long(), 16 * torch.rand(T, n, generator=g, device="cuda"))
    st["logits"] = logits.to(_type(case["dtype"]))
    return st


# ------------------------------------------------------------ plain forms --
def _scores(x, score):
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    e = torch.exp(x - x.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _route_plain(st):
    """float64 throughout: neighbouring scores decide who is chosen."""
    x = st["logits"].double()
    T, E = x.shape
    G, k = st["groups"], st["k"]
    s = _scores(x, st["score"])
    sel = x if st["bias_v"] is None else s + st["bias_v"].double()
    if G > 1:
        by = (s if st["bias_v"] is None and st["best"] == 2 else sel).view(T, G, E // G)
        group = torch.sort(by, dim=2, descending=True).values[:, :, : st["best"]].sum(2)
        keep = torch.sort(group, dim=1, descending=True, stable=True).indices[:, : st["top_groups"]]
        open_ = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, keep, True)
        sel = sel.masked_fill(~open_.repeat_interleave(E // G, 1), -math.inf)
    ids = torch.sort(sel, dim=1, descending=True, stable=True).indices[:, :k]
    w = s.gather(1, ids)
    if st["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return (ids.int(), (w * st["factor"]).float()) + _lists(ids, E)


def _experts_plain(st):
    y = st["y"]
    at = st["offsets"].tolist()
    for e in range(st["E"]):
        if at[e] == at[e + 1]:
            continue
        entry = st["order_v"][at[e] : at[e + 1]].long()
        row = entry if st["down"] else entry // st["k"]
        v = torch.matmul(st["qa"][row].float(), st["w"][e].float().t()) * st["a_scale"][row][:, None] * st["w_scale"][e]
        if st["mean"] is not None:
            v = v + st["mean"][row][:, None] * st["w1"][e]
        if st["bias_v"] is not None:
            v = v + st["bias_v"][e]
        if st["act"]:
            gate, up = v.chunk(2, 1)
            v = gate / (1 + torch.exp(-gate)) * up
        y[entry] = v.to(y.dtype)
    return y


def _norm_plain(x, kind, w):
    if kind == "none":
        return x
    if kind == "layer":
        x = x - x.mean(1, keepdim=True)
    x = x * torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
    return x if w is None else x * w


def _residual_norm_plain(st):
    T, d, k = st["T"], st["d"], st["k"]
    u = st["y"].float()
    if k > 1:
        u = (u.view(T, k, d) * st["mix"][:, :, None]).sum(1)
    u = _norm_plain(u, st["post"], st["w_post"])
    if st["gate_v"] is not None:
        u = u * st["gate_v"].float()[st["row"]]
    r = st["r"].float() + u
    h = _norm_plain(r, st["pre"], st["w_pre"])
    if st["scale"] is not None:
        h = h * (1 + st["scale"].float()[st["row"]]) + st["shift"].float()[st["row"]]
    return r.to(st["r"].dtype), h.to(torch.bfloat16)


def _keys(logits):
    """Whole numbers in the order of the logits, equal ones in the order of falling index."""
    bits = (logits.float() + 0.0).view(torch.int32).long()
    up = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
    V = logits.shape[1]
    return up * (1 << 20) + (V - 1 - torch.arange(V, device=logits.device))


def _logprobs_plain(st):
    x = st["logits"].float() * st["scale"]
    tok = st["tokens"].long()
    z = x - x.amax(1, keepdim=True)
    e = torch.exp(z)
    total = e.sum(1, keepdim=True)
    log_total = torch.log(total)
    entropy = log_total[:, 0] - (e * z).sum(1) / total[:, 0]
    lse = x.amax(1) + log_total[:, 0]
    keys = _keys(st["logits"])
    mine = keys.gather(1, tok)
    rank = torch.stack([(keys > mine[:, i : i + 1]).sum(1) for i in range(tok.shape[1])], 1).int()
    top = torch.topk(keys, st["top"], dim=1).indices
    return z.gather(1, tok) - log_total, rank, entropy, lse, top.int(), z.gather(1, top) - log_total


# ------------------------------------------------------- this repository's --
def _run_own(st):
    import rotated_bit_quantized_amd as oq

    op = st["op"]
    if op == "route":
        if "router" not in st:  # the handle and the workspace that a serving loop keeps
            st["router"] = oq.Router(st["E"], st["k"], score=st["score"], bias=st["bias_v"], groups=st["groups"],
                                     top_groups=st["top_groups"], group_best=st["best"], renorm=st["renorm"], factor=st["factor"])
            st["ws"] = torch.empty(oq.oq_route_ws_bytes(st["T"], st["router"]), dtype=torch.uint8, device="cuda")
        return oq.oq_route(st["logits"], st["router"], ids=st["ids"], weights=st["weights"], offsets=st["offsets"], order=st["order"],
                           ws=st["ws"])
    if op == "experts":
        return oq.oq_gemm_w8a8_experts(st["qa"], st["a_scale"], st["w"], st["w_scale"], st["offsets"], st["order_v"],
                                       per=1 if st["down"] else st["k"], act=oq.OQ_ACT_SWIGLU if st["act"] else oq.OQ_ACT_NONE,
                                       mean=st["mean"], w1=st["w1"], bias=st["bias_v"], y=st["y"])
    if op == "residual_norm":
        if "norms" not in st:  # the descriptors that a layer keeps
            kinds = {"none": None, "rms": oq.OQ_NORM_RMS, "layer": oq.OQ_NORM_LAYER}
            st["norms"] = [None if kinds[st[n]] is None else oq.Norm(kinds[st[n]], st["d"], EPS, st["w_" + n]) for n in ("post", "pre")]
        return oq.oq_residual_norm(st["y"], st["r"], weights=st["mix"], post=st["norms"][0], pre=st["norms"][1], gate=st["gate_v"],
                                   scale=st["scale"], shift=st["shift"], row=st["row"], r_out=st["r_out"], h=st["h"])
    if "ws" not in st:
        st["ws"] = torch.empty(oq.oq_logprobs_ws_bytes(st["T"], st["V"], st["n"], st["top"]), dtype=torch.uint8, device="cuda")
    return oq.oq_logprobs(st["logits"], st["tokens"], top=st["top"], scale=st["scale"], ws=st["ws"])


def run(st):
    if own:
        return _run_own(st)
    return {"route": _route_plain, "experts": _experts_plain, "residual_norm": _residual_norm_plain,
            "logprobs": _logprobs_plain}[st["op"]](st)


# ------------------------------------------------------------------- work --
def work(case):
    op, T = case["op"], case["T"]
    if op == "route":
        n, E = T * case["k"], case["E"]
        return {"bytes": T * E * (4 if case["dtype"] == "f32" else 2) + 12 * n + 4 * (E + 1) + (4 * E if case["bias"] else 0),
                "flops": 6 * T * E}
    if op == "experts":
        E, n, K, N = case["E"], T * case["k"], case["K"], case["N"]
        rows = n if case["down"] else T
        reached = E * (1 - (1 - case["k"] / E) ** T)  # experts that have an entry, on average
        vectors = reached * N * (1 + (1 if case["bias"] else 0) + (1 if case["center"] else 0)) + rows * (2 if case["center"] else 1)
        return {"bytes": int(reached * N * K + rows * K + 4 * vectors + n * N * (1 if case["act"] else 2) + 4 * (n + E)),
                "flops": 2 * n * N * K}
    if op == "residual_norm":
        d, k = case["d"], case["k"]
        images = -(-T // case["tokens"])
        table = 2 * images * d * ((1 if case["gate"] else 0) + (2 if case["mod"] else 0))
        vectors = 4 * d * ((case["post"] != "none") + (case["pre"] != "none" and not case["mod"]))
        return {"bytes": T * d * (2 * k + 2 * (4 if case["res"] == "f32" else 2) + 2) + (4 * T * k if k > 1 else 0) + table + vectors
                + (4 * T if table else 0), "flops": T * d * (2 * k + 10)}
    V, n, top = case["V"], case["n"], case["top"]
    return {"bytes": T * V * (4 if case["dtype"] == "f32" else 2) + T * (12 * n + 8 + 8 * top), "flops": 6 * T * V}


# ------------------------------------------------------------------ exact --
def _exact_route(st):
    x = st["logits"].double()
    T, E = x.shape
    G, k = st["groups"], st["k"]
    s = torch.sigmoid(x) if st["score"] == "sigmoid" else torch.softmax(x, 1)
    sel = x if st["bias_v"] is None else s + st["bias_v"]
    allowed = torch.ones(T, G, dtype=torch.bool, device=x.device)
    if G > 1:
        each = (s if st["bias_v"] is None and st["best"] == 2 else sel).unflatten(1, (G, E // G))
        first = each.amax(2)
        group = first if st["best"] == 1 else first + torch.topk(each, 2, 2).values[:, :, 1]
        allowed[:] = False
        for _ in range(st["top_groups"]):  # the best group still closed, the lowest number of equal ones
            g = group.masked_fill(allowed, -math.inf)
            allowed |= torch.arange(G, device=x.device) == (g == g.amax(1, keepdim=True)).int().argmax(1)[:, None]
    left = sel.unflatten(1, (G, E // G)).masked_fill(~allowed[:, :, None], -math.inf).flatten(1)
    ids = torch.empty(T, k, dtype=torch.int64, device=x.device)
    for j in range(k):
        first = (left == left.amax(1, keepdim=True)).int().argmax(1)
        ids[:, j] = first
        left.scatter_(1, first[:, None], -math.inf)
    w = torch.gather(s, 1, ids)
    if st["renorm"]:
        if st["score"] == "softmax":  # the softmax of the chosen alone
            w = torch.softmax(torch.gather(x, 1, ids), 1)
        else:
            w = w / w.sum(1, keepdim=True)
    host = ids.flatten().tolist()
    at = sorted(range(T * k), key=host.__getitem__)
    starts, seen = [0] * (E + 1), [0] * E
    for e in host:
        seen[e] += 1
    for e in range(E):
        starts[e + 1] = starts[e] + seen[e]
    new = lambda v: torch.tensor(v, dtype=torch.int32, device=x.device)  # noqa: E731
    return ids.int(), w * st["factor"], new(starts), new(at)


def exact(case, seed):
    st = prepare(case, seed)
    op, T = case["op"], case["T"]
    if op == "route":
        return _exact_route(st)
    if op == "experts":
        n, N = T * case["k"], case["N"]
        out = torch.empty(n, N, dtype=torch.float64, device="cuda")
        at = st["offsets"].tolist()
        for e in range(case["E"]):  # int8 products and their sums are whole numbers below 2^53
            mine = st["order_v"][at[e] : at[e + 1]].long()
            rows = mine if case["down"] else torch.div(mine, case["k"], rounding_mode="floor")
            v = torch.outer(st["a_scale"][rows].double(), st["w_scale"][e].double()) * (st["qa"][rows].double() @ st["w"][e].double().t())
            if case["center"]:
                v += torch.outer(st["mean"][rows].double(), st["w1"][e].double())
            if case["bias"]:
                v += st["bias_v"][e].double()
            out[mine] = v
        if case["act"]:
            return torch.sigmoid(out[:, : N // 2]) * out[:, : N // 2] * out[:, N // 2 :]
        return out
    if op == "residual_norm":
        d, k = case["d"], case["k"]
        r_out = torch.empty(T, d, dtype=torch.float64, device="cuda")
        h_out = torch.empty(T, d, dtype=torch.float64, device="cuda")

        def norm(x, kind, w):
            if kind == "none":
                return x
            centre = x.mean(1, keepdim=True) if kind == "layer" else 0.0
            x = (x - centre) / torch.sqrt(((x - centre) ** 2).sum(1, keepdim=True) / d + EPS)
            return x if w is None else w.double() * x

        for t in range(0, T, 4096):
            rows = slice(t, min(T, t + 4096))
            y = st["y"].view(T, k, d)[rows].double()
            u = y[:, 0] if k == 1 else (st["mix"][rows].double()[:, :, None] * y).sum(1)
            u = norm(u, case["post"], st["w_post"])
            image = st["row"][rows].long()
            if case["gate"]:
                u = st["gate_v"][image].double() * u
            r = st["r"][rows].double() + u
            h = norm(r, case["pre"], st["w_pre"])
            if case["mod"]:
                h = h + h * st["scale"][image].double() + st["shift"][image].double()
            r_out[rows], h_out[rows] = r, h
        return r_out, h_out
    tok, top, V = st["tokens"].long(), case["top"], case["V"]
    got = [[] for _ in range(6)]
    for t in range(0, T, 256):
        raw = st["logits"][t : t + 256]
        x = raw.double()
        logp = torch.log_softmax(x * case["scale"], 1)
        mine = tok[t : t + 256]
        lower = torch.arange(V, device="cuda")
        rank = [((x > x.gather(1, mine[:, i : i + 1])) | ((x == x.gather(1, mine[:, i : i + 1])) & (lower < mine[:, i : i + 1]))).sum(1)
                for i in range(mine.shape[1])]
        ids = torch.empty(len(x), top, dtype=torch.int64, device="cuda")
        left = x.clone()
        for j in range(top):
            first = (left == left.amax(1, keepdim=True)).int().argmax(1)
            ids[:, j] = first
            left.scatter_(1, first[:, None], -math.inf)
        parts = (logp.gather(1, mine), torch.stack(rank, 1).int(), -(logp.exp() * logp).sum(1), torch.logsumexp(x * case["scale"], 1),
                 ids.int(), logp.gather(1, ids))
        for g, p in zip(got, parts):
            g.append(p)
    return tuple(torch.cat(g) for g in got)
