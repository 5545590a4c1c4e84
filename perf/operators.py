"""Top-k routing and 8-bit integer products: what is measured of them.

Four operators: ``route_topk`` (scores, balance bias, groups, top-k, renormalised
weights from router logits), ``route_topk_backward`` (its gradient), ``int8_linear``
(a product in 8-bit integers with a scale for each token and output channel) and
``forward_int8`` (the expert sum of the layer with both expert products in 8-bit
integers).  With ``own`` false ``run`` computes their plain forms.
"""
import math

import torch

own = False


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one decoded token: every microsecond is latency
        dict(name="route_one_token", op="route", T=1, E=256, k=8, scores="sigmoid", bias=True, n_group=8,
             topk_group=4, renorm=True, scale=2.5, dtype="f32", padded=False),
        # a batch of verification chunks with a ragged end, plain softmax weights of bf16 logits, some rows
        # padding (no expert allowed)
        dict(name="route_batch", op="route", T=509, E=64, k=6, scores="softmax", bias=False, n_group=1,
             topk_group=1, renorm=False, scale=1.0, dtype="bf16", padded=True),
        # a long prefill over many experts, chosen by biased sigmoid scores inside the best groups
        dict(name="route_long", op="route", T=32749, E=256, k=8, scores="sigmoid", bias=True, n_group=8,
             topk_group=4, renorm=True, scale=2.5, dtype="f32", padded=False),
        # the gradient at a training sequence of 4096 tokens over 64 experts
        dict(name="grad_seq4096", op="grad", T=4096, E=64, k=8, scores="softmax", renorm=False, scale=1.0,
             dtype="bf16", padded=True),
        # and over a long batch with many experts
        dict(name="grad_long", op="grad", T=16381, E=256, k=8, scores="sigmoid", renorm=True, scale=2.5,
             dtype="f32", padded=False),
        # one token through a dense 8-bit layer: the weights' bytes count
        dict(name="linear_one_token", op="linear", T=1, K=4096, O=4096, dtype="bf16", bias=False),
        # a verification chunk through the first layer of the dense FFN of the same size (64 * 128 rows)
        dict(name="linear_chunk32", op="linear", T=32, K=2048, O=8192, dtype="bf16", bias=False),
        # odd sizes, fp32 in and out, with a bias
        dict(name="linear_ragged", op="linear", T=333, K=2064, O=1007, dtype="f32", bias=True),
        # a prefill of 4096 tokens: the products count
        dict(name="linear_seq4096", op="linear", T=4096, K=4096, O=4096, dtype="bf16", bias=False),
        # one decoded token through its 8 experts
        dict(name="experts_one_token", op="experts", T=1, d_h=2048, E=64, d_e=128, gates="topk", k=8, bias=False),
        # a verification chunk with gates of a ReLU router (about a fifth active, neighbours alike, some
        # tokens with no expert), expert biases given
        dict(name="experts_chunk32", op="experts", T=32, d_h=2048, E=64, d_e=128, gates="relu", k=0, bias=True),
        # a prefill of 4096 tokens, 8 of 64 experts each
        dict(name="experts_seq4096", op="experts", T=4096, d_h=2048, E=64, d_e=128, gates="topk", k=8, bias=False),
    ]


def _logu(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "grad", "linear", "experts"])
    if op == "route":
        G = rng.choice([1, 1, 2, 4, 8])
        per = rng.randint(4, 256 // G)
        E, g = G * per, rng.randint(1, G)
        return dict(op=op, T=_logu(rng, 1, 32749), E=E, k=rng.randint(1, min(16, g * per)),
                    scores=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, n_group=G, topk_group=g,
                    renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5, 16.0]), dtype=rng.choice(["f32", "bf16"]),
                    padded=rng.random() < 0.4)
    if op == "grad":
        E, renorm = rng.randint(4, 256), rng.random() < 0.6   # one renormalised weight is constant: no gradient
        return dict(op=op, T=_logu(rng, 1, 16381), E=E, k=rng.randint(2 if renorm else 1, min(16, E)),
                    scores=rng.choice(["softmax", "sigmoid"]), renorm=renorm,
                    scale=rng.choice([1.0, 2.5, 16.0]), dtype=rng.choice(["f32", "bf16"]), padded=rng.random() < 0.4)
    if op == "linear":
        while True:
            T, K, O = _logu(rng, 1, 4096), 16 * _logu(rng, 8, 512), _logu(rng, 64, 8192)
            if T * K * O <= 4096 ** 3:
                return dict(op=op, T=T, K=K, O=O, dtype=rng.choice(["f32", "bf16"]), bias=rng.random() < 0.5)
    while True:
        T, d_h = _logu(rng, 1, 4096), 128 * _logu(rng, 2, 32)
        E, d_e = rng.randint(8, 128), 128 * rng.choice([1, 1, 1, 2, 3, 4])
        if T * E * d_e * d_h <= 4096 * 64 * 128 * 2048 and E * d_e * d_h <= 128 * 128 * 4096:
            gates = rng.choice(["topk", "topk", "relu"])
            return dict(op=op, T=T, d_h=d_h, E=E, d_e=d_e, gates=gates,
                        k=rng.randint(1, min(8, E // 4)) if gates == "topk" else 0, bias=rng.random() < 0.4)


# ----------------------------------------------------------------- inputs --

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _quantized_weight(gen, fan_in, *shape):
    """A weight of N(0, 1/fan_in), as int8 values and a scale for each output channel (the last axis is the input's)."""
    w = _normal(gen, *shape) * fan_in ** -0.5
    s = w.abs().amax(-1) / 127
    return torch.round(w / s[..., None]).clamp(-127, 127).to(torch.int8), s


def _logits(gen, c):
    """Router logits: a token's own part and a part of each expert's (some are popular)."""
    z = 1.3 * _normal(gen, c["T"], c["E"]) + 0.7 * _normal(gen, 1, c["E"])
    if c["padded"]:
        z = z.masked_fill(torch.rand(c["T"], 1, generator=gen, device="cuda") < 0.05, float("-inf"))
    return z.to(_DT[c["dtype"]])


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = dict(case=c)
    if c["op"] == "route":
        st["logits"] = _logits(gen, c)
        st["bias"] = 0.2 * _normal(gen, c["E"]) if c["bias"] else None
    elif c["op"] == "grad":
        st["logits"] = _logits(gen, c)
        order = torch.sort(st["logits"].float(), dim=-1, descending=True, stable=True)
        ids = order.indices[:, : c["k"]].to(torch.int32)
        st["ids"] = ids.masked_fill(order.values[:, : c["k"]] == float("-inf"), -1).contiguous()
        st["d_weights"] = _normal(gen, c["T"], c["k"])
    elif c["op"] == "linear":
        st["x"] = (_normal(gen, c["T"], c["K"]) * (1 + 0.5 * _normal(gen, 1, c["K"]).abs())).to(_DT[c["dtype"]])
        st["W"], st["s_w"] = _quantized_weight(gen, c["K"], c["O"], c["K"])
        st["bias"] = 0.1 * _normal(gen, c["O"]) if c["bias"] else None
    else:
        T, d_h, E, d_e = c["T"], c["d_h"], c["E"], c["d_e"]
        st["x"] = _normal(gen, T, d_h).to(torch.bfloat16)
        st["W_in"], st["s_in"] = _quantized_weight(gen, d_h, E, d_e, d_h)
        st["W_out"], st["s_out"] = _quantized_weight(gen, d_e, E, d_h, d_e)
        st["b_in"] = _normal(gen, E, d_e) * d_h ** -0.5 if c["bias"] else None
        st["b_out"] = _normal(gen, E, d_h) * d_e ** -0.5 if c["bias"] else None
        if c["gates"] == "topk":
            z = 1.3 * _normal(gen, T, E) + 0.7 * _normal(gen, 1, E)
            top = torch.topk(z, c["k"], dim=-1)
            st["gates"] = torch.zeros(T, E, device="cuda").scatter_(1, top.indices, torch.softmax(top.values, -1))
        else:
            runs = torch.rand((T + 7) // 8, E, generator=gen, device="cuda") < 0.22
            on = runs.repeat_interleave(8, 0)[:T] & (torch.rand(T, E, generator=gen, device="cuda") < 0.9)
            on &= torch.rand(T, 1, generator=gen, device="cuda") >= 0.05
            st["gates"] = torch.where(on, _normal(gen, T, E).abs(), 0.0).contiguous()
    if own:   # the scratch buffer that a program keeps for its shapes
        import chunk_sparse_moe_b200 as bffn
        if c["op"] == "linear":
            st["workspace"] = bffn.Workspace.for_int8_linear(c["T"], c["K"], c["O"])
        elif c["op"] == "experts":
            st["workspace"] = bffn.Workspace.for_forward_int8(c["T"], c["d_h"], c["E"], c["d_e"])
    return st


# -------------------------------------------------------------------- run --

def run(state):
    c = state["case"]
    if own:
        import chunk_sparse_moe_b200 as bffn
        if c["op"] == "route":
            return bffn.route_topk(state["logits"], c["k"], scores=c["scores"], bias=state["bias"],
                                   n_group=c["n_group"], topk_group=c["topk_group"], renormalize=c["renorm"],
                                   scale=c["scale"])
        if c["op"] == "grad":
            return bffn.route_topk_backward(state["logits"], state["ids"], state["d_weights"], scores=c["scores"],
                                            renormalize=c["renorm"], scale=c["scale"])
        if c["op"] == "linear":
            return bffn.int8_linear(state["x"], state["W"], state["s_w"], bias=state["bias"],
                                    workspace=state["workspace"])
        return bffn.forward_int8(state["x"], state["gates"], state["W_in"], state["s_in"], state["W_out"],
                                 state["s_out"], b_in=state["b_in"], b_out=state["b_out"],
                                 workspace=state["workspace"])
    if c["op"] == "route":
        return _route(state["logits"], state["bias"], c)
    if c["op"] == "grad":
        return _grad(state["logits"], state["ids"], state["d_weights"], c)
    if c["op"] == "linear":
        return _linear(state["x"], state["W"], state["s_w"], state["bias"])
    return _experts(state)


# ------------------------------------------------------------- plain forms --

def _scores(z, kind):
    """Softmax or sigmoid scores in z's type; an expert whose logit is -inf has score 0."""
    if kind == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    e = torch.exp(z - z.amax(-1, keepdim=True).clamp(min=torch.finfo(z.dtype).min))
    return e / e.sum(-1, keepdim=True).clamp(min=torch.finfo(z.dtype).tiny)


def _route(logits, bias, c):
    """The choice in 64 bits (values next to a border decide it), the weights in 32."""
    T, E, k = c["T"], c["E"], c["k"]
    z = logits.float()
    off = z == float("-inf")
    if bias is None and c["n_group"] == 1:
        choice = z.double()   # both kinds of score grow with the logit
    else:
        choice = _scores(z.double(), c["scores"]) + (0 if bias is None else bias.double())
        choice = choice.masked_fill(off, float("-inf"))
    if c["n_group"] > 1:
        # a group counts the sum of its two best scores; the best topk_group groups take part
        per = choice.view(T, c["n_group"], E // c["n_group"])
        two = torch.sort(per, dim=-1, descending=True).values[..., :2]
        group = torch.where(two == float("-inf"), 0.0, two).sum(-1)
        group = group.masked_fill(two[..., 0] == float("-inf"), float("-inf"))
        best = torch.sort(group, dim=-1, descending=True, stable=True).indices[:, : c["topk_group"]]
        kept = torch.zeros_like(group, dtype=torch.bool).scatter_(1, best, True)
        choice = choice.masked_fill(~kept[:, :, None].expand_as(per).reshape(T, E), float("-inf"))
    order = torch.sort(choice, dim=-1, descending=True, stable=True)   # ties: the lowest index first
    ids = order.indices[:, :k]
    none = order.values[:, :k] == float("-inf")
    s = _scores(z, c["scores"]).gather(1, ids).masked_fill(none, 0.0)
    if c["renorm"]:
        s = s / s.sum(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).tiny)
    weights = s * c["scale"]
    gates = torch.zeros(T, E, device=z.device).scatter_add_(1, ids, weights)
    return gates, ids.masked_fill(none, -1).to(torch.int32), weights


def _grad(logits, ids, d_weights, c):
    """d_logits of the weights of the chosen experts; the choice itself has no gradient."""
    z = logits.float()
    s = _scores(z, c["scores"])
    none, at = ids < 0, ids.clamp(min=0).long()
    chosen = s.gather(1, at).masked_fill(none, 0.0)
    dw = d_weights.masked_fill(none, 0.0) * c["scale"]
    if c["renorm"]:
        total = chosen.sum(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).tiny)
        dw = (dw - (dw * chosen).sum(-1, keepdim=True) / total) / total
        dw = dw.masked_fill(none, 0.0)
    ds = torch.zeros_like(z).scatter_add_(1, at, dw)
    if c["scores"] == "sigmoid":
        dz = ds * s * (1 - s)
    else:
        dz = s * (ds - (dw * chosen).sum(-1, keepdim=True))
    return dz.to(logits.dtype)


def _quantized(v):
    """Whole numbers in [-127, 127] and the scale of each row (last axis).  In 64 bits (v's) a value next to the border
    of two whole numbers goes to the right one."""
    amax = v.abs().amax(-1, keepdim=True)
    q = torch.round(v * 127 / torch.where(amax > 0, amax, 1.0))
    return q.float(), (amax / 127).float()


def _whole_product(a, b):
    """a b^T of whole numbers of at most 127, exactly: fp32 holds every sum below 2^24, 64 bits any that can be met."""
    if a.shape[-1] * 127 * 127 < 2 ** 24:
        return a.float() @ b.float().T
    return (a.double() @ b.double().T).float()


def _linear(x, W, s_w, bias):
    q, s = _quantized(x.double())
    y = _whole_product(q, W) * s_w * s
    if bias is not None:
        y = y + bias
    return y.to(x.dtype)


def _experts(st):
    T, E, d_e, d_h = st["x"].shape[0], *st["W_in"].shape
    g = st["gates"]
    q, s = _quantized(st["x"].double())
    z = _whole_product(q, st["W_in"].view(E * d_e, d_h)) * st["s_in"].view(-1) * s
    if st["b_in"] is not None:
        z = z + st["b_in"].view(-1)
    h = (z / (1 + torch.exp(-z))).view(T, E, d_e)
    hq, hs = _quantized(h)
    hs = torch.where(g != 0, hs[..., 0] * g, 0.0)
    # the sum over experts as one product in 32 bits: the scales differ from expert to expert
    a = (hq * hs[..., None]).view(T, E * d_e)
    b = st["W_out"].float() * st["s_out"][..., None]
    y = a @ b.permute(0, 2, 1).reshape(E * d_e, d_h)
    if st["b_out"] is not None:
        y = y + g @ st["b_out"]
    return y.to(st["x"].dtype)


# ------------------------------------------------------------------- exact --

def _exact_row_scores(z, kind):
    return torch.sigmoid(z) if kind == "sigmoid" else torch.nan_to_num(torch.softmax(z, -1))


def _exact_int8(v):
    amax = v.abs().max(-1, keepdim=True).values
    step = amax / 127
    return torch.where(amax > 0, torch.round(v / step), torch.zeros_like(v)), step


def exact(case, seed):
    c = case
    st = prepare(case, seed)
    if c["op"] == "route":
        z = st["logits"].double()
        s = _exact_row_scores(z, c["scores"])
        choice = s if st["bias"] is None else s + st["bias"].double()
        choice = torch.where(z > float("-inf"), choice, torch.full_like(z, -1e30))
        T, E, G = c["T"], c["E"], c["n_group"]
        if G > 1:
            groups = choice.reshape(T, G, E // G)
            value = groups.topk(2, -1).values.sum(-1) if E // G > 1 else groups[..., 0]
            rank = torch.argsort(value, dim=1, descending=True, stable=True)
            out = rank[:, c["topk_group"]:].repeat_interleave(E // G, 1) * (E // G)
            out = out + torch.arange(E // G, device=z.device).repeat(G - c["topk_group"])
            choice = choice.scatter(1, out, -1e30)
        ids = torch.argsort(choice, dim=1, descending=True, stable=True)[:, : c["k"]]
        live = torch.gather(choice, 1, ids) > -1e29
        w = torch.where(live, torch.gather(s, 1, ids), torch.zeros_like(s[:, : c["k"]]))
        if c["renorm"]:
            w = torch.where(live, w / w.sum(1, keepdim=True), torch.zeros_like(w))
        w = w * c["scale"]
        gates = torch.zeros_like(z)
        gates.scatter_(1, torch.where(live, ids, ids[:, :1]), 0.0)
        gates = gates.scatter_add(1, ids, w)
        return gates, torch.where(live, ids, torch.full_like(ids, -1)).to(torch.int32), w
    if c["op"] == "grad":
        z = st["logits"].double().requires_grad_()
        live = st["ids"] >= 0
        rows = torch.where(live.any(1, keepdim=True), z, torch.zeros_like(z))
        s = torch.sigmoid(rows) if c["scores"] == "sigmoid" else torch.softmax(rows, -1)
        w = torch.gather(s, 1, st["ids"].clamp(min=0).long()) * live
        if c["renorm"]:
            w = w / torch.where(live.any(1, keepdim=True), w.sum(1, keepdim=True), torch.ones_like(w[:, :1]))
        (w * c["scale"] * st["d_weights"].double()).sum().backward()
        return z.grad
    if c["op"] == "linear":
        q, step = _exact_int8(st["x"].double())
        y = (q * step) @ (st["W"].double() * st["s_w"].double()[:, None]).T
        return y if st["bias"] is None else y + st["bias"].double()
    x, g = st["x"].double(), st["gates"].double()
    q, step = _exact_int8(x)
    y = torch.zeros_like(x)
    for e in range(c["E"]):
        t = g[:, e].nonzero()[:, 0]
        z = (q[t] * step[t]) @ (st["W_in"][e].double() * st["s_in"][e].double()[:, None]).T
        z = z if st["b_in"] is None else z + st["b_in"][e].double()
        hq, hstep = _exact_int8(z * torch.sigmoid(z))
        o = (hq * hstep) @ (st["W_out"][e].double() * st["s_out"][e].double()[:, None]).T
        o = o if st["b_out"] is None else o + st["b_out"][e].double()
        y.index_add_(0, t, o * g[t, e, None])
    return y


# -------------------------------------------------------------------- work --

def work(case):
    """Each input read once, each output written once; of the experts' weights those that some token uses, in
    expectation over the inputs; two operations for each product of a token with a weight that it needs."""
    c = case
    size = {"f32": 4, "bf16": 2}
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": T * E * (size[c["dtype"]] + 4) + 8 * T * k + (4 * E if c["bias"] else 0), "flops": 6 * T * E}
    if c["op"] == "grad":
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": T * E * 2 * size[c["dtype"]] + 8 * T * k, "flops": 6 * T * E}
    if c["op"] == "linear":
        T, K, O = c["T"], c["K"], c["O"]
        return {"bytes": size[c["dtype"]] * T * (K + O) + O * K + 4 * O * (2 if c["bias"] else 1), "flops": 2 * T * K * O}
    T, d_h, E, d_e = c["T"], c["d_h"], c["E"], c["d_e"]
    if c["gates"] == "topk":
        pairs, used = T * c["k"], E * (1 - (1 - c["k"] / E) ** T)
    else:
        pairs, used = T * E * 0.22 * 0.9 * 0.95, E * (1 - 0.78 ** math.ceil(T / 8))
    per = 2 * d_h * d_e + 4 * (d_h + d_e) * (2 if c["bias"] else 1)
    return {"bytes": int(4 * T * d_h + 4 * T * E + used * per), "flops": int(4 * pairs * d_h * d_e)}
