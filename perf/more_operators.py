"""Cases for turning a dense layer into one with experts and training it on a
teacher, with plain forms to hold the kernels to:

* ``route``: the top-k routing of every position to its experts: ids, weights,
  the order that groups the rows by expert, and the balance and z losses;
  forward, or forward and the gradient of the router's logits.
* ``experts``: the feed-forward network of the chosen experts, gathered,
  weighted and summed; the forward alone, or forward and backward.
* ``products``: matrix products over ragged groups of rows, each group against
  its own matrix; the forward alone, or with both gradients.
* ``distill``: the divergence of a vocabulary projection's distribution from a
  teacher's stored top logits, the n x V logits never kept; the forward alone,
  or forward and backward.

``own`` selects the framework's entry points; otherwise ``run`` computes the
operators in elementary torch operations in fp32 (long sums in fp64).
"""
import math

import torch

own = False


# ------------------------------------------------------------------ the cases

def _route(name, back, n, experts, k, dtype, norm, balance, z, masked):
    return {"name": name, "op": "route", "back": back, "n": n, "experts": experts, "k": k, "dtype": dtype, "norm": norm,
            "balance": balance, "z": z, "masked": masked}


def _experts(name, train, n, h, f, experts, k, act, skew):
    return {"name": name, "op": "experts", "train": train, "n": n, "h": h, "f": f, "experts": experts, "k": k, "act": act,
            "skew": skew}


def _products(name, train, rows, k, n, groups, out, skew):
    return {"name": name, "op": "products", "train": train, "rows": rows, "k": k, "n": n, "groups": groups, "out": out,
            "skew": skew}


def _distill(name, train, n, h, vocab, k, temperature, teacher, masked):
    return {"name": name, "op": "distill", "train": train, "n": n, "h": h, "vocab": vocab, "k": k, "temperature": temperature,
            "teacher": teacher, "masked": masked}


def listed():
    return [
        # the next token of a few sequences: the latency of a call
        _route("route_tokens", False, 16, 64, 4, "float32", True, 0.0, 0.0, False),
        # a training batch with padded positions and both losses
        _route("route_train", True, 32768, 64, 6, "float32", False, 0.01, 0.001, True),
        # one new token: the weights of its four experts are all there is to read
        _experts("experts_token", False, 1, 2048, 1024, 64, 4, "swiglu", 0.5),
        # one new token of each of 48 sequences: nearly every expert, few rows each
        _experts("experts_batch", False, 48, 2560, 2048, 32, 4, "swiglu", 0.5),
        # a prompt through many small experts
        _experts("experts_prompt", False, 5000, 2048, 1408, 64, 6, "swiglu", 0.5),
        # a training step of the 4096-wide layer turned into eight experts of its own size
        _experts("experts_train", True, 4096, 4096, 14336, 8, 2, "swiglu", 0.3),
        # a training step at odd sizes, uneven experts, the GeLU network
        _experts("experts_ragged_train", True, 3001, 1000, 2744, 12, 3, "gelu_tanh", 1.0),
        # projections of grouped rows, some groups empty, odd sizes
        _products("products_ragged", False, 3001, 1304, 776, 40, "float32", 1.5),
        # grouped rows with both gradients
        _products("products_train", True, 16384, 2560, 2048, 16, "bfloat16", 0.7),
        # one short sequence: the latency of a call
        _distill("distill_short", True, 100, 256, 5000, 16, 1.0, "logits", False),
        # evaluation of a student against stored log-probabilities, padded rows
        _distill("distill_eval", False, 4001, 2048, 50257, 64, 1.0, "logprobs", True),
        # a training step of the 2560-wide model over its vocabulary
        _distill("distill_train", True, 8000, 2560, 50257, 32, 2.0, "logits", False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "experts", "experts", "products", "distill"])
    if op == "route":
        experts = rng.choice([8, 12, 16, 32, 64, 64, 128, 160, 256])
        c = _route("", rng.random() < 0.5, _log(rng, 1, 32768), experts, rng.randint(1, 8), rng.choice(["float32", "bfloat16"]),
                   rng.random() < 0.5, rng.choice([0.0, 0.01]), rng.choice([0.0, 0.001]), rng.random() < 0.5)
    elif op == "experts":
        train = rng.random() < 0.5
        experts = rng.choice([4, 8, 12, 16, 32, 64])
        k = min(experts, rng.choice([1, 2, 2, 4, 6, 8]))
        h, f = 8 * _log(rng, 16, 512), 8 * _log(rng, 16, 512)
        top = min(8e12 / ((18 if train else 6) * k * h * f), 2.0 ** 28 / (k * max(h, f)))
        c = _experts("", train, _log(rng, 1, max(2, min(16384, top))), h, f, experts, k,
                     rng.choice(["swiglu", "swiglu", "gelu_erf", "gelu_tanh"]), rng.choice([0.0, 0.5, 1.0]))
    elif op == "products":
        c = _products("", rng.random() < 0.5, _log(rng, 1, 16384), 8 * _log(rng, 4, 320), 8 * _log(rng, 4, 256),
                      rng.choice([1, 3, 8, 16, 40, 64]), rng.choice(["float32", "bfloat16"]), rng.choice([0.0, 0.7, 1.5]))
    else:
        h, vocab = 8 * _log(rng, 8, 320), _log(rng, 300, 50257)
        c = _distill("", rng.random() < 0.6, _log(rng, 1, min(8000, 2 ** 28 // vocab)), h, vocab, rng.choice([1, 4, 16, 32, 50, 64]),
                     rng.choice([1.0, 1.0, 1.5, 2.0, 4.0]), rng.choice(["logits", "logprobs"]), rng.random() < 0.5)
    del c["name"]
    return c


def _group_sizes(c):
    """Rows of each group, fixed by the case: uneven by `skew`, some empty when
    the skew is large, an eighth of the rows behind the last group."""
    rows, groups = c["rows"] - c["rows"] // 8, c["groups"]
    state, share = 4321 + 13 * c["rows"] + groups, []
    for _ in range(groups):
        state = (state * 1103515245 + 12345) % 2 ** 31
        u = (state >> 8) / 2.0 ** 23
        share.append(0.0 if c["skew"] > 1 and u < 0.2 else math.exp(4 * c["skew"] * (u - 0.5)))
    if not sum(share):
        share[0] = 1.0
    total, sizes, acc, at = sum(share), [], 0.0, 0
    for v in share:
        acc += v
        to = min(rows, int(round(rows * acc / total)))
        sizes.append(to - at)
        at = to
    return sizes


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _matrices(g, count, rows, cols):
    """[count, rows, cols] bf16 of the size that keeps products near one."""
    w = torch.empty(count, rows, cols, device="cuda", dtype=torch.bfloat16)
    for i in range(count):
        w[i] = _randn(g, rows, cols, scale=cols ** -0.5)
    return w


def _dtype(name):
    return {"float32": torch.float32, "bfloat16": torch.bfloat16}[name]


def prepare(c, seed):
    return {"route": _prepare_route, "experts": _prepare_experts, "products": _prepare_products,
            "distill": _prepare_distill}[c["op"]](c, _gen(seed))


def _prepare_route(c, g):
    n, E, k = c["n"], c["experts"], c["k"]
    # experts differ in how often they are wanted
    z = 1.5 * torch.randn(n, E, generator=g, device="cuda") + 0.5 * torch.randn(E, generator=g, device="cuda")
    if c["masked"]:  # padded positions see no expert, some positions only a few
        u = torch.rand(n, 1, generator=g, device="cuda")
        few = (u > 0.97) & (torch.rand(n, E, generator=g, device="cuda") < 0.9)
        z = z.masked_fill((u < 0.1) | few, -math.inf)
    st = {"case": c, "logits": z.to(_dtype(c["dtype"])), "ids": torch.empty(n, k, device="cuda", dtype=torch.int32),
          "weights": torch.empty(n, k, device="cuda"), "offsets": torch.empty(E + 2, device="cuda", dtype=torch.int32),
          "order": torch.empty(n * k, device="cuda", dtype=torch.int32),
          "slot": torch.empty(n * k, device="cuda", dtype=torch.int32), "loss": torch.empty(1, device="cuda")}
    if c["back"]:
        st["dweights"] = torch.randn(n, k, generator=g, device="cuda") / n
        st["dlogits"] = torch.empty_like(st["logits"])
    return st


def _prepare_experts(c, g):
    n, h, f, E, k = c["n"], c["h"], c["f"], c["experts"], c["k"]
    # the routes that the router's call left: ids, weights, and the rows in the experts' order
    z = torch.randn(n, E, generator=g, device="cuda") + c["skew"] * torch.randn(E, generator=g, device="cuda")
    top, ids = z.topk(k, -1)
    key, order = ids.flatten().sort(stable=True)
    slot = torch.empty_like(order)
    slot[order] = torch.arange(n * k, device="cuda")
    counts = torch.bincount(key, minlength=E)
    zero = counts.new_zeros(1)
    offsets = torch.cat((zero, counts.cumsum(0), zero + n))
    st = {"case": c, "ids": ids.int(), "weights": torch.softmax(top, -1).to(torch.bfloat16), "offsets": offsets.int(),
          "order": order.int(), "slot": slot.int(), "counts": counts.tolist(), "x": _randn(g, n, h),
          "w1": _matrices(g, E, f, h), "w3": _matrices(g, E, f, h) if c["act"] == "swiglu" else None,
          "w2": _matrices(g, E, h, f), "y": torch.empty(n, h, device="cuda", dtype=torch.bfloat16)}
    if c["train"]:
        st["dy"] = _randn(g, n, h)
        st["dx"], st["dweights"] = torch.empty_like(st["x"]), torch.empty_like(st["weights"])
        st["dw"] = {w: torch.empty_like(st[w]) for w in ("w1", "w3", "w2") if st[w] is not None}
    return st


def _prepare_products(c, g):
    rows, k, n, G = c["rows"], c["k"], c["n"], c["groups"]
    sizes = _group_sizes(c)
    ends = torch.tensor([0] + sizes, device="cuda").cumsum(0).int()
    st = {"case": c, "sizes": sizes, "offsets": ends, "x": _randn(g, rows, k), "w": _matrices(g, G, n, k),
          "y": torch.zeros(rows, n, device="cuda", dtype=_dtype(c["out"]))}
    if c["train"]:
        st["dy"], st["dx"] = _randn(g, rows, n), torch.zeros(rows, k, device="cuda", dtype=_dtype(c["out"]))
        st["dw"] = torch.empty(G, n, k, device="cuda")
    return st


def _prepare_distill(c, g):
    n, h, V, k = c["n"], c["h"], c["vocab"], c["k"]
    st = {"case": c, "x": _randn(g, n, h), "w": _randn(g, V, h, scale=2.0 * h ** -0.5)}
    # a teacher's top entries: distinct ids in falling order, near-Zipf values
    ids = torch.randint(0, V, (n, k), generator=g, device="cuda")
    ids = (ids[:, :1] + torch.arange(k, device="cuda") * (V // k)) % V if k > V // 8 else _distinct(ids, V)
    v = torch.randn(n, k, generator=g, device="cuda").mul(1.5).sort(-1, descending=True).values
    if c["teacher"] == "logprobs":  # the rest of the mass is outside the stored entries
        v = torch.log_softmax(v, -1) + math.log(0.9)
    ids = ids.int()
    if c["masked"]:  # fewer entries in some rows, none in others
        kept = torch.randint(0, 2 * k, (n, 1), generator=g, device="cuda")
        ids = ids.masked_fill(torch.arange(k, device="cuda") >= kept, -1)
    st["ids"], st["teacher"], st["row_weight"] = ids.contiguous(), v, None
    if c["masked"]:  # padded rows count nothing, the others alike
        keep = (torch.rand(n, generator=g, device="cuda") < 0.85).float()
        st["row_weight"] = keep / keep.sum().clamp(min=1)
    st["loss"] = torch.empty(1, device="cuda")
    if c["train"]:
        st["dx"], st["dw"] = torch.empty_like(st["x"]), torch.empty_like(st["w"])
    return st


def _distinct(ids, V):
    """Row by row distinct ids: the sorted draws pushed apart, shuffled back."""
    k = ids.shape[1]
    s = (ids % (V - k)).sort(-1).values + torch.arange(k, device=ids.device)
    return s.gather(-1, (ids.argsort(-1)).argsort(-1))


# ------------------------------------------------------------------ the framework's calls

ACTS = {"gelu_erf": 0, "gelu_tanh": 1, "swiglu": 2}


def _kept(st, what, nbytes):
    """A buffer that a program keeps beside its tensors."""
    if what not in st:
        st[what] = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device="cuda")
    return st[what]


def _own_route(st):
    import blockwise_attention_ffn_gb300 as bpt
    from blockwise_attention_ffn_gb300.presets import MoeConfig
    c = st["case"]
    cfg = MoeConfig(n=c["n"], h=64, ffn_dim=64, n_experts=c["experts"], top_k=c["k"], norm_topk=int(c["norm"]),
                    logits_dtype=int(c["dtype"] == "bfloat16"), weights_dtype=0, balance_coef=c["balance"], z_coef=c["z"])
    route = bpt.MoeRoute(st["ids"], st["weights"], st["offsets"], st["order"], st["slot"])
    ws = _kept(st, "ws", bpt.bpt_moe_route_workspace_bytes(cfg))
    bpt.bpt_moe_route_fwd(cfg, st["logits"], route, st["loss"], ws)
    got = {w: st[w] for w in ("ids", "weights", "offsets", "order", "slot", "loss")}
    if c["back"]:
        bpt.bpt_moe_route_bwd(cfg, st["logits"], route, st["dweights"], 1.0, st["dlogits"])
        got["dlogits"] = st["dlogits"]
    return got


def _own_experts(st):
    import blockwise_attention_ffn_gb300 as bpt
    from blockwise_attention_ffn_gb300.presets import MoeConfig
    c = st["case"]
    cfg = MoeConfig(n=c["n"], h=c["h"], ffn_dim=c["f"], n_experts=c["experts"], top_k=c["k"], act=ACTS[c["act"]],
                    weights_dtype=1, grads_dtype=1)
    route = bpt.MoeRoute(st["ids"], st["weights"], st["offsets"], st["order"], st["slot"])
    passes = (bpt.BPT_PASS_FWD, bpt.BPT_PASS_BWD) if c["train"] else (bpt.BPT_PASS_FWD,)
    if "ws" not in st:
        _kept(st, "ws", max(bpt.bpt_moe_ffn_workspace_bytes(cfg, p) for p in passes))
    saved = None
    if c["train"]:
        saved = st["saved"] if "saved" in st else _kept(st, "saved", bpt.bpt_moe_saved_bytes(cfg))
    bpt.bpt_moe_ffn_fwd(cfg, route, st["x"], st["w1"], st["w3"], st["w2"], st["y"], saved, st["ws"])
    if not c["train"]:
        return st["y"]
    dw = st["dw"]
    bpt.bpt_moe_ffn_bwd(cfg, route, st["x"], st["w1"], st["w3"], st["w2"], saved, st["dy"], st["dx"], st["dweights"], dw["w1"],
                        dw.get("w3"), dw["w2"], st["ws"])
    return {"y": st["y"], "dx": st["dx"], "dweights": st["dweights"], "dw": dw}


def _own_products(st):
    import blockwise_attention_ffn_gb300 as bpt
    from blockwise_attention_ffn_gb300.presets import GroupedConfig
    c = st["case"]
    out = int(c["out"] == "bfloat16")
    cfg = GroupedConfig(rows=c["rows"], n=c["n"], k=c["k"], groups=c["groups"], form=bpt.BPT_GROUPED_NT, out_dtype=out)
    bpt.bpt_grouped_gemm(cfg, st["x"], st["w"], st["offsets"], st["y"])
    if not c["train"]:
        return st["y"]
    # dx [rows, k] = dy [rows, n] w [n, k], dw [n, k] = dy^T x of each group
    bpt.bpt_grouped_gemm(cfg.with_(n=c["k"], k=c["n"], form=bpt.BPT_GROUPED_NN), st["dy"], st["w"], st["offsets"], st["dx"])
    bpt.bpt_grouped_gemm(cfg.with_(n=c["k"], k=c["n"], form=bpt.BPT_GROUPED_TN, out_dtype=0), st["dy"], st["x"], st["offsets"],
                         st["dw"])
    return {"y": st["y"], "dx": st["dx"], "dw": st["dw"]}


def _own_distill(st):
    import blockwise_attention_ffn_gb300 as bpt
    from blockwise_attention_ffn_gb300.presets import DistillConfig
    c = st["case"]
    cfg = DistillConfig(n=c["n"], h=c["h"], vocab=c["vocab"], top_k=c["k"], temperature=c["temperature"],
                        teacher=int(c["teacher"] == "logprobs"), grads_dtype=1)
    passes = (bpt.BPT_PASS_FWD, bpt.BPT_PASS_BWD) if c["train"] else (bpt.BPT_PASS_FWD,)
    if "ws" not in st:
        _kept(st, "ws", max(bpt.bpt_lm_distill_workspace_bytes(cfg, p) for p in passes))
    saved = st["saved"] if "saved" in st else _kept(st, "saved", bpt.bpt_lm_distill_saved_bytes(cfg))
    bpt.bpt_lm_distill_fwd(cfg, st["x"], st["w"], st["ids"], st["teacher"], st["row_weight"], st["loss"], saved, st["ws"])
    if not c["train"]:
        return st["loss"]
    bpt.bpt_lm_distill_bwd(cfg, st["x"], st["w"], st["row_weight"], saved, 1.0, st["dx"], st["dw"], st["ws"])
    return {"loss": st["loss"], "dx": st["dx"], "dw": st["dw"]}


# ------------------------------------------------------------------ the plain forms

def _plain_route(st):
    c = st["case"]
    n, E, k = c["n"], c["experts"], c["k"]
    z = st["logits"].float()
    top, idx = z.sort(dim=-1, descending=True, stable=True)  # ties to the lowest index
    top, idx = top[:, :k], idx[:, :k]
    seen = top > -math.inf
    ids = torch.where(seen, idx, -1)
    m = top[:, :1].clamp(min=-3e38)
    ex = (z - m).exp()
    total = ex.sum(-1, keepdim=True)
    prob = ex / total.clamp(min=1e-38)
    if c["norm"]:
        w = (top - m).exp()
        w = w / w.sum(-1, keepdim=True).clamp(min=1e-38)
    else:
        w = torch.where(seen, prob.gather(-1, idx), 0.0)
    key, order = torch.where(seen, idx, E).flatten().sort(stable=True)
    order = torch.where(key < E, order, -1)
    counts = (torch.arange(E + 1, device="cuda")[:, None] > key).sum(-1)  # rows of the experts before
    at = torch.empty(n * k + 1, dtype=torch.int64, device="cuda")
    at[order] = torch.arange(n * k, device="cuda")
    slot = torch.where(seen.flatten(), at[:-1], -1)
    live = seen[:, :1].sum()
    share = counts.diff().double()
    nv = live.double().clamp(min=1)
    lse = torch.where(seen[:, 0], (m + total.log())[:, 0], 0.0)
    loss = c["balance"] * E / (nv * k) * (share * prob.sum(0, dtype=torch.float64) / nv).sum() + c["z"] * lse.double().square().sum() / nv
    got = {"ids": ids.int(), "weights": w, "offsets": torch.cat((counts, live[None])).int(), "order": order.int(), "slot": slot.int(),
           "loss": loss.float().view(1)}
    if c["back"]:
        dw = st["dweights"] * seen
        if c["norm"]:
            dtop = w * (dw - (dw * w).sum(-1, keepdim=True))
            dz = torch.zeros_like(z).scatter_add_(-1, idx, dtop)
            gp = torch.zeros_like(z)
        else:
            dz = torch.zeros_like(z)
            gp = torch.zeros_like(z).scatter_add_(-1, idx, dw)
        gp = gp + (c["balance"] * E / (nv * nv * k) * share).float()
        dz = dz + prob * (gp - (gp * prob).sum(-1, keepdim=True) + (2 * c["z"] / nv).float() * lse[:, None])
        got["dlogits"] = dz.to(st["logits"].dtype)
    return got


def _act(kind, g, u):
    """The network's activation and its slopes by g and by u."""
    if kind == "swiglu":
        s = 1 / (1 + (-g).exp())
        return g * s * u, u * s * (1 + g * (1 - s)), g * s
    if kind == "gelu_erf":
        cdf = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * cdf, cdf + g * (-0.5 * g * g).exp() / math.sqrt(2 * math.pi), None
    c = math.sqrt(2 / math.pi)
    t = (c * (g + 0.044715 * g * g * g)).tanh()
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g), None


def _plain_experts(st):
    c = st["case"]
    n, h, k = c["n"], c["h"], c["k"]
    token, slot = st["order"].long() // k, st["slot"].long()
    rows = st["x"].float()[token]
    w = st["weights"].float().flatten()[st["order"].long()][:, None]
    parts, kept, at = [], [], 0
    for e, count in enumerate(st["counts"]):  # an expert is a product of its own
        x = rows[at:at + count]
        g = x @ st["w1"][e].float().T
        u = None if st["w3"] is None else x @ st["w3"][e].float().T
        a, by_g, by_u = _act(c["act"], g, u)
        parts.append(a @ st["w2"][e].float().T)
        if c["train"]:
            kept.append((x, a, by_g, by_u))
        at += count
    ys = torch.cat(parts)
    y = (ys * w)[slot].view(n, k, h).sum(1).to(torch.bfloat16)
    if not c["train"]:
        return y
    dys = st["dy"].float()[token]
    dweights = (ys * dys).sum(-1)[slot].view(n, k).to(torch.bfloat16)
    dys = dys * w
    dw = {m: torch.empty_like(t) for m, t in st["dw"].items()}
    parts, at = [], 0
    for e, (x, a, by_g, by_u) in enumerate(kept):
        dy = dys[at:at + len(x)]
        da = dy @ st["w2"][e].float()
        dw["w2"][e] = dy.T @ a
        dg = da * by_g
        dw["w1"][e] = dg.T @ x
        dx = dg @ st["w1"][e].float()
        if by_u is not None:
            du = da * by_u
            dw["w3"][e] = du.T @ x
            dx += du @ st["w3"][e].float()
        parts.append(dx)
        at += len(x)
    dx = torch.cat(parts)[slot].view(n, k, h).sum(1).to(torch.bfloat16)
    return {"y": y, "dx": dx, "dweights": dweights, "dw": dw}


def _plain_products(st):
    c = st["case"]
    G, sizes = c["groups"], st["sizes"]
    rest = [c["rows"] - sum(sizes)]  # behind the last group: left as they are
    x = st["x"].float().split(sizes + rest)
    y = torch.cat([x[e] @ st["w"][e].float().T for e in range(G)] + [torch.zeros(*rest, c["n"], device="cuda")]).to(st["y"].dtype)
    if not c["train"]:
        return y
    dy = st["dy"].float().split(sizes + rest)
    dx = torch.cat([dy[e] @ st["w"][e].float() for e in range(G)] + [torch.zeros(*rest, c["k"], device="cuda")]).to(st["dx"].dtype)
    return {"y": y, "dx": dx, "dw": torch.stack([dy[e].T @ x[e] for e in range(G)])}


def _plain_distill(st):
    c = st["case"]
    n, T = c["n"], c["temperature"]
    ids = st["ids"].long()
    there = ids >= 0
    v = st["teacher"].masked_fill(~there, -math.inf)
    if c["teacher"] == "logits":
        v = v / T
        v = v - v.amax(-1, keepdim=True).clamp(min=-3e38)
        v = v - v.exp().sum(-1, keepdim=True).log().clamp(min=-3e38)
    p = v.exp()
    z = (st["x"].float() @ st["w"].float().T).div_(T)
    m = z.amax(-1, keepdim=True)
    total = (z - m).exp_().sum(-1, keepdim=True)
    lse = m + total.log()
    picked = z.gather(-1, ids.clamp(min=0))
    kl = torch.where(there, p * (v - picked + lse), 0.0).sum(-1)
    share = torch.full((n,), 1.0 / n, device="cuda") if st["row_weight"] is None else st["row_weight"]
    loss = (T * T * (share * kl).sum(dtype=torch.float64)).float().view(1)
    if not c["train"]:
        return loss
    dz = z.sub_(lse).exp_().mul_(p.sum(-1, keepdim=True)).scatter_add_(-1, ids.clamp(min=0), -p)
    dz.mul_((T * share)[:, None])
    return {"loss": loss, "dx": (dz @ st["w"].float()).to(torch.bfloat16), "dw": (dz.T @ st["x"].float()).to(torch.bfloat16)}


def run(st):
    op = st["case"]["op"]
    if own:
        return {"route": _own_route, "experts": _own_experts, "products": _own_products, "distill": _own_distill}[op](st)
    return {"route": _plain_route, "experts": _plain_experts, "products": _plain_products, "distill": _plain_distill}[op](st)


# ------------------------------------------------------------------ what a pass cannot do without

def work(c):
    if c["op"] == "route":
        n, E, k = c["n"], c["experts"], c["k"]
        e = 4 if c["dtype"] == "float32" else 2
        byte = n * E * e + 16 * n * k + 4 * (E + 2)
        if c["back"]:
            byte += n * E * 2 * e + 8 * n * k
        return {"bytes": byte, "flops": n * E * (20 if c["back"] else 8)}
    if c["op"] == "experts":
        n, h, f, E, k = c["n"], c["h"], c["f"], c["experts"], c["k"]
        mats = 3 if c["act"] == "swiglu" else 2
        active = E * (1 - (1 - k / E) ** n)  # experts that some position is sent to
        byte = 2 * active * mats * h * f + 4 * n * h + 14 * n * k
        flops = 2 * n * k * mats * h * f
        if c["train"]:
            byte += 2 * E * mats * h * f + 4 * n * h + 4 * n * k
            flops *= 3
        return {"bytes": int(byte), "flops": flops}
    if c["op"] == "products":
        sizes = _group_sizes(c)
        rows, some, o = sum(sizes), sum(s > 0 for s in sizes), 4 if c["out"] == "float32" else 2
        byte, flops = 2 * rows * c["k"] + 2 * some * c["k"] * c["n"] + o * rows * c["n"], 2 * rows * c["k"] * c["n"]
        if c["train"]:
            byte += 2 * rows * c["n"] + o * rows * c["k"] + 4 * c["groups"] * c["k"] * c["n"]
            flops *= 3
        return {"bytes": byte, "flops": flops}
    n, h, V, k = c["n"], c["h"], c["vocab"], c["k"]
    byte = 2 * n * h + 2 * V * h + 8 * n * k + 4
    if c["train"]:  # the logits are formed again: they are not kept
        byte += 2 * n * h + 2 * V * h
    return {"bytes": byte, "flops": (8 if c["train"] else 2) * n * h * V}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_route(c, st):
    n, E, k = c["n"], c["experts"], c["k"]
    z = st["logits"].double()
    left, ids, tops = z.clone(), [], []
    for _ in range(k):  # the largest one left, the first of equals
        top = left.max(-1, keepdim=True).values
        first = (left == top).int().argmax(-1, keepdim=True)
        ids.append(torch.where(top > -math.inf, first, -1))
        tops.append(top)
        left.scatter_(-1, first, -math.inf)
    ids, tops = torch.cat(ids, -1), torch.cat(tops, -1)
    live = ids[:, 0] >= 0
    lse = torch.where(live, torch.logsumexp(z, -1), 0.0)
    prob = torch.where(live[:, None], torch.exp(z - lse[:, None]), 0.0)
    of = torch.where(live, torch.logsumexp(tops, -1), 0.0) if c["norm"] else lse
    w = torch.where(ids >= 0, torch.exp(tops - of[:, None]), 0.0)
    flat = ids.flatten()
    lists = [(flat == e).nonzero()[:, 0] for e in range(E)]
    order, slot = torch.full_like(flat, -1), torch.full_like(flat, -1)
    offsets, at = [0], 0
    for rows in lists:
        order[at:at + len(rows)] = rows
        slot[rows] = torch.arange(at, at + len(rows), device="cuda")
        at += len(rows)
        offsets.append(at)
    nv = max(1, int(live.sum()))
    share = torch.tensor(offsets, dtype=torch.float64, device="cuda").diff() / (nv * k)
    loss = c["balance"] * E * (share * prob.mean(0) * n / nv).sum() + c["z"] * (lse * lse).sum() / nv
    got = {"ids": ids.int(), "weights": w, "offsets": torch.tensor(offsets + [int(live.sum())], dtype=torch.int32), "order": order.int(),
           "slot": slot.int(), "loss": loss.view(1)}
    if c["back"]:
        dw = torch.where(ids >= 0, st["dweights"].double(), 0.0)
        # d log w_j / dz_e = [e = id_j] - q_e, with q the softmax that the weights were taken of
        one = torch.zeros_like(z).scatter_add_(-1, ids.clamp(min=0), torch.where(ids >= 0, dw * w, 0.0))
        q = torch.zeros_like(z).scatter_add_(-1, ids.clamp(min=0), w) if c["norm"] else prob
        dz = one - q * (dw * w).sum(-1, keepdim=True)
        b = c["balance"] * E / nv * share
        dz += prob * b - prob * (prob @ b)[:, None]
        dz += 2 * c["z"] / nv * lse[:, None] * prob
        got["dlogits"] = dz
    return got


def _exact_experts(c, st):
    n, h, f, E, k = c["n"], c["h"], c["f"], c["experts"], c["k"]
    if work(c)["flops"] > 6e12:
        return None
    x, ids, w = st["x"].double(), st["ids"], st["weights"].double()
    dy = st["dy"].double() if c["train"] else None
    y, dx, dweights = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(w)
    dw = {m: torch.zeros(t.shape, dtype=torch.float64, device="cuda") for m, t in st["dw"].items()} if c["train"] else {}
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        a1, a2 = st["w1"][e].double(), st["w2"][e].double()
        a3 = None if st["w3"] is None else st["w3"][e].double()
        with torch.enable_grad():
            g = (x[t] @ a1.T).requires_grad_()
            u = None if a3 is None else (x[t] @ a3.T).requires_grad_()
            if a3 is not None:
                a = torch.nn.functional.silu(g) * u
            else:
                a = torch.nn.functional.gelu(g, approximate="tanh" if c["act"] == "gelu_tanh" else "none")
        out = a.detach() @ a2.T
        y.index_add_(0, t, out * w[t, j, None])
        if not c["train"]:
            continue
        dweights[t, j] = (out * dy[t]).sum(-1)
        d = dy[t] * w[t, j, None]
        dw["w2"][e] = d.T @ a.detach()
        slopes = torch.autograd.grad(a, [g] if u is None else [g, u], d @ a2)
        dw["w1"][e] = slopes[0].T @ x[t]
        dx.index_add_(0, t, slopes[0] @ a1)
        if u is not None:
            dw["w3"][e] = slopes[1].T @ x[t]
            dx.index_add_(0, t, slopes[1] @ a3)
    return {"y": y, "dx": dx, "dweights": dweights, "dw": dw} if c["train"] else y


def _exact_products(c, st):
    if work(c)["flops"] > 6e12:
        return None
    group = torch.full((c["rows"],), -1, device="cuda")
    for e in range(c["groups"]):
        group[int(st["offsets"][e]):int(st["offsets"][e + 1])] = e
    y = torch.zeros(c["rows"], c["n"], dtype=torch.float64, device="cuda")
    dx = torch.zeros(c["rows"], c["k"], dtype=torch.float64, device="cuda")
    dw = torch.zeros(c["groups"], c["n"], c["k"], dtype=torch.float64, device="cuda")
    for e in range(c["groups"]):
        r = group == e
        x, w = st["x"][r].double(), st["w"][e].double()
        y[r] = torch.einsum("rk,nk->rn", x, w)
        if c["train"]:
            dy = st["dy"][r].double()
            dx[r] = torch.einsum("rn,nk->rk", dy, w)
            dw[e] = torch.einsum("rn,rk->nk", dy, x)
    return {"y": y, "dx": dx, "dw": dw} if c["train"] else y


def _exact_distill(c, st):
    n, h, V, T = c["n"], c["h"], c["vocab"], c["temperature"]
    if work(c)["flops"] > 9e12:
        return None
    w, total = st["w"].double(), 0.0
    dx, dw = torch.zeros(n, h, dtype=torch.float64, device="cuda"), torch.zeros(V, h, dtype=torch.float64, device="cuda")
    for r0 in range(0, n, 1024):
        r = slice(r0, min(n, r0 + 1024))
        x, ids, t = st["x"][r].double(), st["ids"][r].long(), st["teacher"][r].double()
        share = torch.full((len(x),), 1.0 / n, dtype=torch.float64, device="cuda") if st["row_weight"] is None else st["row_weight"][r].double()
        gone = ids < 0
        if c["teacher"] == "logits":
            t = (t / T).masked_fill(gone, -math.inf)
            p = torch.where(gone, 0.0, torch.softmax(torch.where(gone.all(-1, keepdim=True), 0.0, t), -1))
        else:
            p = torch.where(gone, 0.0, torch.exp(t))
        logq = torch.log_softmax(x @ w.T / T, -1)
        total += float(T * T * (share[:, None] * (torch.special.xlogy(p, p) - p * logq.gather(-1, ids.clamp(min=0)))).sum())
        if c["train"]:
            dz = torch.exp(logq) * p.sum(-1, keepdim=True)
            dz.scatter_add_(-1, ids.clamp(min=0), -p)
            dz *= T * share[:, None]
            dx[r] = dz @ w
            dw += dz.T @ x
    loss = torch.tensor([total], dtype=torch.float64)
    return {"loss": loss, "dx": dx, "dw": dw} if c["train"] else loss


def exact(c, seed):
    st = prepare(c, seed)
    return {"route": _exact_route, "experts": _exact_experts, "products": _exact_products, "distill": _exact_distill}[c["op"]](c, st)
