"""Cases for the training operators around a layer's attention and its weight
gradients, with plain forms to hold the kernels to:

* ``norm_rope``: the norm of every query and key head (RMS over the head's d
  columns, times a weight) and the rotary position embedding in the same pass,
  on the packed projection buffer [b*s, (H + 2 H_kv) d]; forward and backward.
* ``attention``: attention on that buffer with a window of keys per query row
  (documents packed into one sequence, prefixes, sliding windows, padding),
  a tanh cap of the scores and a per-head bias linear in the distance; the
  forward alone, or forward and backward.
* ``clip``: the global norm of a list of gradients and their scaled copies.

``own`` selects the framework's entry points; otherwise ``run`` computes the
operators in elementary torch operations in fp32 (angles and totals in fp64).
"""
import math

import torch

own = False


# ------------------------------------------------------------------ the cases

def _attn(name, train, b, s, heads, kv_heads, d, mask, size, cap, slopes):
    return {"name": name, "op": "attention", "train": train, "b": b, "s": s, "heads": heads, "kv_heads": kv_heads,
            "d": d, "mask": mask, "size": size, "cap": cap, "slopes": slopes}


def _rope(name, back, b, s, heads, kv_heads, d, doc):
    return {"name": name, "op": "norm_rope", "back": back, "b": b, "s": s, "heads": heads, "kv_heads": kv_heads, "d": d,
            "doc": doc}


def _clip(name, layers, h, ffn, kind, dtype, limit):
    return {"name": name, "op": "clip", "layers": layers, "h": h, "ffn": ffn, "kind": kind, "dtype": dtype, "limit": limit}


def listed():
    return [
        # one short prompt through a small layer: the latency of a call
        _attn("attention_short", False, 1, 200, 4, 4, 64, "docs", 64, 0.0, False),
        # a packed batch row of the grouped-query layer with capped scores: evaluation
        _attn("attention_docs_cap", False, 1, 8192, 32, 8, 128, "docs", 1500, 50.0, False),
        # a training step of the 32 x 80 layer whose positions are a distance bias
        _attn("attention_bias_train", True, 2, 2000, 32, 32, 80, "causal", 0, 0.0, True),
        # prefix-masked pairs padded to the longest, every modifier at once, odd lengths
        _attn("attention_prefix_train", True, 3, 1111, 12, 4, 96, "prefix", 300, 30.0, True),
        # a long training row of packed documents, grouped-query heads, capped scores
        _attn("attention_long_train", True, 1, 16384, 16, 4, 128, "docs", 4000, 30.0, False),
        # new tokens of eight sequences at far positions: the latency of a call
        _rope("norm_rope_tokens", False, 8, 1, 32, 8, 128, 0),
        # the long row of the grouped-query layer
        _rope("norm_rope_long", False, 1, 65536, 32, 8, 128, 0),
        # an odd batch of small heads
        _rope("norm_rope_ragged_back", True, 3, 777, 6, 2, 112, 100),
        # the training row of the 32 x 80 layer, positions restarting with each document
        _rope("norm_rope_train_back", True, 1, 32768, 32, 32, 80, 3000),
        # one small layer: the latency of a call
        _clip("clip_small", 1, 256, 1024, "gpt", "float32", 0.5),
        # the gradients of one grouped-query layer kept in bf16
        _clip("clip_layer_bf16", 1, 4096, 14336, "llama", "bfloat16", 1.0),
        # the fp32 gradients of a stack of 24 layers of width 2048
        _clip("clip_stack", 24, 2048, 8192, "gpt", "float32", 1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "norm_rope", "clip"])
    if op == "attention":
        train = rng.random() < 0.6
        d = rng.choice([64, 80, 96, 112, 128])
        kv_heads = rng.choice([1, 2, 4, 8])
        heads = kv_heads * rng.choice([1, 2, 3, 4])
        b = rng.choice([1, 1, 2, 3])
        s = _log(rng, 1, min(16384, int(math.sqrt(2.0 ** 31 / (b * heads)))))
        mask = rng.choice(["causal", "docs", "docs_both", "prefix", "window", "padded", "all"])
        c = _attn("", train, b, s, heads, kv_heads, d, mask, _log(rng, 1, max(2, s)), rng.choice([0.0, 20.0, 30.0, 50.0]),
                  rng.random() < 0.4)
    elif op == "norm_rope":
        kv_heads = rng.choice([1, 2, 4, 8, 16])
        heads = kv_heads * rng.choice([1, 2, 4])
        d = rng.choice([64, 80, 96, 112, 128])
        b = rng.choice([1, 2, 3, 8])
        c = _rope("", rng.random() < 0.5, b, _log(rng, 1, max(2, 2 ** 28 // (b * (heads + 2 * kv_heads) * d))), heads,
                  kv_heads, d, rng.choice([0, 0, 50, 1000]))
    else:
        h = 8 * _log(rng, 4, 256)
        c = _clip("", _log(rng, 1, 12), h, 8 * _log(rng, 8, 1024), rng.choice(["gpt", "llama"]),
                  rng.choice(["float32", "float32", "bfloat16", "mixed"]), rng.choice([0.01, 1.0, 1.0, 1e6]))
    del c["name"]
    return c


def _windows(c):
    """The mask as [begin, end) of the keys of each query row, two lists of
    b*s; None where the causal flag alone says it.  Fixed by the case."""
    b, s, m, size = c["b"], c["s"], c["mask"], max(1, c["size"])
    if m in ("causal", "all"):
        return None, None
    lo, hi = [], []
    state = 12345 + 7 * s + size
    for i in range(b):
        if m in ("docs", "docs_both"):
            at = 0
            while at < s:  # document lengths between a quarter and nearly twice the size
                state = (state * 1103515245 + 12345) % 2 ** 31
                n = min(s - at, max(1, size // 4 + (state >> 8) * (3 * size // 2) // 2 ** 23))
                lo += [at] * n
                hi += [at + n] * n
                at += n
        elif m == "window":
            lo += [max(0, q - size + 1) for q in range(s)]
            hi += [s] * s
        else:  # prefix: bidirectional up to `size`, causal after; both: rows past the sequence's length see nothing
            n = s - (i * s) // 4 if b > 1 else s - s // 8
            p = min(size, n) if m == "prefix" else 0
            lo += [0] * s
            hi += [max(q + 1, p) if q < n else 0 for q in range(s)]
    return lo, (None if m == "window" else hi)


def _is_causal(c):
    return c["mask"] in ("causal", "docs", "window")


def _shapes(c):
    h, f = c["h"], c["ffn"]
    if c["kind"] == "gpt":
        one = [(h,), (h,), (h, h), (h,), (h, h), (h,), (h, h), (h,), (h, h), (h,), (h,), (h,), (f, h), (f,), (h, f), (h,)]
    else:
        kv = max(8, h // 4)
        one = [(h,), (h, h), (kv, h), (kv, h), (h, h), (h,), (f, h), (h, f), (f, h)]
    return one * c["layers"]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def prepare(c, seed):
    g = _gen(seed)
    if c["op"] == "clip":
        # every tensor's gradient has its own scale, as layers differ
        kinds = {"float32": [torch.float32], "bfloat16": [torch.bfloat16], "mixed": [torch.float32, torch.bfloat16]}[c["dtype"]]
        shapes = _shapes(c)
        scale = torch.rand(len(shapes), generator=torch.Generator().manual_seed(seed)).mul(-6).exp2().tolist()
        grads = [_randn(g, *sh, scale=1e-3 * scale[i], dtype=kinds[i % len(kinds)]) for i, sh in enumerate(shapes)]
        # the scaled copies go to one buffer per type, tensor after tensor
        flat = {k: torch.zeros(sum(t.numel() for t in grads if t.dtype == k), device="cuda", dtype=k) for k in kinds}
        at, out = dict.fromkeys(kinds, 0), []
        for t in grads:
            out.append(flat[t.dtype][at[t.dtype]:at[t.dtype] + t.numel()].view(t.shape))
            at[t.dtype] += t.numel()
        return {"case": c, "grads": grads, "flat": flat, "out": out, "norm": torch.zeros(1, device="cuda")}
    b, s, H, K, d = c["b"], c["s"], c["heads"], c["kv_heads"], c["d"]
    rows, width = b * s, (H + 2 * K) * d
    if c["op"] == "norm_rope":
        st = {"case": c, "qkv": _randn(g, rows, width, scale=2.0),
              "wq": (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16),
              "wk": (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16), "positions": None}
        if s == 1:  # single new tokens, each at its own place of a long sequence
            st["positions"] = torch.randint(0, 131072, (rows,), generator=g, device="cuda", dtype=torch.int32)
        elif c["doc"]:
            st["positions"] = (torch.arange(s, device="cuda", dtype=torch.int32) % c["doc"]).repeat(b)
        if c["back"]:
            st["dout"] = _randn(g, rows, width)
            st["dwq"], st["dwk"] = (torch.zeros(d, device="cuda") for _ in range(2))
        st["out"] = torch.empty_like(st["qkv"])
        return st
    qkv = _randn(g, rows, width)
    qkv[:, :H * d] *= 2  # trained heads are more decided than random ones
    lo, hi = _windows(c)
    st = {"case": c, "qkv": qkv, "o": torch.empty(rows, H * d, device="cuda", dtype=torch.bfloat16),
          "lse": torch.empty(b, H, (s + 127) // 128 * 128, device="cuda"),
          "lo": None if lo is None else torch.tensor(lo, dtype=torch.int32, device="cuda"),
          "hi": None if hi is None else torch.tensor(hi, dtype=torch.int32, device="cuda"),
          "slopes": torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H).float() if c["slopes"] else None}
    if c["train"]:
        st["dout"] = _randn(g, rows, H * d)
        st["dqkv"] = torch.empty_like(qkv)
    return st


# ------------------------------------------------------------------ the framework's calls

def _config(c, **more):
    from blockwise_attention_ffn_gb300.presets import LayerConfig
    return LayerConfig(b=c["b"], s=c["s"], h=c["heads"] * c["d"], n_heads=c["heads"], n_kv_heads=c["kv_heads"],
                       head_dim=c["d"], ffn_dim=64, **more)


def _workspace(st, nbytes):
    """The workspace that a program keeps beside its buffers."""
    if "ws" not in st:
        st["ws"] = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device="cuda")
    return st["ws"]


def _run_own(st):
    import blockwise_attention_ffn_gb300 as bpt
    c = st["case"]
    if c["op"] == "clip":
        ws = _workspace(st, bpt.bpt_clip_workspace_bytes())
        bpt.bpt_clip_grads(st["grads"], c["limit"], st["norm"], ws, out=st["out"])
        return {"norm": st["norm"], "out": list(st["flat"].values())}
    if c["op"] == "norm_rope":
        cfg = _config(c, rope_base=500000.0)
        if not c["back"]:
            bpt.bpt_qk_norm_rope_fwd(cfg, st["qkv"], st["wq"], st["wk"], st["positions"], st["out"])
            return st["out"]
        ws = _workspace(st, bpt.bpt_qk_norm_rope_workspace_bytes(cfg))
        bpt.bpt_qk_norm_rope_bwd(cfg, st["qkv"], st["wq"], st["wk"], st["positions"], st["dout"], st["out"], st["dwq"],
                                 st["dwk"], ws)
        return {"dqkv": st["out"], "dwq": st["dwq"], "dwk": st["dwk"]}
    cfg = _config(c, causal=int(_is_causal(c)))
    mod = bpt.ScoreMod(row_begin=st["lo"], row_end=st["hi"], slopes=st["slopes"], softcap=c["cap"])
    bpt.bpt_attention_mod_fwd(cfg, mod, st["qkv"], st["o"], st["lse"])
    got = {"o": st["o"], "lse": st["lse"]}
    if c["train"]:
        ws = _workspace(st, bpt.bpt_attention_mod_bwd_workspace_bytes(cfg))
        bpt.bpt_attention_mod_bwd(cfg, mod, st["qkv"], st["o"], st["lse"], st["dout"], st["dqkv"], ws)
        got["dqkv"] = st["dqkv"]
    return got


# ------------------------------------------------------------------ the plain forms

def _rotation(c, positions):
    """cos and sin [rows, 1, d/2] of each row's angles, formed in fp64."""
    b, s, d = c["b"], c["s"], c["d"]
    if positions is None:
        positions = torch.arange(s, device="cuda").repeat(b)
    theta = 500000.0 ** (-2.0 * torch.arange(d // 2, device="cuda", dtype=torch.float64) / d)
    a = positions.double()[:, None] * theta
    return a.cos().float()[:, None], a.sin().float()[:, None]


def _rotate(x, cos, sin):
    u, v = x.chunk(2, -1)
    return torch.cat((u * cos - v * sin, u * sin + v * cos), -1)


def _run_norm_rope(st):
    c = st["case"]
    H, K, d = c["heads"], c["kv_heads"], c["d"]
    rows = c["b"] * c["s"]
    cos, sin = _rotation(c, st["positions"])
    x = st["qkv"].view(rows, H + 2 * K, d)[:, :H + K].float()
    w = torch.cat((st["wq"].float().expand(H, d), st["wk"].float().expand(K, d)))
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-5)
    if not c["back"]:
        y = _rotate(x * r * w, cos, sin).to(torch.bfloat16)
        return torch.cat((y.view(rows, -1), st["qkv"][:, (H + K) * d:]), 1)
    dn = _rotate(st["dout"].view(rows, H + 2 * K, d)[:, :H + K].float(), cos, -sin)
    n = x * r
    dw = (dn * n).sum(0)
    g = dn * w
    dx = (r * (g - n * (g * n).mean(-1, keepdim=True))).to(torch.bfloat16)
    return {"dqkv": torch.cat((dx.view(rows, -1), st["dout"][:, (H + K) * d:]), 1), "dwq": dw[:H].sum(0), "dwk": dw[H:].sum(0)}


def _run_attention(st):
    c = st["case"]
    b, s, H, K, d = c["b"], c["s"], c["heads"], c["kv_heads"], c["d"]
    q, k, v = st["qkv"].view(b, s, H + 2 * K, d).float().transpose(1, 2).split((H, K, K), 1)
    q = q.reshape(b, K, H // K, s, d)
    k, v = k[:, :, None], v[:, :, None]
    i = torch.arange(s, device="cuda")
    off = torch.zeros(b, 1, 1, s, s, dtype=torch.bool, device="cuda")
    if _is_causal(c):
        off |= i > i[:, None]
    if st["lo"] is not None:
        off |= i < st["lo"].view(b, 1, 1, s, 1)
    if st["hi"] is not None:
        off |= i >= st["hi"].view(b, 1, 1, s, 1)
    x = (q @ k.transpose(-1, -2)).mul_(d ** -0.5)
    t = None
    if c["cap"]:
        t = x.div_(c["cap"]).tanh_()
        x = t * c["cap"]
    if st["slopes"] is not None:
        x = x - st["slopes"].view(K, H // K, 1, 1) * (i - i[:, None]).abs()
    x.masked_fill_(off, -math.inf)
    m = x.amax(-1, keepdim=True).clamp_(min=-3e38)
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(total.clamp(min=1e-38))
    o = p @ v
    lse = torch.zeros_like(st["lse"])
    lse[:, :, :s] = torch.where(total > 0, m + total.log(), -math.inf).view(b, H, s)
    got = {"o": o.view(b, H, s, d).transpose(1, 2).reshape(b * s, H * d).to(torch.bfloat16), "lse": lse}
    if c["train"]:
        do = st["dout"].view(b, s, H, d).float().transpose(1, 2).reshape(b, K, H // K, s, d)
        dv = (p.transpose(-1, -2) @ do).sum(2)
        ds = (do @ v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p)
        if t is not None:
            ds.mul_(t.square_().neg_().add_(1))
        ds.mul_(d ** -0.5)
        dq = (ds @ k).view(b, H, s, d)
        dk = (ds.transpose(-1, -2) @ q).sum(2)
        got["dqkv"] = torch.cat((dq, dk, dv), 1).transpose(1, 2).reshape(b * s, -1).to(torch.bfloat16)
    return got


def _run_clip(st):
    grads = st["grads"]
    norm = torch.stack([g.float().square().sum(dtype=torch.float64) for g in grads]).sum().sqrt().float()
    scale = (st["case"]["limit"] / (norm + 1e-6)).clamp(max=1.0)
    return {"norm": norm.view(1), "out": [torch.cat([g.float().mul(scale).to(k).view(-1) for g in grads if g.dtype == k])
                                          for k in st["flat"]]}


def run(st):
    if own:
        return _run_own(st)
    return {"norm_rope": _run_norm_rope, "attention": _run_attention, "clip": _run_clip}[st["case"]["op"]](st)


# ------------------------------------------------------------------ what a pass cannot do without

def work(c):
    if c["op"] == "clip":
        n, byte = 0, 0
        for i, sh in enumerate(_shapes(c)):
            e = math.prod(sh)
            n += e
            byte += e * (4 if c["dtype"] == "float32" or (c["dtype"] == "mixed" and i % 2 == 0) else 2)
        return {"bytes": 2 * byte + 4, "flops": 3 * n}
    b, s, H, K, d = c["b"], c["s"], c["heads"], c["kv_heads"], c["d"]
    rows, width = b * s, (H + 2 * K) * d
    if c["op"] == "norm_rope":
        heads = (H + K) * d
        if c["back"]:  # dV passes through: read and written, its qkv columns unread
            return {"bytes": 2 * rows * (heads + 2 * width) + 8 * d, "flops": 20 * rows * heads}
        return {"bytes": 4 * rows * width, "flops": 8 * rows * heads}
    lo, hi = _windows(c)
    causal, pairs = _is_causal(c), 0
    if lo is None:
        pairs = b * (s * (s + 1) // 2 if causal else s * s)
    else:
        for r in range(b * s):
            e = s if hi is None else hi[r]
            pairs += max(0, (min(e, r % s + 1) if causal else e) - lo[r])
    byte = 2 * rows * (width + H * d) + 4 * rows * H
    if c["train"]:
        byte += 2 * rows * (H * d + width)
    return {"bytes": byte, "flops": (14 if c["train"] else 4) * pairs * H * d}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_attention(c, st):
    """Query rows in blocks, each against the keys that some row of it sees."""
    b, s, H, K, d = c["b"], c["s"], c["heads"], c["kv_heads"], c["d"]
    lo, hi = _windows(c)
    lo = [0] * (b * s) if lo is None else lo
    hi = [s] * (b * s) if hi is None else list(hi)
    if _is_causal(c):
        hi = [min(e, r % s + 1) for r, e in enumerate(hi)]
    step = 256
    blocks = []
    for bi in range(b):
        for r0 in range(0, s, step):
            rows = [(lo[bi * s + r], hi[bi * s + r]) for r in range(r0, min(s, r0 + step))]
            seen = [w for w in rows if w[1] > w[0]]
            blocks.append((bi, r0, r0 + len(rows), min([w[0] for w in seen], default=0), max([w[1] for w in seen], default=0)))
    pairs = sum((r1 - r0) * (k1 - k0) for _, r0, r1, k0, k1 in blocks)
    if pairs * H * d * (14 if c["train"] else 4) > 4e12:
        return None
    lo64, hi64 = (torch.tensor(w, device="cuda").view(b, s) for w in (lo, hi))
    x = st["qkv"].view(b, s, H + 2 * K, d).double()
    o = torch.zeros(b, s, H, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["lse"].shape, dtype=torch.float64, device="cuda")
    lse[:, :, :s] = -math.inf
    dx = torch.zeros_like(x)
    head_of = torch.arange(H, device="cuda") // (H // K)
    for bi, r0, r1, k0, k1 in blocks:
        if k1 <= k0:
            continue
        q = x[bi, r0:r1, :H].transpose(0, 1)
        k = x[bi, k0:k1, H:H + K].transpose(0, 1)[head_of]
        v = x[bi, k0:k1, H + K:].transpose(0, 1)[head_of]
        y = torch.einsum("hqd,hkd->hqk", q, k) / math.sqrt(d)
        slope = torch.ones_like(y)
        if c["cap"]:
            u = torch.tanh(y / c["cap"])
            y, slope = c["cap"] * u, 1 - u * u
        i, j = torch.arange(r0, r1, device="cuda")[:, None], torch.arange(k0, k1, device="cuda")
        if st["slopes"] is not None:
            y = y - st["slopes"].double()[:, None, None] * (i - j).abs()
        ok = (j >= lo64[bi, r0:r1, None]) & (j < hi64[bi, r0:r1, None])
        y = torch.where(ok, y, -math.inf)
        z = torch.logsumexp(y, -1)
        lse[bi, :, r0:r1] = z
        p = torch.where(ok, torch.exp(y - torch.where(z.isinf(), 0.0, z)[..., None]), 0.0)
        ob = torch.einsum("hqk,hkd->hqd", p, v)
        o[bi, r0:r1] = ob.transpose(0, 1)
        if c["train"]:
            do = st["dout"].view(b, s, H, d)[bi, r0:r1].double().transpose(0, 1)
            ds = p * (torch.einsum("hqd,hkd->hqk", do, v) - (do * ob).sum(-1, keepdim=True)) * slope / math.sqrt(d)
            dx[bi, r0:r1, :H] = torch.einsum("hqk,hkd->qhd", ds, k)
            dk = torch.einsum("hqk,hqd->hkd", ds, q).view(K, H // K, k1 - k0, d).sum(1)
            dv = torch.einsum("hqk,hqd->hkd", p, do).view(K, H // K, k1 - k0, d).sum(1)
            dx[bi, k0:k1, H:H + K] += dk.transpose(0, 1)
            dx[bi, k0:k1, H + K:] += dv.transpose(0, 1)
    got = {"o": o.view(b * s, H * d), "lse": lse}
    if c["train"]:
        got["dqkv"] = dx.view(b * s, -1)
    return got


def exact(c, seed):
    st = prepare(c, seed)
    if c["op"] == "attention":
        return _exact_attention(c, st)
    if c["op"] == "clip":
        if sum(g.numel() for g in st["grads"]) > 3e8:
            return None
        norm = math.sqrt(sum(float((g.double() ** 2).sum()) for g in st["grads"]))
        by = min(1.0, c["limit"] / (norm + 1e-6))
        for o, g in zip(st["out"], st["grads"]):
            o.zero_()
        return {"norm": torch.tensor([norm], dtype=torch.float64),
                "out": [torch.cat([(g.double() * by).flatten() for g in st["grads"] if g.dtype == k]) for k in st["flat"]]}
    b, s, H, K, d = c["b"], c["s"], c["heads"], c["kv_heads"], c["d"]
    rows = b * s
    if rows * (H + 2 * K) * d > 5e8:
        return None
    x = st["qkv"].double().view(rows, H + 2 * K, d)
    pos = torch.arange(rows, device="cuda") % s if st["positions"] is None else st["positions"]
    # the pair (i, i + d/2) as a complex number, turned by e^(i angle)
    turn = torch.polar(torch.ones(1, dtype=torch.float64, device="cuda"),
                       pos.double()[:, None] * torch.pow(500000.0, -torch.arange(0, d, 2, device="cuda").double() / d))[:, None]
    pair = lambda t: torch.complex(t[..., :d // 2].contiguous(), t[..., d // 2:].contiguous())  # noqa: E731
    flat = lambda z: torch.cat((z.real, z.imag), -1)  # noqa: E731
    out, dws = [], []
    for at, n, w in ((0, H, st["wq"].double()), (H, K, st["wk"].double())):
        u = x[:, at:at + n]
        unit = u / torch.sqrt((u * u).sum(-1, keepdim=True) / d + 1e-5)
        if not c["back"]:
            out.append(flat(pair(unit * w) * turn))
            continue
        g = flat(pair(st["dout"].double().view(rows, H + 2 * K, d)[:, at:at + n]) * turn.conj())
        dws.append((g * unit).sum((0, 1)))
        g = g * w
        size = torch.sqrt((u * u).sum(-1, keepdim=True) / d + 1e-5)
        out.append((g - unit * (g * unit).sum(-1, keepdim=True) / d) / size)
    rest = (st["dout"] if c["back"] else st["qkv"]).double().view(rows, H + 2 * K, d)[:, H + K:]
    y = torch.cat((*out, rest), 1).view(rows, -1)
    return {"dqkv": y, "dwq": dws[0], "dwk": dws[1]} if c["back"] else y
