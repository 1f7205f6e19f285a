"""Measured cases of the layer around latent attention: the per-head products of
its absorbed and expanded forms, causal attention over expanded keys and values,
and the norms of queries and latents with the rotation and the pool write.

With ``own`` false ``run`` computes them with elementary torch operations; with
``own`` true it calls this package's entry points on the same inputs.
"""
import math

import torch

own = False

LATENT, ROPE, NOPE, VALUE, HEADS = 512, 64, 128, 128, 64
ROW, HEAD = LATENT + ROPE, NOPE + ROPE
SCALE = HEAD ** -0.5
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6


def listed():
    return [
        # queries of one request's 8 draft nodes taken to the latent space: a step with a batch of one
        {"name": "absorb 8 tokens", "op": "product", "form": "absorb", "tokens": 8, "heads": 64, "part": 128,
         "dtype": "bf16"},
        # 4 requests x 16 nodes, the attention's latent outputs taken to the heads' values
        {"name": "values 64 tokens", "op": "product", "form": "values", "tokens": 64, "heads": 64, "part": 128,
         "dtype": "bf16"},
        # 16 requests x 64 nodes
        {"name": "absorb 1024 tokens", "op": "product", "form": "absorb", "tokens": 1024, "heads": 64, "part": 128,
         "dtype": "bf16"},
        # keys and values of a prompt's cached latents: every head's 128 + 128 from the one latent of a token
        {"name": "expand 8191 tokens", "op": "product", "form": "expand", "tokens": 8191, "heads": 64, "part": 256,
         "dtype": "fp16"},
        # a short prompt
        {"name": "prefill 1x256", "op": "prefill", "bs": 1, "new": 256, "cached": 0, "ragged": False, "heads": 64,
         "dtype": "bf16", "pad": 0},
        # chunks of two prompts behind their cached beginnings
        {"name": "prefill 2x(5760+1000)", "op": "prefill", "bs": 2, "new": 1000, "cached": 5760, "ragged": False,
         "heads": 64, "dtype": "bf16", "pad": 0},
        # prompts of all lengths on a rank with half of the heads, in buffers with rows to spare
        {"name": "prefill 9 ragged fp16", "op": "prefill", "bs": 9, "new": 1777, "cached": 333, "ragged": True,
         "heads": 32, "dtype": "fp16", "pad": 37},
        # the short last chunk of a long prompt on a rank with few heads
        {"name": "prefill 1x(32768+60)", "op": "prefill", "bs": 1, "new": 60, "cached": 32768, "ragged": False,
         "heads": 8, "dtype": "bf16", "pad": 0},
        # a long prompt in one piece
        {"name": "prefill 1x8192", "op": "prefill", "bs": 1, "new": 8192, "cached": 0, "ragged": False, "heads": 64,
         "dtype": "bf16", "pad": 0},
        # a batch of one: 8 draft nodes, latents normalised and written, queries turned
        {"name": "norm rope 8 tokens", "op": "norm", "tokens": 8, "valid": 8, "dtype": "bf16", "layout": "interleaved",
         "q_norm": False, "max_pos": 4096, "slots": 4096},
        # 16 requests x 64 nodes in a padded batch, every query head normalised too
        {"name": "norm rope 1024 tokens", "op": "norm", "tokens": 1100, "valid": 1024, "dtype": "bf16",
         "layout": "interleaved", "q_norm": True, "max_pos": 163840, "slots": 65536},
        # a prefill chunk of fp16 projections, half layout
        {"name": "norm rope 8191 tokens", "op": "norm", "tokens": 8191, "valid": 8191, "dtype": "fp16",
         "layout": "half", "q_norm": True, "max_pos": 131072, "slots": 16384},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["product", "prefill", "norm"])
    if op == "product":
        form = rng.choice(["absorb", "values", "expand"])
        heads = rng.choice([4, 8, 20, 32, 40, 64, 128])
        part = rng.choice([64, 96, 128, 160, 256] if form != "absorb" else [64, 96, 128, 160, 200])
        return {"op": op, "form": form, "tokens": _log_int(rng, 1, min(20000, 8000 * 64 * 128 // (heads * part))),
                "heads": heads, "part": part, "dtype": rng.choice(["bf16", "fp16"])}
    if op == "prefill":
        heads, bs = rng.choice([4, 8, 20, 32, 40, 64, 128]), _log_int(rng, 1, 16)
        most = 2_100_000_000 // (bs * heads)  # pairs of a query and a key it sees, a head
        new = _log_int(rng, 1, min(8000 // bs, int(math.sqrt(2 * most)) - 1))
        cached = _log_int(rng, 1, max(1, min(most // new - new, 3_000_000 // (bs * heads)))) if rng.random() < 0.6 else 0
        return {"op": op, "bs": bs, "new": new, "cached": cached, "ragged": rng.random() < 0.7, "heads": heads,
                "dtype": rng.choice(["bf16", "fp16"]), "pad": rng.choice([0, 0, 1, 29])}
    tokens = _log_int(rng, 1, 8000)
    return {"op": op, "tokens": tokens, "valid": rng.randint((tokens + 1) // 2, tokens),
            "dtype": rng.choice(["bf16", "fp16", "fp32"]), "layout": rng.choice(["interleaved", "half"]),
            "q_norm": rng.random() < 0.6, "max_pos": _log_int(rng, 1000, 1000000), "slots": 16384}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 31)


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    return {"product": _prepare_product, "prefill": _prepare_prefill, "norm": _prepare_norm}[case["op"]](case, g)


def _prepare_product(case, g):
    """Weights as one up-projection [heads, part, latent] keeps them; its
    transpose, for the products from the latent, is a view."""
    n, h, part, dtype = case["tokens"], case["heads"], case["part"], DTYPES[case["dtype"]]
    up = _normal(g, (h, part, LATENT), dtype, LATENT ** -0.5)
    if case["form"] == "absorb":  # the plain part of every query head, into rows of latent + rope
        x = _normal(g, (n, h, part + ROPE), dtype)[:, :, :part]
        rows = torch.zeros((n, h, ROW), dtype=dtype, device="cuda")
        return {"case": case, "x": x, "w": up, "out": rows[:, :, :LATENT]}
    if case["form"] == "values":  # the attention's outputs
        x = _normal(g, (n, h, LATENT), dtype, 0.3)
    else:                         # one latent row a token, shared by the heads
        x = _normal(g, (n, ROW), dtype)[:, None, :LATENT].expand(n, h, LATENT)
    return {"case": case, "x": x, "w": up.transpose(1, 2), "out": torch.zeros((n, h, part), dtype=dtype, device="cuda")}


def _lengths(case):
    """New and cached tokens of the requests, in rising order: evenly spread over
    a fifth of the longest and the longest, and over none and the most."""
    bs = case["bs"]
    if not case["ragged"]:
        return [case["new"]] * bs, [case["cached"]] * bs
    return ([max(1, int(case["new"] * (0.2 + 0.8 * (r + 0.5) / bs))) for r in range(bs)],
            [int(case["cached"] * (r + 0.5) / bs) for r in range(bs)])


def _shuffled(values, g):
    return [values[i] for i in torch.randperm(len(values), generator=g, device="cuda").tolist()]


def _prepare_prefill(case, g):
    h, dtype = case["heads"], DTYPES[case["dtype"]]
    new, cached = (_shuffled(x, g) for x in _lengths(case))
    total_q, total_k = sum(new), sum(new) + sum(cached)
    q = _normal(g, (total_q + case["pad"], h, HEAD), dtype, 1.5)
    kv = _normal(g, (total_k + case["pad"], h, NOPE + VALUE), dtype)   # as the expansion leaves them
    latents = _normal(g, (total_k + case["pad"], ROW), dtype)          # rows of the cache: the shared rotated key behind
    ends = lambda n, t: torch.tensor([0] + n, dtype=t, device="cuda").cumsum(0).to(t)  # noqa: E731
    st = {"case": case, "q": q, "k_nope": kv[:, :, :NOPE], "v": kv[:, :, NOPE:], "k_rope": latents[:, LATENT:],
          "new": new, "cached": cached, "qo_indptr": ends(new, torch.int64),
          "kv_indptr": ends([a + b for a, b in zip(new, cached)], torch.int32),
          "out": torch.zeros((total_q + case["pad"], h, VALUE), dtype=dtype, device="cuda"),
          "lse": torch.zeros((total_q + case["pad"], h), dtype=torch.float32, device="cuda"), "plan": {}}
    return st


def _turns(freq):
    """Frequencies as 64-bit fractions of a turn, the form the rotation reads."""
    return torch.tensor([int(x / (2 * math.pi) * 2.0 ** 64) for x in freq.tolist()], dtype=torch.int64)


def _prepare_norm(case, g):
    tokens, dtype = case["tokens"], DTYPES[case["dtype"]]
    freq = 10000.0 ** (-torch.arange(0, ROPE, 2, dtype=torch.float64) / ROPE)
    # queries and latents as the projections leave them: heads and tokens of different size
    size = torch.exp(torch.randn((tokens, HEADS, 1), generator=g, device="cuda"))
    proj = (torch.randn((tokens, HEADS, HEAD), generator=g, device="cuda") * size).to(dtype)
    down = (torch.randn((tokens, ROW), generator=g, device="cuda") * (0.1 + size[:, 0])).to(dtype)
    weight = lambda n: (1 + 0.2 * torch.randn((n,), generator=g, device="cuda")).to(dtype)  # noqa: E731
    return {"case": case, "q_in": proj, "q_weight": weight(HEAD) if case["q_norm"] else None, "c_in": down[:, :LATENT],
            "c_weight": weight(LATENT), "k_in": down[:, LATENT:],
            "q_nope": torch.zeros((tokens, HEADS, NOPE), dtype=dtype, device="cuda"),
            "q": _normal(g, (tokens, HEADS, ROW), dtype), "pool": _normal(g, (case["slots"], ROW), torch.bfloat16),
            "slots": torch.randperm(case["slots"], generator=g, device="cuda")[:tokens].contiguous(),
            "positions": torch.randint(0, case["max_pos"], (tokens,), generator=g, device="cuda"),
            "freq": freq.cuda(), "turns": _turns(freq).cuda(),
            "valid": torch.tensor([case["valid"]], dtype=torch.int64, device="cuda")}


# -------------------------------------------------------------- one pass

_package = None


def _own():
    global _package
    if _package is None:
        import paged_mla_speculative_tree_gb300
        _package = paged_mla_speculative_tree_gb300
    return _package


def run(state):
    op = state["case"]["op"]
    if op == "product":
        return _run_product(state)
    if op == "prefill":
        return _run_prefill(state)
    return _run_norm(state)


def _run_product(s):
    if own:
        _own().head_product(s["x"], s["w"], s["out"])
        return {"out": s["out"]}
    y = torch.matmul(s["x"].float().transpose(0, 1), s["w"].float()).transpose(0, 1)
    s["out"].copy_(y)
    return {"out": s["out"]}


def _plan(s):
    """What a serving program keeps for its batches: the bounds and the workspace."""
    if not s["plan"]:
        keys = [a + b for a, b in zip(s["new"], s["cached"])]
        s["plan"]["own"] = _own().MlaPrefill(len(keys), max(s["new"]), s["q"].shape[0], max(keys), s["case"]["heads"])
    return s["plan"]["own"]


def _run_prefill(s):
    out = {"out": s["out"], "lse": s["lse"]}
    if own:
        _plan(s)(s["q"], s["k_nope"], s["k_rope"], s["v"], s["qo_indptr"], s["kv_indptr"], SCALE, s["out"], s["lse"])
        return out
    # every request padded to the longest; request r's query i is at its position cached + i
    n, length = max(s["new"]), max(a + b for a, b in zip(s["new"], s["cached"]))
    new = (s["qo_indptr"][1:] - s["qo_indptr"][:-1])[:, None]
    keys = (s["kv_indptr"][1:] - s["kv_indptr"][:-1]).long()[:, None]
    i, j = torch.arange(n, device="cuda")[None], torch.arange(length, device="cuda")[None]
    row = s["qo_indptr"][:-1, None] + torch.minimum(i, new - 1)
    key = s["kv_indptr"][:-1, None].long() + torch.minimum(j, keys - 1)
    q = s["q"][row].float().transpose(1, 2)                                     # [bs, heads, n, 192]
    k_nope, v = s["k_nope"][key].float().transpose(1, 2), s["v"][key].float().transpose(1, 2)
    k_rope = s["k_rope"][key].float()[:, None]
    z = torch.matmul(q[..., :NOPE], k_nope.transpose(-1, -2))
    z += torch.matmul(q[..., NOPE:], k_rope.transpose(-1, -2))
    z *= SCALE
    hidden = j[:, None, :] > (keys - new + i)[:, :, None]                       # the keys behind the query's own
    z.masked_fill_(hidden[:, None], -math.inf)
    top = z.amax(dim=-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = z.sub_(top).exp_()
    total = e.sum(dim=-1, keepdim=True)
    o = torch.matmul(e, v) / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total))[..., 0]
    real = i < new
    s["out"][row[real]] = o.transpose(1, 2)[real].to(s["out"].dtype)
    s["lse"][row[real]] = lse.transpose(1, 2)[real]
    return out


def _normalised(x, weight):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * weight.float()


def _rotate(x, cos, sin, layout):
    if layout == "interleaved":
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
    a, b = x[..., :ROPE // 2], x[..., ROPE // 2:]
    return torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)


def _run_norm(s):
    case = s["case"]
    out = {"q": s["q"], "q_nope": s["q_nope"], "pool": s["pool"]}
    if own:
        p = _own()
        p.norm_rope_write(s["turns"], s["positions"], EPS, layout=p.ROPE_HALF if case["layout"] == "half" else p.ROPE_INTERLEAVED,
                          q_in=s["q_in"], q_weight=s["q_weight"], q_nope=s["q_nope"] if case["q_norm"] else None,
                          q_rope=s["q"][:, :, LATENT:], c_in=s["c_in"], c_weight=s["c_weight"], k_in=s["k_in"],
                          out_cache_loc=s["slots"], kv_pool=s["pool"], num_valid=s["valid"])
        return out
    n = case["valid"]
    angle = s["positions"][:n, None].double() * s["freq"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    q = _normalised(s["q_in"][:n], s["q_weight"]) if case["q_norm"] else s["q_in"][:n].float()
    if case["q_norm"]:
        s["q_nope"][:n] = q[..., :NOPE].to(s["q"].dtype)
    s["q"][:n, :, LATENT:] = _rotate(q[..., NOPE:], cos[:, None], sin[:, None], case["layout"]).to(s["q"].dtype)
    latent = _normalised(s["c_in"][:n], s["c_weight"])
    row = torch.cat([latent, _rotate(s["k_in"][:n].float(), cos, sin, case["layout"])], dim=1)
    s["pool"][s["slots"][:n]] = row.to(torch.bfloat16)
    return out


# ------------------------------------------------------ floors and 64 bits

def work(case):
    if case["op"] == "product":
        n, h, part, e = case["tokens"], case["heads"], case["part"], SIZES[case["dtype"]]
        x = n * (LATENT if case["form"] == "expand" else h * (part if case["form"] == "absorb" else LATENT))
        y = n * h * (LATENT if case["form"] == "absorb" else part)
        return {"bytes": e * (x + y + h * part * LATENT), "flops": 2 * n * h * part * LATENT}
    if case["op"] == "prefill":
        h, size, (new, cached) = case["heads"], SIZES[case["dtype"]], _lengths(case)
        rows, keys = sum(new), sum(new) + sum(cached)
        # of a ragged batch, the mean over the orders in which new and cached tokens meet
        pairs = sum(n * (n + 1) for n in new) / 2 + rows * sum(cached) / case["bs"]
        return {"bytes": size * (rows * h * (HEAD + VALUE) + keys * (h * (NOPE + VALUE) + ROPE)) + 4 * rows * h,
                "flops": 2 * pairs * h * (HEAD + VALUE)}
    e, n = SIZES[case["dtype"]], case["valid"]
    read = HEAD if case["q_norm"] else ROPE
    return {"bytes": n * (2 * HEADS * read * e + ROW * (e + 2) + 16), "flops": n * (HEADS * read + ROW) * 6}


def exact(case, seed):
    s = prepare(case, seed)
    return {"product": _exact_product, "prefill": _exact_prefill, "norm": _exact_norm}[case["op"]](s)


def _exact_product(s):
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    for h in range(out.shape[1]):
        out[:, h] = s["x"][:, h].double() @ s["w"][h].double()
    return {"out": out}


def _exact_prefill(s):
    """Request by request and head by head, as a softmax over the visible keys."""
    out, lse = s["out"].double(), s["lse"].double()
    qa, ka = s["qo_indptr"].tolist(), s["kv_indptr"].tolist()
    for r, (n, p) in enumerate(zip(s["new"], s["cached"])):
        seen = torch.ones((n, n + p), dtype=torch.bool, device="cuda").tril(p)
        rows, keys = slice(qa[r], qa[r + 1]), slice(ka[r], ka[r + 1])
        for h in range(out.shape[1]):
            k = torch.cat([s["k_nope"][keys, h], s["k_rope"][keys]], dim=1).double()
            z = (s["q"][rows, h].double() @ k.t()) * SCALE
            z = torch.where(seen, z, torch.full_like(z, -math.inf))
            lse[rows, h] = torch.logsumexp(z, dim=1)
            out[rows, h] = torch.exp(z - lse[rows, h, None]) @ s["v"][keys, h].double()
    return {"out": out, "lse": lse}


def _exact_norm(s):
    """Norms by the vectors' lengths; the pairs as complex numbers, turned by exp(i * position * frequency)."""
    case, n = s["case"], s["case"]["valid"]
    turn = torch.exp(1j * torch.remainder(s["positions"][:n, None].double() * s["freq"], 2 * math.pi))

    def unit(x, w):
        x = x.double()
        return x / torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / x.shape[-1] + EPS) * w.double()

    def turned(x, w):
        pairs = x.unflatten(-1, (-1, 2)) if case["layout"] == "interleaved" else x.unflatten(-1, (2, -1)).transpose(-1, -2)
        y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * w)
        return (y if case["layout"] == "interleaved" else y.transpose(-1, -2)).flatten(-2)

    q, q_nope, pool = s["q"].double(), s["q_nope"].double(), s["pool"].double()
    x = unit(s["q_in"][:n], s["q_weight"]) if case["q_norm"] else s["q_in"][:n].double()
    if case["q_norm"]:
        q_nope[:n] = x[..., :NOPE]
    q[:n, :, LATENT:] = turned(x[..., NOPE:], turn[:, None])
    pool[s["slots"][:n]] = torch.cat([unit(s["c_in"][:n], s["c_weight"]), turned(s["k_in"][:n].double(), turn)], dim=1)
    return {"q": q, "q_nope": q_nope, "pool": pool}
