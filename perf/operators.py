"""Measured cases of the steps around verify attention: page tables and slot
maps from request lengths, rotary positions with the write into the latent
pool, and token log probabilities.

With ``own`` false ``run`` computes them with elementary torch operations; with
``own`` true it calls this package's entry points on the same inputs.
"""
import math

import torch

own = False

LATENT, ROPE, HEADS = 512, 64, 64
ROW = LATENT + ROPE
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # one request's 8 draft nodes: the latency of a step with a batch of one
        {"name": "logprobs 8x32000 bf16", "op": "logprobs", "rows": 8, "vocab": 32000, "dtype": "bf16", "top": 1,
         "tokens": 8, "by_row": True, "temperature": False, "pad": 0},
        # 4 requests x 16 nodes, odd vocabulary (rows start at odd addresses), scored under their parents' rows
        {"name": "logprobs 64x50257 fp16", "op": "logprobs", "rows": 64, "vocab": 50257, "dtype": "fp16", "top": 20,
         "tokens": 63, "by_row": False, "temperature": True, "pad": 0},
        # 16 requests x 64 nodes: target tokens, scores and five alternatives of a large verify step
        {"name": "logprobs 1024x131072 bf16", "op": "logprobs", "rows": 1024, "vocab": 131072, "dtype": "bf16",
         "top": 5, "tokens": 1024, "by_row": False, "temperature": True, "pad": 0},
        # prompt scoring with fp32 logits kept in a padded buffer
        {"name": "logprobs 515x100003 fp32", "op": "logprobs", "rows": 515, "vocab": 100003, "dtype": "fp32",
         "top": 8, "tokens": 515, "by_row": True, "temperature": False, "pad": 61},
        # a batch of one: 8 draft nodes rotated and written
        {"name": "rope 8 tokens", "op": "rope", "tokens": 8, "dtype": "bf16", "layout": "interleaved",
         "scaling": "none", "max_pos": 4096, "slots": 4096, "valid": 8},
        # 16 requests x 64 nodes at far positions, a padded capacity of 1100 rows
        {"name": "rope 1024 tokens far", "op": "rope", "tokens": 1100, "dtype": "bf16", "layout": "interleaved",
         "scaling": "ramp", "max_pos": 163840, "slots": 65536, "valid": 1024},
        # a prefill chunk of fp16 projections, half layout
        {"name": "rope 8191 tokens half", "op": "rope", "tokens": 8191, "dtype": "fp16", "layout": "half",
         "scaling": "wavelength", "max_pos": 131072, "slots": 16384, "valid": 8191},
        # a decode step's batch of four
        {"name": "slots 4x5760+16", "op": "slots", "bs": 4, "prefix": 5760, "ragged": False, "tree": 16, "page": 64,
         "chain": False},
        # a ragged batch with single-slot pages
        {"name": "slots 192 ragged page 1", "op": "slots", "bs": 192, "prefix": 16000, "ragged": True, "tree": 31,
         "page": 1, "chain": True},
        # the longest contexts: 33.5 M prefix keys
        {"name": "slots 256x131072+64", "op": "slots", "bs": 256, "prefix": 131072, "ragged": False, "tree": 64,
         "page": 64, "chain": False},
        # one draft step of 256 sequences: pages for the trees, then all of them rolled back
        {"name": "pages 256 rows tree step", "op": "pages", "rows": 256, "held": 300, "grow": 64, "page": 16},
        # 64 prompts of up to 32768 tokens admitted with single-slot pages, then released
        {"name": "pages 64 prompts page 1", "op": "pages", "rows": 64, "held": 0, "grow": 32768, "page": 1},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "rope", "slots", "pages"])
    if op == "logprobs":
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        vocab = _log_int(rng, 1000, 200000)
        rows = _log_int(rng, 1, min(1024, 250_000_000 // (vocab * SIZES[dtype])))
        return {"op": op, "rows": rows, "vocab": vocab, "dtype": dtype, "top": rng.randint(1, 32),
                "tokens": _log_int(rng, 1, 2048), "by_row": False, "temperature": rng.random() < 0.5,
                "pad": rng.choice([0, 0, 1, 7, 64])}
    if op == "rope":
        tokens = _log_int(rng, 1, 8000)
        return {"op": op, "tokens": tokens, "dtype": rng.choice(["bf16", "fp16", "fp32"]),
                "layout": rng.choice(["interleaved", "half"]),
                "scaling": rng.choice(["none", "linear", "ramp", "wavelength"]),
                "max_pos": _log_int(rng, 1000, 1000000), "slots": 16384, "valid": rng.randint((tokens + 1) // 2, tokens)}
    if op == "slots":
        bs = _log_int(rng, 1, 512)
        return {"op": op, "bs": bs, "prefix": _log_int(rng, 16, min(131072, 30_000_000 // bs)),
                "ragged": rng.random() < 0.7, "tree": _log_int(rng, 1, 200), "page": rng.choice([1, 16, 32, 48, 64, 128]),
                "chain": rng.random() < 0.3}
    rows = _log_int(rng, 1, 4000)
    page = rng.choice([1, 16, 32, 48, 64])
    return {"op": op, "rows": rows, "held": _log_int(rng, 1, 1000), "grow": _log_int(rng, 1, min(32768, 2_000_000 // rows)),
            "page": page}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)


def _ints(g, lo, hi, n, dtype=torch.int32):
    """n uniform integers of [lo, hi]."""
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int64).to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    return {"logprobs": _prepare_logprobs, "rope": _prepare_rope, "slots": _prepare_slots,
            "pages": _prepare_pages}[case["op"]](case, g)


def _prepare_logprobs(case, g):
    """Logits of a language model: a broad bulk, a few likely tokens a row, and
    ids at the end that are masked out with -inf."""
    rows, vocab, stride = case["rows"], case["vocab"], case["vocab"] + case["pad"]
    dtype = DTYPES[case["dtype"]]
    buf = torch.empty((rows, stride), dtype=dtype, device="cuda")
    for a in range(0, rows, 128):
        part = torch.randn((min(128, rows - a), stride), generator=g, device="cuda") * 2.5
        buf[a:a + 128] = part.to(dtype)
    likely = torch.randint(0, vocab, (rows, 6), generator=g, device="cuda")
    lift = torch.rand((rows, 6), generator=g, device="cuda") * 10 + 6
    buf.scatter_(1, likely, lift.to(dtype))
    logits = buf[:, :vocab]
    masked = vocab // 500
    if masked:
        logits[:, vocab - masked:] = -math.inf
    n, k = case["tokens"], case["top"]
    tokens = torch.randint(0, vocab - masked, (n,), generator=g, device="cuda").to(torch.int32)
    st = {"case": case, "logits": logits, "tokens": tokens, "token_rows": None, "inv_temperature": None}
    if not case["by_row"]:
        st["token_rows"] = _ints(g, 0, rows - 1, n)
        hot = torch.rand((n,), generator=g, device="cuda") < 0.7  # drafts are mostly likely tokens
        pick = likely[st["token_rows"].long(), torch.arange(n, device="cuda") % 6]
        st["tokens"] = torch.where(hot & (pick < vocab - masked), pick, tokens.long()).to(torch.int32)
    if case["temperature"]:
        st["inv_temperature"] = 1.0 / (torch.rand((rows,), generator=g, device="cuda") * 1.2 + 0.3)
    st["logprobs"] = torch.zeros(n, dtype=torch.float32, device="cuda")
    st["stats"] = torch.zeros((3, rows), dtype=torch.float32, device="cuda")
    st["top_tokens"] = torch.zeros((k, rows), dtype=torch.int32, device="cuda")
    st["top_logprobs"] = torch.zeros((k, rows), dtype=torch.float32, device="cuda")
    return st


def _frequencies(scaling):
    """Angle per position of each rotated pair, and the amplitude (64 bits).

    ramp: a linear ramp between kept and divided frequencies over the pairs
    that turn between beta_fast and beta_slow times in the original length;
    wavelength: kept, divided or blended by each pair's wavelength."""
    base, factor, length = 10000.0, 40.0, 4096.0
    f = base ** (-torch.arange(0, ROPE, 2, dtype=torch.float64) / ROPE)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "ramp":
        at = lambda turns: ROPE * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), ROPE - 1)
        ramp = ((torch.arange(ROPE // 2, dtype=torch.float64) - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    if scaling == "wavelength":
        low, high, factor, length = 1.0, 4.0, 8.0, 8192.0
        turns = length * f / (2 * math.pi)
        s = (turns - low) / (high - low)
        mid = (1 - s) * f / factor + s * f
        return torch.where(turns > high, f, torch.where(turns < low, f / factor, mid)), 1.0
    return f, 1.0


def _turns(freq):
    """Frequencies as 64-bit fractions of a turn, the form the rotation reads."""
    return torch.tensor([int(x / (2 * math.pi) * 2.0 ** 64) for x in freq.tolist()], dtype=torch.int64)


def _prepare_rope(case, g):
    tokens, valid, dtype = case["tokens"], case["valid"], DTYPES[case["dtype"]]
    freq, amplitude = _frequencies(case["scaling"])
    # queries as the projection leaves them: 128 plain dims and 64 to rotate a head
    proj = torch.randn((tokens, HEADS, 128 + ROPE), generator=g, device="cuda", dtype=dtype)
    # latent and key part as one down-projection leaves them
    down = torch.randn((tokens, LATENT + ROPE), generator=g, device="cuda", dtype=dtype)
    q = torch.randn((tokens, HEADS, ROW), generator=g, device="cuda", dtype=dtype)
    pool = torch.randn((case["slots"], ROW), generator=g, device="cuda", dtype=torch.bfloat16)
    slots = torch.randperm(case["slots"], generator=g, device="cuda")[:tokens].contiguous()
    positions = torch.randint(0, case["max_pos"], (tokens,), generator=g, device="cuda")
    return {"case": case, "q_in": proj[:, :, 128:], "c_in": down[:, :LATENT], "k_in": down[:, LATENT:], "q": q,
            "pool": pool, "slots": slots, "positions": positions, "freq": freq.cuda(), "turns": _turns(freq).cuda(),
            "amplitude": amplitude, "valid": torch.tensor([valid], dtype=torch.int64, device="cuda")}


def _trees(case, bs, sizes, g):
    """Parent index of each node: a chain, or uniform over the earlier nodes."""
    node = torch.cat([torch.arange(n) for n in sizes]).cuda()
    if case["chain"]:
        return (node - 1).to(torch.int32)
    r = torch.rand((node.numel(),), generator=g, device="cuda", dtype=torch.float64)
    return ((r * (node + 1)).long() - 1).clamp(max=node - 1).to(torch.int32)


def _prepare_slots(case, g):
    bs, page = case["bs"], case["page"]
    if case["ragged"]:
        p = _ints(g, case["prefix"] // 8, case["prefix"], bs)
        n = _ints(g, 1, case["tree"], bs)
    else:
        p = torch.full((bs,), case["prefix"], dtype=torch.int32, device="cuda")
        n = torch.full((bs,), case["tree"], dtype=torch.int32, device="cuda")
    max_pages = (case["prefix"] + case["tree"] + page - 1) // page
    num_rows = bs + 3  # a few rows of the table belong to nobody in this batch
    pages = num_rows * max_pages
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).reshape(num_rows, max_pages)
    kv, q = bs * case["prefix"], bs * case["tree"]  # capacities: a ragged batch leaves the ends as they are
    return {"case": case, "p": p, "n": n, "parents": _trees(case, bs, n.tolist(), g), "table": table,
            "rows": torch.randperm(num_rows, generator=g, device="cuda")[:bs].to(torch.int32), "num_pages": pages,
            "kv_indptr": torch.zeros(bs + 1, dtype=torch.int32, device="cuda"),
            "kv_indices": torch.zeros(kv, dtype=torch.int64, device="cuda"),
            "qo_indptr": torch.zeros(bs + 1, dtype=torch.int64, device="cuda"),
            "out_cache_loc": torch.zeros(q, dtype=torch.int64, device="cuda"),
            "positions": torch.zeros(q, dtype=torch.int64, device="cuda")}


def _prepare_pages(case, g):
    rows, page = case["rows"], case["page"]
    before = _ints(g, 0, case["held"], rows)
    after = before + _ints(g, 1, case["grow"], rows)
    max_pages = (case["held"] + case["grow"] + page - 1) // page
    held = (before + page - 1) // page
    taken = int(held.sum())
    pages = rows * max_pages + 5
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((rows, max_pages), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(max_pages, device="cuda")[None] < held[:, None]] = order[:taken]
    free = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    free[:pages - taken] = order[taken:]
    return {"case": case, "before": before, "after": after, "table": table, "held": held.to(torch.int32), "free": free,
            "num_free": torch.tensor([pages - taken], dtype=torch.int32, device="cuda")}


# -------------------------------------------------------------- one pass

_binding = None


def _own():
    global _binding
    if _binding is None:
        from paged_mla_speculative_tree_gb300 import binding
        _binding = binding
    return _binding


def run(state):
    op = state["case"]["op"]
    if op == "logprobs":
        return _run_logprobs(state)
    if op == "rope":
        return _run_rope(state)
    if op == "slots":
        return _run_slots(state)
    return _run_pages(state)


def _run_logprobs(s):
    out = {"logprobs": s["logprobs"], "stats": s["stats"], "top_tokens": s["top_tokens"],
           "top_logprobs": s["top_logprobs"]}
    if own:
        _own().token_logprobs(s["logits"], s["stats"], s["tokens"], s["logprobs"], s["top_tokens"], s["top_logprobs"],
                              token_rows=s["token_rows"], inv_temperature=s["inv_temperature"])
        return out
    logits = s["logits"].float()
    rows, vocab = logits.shape
    k = s["case"]["top"]
    scale = s["inv_temperature"][:, None] if s["inv_temperature"] is not None else 1.0
    top = logits.max(dim=1, keepdim=True).values
    d = (logits - top) * scale
    e = torch.exp(d)
    total = e.sum(dim=1)
    log_total = torch.log(total)
    weighted = torch.where(e > 0, e * d, torch.zeros_like(e)).sum(dim=1)
    out["stats"] = torch.stack([top[:, 0] * (scale[:, 0] if torch.is_tensor(scale) else scale), log_total,
                                log_total - weighted / total])
    row = s["token_rows"].long() if s["token_rows"] is not None else torch.arange(rows, device="cuda")
    out["logprobs"] = d[row, s["tokens"].long()] - log_total[row]
    # order by (logit, lowest id): the value's bits, made monotone, above the id's complement
    bits = (logits + 0.0).view(torch.int32)
    bits = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    key = (bits << 32) | (vocab - 1 - torch.arange(vocab, device="cuda"))[None]
    ids = vocab - 1 - (torch.topk(key, k, dim=1, sorted=True).values & 0xFFFFFFFF)
    value = torch.gather(logits, 1, ids)
    none = value == -math.inf
    out["top_tokens"] = torch.where(none, torch.full_like(ids, -1), ids).t().to(torch.int32)
    out["top_logprobs"] = (torch.gather(d, 1, ids) - log_total[:, None]).t()
    return out


def _rotate(x, cos, sin, layout):
    x = x.float()
    if layout == "interleaved":
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
    a, b = x[..., :ROPE // 2], x[..., ROPE // 2:]
    return torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)


def _run_rope(s):
    case = s["case"]
    if own:
        b = _own()
        b.rope_write(s["turns"], s["positions"], layout=b.ROPE_HALF if case["layout"] == "half" else b.ROPE_INTERLEAVED,
                     amplitude=s["amplitude"], q_in=s["q_in"], q_out=s["q"][:, :, LATENT:], k_in=s["k_in"],
                     c_in=s["c_in"], out_cache_loc=s["slots"], kv_pool=s["pool"], num_valid=s["valid"])
        return {"q": s["q"], "pool": s["pool"]}
    n = case["valid"]
    angle = s["positions"][:n, None].double() * s["freq"]
    cos, sin = (torch.cos(angle) * s["amplitude"]).float(), (torch.sin(angle) * s["amplitude"]).float()
    s["q"][:n, :, LATENT:] = _rotate(s["q_in"][:n], cos[:, None], sin[:, None], case["layout"]).to(s["q"].dtype)
    row = torch.cat([s["c_in"][:n].float(), _rotate(s["k_in"][:n], cos, sin, case["layout"])], dim=1)
    s["pool"][s["slots"][:n]] = row.to(torch.bfloat16)
    return {"q": s["q"], "pool": s["pool"]}


def _run_slots(s):
    names = ("kv_indptr", "kv_indices", "qo_indptr", "out_cache_loc", "positions")
    case = s["case"]
    if own:
        _own().slot_map_build(s["table"], s["p"], s["n"], case["page"], s["kv_indptr"], s["kv_indices"], s["qo_indptr"],
                              s["out_cache_loc"], s["positions"], rows=s["rows"], parents=s["parents"],
                              num_pages=s["num_pages"])
        return {k: s[k] for k in names}
    page, p, n = case["page"], s["p"].long(), s["n"].long()
    bs = p.numel()
    kv_ptr, qo_ptr = torch.zeros(bs + 1, dtype=torch.int64, device="cuda"), torch.zeros(bs + 1, dtype=torch.int64, device="cuda")
    kv_ptr[1:], qo_ptr[1:] = torch.cumsum(p, 0), torch.cumsum(n, 0)

    def slots(r, at):
        return s["table"][s["rows"].long()[r], at // page].long() * page + at % page

    r = torch.repeat_interleave(torch.arange(bs, device="cuda"), p)
    s["kv_indices"][:r.numel()] = slots(r, torch.arange(r.numel(), device="cuda") - kv_ptr[r])
    r = torch.repeat_interleave(torch.arange(bs, device="cuda"), n)
    t = torch.arange(r.numel(), device="cuda") - qo_ptr[r]
    # depth by doubling: each node's ancestor 1, 2, 4, ... steps up; -1 is above the root
    up = torch.where(s["parents"] >= 0, s["parents"] + qo_ptr[r], -1)
    depth = (up >= 0).long()
    for _ in range(max(1, case["tree"].bit_length())):
        over = up.clamp(min=0)
        depth = depth + torch.where(up >= 0, depth[over], 0)
        up = torch.where(up >= 0, up[over], -1)
    s["out_cache_loc"][:r.numel()] = slots(r, p[r] + t)
    s["positions"][:r.numel()] = p[r] + depth
    s["kv_indptr"].copy_(kv_ptr)
    s["qo_indptr"].copy_(qo_ptr)
    return {k: s[k] for k in names}


def _pages_to(s, lens):
    """Every row grown or shrunk to hold lens tokens: released pages go on top
    of the free list, the last row's last page first; new pages come off it."""
    page, table, held, free, num = s["case"]["page"], s["table"], s["held"], s["free"], s["num_free"]
    need = (lens + page - 1) // page

    def items(lo, hi):
        """(row, page index) of entries [lo, hi) of every row, in order."""
        c = (hi - lo).clamp(min=0).long()
        r = torch.repeat_interleave(torch.arange(c.numel(), device="cuda"), c)
        return r, lo.long()[r] + torch.arange(r.numel(), device="cuda") - (torch.cumsum(c, 0) - c)[r]

    out_r, out_j = items(need, held)
    in_r, in_j = items(held, need)
    free[num.long() + out_r.numel() - 1 - torch.arange(out_r.numel(), device="cuda")] = table[out_r, out_j]
    num += out_r.numel()
    table[in_r, in_j] = free[num.long() - 1 - torch.arange(in_r.numel(), device="cuda")]
    num -= in_r.numel()
    held.copy_(need)


def _run_pages(s):
    if own:
        update, page = _own().page_table_update, s["case"]["page"]
        update(s["after"], page, s["table"], s["held"], s["free"], s["num_free"])
        update(s["before"], page, s["table"], s["held"], s["free"], s["num_free"])
    else:
        _pages_to(s, s["after"])
        _pages_to(s, s["before"])
    return {k: s[k] for k in ("table", "held", "free", "num_free")}


# ------------------------------------------------------ floors and 64 bits

def work(case):
    if case["op"] == "logprobs":
        read = case["rows"] * case["vocab"] * SIZES[case["dtype"]]
        return {"bytes": read + case["rows"] * (16 + 8 * case["top"]) + 12 * case["tokens"],
                "flops": 6 * case["rows"] * case["vocab"]}
    if case["op"] == "rope":
        e, n = SIZES[case["dtype"]], case["valid"]
        return {"bytes": n * (2 * HEADS * ROPE * e + ROW * (e + 2) + 16), "flops": 3 * n * (HEADS + 1) * ROPE}
    if case["op"] == "slots":
        mean = 9 / 16 if case["ragged"] else 1.0
        kv, q = mean * case["bs"] * case["prefix"], (0.5 if case["ragged"] else 1.0) * case["bs"] * case["tree"]
        return {"bytes": kv * (8 + 4 / case["page"]) + q * 20 + 24 * case["bs"], "flops": 0}
    moved = case["rows"] * max(1, case["grow"] / 2 / case["page"])
    return {"bytes": 2 * moved * 8 + 24 * case["rows"], "flops": 0}


def exact(case, seed):
    s = prepare(case, seed)
    return {"logprobs": _exact_logprobs, "rope": _exact_rope}.get(case["op"], _exact_whole)(s)


def _exact_whole(s):
    """Slot maps and page tables are whole numbers: there is nothing to round."""
    return None


def _exact_logprobs(s):
    logits, n, k = s["logits"], s["tokens"].numel(), s["case"]["top"]
    rows, vocab = logits.shape
    lse = torch.empty(rows, dtype=torch.float64, device="cuda")
    top, entropy = torch.empty_like(lse), torch.empty_like(lse)
    best = torch.empty((k, rows), dtype=torch.float64, device="cuda")
    scale = s["inv_temperature"].double() if s["inv_temperature"] is not None else torch.ones_like(lse)
    for a in range(0, rows, 64):
        z = logits[a:a + 64].double() * scale[a:a + 64, None]
        lse[a:a + 64] = torch.logsumexp(z, dim=1)
        top[a:a + 64] = z.amax(dim=1)
        lp = z - lse[a:a + 64, None]
        entropy[a:a + 64] = -(lp.exp() * lp.clamp(min=-1e4)).sum(dim=1)
        best[:, a:a + 64] = torch.sort(lp, dim=1, descending=True).values[:, :k].t()
    row = s["token_rows"].long() if s["token_rows"] is not None else torch.arange(n, device="cuda")
    given = logits[row, s["tokens"].long()].double() * scale[row] - lse[row]
    return {"logprobs": given, "stats": torch.stack([top, lse - top, entropy]), "top_tokens": None, "top_logprobs": best}


def _exact_rope(s):
    """The pairs as complex numbers, turned by exp(i * position * frequency)."""
    case, n = s["case"], s["case"]["valid"]
    turn = torch.polar(torch.full((n, ROPE // 2), s["amplitude"], dtype=torch.float64, device="cuda"),
                       torch.remainder(s["positions"][:n, None].double() * s["freq"], 2 * math.pi))

    def turned(x, w):
        x = x.double()
        pairs = x.unflatten(-1, (-1, 2)) if case["layout"] == "interleaved" else x.unflatten(-1, (2, -1)).transpose(-1, -2)
        y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * w)
        return (y if case["layout"] == "interleaved" else y.transpose(-1, -2)).flatten(-2)

    q, pool = s["q"].double(), s["pool"].double()
    q[:n, :, LATENT:] = turned(s["q_in"][:n], turn[:, None])
    pool[s["slots"][:n]] = torch.cat([s["c_in"][:n].double(), turned(s["k_in"][:n], turn)], dim=1)
    return {"q": q, "pool": pool}
