"""Measured cases of the group-rollout operators, with their plain forms.

Four operators of a rollout that samples groups of responses with filters, and
of the learner that scores what it sampled:

* ``tables``  block tables and the slot map of the tokens a step adds;
* ``attn``    decode attention of groups that share a prompt's cache;
* ``sample``  temperature, top-k, top-p and min-p sampling from given uniforms;
* ``keep``    the logprob over the kept tokens, forward and backward.
"""

import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a small server: every response adds one token
        {"name": "tables_step_64", "op": "tables", "B": 64, "page": 16, "len_lo": 0,
         "len_hi": 8192, "new_lo": 1, "new_hi": 1, "shape_seed": 1},
        # admission of many prompts at once: whole prompts get pages and slots
        {"name": "tables_admit_3000", "op": "tables", "B": 3000, "page": 16, "len_lo": 0,
         "len_hi": 0, "new_lo": 1, "new_hi": 2048, "shape_seed": 2},
        # one prompt, eight fresh responses: latency
        {"name": "attn_one_prompt", "op": "attn", "dtype": "bf16", "prompts": 1, "per": 8,
         "ragged": False, "pre_lo": 700, "pre_hi": 700, "len_lo": 1, "len_hi": 64, "Hq": 12,
         "Hkv": 2, "D": 128, "page": 16, "shape_seed": 3},
        # ragged groups, empty prompts and responses, odd pages, one head a KV head
        {"name": "attn_ragged_mha", "op": "attn", "dtype": "f16", "prompts": 7, "per": 5,
         "ragged": True, "pre_lo": 0, "pre_hi": 3000, "len_lo": 0, "len_hi": 900, "Hq": 16,
         "Hkv": 16, "D": 64, "page": 24, "shape_seed": 4},
        # the 16 x 8 batch of a long-response run, half way through
        {"name": "attn_group_16x8", "op": "attn", "dtype": "bf16", "prompts": 16, "per": 8,
         "ragged": False, "pre_lo": 512, "pre_hi": 4096, "len_lo": 1024, "len_hi": 8192, "Hq": 32,
         "Hkv": 8, "D": 128, "page": 16, "shape_seed": 5},
        # long shared contexts with many responses each, early in their decode
        {"name": "attn_long_prefix", "op": "attn", "dtype": "bf16", "prompts": 4, "per": 32,
         "ragged": False, "pre_lo": 50000, "pre_hi": 98304, "len_lo": 1, "len_hi": 512, "Hq": 32,
         "Hkv": 8, "D": 128, "page": 64, "shape_seed": 6},
        # a single stream's next token: latency
        {"name": "sample_one_row", "op": "sample", "dtype": "f32", "T": 1, "V": 151936, "pad": 0,
         "filters": "p", "std": 2.0, "peak": 10.0, "keep": False, "shape_seed": 7},
        # a batch of requests, each with its own filters, logits of the LM head in fp32
        {"name": "sample_mixed_64", "op": "sample", "dtype": "f32", "T": 64, "V": 151936,
         "pad": 0, "filters": "mixed", "std": 2.0, "peak": 9.0, "keep": True, "shape_seed": 8},
        # a large rollout batch with nucleus sampling, bf16 logits, flat rows among them
        {"name": "sample_nucleus_512", "op": "sample", "dtype": "bf16", "T": 512, "V": 151936,
         "pad": 0, "filters": "p", "std": 3.0, "peak": 0.0, "keep": True, "shape_seed": 9},
        # a short response scored under its kept tokens: odd vocabulary, padded rows
        {"name": "keep_odd_small", "op": "keep", "dtype": "f16", "T": 33, "V": 32003, "pad": 5,
         "kept_hi": 64, "std": 2.0, "shape_seed": 10},
        # learner rows with the rollout's kept sets
        {"name": "keep_rows_4096", "op": "keep", "dtype": "bf16", "T": 4096, "V": 151936,
         "pad": 0, "kept_hi": 256, "std": 2.0, "shape_seed": 11},
        # learner rows of an unfiltered rollout at a temperature, fp32 logits
        {"name": "keep_all_1024", "op": "keep", "dtype": "f32", "T": 1024, "V": 151936,
         "pad": 0, "kept_hi": 0, "std": 2.0, "shape_seed": 12},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "attn", "attn", "sample", "sample", "keep", "keep"])
    seed = rng.randrange(1 << 30)
    if op == "tables":
        admit = rng.random() < 0.5
        return {"op": op, "B": _log(rng, 1, 3000), "page": rng.choice([1, 8, 16, 24, 64, 100]),
                "len_lo": 0, "len_hi": 0 if admit else _log(rng, 16, 8192), "new_lo": 0,
                "new_hi": _log(rng, 2, 1024) if admit else rng.randint(1, 4), "shape_seed": seed}
    if op == "attn":
        hkv = rng.choice([1, 2, 4, 8, 16])
        prompts, per, rep = _log(rng, 1, 16), _log(rng, 1, 32), rng.choice([1, 2, 4, 6, 8])
        most = min(200_000_000, 30_000_000_000 // (per * rep)) // (hkv * prompts * 128)
        pre = max(1, min(_log(rng, 1, 98304), most))
        own_len = max(1, min(_log(rng, 1, 8192), most // per))
        return {"op": op, "dtype": rng.choice(["bf16", "f16"]), "prompts": prompts, "per": per,
                "ragged": rng.random() < 0.5, "pre_lo": rng.choice([0, pre // 2]), "pre_hi": pre,
                "len_lo": rng.choice([0, own_len // 2]), "len_hi": own_len,
                "Hq": hkv * rep, "Hkv": hkv,
                "D": rng.choice([64, 80, 96, 128]), "page": rng.choice([8, 16, 24, 64, 100]),
                "shape_seed": seed}
    V = rng.choice([151936, _log(rng, 100, 151936)])
    T = _log(rng, 1, max(2, min(4096, 70_000_000 // V)))
    common = {"op": op, "dtype": rng.choice(["f32", "bf16", "f16"]), "T": T, "V": V,
              "pad": rng.choice([0, 0, rng.randint(1, 40)]), "std": rng.choice([0.5, 2.0, 3.0]),
              "shape_seed": seed}
    if op == "sample":
        return {**common, "filters": rng.choice(["p", "k", "min_p", "mixed", "none"]),
                "peak": rng.choice([0.0, 5.0, 10.0]), "keep": rng.random() < 0.7}
    return {**common, "kept_hi": rng.choice([0, _log(rng, 1, min(V // 2, 2048))])}


# ------------------------------------------------------------------ shapes (a case's alone)
def _table_lens(case):
    rng = random.Random(case["shape_seed"])
    lens = [rng.randint(case["len_lo"], case["len_hi"]) for _ in range(case["B"])]
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["B"])]
    return lens, new


def _attn_lens(case):
    rng = random.Random(case["shape_seed"])
    sizes = [rng.randint(0, 2 * case["per"] - 1) if case["ragged"] else case["per"]
             for _ in range(case["prompts"])]
    if sum(sizes) == 0:
        sizes[0] = 1
    pre = [rng.randint(case["pre_lo"], case["pre_hi"]) for _ in sizes]
    lens = [rng.randint(case["len_lo"], case["len_hi"]) for _ in range(sum(sizes))]
    return sizes, pre, lens


def _kept_counts(case):
    rng = random.Random(case["shape_seed"])
    hi = min(case["kept_hi"], case["V"])
    return [_log(rng, 1, hi) for _ in range(case["T"])]


def work(case):
    op = case["op"]
    if op == "tables":
        p = case["page"]
        lens, new = _table_lens(case)
        fresh = sum(-(-(a + b) // p) - -(-a // p) for a, b in zip(lens, new))
        B = case["B"]
        return {"bytes": 8 * B + 8 * fresh + 8 * sum(new) + 8 * (B + 1), "flops": 4 * sum(new)}
    if op == "attn":
        sizes, pre, lens = _attn_lens(case)
        B = sum(sizes)
        tokens = sum(a for a, n in zip(pre, sizes) if n) + sum(lens)
        pairs = sum(a * n for a, n in zip(pre, sizes)) + sum(lens)
        return {"bytes": tokens * 2 * case["Hkv"] * case["D"] * 2 +
                B * case["Hq"] * (case["D"] * 4 + 4),
                "flops": 4 * case["Hq"] * case["D"] * pairs}
    T, V = case["T"], case["V"]
    size = 4 if case["dtype"] == "f32" else 2
    words = (V + 31) // 32
    if op == "sample":
        return {"bytes": T * (V * size + (words * 4 if case["keep"] else 0) + 32),
                "flops": 6 * T * V}
    kept = sum(_kept_counts(case)) if case["kept_hi"] else T * V
    mask = T * words * 4 if case["kept_hi"] else 0
    return {"bytes": mask + kept * size + T * V * size + T * 24, "flops": 10 * kept}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _logits(case, g):
    T, V = case["T"], case["V"]
    z = torch.empty(T, V + case["pad"], dtype=DTYPES[case["dtype"]], device="cuda")
    z.normal_(0.0, case["std"], generator=g)
    if case.get("peak"):
        # some twenty likely tokens a row, as a language model's rows have them
        n = min(20, V)
        at = torch.randint(0, V, (T, n), generator=g, device="cuda")
        up = case["peak"] * (0.4 + 0.6 * torch.rand(T, n, generator=g, device="cuda"))
        z.scatter_(1, at, up.to(z.dtype))
    if V >= 64:
        z[:, 17:V:1009] = float("-inf")  # tokens that are never to be sampled
    return z[:, :V]


def _prepare_tables(case, seed):
    g = _gen(seed)
    lens, new = _table_lens(case)
    p, B = case["page"], case["B"]
    width = max(1, max(-(-(a + b) // p) for a, b in zip(lens, new)))
    old = torch.tensor([-(-a // p) for a in lens], device="cuda")
    n_old = int(old.sum())
    fresh = sum(-(-(a + b) // p) - -(-a // p) for a, b in zip(lens, new))
    pages = torch.randperm(n_old + fresh + 5, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    have = torch.arange(width, device="cuda") < old[:, None]
    table[have] = pages[:n_old]
    return {"table": table, "free": pages[n_old:].contiguous(), "page": p, "n_slots": sum(new),
            "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
            "new": torch.tensor(new, dtype=torch.int32, device="cuda")}


def _pages(counts, perm, first):
    width = max(1, max(counts, default=1))
    table = torch.full((len(counts), width), -1, dtype=torch.int32, device="cuda")
    have = torch.arange(width, device="cuda") < torch.tensor(counts, device="cuda")[:, None]
    table[have] = perm[first:first + sum(counts)]
    return table


def _prepare_attn(case, seed):
    g = _gen(seed)
    sizes, pre, lens = _attn_lens(case)
    p, hkv, D, dt = case["page"], case["Hkv"], case["D"], DTYPES[case["dtype"]]
    B = sum(sizes)
    n_pre, n_own = [-(-a // p) for a in pre], [-(-a // p) for a in lens]
    n_pages = sum(n_pre) + sum(n_own) + 3
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    k = torch.empty(n_pages, p, hkv, D, dtype=dt, device="cuda").normal_(generator=g)
    v = torch.empty(n_pages, p, hkv, D, dtype=dt, device="cuda").normal_(generator=g)
    q = torch.empty(B, case["Hq"], D, dtype=dt, device="cuda").normal_(0, 2, generator=g)
    cu = [0]
    for n in sizes:
        cu.append(cu[-1] + n)
    group = [i for i, n in enumerate(sizes) for _ in range(n)]
    place = [j for n in sizes for j in range(n)]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"q": q, "k": k, "v": v, "prefix_table": _pages(n_pre, perm, 0),
            "prefix_lens": i32(pre), "cu_group": i32(cu),
            "table": _pages(n_own, perm, sum(n_pre)), "lens": i32(lens),
            "group": torch.tensor(group, device="cuda"),
            "place": torch.tensor(place, device="cuda"), "most": max(sizes)}


def _prepare_sample(case, seed):
    g = _gen(seed)
    T, V = case["T"], case["V"]
    rng = random.Random(case["shape_seed"])
    kind = case["filters"]
    pick = {"k": lambda: (rng.choice([1, 20, 50, 1000]), 1.0, 0.0),
            "p": lambda: (0, rng.choice([0.8, 0.9, 0.95, 0.99]), 0.0),
            "min_p": lambda: (0, 1.0, rng.choice([0.02, 0.05, 0.1])),
            "none": lambda: (0, 1.0, 0.0)}
    rows = [pick[kind if kind != "mixed" else rng.choice(["k", "p", "min_p", "none", "all"])]()
            if kind != "mixed" else
            (rng.choice([0, 1, 40, 500]), rng.choice([1.0, 0.9, 0.97]),
             rng.choice([0.0, 0.01, 0.05])) for _ in range(T)]
    temp = [rng.choice([1.0, 1.0, 0.7, 1.3] + ([0.0] if kind == "mixed" else []))
            for _ in range(T)]
    f32 = lambda x: torch.tensor(x, dtype=torch.float32, device="cuda")  # noqa: E731
    return {"logits": _logits(case, g), "keep": case["keep"], "temperature": f32(temp),
            "top_k": torch.tensor([r[0] for r in rows], dtype=torch.int32, device="cuda"),
            "top_p": f32([r[1] for r in rows]), "min_p": f32([r[2] for r in rows]),
            "uniform": torch.rand(T, generator=g, device="cuda")}


def _pack(kept):
    T, V = kept.shape
    words = torch.zeros(T, (V + 31) // 32 * 32, dtype=torch.bool, device=kept.device)
    words[:, :V] = kept
    bit = (1 << torch.arange(32, device=kept.device)).to(torch.int32)  # bit 31 wraps to the sign
    return (words.view(T, -1, 32) * bit).sum(-1, dtype=torch.int32)


def _prepare_keep(case, seed):
    g = _gen(seed)
    T, V = case["T"], case["V"]
    logits = _logits({**case, "peak": 0.0}, g)
    rng = random.Random(case["shape_seed"])
    temp = torch.tensor([rng.choice([1.0, 0.7, 1.3]) for _ in range(T)], device="cuda")
    keep = None
    if case["kept_hi"]:
        # the rollout's weights were others: its likeliest tokens are not quite these
        n = torch.tensor(_kept_counts(case), device="cuda")
        most = int(n.max())
        keep = torch.empty(T, (V + 31) // 32, dtype=torch.int32, device="cuda")
        tokens = torch.empty(T, dtype=torch.int32, device="cuda")
        for r in range(0, T, 256):
            z = logits[r:r + 256].float()
            z += 0.3 * torch.randn(z.shape, generator=g, device="cuda")
            at = z.topk(most, dim=1).indices
            kept = torch.zeros(z.shape, dtype=torch.bool, device="cuda")
            kept.scatter_(1, at, torch.arange(most, device="cuda") < n[r:r + 256, None])
            keep[r:r + 256] = _pack(kept)
            choice = (torch.rand(len(z), generator=g, device="cuda") * n[r:r + 256]).long()
            tokens[r:r + 256] = at.gather(1, choice[:, None])[:, 0].to(torch.int32)
    else:
        tokens = (torch.randint(0, (V + 1) // 2, (T,), generator=g, device="cuda") * 2
                  ).clamp(max=V - 1).to(torch.int32)
        if V >= 64:
            tokens = torch.where((tokens - 17) % 1009 == 0, tokens - 1, tokens)
    coef = torch.randn(T, generator=g, device="cuda") / T
    return {"logits": logits, "tokens": tokens, "keep": keep, "temperature": temp, "coef": coef}


def prepare(case, seed):
    make = {"tables": _prepare_tables, "attn": _prepare_attn, "sample": _prepare_sample,
            "keep": _prepare_keep}
    return {"op": case["op"], **make[case["op"]](case, seed)}


# ------------------------------------------------------------------ the framework's calls
def _own_tables(s):
    import invariant_logprobs_gb300 as rz
    slots, cu, used = rz.rz_page_tables(s["lens"], s["new"], s["free"], s["page"], s["table"],
                                        s["n_slots"])
    return {"table": s["table"], "slots": slots, "cu": cu, "used": used}


def _own_attn(s):
    import invariant_logprobs_gb300 as rz
    out, lse = rz.rz_group_decode_attn(s["q"], s["k"], s["v"], s["table"], s["lens"],
                                       prefix_table=s["prefix_table"],
                                       prefix_lens=s["prefix_lens"], cu_group=s["cu_group"])
    return {"out": out, "lse": lse}


def _own_sample(s):
    import invariant_logprobs_gb300 as rz
    tokens, logprob, kept, keep = rz.rz_filter_sample(
        s["logits"], s["uniform"], temperature=s["temperature"], top_k=s["top_k"],
        top_p=s["top_p"], min_p=s["min_p"], want_keep=s["keep"])
    out = {"tokens": tokens, "logprob": logprob, "kept": kept}
    return {**out, "keep": keep} if s["keep"] else out


def _own_keep(s):
    import invariant_logprobs_gb300 as rz
    logprob, lse = rz.rz_keep_logprob(s["logits"], s["tokens"], keep=s["keep"],
                                      temperature=s["temperature"])
    dlogits = rz.rz_keep_logprob_bwd(s["logits"], s["tokens"], lse, s["coef"], keep=s["keep"],
                                     temperature=s["temperature"])
    return {"logprob": logprob, "lse": lse, "dlogits": dlogits}


# ------------------------------------------------------------------ plain forms
def _plain_tables(s):
    p, table, lens, new = s["page"], s["table"], s["lens"].long(), s["new"].long()
    zero = torch.zeros(1, dtype=torch.int64, device=table.device)
    old, full = (lens + p - 1) // p, (lens + new + p - 1) // p
    first = torch.cat([zero, torch.cumsum(full - old, 0)])
    col = torch.arange(table.shape[1], device=table.device)
    at = (first[:-1, None] + col - old[:, None]).clamp(0, len(s["free"]) - 1)
    table.copy_(torch.where((col >= old[:, None]) & (col < full[:, None]), s["free"][at], table))
    cu = torch.cat([zero, torch.cumsum(new, 0)])
    t = torch.arange(s["n_slots"], device=table.device)
    req = torch.searchsorted(cu[1:], t, right=True)
    pos = lens[req] + t - cu[req]
    return {"table": table, "slots": table[req, pos // p].long() * p + pos % p, "cu": cu,
            "used": first[-1:].to(torch.int32)}


def _gathered(cache, table):
    rows = cache[table.clamp(min=0).long()].float()
    return rows.flatten(1, 2)  # [rows, tokens, Hkv, D]


def _plain_attn(s):
    q, (B, Hq, D) = s["q"].float(), s["q"].shape
    hkv, P, most = s["k"].shape[2], len(s["prefix_lens"]), s["most"]
    q = (q / math.sqrt(D)).view(B, hkv, Hq // hkv, D)
    by_group = torch.zeros(P, most, hkv, Hq // hkv, D, device=q.device)
    by_group[s["group"], s["place"]] = q
    seen = lambda n, t: torch.arange(t, device=q.device) < n[:, None]  # noqa: E731
    pk, pv = _gathered(s["k"], s["prefix_table"]), _gathered(s["v"], s["prefix_table"])
    ok, ov = _gathered(s["k"], s["table"]), _gathered(s["v"], s["table"])
    a = torch.einsum("pghrd,pthd->pghrt", by_group, pk)
    a = torch.where(seen(s["prefix_lens"], a.shape[-1])[:, None, None, None], a, -math.inf)
    b = torch.einsum("bhrd,bthd->bhrt", q, ok)
    b = torch.where(seen(s["lens"], b.shape[-1])[:, None, None], b, -math.inf)
    m_a, m_b = a.amax(-1, keepdim=True), b.amax(-1, keepdim=True)
    mine = lambda x: x[s["group"], s["place"]]  # noqa: E731
    m = torch.maximum(mine(m_a), m_b)
    safe = torch.where(m > -math.inf, m, 0.0)
    safe_a = torch.zeros_like(m_a)
    safe_a[s["group"], s["place"]] = safe
    ea, eb = torch.exp(a - safe_a), torch.exp(b - safe)
    total = mine(ea.sum(-1, keepdim=True)) + eb.sum(-1, keepdim=True)
    out = mine(torch.einsum("pghrt,pthd->pghrd", ea, pv)) + torch.einsum("bhrt,bthd->bhrd", eb, ov)
    out = torch.where(total > 0, out / total, 0.0)
    lse = safe + torch.log(total)
    return {"out": out.reshape(B, Hq, D).to(s["q"].dtype), "lse": lse.reshape(B, Hq)}


def _plain_sample(s):
    z = s["logits"].float()
    T, V = z.shape
    greedy = s["temperature"] == 0
    tau = torch.where(greedy, 1.0, s["temperature"]).double()[:, None]
    k = torch.where(s["top_k"] > 0, s["top_k"], V)
    k = torch.where(greedy, 1, k)[:, None]
    p, min_p = s["top_p"].double()[:, None], s["min_p"].double()[:, None]
    v, at = torch.sort(z, dim=-1, descending=True, stable=True)
    x = (v.double() - v[:, :1].double()) / tau
    w = torch.exp(x)
    rank = torch.arange(V, device=z.device)
    mass = torch.where(rank < k, w, 0.0)
    before = torch.cumsum(mass, -1) - mass
    total = mass.sum(-1, keepdim=True)
    fits = (rank < k) & ((before < p * total) | (p >= 1) | (rank == 0))
    fits &= (x >= torch.log(min_p)) & (v > -math.inf)
    kept = torch.zeros(T, V, dtype=torch.bool, device=z.device).scatter_(1, at, fits)
    x = (z.double() - v[:, :1].double()) / tau
    cum = torch.cumsum(torch.where(kept, torch.exp(x), 0.0), -1)
    mass = cum[:, -1:]
    token = (cum <= s["uniform"].double()[:, None] * mass).sum(-1, keepdim=True)
    logprob = (x.gather(1, token) - torch.log(mass))[:, 0].float()
    out = {"tokens": token[:, 0].to(torch.int32), "logprob": logprob,
           "kept": fits.sum(-1).to(torch.int32)}
    return {**out, "keep": _pack(kept)} if s["keep"] else out


def _unpack(words, V):
    bit = torch.arange(32, dtype=torch.int32, device=words.device)
    return (((words[:, :, None] >> bit) & 1) != 0).flatten(1)[:, :V]


def _plain_keep(s):
    tau = s["temperature"][:, None]
    x = s["logits"].float() / tau
    if s["keep"] is not None:
        x = torch.where(_unpack(s["keep"], x.shape[1]), x, -math.inf)
    m = x.amax(-1, keepdim=True)
    lse = m + torch.log(torch.exp(x - m).sum(-1, keepdim=True))
    token = s["tokens"].long()[:, None]
    logprob = x.gather(1, token) - lse
    g = s["coef"][:, None] / tau
    d = -g * torch.exp(x - lse)
    d.scatter_add_(1, token, g)
    return {"logprob": logprob[:, 0], "lse": lse[:, 0], "dlogits": d.to(s["logits"].dtype)}


def run(state):
    if own:
        return {"tables": _own_tables, "attn": _own_attn, "sample": _own_sample,
                "keep": _own_keep}[state["op"]](state)
    return {"tables": _plain_tables, "attn": _plain_attn, "sample": _plain_sample,
            "keep": _plain_keep}[state["op"]](state)


# ------------------------------------------------------------------ in 64 bits
def _exact_attn(s, case):
    sizes, pre, lens = _attn_lens(case)
    B, Hq, D = s["q"].shape
    hkv = s["k"].shape[2]
    rep = Hq // hkv
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")

    def cached(cache, pages, n, h):
        return cache[pages.long(), :, h].double().flatten(0, 1)[:n]

    first = 0
    for i, n in enumerate(sizes):
        n_pages = -(-pre[i] // case["page"])
        for h in range(hkv):
            heads = slice(h * rep, (h + 1) * rep)
            pages = s["prefix_table"][i, :n_pages]
            pk, pv = cached(s["k"], pages, pre[i], h), cached(s["v"], pages, pre[i], h)
            for b in range(first, first + n):
                mine = s["table"][b, :-(-lens[b] // case["page"])]
                key = torch.cat([pk, cached(s["k"], mine, lens[b], h)])
                val = torch.cat([pv, cached(s["v"], mine, lens[b], h)])
                if len(key):
                    score = s["q"][b, heads].double() @ key.T * D ** -0.5
                    lse[b, heads] = torch.logsumexp(score, -1)
                    out[b, heads] = torch.softmax(score, -1) @ val
        first += n
    return {"out": out, "lse": lse}


def _exact_sample(s):
    lps = []
    T, V = s["logits"].shape
    for r in range(T):
        tau, k = float(s["temperature"][r]), int(s["top_k"][r])
        p, min_p = float(s["top_p"][r]), float(s["min_p"][r])
        if tau == 0:
            lps.append(0.0)
            continue
        order = torch.sort(-s["logits"][r].double(), stable=True)
        x = (order.values[0] - order.values) / tau
        n = k if 0 < k < V else V
        n = min(n, int((x > -math.inf).sum()))
        head = torch.exp(x[:n])
        if p < 1:
            part = torch.cumsum(head, 0) / head.sum()
            n = min(n, 1 + int((part < p).sum()))
        if min_p > 0:
            n = min(n, int((torch.exp(x) >= min_p).sum()))
        mine = order.indices[:n].sort().values
        prob = torch.softmax((s["logits"][r].double() / tau)[mine], 0)
        j = int((torch.cumsum(prob, 0) <= float(s["uniform"][r])).sum())
        lps.append(math.log(float(prob[min(j, n - 1)])))
    logprob = torch.tensor(lps, dtype=torch.float64, device="cuda")
    out = {"tokens": None, "logprob": logprob, "kept": None}
    return {**out, "keep": None} if s["keep"] else out


def _exact_keep(s):
    T, V = s["logits"].shape
    logprob, lse = [], []
    d = torch.zeros(T, V, dtype=torch.float64, device="cuda")
    bit = torch.arange(V, device="cuda")
    for r in range(T):
        x = s["logits"][r].double() / s["temperature"][r].double()
        if s["keep"] is not None:
            x = x.masked_fill((s["keep"][r][bit // 32] >> (bit % 32)) & 1 == 0, -math.inf)
        lp = torch.log_softmax(x, 0)
        a = s["tokens"][r].long()
        lse.append(torch.logsumexp(x, 0))
        logprob.append(lp[a])
        d[r] = -torch.exp(lp)
        d[r, a] += 1
        d[r] *= s["coef"][r].double() / s["temperature"][r].double()
    return {"logprob": torch.stack(logprob), "lse": torch.stack(lse), "dlogits": d}


def exact(case, seed):
    if case["op"] == "tables":
        return None
    s = prepare(case, seed)
    if case["op"] == "attn":
        return _exact_attn(s, case)
    return _exact_sample(s) if case["op"] == "sample" else _exact_keep(s)
