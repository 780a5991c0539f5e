"""The operators around a verification round, as cases that can be timed and compared.

A round of speculative decoding draws draft tokens, runs the target (and the
drafter) over the new tokens against a paged key-value cache, and verifies.
Each case is one call of that loop:

``sample``    tokens drawn from logits under temperature, top-k, top-p and
              min-p, by inverse CDF from given uniforms (``spec_sample``)
``truncate``  the same truncation written as logits, -inf outside, which keeps
              verification lossless for truncated sampling (``spec_truncate``)
``append``    keys and values of the new tokens written into the cache's pages
              (``spec_kv_append``)
``attend``    attention of a chunk of new tokens per request over its pages,
              causal (the target's pass, single tokens, prompts) or not (a block
              drafter's), with grouped heads (``spec_paged_attention``)

``run`` computes them in elementary torch operations, or through the
library's entry points where ``own`` is true.
"""

import math
import random

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # One token of one request: the latency of a sampling step.
        {"name": "sample_one_row", "op": "sample", "B": 1, "n": 1, "V": 151936, "dtype": "bf16",
         "mix": "all"},
        # Requests without top-k over an odd vocabulary in single precision.
        {"name": "sample_odd", "op": "sample", "B": 37, "n": 1, "V": 50021, "dtype": "f32",
         "mix": "top_p"},
        # The draft tokens of a serving batch: 128 requests of 16 positions.
        {"name": "sample_128_requests", "op": "sample", "B": 128, "n": 16, "V": 151936,
         "dtype": "bf16", "mix": "all"},
        # The target's rows of one request, 16 drafts and the bonus position.
        {"name": "truncate_one_request", "op": "truncate", "B": 1, "n": 17, "V": 151936,
         "dtype": "bf16", "mix": "all"},
        # The target's rows of 32 requests in single precision.
        {"name": "truncate_32_requests", "op": "truncate", "B": 32, "n": 17, "V": 151936,
         "dtype": "f32", "mix": "all"},
        # The new tokens of 32 verified requests, up to 17 each.
        {"name": "append_verify", "op": "append", "B": 32, "new": 17, "ragged": True,
         "context": 4096, "heads": 32, "kv_heads": 8, "width": 128, "page": 16},
        # Prompts: 16 requests of 2048 tokens.
        {"name": "append_prompts", "op": "append", "B": 16, "new": 2048, "ragged": False,
         "context": 0, "heads": 32, "kv_heads": 8, "width": 128, "page": 64},
        # One token of one request: latency.
        {"name": "attend_one_token", "op": "attend", "B": 1, "new": 1, "ragged": False,
         "context": 8000, "heads": 32, "kv_heads": 8, "width": 128, "page": 16, "causal": True,
         "window": 0},
        # Single tokens of a serving batch with long contexts.
        {"name": "attend_decode_64", "op": "attend", "B": 64, "new": 1, "ragged": False,
         "context": 16384, "heads": 32, "kv_heads": 8, "width": 128, "page": 64, "causal": True,
         "window": 0},
        # Verification of 32 requests, each with its own length of up to 17 tokens.
        {"name": "attend_verify_32", "op": "attend", "B": 32, "new": 17, "ragged": True,
         "context": 8192, "heads": 32, "kv_heads": 8, "width": 128, "page": 16, "causal": True,
         "window": 0},
        # A small block drafter: blocks of 16 positions that see each other; odd sharing of heads.
        {"name": "attend_block_drafter", "op": "attend", "B": 48, "new": 16, "ragged": False,
         "context": 1500, "heads": 14, "kv_heads": 2, "width": 64, "page": 32, "causal": False,
         "window": 0},
        # A chunk of two prompts behind what the cache holds of them.
        {"name": "attend_prompt_chunk", "op": "attend", "B": 2, "new": 4096, "ragged": False,
         "context": 8192, "heads": 32, "kv_heads": 8, "width": 128, "page": 64, "causal": True,
         "window": 0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["sample", "truncate", "append", "attend"])
    if op in ("sample", "truncate"):
        V = _log_int(rng, 300, 151936)
        n = rng.randint(1, 17)
        B = _log_int(rng, 1, max(1, min(128, 40000000 // (n * V))))
        return {"op": op, "B": B, "n": n, "V": V, "dtype": rng.choice(["bf16", "f32"]),
                "mix": rng.choice(["all", "top_p", "top_k", "flat"])}
    case = {"op": op, "B": _log_int(rng, 1, 64), "ragged": rng.random() < 0.5,
            "new": rng.choice([1, rng.randint(2, 17), _log_int(rng, 18, 1000)]),
            "context": _log_int(rng, 1, 16384), "kv_heads": rng.choice([1, 2, 4, 8]),
            "width": rng.choice([64, 128]), "page": rng.choice([16, 32, 64, 128])}
    case["heads"] = case["kv_heads"] * rng.choice([1, 2, 3, 4, 5, 7, 8])
    if case["new"] > 17:
        case["B"] = min(case["B"], 8)
    if op == "attend":
        case["causal"] = rng.random() < 0.7
        case["window"] = rng.choice([0, 0, _log_int(rng, 16, 4096)]) if case["causal"] else 0
    return case


def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _sizes(case):
    """(new tokens, cache entries with them) of each request, the same for every seed."""
    rng = random.Random(1000003 * case["B"] + 1009 * case["context"] + case["new"])
    new = [rng.randint(1, case["new"]) if case["ragged"] else case["new"]
           for _ in range(case["B"])]
    old = [rng.randint(case["context"] // 2, case["context"]) if case["B"] > 1
           else case["context"] for _ in new]
    return new, [a + b for a, b in zip(new, old)]


def _prepare_logits(case, seed):
    B, n, V = case["B"], case["n"], case["V"]
    g = _generator(seed)
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    logits = torch.empty((B, n, V), dtype=dt, device=DEV)
    # Zipf logits over a permutation of the vocabulary per request; "flat" rows without it.
    tail = -1.1 * torch.log(torch.arange(1, V + 1, device=DEV, dtype=torch.float32))
    for b in range(B):
        z = torch.randn((n, V), generator=g, device=DEV)
        if case["mix"] != "flat":
            z += tail[torch.randperm(V, generator=g, device=DEV)]
        logits[b] = z

    def pick(values):
        return torch.tensor(values, device=DEV)[
            torch.randint(0, len(values), (B,), generator=g, device=DEV)]

    # Every request has its own settings; one in ten is greedy.
    temperature = 0.5 + 0.8 * torch.rand(B, generator=g, device=DEV)
    temperature[torch.rand(B, generator=g, device=DEV) < 0.1] = 0.0
    off = case["mix"] == "top_p"
    top_k = pick([0, 0, 0, 0] if off else [0, 20, 50, 400]).to(torch.int32)
    top_p = pick([1.0, 1.0] if case["mix"] == "top_k" else [1.0, 0.8, 0.95, 0.99]).float()
    min_p = pick([0.0, 0.0] if off else [0.0, 0.0, 0.02, 0.1]).float()
    s = {"logits": logits, "temperature": temperature, "top_k": top_k, "top_p": top_p,
         "min_p": min_p, "uniforms": torch.rand((B, n), generator=g, device=DEV)}
    if own:
        import speculative_decoding_verification_58_gb300 as sv
        s["sampler"] = sv.Sampler(logits, temperature, s["uniforms"], top_k=top_k, top_p=top_p,
                                  min_p=min_p)
    return s


def _prepare_cache(case, seed):
    g = _generator(seed)
    new, total = _sizes(case)
    B, page, Hk, D = case["B"], case["page"], case["kv_heads"], case["width"]
    pages = [-(-t // page) for t in total]
    pool = sum(pages) + 3
    order = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    # The pages of a request lie anywhere in the pool; what it does not use yet is -1.
    table = torch.full((B, max(pages) + 2), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, p in enumerate(pages):
        table[b, :p] = order[at:at + p]
        at += p
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    bf = torch.bfloat16

    def normal(*shape):
        return torch.empty(shape, dtype=bf, device=DEV).normal_(generator=g)

    s = {"k_cache": normal(pool, page, Hk, D), "v_cache": normal(pool, page, Hk, D),
         "table": table, "new": new, "total": total, "start": start,
         "new_start": torch.tensor(start, dtype=torch.int32, device=DEV),
         "kv_len": torch.tensor(total, dtype=torch.int32, device=DEV)}
    rows = start[-1]
    if case["op"] == "append":
        s["k_new"], s["v_new"] = normal(rows, Hk, D), normal(rows, Hk, D)
    else:
        # Scores of standard deviation 2.
        s["q"] = normal(rows, case["heads"], D).mul_(2.0)
        s["causal"], s["window"] = case["causal"], case["window"]
    if own:
        import speculative_decoding_verification_58_gb300 as sv
        if case["op"] == "append":
            s["cache"] = sv.PagedCache(s["k_cache"], s["v_cache"], table, s["new_start"],
                                       s["kv_len"], k_new=s["k_new"], v_new=s["v_new"])
        else:
            s["cache"] = sv.PagedCache(s["k_cache"], s["v_cache"], table, s["new_start"],
                                       s["kv_len"], q=s["q"], causal=s["causal"],
                                       window=s["window"], need_lse=True)
    return s


def prepare(case, seed):
    s = (_prepare_logits if case["op"] in ("sample", "truncate") else _prepare_cache)(case, seed)
    s["op"] = case["op"]
    return s


def _plain_kept(s):
    """Rows sorted by logit (ties: lower index first): masses in that order, which of them are
    kept, and the order; greedy rows keep their first."""
    z = s["logits"].flatten(0, 1)
    n = s["logits"].shape[1]

    def rows(t):
        return t.repeat_interleave(n)[:, None]

    T = rows(s["temperature"]).double()
    greedy = T == 0
    zs, order = torch.sort(z, dim=1, descending=True, stable=True)
    zs = zs.double()
    x = (zs - zs[:, :1]) / torch.where(greedy, 1.0, T)
    mass = torch.exp(x)
    place = torch.arange(z.shape[1], device=z.device)[None, :]
    k = rows(s["top_k"])
    keep = place < torch.where(k > 0, k, z.shape[1])
    mass = torch.where(keep, mass, 0.0)
    upto = torch.cumsum(mass, 1)
    p = rows(s["top_p"]).double()
    # An entry belongs to the shortest prefix while what comes before it is too little.
    keep &= (p >= 1) | (upto - mass < p * upto[:, -1:])
    keep &= mass >= rows(s["min_p"]).double()
    keep &= ~greedy | (place == 0)
    return z, mass, keep, order


def _plain_sample(s):
    z, mass, keep, order = _plain_kept(s)
    p = torch.zeros_like(mass).scatter_(1, order, torch.where(keep, mass, 0.0))
    cdf = torch.cumsum(p, 1)
    level = s["uniforms"].flatten()[:, None].double() * cdf[:, -1:]
    return (cdf <= level).sum(1).to(torch.int32).view(s["uniforms"].shape)


def _plain_truncate(s):
    z, _, keep, order = _plain_kept(s)
    kept = torch.zeros_like(keep).scatter_(1, order, keep)
    return torch.where(kept, z, -math.inf).view(s["logits"].shape)


def _slots(s, b, first, last):
    """Page and slot of a request's entries first .. last - 1."""
    page = s["k_cache"].shape[1]
    at = torch.arange(first, last, device=DEV)
    return s["table"][b].long()[at // page], at % page


def _plain_append(s):
    for b, (n, total) in enumerate(zip(s["new"], s["total"])):
        page, slot = _slots(s, b, total - n, total)
        r = s["start"][b]
        s["k_cache"][page, slot] = s["k_new"][r:r + n]
        s["v_cache"][page, slot] = s["v_new"][r:r + n]
    return s["k_cache"], s["v_cache"]


def _plain_attend(s):
    out, lse = [], []
    Hk, D = s["k_cache"].shape[2:]
    for b, (n, total) in enumerate(zip(s["new"], s["total"])):
        page, slot = _slots(s, b, 0, total)
        k = s["k_cache"][page, slot].float().permute(1, 2, 0)[:, None]
        v = s["v_cache"][page, slot].float().transpose(0, 1)[:, None]
        r = s["start"][b]
        q = s["q"][r:r + n].float().view(n, Hk, -1, D).permute(1, 2, 0, 3)
        z = (q @ k) * (1.0 / math.sqrt(D))
        if s["causal"]:
            at = torch.arange(total, device=DEV)[None, :]
            mine = torch.arange(total - n, total, device=DEV)[:, None]
            hidden = at > mine
            if s["window"] > 0:
                hidden |= at <= mine - s["window"]
            z = z.masked_fill_(hidden, -math.inf)
        m = z.amax(-1, keepdim=True)
        z = z.sub_(m).exp_()
        total_mass = z.sum(-1, keepdim=True)
        out.append(((z @ v) / total_mass).permute(2, 0, 1, 3).reshape(n, -1, D))
        lse.append((m + torch.log(total_mass))[..., 0].permute(2, 0, 1).reshape(n, -1))
    return torch.cat(out).to(s["q"].dtype), torch.cat(lse)


def run(state):
    op = state["op"]
    if not own:
        return {"sample": _plain_sample, "truncate": _plain_truncate, "append": _plain_append,
                "attend": _plain_attend}[op](state)
    if op == "sample":
        return state["sampler"].sample()
    if op == "truncate":
        return state["sampler"].truncate()
    if op == "append":
        return state["cache"].append()
    return state["cache"].attend()


def _seen(case):
    """Per request: entries that some new token sees, and pairs of a new token and an entry."""
    seen = []
    for n, total in zip(*_sizes(case)):
        if not case["causal"]:
            seen.append((total, n * total))
            continue
        w = case["window"] or total
        first = max(0, total - n + 1 - w)
        # Token t sees min(total - n + t + 1, w) entries.
        full = max(0, min(n, total - w))  # tokens that see a whole window
        rest = n - full
        a = total - n + 1
        seen.append((total - first, full * w + rest * a + rest * (rest - 1) // 2))
    return seen


def work(case):
    op = case["op"]
    if op in ("sample", "truncate"):
        es = 4 if case["dtype"] == "f32" else 2
        rows, V = case["B"] * case["n"], case["V"]
        once = rows * V * es + 16 * case["B"]
        return {"bytes": once + (8 * rows if op == "sample" else rows * V * es),
                "flops": 4 * rows * V}
    new, total = _sizes(case)
    Hk, D = case["kv_heads"], case["width"]
    rows = sum(new)
    index = 4 * sum(-(-t // case["page"]) for t in total) + 8 * case["B"]
    if op == "append":
        return {"bytes": 2 * 2 * rows * Hk * D * 2 + 4 * rows, "flops": rows * Hk * D}
    seen = _seen(case)
    H = case["heads"]
    return {"bytes": sum(e for e, _ in seen) * Hk * D * 4 + rows * H * (4 * D + 4) + index,
            "flops": 4 * sum(p for _, p in seen) * H * D}


def _exact_kept(s, b, i):
    """Kept entries of one row, as a truth value per index, and their masses."""
    z = s["logits"][b, i].double()
    V = z.numel()
    T = float(s["temperature"][b])
    kept = torch.zeros(V, dtype=torch.bool, device=DEV)
    if T == 0.0:
        kept[int(torch.nonzero(z == z.max())[0])] = True
        return kept, kept.double()
    w = torch.exp((z - z.max()) / T)
    ranked = torch.argsort(-z, stable=True)
    k, p, m = int(s["top_k"][b]), float(s["top_p"][b]), float(s["min_p"][b])
    if k > 0:
        ranked = ranked[:k]
    if p < 1.0:
        c = torch.cumsum(w[ranked], 0)
        count = int(torch.searchsorted(c, p * c[-1:])[0]) + 1  # first place that reaches p
        ranked = ranked[:count]
    kept[ranked] = True
    kept &= w >= m
    return kept, torch.where(kept, w, 0.0)


def _exact_logits(case, s):
    B, n = case["B"], case["n"]
    if B * n > 700:  # a row at a time takes about 1 ms
        return None
    if case["op"] == "sample":
        out = torch.zeros((B, n), dtype=torch.int32, device=DEV)
    else:
        out = torch.full(s["logits"].shape, -math.inf, dtype=torch.float64, device=DEV)
    for b in range(B):
        for i in range(n):
            kept, w = _exact_kept(s, b, i)
            if case["op"] == "sample":
                c = torch.cumsum(w, 0)
                out[b, i] = torch.searchsorted(c, float(s["uniforms"][b, i]) * c[-1:],
                                               right=True)[0]
            else:
                out[b, i, kept] = s["logits"][b, i, kept].double()
    return out


def _exact_append(s):
    caches = []
    page = s["k_cache"].shape[1]
    for cache, fresh in ((s["k_cache"], s["k_new"]), (s["v_cache"], s["v_new"])):
        flat = cache.double().flatten(0, 1)
        for b, (n, total) in enumerate(zip(s["new"], s["total"])):
            at = torch.arange(total - n, total, device=DEV)
            row = s["table"][b].long().index_select(0, at // page) * page + at % page
            flat.index_copy_(0, row, fresh[s["start"][b]:s["start"][b + 1]].double())
        caches.append(flat.view(cache.shape))
    return tuple(caches)


def _exact_attend(case, s):
    if work(case)["flops"] > 2e12:  # double precision runs at about 1 TFLOP/s
        return None
    H, D = case["heads"], case["width"]
    G = H // case["kv_heads"]
    rows = s["start"][-1]
    out = torch.zeros((rows, H, D), dtype=torch.float64, device=DEV)
    lse = torch.zeros((rows, H), dtype=torch.float64, device=DEV)
    for b, (n, total) in enumerate(zip(s["new"], s["total"])):
        used = s["table"][b, :-(-total // case["page"])].long()
        k = s["k_cache"][used].flatten(0, 1)[:total].double()
        v = s["v_cache"][used].flatten(0, 1)[:total].double()
        r = s["start"][b]
        for t0 in range(0, n, 256):  # 256 tokens at a time
            t1 = min(n, t0 + 256)
            away = (torch.arange(t0, t1, device=DEV)[:, None] + (total - n)
                    - torch.arange(total, device=DEV)[None, :])
            sees = torch.ones_like(away, dtype=torch.bool)
            if case["causal"]:
                sees = away >= 0
                if case["window"]:
                    sees &= away < case["window"]
            for h in range(H):
                z = s["q"][r + t0:r + t1, h].double() @ k[:, h // G].t() / math.sqrt(D)
                z = torch.where(sees, z, -math.inf)
                lse[r + t0:r + t1, h] = torch.logsumexp(z, 1)
                out[r + t0:r + t1, h] = torch.softmax(z, 1) @ v[:, h // G]
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("sample", "truncate"):
        return _exact_logits(case, s)
    return _exact_append(s) if case["op"] == "append" else _exact_attend(case, s)
