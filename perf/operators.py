"""The paged-cache operators over the range they are used in: appending new keys, attention of new tokens over the
cache, the attention weight each cached key has received, and eviction by it. `run` computes one of them, either in
plain torch operations (fp32) or through the library's entry points."""

import math

import torch

own = False

# Head layouts are this library's workloads': 32 query heads over 8 K/V heads at d = 128 (its grouped-query and decode
# shapes), 12 heads at d = 64 (GPT-2), 16 at d = 64 (BERT-large), 32 over 32.
GQA = {"H": 32, "Hkv": 8, "d": 128}
GPT2 = {"H": 12, "Hkv": 12, "d": 64}


def listed():
    return [
        # One user's next token over a short context: the smallest call, where latency counts.
        {"name": "attend_one", "op": "attend", "B": 1, "Lq": 1, "Lk": 777, "page": 16, "causal": True, "packed": False, **GQA},
        # The decode step of a full server: ragged lengths up to the library's long context.
        {"name": "attend_step", "op": "attend", "B": 32, "Lq": 1, "Lk": 8192, "page": 64, "causal": True, "packed": False, **GQA},
        # The same for small heads without groups.
        {"name": "attend_step_d64", "op": "attend", "B": 48, "Lq": 1, "Lk": 1024, "page": 16, "causal": True, "packed": False, **GPT2},
        # A few drafted tokens per sequence checked at once.
        {"name": "attend_draft", "op": "attend", "B": 16, "Lq": 5, "Lk": 4099, "page": 32, "causal": True, "packed": False, **GQA},
        # Prompt chunks of some sequences beside single tokens of others, in one packed batch.
        {"name": "attend_mixed", "op": "attend", "B": 6, "Lq": 509, "Lk": 6001, "page": 128, "causal": True, "packed": True, **GQA},
        # A long prompt's last chunk: bound by the tensor cores.
        {"name": "attend_chunk", "op": "attend", "B": 1, "Lq": 2048, "Lk": 16384, "page": 64, "causal": True, "packed": False, **GQA},
        # One token of each of 64 sequences into the cache; and a packed batch of prompts.
        {"name": "append_step", "op": "append", "B": 64, "Lq": 1, "Lk": 2000, "page": 16, "causal": True, "packed": False, **GQA},
        {"name": "append_prompts", "op": "append", "B": 7, "Lq": 4096, "Lk": 4096, "page": 64, "causal": True, "packed": True, **GQA},
        # The weights' update after a decode step, and after a prompt chunk.
        {"name": "weights_step", "op": "weights", "B": 16, "Lq": 1, "Lk": 8192, "page": 64, "causal": True, "packed": False, **GQA},
        {"name": "weights_chunk", "op": "weights", "B": 2, "Lq": 700, "Lk": 8192, "page": 128, "causal": True, "packed": True, **GQA},
        # One short sequence cut down; and a batch that reaches its budget.
        {"name": "evict_one", "op": "evict", "B": 1, "Lq": 1, "Lk": 1030, "page": 16, "causal": True, "packed": False, "keep": 512, "recent": 64, **GQA},
        {"name": "evict_batch", "op": "evict", "B": 12, "Lq": 1, "Lk": 8192, "page": 64, "causal": True, "packed": False, "keep": 2050, "recent": 256, **GQA},
    ]


def draw(rng):
    def logs(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["attend", "attend", "attend", "append", "weights", "weights", "evict"])
    heads = rng.choice([GQA, GPT2, {"H": 16, "Hkv": 16, "d": 64}, {"H": 32, "Hkv": 32, "d": 128}, {"H": 28, "Hkv": 4, "d": 128},
                        {"H": 24, "Hkv": 8, "d": 64}, {"H": 8, "Hkv": 1, "d": 128}])
    Lk = logs(64, 16384)
    Lq = 1 if op == "evict" else rng.choice([1, 1, rng.randint(2, 9), logs(10, 2048)])
    Lq = min(Lq, Lk)
    # At most the largest listed case's cache (32 x 8192 keys of 8 heads, d = 128) and products (2048 x 16384, 32 heads).
    most = min(32 * 8192 * 1024 / (Lk * heads["Hkv"] * heads["d"]), 2048 * 16384 * 4096 / (Lq * Lk * heads["H"] * heads["d"]))
    B = logs(1, max(1, min(48, int(most))))
    case = {"op": op, "B": B, "Lq": Lq, "Lk": Lk, "page": rng.choice([16, 32, 64, 128, 256]), "causal": rng.random() < 0.8,
            "packed": Lq > 1 and rng.random() < 0.5, **heads}
    if op == "evict":
        case["keep"] = logs(16, max(16, Lk - 1))
        case["recent"] = rng.randint(0, case["keep"])
    return case


def lengths(c):
    """Query and key lengths of the sequences: ragged, the first the longest; in a packed batch every third sequence has one token."""
    lk = [max(1, c["Lk"] - (b * 7919) % max(1, c["Lk"] // 2)) for b in range(c["B"])]
    lq = [c["Lq"]] * c["B"]
    if c["packed"]:
        lq = [(c["Lq"], 1, c["Lq"] // 2 + 1)[b % 3] for b in range(c["B"])]
    return lq, [max(n, m) for n, m in zip(lk, lq)]


class State:
    pass


def prepare(case, seed):
    c, s = case, State()
    g = torch.Generator("cuda").manual_seed(seed)
    lq, lk = lengths(c)
    B, P = c["B"], c["page"]
    used = [-(-n // P) for n in lk]
    width = max(used) + 1
    total = sum(used) + 3  # some pages of the pool belong to nobody
    s.c, s.lq, s.lk, s.max_q, s.max_k = c, lq, lk, max(lq), max(lk)
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32).cpu()
    table = torch.zeros(B, width, dtype=torch.int32)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    s.table = table.cuda()
    s.seqlens_k = torch.tensor(lk, dtype=torch.int32, device="cuda")
    rows = sum(lq)
    cu = [0]
    for n in lq:
        cu.append(cu[-1] + n)
    s.cu = torch.tensor(cu, dtype=torch.int32, device="cuda") if c["packed"] else None
    lead = (rows,) if c["packed"] else (B, c["Lq"])

    def bf16(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)

    s.k_cache = bf16(total, P, c["Hkv"], c["d"], std=1.5)
    s.v_cache = bf16(total, P, c["Hkv"], c["d"])
    s.scale = 1.0 / math.sqrt(c["d"])
    if c["op"] in ("attend", "weights"):
        s.q = bf16(*lead, c["H"], c["d"], std=1.5)
    if c["op"] == "append":
        s.k, s.v = bf16(*lead, c["Hkv"], c["d"], std=1.5), bf16(*lead, c["Hkv"], c["d"])
    if c["op"] != "attend":
        # Attention weight is heavy-tailed, and keys that nothing has looked at yet have none.
        w = torch.randn(total, c["Hkv"], P, generator=g, device="cuda")
        s.weights0 = torch.where(w > -1.5, torch.exp(2.0 * w), 0.0)
        s.weights = s.weights0.clone()
    if c["op"] == "weights":
        s.lse = _attend(s, values=False)[1]
    return s


# ---------------------------------------------------------------------------------------------- plain forms


def _padded(s, x):
    """[B, max_q, heads, d] of the new tokens (a packed batch padded), and which of its rows exist."""
    n = torch.tensor(s.lq, device="cuda")
    i = torch.arange(s.max_q, device="cuda")
    live = i[None] < n[:, None]
    if not s.c["packed"]:
        return x, live
    row = (s.cu[:-1, None] + i[None]).clamp(max=x.shape[0] - 1).long()
    return x[row], live


def _unpadded(s, x, live):
    return x[live] if s.c["packed"] else x


def _gathered(s, cache):
    """[B, keys, Hkv, d] fp32 of a cache's keys, zero past each sequence's length."""
    P = s.c["page"]
    n = -(-s.max_k // P)
    x = cache[s.table[:, :n].long()].reshape(s.c["B"], n * P, s.c["Hkv"], s.c["d"])[:, :s.max_k].float()
    dead = torch.arange(s.max_k, device="cuda")[None] >= s.seqlens_k[:, None]
    return x.masked_fill(dead[:, :, None, None], 0.0)


def _scores(s):
    """Masked scaled scores [B, Hkv, G, max_q, keys] and the rows that exist."""
    c = s.c
    q, live = _padded(s, s.q)
    q = q.float().reshape(c["B"], s.max_q, c["Hkv"], c["H"] // c["Hkv"], c["d"])
    x = torch.einsum("bqhgd,bkhd->bhgqk", q, _gathered(s, s.k_cache)) * s.scale
    j = torch.arange(s.max_k, device="cuda")
    last = s.seqlens_k.long()[:, None].expand(-1, s.max_q)
    if c["causal"]:
        n = torch.tensor(s.lq, device="cuda")
        last = torch.arange(s.max_q, device="cuda")[None] + 1 + (s.seqlens_k.long() - n)[:, None]
        last = torch.minimum(last, s.seqlens_k.long()[:, None])
    hidden = j[None, None] >= last[:, :, None]
    return x.masked_fill_(hidden[:, None, None], -math.inf), live


def _attend(s, values=True):
    c = s.c
    x, live = _scores(s)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x.sub_(torch.where(m == -math.inf, 0.0, m)))
    total = p.sum(-1, keepdim=True)
    lse = (m + torch.log(total)).squeeze(-1).reshape(c["B"], c["H"], s.max_q)
    lse = lse.transpose(0, 1)[:, live].contiguous() if c["packed"] else lse
    if not values:
        return None, lse
    o = torch.einsum("bhgqk,bkhd->bqhgd", p, _gathered(s, s.v_cache))
    o = o / torch.where(total == 0, 1.0, total).squeeze(-1).permute(0, 3, 1, 2)[..., None]
    return _unpadded(s, o.reshape(c["B"], s.max_q, c["H"], c["d"]).to(torch.bfloat16), live), lse


def _slots(s, j):
    """Page and slot of the keys j [B, n]."""
    P = s.c["page"]
    return s.table.gather(1, (j // P).long()).long(), (j % P).long()


def _append(s):
    n = torch.tensor(s.lq, device="cuda")
    i = torch.arange(s.max_q, device="cuda")
    (k, live), (v, _) = _padded(s, s.k), _padded(s, s.v)
    j = (s.seqlens_k - n)[:, None] + i[None]
    page, slot = _slots(s, torch.where(live, j, 0))  # a packed batch's padding has no place of its own
    page, slot = page[live], slot[live]
    s.k_cache[page, slot] = k[live]
    s.v_cache[page, slot] = v[live]
    s.weights[page, :, slot] = 0.0
    return s.k_cache, s.v_cache, s.weights


def _weights(s):
    c = s.c
    x, live = _scores(s)
    if c["packed"]:
        lse = torch.full((c["B"], s.max_q, c["H"]), math.inf, device="cuda")
        lse[live] = s.lse.t()
        lse = lse.transpose(1, 2)
    else:
        lse = s.lse
    lse = torch.where(lse == -math.inf, math.inf, lse).reshape(c["B"], c["Hkv"], c["H"] // c["Hkv"], s.max_q, 1)
    add = torch.exp(x.sub_(lse)).sum((2, 3))  # [B, Hkv, keys]
    j = torch.arange(s.max_k, device="cuda")[None].expand(c["B"], -1)
    there = j < s.seqlens_k[:, None]
    page, slot = _slots(s, j)
    s.weights[page[there], :, slot[there]] += add.transpose(1, 2)[there]
    return s.weights


def _evict(s):
    c = s.c
    keep, B, Hkv = c["keep"], c["B"], c["Hkv"]
    L = s.seqlens_k.long()
    j = torch.arange(s.max_k, device="cuda")[None].expand(B, -1)
    page, slot = _slots(s, j)
    w = s.weights[page, :, slot].transpose(1, 2)  # [B, Hkv, keys]
    rank = w.masked_fill((j >= (L - c["recent"])[:, None])[:, None], math.inf).masked_fill((j >= L[:, None])[:, None], -math.inf)
    first = torch.sort(rank, dim=-1, descending=True, stable=True).indices
    n = min(keep, s.max_k)
    kept = torch.sort(first[:, :, :n].masked_fill(torch.arange(n, device="cuda") >= L[:, None, None], s.max_k), dim=-1).values
    gone = kept == s.max_k
    cut = L > keep
    full = torch.full((B, Hkv, keep), -1, dtype=torch.int32, device="cuda")
    full[:, :, :n] = kept.masked_fill(gone, -1).to(torch.int32)
    b, h, t = torch.where((~gone) & cut[:, None, None])
    old = kept[b, h, t]
    to, at, src, off = page[b, t], slot[b, t], page[b, old], slot[b, old]
    s.k_cache[to, at, h] = s.k_cache[src, off, h]
    s.v_cache[to, at, h] = s.v_cache[src, off, h]
    s.weights[to, h, at] = s.weights[src, h, off]
    return full, torch.minimum(L, torch.tensor(keep, device="cuda")).to(torch.int32)


def run(s):
    c = s.c
    op = c["op"]
    if op == "evict":
        s.weights.copy_(s.weights0)  # what the steps before would have left; eviction itself moves them
    if own:
        import exact_io_aware_38_gb300 as fa
        tokens = dict(cu_seqlens_q=s.cu, max_seqlen_q=s.max_q) if c["packed"] else {}
        if op == "attend":
            o, lse = fa.fwd_paged(s.q, s.k_cache, s.v_cache, s.table, s.seqlens_k, max_seqlen_k=s.max_k, causal=c["causal"],
                                  scale=s.scale, **tokens)
            return {"o": o, "lse": lse}
        if op == "append":
            fa.paged_append(s.k, s.v, s.k_cache, s.v_cache, s.table, s.seqlens_k, key_weights=s.weights, **tokens)
            return {"k": s.k_cache, "v": s.v_cache, "weights": s.weights}
        if op == "weights":
            fa.paged_key_weights(s.q, s.k_cache, s.table, s.seqlens_k, s.lse, s.weights, max_seqlen_k=s.max_k,
                                 causal=c["causal"], scale=s.scale, **tokens)
            return {"weights": s.weights}
        kept, n = fa.paged_evict(s.k_cache, s.v_cache, s.weights, s.table, s.seqlens_k, c["keep"], recent=c["recent"],
                                 max_seqlen_k=s.max_k)
    elif op == "attend":
        o, lse = _attend(s)
        return {"o": o, "lse": lse}
    elif op == "append":
        k, v, w = _append(s)
        return {"k": k, "v": v, "weights": w}
    elif op == "weights":
        return {"weights": _weights(s)}
    else:
        kept, n = _evict(s)
    return {"kept": kept, "seqlens": n, "k": s.k_cache, "v": s.v_cache, "weights": s.weights}


def work(case):
    c = case
    lq, lk = lengths(c)
    H, Hkv, d = c["H"], c["Hkv"], c["d"]
    tokens, keys = sum(lq), sum(lk)
    pairs = sum(n * m - (n * (n - 1) // 2 if c["causal"] else 0) for n, m in zip(lq, lk))
    if c["op"] == "attend":
        return {"bytes": 4 * keys * Hkv * d + 4 * tokens * H * d + 4 * tokens * H, "flops": 4 * pairs * H * d}
    if c["op"] == "append":
        return {"bytes": 8 * tokens * Hkv * d + 4 * tokens * Hkv, "flops": 0}
    if c["op"] == "weights":
        return {"bytes": 2 * keys * Hkv * d + 2 * tokens * H * d + 4 * tokens * H + 8 * keys * Hkv, "flops": 2 * pairs * H * d}
    # The step's weights are put in place (read and written), then read once; kept rows move but for those already at their place.
    pool = (sum(-(-n // c["page"]) for n in lk) + 3) * c["page"] * Hkv
    moved = sum(c["keep"] for n in lk if n > c["keep"]) * Hkv
    return {"bytes": 8 * pool + 4 * keys * Hkv + moved * (8 * d + 8) + 4 * c["B"] * Hkv * c["keep"], "flops": 0}


# ---------------------------------------------------------------------------------------------- from the definitions


def exact(case, seed):
    """One sequence and K/V head at a time, in fp64; data movement by plain index lists."""
    s = prepare(case, seed)
    c = case
    P, G, Hkv = c["page"], c["H"] // c["Hkv"], c["Hkv"]
    first = [0]
    for n in s.lq:
        first.append(first[-1] + n)

    def place(b, j):
        return s.table[b, j // P].long(), j % P

    def new(x, b):
        return x[first[b]:first[b + 1]] if c["packed"] else x[b]

    def probabilities(b, h, lse=None):
        n, L = s.lq[b], s.lk[b]
        j = torch.arange(L, device="cuda")
        page, slot = place(b, j)
        q = new(s.q, b)[:, h * G:(h + 1) * G].double().transpose(0, 1)  # [G, n, d]
        x = (q @ s.k_cache[page, slot, h].double().t()) * s.scale
        if c["causal"]:
            i = torch.arange(n, device="cuda")
            x[:, j[None] > (i + L - n)[:, None]] = -math.inf
        if lse is not None:
            return torch.exp(x - lse[..., None]), None
        lse = torch.logsumexp(x, -1)
        return torch.exp(x - lse[..., None]), lse

    if c["op"] == "attend":
        o = torch.zeros(s.q.shape, dtype=torch.float64, device="cuda")
        lse = torch.zeros((c["H"], s.q.shape[0]) if c["packed"] else (c["B"], c["H"], c["Lq"]), dtype=torch.float64, device="cuda")
        for b in range(c["B"]):
            page, slot = place(b, torch.arange(s.lk[b], device="cuda"))
            for h in range(Hkv):
                p, l = probabilities(b, h)
                new(o, b)[:, h * G:(h + 1) * G] = (p @ s.v_cache[page, slot, h].double()).transpose(0, 1)
                if c["packed"]:
                    lse[h * G:(h + 1) * G, first[b]:first[b + 1]] = l
                else:
                    lse[b, h * G:(h + 1) * G] = l
        return {"o": o, "lse": lse}
    w = s.weights0.double()
    if c["op"] == "weights":
        for b in range(c["B"]):
            page, slot = place(b, torch.arange(s.lk[b], device="cuda"))
            for h in range(Hkv):
                l = s.lse[h * G:(h + 1) * G, first[b]:first[b + 1]] if c["packed"] else s.lse[b, h * G:(h + 1) * G]
                w[page, h, slot] += probabilities(b, h, l.double())[0].sum((0, 1))
        return {"weights": w}
    k, v = s.k_cache.double(), s.v_cache.double()
    if c["op"] == "append":
        for b in range(c["B"]):
            page, slot = place(b, torch.arange(s.lk[b] - s.lq[b], s.lk[b], device="cuda"))
            k[page, slot], v[page, slot], w[page, :, slot] = new(s.k, b).double(), new(s.v, b).double(), 0.0
        return {"k": k, "v": v, "weights": w}
    k0, v0, w0 = k.clone(), v.clone(), w.clone()
    for b in range(c["B"]):
        L = s.lk[b]
        if L <= c["keep"]:
            continue
        old = L - c["recent"]
        for h in range(Hkv):
            page, slot = place(b, torch.arange(old, device="cuda"))
            seen = w0[page, h, slot].tolist()
            chosen = sorted(sorted(range(old), key=lambda j: (-seen[j], j))[:c["keep"] - c["recent"]]) + list(range(old, L))
            src, off = place(b, torch.tensor(chosen, device="cuda"))
            to, at = place(b, torch.arange(c["keep"], device="cuda"))
            k[to, at, h], v[to, at, h], w[to, h, at] = k0[src, off, h], v0[src, off, h], w0[src, h, off]
    return {"kept": None, "seqlens": None, "k": k, "v": v, "weights": w}
