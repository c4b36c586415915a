"""The operators of a paged K/V cache held in 8 bits, over the range they are used in: writing new keys and values as
e4m3 rows with an exponent each, attention of new tokens over such a cache, and reading rows back in bf16. `run` computes
one of them, either in plain torch operations (fp32) or through the library's entry points.

A row of d values (a token's, of one K/V head) is y 2^(code - 127) with e4m3 numbers y: code = floor(log2 max|x|) + 120, at
least 47; 0 for a row of zeros; 255 for one with NaN or an infinity. Codes lie as uint8 [page][head][slot][K, V]."""

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
        {"name": "attend_step", "op": "attend", "B": 64, "Lq": 1, "Lk": 8192, "page": 64, "causal": True, "packed": False, **GQA},
        # The same for small heads without groups.
        {"name": "attend_step_d64", "op": "attend", "B": 48, "Lq": 1, "Lk": 1024, "page": 16, "causal": True, "packed": False, **GPT2},
        # Two very long documents: few sequences, whose keys have to be divided.
        {"name": "attend_long", "op": "attend", "B": 2, "Lq": 1, "Lk": 131071, "page": 128, "causal": True, "packed": False, **GQA},
        # A few drafted tokens per sequence checked at once.
        {"name": "attend_draft", "op": "attend", "B": 16, "Lq": 5, "Lk": 4099, "page": 32, "causal": True, "packed": False, **GQA},
        # Prompt chunks of some sequences beside single tokens of others, in one packed batch.
        {"name": "attend_mixed", "op": "attend", "B": 6, "Lq": 509, "Lk": 6001, "page": 128, "causal": True, "packed": True, **GQA},
        # A long prompt's last chunk: bound by the tensor cores.
        {"name": "attend_chunk", "op": "attend", "B": 1, "Lq": 2048, "Lk": 16384, "page": 64, "causal": True, "packed": False, **GQA},
        # One token of each of 64 sequences into the cache; and a packed batch of prompts.
        {"name": "append_step", "op": "append", "B": 64, "Lq": 1, "Lk": 2000, "page": 16, "causal": True, "packed": False, **GQA},
        {"name": "append_prompts", "op": "append", "B": 7, "Lq": 4096, "Lk": 4096, "page": 64, "causal": True, "packed": True, **GQA},
        # A short cached prefix taken out of the cache; and a packed batch of long ones.
        {"name": "read_one", "op": "read", "B": 1, "Lq": 300, "Lk": 301, "page": 16, "causal": True, "packed": False, **GPT2},
        {"name": "read_prompts", "op": "read", "B": 9, "Lq": 8191, "Lk": 8191, "page": 64, "causal": True, "packed": True, **GQA},
    ]


def draw(rng):
    def logs(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["attend", "attend", "attend", "attend", "append", "read"])
    heads = rng.choice([GQA, GPT2, {"H": 16, "Hkv": 16, "d": 64}, {"H": 32, "Hkv": 32, "d": 128}, {"H": 28, "Hkv": 4, "d": 128},
                        {"H": 24, "Hkv": 8, "d": 64}, {"H": 8, "Hkv": 1, "d": 128}])
    Lk = logs(64, 16384)
    Lq = logs(1, Lk) if op == "read" else rng.choice([1, 1, rng.randint(2, 9), rng.randint(10, 80), logs(10, 2048)])
    Lq = min(Lq, Lk)
    # At most the largest listed case's cache (64 x 8192 keys of 8 heads, d = 128) and products (2048 x 16384, 32 heads).
    most = min(64 * 8192 * 1024 / (Lk * heads["Hkv"] * heads["d"]), 2048 * 16384 * 4096 / (Lq * Lk * heads["H"] * heads["d"]))
    B = logs(1, max(1, min(64, int(most))))
    return {"op": op, "B": B, "Lq": Lq, "Lk": Lk, "page": rng.choice([8, 16, 32, 64, 128, 256]), "causal": rng.random() < 0.8,
            "packed": Lq > 1 and rng.random() < 0.5, **heads}


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
    B, P, Hkv, d = c["B"], c["page"], c["Hkv"], c["d"]
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
    s.live = torch.arange(s.max_q, device="cuda")[None] < torch.tensor(lq, device="cuda")[:, None]
    lead = (rows,) if c["packed"] else (B, c["Lq"])

    def rand(*shape, std=1.0, spread=0.0):
        # Some tokens' rows are larger than others', by a factor each: exponents differ from row to row.
        x = torch.randn(*shape, generator=g, device="cuda")
        size = torch.randn(*shape[:-1], 1, generator=g, device="cuda") * spread if spread else None
        return x * std if size is None else x * (torch.exp(size) * std)

    codes = []
    for name, std, spread in (("k_cache", 1.5, 0.2), ("v_cache", 1.0, 0.7)):
        y, code = quantised(rand(total, P, Hkv, d, std=std, spread=spread))
        setattr(s, name, y)
        codes.append(code)
    s.scales = torch.stack(codes, -1).transpose(1, 2).contiguous()
    s.scale = 1.0 / math.sqrt(d)
    if c["op"] == "attend":
        s.q = rand(*lead, c["H"], d, std=1.5).to(torch.bfloat16)
    if c["op"] == "append":
        s.k = rand(*lead, Hkv, d, std=1.5, spread=0.2).to(torch.bfloat16)
        s.v = rand(*lead, Hkv, d, spread=0.7).to(torch.bfloat16)
    if c["op"] == "read":
        s.k, s.v = (torch.zeros(*lead, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    return s


# ---------------------------------------------------------------------------------------------- plain forms


def power(n):
    """2^n in fp32, of whole numbers from -126 to 127 (a pow need not be exact)."""
    return ((n.int() + 127) << 23).view(torch.float32)


def quantised(x):
    """e4m3 values and codes of finite rows x [..., d] (fp32 or bf16)."""
    x = x.float()
    top = x.abs().amax(-1)
    code = torch.where(top == 0, 0, (torch.frexp(top).exponent - 1 + 120).clamp(min=47))
    return (x * power(127 - code)[..., None]).to(torch.float8_e4m3fn), code.to(torch.uint8)


def _places(s, j):
    """Page and slot of the keys j [B, n]."""
    P = s.c["page"]
    return s.table.gather(1, (j // P).long()).long(), (j % P).long()


def _new_places(s):
    """Page and slot of the rows that exist, in their order."""
    n = torch.tensor(s.lq, device="cuda")
    j = (s.seqlens_k - n)[:, None] + torch.arange(s.max_q, device="cuda")[None]
    page, slot = _places(s, torch.where(s.live, j, 0))
    return page[s.live], slot[s.live]


def _rows(s, which, page, slot):
    """fp32 rows [..., Hkv, d] of the keys (0) or values (1) at these places."""
    y = (s.k_cache, s.v_cache)[which].view(torch.uint8)[page, slot].view(torch.float8_e4m3fn).float()
    code = s.scales[page, :, slot, which].int()
    return y * torch.where(code == 0, 0.0, power(code.clamp(min=1) - 127))[..., None]


def _gathered(s, which):
    """[B, keys, Hkv, d] fp32, zero past each sequence's length."""
    j = torch.arange(s.max_k, device="cuda")[None].expand(s.c["B"], -1)
    dead = j >= s.seqlens_k[:, None]
    return _rows(s, which, *_places(s, j)).masked_fill(dead[:, :, None, None], 0.0)


def _attend(s):
    c = s.c
    B, H, Hkv, d = c["B"], c["H"], c["Hkv"], c["d"]
    q = s.q
    if c["packed"]:
        i = torch.arange(s.max_q, device="cuda")
        q = q[(s.cu[:-1, None] + i[None]).clamp(max=q.shape[0] - 1).long()]
    q = q.float().reshape(B, s.max_q, Hkv, H // Hkv, d)
    x = torch.einsum("bqhgd,bkhd->bhgqk", q, _gathered(s, 0)) * s.scale
    j = torch.arange(s.max_k, device="cuda")
    last = s.seqlens_k.long()[:, None].expand(-1, s.max_q)
    if c["causal"]:
        n = torch.tensor(s.lq, device="cuda")
        last = torch.minimum(torch.arange(s.max_q, device="cuda")[None] + 1 + (s.seqlens_k.long() - n)[:, None], last)
    x.masked_fill_((j[None, None] >= last[:, :, None])[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x.sub_(torch.where(m == -math.inf, 0.0, m)))
    total = p.sum(-1, keepdim=True)
    lse = (m + torch.log(total)).squeeze(-1).reshape(B, H, s.max_q)
    o = torch.einsum("bhgqk,bkhd->bqhgd", p, _gathered(s, 1))
    o = o / torch.where(total == 0, 1.0, total).squeeze(-1).permute(0, 3, 1, 2)[..., None]
    o = o.reshape(B, s.max_q, H, d).to(torch.bfloat16)
    if c["packed"]:
        return o[s.live], lse.transpose(0, 1)[:, s.live].contiguous()
    return o, lse


def _append(s):
    page, slot = _new_places(s)
    for which, (x, cache) in enumerate(((s.k, s.k_cache), (s.v, s.v_cache))):
        y, code = quantised(x.reshape(-1, *x.shape[-2:]))
        cache.view(torch.uint8)[page, slot] = y.view(torch.uint8)
        s.scales[page, :, slot, which] = code


def _read(s):
    page, slot = _new_places(s)
    for which, out in enumerate((s.k, s.v)):
        out.copy_(_rows(s, which, page, slot).to(torch.bfloat16).reshape(out.shape))


def run(s):
    c = s.c
    op = c["op"]
    if own:
        import exact_io_aware_38_gb300 as fa
        tokens = dict(cu_seqlens_q=s.cu, max_seqlen_q=s.max_q) if c["packed"] else {}
        if op == "attend":
            o, lse = fa.fwd_paged_fp8(s.q, s.k_cache, s.v_cache, s.scales, s.table, s.seqlens_k, max_seqlen_k=s.max_k,
                                      causal=c["causal"], scale=s.scale, **tokens)
        elif op == "append":
            fa.paged_append_fp8(s.k, s.v, s.k_cache, s.v_cache, s.scales, s.table, s.seqlens_k, **tokens)
        else:
            fa.paged_read_fp8(s.k, s.v, s.k_cache, s.v_cache, s.scales, s.table, s.seqlens_k, **tokens)
    elif op == "attend":
        o, lse = _attend(s)
    elif op == "append":
        _append(s)
    else:
        _read(s)
    if op == "attend":
        return {"o": o, "lse": lse}
    if op == "append":
        return {"k": s.k_cache, "v": s.v_cache, "scales": s.scales}
    return {"k": s.k, "v": s.v}


def work(case):
    c = case
    lq, lk = lengths(c)
    H, Hkv, d = c["H"], c["Hkv"], c["d"]
    tokens, keys = sum(lq), sum(lk)
    if c["op"] != "attend":  # a row in bf16 on one side, in bytes and an exponent on the other
        return {"bytes": tokens * Hkv * (6 * d + 2), "flops": 0}
    pairs = sum(n * m - (n * (n - 1) // 2 if c["causal"] else 0) for n, m in zip(lq, lk))
    return {"bytes": keys * Hkv * (2 * d + 2) + 4 * tokens * H * d + 4 * tokens * H, "flops": 4 * pairs * H * d}


# ---------------------------------------------------------------------------------------------- from the definitions


def _e4m3():
    """The numbers of the 256 bytes: sign, 4 exponent bits biased by 7, 3 bits of fraction; all ones is NaN."""
    out = []
    for n in range(256):
        e, f = n >> 3 & 15, n & 7
        x = math.nan if n & 127 == 127 else f * 2.0**-9 if e == 0 else (8 + f) * 2.0**(e - 10)
        out.append(-x if n & 128 else x)
    return torch.tensor(out, dtype=torch.float64, device="cuda")


def exact(case, seed):
    """One sequence (and K/V head) at a time, in fp64; data movement by plain index lists."""
    s = prepare(case, seed)
    c = case
    P, G, Hkv = c["page"], c["H"] // c["Hkv"], c["Hkv"]
    number = _e4m3()
    first = [0]
    for n in s.lq:
        first.append(first[-1] + n)

    def place(b, j):
        return s.table[b, j // P].long(), j % P

    def new(x, b):
        return x[first[b]:first[b + 1]] if c["packed"] else x[b]

    def row(which, page, slot, h):
        y = number[(s.k_cache, s.v_cache)[which].view(torch.uint8)[page, slot, h].long()]
        return y * (s.scales[page, h, slot, which].long() - 127 + 1023 << 52).view(torch.float64)[:, None]

    if c["op"] == "attend":
        o = torch.zeros(s.q.shape, dtype=torch.float64, device="cuda")
        lse = torch.zeros((c["H"], s.q.shape[0]) if c["packed"] else (c["B"], c["H"], c["Lq"]), dtype=torch.float64, device="cuda")
        for b in range(c["B"]):
            n, L = s.lq[b], s.lk[b]
            j = torch.arange(L, device="cuda")
            page, slot = place(b, j)
            for h in range(Hkv):
                q = new(s.q, b)[:, h * G:(h + 1) * G].double().transpose(0, 1)  # [G, n, d]
                x = (q @ row(0, page, slot, h).t()) * s.scale
                if c["causal"]:
                    i = torch.arange(n, device="cuda")
                    x[:, j[None] > (i + L - n)[:, None]] = -math.inf
                l = torch.logsumexp(x, -1)
                new(o, b)[:, h * G:(h + 1) * G] = (torch.exp(x - l[..., None]) @ row(1, page, slot, h)).transpose(0, 1)
                if c["packed"]:
                    lse[h * G:(h + 1) * G, first[b]:first[b + 1]] = l
                else:
                    lse[b, h * G:(h + 1) * G] = l
        return {"o": o, "lse": lse}
    if c["op"] == "read":
        k, v = (torch.zeros(x.shape, dtype=torch.float64, device="cuda") for x in (s.k, s.v))
        for b in range(c["B"]):
            page, slot = place(b, torch.arange(s.lk[b] - s.lq[b], s.lk[b], device="cuda"))
            for h in range(Hkv):
                new(k, b)[:, h], new(v, b)[:, h] = row(0, page, slot, h), row(1, page, slot, h)
        return {"k": k, "v": v}
    out = []
    for x, cache in ((s.k, s.k_cache), (s.v, s.v_cache)):
        y = number[cache.view(torch.uint8).long()]
        for b in range(c["B"]):
            page, slot = place(b, torch.arange(s.lk[b] - s.lq[b], s.lk[b], device="cuda"))
            r = new(x, b).double()
            below = torch.frexp(r.abs().amax(-1, keepdim=True).clamp(min=2.0**-73)).exponent  # max|r| is in [2^(below - 1), 2^below)
            r = r * (8 - below.long() + 1023 << 52).view(torch.float64)
            step = (torch.frexp(r.abs().clamp(min=2.0**-6)).exponent.long() - 4 + 1023 << 52).view(torch.float64)
            y[page, slot] = torch.round(r / step) * step  # (to even)
        out.append(y)
    return {"k": out[0], "v": out[1], "scales": None}
