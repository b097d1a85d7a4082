"""Cases of the paged-cache operators: tables, 8-bit store, decode attention, prompt attention.

The four operators serve a model whose KV cache lives in pages of 16 tokens, in
8 bits (e4m3) with one power-of-two scale for each page, KV head and K or V:

  tables   pages for the new tokens of every request and each token's slot
  store    new K/V rows quantised into their pages
  decode   one query token per request over its pages (all, or a selection)
  prompt   causal attention over packed prompts, before their K/V is stored

`run` computes them with elementary torch operations, or, where `own` is true,
through this package's calls.  Head dimension 128 and 16 tokens per page
throughout; head counts as in the repository's workloads (32/8, 64/8) and odd ones.
"""
import math
import random

import torch

own = False

D = 128       # head dimension
BS = 16       # tokens per page
E_LOW, E_HIGH = -60, 119  # range of a page's scale exponent


# ------------------------------------------------------------------ the cases
def _text(values):
    return ",".join(str(v) for v in values)


def _lens(text):
    return [int(v) for v in text.split(",")]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def listed():
    r = random.Random(16)
    return [
        # one short chat turn: latency
        {"name": "prompt_short", "op": "prompt", "hq": 32, "hkv": 8, "lens": "17", "pad": 0},
        # a serving batch of prompts, packed, behind it the padding of a fixed-size buffer
        {"name": "prompt_packed", "op": "prompt", "hq": 32, "hkv": 8, "lens": "1,517,2048,3,96,4001,129,1280,760,2500,64,31",
         "pad": 30},
        # wide groups (8 query heads per KV head), a few middle-sized documents
        {"name": "prompt_wide_group", "op": "prompt", "hq": 64, "hkv": 8, "lens": "2100,1023,3333", "pad": 0},
        # one long document: compute
        {"name": "prompt_long", "op": "prompt", "hq": 32, "hkv": 8, "lens": "16384", "pad": 0},
        # a single user early in a conversation: latency
        {"name": "decode_single", "op": "decode", "hq": 32, "hkv": 8, "lens": "700", "kb": 0},
        # a serving batch of very different contexts, one slot empty: bandwidth
        {"name": "decode_batch", "op": "decode", "hq": 32, "hkv": 8,
         "lens": _text([0, 1, 32768, 16] + [_log_int(r, 64, 32768) for _ in range(12)] + [r.randint(1, 32768) for _ in range(16)]),
         "kb": 0},
        # one user at 128K tokens: the work of one request split over the whole GPU
        {"name": "decode_long", "op": "decode", "hq": 64, "hkv": 8, "lens": "131072", "kb": 0},
        # the sparse path: a 2,048-token budget of blocks per KV head at 32K tokens
        {"name": "decode_selected", "op": "decode", "hq": 32, "hkv": 8, "lens": _text([32768] * 32), "kb": 128},
        # one decode step's new tokens, most of them inside a page that already holds some
        {"name": "store_step", "op": "store", "hkv": 8, "old": _text([r.randint(0, 4000) for _ in range(32)]),
         "new": _text([1] * 32), "pad": 0},
        # packed prompts written after their attention, some continuing a page
        {"name": "store_prompts", "op": "store", "hkv": 8, "old": "0,0,37,0,160,0,9,0", "new": "4096,511,2000,1,333,6000,7,2222",
         "pad": 14},
        # the tables of one decode step of a large batch
        {"name": "tables_step", "op": "tables", "old": _text([r.randint(1, 4000) for _ in range(256)]), "new": _text([1] * 256),
         "pad": 0},
        # the tables of a wave of long prompts
        {"name": "tables_prompts", "op": "tables", "old": _text([r.choice((0, 0, 5, 1000)) for _ in range(64)]),
         "new": _text([_log_int(r, 1000, 131072) for _ in range(64)]), "pad": 1000},
    ]


def draw(rng):
    op = rng.choice(("prompt", "prompt", "decode", "decode", "decode", "store", "tables"))
    hkv = rng.choice((1, 2, 4, 5, 8))
    hq = hkv * rng.choice((1, 2, 3, 4, 6, 7, 8))
    if op == "prompt":
        room = 16384 ** 2 * 32 // hq  # score elements of one head that the largest listed case has
        longest = _log_int(rng, 1, 12000)
        count = max(1, min(_log_int(rng, 1, 40), room // (longest * longest)))
        return {"op": op, "hq": hq, "hkv": hkv, "lens": _text([longest] + [_log_int(rng, 1, longest) for _ in range(count - 1)]),
                "pad": rng.choice((0, 0, 1, 77))}
    if op == "decode":
        longest = _log_int(rng, 1, 131072)
        count = max(1, min(_log_int(rng, 1, 200), 32 * 32768 * 8 // (longest * hkv)))
        lens = [longest] + [rng.randint(0, longest) for _ in range(count - 1)]
        return {"op": op, "hq": hq, "hkv": hkv, "lens": _text(lens), "kb": rng.choice((0, 0, rng.randint(1, 256)))}
    count = _log_int(rng, 1, 200)
    old = [rng.choice((0, rng.randint(1, 5000))) for _ in range(count)]
    most = max(1, (16000 * 8 // hkv if op == "store" else 2000000) // count)
    new = [rng.choice((1, _log_int(rng, 1, most))) for _ in range(count)]
    return {"op": op, **({"hkv": hkv} if op == "store" else {}), "old": _text(old), "new": _text(new), "pad": rng.choice((0, 3, 100))}


def work(case):
    op = case["op"]
    if op == "prompt":
        n = _lens(case["lens"])
        pairs = sum(x * (x + 1) // 2 for x in n)
        return {"bytes": 2 * D * sum(n) * (2 * case["hq"] + 2 * case["hkv"]) + 4 * (len(n) + 1), "flops": 4 * D * case["hq"] * pairs}
    if op == "decode":
        kb = case["kb"]
        # pages that are read, of one head; with a selection the whole of each chosen block
        pages = sum(min(kb, -(-x // BS)) if kb else -(-x // BS) for x in _lens(case["lens"])) * case["hkv"]
        b = len(_lens(case["lens"]))
        tables = 4 * (pages * 2 if kb else pages // case["hkv"]) + 4 * b
        return {"bytes": pages * (2 * BS * D + 8) + tables + 2 * 2 * b * case["hq"] * D,
                "flops": 4 * D * BS * pages * (case["hq"] // case["hkv"])}
    old, new = _lens(case["old"]), _lens(case["new"])
    rows = sum(new)
    if op == "store":
        # bf16 rows in, 8-bit rows out, a slot for each row, a scale for each page, head and K or V
        runs = sum(-(-(o + n) // BS) - o // BS for o, n in zip(old, new))
        return {"bytes": case["hkv"] * (2 * D * 3 * rows + 8 * runs) + 4 * (rows + case["pad"]), "flops": 4 * D * case["hkv"] * rows}
    pages = sum(-(-(o + n) // BS) - -(-o // BS) for o, n in zip(old, new))
    return {"bytes": 4 * (rows + case["pad"] + 2 * pages + 4 * len(old) + 2), "flops": rows}


# ------------------------------------------------------------------ the inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)


def _randn(shape, g, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _paged_inputs(old, new, g):
    """Tables of requests that hold `old` tokens, in pages shuffled over the pool, and the free pages."""
    b = len(old)
    held = [-(-o // BS) for o in old]
    need = [-(-(o + n) // BS) for o, n in zip(old, new)]
    pages = sum(need) + 7
    order = torch.randperm(pages, generator=g, device="cuda").int()
    nb = max(1, max(need))
    table = torch.full((b, nb), -1, dtype=torch.int32, device="cuda")
    cols = torch.arange(nb, device="cuda")[None, :] < _ints(held)[:, None]
    table[cols] = order[: sum(held)]
    return pages, table, order[sum(held):].contiguous(), sum(held)


def _cache(pages, batch, nb, hq, hkv):
    """The handle that a user's program keeps for its cache (the package's path only)."""
    from sparse_decode_attention_oasis_gb300.paged import PagedKV

    return PagedKV(n_pages=pages, batch=batch, nb_max=nb, n_q_heads=hq, n_kv_heads=hkv)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"op": op}
    if op == "prompt":
        lens, hq, hkv = _lens(case["lens"]), case["hq"], case["hkv"]
        rows = sum(lens) + case["pad"]
        # one buffer of a fused projection: queries, keys and values are slices of its rows
        qkv = _randn((rows, hq + 2 * hkv, D), g)
        qkv[:, :hq] *= 1.5
        s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], lens=lens,
                 start=_ints([sum(lens[:i]) for i in range(len(lens) + 1)]),
                 out=torch.full((rows, hq, D), 0.25, dtype=torch.bfloat16, device="cuda"))
        return s
    if op == "decode":
        lens, hq, hkv = _lens(case["lens"]), case["hq"], case["hkv"]
        b = len(lens)
        pages, table, _, _ = _paged_inputs(lens, [0] * b, g)
        # 8-bit values of normal keys and values whose size differs from page to page
        e = torch.randint(-9, -5, (pages, hkv, 2), generator=g, device="cuda")
        scale = torch.exp2(e.float())
        kv = torch.empty((pages, hkv, 2, BS, D), dtype=torch.uint8, device="cuda")
        for at in range(0, pages, 32768):  # in parts: the 32-bit draws of a large pool are larger than the pool
            part = kv[at:at + 32768]
            x = torch.randn(part.shape, generator=g, device="cuda").mul_(64.0).clamp_(-448, 448)
            part.copy_(x.to(torch.float8_e4m3fn).view(torch.uint8))
        s.update(q=_randn((b, hq, D), g), kv=kv, scale=scale, table=table, ctx=_ints(lens), hkv=hkv, sel=None, nsel=None,
                 out=torch.zeros((b, hq, D), dtype=torch.bfloat16, device="cuda"))
        if case["kb"]:
            kb, nb = case["kb"], table.shape[1]
            held = torch.div(s["ctx"] + (BS - 1), BS, rounding_mode="floor")
            n = held.clamp(max=kb)
            rank = torch.rand((b, hkv, nb), generator=g, device="cuda")
            rank.masked_fill_(torch.arange(nb, device="cuda")[None, None] >= held[:, None, None], 2.0)
            best = rank.argsort(dim=-1)[..., :kb]
            if best.shape[-1] < kb:
                best = torch.nn.functional.pad(best, (0, kb - best.shape[-1]))
            keep = torch.arange(kb, device="cuda")[None, None] < n[:, None, None]
            best = torch.where(keep, best, 1 << 30).sort(dim=-1).values
            s["sel"] = torch.where(keep, best, -1).int().contiguous()
            s["nsel"] = n[:, None].expand(b, hkv).int().contiguous()
        if own:
            s["cache"] = _cache(pages, b, table.shape[1], hq, hkv)
            s["cache"].adopt(kv=kv[None], scale=scale[None], table=table)
        return s
    old, new = _lens(case["old"]), _lens(case["new"])
    pages, table, free, held = _paged_inputs(old, new, g)
    b, rows = len(old), sum(new) + case["pad"]
    total = [o + n for o, n in zip(old, new)]
    if op == "tables":
        s.update(old=_ints(old), total=_ints(total), table=table, rows=rows, n_free=_ints([pages - held]),
                 free=torch.cat([free, torch.full((held,), -1, dtype=torch.int32, device="cuda")]))
        if own:
            s["cache"] = _cache(pages, b, table.shape[1], 8, 8)
            s["cache"].adopt(table=table, free=s["free"], lens=s["old"], n_free=s["n_free"])
        return s
    hkv = case["hkv"]
    kv = torch.zeros((pages, hkv, 2, BS, D), dtype=torch.uint8, device="cuda")
    scale = torch.ones((pages, hkv, 2), device="cuda")
    firsts = [o // BS for o in old]
    for i, o in enumerate(old):  # the pages that new tokens continue hold earlier ones
        if o % BS:
            p = int(table[i, firsts[i]])
            x = torch.randn((hkv, 2, BS, D), generator=g, device="cuda")
            e = _exponent(x[:, :, : o % BS].abs().amax(dim=(2, 3)))
            scale[p] = torch.exp2(e.float())
            x[:, :, o % BS:] = 0
            kv[p] = (x * torch.exp2(-e.float())[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    slots = []
    at, spare = 0, free.flip(0)  # pages are taken from the end of the free list
    for i, (o, n) in enumerate(zip(old, new)):
        have, want = -(-o // BS), -(-(o + n) // BS)
        own_pages = torch.cat([table[i, :have], spare[at:at + want - have]])
        at += want - have
        t = torch.arange(o, o + n, device="cuda")
        slots.append(own_pages[t // BS].long() * BS + t % BS)
    slots.append(torch.full((case["pad"],), -1, device="cuda"))
    # one buffer of a fused projection; sizes that differ from token to token, and an outlier channel
    rowsize = torch.exp2(torch.randint(-1, 3, (rows, 1, 1), generator=g, device="cuda").float())
    kvrows = torch.randn((rows, 2 * hkv, D), generator=g, device="cuda") * rowsize
    kvrows[:, :hkv, 5] *= 8
    kvrows = kvrows.to(torch.bfloat16)
    s.update(k=kvrows[:, :hkv], v=kvrows[:, hkv:], slots=torch.cat(slots).int(), kv=kv, scale=scale)
    if own:
        s["cache"] = _cache(pages, b, table.shape[1], hkv, hkv)
        s["cache"].adopt(kv=kv[None], scale=scale[None], table=table)
    return s


# ------------------------------------------------------------------ the plain forms
def _plain_prompt(s):
    q, k, v, lens = s["q"], s["k"], s["v"], _ints(s["lens"]).long()
    hkv, group, n = k.shape[1], q.shape[1] // k.shape[1], max(s["lens"])
    t = torch.arange(n, device="cuda")
    valid = t[None] < lens[:, None]                                            # [B, n]
    at = torch.where(valid, s["start"][:-1, None].long() + t[None], 0)
    zero = torch.zeros((), device="cuda")

    def padded(x):                                                             # [B, heads, n, D]
        return torch.where(valid[:, :, None, None], x[at].float(), zero).transpose(1, 2)

    b = len(s["lens"])
    qp = padded(q).reshape(b, hkv, group * n, D)
    score = torch.matmul(qp, padded(k).transpose(-1, -2)).view(b, hkv, group, n, n)
    score.mul_(1.0 / math.sqrt(D)).masked_fill_(t[None, :] > t[:, None], -math.inf)
    score.sub_(score.amax(dim=-1, keepdim=True)).exp_()
    total = score.sum(dim=-1, keepdim=True)
    o = torch.matmul(score.view(b, hkv, group * n, n), padded(v)).view(b, hkv, group, n, D) / total
    s["out"][at[valid]] = o.permute(0, 3, 1, 2, 4).reshape(b, n, hkv * group, D)[valid].to(torch.bfloat16)
    return s["out"]


def _plain_decode(s):
    q, kv, scale, table, ctx, hkv = s["q"], s["kv"], s["scale"], s["table"].long(), s["ctx"].long(), s["hkv"]
    b, hq, nb = q.shape[0], q.shape[1], table.shape[1]
    if s["sel"] is None:
        blocks = torch.arange(nb, device="cuda").expand(b, hkv, nb)
        chosen = torch.ones_like(blocks, dtype=torch.bool)
    else:
        blocks = s["sel"].long()
        chosen = torch.arange(blocks.shape[-1], device="cuda") < s["nsel"][..., None]
        blocks = blocks.clamp(min=0)
    n = blocks.shape[-1]
    page = table[:, None].expand(b, hkv, nb).gather(2, blocks)
    chosen = chosen & (page >= 0)
    page = page.clamp(min=0)
    head = torch.arange(hkv, device="cuda")[None, :, None]
    valid = chosen[..., None] & (blocks[..., None] * BS + torch.arange(BS, device="cuda") < ctx[:, None, None, None])
    valid = valid.view(b, hkv, 1, n * BS)
    zero = torch.zeros((), device="cuda")

    def rows(which):                                                           # [B, hkv, tokens, D]
        x = kv[page, head, which].view(torch.float8_e4m3fn).float() * scale[page, head, which][..., None, None]
        return torch.where(valid.view(b, hkv, n * BS, 1), x.view(b, hkv, n * BS, D), zero)

    score = torch.matmul(q.float().view(b, hkv, hq // hkv, D), rows(0).transpose(-1, -2)) * (1.0 / math.sqrt(D))
    score = score.masked_fill(~valid, -math.inf)
    top = score.amax(dim=-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, zero, top))
    total = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p, rows(1)) / torch.where(total == 0, torch.ones_like(total), total)
    s["out"].copy_(o.view(b, hq, D))
    return s["out"]


def _exponent(amax):
    """The least e with amax <= 448 * 2^e, inside the scales' range."""
    m, x = torch.frexp(amax)
    return torch.where(amax > 0, x - 9 + (m > 0.875), E_LOW).clamp(E_LOW, E_HIGH)


def _plain_store(s):
    slots = s["slots"].long()
    used = slots >= 0
    slots = slots[used]
    x = torch.stack([s["k"][used], s["v"][used]], dim=2).float()               # [rows, hkv, 2, D]
    page, pos = slots // BS, slots % BS
    first = torch.ones_like(page, dtype=torch.bool)
    first[1:] = page[1:] != page[:-1]
    run = first.cumsum(0) - 1                                                  # the page's group of rows
    page_of, pos_of = page[first], pos[first]
    amax = x.new_zeros((page_of.numel(),) + x.shape[1:3]).index_reduce_(0, run, x.abs().amax(dim=-1), "amax")
    kept = torch.arange(BS, device="cuda")[None] < pos_of[:, None]             # tokens that the page holds already
    before = s["scale"][page_of]
    e_old = torch.frexp(before)[1] - 1
    e = _exponent(amax)
    e = torch.where((pos_of > 0)[:, None, None], torch.maximum(e, e_old), e)
    shift = torch.exp2((e_old - e).float())[..., None, None]
    old = s["kv"][page_of].view(torch.float8_e4m3fn).float() * shift
    again = torch.where(kept[:, None, None, :, None], old.to(torch.float8_e4m3fn).view(torch.uint8), s["kv"][page_of])
    s["kv"][page_of] = again
    s["scale"][page_of] = torch.exp2(e.float())
    y = (x * torch.exp2(-e.float())[run][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    s["kv"][page, :, :, pos] = y
    return {"pages": s["kv"].view(torch.float8_e4m3fn), "scale": s["scale"]}


def _plain_tables(s):
    old, total, table, rows = s["old"].long(), s["total"].long(), s["table"], s["rows"]
    b = old.numel()
    held, want = (old + BS - 1) // BS, (total + BS - 1) // BS
    need, grow = want - held, total - old
    zero = torch.zeros(1, dtype=torch.long, device="cuda")
    first_page, start = torch.cat([zero, need.cumsum(0)]), torch.cat([zero, grow.cumsum(0)])
    who = torch.repeat_interleave(torch.arange(b, device="cuda"), need)
    k = torch.arange(who.numel(), device="cuda")
    table[who, held[who] + k - first_page[who]] = s["free"][s["n_free"].long() - 1 - k]
    who = torch.repeat_interleave(torch.arange(b, device="cuda"), grow)
    at = old[who] + torch.arange(who.numel(), device="cuda") - start[who]
    slots = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    slots[: who.numel()] = table[who, at // BS] * BS + (at % BS).int()
    return {"slots": slots, "start": start.int(), "table": table, "lens": s["total"].clone(),
            "n_free": s["n_free"] - first_page[-1:].int()}


# ------------------------------------------------------------------ one pass
def run(state):
    s = state
    if own:
        op = s["op"]
        if op == "prompt":
            from sparse_decode_attention_oasis_gb300.paged import prompt_attn

            return prompt_attn(s["q"], s["k"], s["v"], s["start"], out=s["out"])
        if op == "decode":
            return s["cache"].decode(s["q"], s["ctx"], sel=s["sel"], nsel=s["nsel"], out=s["out"])
        if op == "store":
            s["cache"].store(s["k"], s["v"], s["slots"])
            return {"pages": s["kv"].view(torch.float8_e4m3fn), "scale": s["scale"]}
        plan = s["cache"].extend(s["total"], s["rows"])
        return {"slots": plan.slot_map, "start": plan.row_start, "table": s["table"], "lens": plan.lens, "n_free": plan.n_free}
    return {"prompt": _plain_prompt, "decode": _plain_decode, "store": _plain_store, "tables": _plain_tables}[s["op"]](s)


# ------------------------------------------------------------------ in 64 bits
def _exact_prompt(s):
    out = torch.full(s["q"].shape, 0.25, dtype=torch.float64, device="cuda")
    group, at = s["q"].shape[1] // s["k"].shape[1], 0
    for n in s["lens"]:
        for h in range(s["q"].shape[1]):
            k, v = (s[x][at:at + n, h // group].double() for x in "kv")
            for r in range(0, n, 8192):  # rows in parts
                q = s["q"][at + r:min(at + r + 8192, at + n), h].double()
                w = (q @ k.T) / math.sqrt(D)
                w = torch.softmax(w + torch.full_like(w, -math.inf).triu_(r + 1), dim=-1)
                out[at + r:at + r + q.shape[0], h] = w @ v
        at += n
    return out


def _exact_decode(s):
    q, out = s["q"].double(), torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group, lens = q.shape[1] // s["hkv"], s["ctx"].tolist()
    for i, n in enumerate(lens):
        for h in range(s["hkv"]):
            blocks = range(-(-n // BS)) if s["sel"] is None else s["sel"][i, h, : int(s["nsel"][i, h])].tolist()
            t = torch.tensor([x * BS + j for x in blocks for j in range(BS) if x * BS + j < n], dtype=torch.long, device="cuda")
            if not t.numel():
                continue
            page = s["table"][i].long()[t // BS]
            k, v = (s["kv"][page, h, w, t % BS].view(torch.float8_e4m3fn).double() * s["scale"][page, h, w].double()[:, None]
                    for w in (0, 1))
            rows = slice(h * group, (h + 1) * group)
            out[i, rows] = torch.softmax(q[i, rows] @ k.T / math.sqrt(D), dim=-1) @ v
    return out


def _exact_e4m3(x):
    """x in 64 bits rounded to the nearest e4m3 value, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))).clamp(min=-6) - 3)
    return torch.round(x / step) * step


def _exact_store(s):
    values, scale = s["kv"].view(torch.float8_e4m3fn).double(), s["scale"].double().clone()
    slots, at = s["slots"].tolist(), 0
    while at < len(slots):
        end = at + 1
        while slots[at] >= 0 and end < len(slots) and slots[end] // BS == slots[at] // BS:
            end += 1
        if slots[at] >= 0:
            p, first = divmod(slots[at], BS)
            rows = torch.stack([s["k"][at:end], s["v"][at:end]], dim=1).double().permute(2, 1, 0, 3)  # [hkv, 2, rows, D]
            most = rows.abs().amax(dim=(2, 3))
            low = torch.floor(torch.log2(most.clamp(min=2.0 ** -200) / 448)) - 1
            need = low + sum((most > 448 * torch.exp2(low + i)).double() for i in range(3))  # the least that holds it
            e = torch.exp2(need.clamp(E_LOW, E_HIGH))
            if first:
                e = torch.maximum(e, scale[p])
                values[p, :, :, :first] = _exact_e4m3(values[p, :, :, :first] * (scale[p] / e)[..., None, None])
            scale[p] = e
            values[p, :, :, first:first + end - at] = _exact_e4m3(rows / e[..., None, None])
        at = end
    return {"pages": values, "scale": scale}


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "tables":
        return None  # whole numbers
    return {"prompt": _exact_prompt, "decode": _exact_decode, "store": _exact_store}[s["op"]](s)
