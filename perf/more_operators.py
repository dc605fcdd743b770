"""The attention half of a decoder block over a key-value cache held in 8 bits, as cases to be measured.

Four operators: new tokens' keys and values into the cache (``append``),
attention of new tokens over it (``attention``), the cached tokens' values
(``read``) and a sequence that continues another one (``fork``).  The cache
holds pages of P tokens; a full page has 8-bit codes with one scale for its
keys and one for its values of each head, a sequence's last, incomplete page is
kept as it came.  Each case runs in its plain form (elementary torch
operations in 32 bits) or, with ``own`` set, through the framework's entry
points.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    # len: tokens of the longest sequence before the call; new: its new tokens (ragged: other sequences have
    # anything from none to as many); heads per kv head: group
    return [
        # the tokens of a decode batch; some complete their page
        {"name": "append decode", "op": "append", "B": 64, "len": 4095, "new": 1, "ragged": False, "kv": 8, "D": 128,
         "page": 16, "dtype": "bf16", "fork": False},
        # chunks of ragged lengths that continue shared prefixes in the middle of a page
        {"name": "append ragged chunks", "op": "append", "B": 9, "len": 777, "new": 501, "ragged": True, "kv": 5,
         "D": 64, "page": 32, "dtype": "f16", "fork": True},
        # prompts into an empty cache
        {"name": "append prompts", "op": "append", "B": 4, "len": 0, "new": 8192, "ragged": False, "kv": 8, "D": 128,
         "page": 64, "dtype": "bf16", "fork": False},
        # one decoded token of one short sequence (latency)
        {"name": "attention one token", "op": "attention", "B": 1, "len": 600, "new": 1, "ragged": False, "kv": 2,
         "group": 8, "D": 128, "page": 64, "dtype": "bf16", "window": 0},
        # a decode batch of ragged lengths
        {"name": "attention decode", "op": "attention", "B": 64, "len": 8191, "new": 1, "ragged": False, "kv": 8,
         "group": 8, "D": 128, "page": 64, "dtype": "bf16", "window": 0},
        # one decoded token of a very long sequence
        {"name": "attention long", "op": "attention", "B": 1, "len": 131000, "new": 1, "ragged": False, "kv": 4,
         "group": 7, "D": 128, "page": 128, "dtype": "f16", "window": 0},
        # a mixed batch of chunks and single tokens in a layer with a sliding window, odd head counts, small pages
        {"name": "attention mixed window", "op": "attention", "B": 9, "len": 1777, "new": 501, "ragged": True, "kv": 5,
         "group": 3, "D": 64, "page": 16, "dtype": "f16", "window": 1000},
        # the second chunk of two prompts
        {"name": "attention prefill", "op": "attention", "B": 2, "len": 4096, "new": 4096, "ragged": False, "kv": 8,
         "group": 4, "D": 128, "page": 64, "dtype": "bf16", "window": 0},
        # a short sequence handed to another process
        {"name": "read short", "op": "read", "B": 1, "len": 300, "new": 301, "kv": 2, "D": 128, "page": 64,
         "dtype": "bf16"},
        # ragged sequences moved out of the cache
        {"name": "read sequences", "op": "read", "B": 8, "len": 0, "new": 8191, "kv": 8, "D": 128, "page": 64,
         "dtype": "bf16"},
        # four samples of one prompt
        {"name": "fork samples", "op": "fork", "B": 1, "copies": 4, "len": 601, "kv": 2, "D": 128, "page": 64,
         "dtype": "bf16"},
        # the sequences of many beams after a selection
        {"name": "fork beams", "op": "fork", "B": 32, "copies": 4, "len": 2047, "kv": 8, "D": 128, "page": 64,
         "dtype": "bf16"},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, its logarithm even."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "read", "fork"])
    kv, D, dtype = rng.choice([1, 2, 3, 4, 5, 8]), rng.choice([64, 128, 128, 192, 256]), rng.choice(["bf16", "bf16", "f16"])
    c = {"op": op, "kv": kv, "D": D, "page": rng.choice([16, 32, 64, 128]), "dtype": dtype}
    B = _spread(rng, 1, 128)
    if op == "fork":
        copies = rng.randint(1, 8)
        n = _spread(rng, 1, 4096)
        return {**c, "B": max(1, B // copies), "copies": copies, "len": n + (n % c["page"] == 0)}
    # as many tokens in the cache as the listed decode batch has, or fewer
    most = 64 * 8192 * 8 * 128 // (kv * D * B)
    held = min(_spread(rng, 1, 131072), most // 2)
    if op == "read":
        return {**c, "B": B, "len": held // 2, "new": min(max(1, held // 2), 4 * 8192 * 8 * 128 // (kv * D * B)),
                "dtype": rng.choice([dtype, "f32"])}
    if op == "append":
        new = min(rng.choice([1, _spread(rng, 2, 4096)]), 4 * 8192 * 8 * 128 // (kv * D * B))
        held = rng.choice([0, held // 4]) if new > 1 else held
        # a chunk behind older tokens replaces those of an incomplete page, so it goes to a fork of them
        return {**c, "B": B, "len": held, "new": new, "ragged": rng.random() < 0.5,
                "fork": held > 0 and (new > 1 or rng.random() < 0.5)}
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    # the padded batch's products: no more than those of the listed chunks
    most = 2 * 4096 * 8192 * 32 * 128 // (2 * B * held * kv * group * D)
    new = min(rng.choice([1, _spread(rng, 2, 4096)]), max(1, most), held)
    return {**c, "B": B, "len": held, "new": new, "ragged": rng.random() < 0.5, "group": group,
            "window": rng.choice([0, 0, rng.randint(1, 2000)])}


def _counts(c):
    """Tokens that each sequence holds before the call, and its new ones."""
    rng = random.Random(c["B"] * 1000003 + c["len"])
    held = [c["len"]] + [rng.randint(c["len"] // 4, c["len"]) for _ in range(c["B"] - 1)]
    if c["op"] == "fork":
        return held, [0] * c["B"]
    if c["op"] == "read":
        return held, [max(1, c["new"] - 37 * i) for i in range(c["B"])]
    most = c["new"]
    return held, [most] + [rng.choice([0, 1, rng.randint(0, most)]) if c["ragged"] else most for _ in range(c["B"] - 1)]


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(counts):
    total = [0]
    for n in counts:
        total.append(total[-1] + n)
    return total


def _touched(held, new, table, slots, P):
    """The pages that new tokens fall on, as index tensors: the sequence's table entry, the tokens' places among the
    new ones (-1: an older token or none) and whether a page gets full."""
    first = torch.tensor(_starts(new)[:-1], device="cuda")
    h, n = torch.tensor(held, device="cuda"), torch.tensor(new, device="cuda")
    pages = torch.where(n > 0, (h + n + P - 1) // P - h // P, 0)
    seq = torch.repeat_interleave(torch.arange(len(held), device="cuda"), pages)
    number = torch.arange(seq.numel(), device="cuda") - (pages.cumsum(0) - pages)[seq] + (h // P)[seq]
    pos = number[:, None] * P + torch.arange(P, device="cuda")
    place = torch.where((pos >= h[seq, None]) & (pos < (h + n)[seq, None]), first[seq, None] + pos - h[seq, None], -1)
    full = (h + n)[seq] >= (number + 1) * P
    return {"place": place, "older": pos < h[seq, None], "slot": slots.long()[seq], "full": full.nonzero()[:, 0],
            "part": (~full).nonzero()[:, 0], "page": table.long()[seq, number][full]}


def prepare(case, seed):
    c, gen = case, torch.Generator(device="cuda").manual_seed(seed)
    kv, D, P = c["kv"], c["D"], c["page"]
    dt = DTYPES["bf16" if c["dtype"] == "f32" else c["dtype"]]
    held, new = _counts(c)
    B, forks = c["B"], c["B"] * c["copies"] if c["op"] == "fork" else c["B"] if c.get("fork") else 0
    # tokens in the cache before the call (attention's and read's own among them)
    inside = [h + n for h, n in zip(held, new)] if c["op"] in ("attention", "read") else held

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    spread_k, spread_v = torch.exp(0.5 * normal(kv, D)), torch.exp(0.3 * normal(kv, D))

    def tokens(n):
        """keys with larger channels, values around a mean"""
        return (spread_k * normal(n, kv, D)).to(dt), (spread_v * (normal(n, kv, D) + 0.3)).to(dt)

    # sequences own scattered pages; a fork shares its parent's full pages and has the rest of its own
    rows = B + forks
    parent = [i % B for i in range(forks)]
    need = [-(-(h + n) // P) for h, n in zip(held, new)]
    width = max(need) + 2
    own_pages = need + [need[p] - held[p] // P + 1 for p in parent]
    pages = sum(own_pages) + 3
    ids = torch.randperm(pages, generator=gen, device="cuda", dtype=torch.int32)
    at = torch.zeros((rows, width), dtype=torch.int64)
    starts = _starts(own_pages)
    for i in range(rows):
        skip = held[parent[i - B]] // P if i >= B else 0
        count = own_pages[i]
        at[i, skip:skip + count] = torch.arange(starts[i], starts[i] + count)
    table = ids[at.cuda()].contiguous()
    slots = torch.randperm(rows + 2, generator=gen, device="cuda", dtype=torch.int32)[:rows].contiguous()
    s = {"case": c, "pages": pages, "slot_count": rows + 2, "table": table, "slots": slots, "lens": _ints(held + [0] * forks),
         "cu": _ints(_starts(new)), "past": tokens(sum(inside)), "inside": inside, "parent": parent,
         "tokens": sum(new)}

    # the cache in its plain layout: codes and scales of full pages, the last tokens as they are
    s["codes"] = torch.zeros((pages, 2, kv, P, D), dtype=torch.int8, device="cuda")
    s["scales"] = torch.zeros((pages, 2, kv), device="cuda")
    s["tails"] = torch.zeros((rows + 2, 2, kv, P, D), dtype=dt, device="cuda")
    _write(s, *s["past"], _touched([0] * B, inside, table, slots, P))

    if c["op"] == "append":
        s["k"], s["v"] = tokens(sum(new))
        if forks:
            s["src"], s["dst"] = _ints(parent), _ints(list(range(B, 2 * B)))
        # the appended tokens' sequences: the forks, where there are any
        s["t_table"], s["t_slots"] = table[-B:], slots[-B:]
        s["touched"] = _touched(held, new, s["t_table"], s["t_slots"], P)
        # all tokens of the pages that changed are read back
        back = [h // P * P if n else h for h, n in zip(held, new)]
        s["back"] = _read_plan(s, back, [h + n - b for h, n, b in zip(held, new, back)], s["t_table"], s["t_slots"])
    elif c["op"] == "attention":
        heads = kv * c["group"]
        s["q"] = (1.5 * normal(sum(new), heads, D) / spread_k.repeat_interleave(c["group"], 0)).to(dt)
        # the tokens' places in the padded batch
        n = torch.tensor(new, device="cuda")
        s["row"] = torch.repeat_interleave(torch.arange(B, device="cuda"), n)
        s["col"] = torch.arange(sum(new), device="cuda") - torch.tensor(_starts(new)[:-1], device="cuda")[s["row"]]
        s["most"] = max(new)
        s["end"] = torch.tensor(inside, device="cuda")
    elif c["op"] == "read":
        s["back"] = _read_plan(s, held, new, table, slots)
    else:
        s["src"], s["dst"] = _ints(parent), _ints(list(range(B, rows)))
        last = [held[p] % P for p in parent]
        s["back"] = _read_plan(s, [held[p] - n for p, n in zip(parent, last)], last, table[B:], slots[B:])
    return s


def _read_plan(s, start, count, table, slots):
    """Where the `count` last tokens of sequences, from `start` on, are: pages, or the kept tokens of a slot."""
    P = s["case"]["page"]
    n, b = torch.tensor(count, device="cuda"), torch.tensor(start, device="cuda")
    seq = torch.repeat_interleave(torch.arange(len(count), device="cuda"), n)
    pos = torch.arange(seq.numel(), device="cuda") - (n.cumsum(0) - n)[seq] + b[seq]
    return {"table": table, "slots": slots, "lens": _ints(start), "cu": _ints(_starts(count)), "tokens": sum(count),
            "seq": seq, "number": pos // P, "offset": pos % P, "kept": pos // P == ((b + n) // P)[seq]}


# --- plain forms ---------------------------------------------------------------

def _write(s, k, v, plan):
    """Keys and values into the plain cache: the touched pages' tokens together, a full page quantized with one scale
    for its keys and one for its values of each head."""
    new = torch.stack((k, v), 1)
    place = plan["place"]
    x = torch.zeros((place.shape[0], *s["tails"].shape[1:]), dtype=k.dtype, device=k.device)
    if new.shape[0]:
        x = torch.where((place >= 0)[:, None, None, :, None], new[place.clamp(min=0)].permute(0, 2, 3, 1, 4), x)
    x = torch.where(plan["older"][:, None, None, :, None], s["tails"][plan["slot"]], x)
    full, part = plan["full"], plan["part"]
    f = x[full].float()
    top = f.abs().amax((3, 4))
    some = top >= 2.0 ** -119
    most = torch.full_like(top, 127.0)  # a tensor: a number on either side of / may become a reciprocal
    top = torch.where(some, top, most)
    code = (f * torch.div(most, top)[..., None, None]).round()
    s["codes"][plan["page"]] = torch.where(some[..., None, None], code, 0.0).to(torch.int8)
    s["scales"][plan["page"]] = torch.where(some, torch.div(top, most), 0.0)
    s["tails"][plan["slot"][part]] = x[part]


def _values(s, plan, dtype):
    page = plan["table"].long()[plan["seq"], plan["number"].clamp(max=plan["table"].shape[1] - 1)]
    # a full page's codes times their scale, or the value as it came
    x = s["codes"][page, :, :, plan["offset"]].float() * s["scales"][page][..., None]
    kept = s["tails"][plan["slots"].long()[plan["seq"]], :, :, plan["offset"]].float()
    x = torch.where(plan["kept"][:, None, None, None], kept, x).to(dtype)
    return x[:, 0].contiguous(), x[:, 1].contiguous()


def _forked(s):
    P, src, dst = s["case"]["page"], s["src"].long(), s["dst"].long()
    table, lens, slots = s["table"], s["lens"], s["slots"].long()
    number = torch.arange(table.shape[1], device="cuda")
    table[dst] = torch.where(number < (lens[src] // P)[:, None], table[src], table[dst])
    lens[dst] = lens[src]
    s["tails"][slots[dst]] = s["tails"][slots[src]]


def _append(s, c):
    if c["fork"]:
        _forked(s)
    _write(s, s["k"], s["v"], s["touched"])
    return _values(s, s["back"], DTYPES[c["dtype"]])


def _attention(s, c):
    B, kv, G, D, P, most = c["B"], c["kv"], c["group"], c["D"], c["page"], s["most"]
    table, end = s["table"].long(), s["end"]
    x = s["codes"][table].float() * s["scales"][table][..., None, None]  # [B, W, 2, kv, P, D]
    x[torch.arange(B, device="cuda"), end // P] = s["tails"][s["slots"].long()].float()
    n = x.shape[1] * P
    k = x[:, :, 0].permute(0, 2, 4, 1, 3).reshape(B * kv, D, n)
    v = x[:, :, 1].permute(0, 2, 1, 3, 4).reshape(B * kv, n, D)
    q = torch.zeros((B, most, kv, G, D), device="cuda")
    q[s["row"], s["col"]] = s["q"].float().view(-1, kv, G, D)
    q = q.permute(0, 2, 1, 3, 4).reshape(B * kv, most * G, D)
    score = torch.matmul(q * D ** -0.5, k).view(B, kv, most, G, n)
    pos = s["lens"][:, None].long() + torch.arange(most, device="cuda")
    j = torch.arange(n, device="cuda")
    seen = (j <= pos[..., None]) & (j < end[:, None, None])
    if c["window"]:
        seen = seen & (j > pos[..., None] - c["window"])
    score.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(torch.where(top > -math.inf, top, 0.0)).exp_()
    total = score.sum(-1, keepdim=True)
    out = torch.matmul(score.view(B * kv, most * G, n), v).view(B, kv, most, G, D) / torch.where(total > 0, total, 1.0)
    out = out.permute(0, 2, 1, 3, 4)[s["row"], s["col"]]
    return out.reshape(-1, kv * G, D).to(s["q"].dtype)


def _read(s, c):
    return _values(s, s["back"], DTYPES[c["dtype"]])


def _fork(s, c):
    _forked(s)
    return (s["table"], s["lens"], *_values(s, s["back"], DTYPES[c["dtype"]]))


# --- the framework's calls -----------------------------------------------------

def _own(s, c):
    from nvfp4_token_quant_amd import binding
    if "cache" not in s:  # a program's cache holds the tokens of earlier calls
        s["cache"] = binding.KvCache(s["pages"], s["slot_count"], c["kv"], c["D"], page_size=c["page"])
        B = c["B"]
        binding.kv_append(s["cache"], *s["past"], s["table"][:B], torch.zeros_like(s["lens"][:B]), s["slots"][:B],
                          cu=_ints(_starts(s["inside"])))
    cache = s["cache"]

    def back():
        p = s["back"]
        return binding.kv_read(cache, p["table"], p["lens"], p["slots"], cu=p["cu"], tokens=p["tokens"],
                               dtype=DTYPES[c["dtype"]])

    if c["op"] == "append":
        if c["fork"]:
            binding.kv_fork(cache, s["table"], s["lens"], s["slots"], s["src"], s["dst"])
        one = c["new"] == 1 and not c["ragged"]
        binding.kv_append(cache, s["k"], s["v"], s["t_table"], s["lens"][-c["B"]:], s["t_slots"],
                          cu=None if one else s["cu"])
        return back()
    if c["op"] == "attention":
        one = c["new"] == 1 and not c["ragged"]
        return binding.kv_attention(cache, s["q"], s["table"], s["lens"], s["slots"], cu=None if one else s["cu"],
                                    window=c["window"])
    if c["op"] == "read":
        return back()
    binding.kv_fork(cache, s["table"], s["lens"], s["slots"], s["src"], s["dst"])
    return (s["table"], s["lens"], *back())


def run(state):
    c = state["case"]
    if own:
        return _own(state, c)
    return {"append": _append, "attention": _attention, "read": _read, "fork": _fork}[c["op"]](state, c)


def work(case):
    c, b = case, SIZES[case["dtype"]]
    held, new = _counts(c)
    kv, D, P = c["kv"], c["D"], c["page"]
    token = 2 * kv * D  # values of a token
    if c["op"] == "append":
        whole = sum((h + n) // P * P - h // P * P for h, n in zip(held, new))
        kept = sum(min((h + n) % P, n) for h, n in zip(held, new))
        older = sum(h % P for h, n in zip(held, new) if n)
        back = sum(h + n - h // P * P for h, n in zip(held, new) if n)
        scales = whole // P * 2 * kv * 4
        return {"bytes": token * (b * sum(new) + whole + 2 * kept + 2 * older * (2 if c["fork"] else 1) + b * back)
                + scales, "flops": 4 * token * whole}
    if c["op"] == "attention":
        w = c["window"] or 1 << 60
        seen = [min(h + n, n + w - 1) if n else 0 for h, n in zip(held, new)]
        pairs = sum(sum(min(h + i + 1, w) for i in range(n)) for h, n in zip(held, new))
        return {"bytes": sum(seen) * kv * 2 * D + sum(-(-m // P) for m in seen) * kv * 8
                + 2 * sum(new) * kv * c["group"] * D * b, "flops": 4 * D * kv * c["group"] * pairs}
    if c["op"] == "read":
        kept = sum(min((h + n) % P, n) for h, n in zip(held, new))
        return {"bytes": token * (sum(new) * (b + 1) + kept), "flops": token * sum(new)}
    copies = c["copies"]
    return {"bytes": copies * sum(token * (4 + b) * (h % P) + 8 * (h // P) + 8 for h in held) - 2 * token * (copies - 1)
            * sum(h % P for h in held), "flops": token * copies * sum(h % P for h in held)}


# --- the definitions in 64 bits ------------------------------------------------

def _token_values(s, x, lens):
    """What the cache gives for the tokens x [n, kv, D] of sequences with `lens` tokens each, in 64 bits."""
    P, out, first = s["case"]["page"], [], 0
    for n in lens:
        y = x[first:first + n].double()
        first += n
        whole = n // P * P
        page = y[:whole].view(-1, P, *y.shape[1:])
        # a code is the nearest whole number to x times the 32-bit number 127 / max|x|, that product in 32 bits
        top = page.abs().amax(dim=(1, 3), keepdim=True)
        none = top < 2.0 ** -119
        factor = torch.where(none, 0.0, 127.0 / top.clamp(min=2.0 ** -119)).float().double()
        unit = torch.where(none, 0.0, top / 127.0).float().double()
        page = torch.round((page * factor).float().double()) * unit
        out.append(torch.cat((page.reshape(whole, *y.shape[1:]), y[whole:])))
    return out


def exact(case, seed):
    s, c = prepare(case, seed), case
    held, new = _counts(c)
    P = c["page"]
    past_k, past_v = (t.split(s["inside"]) for t in s["past"])
    if c["op"] == "append":
        ks, vs = s["k"].split(new), s["v"].split(new)
        total = [h + n for h, n in zip(held, new)]
        out = []
        for past, now in ((past_k, ks), (past_v, vs)):
            x = torch.cat([torch.cat(p) for p in zip(past, now)])
            # the tokens of the pages that new tokens fall on
            y = _token_values(s, x, total)
            out.append(torch.cat([v[h // P * P if n else h:] for v, h, n in zip(y, held, new)]))
        return tuple(out)
    k, v = (_token_values(s, x, s["inside"]) for x in s["past"])
    if c["op"] == "read":
        return tuple(torch.cat([y[h:] for y, h in zip(x, held)]) for x in (k, v))
    if c["op"] == "fork":
        last = [[x[p][held[p] // P * P:] for p in s["parent"]] for x in (k, v)]
        return (None, None, torch.cat(last[0]), torch.cat(last[1]))
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    first = 0
    for i, (h, n) in enumerate(zip(held, new)):
        q = s["q"][first:first + n].double()
        if n:
            j, p = torch.arange(h + n, device="cuda"), torch.arange(h, h + n, device="cuda")[:, None]
            hidden = (j > p) | (j <= p - (c["window"] or h + n))
            for head in range(q.shape[1]):
                w = (q[:, head] @ k[i][:, head // c["group"]].t()) / math.sqrt(c["D"])
                w = torch.softmax(torch.where(hidden, -math.inf, w), 1)
                out[first:first + n, head] = w @ v[i][:, head // c["group"]]
        first += n
    return out
