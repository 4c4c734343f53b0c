"""Operators around the key-value cache in their plain form, the cases that they
are measured at, and the same calls through the library.

Operators: `rotate` turns the heads of rows by their positions (rotary
positions: halves or pairs, part of the head, scaled for long contexts),
optionally after a norm of each head; `append` does that to the queries and
keys of new tokens and quantizes keys and values into their pages in the same
pass; `shared` is attention for a batch whose sequences begin with the same
tokens, group by group; `read` gives tokens of the cache back as rows.

The cache holds keys and values in 8 bits (e4m3, largest value 448) with one
power-of-two scale for every block of 16 tokens of a head, in pages of `page`
tokens:

    k        uint8 [layers][pages][kv heads][page tokens][head dim]
    v        uint8 [layers][pages][kv heads][page tokens / 4][head dim][4]
    scales   fp32  [layers][pages][kv heads][page tokens / 16], one array each
"""
import math

import torch

own = False

BLOCK = 16          # tokens under one scale
TOP = 448.0         # largest e4m3 value
LOW, HIGH = -40, 100  # exponents that a scale may have
EPS = 1e-6          # of the norms


def listed():
    return [
        # the queries of one decoded token, as the projection leaves them: a latency
        {"name": "rotate_token", "op": "rotate", "rows": 1, "heads": 28, "dim": 128, "dims": 128,
         "layout": "halves", "type": "fp32", "to": "bf16", "norm": False, "scaling": "plain",
         "base": 1e6, "start": 14449},
        # all queries of the prompt of a 32-minute recording: pairs, part of the
        # head, context extended four times, each head normed
        {"name": "rotate_prompt", "op": "rotate", "rows": 14449, "heads": 32, "dim": 128, "dims": 96,
         "layout": "pairs", "type": "bf16", "to": "bf16", "norm": True, "scaling": "ramp",
         "base": 1e4, "start": 0},
        # one decoded token of one sequence, 28 query heads over 4: a latency
        {"name": "append_token", "op": "append", "seqs": 1, "heads": 28, "kv": 4, "dim": 128,
         "page": 64, "rows": 1, "length": 1025, "type": "fp32", "dims": 128, "layout": "halves",
         "norm": False, "scaling": "plain", "base": 1e6},
        # a full server decoding: 64 sequences of every length, normed heads
        {"name": "append_batch", "op": "append", "seqs": 64, "heads": 32, "kv": 8, "dim": 128,
         "page": 64, "rows": 1, "length": 2000, "type": "fp32", "dims": 128, "layout": "halves",
         "norm": True, "scaling": "smooth", "base": 1e6},
        # the recording's prompt, straight from the fp32 projection
        {"name": "append_prompt", "op": "append", "seqs": 1, "heads": 28, "kv": 4, "dim": 128,
         "page": 64, "rows": 14449, "length": 14449, "type": "fp32", "dims": 128,
         "layout": "halves", "norm": False, "scaling": "plain", "base": 1e6},
        # chunks of several prompts, heads of 64 of which an odd number of pairs turns
        {"name": "append_chunks", "op": "append", "seqs": 5, "heads": 32, "kv": 8, "dim": 64,
         "page": 16, "rows": 701, "length": 3001, "type": "bf16", "dims": 50, "layout": "halves",
         "norm": True, "scaling": "linear", "base": 1e4},
        # beams over a long recording
        {"name": "shared_beams", "op": "shared", "seqs": 8, "groups": 1, "heads": 28, "kv": 4,
         "dim": 128, "page": 64, "rows": 1, "prefix": 14449, "suffix": 120, "window": 0, "sinks": 0},
        # a full server whose requests begin with the same instructions
        {"name": "shared_server", "op": "shared", "seqs": 64, "groups": 1, "heads": 32, "kv": 8,
         "dim": 128, "page": 64, "rows": 1, "prefix": 4096, "suffix": 2000, "window": 0, "sinks": 0},
        # several instructions of odd lengths, drafts of five tokens to be checked
        {"name": "shared_drafts", "op": "shared", "seqs": 24, "groups": 3, "heads": 32, "kv": 8,
         "dim": 64, "page": 16, "rows": 5, "prefix": 3501, "suffix": 300, "window": 0, "sinks": 0},
        # streaming under a window with a few first tokens that stay visible
        {"name": "shared_window", "op": "shared", "seqs": 32, "groups": 2, "heads": 32, "kv": 8,
         "dim": 128, "page": 32, "rows": 1, "prefix": 6001, "suffix": 400, "window": 2048, "sinks": 4},
        # the last ragged chunk of a prompt comes back for another step
        {"name": "read_chunk", "op": "read", "seqs": 1, "kv": 4, "dim": 128, "page": 64, "rows": 113,
         "length": 14449, "type": "fp32"},
        # whole sequences leave the card, or go to a model that wants them in 16 bits
        {"name": "read_sequences", "op": "read", "seqs": 6, "kv": 8, "dim": 128, "page": 32,
         "rows": 14449, "length": 14449, "type": "bf16"},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _turning(rng, dim):
    """How a case's heads turn: whole ones, or any even part of them."""
    return {"dims": rng.choice([dim, dim, dim // 2, 2 * rng.randint(1, dim // 2)]),
            "layout": rng.choice(["halves", "halves", "pairs"]), "norm": rng.random() < 0.5,
            "scaling": rng.choice(["plain", "linear", "base", "ramp", "smooth"]),
            "base": rng.choice([1e4, 5e5, 1e6])}


def draw(rng):
    op = rng.choice(["rotate", "append", "append", "shared", "shared", "shared", "read"])
    kv, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    if op == "rotate":
        return {"op": op, "rows": _log(rng, 1, 14000), "heads": rng.randint(1, 32), "dim": dim,
                "type": rng.choice(["bf16", "fp32"]), "to": rng.choice(["bf16", "bf16", "fp32"]),
                "start": _log(rng, 1, 200000), **_turning(rng, dim)}
    base = {"kv": kv, "dim": dim, "page": rng.choice([16, 32, 64, 128])}
    if op in ("append", "read"):
        seqs = _log(rng, 1, 64)
        length = _log(rng, 1, 14000 // seqs + 1)
        rows = min(rng.choice([1, _log(rng, 1, length), length]), length)
        case = {"op": op, "seqs": seqs, "rows": rows, "length": length,
                "type": rng.choice(["bf16", "fp32"]), **base}
        if op == "append":
            case |= {"heads": kv * rng.choice([1, 2, 4, 6, 7]), **_turning(rng, dim)}
            case["heads"] = min(case["heads"], 32)
        return case
    seqs = _log(rng, 2, 64)
    prefix, suffix = _log(rng, 16, 14000), _log(rng, 1, 2000)
    while seqs * (prefix + suffix) * kv * dim > 64 * 6096 * 8 * 128:
        prefix = prefix // 2 + 1
    rows = rng.choice([1, 1, 1, 2, 5])
    masks = {"window": 0, "sinks": 0}
    if rng.random() < 0.3:
        masks = {"window": _log(rng, 16, 8000), "sinks": rng.choice([0, 1, 4, 20])}
    return {"op": op, "seqs": seqs, "groups": rng.randint(1, min(6, seqs)),
            "heads": kv * rng.choice([1, 2, 4, 7] if kv < 8 else [1, 2, 4]), "rows": min(rows, suffix),
            "prefix": prefix, "suffix": suffix, **masks, **base}


# ------------------------------------------------------------------ inputs
def _spread(top, n, low=1):
    """n numbers: the largest first, the others over the whole range."""
    return [top] + [low + int((top - low) * ((i * 0.6180339887) % 1.0)) for i in range(1, n)]


def _prefixes(case):
    return _spread(case["prefix"], case["groups"], max(1, case["prefix"] // 3))


def _first(case):
    """The groups' first sequences, and the end: one and one, two, .. parts of the others."""
    n, g = case["seqs"], case["groups"]
    return [i + (n - g) * i * (i + 1) // (g * (g + 1)) for i in range(g + 1)]


def _group_of(case):
    first = _first(case)
    return [max(g for g in range(case["groups"]) if first[g] <= s) for s in range(case["seqs"])]


def _lengths(case):
    """Tokens of each sequence, new ones included."""
    if case["op"] != "shared":
        return _spread(case["length"], case["seqs"])
    more, prefix = _spread(case["suffix"], case["seqs"]), _prefixes(case)
    return [prefix[g] + n for g, n in zip(_group_of(case), more)]


def _rows(case):
    """New tokens of each sequence: the case's, as far as it has so many."""
    return [min(case["rows"], n) for n in _lengths(case)]


#: How far contexts are stretched: factor, tokens of the original context, and
#: between how many turns over it a pair goes from stretched to left alone.
SCALED = {"plain": (1.0, 0, 0.0, 0.0), "linear": (2.5, 0, 0.0, 0.0), "base": (3.0, 0, 0.0, 0.0),
          "ramp": (4.0, 4096, 1.0, 32.0), "smooth": (8.0, 8192, 1.0, 4.0)}


def _frequencies(case):
    """Radians a token of each pair, and the factor of what is turned."""
    n, base = case["dims"], case["base"]
    factor, original, low, high = SCALED[case["scaling"]]
    if case["scaling"] == "base" and n > 2:
        base *= factor ** (n / (n - 2))
    f = [base ** (-2 * i / n) for i in range(n // 2)]
    if case["scaling"] == "linear":
        f = [x / factor for x in f]
    if case["scaling"] == "smooth":  # by the turns that a pair makes over the original context
        kept = [min(1.0, max(0.0, (original * x / (2 * math.pi) - low) / (high - low))) for x in f]
        f = [x * k + x / factor * (1 - k) for x, k in zip(f, kept)]
    if case["scaling"] == "ramp":    # by the pair's number, between those that make so many turns
        def pair(turns):
            return n * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
        a, b = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), n - 1)
        b = b + 0.001 if a == b else b
        gone = [min(1.0, max(0.0, (i - a) / (b - a))) for i in range(n // 2)]
        f = [x * (1 - g) + x / factor * g for x, g in zip(f, gone)]
    return f, 0.1 * math.log(factor) + 1 if case["scaling"] == "ramp" else 1.0


def _exponent(top):
    """Exponent of the scale of blocks whose largest magnitude is `top`: the
    least with top <= 448 * 2^e."""
    m, e = torch.frexp(top)
    e = e - 9 + (m > 0.875).to(e.dtype)
    return torch.where(top > 0, e, torch.full_like(e, LOW)).clamp(LOW, HIGH)


def _power(e):
    """2^e in 32 bits, exactly, for whole e in -126 .. 127."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _codes(x, exponent):
    """e4m3 codes of x / 2^exponent, to nearest even."""
    x = (x * _power(-exponent)).clamp(-TOP, TOP)
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def _cache(case, pages, g):
    """A cache of one layer with something in every place: keys with a few
    strong channels, values of another size in every head."""
    kv, dim, page = case["kv"], case["dim"], case["page"]
    loud = 1 + 3 * (torch.rand(kv, 1, 1, dim, generator=g, device="cuda") < 0.05)
    size = torch.exp2(2 * torch.randn(kv, 1, 1, 1, generator=g, device="cuda"))
    st = {}
    for name, gain in (("k", loud), ("v", size)):
        one = torch.randn(pages, kv, page // BLOCK, BLOCK, dim, generator=g, device="cuda") * gain
        e = _exponent(one.abs().amax((3, 4)))
        c = _codes(one, e[..., None, None])
        if name == "v":
            c = c.reshape(pages, kv, page // 4, 4, dim).transpose(3, 4).contiguous()
        else:
            c = c.reshape(pages, kv, page, dim)
        st[name], st[name + "_scale"] = c[None], _power(e)[None]
    return st


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _pages(case):
    """The page table as lists of places in an order of pages, the number of
    pages, and (from, to, blocks) of the pages that a shared prefix ends in."""
    page, lengths = case["page"], _lengths(case)
    width = -(-max(lengths) // page) + 1
    if case["op"] != "shared":
        rows, at = [], 0
        for n in lengths:
            need = -(-n // page)
            rows.append(list(range(at, at + need)) + [-1] * (width - need))
            at += need
        return rows, at, []
    rows, at, copies, prefix, first = [], 0, [], _prefixes(case), _first(case)
    for s, (g, n) in enumerate(zip(_group_of(case), lengths)):
        whole, need = prefix[g] // page, -(-n // page)
        shared = rows[first[g]][:whole] if s > first[g] else list(range(at, at + whole))
        at += whole if s == first[g] else 0
        row = shared + list(range(at, at + need - whole))
        at += need - whole
        if prefix[g] % page and s > first[g]:  # each has a copy of a page in part
            copies.append((rows[first[g]][whole], row[whole], -(-(prefix[g] % page) // BLOCK)))
        rows.append(row + [-1] * (width - need))
    return rows, at, copies


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dim, kv, heads = case["dim"], case.get("kv", 0), case.get("heads", 0)
    if case["op"] == "rotate":
        rows, counts = case["rows"], [case["rows"]]
        st = {"positions": case["start"] + torch.arange(rows, device="cuda", dtype=torch.int32)}
    else:
        place, used, copies = _pages(case)
        pages = used + 3
        st = _cache(case, pages, g)
        order = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int32)
        place = torch.tensor(place, device="cuda")
        st["table"] = torch.where(place < 0, -1, order[place.clamp(min=0)]).int()
        if copies:
            src, dst = (order[torch.tensor([c[i] for c in copies], device="cuda")].long() for i in (0, 1))
            blocks = torch.arange(case["page"] // BLOCK, device="cuda")
            over = (blocks < torch.tensor([c[2] for c in copies], device="cuda")[:, None])[:, None, :]
            for name in ("k", "v"):
                c = st[name][0].reshape(pages, kv, len(blocks), BLOCK * dim)
                c[dst] = torch.where(over[..., None], c[src], c[dst])
                s = st[name + "_scale"][0]
                s[dst] = torch.where(over, s[src], s[dst])
        counts = _rows(case)
        rows = sum(counts)
        starts = [0]
        for r in counts:
            starts.append(starts[-1] + r)
        st |= {"row_start": _int32(starts), "kv_len": _int32(_lengths(case)), "total": rows}
    kind = torch.float32 if case.get("type") == "fp32" else torch.bfloat16
    if case["op"] == "read":
        st["k_rows"], st["v_rows"] = (torch.empty(rows, kv * dim, dtype=kind, device="cuda")
                                      for _ in range(2))
    else:
        # rows as a projection leaves them: q, k and v of a token side by side,
        # some channels louder than others
        loud = 1 + 3 * (torch.rand((heads + 2 * kv) * dim, generator=g, device="cuda") < 0.05)
        y = (torch.randn(rows, (heads + 2 * kv) * dim, generator=g, device="cuda") * loud).to(kind)
        st["q"], st["new_k"], st["new_v"] = (
            y[:, :heads * dim], y[:, heads * dim:(heads + kv) * dim], y[:, (heads + kv) * dim:])
        to = torch.float32 if case.get("to") == "fp32" else torch.bfloat16
        st["out"] = torch.empty(rows, heads * dim, dtype=to, device="cuda")
    if case.get("norm"):
        st["q_weight"], st["k_weight"] = (1 + 0.2 * torch.randn(dim, generator=g, device="cuda")
                                          for _ in range(2))
    if case["op"] == "shared":
        st["lse"] = torch.empty(rows, heads, dtype=torch.float32, device="cuda")
        st["first"], st["prefix_len"] = _int32(_first(case)), _int32(_prefixes(case))
    st["case"] = case
    if "dims" in case:
        f, st["gain"] = _frequencies(case)
        st["frequencies"] = torch.tensor(f, dtype=torch.float64, device="cuda")
    if own:
        _handles(st)
    return st


def _handles(st):
    """What a user's program keeps beside its tensors: the library's views of
    them, and the workspace."""
    from bit_weight_only_amd import nf4
    case = st["case"]
    st["nf4"] = nf4
    if "dims" in case:
        factor, original, low, high = SCALED[case["scaling"]]
        st["rotary"] = nf4.Rotary(
            case["dims"], getattr(nf4, "NF4_ROTARY_" + case["layout"].upper()), case["base"],
            scaling=getattr(nf4, "NF4_SCALING_" + case["scaling"].upper()), factor=factor,
            original=original, low=low, high=high, gain=st["gain"])
    if case["op"] == "rotate":
        return
    st["cache"] = c = nf4.KVCache(*st["k"].shape[:3], case["page"], case["dim"], k=st["k"],
                                  v=st["v"], k_scale=st["k_scale"], v_scale=st["v_scale"])
    st["batch"] = b = nf4.KVBatch(st["kv_len"], st["table"], row_start=st["row_start"],
                                  rows=st["total"], max_rows=max(_rows(case)),
                                  max_len=max(_lengths(case)))
    if case["op"] == "shared":
        first, rows = _first(case), _rows(case)
        st["groups"] = nf4.KVGroups(st["prefix_len"], st["first"], max_prefix=case["prefix"],
                                    max_rows=max(sum(rows[a:b]) for a, b in zip(first, first[1:])))
        n = nf4.nf4_kv_attention_shared_workspace_bytes(c, b, st["groups"], case["heads"],
                                                        case["window"], case["sinks"])
        st["ws"] = torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda")


# --------------------------------------------------------------- one pass
def run(st):
    return {"rotate": _rotate, "append": _append, "shared": _shared, "read": _read}[st["case"]["op"]](st)


def _type(st):
    return st["nf4"].NF4_KV_F32 if st["case"]["type"] == "fp32" else st["nf4"].NF4_KV_BF16


def _turned(st, x, at, weight):
    """Heads x [rows][heads][dim] (32 or 64 bits) at positions `at`: normed, then turned."""
    case = st["case"]
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.to(x.dtype)
    n = case["dims"]
    angle = (at.double()[:, None] * st["frequencies"])[:, None]
    c, s = (angle.cos() * st["gain"]).to(x.dtype), (angle.sin() * st["gain"]).to(x.dtype)
    if case["layout"] == "halves":
        a, b = x[..., :n // 2], x[..., n // 2:n]
        return torch.cat([a * c - b * s, a * s + b * c, x[..., n:]], -1)
    a, b = x[..., :n:2], x[..., 1:n:2]
    y = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    return torch.cat([y, x[..., n:]], -1)


def _rotate(st):
    case, q, out = st["case"], st["q"], st["out"]
    if own:
        nf4 = st["nf4"]
        nf4.nf4_rotate(st["rotary"], q, q.stride(0), _type(st), st["positions"], case["rows"],
                       case["heads"], case["dim"], st.get("q_weight"), EPS, out, out.stride(0),
                       nf4.NF4_KV_F32 if case["to"] == "fp32" else nf4.NF4_KV_BF16)
        return out
    x = q.float().reshape(case["rows"], -1, case["dim"])
    return _turned(st, x, st["positions"], st.get("q_weight")).reshape(case["rows"], -1).to(out.dtype)


def _whole(st):
    """The cache: codes as the e4m3 values they are, and the scales."""
    return {"k": st["k"].view(torch.float8_e4m3fn), "v": st["v"].view(torch.float8_e4m3fn),
            "k_scale": st["k_scale"], "v_scale": st["v_scale"]}


def _positions(st):
    """Position of each row, and its sequence."""
    counts = (st["row_start"][1:] - st["row_start"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(len(counts), device="cuda"), counts, output_size=st["total"])
    row = torch.arange(st["total"], device="cuda")
    return row - st["row_start"][1:][seq] + st["kv_len"][seq], seq


def _append(st):
    case = st["case"]
    if own:
        q, k, v = st["q"], st["new_k"], st["new_v"]
        st["nf4"].nf4_kv_append_rotated(
            st["cache"], 0, st["batch"], st["rotary"], q, q.stride(0), case["heads"],
            st.get("q_weight"), k, k.stride(0), st.get("k_weight"), v, v.stride(0), _type(st), EPS,
            st["out"])
        return {"q": st["out"], **_whole(st)}
    kv, dim, page, total = case["kv"], case["dim"], case["page"], st["total"]
    at, _ = _positions(st)
    q = _turned(st, st["q"].float().reshape(total, -1, dim), at, st.get("q_weight"))
    fresh = {"k": _turned(st, st["new_k"].float().reshape(total, kv, dim), at, st.get("k_weight")),
             "v": st["new_v"].float().reshape(total, kv, dim)}
    pages = st["k"].shape[1]
    kv_len, count = st["kv_len"].long(), (st["row_start"][1:] - st["row_start"][:-1]).long()
    begin = kv_len - count
    most = -(-max(_rows(case)) // BLOCK) + 1  # blocks that a sequence's new tokens can touch
    block = begin[:, None] // BLOCK + torch.arange(most, device="cuda")
    seq, which = torch.nonzero(block * BLOCK < kv_len[:, None], as_tuple=True)
    block = block[seq, which]
    token = block[:, None] * BLOCK + torch.arange(BLOCK, device="cuda")
    old = token < begin[seq, None]
    new = ~old & (token < kv_len[seq, None])
    row = (st["row_start"][seq, None] + token - begin[seq, None]).clamp(0, total - 1)
    place = st["table"][seq, block * BLOCK // page].long() * (page // BLOCK) + block % (page // BLOCK)
    for name in ("k", "v"):
        codes = st[name][0].reshape(pages, kv, page // BLOCK, -1).transpose(1, 2)
        scales = st[name + "_scale"][0].transpose(1, 2)
        p, b = place // (page // BLOCK), place % (page // BLOCK)
        had = codes[p, b]                                              # [blocks][kv][bytes]
        if name == "k":
            had = had.reshape(-1, kv, BLOCK, dim)
        else:
            had = had.reshape(-1, kv, 4, dim, 4).transpose(3, 4).reshape(-1, kv, BLOCK, dim)
        was = scales[p, b]
        x = fresh[name][row].transpose(1, 2)
        is_new, is_old = new[:, None, :, None], old[:, None, :, None]
        e = _exponent(torch.where(is_new, x.abs(), 0.0).amax((2, 3)))
        _, e_was = torch.frexp(was)
        e = torch.where(old.any(1)[:, None], torch.maximum(e, e_was - 1), e)
        kept = had.view(torch.float8_e4m3fn).float() * was[:, :, None, None]
        out = _codes(torch.where(is_new, x, kept), e[:, :, None, None])
        out = torch.where(is_new | is_old, out, had)
        if name == "v":
            out = out.reshape(-1, kv, 4, 4, dim).transpose(3, 4)
        codes[p, b] = out.reshape(-1, kv, BLOCK * dim)
        scales[p, b] = _power(e)
    return {"q": q.reshape(total, -1).to(torch.bfloat16), **_whole(st)}


def _dense(st, name):
    """Codes times scales of the whole cache, [pages][kv][page tokens][dim] in 32 bits."""
    case = st["case"]
    kv, dim, page = case["kv"], case["dim"], case["page"]
    x = st[name][0].view(torch.float8_e4m3fn).float()
    x = x.transpose(3, 4) if name == "v" else x
    x = x.reshape(-1, kv, page // BLOCK, BLOCK, dim) * st[name + "_scale"][0][..., None, None]
    return x.reshape(-1, kv, page, dim)


def _shared(st):
    case = st["case"]
    heads, kv, dim, page = case["heads"], case["kv"], case["dim"], case["page"]
    if own:
        q, ws = st["q"], st["ws"]
        st["nf4"].nf4_kv_attention_shared(
            st["cache"], 0, st["batch"], st["groups"], q, q.stride(0), heads, dim ** -0.5,
            case["window"], case["sinks"], st["out"], st["lse"], ws, ws.numel())
        return {"out": st["out"], "lse": st["lse"]}
    table = st["table"].long().clamp(min=0)
    seqs, width = table.shape
    kv_len, count = st["kv_len"].long(), (st["row_start"][1:] - st["row_start"][:-1]).long()
    k, v = (_dense(st, name)[table].transpose(1, 2).reshape(seqs, kv, width * page, dim)
            for name in ("k", "v"))
    most = max(_rows(case))
    r = torch.arange(most, device="cuda")
    row = (st["row_start"][:-1, None] + r).clamp(max=st["total"] - 1)
    q = st["q"].float().reshape(-1, kv, heads // kv, dim)[row]          # [seqs][rows][kv][group][dim]
    q = q.permute(0, 2, 3, 1, 4).reshape(seqs, kv, -1, dim)
    s = (q @ k.transpose(2, 3)) * dim ** -0.5
    at = (kv_len - count)[:, None, None] + r[:, None]                   # position of each row
    key = torch.arange(width * page, device="cuda")
    seen = key <= at
    if case["window"]:
        seen &= (key > at - case["window"]) | (key < case["sinks"])
    s = s.reshape(seqs, kv, heads // kv, most, -1).masked_fill_(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.reshape(seqs, kv, -1, width * page) @ v).reshape(*total.shape[:-1], dim) / total
    lse = (top + total.log())[..., 0]
    mine = torch.nonzero(r < count[:, None], as_tuple=True)             # rows in order
    o = o.permute(0, 3, 1, 2, 4)[mine].reshape(-1, heads * dim)
    return {"out": o.to(torch.bfloat16), "lse": lse.permute(0, 3, 1, 2)[mine].reshape(-1, heads)}


def _read(st):
    k, v = st["k_rows"], st["v_rows"]
    if own:
        st["nf4"].nf4_kv_read(st["cache"], 0, st["batch"], k, k.stride(0), v, v.stride(0), _type(st))
        return {"k": k, "v": v}
    page = st["case"]["page"]
    at, seq = _positions(st)
    p = st["table"].long()[seq, at // page]
    return {n: _dense(st, n)[p, :, at % page].reshape(st["total"], -1).to(k.dtype) for n in ("k", "v")}


# ------------------------------------------------------------ what it costs
def _span(first, last, low, high, window, sinks):
    """(pairs, keys): keys in low .. high - 1 that the rows at positions first
    .. last see, summed over the rows, and those that any of them sees."""
    pairs, spans = 0, []
    for at in range(first, last + 1):
        a, b = max(low, at - window + 1 if window else 0), min(high, at + 1)
        s = max(0, min(sinks, high, a) - low) if window else 0
        pairs += max(0, b - a) + s
        spans.append((a, b))
    a, b = min(x for x, _ in spans), max(x for _, x in spans)
    s = max(0, min(sinks, high, a) - low) if window else 0
    return pairs, max(0, b - a) + s


def work(case):
    kv, dim, heads, size = case.get("kv", 0), case["dim"], case.get("heads", 0), 4 if case.get("type") == "fp32" else 2
    if case["op"] == "rotate":
        values = case["rows"] * heads * dim
        return {"bytes": values * (size + (4 if case["to"] == "fp32" else 2)),
                "flops": values * (10 if case["norm"] else 6)}
    rows = sum(_rows(case))
    codes = 2 * rows * kv * (dim + 4 / BLOCK)
    if case["op"] == "append":
        return {"bytes": rows * (heads * dim * (size + 2) + 2 * kv * dim * size) + codes,
                "flops": rows * (heads + kv) * dim * 8}
    if case["op"] == "read":
        return {"bytes": codes + 2 * rows * kv * dim * size, "flops": 2 * rows * kv * dim}
    pairs = keys = 0
    lengths, counts, prefix, first = _lengths(case), _rows(case), _prefixes(case), _first(case)
    for g, n in enumerate(prefix):  # a prefix is read once for all of its sequences
        seen = []
        for s in range(first[g], first[g + 1]):
            at = lengths[s] - counts[s], lengths[s] - 1, case["window"], case["sinks"]
            p, k = _span(*at[:2], n, lengths[s], *at[2:])
            q, shared = _span(*at[:2], 0, n, *at[2:])
            pairs, keys = pairs + p + q, keys + k
            seen.append(shared)
        keys += max(seen, default=0)
    return {"bytes": 2 * keys * kv * (dim + 4 / BLOCK) + rows * heads * (4 * dim + 4),
            "flops": 4 * pairs * heads * dim}


# ------------------------------------------------------- the definition, 64 bits
def _values():
    """The 256 values of e4m3: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    x = [(1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7) if c > 7 else c / 8 * 2.0 ** -6 for c in range(127)]
    x = torch.tensor(x + [math.nan], dtype=torch.float64, device="cuda")
    return torch.cat([x, -x])


def _power64(e):
    """2^e in 64 bits, exactly, for whole e."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def exact(case, seed):
    st = prepare(case, seed)
    return {"rotate": _exact_rotate, "append": _exact_append, "shared": _exact_shared,
            "read": _exact_read}[case["op"]](st, case)


def _exact_turn(st, case, x, at, weight):
    """The definition as complex numbers: a pair is a + ib, turned by e^(i angle)."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.double()
    n = case["dims"]
    where = torch.arange(n, device="cuda")
    a, b = (where[:n // 2], where[n // 2:]) if case["layout"] == "halves" else (where[::2], where[1::2])
    f, gain = _frequencies(case)
    angle = at.double()[:, None, None] * torch.tensor(f, dtype=torch.float64, device="cuda")
    z = torch.complex(x[..., a], x[..., b]) * torch.polar(torch.full_like(angle, gain), angle)
    y = x.clone()
    y[..., a], y[..., b] = z.real, z.imag
    return y


def _exact_rotate(st, case):
    x = st["q"].reshape(case["rows"], -1, case["dim"])
    return _exact_turn(st, case, x, st["positions"], st.get("q_weight")).reshape(case["rows"], -1)


def _round_e4m3(x):
    """The nearest e4m3 value, ties to the even mantissa."""
    _, e = torch.frexp(x)
    step = _power64((e - 1).clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-TOP, TOP)


def _exact_append(st, case):
    kv, dim, page, heads = case["kv"], case["dim"], case["page"], case["heads"]
    value = _values()
    out = {"q": torch.empty(st["total"], heads * dim, dtype=torch.float64, device="cuda")}
    for name in ("q", "k", "v"):
        if name != "q":
            c = st[name][0]
            if name == "v":
                c = c.transpose(3, 4).reshape(-1, kv, page, dim)
            codes, scale = value[c.long()], st[name + "_scale"][0].double()
        for s in range(case["seqs"]):
            n, r0, r1 = int(st["kv_len"][s]), int(st["row_start"][s]), int(st["row_start"][s + 1])
            begin = n - (r1 - r0)
            new = st[name if name == "q" else "new_" + name][r0:r1].double().reshape(r1 - r0, -1, dim)
            if name != "v":
                at = torch.arange(begin, n, device="cuda")
                new = _exact_turn(st, case, new, at, st.get(name + "_weight"))
            if name == "q":
                out["q"][r0:r1] = new.reshape(r1 - r0, -1)
                continue
            lo, hi = begin // BLOCK, -(-n // BLOCK)
            t = torch.arange(lo * BLOCK, hi * BLOCK, device="cuda")
            at = st["table"][s].long()[t // page]
            had, was = codes[at, :, t % page], scale[at, :, t % page // BLOCK]  # [tokens][kv][dim], [tokens][kv]
            x = had * was[..., None]
            x[begin - lo * BLOCK:n - lo * BLOCK] = new
            fresh = ((t >= begin) & (t < n))[:, None, None]
            top = torch.where(fresh, x.abs(), 0.0).reshape(-1, BLOCK, kv, dim).amax((1, 3))
            scales = _power64(torch.arange(LOW, HIGH + 1, device="cuda"))
            least = torch.searchsorted(TOP * scales, top.contiguous())  # the least that holds it
            e = scales[least.clamp(max=HIGH - LOW)]
            if begin % BLOCK:
                e[0] = torch.maximum(e[0], was[0])
            e = e.repeat_interleave(BLOCK, 0)
            y = _round_e4m3(x / e[..., None])
            codes[at, :, t % page] = torch.where((t < n)[:, None, None], y, had)
            scale[at, :, t % page // BLOCK] = e
        if name == "v":
            codes = codes.reshape(-1, kv, page // 4, 4, dim).transpose(3, 4)
        if name != "q":
            out[name], out[name + "_scale"] = codes.reshape(st[name].shape), scale[None]
    return out


def _exact_rows(st, case, s, h, t):
    """Keys and values of head h at tokens t of sequence s."""
    value, page = _values(), case["page"]
    at = st["table"][s].long()[t // page]
    k = value[st["k"][0, at, h, t % page].long()]
    v = value[st["v"][0, at, h, t % page // 4, :, t % 4].long()]
    return (k * st["k_scale"][0, at, h, t % page // BLOCK].double()[:, None],
            v * st["v_scale"][0, at, h, t % page // BLOCK].double()[:, None])


def _exact_shared(st, case):
    kv, dim, heads = case["kv"], case["dim"], case["heads"]
    group = heads // kv
    out = torch.zeros(st["total"], heads, dim, dtype=torch.float64, device="cuda")
    lse = torch.full((st["total"], heads), -math.inf, dtype=torch.float64, device="cuda")
    q = st["q"].double().reshape(-1, heads, dim)
    for s, (n, r) in enumerate(zip(_lengths(case), _rows(case))):
        r0 = sum(_rows(case)[:s])
        t = torch.arange(n, device="cuda")
        at = n - r + torch.arange(r, device="cuda")
        hidden = t > at[:, None]
        if case["window"]:
            hidden |= (t <= at[:, None] - case["window"]) & (t >= case["sinks"])
        for h in range(kv):
            k, v = _exact_rows(st, case, s, h, t)
            x = (q[r0:r0 + r, h * group:(h + 1) * group].reshape(-1, dim) @ k.T) / math.sqrt(dim)
            x = x.reshape(r, group, n).masked_fill_(hidden[:, None], -math.inf)
            z = torch.logsumexp(x, -1)
            out[r0:r0 + r, h * group:(h + 1) * group] = \
                (x.sub_(z[..., None]).exp_().reshape(-1, n) @ v).reshape(r, group, dim)
            lse[r0:r0 + r, h * group:(h + 1) * group] = z
    return {"out": out.reshape(-1, heads * dim), "lse": lse}


def _exact_read(st, case):
    kv, dim = case["kv"], case["dim"]
    out = {n: torch.empty(st["total"], kv, dim, dtype=torch.float64, device="cuda") for n in ("k", "v")}
    r0 = 0
    for s, (n, r) in enumerate(zip(_lengths(case), _rows(case))):
        t = torch.arange(n - r, n, device="cuda")
        for h in range(kv):
            out["k"][r0:r0 + r, h], out["v"][r0:r0 + r, h] = _exact_rows(st, case, s, h, t)
        r0 += r
    return {n: x.reshape(st["total"], -1) for n, x in out.items()}
