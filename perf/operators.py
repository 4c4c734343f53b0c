"""The key-value cache operators in their plain form, the cases that they are
measured at, and the same calls through the library.

The cache holds keys and values in 8 bits (e4m3: 4 exponent bits, 3 mantissa
bits, largest value 448) with one power-of-two scale for every block of 16
tokens of a head.  It lies in pages of `page` tokens that any sequence may own:

    k        uint8 [layers][pages][kv heads][page tokens][head dim]
    v        uint8 [layers][pages][kv heads][page tokens / 4][head dim][4]
    scales   fp32  [layers][pages][kv heads][page tokens / 16], one array each

Operators: `append` quantizes new tokens into the pages; `attention` reads
them (prompts and single tokens, causal, optionally with a sliding window and
a few first tokens that stay visible); `branch` releases, forks and extends
sequences; `compact` moves the live pages to the front of the pool.
"""
import math

import torch

own = False

BLOCK = 16          # tokens under one scale
TOP = 448.0         # largest e4m3 value
LOW, HIGH = -40, 100  # exponents that a scale may have


def listed():
    return [
        # one decoded token of one sequence goes into the cache: a latency
        {"name": "append_token", "op": "append", "seqs": 1, "kv": 4, "dim": 128, "page": 64,
         "rows": 1, "length": 1025, "type": "bf16"},
        # the prompt of a 32-minute recording, straight from the fp32 projection
        {"name": "append_prompt", "op": "append", "seqs": 1, "kv": 8, "dim": 128, "page": 64,
         "rows": 14449, "length": 14449, "type": "fp32"},
        # one token of a short conversation, 28 query heads over 4
        {"name": "decode_short", "op": "attention", "seqs": 1, "heads": 28, "kv": 4, "dim": 128,
         "page": 16, "rows": 1, "length": 113, "window": 0, "sinks": 0},
        # two slots decoding at the end of a long recording
        {"name": "decode_long", "op": "attention", "seqs": 2, "heads": 28, "kv": 4, "dim": 128,
         "page": 64, "rows": 1, "length": 14449, "window": 0, "sinks": 0},
        # a full server: 64 sequences of every length, 32 query heads over 8
        {"name": "decode_batch", "op": "attention", "seqs": 64, "heads": 32, "kv": 8, "dim": 128,
         "page": 64, "rows": 1, "length": 16384, "window": 0, "sinks": 0},
        # an ordinary prompt in one chunk
        {"name": "prefill_1024", "op": "attention", "seqs": 1, "heads": 28, "kv": 4, "dim": 128,
         "page": 64, "rows": 1024, "length": 1024, "window": 0, "sinks": 0},
        # the last, ragged chunk of the long recording's prompt over all before it
        {"name": "prefill_tail", "op": "attention", "seqs": 1, "heads": 28, "kv": 4, "dim": 128,
         "page": 64, "rows": 113, "length": 14449, "window": 0, "sinks": 0},
        # that prompt as one sequence
        {"name": "prefill_recording", "op": "attention", "seqs": 1, "heads": 28, "kv": 4,
         "dim": 128, "page": 64, "rows": 14449, "length": 14449, "window": 0, "sinks": 0},
        # streaming decode: an odd window and four first tokens, small pages, heads of 64
        {"name": "window_decode", "op": "attention", "seqs": 48, "heads": 32, "kv": 8, "dim": 64,
         "page": 16, "rows": 1, "length": 20001, "window": 1500, "sinks": 4},
        # three prompts of different lengths under a window
        {"name": "window_prefill", "op": "attention", "seqs": 3, "heads": 32, "kv": 8, "dim": 128,
         "page": 32, "rows": 6001, "length": 6001, "window": 1024, "sinks": 4},
        # beams: every parent continues in several children with room to go on
        {"name": "pages_branch", "op": "branch", "layers": 28, "kv": 4, "dim": 128, "page": 64,
         "pages": 512, "parents": 8, "children": 32, "length": 1000, "add": 70},
        # a pool after long use: a third of its pages free, all over it
        {"name": "pages_compact", "op": "compact", "layers": 4, "kv": 8, "dim": 128, "page": 64,
         "pages": 2000, "seqs": 96, "shared": 4, "free": 0.33},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "prefill", "prefill", "branch", "compact"])
    kv = rng.choice([1, 2, 4, 8])
    base = {"kv": kv, "dim": rng.choice([64, 128]), "page": rng.choice([16, 32, 64, 128])}
    if op == "append":
        seqs = _log(rng, 1, 64)
        length = _log(rng, 1, 14000 // seqs + 1)
        rows = rng.choice([1, _log(rng, 1, length), length])
        return {"op": "append", "seqs": seqs, "rows": min(rows, length), "length": length,
                "type": rng.choice(["bf16", "fp32"]), **base}
    masks = {"window": 0, "sinks": 0}
    if op == "decode":
        seqs, heads = _log(rng, 1, 64), kv * rng.choice([1, 2, 4, 6, 7, 8])
        length = _log(rng, 1, 16000)
        if rng.random() < 0.4:
            masks = {"window": _log(rng, 1, 4000), "sinks": rng.choice([0, 1, 4, 20])}
        return {"op": "attention", "seqs": seqs, "heads": heads, "rows": rng.choice([1, 1, 1, 2, 5]),
                "length": length, **masks, **base}
    if op == "prefill":
        seqs, heads = rng.choice([1, 1, 2, 5]), kv * rng.choice([1, 2, 4, 7, 8])
        rows = _log(rng, 17, 8000 // seqs)
        length = rows + rng.choice([0, 0, _log(rng, 1, 6000 // seqs)])
        if rng.random() < 0.4:
            masks = {"window": _log(rng, 16, 4000), "sinks": rng.choice([0, 1, 4, 20])}
        heads = heads if heads * rows < 60000 else kv
        return {"op": "attention", "seqs": seqs, "heads": heads, "rows": rows, "length": length,
                **masks, **base}
    if op == "branch":
        parents = _log(rng, 1, 8)
        length = _log(rng, 1, 3000)
        children = parents * rng.randint(1, 4)
        add = _log(rng, 1, 200)
        pages = parents * (length // base["page"] + 1) + children * (add // base["page"] + 3)
        return {"op": "branch", "layers": rng.randint(1, 28), "pages": pages + rng.randint(0, 40),
                "parents": parents, "children": children, "length": length, "add": add, **base}
    seqs = _log(rng, 2, 96)
    return {"op": "compact", "layers": rng.randint(1, 4), "pages": _log(rng, 8 * seqs, 2000 + 8 * seqs),
            "seqs": seqs, "shared": rng.randint(0, 4), "free": round(rng.uniform(0.05, 0.8), 3), **base}


# ------------------------------------------------------------------ inputs
def _lengths(case):
    """Tokens of each sequence, new ones included: the longest first, the
    others spread over the whole range."""
    n, top = case.get("seqs", case.get("parents", 1)), case["length"]
    return [top] + [1 + int((top - 1) * ((i * 0.6180339887) % 1.0)) for i in range(1, n)]


def _rows(case):
    """New tokens of each sequence: the case's, as far as it has so many."""
    return [min(case["rows"], n) for n in _lengths(case)]


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


def _cache(case, layers, pages, g):
    """A cache with something in every place: keys with a few strong
    channels, values of another size in every head."""
    kv, dim, page = case["kv"], case["dim"], case["page"]
    loud = 1 + 3 * (torch.rand(kv, 1, 1, dim, generator=g, device="cuda") < 0.05)
    size = torch.exp2(2 * torch.randn(kv, 1, 1, 1, generator=g, device="cuda"))
    st = {}
    for name, gain in (("k", loud), ("v", size)):
        one = torch.randn(pages, kv, page // BLOCK, BLOCK, dim, generator=g, device="cuda") * gain
        e = _exponent(one.abs().amax((3, 4)))
        c = _codes(one, e[..., None, None])
        if name == "v":
            c = c.reshape(pages, kv, page // 4, 4, dim).transpose(3, 4)
            c = c.reshape(pages, kv, page // 4, dim, 4)
        else:
            c = c.reshape(pages, kv, page, dim)
        s = _power(e)
        # layers differ by where their pages lie
        st[name] = torch.stack([c.roll(i, 0) for i in range(layers)]).contiguous()
        st[name + "_scale"] = torch.stack([s.roll(i, 0) for i in range(layers)]).contiguous()
    return st


def _table(lengths, page, pages, width, g):
    """A page table whose sequences own pages all over the pool, -1 past
    their ends, and the reference counts of the pages."""
    need = [-(-n // page) for n in lengths]
    order = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int32)
    table = torch.full((len(lengths), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[order[:at].long()] = 1
    return table, refs


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, page = case["op"], case["page"]
    if op == "compact":
        return _prepare_compact(case, g)
    lengths = _lengths(case)
    if op == "branch":
        st = _cache(case, case["layers"], case["pages"], g)
        n, c = case["parents"], case["children"]
        width = (case["length"] + case["add"]) // page + 2
        table, refs = _table(lengths, page, case["pages"], width, g)
        table = torch.cat([table, table.new_full((c, width), -1)])
        st |= {"table": table, "refs": refs, "len": _int32(lengths + [0] * c),
               "missing": _int32([0]), "child": _int32(list(range(n, n + c))),
               "parent": torch.randint(0, n, (c,), generator=g, device="cuda", dtype=torch.int32),
               "add": _int32([0] * n + [case["add"]] * c)}
    else:
        need = sum(-(-n // page) for n in lengths)
        st = _cache(case, 1, need + 3, g)
        width = -(-max(lengths) // page) + 1
        st["table"], _ = _table(lengths, page, need + 3, width, g)
        rows = _rows(case)
        starts = [0]
        for r in rows:
            starts.append(starts[-1] + r)
        st |= {"row_start": _int32(starts), "kv_len": _int32(lengths), "total": starts[-1]}
        kv, dim = case["kv"], case["dim"]
        kind = torch.float32 if case.get("type") == "fp32" else torch.bfloat16
        # rows as a projection leaves them: q, k and v of a token side by side
        heads = case.get("heads", 0)
        y = torch.randn(starts[-1], (heads + 2 * kv) * dim, generator=g, device="cuda").to(kind)
        st["q"], st["new_k"], st["new_v"] = (
            y[:, :heads * dim], y[:, heads * dim:(heads + kv) * dim], y[:, (heads + kv) * dim:])
        if op == "attention":
            st["out"] = torch.empty(starts[-1], heads * dim, dtype=torch.bfloat16, device="cuda")
            st["lse"] = torch.empty(starts[-1], heads, dtype=torch.float32, device="cuda")
    st["case"] = case
    if own:
        _handles(st)
    return st


def _prepare_compact(case, g):
    pages, seqs = case["pages"], case["seqs"]
    st = _cache(case, case["layers"], pages, g)
    live = pages - int(pages * case["free"])
    shared = min(case["shared"], live - 1)
    each = max(1, (live - shared) // seqs)
    order = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int32)
    first = order[:shared].expand(seqs, shared)  # a prefix that all sequences share
    rest = order[shared:shared + seqs * each].reshape(seqs, each)
    table = torch.full((seqs, shared + each + 3), -1, dtype=torch.int32, device="cuda")
    table[:, :shared + each] = torch.cat([first, rest], 1)
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[order[:shared].long()] = seqs
    refs[rest.reshape(-1).long()] = 1
    st |= {"table": table, "refs": refs, "refs_out": torch.empty_like(refs),
           "table_out": torch.empty_like(table), "case": case}
    if own:
        _handles(st)
    return st


def _handles(st):
    """What a user's program keeps beside its tensors: the library's views of
    them, and the workspace."""
    from bit_weight_only_amd import nf4
    case = st["case"]
    st["nf4"] = nf4
    st["cache"] = c = nf4.KVCache(*st["k"].shape[:3], case["page"], case["dim"], k=st["k"],
                                  v=st["v"], k_scale=st["k_scale"], v_scale=st["v_scale"])
    if case["op"] in ("append", "attention"):
        st["batch"] = b = nf4.KVBatch(st["kv_len"], st["table"], row_start=st["row_start"],
                                      rows=st["total"], max_rows=max(_rows(case)),
                                      max_len=case["length"])
        if case["op"] == "attention":
            n = nf4.nf4_kv_attention_workspace_bytes(c, b, case["heads"], case["window"],
                                                     case["sinks"])
            st["ws"] = torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda")
    else:
        length = st.get("len")
        st["pool"] = nf4.KVPool(st["refs"], st["table"],
                                torch.zeros(len(st["table"]), dtype=torch.int32, device="cuda")
                                if length is None else length, st.get("missing"))
        if case["op"] == "compact":
            n = nf4.nf4_kv_compact_workspace_bytes(c)
            st["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")


# --------------------------------------------------------------- one pass
def run(st):
    return {"append": _append, "attention": _attention, "branch": _branch,
            "compact": _compact}[st["case"]["op"]](st)


def _whole(st):
    """The cache: codes as the e4m3 values they are, and the scales."""
    return {"k": st["k"].view(torch.float8_e4m3fn), "v": st["v"].view(torch.float8_e4m3fn),
            "k_scale": st["k_scale"], "v_scale": st["v_scale"]}


def _append(st):
    case = st["case"]
    if own:
        nf4, k, v = st["nf4"], st["new_k"], st["new_v"]
        kind = nf4.NF4_KV_F32 if case["type"] == "fp32" else nf4.NF4_KV_BF16
        nf4.nf4_kv_append(st["cache"], 0, st["batch"], k, k.stride(0), v, v.stride(0), kind)
        return _whole(st)
    kv, dim, page = case["kv"], case["dim"], case["page"]
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
    row = (st["row_start"][seq, None] + token - begin[seq, None]).clamp(0, st["total"] - 1)
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
        x = st["new_" + name].float().reshape(-1, kv, dim)[row].transpose(1, 2)
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
    return _whole(st)


def _attention(st):
    case = st["case"]
    heads, kv, dim, page = case["heads"], case["kv"], case["dim"], case["page"]
    if own:
        q, ws = st["q"], st["ws"]
        st["nf4"].nf4_kv_attention(st["cache"], 0, st["batch"], q, q.stride(0), heads, dim ** -0.5,
                                   case["window"], case["sinks"], st["out"], st["lse"], ws,
                                   ws.numel())
        return {"out": st["out"], "lse": st["lse"]}
    table = st["table"].long().clamp(min=0)
    seqs, width = table.shape
    kv_len, count = st["kv_len"].long(), (st["row_start"][1:] - st["row_start"][:-1]).long()
    k = st["k"][0].view(torch.float8_e4m3fn).float()
    k = k.reshape(-1, kv, page // BLOCK, BLOCK, dim) * st["k_scale"][0][..., None, None]
    v = st["v"][0].view(torch.float8_e4m3fn).float().transpose(3, 4)
    v = v.reshape(-1, kv, page // BLOCK, BLOCK, dim) * st["v_scale"][0][..., None, None]
    k, v = (x.reshape(-1, kv, page, dim)[table].transpose(1, 2).reshape(seqs, kv, width * page, dim)
            for x in (k, v))
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


def _pool(st):
    return {"table": st["table"], "refs": st["refs"], "len": st["len"], "missing": st["missing"]}


def _branch(st):
    """The children of the last step go, the parents' next ones come, and each
    gets room for its next tokens."""
    case, child, parent = st["case"], st["child"], st["parent"]
    if own:
        nf4, c, pool = st["nf4"], st["cache"], st["pool"]
        nf4.nf4_kv_release(c, pool, child, case["children"])
        nf4.nf4_kv_fork(c, pool, parent, child, case["children"])
        nf4.nf4_kv_reserve(c, pool, st["add"])
        return {**_pool(st), **_whole(st)}
    page, table, refs, length = case["page"], st["table"], st["refs"], st["len"]
    child, parent = child.long(), parent.long()
    gone = table[child]
    refs.index_add_(0, gone.clamp(min=0).reshape(-1), -(gone >= 0).reshape(-1).int())
    table[child] = -1
    # whole pages are shared, a page in part is copied
    n = length[parent]
    entry = torch.arange(table.shape[1], device="cuda")
    keep = torch.where(entry < (n // page)[:, None], table[parent], -1)
    refs.index_add_(0, keep.clamp(min=0).reshape(-1), (keep >= 0).reshape(-1).int())
    table[child] = keep
    part = torch.nonzero(n % page)[:, 0]
    new = torch.nonzero(refs == 0)[:len(part), 0]
    at = (n[part] // page).long()
    old = table[parent[part], at].long()
    table[child[part], at] = new.int()
    refs[new] = 1
    for name in ("k", "v", "k_scale", "v_scale"):
        st[name][:, new] = st[name][:, old]
    length[child] = n
    # room for the next tokens, lowest free pages in order of rows
    had, length[:] = -(-length // page), length + st["add"]
    want = -(-length // page) - had
    seq = torch.repeat_interleave(torch.arange(len(want), device="cuda"), want)
    rank = torch.arange(len(seq), device="cuda") - (want.cumsum(0) - want)[seq]
    new = torch.nonzero(refs == 0)[:len(seq), 0]
    table[seq, had[seq].long() + rank] = new.int()
    refs[new] = 1
    st["missing"].fill_(0)
    return {**_pool(st), **_whole(st)}


def _compact(st):
    if own:
        nf4, ws = st["nf4"], st["ws"]
        nf4.nf4_kv_compact(st["cache"], st["pool"], st["refs_out"], st["table_out"], ws, ws.numel())
        return {"refs": st["refs_out"], "table": st["table_out"], **_whole(st)}
    refs, table = st["refs"], st["table"]
    page = torch.arange(len(refs), device="cuda")
    live = refs > 0
    n = live.sum()
    src, dst = (torch.nonzero(x)[:, 0] for x in (live & (page >= n), ~live & (page < n)))
    for name in ("k", "v", "k_scale", "v_scale"):
        st[name][:, dst] = st[name][:, src]
    to = page.clone()
    to[src] = dst
    st["table_out"].copy_(torch.where(table >= 0, to[table.long().clamp(min=0)], -1))
    st["refs_out"].zero_().index_add_(0, to[live], refs[live])
    return {"refs": st["refs_out"], "table": st["table_out"], **_whole(st)}


# ------------------------------------------------------------ what it costs
def _page_bytes(case):
    """Codes and scales of one page of one layer, keys and values."""
    return 2 * case["kv"] * case["page"] * (case["dim"] + 4 / BLOCK)


def _seen(first, last, window, sinks):
    """(pairs, keys): keys seen by the rows at positions first .. last,
    summed over the rows, and the keys that any of them sees."""
    pairs = 0
    if not window:
        pairs = (last + 1) * (last + 2) // 2 - first * (first + 1) // 2
        return pairs, last + 1
    for at in range(first, last + 1):
        inside = min(at + 1, window)
        pairs += inside + min(sinks, at + 1 - inside)
    low = max(0, first - window + 1)
    return pairs, last + 1 - low + min(sinks, low)


def work(case):
    kv, dim = case["kv"], case["dim"]
    if case["op"] == "append":
        values = 2 * sum(_rows(case)) * kv * dim
        return {"bytes": values * (5 if case["type"] == "fp32" else 3) + values / dim / BLOCK * 4,
                "flops": 2 * values}
    if case["op"] == "attention":
        seen = [_seen(n - r, n - 1, case["window"], case["sinks"])
                for n, r in zip(_lengths(case), _rows(case))]
        pairs, keys = (sum(x) for x in zip(*seen))
        rows = sum(_rows(case)) * case["heads"]
        return {"bytes": 2 * keys * kv * (dim + 4 / BLOCK) + rows * (4 * dim + 4),
                "flops": 4 * pairs * case["heads"] * dim}
    if case["op"] == "branch":
        part = case["children"] * (case["length"] % case["page"] > 0)
        return {"bytes": 2 * part * case["layers"] * _page_bytes(case) + 8 * case["pages"], "flops": 0}
    live = case["pages"] - int(case["pages"] * case["free"])
    moved = live * case["free"]  # live pages that lie past the live ones' number, on average
    return {"bytes": 2 * moved * case["layers"] * _page_bytes(case) + 8 * case["pages"], "flops": 0}


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
    if case["op"] not in ("append", "attention"):
        return None
    st = prepare(case, seed)
    return (_exact_append if case["op"] == "append" else _exact_attention)(st, case)


def _round_e4m3(x):
    """The nearest e4m3 value, ties to the even mantissa."""
    _, e = torch.frexp(x)
    step = _power64((e - 1).clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-TOP, TOP)


def _exact_append(st, case):
    kv, dim, page = case["kv"], case["dim"], case["page"]
    value = _values()
    out = {}
    for name in ("k", "v"):
        c = st[name][0]
        if name == "v":
            c = c.transpose(3, 4).reshape(-1, kv, page, dim)
        codes, scale = value[c.long()], st[name + "_scale"][0].double()
        for s in range(case["seqs"]):
            n, r0, r1 = int(st["kv_len"][s]), int(st["row_start"][s]), int(st["row_start"][s + 1])
            begin = n - (r1 - r0)
            lo, hi = begin // BLOCK, -(-n // BLOCK)
            t = torch.arange(lo * BLOCK, hi * BLOCK, device="cuda")
            at = st["table"][s].long()[t // page]
            had, was = codes[at, :, t % page], scale[at, :, t % page // BLOCK]  # [tokens][kv][dim], [tokens][kv]
            x = had * was[..., None]
            x[begin - lo * BLOCK:n - lo * BLOCK] = \
                st["new_" + name][r0:r1].double().reshape(-1, kv, dim)
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
        out[name], out[name + "_scale"] = codes.reshape(st[name].shape), scale[None]
    return out


def _exact_attention(st, case):
    kv, dim, page, heads = case["kv"], case["dim"], case["page"], case["heads"]
    group, value = heads // kv, _values()
    out = torch.zeros(st["total"], heads, dim, dtype=torch.float64, device="cuda")
    lse = torch.full((st["total"], heads), -math.inf, dtype=torch.float64, device="cuda")
    q = st["q"].double().reshape(-1, heads, dim)
    for s in range(case["seqs"]):
        n, r0, r1 = int(st["kv_len"][s]), int(st["row_start"][s]), int(st["row_start"][s + 1])
        t = torch.arange(n, device="cuda")
        page_of = st["table"][s].long()[t // page]
        at = n - (r1 - r0) + torch.arange(r1 - r0, device="cuda")
        hidden = t > at[:, None]
        if case["window"]:
            hidden |= (t <= at[:, None] - case["window"]) & (t >= case["sinks"])
        for h in range(kv):
            k = value[st["k"][0, page_of, h, t % page].long()]
            k = k * st["k_scale"][0, page_of, h, t % page // BLOCK].double()[:, None]
            v = value[st["v"][0, page_of, h, t % page // 4, :, t % 4].long()]
            v = v * st["v_scale"][0, page_of, h, t % page // BLOCK].double()[:, None]
            for i in range(group):
                x = q[r0:r1, h * group + i] @ k.T / math.sqrt(dim)
                x.masked_fill_(hidden, -math.inf)
                z = torch.logsumexp(x, 1)
                out[r0:r1, h * group + i] = x.sub_(z[:, None]).exp_() @ v
                lse[r0:r1, h * group + i] = z
    return {"out": out.reshape(-1, heads * dim), "lse": lse}
