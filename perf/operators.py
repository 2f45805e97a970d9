"""What the attention cache's operators are measured on: storing tokens in a paged cache of 8-bit codes, attending over
it (one token a sequence, a few, prompts; whole, or through a sliding window with sinks), and moving its pages.

A cache holds K and V in blocks of 32 tokens of one head.  A block has one exponent e, the smallest integer with
amax <= TOP * 2^e (TOP: 448 for e4m3, 127 for int8), and 8-bit codes RNE(x * 2^-e).  A token's values are code * 2^e.
When a later token of the block needs a larger e, the codes that are there are rounded to the new one.

With `own` false, `run` computes the plain form in elementary torch operations; with `own` true it makes the calls a
user makes of this package.
"""

import math
import random

import torch

own = False

BLOCK = 32                     # tokens that share an exponent
TOP = {"e4m3": 448.0, "int8": 127.0}
ACT = {"f16": torch.float16, "bf16": torch.bfloat16}
DEV = "cuda"

# heads, heads of K and V, head size: the widths 4096, 7168 and 8192 of this repository's layers
HEADS = [(32, 32, 128), (56, 56, 128), (64, 8, 128), (128, 8, 64)]


def _attend(name, n, lo, hi, new_lo, new_hi, heads, page, act, code, window=0, sinks=0, mix=1):
    return dict(name=name, kind="attend", n=n, lo=lo, hi=hi, new_lo=new_lo, new_hi=new_hi, heads=heads[0],
                kv_heads=heads[1], dim=heads[2], page=page, act=act, code=code, window=window, sinks=sinks, mix=mix)


def _append(name, n, lo, hi, new_lo, new_hi, heads, page, act, code, mix=1):
    return dict(name=name, kind="append", n=n, lo=lo, hi=hi, new_lo=new_lo, new_hi=new_hi, heads=heads[0],
                kv_heads=heads[1], dim=heads[2], page=page, act=act, code=code, mix=mix)


def _pages(name, kind, n, lo, hi, heads, page, layers, mix=1):
    return dict(name=name, kind=kind, n=n, lo=lo, hi=hi, heads=heads[0], kv_heads=heads[1], dim=heads[2], page=page,
                layers=layers, mix=mix)


def listed():
    return [
        # a lone user's first words: nothing but latency
        _attend("step one short", 1, 37, 37, 1, 1, HEADS[0], 64, "f16", "e4m3"),
        # a full server between steps: short and long conversations side by side, 8 query heads to a cached head
        _attend("step 64 ragged", 64, 100, 8192, 1, 1, HEADS[2], 64, "f16", "e4m3", mix=2),
        # every query head has its own cached head: the cache is all there is to read
        _attend("step one head each", 16, 3000, 5000, 1, 1, HEADS[0], 32, "bf16", "int8", mix=3),
        # one long document, four guessed tokens checked at once, 16 query heads to a cached head
        _attend("four tokens long cache", 1, 100003, 100003, 4, 4, HEADS[3], 128, "f16", "e4m3"),
        # a prompt's own attention
        _attend("prompt", 1, 4096, 4096, 4096, 4096, HEADS[2], 64, "f16", "e4m3"),
        # prompts taken in pieces, over what earlier pieces left
        _attend("pieces of prompts", 4, 2000, 8000, 100, 1000, HEADS[1], 64, "bf16", "int8", mix=5),
        # long conversations of a model with a window: what falls behind it is not read, but for the first tokens
        _attend("step window sinks", 32, 1000, 32768, 1, 1, HEADS[2], 64, "bf16", "e4m3", window=2048, sinks=4, mix=6),
        # a long prompt of such a model
        _attend("prompt window sinks", 1, 8191, 8191, 8191, 8191, HEADS[0], 64, "f16", "e4m3", window=1024, sinks=4),
        # storing one token of every sequence, and reading back the blocks that changed
        _append("store a step", 64, 100, 2000, 1, 1, HEADS[2], 64, "f16", "e4m3", mix=7),
        # storing prompts
        _append("store prompts", 6, 1, 9000, 500, 4000, HEADS[0], 64, "bf16", "int8", mix=8),
        # a step of a beam search: losers freed, survivors forked into their places, room for a token each
        _pages("beams freed and forked", "fork", 32, 200, 3000, HEADS[2], 64, 4),
        # a pool shrunk after half of its sequences left: the pages in use move to its front
        _pages("pool compacted", "compact", 64, 500, 4000, HEADS[2], 64, 4, mix=9),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    heads, page = rng.choice(HEADS), rng.choice([32, 64, 128])
    act, code, mix = rng.choice(["f16", "bf16"]), rng.choice(["e4m3", "int8"]), rng.randrange(1 << 20)
    kind = rng.choice(["step", "step", "step", "few", "prompt", "pieces", "store", "fork", "compact"])
    window, sinks = (0, 0) if rng.random() < 0.6 else (_log_int(rng, 16, 4096), rng.choice([0, 1, 4, 33]))
    if kind in ("step", "few"):
        n = _log_int(rng, 1, 128)
        most = min(100000, (1 << 19) * 8 // (n * heads[1]))      # tokens a sequence: at most 4 Mi tokens and heads
        hi = _log_int(rng, 8, most)
        new = 1 if kind == "step" else rng.randint(2, 7)
        c = _attend("", n, max(new, _log_int(rng, 1, hi)), max(hi, new), 1 if kind == "step" else 0, new, heads, page,
                    act, code, window, sinks, mix)
    elif kind == "prompt":
        hi = _log_int(rng, 8, 4096)
        n = rng.randint(1, max(1, min(4, 4096 // hi)))
        c = _attend("", n, hi, hi, hi, hi, heads, page, act, code, window, sinks, mix)
    elif kind == "pieces":
        hi, new = _log_int(rng, 300, 8000), _log_int(rng, 16, 300)
        c = _attend("", rng.randint(1, 6), 300, hi, 1, new, heads, page, act, code, window, sinks, mix)
    elif kind == "store":
        n = _log_int(rng, 1, 64)
        new = _log_int(rng, 1, max(1, 8192 // n))
        c = _append("", n, 1, _log_int(rng, 1, 4000), 0 if new > 1 else 1, new, heads, page, act, code, mix)
    elif kind == "fork":
        hi = _log_int(rng, 50, 3000)
        c = _pages("", "fork", _log_int(rng, 1, 32), max(1, hi // 3), hi, HEADS[2], page, rng.randint(1, 4), mix)
    else:
        hi = _log_int(rng, 50, 4000)
        c = _pages("", "compact", _log_int(rng, 2, 64), max(1, hi // 3), hi, HEADS[2], page, rng.randint(1, 4), mix)
    c.pop("name")
    return c


# ---- sizes, from the case alone ----------------------------------------------------------------------


def _sizes(case):
    """(tokens held before the call, new tokens) of every sequence."""
    rng = random.Random(case["mix"])
    total, new = [], []
    for _ in range(case["n"]):
        total.append(_log_int(rng, case["lo"], case["hi"]))
        new.append(rng.randint(case["new_lo"], case["new_hi"]) if "new_lo" in case else 0)
    if not any(new):
        new[0] = case.get("new_hi", 0)
    if case["kind"] == "append":
        return total, new
    new = [min(a, b) for a, b in zip(new, total)]
    return [a - b for a, b in zip(total, new)], new


def _visible(case, i):
    """How many tokens row position i sees."""
    w, s = case["window"], case["sinks"]
    if w == 0 or i + 1 <= w:
        return i + 1
    return w + min(s, i + 1 - w)


def work(case):
    kind = case["kind"]
    kvh, dim = case["kv_heads"], case["dim"]
    if kind in ("fork", "compact"):
        page = kvh * case["page"] * dim * 2 + kvh * (case["page"] // BLOCK) * 2
        s = _page_state(case)
        moved = s["copies"] * page * case["layers"]
        return {"bytes": 2 * moved + 8 * s["entries"] + 8 * s["pages"], "flops": 0}
    before, new = _sizes(case)
    tok = kvh * dim * 2                                   # bytes of a token's codes, K and V
    if kind == "append":
        rows = sum(b % BLOCK + c for b, c in zip(before, new) if c)
        return {"bytes": sum(new) * tok * (2 + 1) + rows * tok * (1 + 2) + rows * kvh * 2 // BLOCK, "flops": 0}
    read, pairs = 0, 0
    for b, c in zip(before, new):
        if c == 0:
            continue
        pairs += sum(_visible(case, i) for i in range(b, b + c))
        seen = b + c
        if case["window"]:
            first = max(0, b - case["window"] + 1)        # the first token that the first row's window holds
            seen = b + c - first + min(first, case["sinks"])
        read += seen
    t = sum(new)
    rows = t * case["heads"]
    return {"bytes": read * (tok + kvh * 2 / BLOCK) + rows * (dim * 4 + 4), "flops": pairs * case["heads"] * dim * 4}


# ---- inputs ------------------------------------------------------------------------------------------


def _gen(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + case["mix"])
    return g


def _kv(case, gen, n, tokens):
    """K and V of `tokens` tokens of n sequences: [n][tokens][kv_heads][dim] in the activations' type.  A few channels of
    K are several times larger than the others, and tokens differ in size, as they do in trained models."""
    kvh, dim, act = case["kv_heads"], case["dim"], ACT[case["act"]]
    out = []
    for spread in (0.8, 0.3):
        chan = torch.exp(spread * torch.randn(kvh, dim, device=DEV, generator=gen))
        size = torch.exp(0.3 * torch.randn(n, tokens, 1, 1, device=DEV, generator=gen))
        x = torch.randn(n, tokens, kvh, dim, device=DEV, generator=gen, dtype=torch.float32)
        out.append(x.mul_(chan).mul_(size).to(act))
    return out


def _inputs(case, seed):
    """Everything random of an attend or append case."""
    gen = _gen(case, seed)
    before, new = _sizes(case)
    n, page = case["n"], case["page"]
    total = [a + b for a, b in zip(before, new)]
    pages = [-(-t // page) for t in total]
    width = max(pages)
    k, v = _kv(case, gen, n, width * page)
    q = torch.randn(sum(new), case["heads"], case["dim"], device=DEV, generator=gen).mul_(1.5).to(ACT[case["act"]])
    pool = sum(pages) + 7
    order = torch.randperm(pool, device=DEV, generator=gen).to(torch.int32)     # pages lie about as after long use
    starts = torch.tensor([0] + pages).cumsum(0).tolist()
    table = torch.full((n, width), -1, dtype=torch.int32, device=DEV)
    col = torch.arange(width, device=DEV)
    held = col[None] < torch.tensor(pages, device=DEV)[:, None]
    table[held] = order[:starts[-1]]
    return dict(k=k, v=v, q=q, table=table, held=held, pool=pool, width=width, before=before, new=new, total=total)


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    if case["kind"] in ("fork", "compact"):
        return _prepare_pages(case, seed)
    x = _inputs(case, seed)
    n, page, width = case["n"], case["page"], x["width"]
    before, new, total = x["before"], x["new"], x["total"]
    pos = torch.arange(width * page, device=DEV)
    lens_b, lens_t = torch.tensor(before, device=DEV), torch.tensor(total, device=DEV)
    new_mask = (pos[None] >= lens_b[:, None]) & (pos[None] < lens_t[:, None])
    s = dict(case=case, q=x["q"], k_new=x["k"][new_mask], v_new=x["v"][new_mask])
    first = [b // BLOCK * BLOCK if c else t for b, c, t in zip(before, new, total)]   # where the changed blocks begin
    seqs, starts = _int(list(range(n))), _int([0] + torch.tensor(new).cumsum(0).tolist())
    filled = lens_t if case["kind"] == "attend" else lens_b                            # what the cache holds at the call
    fill_mask = pos[None] < filled[:, None]
    if own:
        from activation_sparse_decode_relu_amd import KVCache
        cache = KVCache(heads=case["heads"], kv_heads=case["kv_heads"], head_dim=case["dim"], pages=x["pool"],
                        page_tokens=page, max_seqs=n, max_seq_pages=width, act_dtype=case["act"], code=case["code"])
        cache.table.copy_(x["table"])
        cache.refs.zero_()
        cache.refs[x["table"][x["held"]].long()] = 1
        cache.lens.copy_(filled)
        fill = _int([0] + filled.cpu().cumsum(0).tolist())
        cache.append(0, x["k"][fill_mask], x["v"][fill_mask], seqs, fill)
        cache.lens.copy_(lens_t)
        read = [0] + torch.tensor([t - f for t, f in zip(total, first)]).cumsum(0).tolist()
        act, rows = ACT[case["act"]], read[-1]
        s.update(cache=cache, seqs=seqs, starts=starts, most=max(new), first=_int(first), read=_int(read),
                 out=torch.empty_like(x["q"]), lse=torch.empty(x["q"].shape[:2], dtype=torch.float32, device=DEV))
        if case["kind"] == "append":
            s.update(k_out=torch.empty(rows, case["kv_heads"], case["dim"], dtype=act, device=DEV),
                     v_out=torch.empty(rows, case["kv_heads"], case["dim"], dtype=act, device=DEV))
        return s
    # the plain cache: codes [pages][page][kv_heads][dim] and exponents [pages][page / 32][kv_heads]
    table = x["table"]
    for name in ("k", "v"):
        masked = x[name].masked_fill(~fill_mask[:, :, None, None], 0)
        blocks = masked.reshape(n * width * page // BLOCK, BLOCK, case["kv_heads"], case["dim"])
        codes, exps = _encode(blocks.float(), _exponent(blocks.float(), case["code"]), case["code"])
        codes = codes.reshape(n, width, page, case["kv_heads"], case["dim"])
        exps = exps.reshape(n, width, page // BLOCK, case["kv_heads"])
        s[name + "_codes"] = torch.zeros(x["pool"], page, case["kv_heads"], case["dim"], dtype=torch.uint8, device=DEV)
        s[name + "_exps"] = torch.full((x["pool"], page // BLOCK, case["kv_heads"]), -126, dtype=torch.int32, device=DEV)
        s[name + "_codes"][table[x["held"]].long()] = codes[x["held"]]
        s[name + "_exps"][table[x["held"]].long()] = exps[x["held"]]
    s["table"] = table.clamp(min=0).long()
    # where the packed rows belong in a padded batch
    row_mask = torch.arange(max(max(new), 1), device=DEV)[None] < torch.tensor(new, device=DEV)[:, None]
    s["row_mask"], s["pos"], s["lens_b"], s["lens_t"] = row_mask, pos, lens_b, lens_t
    if case["kind"] == "append":
        blk = torch.arange(width * page // BLOCK, device=DEV)
        hit = (blk[None] >= (torch.tensor(first, device=DEV) // BLOCK)[:, None]) & (blk[None] * BLOCK < lens_t[:, None])
        hit &= (torch.tensor(new, device=DEV) > 0)[:, None]
        seq, b = hit.nonzero(as_tuple=True)
        tok = b[:, None] * BLOCK + torch.arange(BLOCK, device=DEV)[None]
        row0 = torch.tensor([0] + new, device=DEV).cumsum(0)[:-1]
        s["at_page"], s["at_slot"] = s["table"][seq, b // (page // BLOCK)], b % (page // BLOCK)
        s["is_old"], s["is_held"] = tok < lens_b[seq][:, None], tok < lens_t[seq][:, None]
        s["is_new"] = ~s["is_old"] & s["is_held"]
        s["src"] = (row0[seq][:, None] + tok - lens_b[seq][:, None]).clamp(0, max(sum(new) - 1, 0))
    return s


# ---- the plain form ----------------------------------------------------------------------------------


def _exponent(x, code):
    """Blocks [b][32][heads][dim] -> the exponent of each block and head [b][heads]."""
    amax = x.abs().amax(dim=(1, 3))
    frac, ex = torch.frexp(amax)                      # amax = frac * 2^ex, frac in [0.5, 1)
    top, top_ex = math.frexp(TOP[code])
    e = ex.to(torch.int32) - top_ex + (frac > top).to(torch.int32)
    return torch.where(amax == 0, torch.full_like(e, -126), e.clamp(-126, 127))


def _pow2(e):
    """2^e as fp32, exactly, for whole e in [-126, 127]."""
    return (e.to(torch.int32) + 127).bitwise_left_shift(23).view(torch.float32)


def _encode(x, e, code):
    scaled = x * _pow2(-e)[:, None, :, None]
    if code == "int8":
        return torch.round(scaled).to(torch.int8).view(torch.uint8), e
    return scaled.to(torch.float8_e4m3fn).view(torch.uint8), e


def _decode(codes, code):
    return codes.view(torch.int8).float() if code == "int8" else codes.view(torch.float8_e4m3fn).float()


def _values(codes, e, code):
    """Codes [...][tokens][heads][dim] with exponents [...][tokens / 32][heads] -> fp32 values."""
    e = e.repeat_interleave(BLOCK, dim=-2)
    return _decode(codes, code) * _pow2(e)[..., None]


def _plain_attend(s):
    case, table = s["case"], s["table"]
    n, h, kvh, dim = case["n"], case["heads"], case["kv_heads"], case["dim"]
    k = _values(s["k_codes"][table].flatten(1, 2), s["k_exps"][table].flatten(1, 2), case["code"])
    v = _values(s["v_codes"][table].flatten(1, 2), s["v_exps"][table].flatten(1, 2), case["code"])
    rows = s["row_mask"].shape[1]
    q = torch.zeros(n, rows, h, dim, device=DEV)
    q[s["row_mask"]] = s["q"].float()
    q = q.reshape(n, rows, kvh, h // kvh, dim).permute(0, 2, 3, 1, 4).reshape(n, kvh, h // kvh * rows, dim)
    scores = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous()).mul_(dim ** -0.5)
    i, j = s["lens_b"][:, None] + torch.arange(rows, device=DEV), s["pos"][None, None]
    seen = (j <= i[:, :, None]) & s["row_mask"][:, :, None]
    if case["window"]:
        seen &= (j > i[:, :, None] - case["window"]) | (j < case["sinks"])
    scores = scores.view(n, kvh, h // kvh, rows, -1).masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores.sub_(torch.where(top.isinf(), torch.zeros_like(top), top)))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.reshape(n, kvh, h // kvh * rows, -1), v.permute(0, 2, 1, 3)).view(n, kvh, h // kvh, rows, dim)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    lse = (top + torch.log(total)).squeeze(-1)
    out = out.permute(0, 3, 1, 2, 4).reshape(n, rows, h, dim)[s["row_mask"]]
    lse = lse.permute(0, 3, 1, 2).reshape(n, rows, h)[s["row_mask"]]
    return {"out": out.to(s["q"].dtype), "lse": lse}


def _plain_append(s):
    case = s["case"]
    act, code = s["k_new"].dtype, case["code"]
    big = torch.finfo(act).max
    got = {}
    for name in ("k", "v"):
        codes, exps = s[name + "_codes"], s[name + "_exps"]
        page, slot = s["at_page"], s["at_slot"]
        grouped = codes.view(codes.shape[0], -1, BLOCK, *codes.shape[2:])
        old, old_e = _decode(grouped[page, slot], code), exps[page, slot]
        fresh = s[name + "_new"][s["src"]].float().masked_fill(~s["is_new"][:, :, None, None], 0)
        has_old = s["is_old"].any(1)[:, None]
        e = torch.where(has_old, torch.maximum(old_e, _exponent(fresh, code)), _exponent(fresh, code))
        kept = (old * _pow2(old_e)[:, None, :, None]).masked_fill(~s["is_old"][:, :, None, None], 0)
        block, e = _encode(kept + fresh, e, code)
        grouped[page, slot] = block
        exps[page, slot] = e
        values = (_decode(block, code) * _pow2(e)[:, None, :, None]).clamp(-big, big)
        got[name] = values[s["is_held"]].to(act)
    return got


# ---- pages -------------------------------------------------------------------------------------------


def _page_state(case):
    """Table, lengths and reference counts before the call, and how many pages the call copies.  fork: 2n slots, the first
    n hold the survivors, the others hypotheses that were forked from them a step ago.  compact: the sequences that are
    left, on pages all over the pool."""
    rng = random.Random(case["mix"] * 31 + 7)
    n, page = case["n"], case["page"]
    total = [_log_int(rng, case["lo"], case["hi"]) for _ in range(n)]
    count = [-(-t // page) for t in total]
    if case["kind"] == "fork":
        src = [rng.randrange(n) for _ in range(n)]
        width = max(-(-(t + 2) // page) for t in total)
        pool = sum(count) + 3 * n + 5
        ids = rng.sample(range(pool), sum(count) + n)
        table = [[ids.pop() if j < c else -1 for j in range(width)] for c in count]
        refs = [0] * pool
        for row in table:
            for p in row:
                if p >= 0:
                    refs[p] += 1
        lens = list(total)
        for i in range(n):
            row = list(table[i])                      # a child of survivor i that has grown by a token
            tail = total[i] // page
            row[tail] = ids.pop()
            table.append(row)
            lens.append(total[i] + 1)
            for p in row:
                if p >= 0:
                    refs[p] += 1
        copies = sum(total[i] % page != 0 for i in src)
        entries = 2 * sum(count[i] for i in src)
        return dict(table=table, lens=lens, refs=refs, src=src, copies=copies, entries=entries, pages=pool, width=width)
    pool = 2 * sum(count)
    ids = rng.sample(range(pool), sum(count))
    refs = [0] * pool
    for p in ids:
        refs[p] = 1
    copies = sum(p >= len(ids) for p in ids)
    width = max(count)
    table = [[ids.pop() if j < c else -1 for j in range(width)] for c in count]
    return dict(table=table, lens=total, refs=refs, src=[], copies=copies, entries=2 * sum(count), pages=pool, width=width)


def _prepare_pages(case, seed):
    st = _page_state(case)
    gen = _gen(case, seed)
    layers, page, kvh, dim = case["layers"], case["page"], case["kv_heads"], case["dim"]
    shapes = {"k": kvh * page * dim, "v": kvh * page * dim, "k_exp": kvh * page // BLOCK, "v_exp": kvh * page // BLOCK}
    # copying does not look into the bytes: a page is what it is
    data = {name: torch.randint(0, 256, (layers, st["pages"], size), dtype=torch.uint8, device=DEV, generator=gen)
            for name, size in shapes.items()}
    meta = dict(table=_int(st["table"]), lens=_int(st["lens"]), refs=_int(st["refs"]))
    s = dict(case=case, saved={k: t.clone() for k, t in meta.items()})
    if case["kind"] == "fork":
        n = case["n"]
        s.update(src=_int(st["src"]), dst=_int(list(range(n, 2 * n))), one=torch.ones(n, dtype=torch.int32, device=DEV))
    if own:
        from activation_sparse_decode_relu_amd import KVCache
        cache = KVCache(heads=case["heads"], kv_heads=kvh, head_dim=dim, pages=st["pages"], page_tokens=page,
                        max_seqs=len(st["lens"]), max_seq_pages=st["width"], layers=layers, buffers={**data, **meta})
        s.update(cache=cache)
    else:
        s.update(data=data, **meta)
    return s


def _copy_pages(data, src, dst):
    for pool in data.values():
        pool[:, dst] = pool[:, src]


def _plain_fork(s):
    page, table, lens, refs, src, dst = s["case"]["page"], s["table"], s["lens"], s["refs"], s["src"].long(), s["dst"].long()
    # free the old hypotheses
    refs.sub_(torch.zeros_like(refs).index_add_(0, table[dst].clamp(min=0).flatten().long(),
                                                (table[dst] >= 0).to(torch.int32).flatten()))
    # the survivors' pages, shared
    table[dst], lens[dst] = table[src], lens[src]
    refs.add_(torch.zeros_like(refs).index_add_(0, table[dst].clamp(min=0).flatten().long(),
                                                (table[dst] >= 0).to(torch.int32).flatten()))
    # room for one token each: a page of its own where the last is full or shared
    at = lens[dst] // page
    last = table[dst, at.long()].clamp(min=0).long()
    copied = (lens[dst] % page != 0) & (refs[last] > 1)
    need = (lens[dst] % page == 0) | copied
    free = torch.argsort((refs > 0).to(torch.int32), stable=True)        # free pages, lowest first
    fresh = free[(need.cumsum(0) - 1).clamp(min=0)]
    table[dst, at.long()] = torch.where(need, fresh.to(torch.int32), table[dst, at.long()])
    refs.index_add_(0, fresh, need.to(torch.int32))
    refs.index_add_(0, last, -copied.to(torch.int32))
    lens[dst] = lens[dst] + 1
    _copy_pages(s["data"], last[copied], fresh[copied])
    return {"table": table, "lens": lens, "refs": refs, **s["data"]}


def _plain_compact(s):
    for name in ("table", "lens", "refs"):
        s[name].copy_(s["saved"][name])
    table, refs = s["table"], s["refs"]
    live = refs > 0
    front = torch.arange(refs.numel(), device=DEV) < live.sum()
    holes, movers = (front & ~live).nonzero().flatten(), (live & ~front).nonzero().flatten()
    where = torch.arange(refs.numel(), device=DEV, dtype=torch.int32)
    where[movers] = holes.to(torch.int32)
    s["table"] = torch.where(table >= 0, where[table.clamp(min=0).long()], table)
    refs[holes] = refs[movers]
    refs[movers] = 0
    _copy_pages(s["data"], movers, holes)
    return {"table": s["table"], "lens": s["lens"], "refs": refs, **s["data"]}


# ---- one pass ----------------------------------------------------------------------------------------


def _cache_state(cache):
    return {"table": cache.table, "lens": cache.lens, "refs": cache.refs, "k": cache.k, "v": cache.v,
            "k_exp": cache.k_exp, "v_exp": cache.v_exp}


def run(s):
    case = s["case"]
    kind = case["kind"]
    if not own:
        return {"attend": _plain_attend, "append": _plain_append, "fork": _plain_fork, "compact": _plain_compact}[kind](s)
    cache = s["cache"]
    if kind == "attend":
        cache.attend(0, s["q"], s["out"], s["seqs"], s["starts"], max_new=s["most"], window=case["window"],
                     sinks=case["sinks"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if kind == "append":
        cache.append(0, s["k_new"], s["v_new"], s["seqs"], s["starts"])
        cache.read(0, s["k_out"], s["v_out"], s["seqs"], s["read"], first=s["first"])
        return {"k": s["k_out"], "v": s["v_out"]}
    if kind == "fork":
        cache.free(s["dst"])
        cache.fork(s["src"], s["dst"])
        cache.reserve(s["dst"], s["one"])
        return _cache_state(cache)
    for name in ("table", "lens", "refs"):
        getattr(cache, name).copy_(s["saved"][name])
    cache.compact()
    return _cache_state(cache)


# ---- the definition in 64 bits -----------------------------------------------------------------------


def _stored64(parts, code):
    """What a cache holds of one head group after storing `parts` ([tokens][kv_heads][dim] each) one after the other:
    fp64 values, from the definition, block by block."""
    bits, low, top = (3, -6, 448.0) if code == "e4m3" else (None, None, 127.0)

    def two(e):                                        # 2^e, exactly
        return (e.long() + 1023).bitwise_left_shift(52).view(torch.float64)

    def need(x):                                       # smallest e with amax <= top 2^e
        amax = x.abs().amax(dim=(0, 2))
        e = torch.ceil(torch.log2(amax.clamp(min=2.0 ** -140) / top)).long()
        e = torch.where(top * two(e - 1) >= amax, e - 1, e)
        e = torch.where(top * two(e) < amax, e + 1, e)
        return torch.where(amax == 0, torch.full_like(e, -126), e.clamp(-126, 127))

    def rounded(x, e):                                 # to the codes' grid
        unit = two(e)[None, :, None]
        y = x / unit
        if bits is None:
            return torch.round(y) * unit
        _, ex = torch.frexp(y)                         # |y| in [2^(ex-1), 2^ex)
        step = two((ex - 1).clamp(min=low) - bits)
        return torch.round(y / step) * step * unit

    held = torch.zeros(0, *parts[0].shape[1:], dtype=torch.float64, device=DEV)
    exps = {}
    for part in parts:
        x, pos = part.double(), held.shape[0]
        at = 0
        pieces = [held[:pos // BLOCK * BLOCK]]
        while at < x.shape[0]:
            blk = (pos + at) // BLOCK
            take = min(x.shape[0] - at, (blk + 1) * BLOCK - (pos + at))
            here = x[at:at + take]
            old = held[blk * BLOCK:pos] if blk * BLOCK < pos else held[:0]
            e = need(here)
            if old.shape[0]:
                e = torch.maximum(e, exps[blk])
            exps[blk] = e
            pieces.append(rounded(torch.cat([old, here]), e))
            at += take
        held = torch.cat(pieces) if x.shape[0] else held
    return held


def _whole64(x, code):
    """As _stored64 for tokens stored in one call, all blocks at once."""
    t = x.shape[0]
    pad = -t % BLOCK
    y = torch.cat([x.double(), torch.zeros(pad, *x.shape[1:], dtype=torch.float64, device=DEV)])
    y = y.reshape(-1, BLOCK, *x.shape[1:]).permute(1, 0, 2, 3)              # a block is a "head" of its own
    b, h, d = y.shape[1:]
    return _stored64([y.reshape(BLOCK, b * h, d)], code).reshape(BLOCK, b, h, d).permute(1, 0, 2, 3).reshape(-1, h, d)[:t]


def exact(case, seed):
    if case["kind"] in ("fork", "compact"):
        return None
    x = _inputs(case, seed)
    code, h, kvh, dim = case["code"], case["heads"], case["kv_heads"], case["dim"]
    if case["kind"] == "append":
        big = torch.finfo(ACT[case["act"]]).max
        got = {"k": [], "v": []}
        for i, (b, c) in enumerate(zip(x["before"], x["new"])):
            if c == 0:
                continue
            edge, end = b // BLOCK * BLOCK, b + c
            cut = min(end, edge + BLOCK)               # the block that held tokens before, then whole blocks
            for name in got:
                src = x[name][i]
                got[name] += [_stored64([src[edge:b], src[b:cut]], code) if b > edge else _whole64(src[edge:cut], code)]
                got[name] += [_whole64(src[cut:end], code)] if end > cut else []
        return {name: torch.cat(got[name]).clamp(-big, big) for name in got}
    outs, lses, row = [], [], 0
    for i, (b, c) in enumerate(zip(x["before"], x["new"])):
        if c == 0:
            continue
        k, v = (_whole64(x[name][i][:b + c], code) for name in ("k", "v"))
        q = x["q"][row:row + c].double().reshape(c, kvh, h // kvh, dim)
        row += c
        where = torch.arange(b, b + c, device=DEV)[:, None]
        j = torch.arange(b + c, device=DEV)[None]
        hidden = j > where
        if case["window"]:
            hidden = hidden | ((j <= where - case["window"]) & (j >= case["sinks"]))
        out = torch.empty(c, kvh, h // kvh, dim, dtype=torch.float64, device=DEV)
        lse = torch.empty(c, kvh, h // kvh, dtype=torch.float64, device=DEV)
        for a in range(kvh):
            for r in range(h // kvh):
                z = (q[:, a, r] @ k[:, a].T) / math.sqrt(dim)
                z[hidden] = -math.inf
                lse[:, a, r] = torch.logsumexp(z, 1)
                out[:, a, r] = torch.exp(z - lse[:, a, r, None]) @ v[:, a]
        outs.append(out.reshape(c, h, dim))
        lses.append(lse.reshape(c, h))
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
