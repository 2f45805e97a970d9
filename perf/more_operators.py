"""What the operators round the attention cache are measured on: products with 4-bit weights, norms and rotation of queries
and keys, and attention of sequences that share the beginning of their caches.

project   y = x W^T + bias + add.  W is in 4 bits: 32 consecutive elements of a row share an fp16 scale.
rotate    each head of q and k: divided by its root mean square, times a weight, then pairs of its first dims turned by
          position times frequency.
shared    attention over a paged cache of 8-bit codes (blocks of 32 tokens of one head share a power of two) where the
          sequences of a group begin with the same pages.

With `own` false, `run` computes the plain form in elementary torch operations; with `own` true it makes the calls a
user makes of this package.
"""

import math
import random

import torch

own = False

GROUP = 32                     # elements of a weight row that share a scale, and tokens of the cache that share an exponent
TOP = {"e4m3": 448.0, "int8": 127.0}
ACT = {"f16": torch.float16, "bf16": torch.bfloat16}
DEV = "cuda"
EPS = 1e-6

# heads, heads of K and V, head size: the widths 4096, 7168 and 8192 of this repository's layers
HEADS = [(32, 32, 128), (56, 56, 128), (64, 8, 128), (128, 8, 64)]


def _project(name, rows, d_in, d_out, act, bias=False, add=False):
    return dict(name=name, kind="project", rows=rows, d_in=d_in, d_out=d_out, act=act, bias=bias, add=add)


def _rotate(name, n, lo, hi, new_lo, new_hi, heads, act, layout, rot, norm, scaling="none", factor=1.0, mix=1):
    return dict(name=name, kind="rotate", n=n, lo=lo, hi=hi, new_lo=new_lo, new_hi=new_hi, heads=heads[0],
                kv_heads=heads[1], dim=heads[2], act=act, layout=layout, rot=rot, norm=norm, scaling=scaling,
                factor=factor, original=8192 if scaling == "bands" else 0, gain=1.1 if scaling == "bands" else 1.0,
                base=500000.0 if scaling == "bands" else 10000.0, mix=mix)


def _shared(name, groups, members_lo, members_hi, lo, hi, own_lo, own_hi, new, heads, page, act, code, layers=2, mix=1):
    return dict(name=name, kind="shared", groups=groups, members_lo=members_lo, members_hi=members_hi, lo=lo, hi=hi,
                own_lo=own_lo, own_hi=own_hi, new=new, heads=heads[0], kv_heads=heads[1], dim=heads[2], page=page, act=act,
                code=code, layers=layers, mix=mix)


def listed():
    return [
        # one token through the toy layer's width: nothing but latency
        _project("project toy", 1, 512, 1536, "f16"),
        # a lone user's token: queries, keys and values of a layer of width 8192 in one product
        _project("project one", 1, 8192, 10240, "bf16", bias=True),
        # a step of 16 conversations: back to the model's width, added to the residual
        _project("project 16 add", 16, 8192, 8192, "f16", add=True),
        # a full server's step
        _project("project 64", 64, 7168, 21504, "bf16"),
        # a prompt
        _project("project prompt", 2000, 4096, 12288, "f16", bias=True),
        # a full server's step: far positions, frequencies scaled for long contexts
        _rotate("rotate step", 64, 100, 100000, 1, 1, HEADS[2], "f16", "half", 128, True, "bands", 8.0),
        # a prompt of a model without norms
        _rotate("rotate prompt", 1, 0, 0, 4096, 4096, HEADS[0], "bf16", "interleaved", 128, False, mix=2),
        # pieces of prompts: half of each head turned
        _rotate("rotate part", 5, 1, 9000, 50, 700, HEADS[3], "f16", "half", 32, True, "linear", 4.0, mix=3),
        # a beam search on a short prompt
        _shared("shared beams", 1, 4, 4, 500, 500, 1, 40, 1, HEADS[0], 64, "f16", "e4m3"),
        # a full server whose conversations begin with the same instructions
        _shared("shared 64", 1, 64, 64, 4096, 4096, 30, 800, 1, HEADS[2], 64, "f16", "e4m3", mix=2),
        # questions about one long document, four guessed tokens each checked at once
        _shared("shared document", 1, 4, 4, 100003, 100003, 5, 300, 4, HEADS[3], 128, "bf16", "int8", mix=3),
        # several groups of several sizes, lone sequences among them
        _shared("shared groups", 6, 1, 9, 100, 6000, 1, 500, 1, HEADS[1], 32, "bf16", "int8", mix=4),
    ]


def _log_int(rng, lo, hi):
    if hi <= 0:
        return 0
    lo = max(lo, 1)
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["project", "project", "rotate", "shared", "shared"])
    act = rng.choice(["f16", "bf16"])
    if kind == "project":
        d_in = GROUP * _log_int(rng, 8, 256)
        d_out = _log_int(rng, 100, 21504)
        rows = rng.choice([1, 1, _log_int(rng, 2, 64), _log_int(rng, 2, 64), _log_int(rng, 65, 2000)])
        rows = min(rows, max(1, 2000 * 4096 * 12288 // (d_in * d_out)))
        c = _project("", rows, d_in, d_out, act, rng.random() < 0.5, rng.random() < 0.5)
    elif kind == "rotate":
        heads = rng.choice(HEADS)
        n = _log_int(rng, 1, 128)
        new = rng.choice([1, _log_int(rng, 1, max(1, 4096 // n))])
        scaling = rng.choice(["none", "linear", "ntk", "bands"])
        c = _rotate("", n, 1, _log_int(rng, 1, 500000), 0 if new > 1 else 1, new, heads, act,
                    rng.choice(["half", "interleaved"]), 16 * rng.randint(1, heads[2] // 16), rng.random() < 0.6, scaling,
                    1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 32.0]), rng.randrange(1 << 20))
    else:
        heads = rng.choice(HEADS)
        groups = _log_int(rng, 1, 8)
        members = _log_int(rng, 2, max(2, 64 // groups))
        most = (48 << 20) // (heads[1] * heads[2])              # tokens held in all: 200 MB of codes in two layers
        own_hi = min(_log_int(rng, 5, 800), most // (2 * groups * members))
        hi = min(_log_int(rng, 40, 100000), most // (2 * groups))
        c = _shared("", groups, rng.choice([1, members]), members, max(1, hi // rng.choice([1, 1, 20])), hi, 1, own_hi,
                    rng.choice([1, 1, 2, 5]), heads, rng.choice([32, 64, 128]), act, rng.choice(["e4m3", "int8"]), 2,
                    rng.randrange(1 << 20))
    c.pop("name")
    return c


def _gen(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + case.get("mix", case.get("rows", 0)))
    return g


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _offsets(counts):
    out = [0]
    for c in counts:
        out.append(out[-1] + c)
    return out


def work(case):
    if case["kind"] == "project":
        rows, d_in, d_out = case["rows"], case["d_in"], case["d_out"]
        weights = d_out * d_in // 2 + d_out * d_in // GROUP * 2
        return {"bytes": weights + rows * (d_in + d_out * (2 if case["add"] else 1)) * 2 + (4 * d_out if case["bias"] else 0),
                "flops": 2 * rows * d_in * d_out}
    if case["kind"] == "rotate":
        elems = sum(_rotate_sizes(case)[1]) * (case["heads"] + case["kv_heads"]) * case["dim"]
        return {"bytes": 4 * elems, "flops": elems * (8 if case["norm"] else 4)}
    g = _shared_sizes(case)
    tok = case["kv_heads"] * (case["dim"] * 2 + 2 / GROUP)
    held = sum(p for p in g["prefix"]) + sum(g["own"])
    pairs = sum(p + o - case["new"] + 1 + i for p, o in zip(g["of"], g["own"]) for i in range(case["new"]))
    rows = len(g["own"]) * case["new"] * case["heads"]
    return {"bytes": case["layers"] * (held * tok + rows * (case["dim"] * 4 + 4)),
            "flops": case["layers"] * pairs * case["heads"] * case["dim"] * 4}


# ---- products with 4-bit weights -----------------------------------------------------------------------


def _project_inputs(case, seed):
    gen = _gen(case, seed)
    rows, d_in, d_out, act = case["rows"], case["d_in"], case["d_out"], ACT[case["act"]]
    # trained weights: rows of different size, quantised by groups
    w = torch.randn(d_out, d_in // GROUP, GROUP, device=DEV, generator=gen)
    w *= d_in ** -0.5 * torch.exp(0.3 * torch.randn(d_out, 1, 1, device=DEV, generator=gen))
    scales = (w.abs().amax(-1) / 7).to(torch.float16)
    q = torch.round(w / scales.float()[..., None]).clamp(-8, 7).to(torch.int8).reshape(d_out, d_in // 2, 2)
    codes = ((q[..., 0] & 15) | (q[..., 1] << 4)).view(torch.uint8)
    chan = torch.exp(0.8 * torch.randn(d_in, device=DEV, generator=gen))     # some channels are far larger than others
    x = (torch.randn(rows, d_in, device=DEV, generator=gen) * chan).to(act)
    s = dict(case=case, codes=codes, scales=scales, x=x, bias=None, add=None)
    if case["bias"]:
        s["bias"] = torch.randn(d_out, device=DEV, generator=gen)
    if case["add"]:
        s["add"] = torch.randn(rows, d_out, device=DEV, generator=gen).to(act)
    return s


def _prepare_project(case, seed):
    s = _project_inputs(case, seed)
    if own:
        from activation_sparse_decode_relu_amd import Linear
        s["linear"] = Linear(s["codes"], s["scales"], act_dtype=case["act"], bias=s["bias"])
        s["y"] = torch.empty(case["rows"], case["d_out"], dtype=s["x"].dtype, device=DEV)
    return s


def _plain_project(s):
    codes = s["codes"]
    low, high = ((codes & 15) ^ 8).float() - 8, ((codes >> 4) ^ 8).float() - 8
    q = torch.stack([low, high], -1).reshape(*s["scales"].shape, GROUP)
    w = (q * s["scales"].float()[..., None]).reshape(codes.shape[0], -1)
    y = s["x"].float() @ w.T
    if s["bias"] is not None:
        y = y + s["bias"]
    if s["add"] is not None:
        y = y + s["add"].float()
    return y.to(s["x"].dtype)


def _exact_project(case, seed):
    s = _project_inputs(case, seed)
    signed = s["codes"].view(torch.int8)
    q = torch.stack([(signed << 4) >> 4, signed >> 4], -1).reshape(*s["scales"].shape, GROUP)
    y = s["x"].double() @ (q.double() * s["scales"].double()[..., None]).reshape(case["d_out"], case["d_in"]).T
    for more in ("bias", "add"):
        if s[more] is not None:
            y += s[more].double()
    return y


# ---- norms and rotation --------------------------------------------------------------------------------


def _rotate_sizes(case):
    """(tokens held before the call, new tokens) of every sequence."""
    rng = random.Random(case["mix"])
    before = [_log_int(rng, case["lo"], case["hi"]) for _ in range(case["n"])]
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["n"])]
    if not any(new):
        new[0] = case["new_hi"]
    return before, new


def _rotate_inputs(case, seed):
    gen = _gen(case, seed)
    before, new = _rotate_sizes(case)
    h, kvh, dim, act = case["heads"], case["kv_heads"], case["dim"], ACT[case["act"]]
    # the rows as the projection leaves them: queries, keys and values side by side
    size = torch.exp(0.5 * torch.randn(sum(new), h + 2 * kvh, 1, device=DEV, generator=gen))
    qkv = (torch.randn(sum(new), h + 2 * kvh, dim, device=DEV, generator=gen) * size).to(act)
    s = dict(case=case, before=before, new=new, q=qkv[:, :h], k=qkv[:, h:h + kvh], q_norm=None, k_norm=None)
    if case["norm"]:
        s["q_norm"], s["k_norm"] = ((1 + 0.2 * torch.randn(dim, device=DEV, generator=gen)).to(act) for _ in range(2))
    return s


def _freqs(case):
    rot = case["rot"]
    base = case["base"]
    if case["scaling"] == "ntk" and rot > 2:
        base *= case["factor"] ** (rot / (rot - 2))
    f = [base ** (-2 * i / rot) for i in range(rot // 2)]
    if case["scaling"] == "linear":
        f = [x / case["factor"] for x in f]
    elif case["scaling"] == "bands":                  # turns within the original length: many stay, few are stretched
        low, high = 1.0, 32.0
        for i, x in enumerate(f):
            keep = min(max((case["original"] * x / (2 * math.pi) - low) / (high - low), 0.0), 1.0)
            f[i] = keep * x + (1 - keep) * x / case["factor"]
    return torch.tensor(f, dtype=torch.float64, device=DEV)


def _positions(s):
    """Position of every row."""
    new = torch.tensor(s["new"], device=DEV)
    first = torch.tensor(s["before"], device=DEV) - (new.cumsum(0) - new)
    return torch.repeat_interleave(first, new) + torch.arange(sum(s["new"]), device=DEV)


def _prepare_rotate(case, seed):
    s = _rotate_inputs(case, seed)
    if own:
        from activation_sparse_decode_relu_amd import KVCache, Rope
        total = [a + b for a, b in zip(s["before"], s["new"])]
        page = 4096
        cache = KVCache(heads=case["heads"], kv_heads=case["kv_heads"], head_dim=case["dim"], pages=1, page_tokens=page,
                        max_seqs=case["n"], max_seq_pages=-(-max(total) // page), act_dtype=case["act"])
        cache.lens.copy_(_int(total))
        rope = Rope(case["dim"], rot_dims=case["rot"], layout=case["layout"], base=case["base"], scaling=case["scaling"],
                    factor=case["factor"], original=case["original"], low=1.0, high=32.0, gain=case["gain"])
        s.update(cache=cache, rope=rope, seqs=_int(list(range(case["n"]))), starts=_int(_offsets(s["new"])),
                 q_out=torch.empty(s["q"].shape, dtype=s["q"].dtype, device=DEV),
                 k_out=torch.empty(s["k"].shape, dtype=s["k"].dtype, device=DEV))
    else:
        s["pos"], s["freqs"] = _positions(s), _freqs(case)
    return s


def _plain_turn(x, norm, cos, sin, case):
    x, rot = x.float(), case["rot"]
    if norm is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * norm.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if case["layout"] == "interleaved" else (x[..., :rot // 2], x[..., rot // 2:rot])
    c, d = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([c, d], -1).flatten(-2) if case["layout"] == "interleaved" else torch.cat([c, d], -1)
    return torch.cat([turned, x[..., rot:]], -1).to(ACT[case["act"]])


def _plain_rotate(s):
    case = s["case"]
    angle = s["pos"].double()[:, None] * s["freqs"]                        # [rows][rot / 2]
    cos, sin = (case["gain"] * torch.cos(angle)).float()[:, None], (case["gain"] * torch.sin(angle)).float()[:, None]
    return {"q": _plain_turn(s["q"], s["q_norm"], cos, sin, case), "k": _plain_turn(s["k"], s["k_norm"], cos, sin, case)}


def _exact_rotate(case, seed):
    s = _rotate_inputs(case, seed)
    pos, f, half = _positions(s).double(), _freqs(case), case["rot"] // 2
    got = {}
    for name in ("q", "k"):
        x = s[name].double()
        if case["norm"]:
            x = x / torch.sqrt(torch.mean(x ** 2, -1, keepdim=True) + EPS) * s[name + "_norm"].double()
        y = x.clone()
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if case["layout"] == "interleaved" else (i, i + half)
            z = torch.polar(torch.full_like(pos, case["gain"]), pos * f[i])[:, None] * torch.complex(x[..., a], x[..., b])
            y[..., a], y[..., b] = z.real, z.imag
        got[name] = y
    return got


# ---- attention of sequences that share their beginning -------------------------------------------------


def _shared_sizes(case):
    """prefix: tokens of each group's common beginning; group: the group of each sequence; of: its common tokens;
    own: its further tokens, the new ones among them."""
    rng = random.Random(case["mix"])
    prefix = [_log_int(rng, case["lo"], case["hi"]) for _ in range(case["groups"])]
    group = [g for g in range(case["groups"]) for _ in range(rng.randint(case["members_lo"], case["members_hi"]))]
    own_tokens = [case["new"] - 1 + _log_int(rng, case["own_lo"], case["own_hi"]) for _ in group]
    return dict(prefix=prefix, group=group, of=[prefix[g] for g in group], own=own_tokens)


def _shared_inputs(case, seed):
    gen = _gen(case, seed)
    g = _shared_sizes(case)
    kvh, dim, act, page, n = case["kv_heads"], case["dim"], ACT[case["act"]], case["page"], len(g["own"])
    total = [p + o for p, o in zip(g["of"], g["own"])]
    # whole pages of the common tokens are held once; each sequence has pages of its own from there on
    whole = [p // page for p in g["prefix"]]
    own_pages = [-(-t // page) - whole[a] for t, a in zip(total, g["group"])]
    pool = sum(whole) + sum(own_pages) + 5
    order = torch.randperm(pool, device=DEV, generator=gen).tolist()         # pages lie about as after long use
    width = max(-(-t // page) for t in total)
    common = [[order.pop() for _ in range(w)] for w in whole]
    table = []
    for a, c in zip(g["group"], own_pages):
        row = common[a] + [order.pop() for _ in range(c)]
        table.append(row + [-1] * (width - len(row)))
    # what every page holds, in the activations' type: one draw for the pool, the common tail of a prefix copied
    data = {}
    for name, spread in (("k", 0.8), ("v", 0.3)):
        chan = torch.exp(spread * torch.randn(case["layers"], 1, 1, kvh, dim, device=DEV, generator=gen))
        size = torch.exp(0.3 * torch.randn(1, pool, page, 1, 1, device=DEV, generator=gen))
        x = torch.randn(case["layers"], pool, page, kvh, dim, device=DEV, generator=gen).mul_(chan).mul_(size).to(act)
        first = {}
        for i, a in enumerate(g["group"]):
            tail = g["prefix"][a] % page
            here = table[i][whole[a]]
            if tail and a in first:
                x[:, here, :tail] = x[:, first[a], :tail]
            first.setdefault(a, here)
        for i, t in enumerate(total):                                        # nothing behind the last token
            if t % page:
                x[:, table[i][t // page], t % page:] = 0
        data[name] = x
    q = torch.randn(case["layers"], n * case["new"], case["heads"], dim, device=DEV, generator=gen).mul_(1.5).to(act)
    return dict(g, n=n, total=total, whole=whole, pool=pool, width=width, table=table, q=q, **data)


def _prepare_shared(case, seed):
    x = _shared_inputs(case, seed)
    page, n, new = case["page"], x["n"], case["new"]
    s = dict(case=case, q=x["q"], group=x["group"], total=x["total"])
    if own:
        from activation_sparse_decode_relu_amd import KVCache
        cache = KVCache(heads=case["heads"], kv_heads=case["kv_heads"], head_dim=case["dim"], pages=x["pool"],
                        page_tokens=page, max_seqs=n, max_seq_pages=x["width"], act_dtype=case["act"], code=case["code"],
                        layers=case["layers"])
        cache.table.copy_(_int(x["table"]))
        used = cache.table[cache.table >= 0]
        cache.refs.index_add_(0, used.long(), torch.ones_like(used))
        cache.lens.copy_(_int(x["total"]))
        # the first of a group stores all of its tokens, the others those behind the common pages
        seen, rows, starts = set(), [], [0]
        for i, a in enumerate(x["group"]):
            at = x["whole"][a] if a in seen else 0
            seen.add(a)
            flat = torch.arange(at * page, x["total"][i], device=DEV)
            rows.append(cache.table[i].long()[flat // page] * page + flat % page)
            starts.append(starts[-1] + flat.numel())
        rows = torch.cat(rows)
        for layer in range(case["layers"]):
            cache.append(layer, x["k"][layer].flatten(0, 1)[rows], x["v"][layer].flatten(0, 1)[rows], _int(list(range(n))),
                         _int(starts))
        members = [x["group"].count(a) for a in range(case["groups"])]
        s.update(cache=cache, seqs=_int(list(range(n))), starts=_int([new * i for i in range(n + 1)]),
                 groups=_int(_offsets(members)), most=max(members) * new,
                 plan=torch.empty(case["groups"] + n, dtype=torch.int32, device=DEV),
                 out=torch.empty_like(x["q"]), lse=torch.empty(x["q"].shape[:3], dtype=torch.float32, device=DEV))
        return s
    # the plain cache: codes [layers][pages][page][kv_heads][dim] and exponents [layers][pages][page / 32][kv_heads]
    for name in ("k", "v"):
        blocks = x[name].reshape(-1, GROUP, case["kv_heads"], case["dim"]).float()
        e = _exponent(blocks, case["code"])
        s[name + "_codes"] = _encode(blocks, e, case["code"]).reshape(x[name].shape)
        s[name + "_exps"] = e.reshape(case["layers"], x["pool"], page // GROUP, case["kv_heads"])
    s["table"] = torch.tensor(x["table"], device=DEV).clamp(min=0)
    return s


def _exponent(x, code):
    """Blocks [b][32][heads][dim] -> the smallest e with amax <= TOP 2^e of each block and head [b][heads]."""
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
        return torch.round(scaled).to(torch.int8).view(torch.uint8)
    return scaled.to(torch.float8_e4m3fn).view(torch.uint8)


def _values(codes, e, code):
    """Codes [tokens][heads][dim] with exponents [tokens / 32][heads] -> fp32 values."""
    x = codes.view(torch.int8).float() if code == "int8" else codes.view(torch.float8_e4m3fn).float()
    return x * _pow2(e).repeat_interleave(GROUP, dim=0)[..., None]


def _plain_shared(s):
    case, new = s["case"], s["case"]["new"]
    h, kvh, dim = case["heads"], case["kv_heads"], case["dim"]
    outs, lses = [], []
    for layer in range(case["layers"]):
        for i, t in enumerate(s["total"]):
            pages = s["table"][i, :-(-t // case["page"])]
            k, v = (_values(s[x + "_codes"][layer, pages].flatten(0, 1), s[x + "_exps"][layer, pages].flatten(0, 1),
                            case["code"])[:t] for x in ("k", "v"))
            q = s["q"][layer, i * new:(i + 1) * new].float().reshape(new, kvh, h // kvh, dim).permute(1, 2, 0, 3)
            scores = torch.matmul(q.reshape(kvh, -1, dim), k.permute(1, 2, 0).contiguous()).view(kvh, h // kvh, new, t)
            scores = scores * dim ** -0.5
            late = torch.arange(t, device=DEV)[None] > torch.arange(t - new, t, device=DEV)[:, None]
            scores = scores.masked_fill(late, -math.inf)
            top = scores.amax(-1, keepdim=True)
            p = torch.exp(scores - top)
            total = p.sum(-1, keepdim=True)
            out = torch.matmul(p.view(kvh, -1, t), v.permute(1, 0, 2).contiguous()).view(kvh, h // kvh, new, dim) / total
            outs.append(out.permute(2, 0, 1, 3).reshape(new, h, dim))
            lses.append((top + torch.log(total))[..., 0].permute(2, 0, 1).reshape(new, h))
    return {"out": torch.cat(outs).to(s["q"].dtype).reshape(s["q"].shape), "lse": torch.cat(lses).reshape(s["q"].shape[:3])}


def _stored64(x, code):
    """Values [tokens][heads][dim] as blocks of 32 tokens of a head are stored, from the definition: fp64."""
    t, h, d = x.shape
    y = torch.cat([x.double(), torch.zeros(-t % GROUP, h, d, dtype=torch.float64, device=DEV)]).reshape(-1, GROUP, h, d)
    amax = y.abs().amax(dim=(1, 3), keepdim=True).clamp(min=2.0 ** -130)
    e = torch.ceil(torch.log2(amax / TOP[code]))
    e = torch.where(TOP[code] * torch.exp2(e - 1) >= amax, e - 1, e)
    e = torch.where(TOP[code] * torch.exp2(e) < amax, e + 1, e).clamp(min=-126)
    z = y / torch.exp2(e)
    if code == "int8":
        z = torch.round(z)
    else:
        step = torch.exp2((torch.frexp(z)[1] - 1).clamp(min=-6).double() - 3)
        z = torch.round(z / step) * step
    return (z * torch.exp2(e)).reshape(-1, h, d)[:t]


def _exact_shared(case, seed):
    x = _shared_inputs(case, seed)
    new, h, kvh, dim, page = case["new"], case["heads"], case["kv_heads"], case["dim"], case["page"]
    out = torch.empty(x["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(x["q"].shape[:3], dtype=torch.float64, device=DEV)
    for layer in range(case["layers"]):
        for i, t in enumerate(x["total"]):
            pages = torch.tensor(x["table"][i][:-(-t // page)], device=DEV)
            k, v = (_stored64(x[name][layer, pages].flatten(0, 1), case["code"])[:t] for name in ("k", "v"))
            hidden = torch.arange(t, device=DEV)[None] > torch.arange(t - new, t, device=DEV)[:, None]
            rows = slice(i * new, (i + 1) * new)
            for a in range(h):
                z = (x["q"][layer, rows, a].double() @ k[:, a // (h // kvh)].T) / math.sqrt(dim)
                z[hidden] = -math.inf
                lse[layer, rows, a] = torch.logsumexp(z, 1)
                out[layer, rows, a] = torch.softmax(z, 1) @ v[:, a // (h // kvh)]
    return {"out": out, "lse": lse}


# ---- one pass ------------------------------------------------------------------------------------------


def prepare(case, seed):
    return {"project": _prepare_project, "rotate": _prepare_rotate, "shared": _prepare_shared}[case["kind"]](case, seed)


def run(s):
    kind = s["case"]["kind"]
    if not own:
        return {"project": _plain_project, "rotate": _plain_rotate, "shared": _plain_shared}[kind](s)
    if kind == "project":
        s["linear"].forward(s["x"], s["y"], add=s["add"])
        return s["y"]
    if kind == "rotate":
        s["cache"].rotate(s["rope"], s["q"], s["q_out"], s["k"], s["k_out"], s["seqs"], s["starts"], q_norm=s["q_norm"],
                          k_norm=s["k_norm"], eps=EPS)
        return {"q": s["q_out"], "k": s["k_out"]}
    # a step: what is shared is found once, then every layer attends
    cache, new = s["cache"], s["case"]["new"]
    cache.share(s["seqs"], s["starts"], s["groups"], s["plan"])
    for layer in range(s["case"]["layers"]):
        cache.attend_shared(layer, s["q"][layer], s["out"][layer], s["seqs"], s["starts"], s["groups"], s["plan"],
                            max_new=new, max_rows=s["most"], lse=s["lse"][layer])
    return {"out": s["out"], "lse": s["lse"]}


def exact(case, seed):
    return {"project": _exact_project, "rotate": _exact_rotate, "shared": _exact_shared}[case["kind"]](case, seed)
