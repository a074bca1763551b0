"""Measured cases of the paged key/value operators: csa2_rotate, csa2_kv_append and csa2_kv_attn.

Each case is one call of one operator.  `run` computes it in elementary torch operations in 32 bits
(64 for angles) when `own` is false, and calls the library when it is true; `exact` is the definition
in 64 bits.  Layouts are those of include/csa2.h: pools [pages][kv_heads][64][dim], a page table
[batch][max_pages], new tokens packed one sequence after another with their bounds in `cu`.
"""
import math

import torch

own = False

PAGE = 64
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}


# ---------------------------------------------------------------- cases

def _rotate(name, tokens, heads, dim, rot, offset, neighbours, axes, dtype, inverse, far):
    return {"name": name, "op": "rotate", "tokens": tokens, "heads": heads, "dim": dim, "rot": rot, "offset": offset,
            "neighbours": neighbours, "axes": axes, "dtype": dtype, "inverse": inverse, "far": far}


def _append(name, batch, new, start, kv_heads, dim, rot, neighbours, axes, dtype, cache, ragged):
    return {"name": name, "op": "append", "batch": batch, "new": new, "start": start, "kv_heads": kv_heads, "dim": dim,
            "rot": rot, "neighbours": neighbours, "axes": axes, "dtype": dtype, "cache": cache, "ragged": ragged}


def _attend(name, batch, new, ctx, heads, kv_heads, dim, dtype, cache, window, ragged):
    return {"name": name, "op": "attend", "batch": batch, "new": new, "ctx": ctx, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "dtype": dtype, "cache": cache, "window": window, "ragged": ragged}


def listed():
    return [
        # the queries of one decode step of 16 sequences: latency
        _rotate("rotate_token", 16, 64, 128, 128, 0, False, 1, "bf16", False, 131072),
        # a chunk of latent queries (64 heads x 512) of which the last 64 channels rotate
        _rotate("rotate_latent_tail", 4096, 64, 512, 64, 448, True, 1, "bf16", False, 1048576),
        # image and video tokens with time, height and width axes; the inverse is the backward pass
        _rotate("rotate_axes_back", 8191, 16, 128, 128, 0, False, 3, "f16", True, 65536),
        # one new token for each of 16 sequences: latency
        _append("append_token", 16, 1, 2000, 8, 128, 128, False, 1, "bf16", "bf16", False),
        # the agent turn: 16 sessions bring 8,192 tokens each, into an 8-bit cache
        _append("append_turn_e4m3", 16, 8192, 1000, 8, 128, 128, False, 1, "bf16", "e4m3", False),
        # prompts of unequal length with three axes; some sequences bring nothing
        _append("append_ragged_axes", 9, 777, 5000, 4, 64, 32, True, 3, "f16", "f16", True),
        # one token of one short sequence: latency
        _attend("attend_token_short", 1, 1, 1000, 16, 2, 128, "bf16", "bf16", 0, False),
        # a decode step of 16 sequences of unequal length up to 32,768 tokens
        _attend("attend_token_long", 16, 1, 32768, 64, 8, 128, "bf16", "bf16", 0, True),
        # four drafted tokens of 8 sequences verified over 65,536 tokens in an 8-bit cache
        _attend("attend_drafts_e4m3", 8, 4, 65536, 64, 8, 128, "bf16", "e4m3", 0, False),
        # a prompt's chunk of 2,048 tokens over 16,384
        _attend("attend_chunk", 1, 2048, 16384, 64, 8, 128, "bf16", "bf16", 0, False),
        # prompts of unequal length through a layer that sees the last 128 tokens
        _attend("attend_ragged_window", 12, 512, 4096, 20, 4, 64, "f16", "f16", 128, True),
        # chunks of unequal length over an 8-bit cache
        _attend("attend_chunk_e4m3", 4, 1024, 8192, 32, 4, 128, "bf16", "e4m3", 0, True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    """One more case: the operator, then its sizes over the listed cases' whole range."""
    while True:
        op = rng.choice(("rotate", "append", "attend", "attend"))
        axes, pairs = rng.choice((1, 1, 3)), rng.random() < 0.5
        if op == "rotate":
            dim = rng.choice((64, 128, 512))
            rot = rng.choice((32, 64, dim if dim < 512 else 128))
            case = _rotate("", _log(rng, 1, 8192), _log(rng, 1, 128), dim, rot, rng.choice((0, dim - rot)), pairs, axes,
                           rng.choice(("bf16", "f16", "f32")), rng.random() < 0.5, _log(rng, 16, 1 << 20))
        elif op == "append":
            dim = rng.choice((64, 128))
            dtype = rng.choice(("bf16", "f16"))
            case = _append("", _log(rng, 1, 64), _log(rng, 1, 8192), _log(rng, 1, 8192), rng.choice((1, 2, 3, 4, 8)), dim,
                           rng.choice((0, 32, dim)), pairs, axes, dtype, rng.choice((dtype, "e4m3")), rng.random() < 0.6)
            case["axes"] = axes if case["rot"] else 1
        else:
            kv_heads = rng.choice((1, 2, 3, 4, 8))
            dtype = rng.choice(("bf16", "f16"))
            new = _log(rng, 1, 2048)
            case = _attend("", _log(rng, 1, 16), new, max(new, _log(rng, 64, 65536)),
                           kv_heads * rng.choice((1, 2, 4, 5, 7, 8, 16)), kv_heads, rng.choice((64, 128)), dtype,
                           rng.choice((dtype, "e4m3")), rng.choice((0, 0, 128, 1000)), rng.random() < 0.6)
        del case["name"]
        if _plain_bytes(case) <= _plain_bytes(listed()[9]) and work(case)["flops"] <= work(listed()[9])["flops"] and \
                work(case)["bytes"] <= work(listed()[7])["bytes"]:
            return case


def _plain_bytes(case):
    """Scores (or cache copies) that the plain form holds in 32 bits."""
    if case["op"] != "attend":
        return 0
    return max(4 * case["batch"] * case["heads"] * case["new"] * case["ctx"],
               4 * case["batch"] * case["kv_heads"] * case["dim"] * case["ctx"])


def _news(case):
    """New tokens of each sequence: `new`, or from `new` down to a single one, with one that brings none."""
    b, n = case["batch"], case["new"]
    if not case["ragged"]:
        return [n] * b
    got = [1 + (n - 1) * ((5 * i) % b) // max(1, b - 1) for i in range(b)]
    got[0] = n
    if b >= 4:
        got[2] = 0
    return got


def _before(case):
    """Tokens that each sequence holds before its new ones."""
    news = _news(case)
    most = case["start"] if case["op"] == "append" else case["ctx"]
    held = [most if not case["ragged"] else most - most * ((3 * i) % case["batch"]) // (case["batch"] + case["batch"] // 3 + 1)
            for i in range(case["batch"])]
    if case["op"] == "append":
        return held
    return [max(0, h - n) for h, n in zip(held, news)]


def _pairs(case):
    """(query, key) pairs that the masks leave, for one head."""
    total = 0
    for new, old in zip(_news(case), _before(case)):
        w = case["window"]
        if w == 0:
            total += new * old + new * (new + 1) // 2
        else:  # the i-th new token sees min(old + i + 1, w) keys
            short = max(0, min(new, w - old))
            total += short * old + short * (short + 1) // 2 + (new - short) * w
    return total


def work(case):
    s = SIZE[case["dtype"]]
    if case["op"] == "rotate":
        n = case["tokens"] * case["heads"]
        return {"bytes": 2 * n * case["dim"] * s + 4 * case["tokens"] * case["axes"], "flops": 3 * n * case["rot"]}
    news, old = _news(case), _before(case)
    width = case["kv_heads"] * case["dim"]
    if case["op"] == "append":
        n = sum(news)
        return {"bytes": 2 * n * width * (s + SIZE[case["cache"]]) + 4 * n * case["axes"],
                "flops": 3 * n * case["kv_heads"] * case["rot"]}
    seen = sum(min(n + o, n + case["window"] - 1 if case["window"] else n + o) for n, o in zip(news, old) if n)
    return {"bytes": 2 * sum(news) * case["heads"] * case["dim"] * s + 2 * seen * width * SIZE[case["cache"]],
            "flops": 4 * case["dim"] * case["heads"] * _pairs(case)}


# ---------------------------------------------------------------- inputs

def _normal(gen, shape, dtype):
    """N(0, 1) values; made in pieces, so that no large 32-bit copy is held."""
    x = torch.empty(shape, dtype=TYPES[dtype], device=DEV)
    flat = x.view(-1)
    for i in range(0, flat.numel(), 1 << 26):
        part = flat[i:i + (1 << 26)]
        part.copy_(torch.randn(part.numel(), generator=gen, device=DEV, dtype=torch.float32))
    return x


def _inv_freq(rot):
    i = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    return (10000.0 ** (-2.0 * i / max(rot, 1))).float()


def _axis_of(case):
    """The axis of each pair: the first half of them time, then height and width by turns."""
    half = case["rot"] // 2
    if case["axes"] == 1:
        return [0] * half
    return [0 if i < half // 2 else 1 + i % 2 for i in range(half)]


def _positions(case, first, gen):
    """int32 [axes][tokens]: the first axis counts up from `first`, the others walk an image of 64 columns."""
    n = first.numel()
    pos = [first]
    if case["axes"] == 3:
        shift = int(torch.randint(0, 1000, (1,), generator=gen, device=DEV))
        at = torch.arange(n, device=DEV) + shift
        pos += [at // 64 % 64, at % 64]
    return torch.stack(pos).int().contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    if case["op"] == "rotate":
        first = torch.randint(0, case["far"], (case["tokens"],), generator=gen, device=DEV)
        return {"case": case, "x": _normal(gen, (case["tokens"], case["heads"], case["dim"]), case["dtype"]),
                "pos": _positions(case, first, gen), "inv_freq": _inv_freq(case["rot"]), "axis": _axis_of(case),
                "axis_at": torch.tensor(_axis_of(case), device=DEV)}
    news, old = _news(case), _before(case)
    pages = [-(-(n + o) // PAGE) for n, o in zip(news, old)]
    table = torch.zeros(case["batch"], max(1, max(pages)), dtype=torch.int32)
    order = torch.randperm(sum(pages) + 3, generator=torch.Generator().manual_seed(seed)).int()
    at = 0
    for b, p in enumerate(pages):
        table[b, :p] = order[at:at + p]
        at += p
    shape = (sum(pages) + 3, case["kv_heads"], PAGE, case["dim"])
    total = sum(news)
    cu = torch.tensor([sum(news[:b]) for b in range(case["batch"] + 1)], dtype=torch.int32, device=DEV)
    held = torch.tensor(old, dtype=torch.int32, device=DEV)
    s = {"case": case, "table": table.to(DEV), "cu": cu, "total": total, "status": torch.zeros(4, dtype=torch.int32, device=DEV),
         "k_pages": _normal(gen, shape, case["cache"]), "v_pages": _normal(gen, shape, case["cache"])}
    if case["op"] == "append":
        s |= {"start": held, "n_tokens": held.clone(), "k": _normal(gen, (total, case["kv_heads"], case["dim"]), case["dtype"]),
              "v": _normal(gen, (total, case["kv_heads"], case["dim"]), case["dtype"])}
        first = torch.cat([torch.arange(o, o + n, device=DEV) for n, o in zip(news, old)])
        if case["rot"]:
            s |= {"pos": _positions(case, first, gen), "inv_freq": _inv_freq(case["rot"]), "axis": _axis_of(case),
                  "axis_at": torch.tensor(_axis_of(case), device=DEV)}
        return s
    s |= {"n_tokens": torch.tensor([n + o for n, o in zip(news, old)], dtype=torch.int32, device=DEV),
          "q": _normal(gen, (total, case["heads"], case["dim"]), case["dtype"]), "scale": 1.0 / math.sqrt(case["dim"])}
    return s


# ---------------------------------------------------------------- the plain form

def _turned(x, s, sign):
    """x [tokens][heads][dim] in 32 bits with its channels rotated; the angles in 64."""
    case = s["case"]
    off, rot = case.get("offset", 0), case["rot"]
    at = s["pos"][s["axis_at"]].double().t() * s["inv_freq"].double()
    cos, sin = at.cos().float()[:, None], (sign * at.sin()).float()[:, None]
    part = x[..., off:off + rot]
    if case["neighbours"]:
        a, b = part[..., 0::2], part[..., 1::2]
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
    a, b = a * cos - b * sin, b * cos + a * sin
    y = x.clone()
    if case["neighbours"]:
        y[..., off:off + rot] = torch.stack((a, b), -1).flatten(-2)
    else:
        y[..., off:off + rot] = torch.cat((a, b), -1)
    return y


def _plain_rotate(s):
    return _turned(s["x"].float(), s, -1.0 if s["case"]["inverse"] else 1.0).to(s["x"].dtype)


def _plain_append(s):
    token = torch.arange(s["total"], device=DEV)
    seq = torch.searchsorted(s["cu"][1:], token, right=True)
    slot = s["start"][seq] + token - s["cu"][seq]
    page = s["table"][seq, slot // PAGE].long()
    k = _turned(s["k"].float(), s, 1.0) if s["case"]["rot"] else s["k"].float()
    top = 448.0 if s["case"]["cache"] == "e4m3" else float("inf")
    s["k_pages"].permute(0, 2, 1, 3)[page, slot % PAGE] = k.clamp(-top, top).to(s["k_pages"].dtype)
    s["v_pages"].permute(0, 2, 1, 3)[page, slot % PAGE] = s["v"].float().clamp(-top, top).to(s["v_pages"].dtype)
    s["n_tokens"].copy_(s["start"] + s["cu"][1:] - s["cu"][:-1])
    return s["k_pages"], s["v_pages"], s["n_tokens"]


def _plain_attend(s):
    case, cu = s["case"], s["cu"]
    b, hk, d, new = case["batch"], case["kv_heads"], case["dim"], case["new"]
    g = case["heads"] // hk
    n = s["n_tokens"][:, None]
    news = (cu[1:] - cu[:-1])[:, None]
    k = s["k_pages"][s["table"]].float().transpose(1, 2).reshape(b, hk, -1, d)
    v = s["v_pages"][s["table"]].float().transpose(1, 2).reshape(b, hk, -1, d)
    key = torch.arange(k.shape[2], device=DEV)
    v = torch.where((key < n)[:, None, :, None], v, 0.0)
    i = torch.arange(new, device=DEV)
    row = (cu[:-1, None] + i).clamp(max=s["total"] - 1)
    at = n - news + i  # the position of each new token
    q = s["q"].float()[row].view(b, new, hk, g, d).permute(0, 2, 3, 1, 4).reshape(b, hk, g * new, d)
    x = (q @ k.transpose(2, 3)).mul_(s["scale"]).view(b, hk, g, new, -1)
    seen = key <= at[..., None]
    if case["window"]:
        seen &= key > at[..., None] - case["window"]
    x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(b, hk, g * new, -1) @ v).view(b, hk, g, new, d) / total.clamp(min=1e-30)
    lse = (top + total.log())[..., 0]
    token = torch.arange(s["total"], device=DEV)
    seq = torch.searchsorted(cu[1:], token, right=True)
    i = token - cu[seq]
    out = o.permute(0, 3, 1, 2, 4).reshape(b, new, hk * g, d)[seq, i]
    return out.to(s["q"].dtype), lse.permute(0, 3, 1, 2).reshape(b, new, hk * g)[seq, i]


# ---------------------------------------------------------------- the library's calls

def _own(s):
    import fp4_sparse_attention_pack_b200 as csa
    case = s["case"]
    if "rotary" not in s and case.get("rot"):  # a program makes its descriptors and workspaces once
        s["rotary"] = csa.rotary(s["inv_freq"], case["rot"], offset=case.get("offset", 0),
                                 neighbours=case["neighbours"], n_axes=case["axes"], axis=s["axis"])
    if case["op"] == "rotate":
        out = torch.empty_like(s["x"])
        csa.rotate(s["rotary"], s["x"], s["pos"], out, inverse=case["inverse"])
        return out
    if "cache" not in s:
        s["cache"] = csa.kv_cache(s["k_pages"], s["v_pages"], s["table"], s["n_tokens"], s["status"])
    if case["op"] == "append":
        csa.kv_append(s["cache"], s["k"], s["v"], s["cu"], case["new"], start=s["start"], rotary=s.get("rotary"), pos=s.get("pos"))
        return s["k_pages"], s["v_pages"], s["n_tokens"]
    if "ws" not in s:
        s["ws"] = torch.empty(csa.kv_attn_workspace(s["cache"], s["total"], case["new"], case["heads"]),
                              dtype=torch.uint8, device=DEV)
    out = torch.empty_like(s["q"])
    lse = torch.empty(s["total"], case["heads"], dtype=torch.float32, device=DEV)
    csa.kv_attn(s["cache"], s["q"], s["cu"], case["new"], s["scale"], out, s["ws"], lse=lse, window=case["window"])
    return out, lse


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_rotate(state) if op == "rotate" else _plain_append(state) if op == "append" else _plain_attend(state)


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_turn(x, s, case, sign):
    """Every pair of channels is a complex number that is multiplied by e^(i * angle)."""
    off, rot = case.get("offset", 0), case["rot"]
    axis = torch.tensor(s["axis"], device=DEV)
    angle = torch.stack([s["pos"].double()[int(a)] * f for a, f in zip(axis, s["inv_freq"].double())], 1)
    unit = torch.polar(torch.ones_like(angle), sign * angle)[:, None]
    y = x.double()
    part = y[..., off:off + rot]
    pair = (part.unflatten(-1, (rot // 2, 2)) if case["neighbours"] else part.unflatten(-1, (2, rot // 2)).transpose(-1, -2)).contiguous()
    z = torch.view_as_real(torch.view_as_complex(pair) * unit)
    y[..., off:off + rot] = z.flatten(-2) if case["neighbours"] else z.transpose(-1, -2).flatten(-2)
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotate":
        return _exact_turn(s["x"], s, case, -1.0 if case["inverse"] else 1.0)
    news, old = _news(case), _before(case)
    bounds, table = s["cu"].tolist(), s["table"].long()
    if case["op"] == "append":
        k = _exact_turn(s["k"], s, case, 1.0) if case["rot"] else s["k"].double()
        pools = []
        for new, pool in ((k, s["k_pages"]), (s["v"].double(), s["v_pages"])):
            pool = pool.double()
            for b, (n, o) in enumerate(zip(news, old)):
                at = torch.arange(o, o + n, device=DEV)
                pool[table[b, at // PAGE], :, at % PAGE] = new[bounds[b]:bounds[b + 1]]
            pools.append(pool)
        return pools[0], pools[1], None
    g = case["heads"] // case["kv_heads"]
    out = torch.zeros(s["total"], case["heads"], case["dim"], dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["total"], case["heads"], dtype=torch.float64, device=DEV)
    for b, (n, o) in enumerate(zip(news, old)):
        if n == 0:
            continue
        lo, hi = bounds[b], bounds[b + 1]
        pages = table[b, :-(-(n + o) // PAGE)]
        at = torch.arange(o, o + n, device=DEV)[:, None, None]
        key = torch.arange(n + o, device=DEV)
        seen = (key <= at) & (key > at - (case["window"] or n + o + 1))
        for h in range(case["kv_heads"]):
            k = s["k_pages"][pages, h].double().flatten(0, 1)[:n + o]
            v = s["v_pages"][pages, h].double().flatten(0, 1)[:n + o]
            x = s["q"][lo:hi, h * g:(h + 1) * g].double() @ k.t() * s["scale"]
            x = torch.where(seen, x, -math.inf)
            lse[lo:hi, h * g:(h + 1) * g] = torch.logsumexp(x, -1)
            out[lo:hi, h * g:(h + 1) * g] = torch.softmax(x, -1) @ v
    return out, lse
