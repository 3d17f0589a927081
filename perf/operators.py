"""The cases over which the operators of the 8-bit paged KV cache are measured,
each in a plain form (elementary torch operations) and as the framework's calls:

  attention  over the paged cache: prompts, chunks behind a prefix, single and
             few tokens; ragged lengths, GQA, causal and windowed
  append     of new keys (turned to their positions) and values, and the read
             of the written pages back to 16-bit values
  rope       rotary positions, forward and gradient
  pages      one step of a scheduler (free, fork, reserve with copy on write),
             and the live pages moved to the front of the pool

A case is a dict of plain values.  Lengths follow from the case alone, values
and page numbers from the seed.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
CODE = {"i8": torch.int8, "e4m3": torch.float8_e4m3fn}
CMAX = {"i8": 127.0, "e4m3": 448.0}
BASE, CTX, FACTOR, LOW, HIGH = 500000.0, 8192, 8.0, 1.0, 4.0


# ---------------------------------------------------------------- the cases

def listed():
    attn = {"op": "attention", "heads": 8, "group": 4, "d": 128, "page": 64, "window": 0,
            "causal": True, "dtype": "bf16"}
    app = {"op": "append", "heads": 8, "d": 128, "page": 64, "dtype": "bf16"}
    rope = {"op": "rope", "heads": 32, "d": 128}
    pages = {"op": "pages", "heads": 8, "d": 128, "page": 64}
    return [
        # one user's chat, single token: latency
        {**attn, "name": "attn_decode_one", "ns": 1, "kv_min": 500, "kv_max": 500, "q_min": 1,
         "q_max": 1, "fmt": "i8", "salt": 1},
        # a serving batch of unlike lengths, single tokens
        {**attn, "name": "attn_decode_batch", "ns": 64, "kv_min": 33, "kv_max": 8190, "q_min": 1,
         "q_max": 1, "fmt": "e4m3", "salt": 2},
        # the benchmark's long KV cache (8 heads x 131072 tokens) for a few users
        {**attn, "name": "attn_decode_long", "ns": 4, "kv_min": 131072, "kv_max": 131072,
         "q_min": 1, "q_max": 1, "fmt": "i8", "salt": 3},
        # a long prompt's chunk behind its cached prefix
        {**attn, "name": "attn_prompt_long", "ns": 1, "kv_min": 16384, "kv_max": 16384,
         "q_min": 4096, "q_max": 4096, "fmt": "i8", "salt": 4},
        # several ragged prompts in one call: smaller heads, a window, short pages
        {**attn, "name": "attn_prompt_ragged", "d": 64, "group": 3, "page": 32, "window": 1000,
         "ns": 9, "kv_min": 200, "kv_max": 3001, "q_min": 100, "q_max": 2000, "fmt": "e4m3",
         "dtype": "f16", "salt": 5},
        # every step of a serving batch writes one token a sequence
        {**app, "name": "append_decode", "ns": 64, "kv_min": 33, "kv_max": 2000, "q_min": 1,
         "q_max": 1, "fmt": "i8", "rot": 128, "layout": "half", "salt": 6},
        # prompts written into the cache
        {**app, "name": "append_prompt", "ns": 7, "kv_min": 1000, "kv_max": 9001, "q_min": 999,
         "q_max": 8192, "fmt": "e4m3", "rot": 64, "layout": "interleaved", "salt": 7},
        # the queries of a serving batch, far positions
        {**rope, "name": "rope_decode", "tokens": 64, "rot": 128, "layout": "half",
         "scaling": "parts", "dtype": "bf16", "back": False, "far": 131072},
        # the gradient over a training batch, part of the head
        {**rope, "name": "rope_train_back", "tokens": 16383, "rot": 64, "layout": "interleaved",
         "scaling": "none", "dtype": "f32", "back": True, "far": 8192},
        # beam search: the losers freed, the winners forked, a token reserved
        {**pages, "name": "pages_beam", "do": "step", "layers": 4, "parents": 4, "children": 12,
         "kv_min": 100, "kv_max": 1500, "grow": 1, "salt": 8},
        # parallel samples of a batch in a deep model
        {**pages, "name": "pages_samples", "do": "step", "layers": 16, "parents": 37,
         "children": 150, "kv_min": 50, "kv_max": 2500, "grow": 70, "salt": 9},
        # a fragmented pool brought together
        {**pages, "name": "pages_compact", "do": "compact", "layers": 4, "parents": 48,
         "children": 0, "kv_min": 10, "kv_max": 8000, "grow": 0, "salt": 10},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "rope", "pages"])
    salt = rng.randrange(1 << 30)
    if op == "rope":
        d = rng.choice([64, 128])
        tokens = _log(rng, 1, 16000)
        return {"op": op, "tokens": tokens, "heads": rng.choice([1, 2, 5, 8, 32]), "d": d,
                "rot": rng.choice([d, d // 2, 32]), "layout": rng.choice(["half", "interleaved"]),
                "scaling": rng.choice(["none", "linear", "ntk", "parts"]),
                "dtype": rng.choice(["bf16", "f16", "f32"]), "back": rng.random() < 0.4,
                "far": _log(rng, 64, 1000000)}
    heads, d = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    if op == "pages":
        compact = rng.random() < 0.4
        parents = _log(rng, 1, 40)
        hi = _log(rng, 20, 2500)
        return {"op": op, "heads": heads, "d": d, "page": page,
                "do": "compact" if compact else "step", "layers": rng.choice([1, 2, 4, 7]),
                "parents": parents, "children": 0 if compact else _log(rng, 1, 120),
                "kv_min": rng.randint(1, min(hi, 50)), "kv_max": hi,
                "grow": 0 if compact else rng.choice([1, 1, 3, 60, 200]), "salt": salt}
    fmt, dtype = rng.choice(["i8", "e4m3"]), rng.choice(["bf16", "bf16", "f16"])
    base = {"op": op, "heads": heads, "d": d, "page": page, "fmt": fmt, "dtype": dtype,
            "salt": salt}
    if op == "append":
        ns = _log(rng, 1, 64)
        new = rng.choice([1, 1, 4, _log(rng, 16, 16384 // ns + 16)])
        kv = new + _log(rng, 1, 4000)
        return {**base, "ns": ns, "kv_min": max(new, kv // 3), "kv_max": kv,
                "q_min": max(1, new // 2), "q_max": new, "rot": rng.choice([0, 32, d]),
                "layout": rng.choice(["half", "interleaved"])}
    ns, group = _log(rng, 1, 64), rng.choice([1, 2, 3, 4, 5, 7, 8])
    kv = _log(rng, 2, min(131072, 400000 // ns))
    q = rng.choice([1, 1, rng.randint(2, 8), _log(rng, 9, 3000)])
    q = max(1, min(q, kv, 400000000 // (ns * heads * group * kv)))
    return {**base, "group": group, "ns": ns, "kv_min": max(1, kv // rng.choice([1, 2, 20])),
            "kv_max": kv, "q_min": max(1, q // 2), "q_max": q,
            "window": rng.choice([0, 0, 0, _log(rng, 1, 4096)]), "causal": rng.random() < 0.9}


def _lengths(case):
    """(cache lengths, new tokens) of the sequences; both ends of a range occur."""
    r = random.Random(case["salt"])
    n = case.get("ns") or case["parents"]
    kv = [r.randint(case["kv_min"], case["kv_max"]) for _ in range(n)]
    kv[0] = case["kv_max"]
    if "q_max" not in case:
        return kv, [0] * n
    q = [r.randint(case["q_min"], case["q_max"]) for _ in range(n)]
    q[0] = case["q_max"]
    return kv, [min(a, b) for a, b in zip(q, kv)]


def _pages(case):
    """Pages of every sequence."""
    return [-(-n // case["page"]) for n in _lengths(case)[0]]


def _cow(case):
    """Which children copy a page of their parent in a step: one of the others
    still holds it (the parent itself does)."""
    kv = _lengths(case)[0]
    return [kv[i % len(kv)] % case["page"] > 0 for i in range(case["children"])]


def work(case):
    op = case["op"]
    if op == "rope":
        x = case["tokens"] * case["heads"] * case["d"]
        return {"bytes": 2 * x * DT[case["dtype"]].itemsize + 8 * case["tokens"],
                "flops": 3 * x * case["rot"] // case["d"]}
    row = case["heads"] * case["d"]
    if op == "pages":
        page = 2 * case["layers"] * (case["page"] * row + 4 * case["heads"])
        meta = 8 * sum(_pages(case))
        if case["do"] == "compact":
            moved = sum(_pages(case)) // 2
            return {"bytes": 2 * moved * page + meta, "flops": 0}
        return {"bytes": 2 * sum(_cow(case)) * page + meta, "flops": 0}
    kv, q = _lengths(case)
    if op == "append":
        new, size = sum(q), DT[case["dtype"]].itemsize
        read = sum(n - (n - m) // case["page"] * case["page"] for n, m in zip(kv, q))
        # new rows in, codes out; the written pages' codes in, their values out
        return {"bytes": 2 * row * (new * (size + 1) + read * (1 + size)), "flops": 6 * row * new}
    seen = reach = 0
    for n, m in zip(kv, q):
        w = case["window"] or n
        lo, hi = n - m, n - 1  # the queries' positions
        if not case["causal"]:
            seen, reach = seen + n * m, reach + n
            continue
        full = max(0, hi - max(lo, w - 1) + 1)
        part = m - full
        seen += full * w + part * (lo + 1) + part * (part - 1) // 2
        reach += n - max(0, lo - w + 1)
    size = DT[case["dtype"]].itemsize
    return {"bytes": 2 * row * reach + 2 * sum(q) * row * case["group"] * size,
            "flops": 4 * case["d"] * case["heads"] * case["group"] * seen}


# ---------------------------------------------------------------- the inputs

def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype).to(DEV)


def _cu(counts):
    out = [0]
    for c in counts:
        out.append(out[-1] + c)
    return _ints(out)


def _tables(case, g, rows, spare):
    """A table of `rows` rows over scattered page numbers and the pages' counts."""
    need = _pages(case)
    pool = sum(need) + spare
    ids = torch.randperm(pool, generator=g, device=DEV)[:sum(need)].to(torch.int32)
    width = max(need) + 4 + case.get("grow", 0) // case["page"]
    table = torch.full((rows, width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = ids[at:at + n]
        at += n
    refs = torch.zeros(pool, dtype=torch.int32, device=DEV)
    refs[ids.long()] = 1
    return table, refs, pool


def _codes(case, g, shape):
    """Random codes as a cache of activations holds them."""
    x = torch.empty(shape, dtype=CODE[case.get("fmt", "i8")], device=DEV)
    for layer in x:  # a layer at a time: bounded 32-bit intermediates
        step = max(1, (1 << 27) // layer[0].numel())
        for at in range(0, layer.shape[0], step):
            part = layer[at:at + step]
            v = torch.randn(part.shape, generator=g, device=DEV)
            if x.dtype == torch.int8:
                part.copy_((v * 40).round_().clamp_(-127, 127))
            else:
                part.copy_((v * 120).clamp_(-448, 448))
    return x


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op, s = case["op"], {"case": dict(case)}
    if op == "rope":
        s["x"] = torch.randn(case["tokens"], case["heads"], case["d"], generator=g,
                             device=DEV).to(DT[case["dtype"]])
        s["pos"] = torch.randint(0, case["far"], (case["tokens"],), generator=g, device=DEV)
        s["rope"] = _rope_params(case)
    else:
        kv, q = _lengths(case)
        rows = len(kv) + case.get("children", 0)
        spare = (case["children"] * (2 + case["grow"] // case["page"]) + 5 if "children" in case
                 else 3)
        if case.get("do") == "compact":
            spare = sum(_pages(case))
        table, refs, pool = _tables(case, g, rows, spare)
        shape = (case.get("layers", 1), pool, case["heads"], case["page"], case["d"])
        s["k"], s["v"] = _codes(case, g, shape), _codes(case, g, shape)
        unit = 40.0 if case.get("fmt", "i8") == "i8" else 120.0
        for name in ("kscale", "vscale"):
            s[name] = (torch.rand(shape[:3], generator=g, device=DEV) + 0.5) / unit
        s["table"], s["refs"] = table, refs
        s["lens"] = _ints(kv + [0] * case.get("children", 0))
        s["list"], s["cu"], s["maxq"], s["maxkv"] = q, _cu(q), max(q), max(kv)
        if s["k"].dtype != torch.int8 and op == "attention":
            # rows behind a sequence's end were never written: any bytes, NaN among them
            for i, n in enumerate(kv):
                if n % case["page"]:
                    last = int(table[i, n // case["page"]])
                    for t in (s["k"], s["v"]):
                        t.view(torch.uint8)[:, last, :, n % case["page"]:] = 0x7F
        if op == "attention":
            s["q"] = torch.randn(sum(q), case["heads"] * case["group"], case["d"], generator=g,
                                 device=DEV).to(DT[case["dtype"]])
        elif op == "append":
            new = (sum(q), case["heads"], case["d"])
            s["new_k"], s["new_v"] = (torch.randn(new, generator=g, device=DEV)
                                      .to(DT[case["dtype"]]) for _ in "kv")
            s["pos"] = torch.cat([torch.arange(n - m, n) for n, m in zip(kv, q)]).to(DEV)
            begin = [(n - m) // case["page"] * case["page"] for n, m in zip(kv, q)]
            s["begin"], back = _ints(begin), [n - b for n, b in zip(kv, begin)]
            s["cu_back"], s["total_back"], s["max_back"] = _cu(back), sum(back), max(back)
            s["rope"] = _rope_params(case) if case["rot"] else None
        else:
            s["table0"], s["refs0"], s["lens0"] = table.clone(), refs.clone(), s["lens"].clone()
            n, c = case["parents"], case["children"]
            s["parents"] = _ints([i % n for i in range(c)])
            s["children"] = _ints([n + i for i in range(c)])
            s["zero"], s["grow"] = _ints([0] * c), _ints([case["grow"]] * c)
    if own:
        import kv_cache_embedding_b200 as tq
        if op != "rope":
            s["cache"] = tq.KV8Cache(s["k"], s["v"], s["kscale"], s["vscale"], s["table"],
                                     s["lens"], s["refs"])
        if s.get("rope"):
            s["rope"] = tq.Rope(**s["rope"])
    return s


def _rope_params(case):
    kind = case.get("scaling", "none")
    p = {"d": case["d"], "rot": case["rot"], "base": BASE, "layout": case["layout"],
         "scaling": kind}
    if kind != "none":
        p["factor"] = FACTOR
    if kind == "parts":
        p.update(ctx=CTX, low=LOW, high=HIGH, amplitude=0.1 * math.log(FACTOR) + 1.0)
    return p


# ---------------------------------------------------------------- the plain forms

def _freqs(p):
    i = torch.arange(0, p["rot"], 2, dtype=torch.float64, device=DEV) / p["rot"]
    base = p["base"]
    if p["scaling"] == "ntk":
        base = base * p["factor"] ** (p["rot"] / (p["rot"] - 2))
    f = base ** -i
    if p["scaling"] == "linear":
        f = f / p["factor"]
    if p["scaling"] == "parts":
        g = ((p["ctx"] * f / (2 * math.pi) - p["low"]) / (p["high"] - p["low"])).clamp(0, 1)
        f = f * (g + (1 - g) / p["factor"])
    return f


def _turn(x, pos, p, back):
    """x [T, H, d] fp32, turned (back: by the transpose) at positions pos [T]."""
    angle = pos.double()[:, None] * _freqs(p)
    a = p.get("amplitude", 1.0)
    c, s = (angle.cos() * a).float()[:, None], (angle.sin() * a).float()[:, None]
    if back:
        s = -s
    r = p["rot"]
    half = p["layout"] == "half"
    x1, x2 = (x[..., :r // 2], x[..., r // 2:r]) if half else (x[..., 0:r:2], x[..., 1:r:2])
    y1, y2 = x1 * c - x2 * s, x2 * c + x1 * s
    y = torch.cat([y1, y2], -1) if half else torch.stack([y1, y2], -1).flatten(-2)
    return torch.cat([y, x[..., r:]], -1)


def _gathered(codes, scale, ids):
    """fp32 values [n, heads, tokens, d] of the pages ids [n, p]."""
    x = codes[ids].float() * scale[ids][..., None, None]  # [n, p, heads, page, d]
    n, p, h, t, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(n, h, p * t, d)


def _attention(s):
    case = s["case"]
    ids = s["table"].clamp_min(0).long()[:, :-(-s["maxkv"] // case["page"])]
    keys = _gathered(s["k"][0], s["kscale"][0], ids)
    vals = _gathered(s["v"][0], s["vscale"][0], ids)
    n, h, t, d = keys.shape
    g, m = case["group"], s["maxq"]
    lens, counts = s["lens"].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    j, i = torch.arange(t, device=DEV), torch.arange(m, device=DEV)
    vals = torch.where((j < lens[:, None])[:, None, :, None], vals, 0.0)
    row = (s["cu"][:-1, None] + i).clamp_max(s["q"].shape[0] - 1)  # [n, m]
    q = s["q"][row].float().reshape(n, m, h, g, d).permute(0, 2, 3, 1, 4).reshape(n, h, g * m, d)
    at = lens[:, None] - counts[:, None] + i  # the queries' positions
    see = (j < lens[:, None, None]).expand(n, m, t)
    if case["causal"]:
        see = see & (j <= at[..., None])
        if case["window"]:
            see = see & (j > at[..., None] - case["window"])
    logits = (q @ keys.transpose(2, 3)).mul_(d ** -0.5).reshape(n, h, g, m, t)
    logits = logits.masked_fill_(~see[:, None, None], -math.inf)
    top = logits.amax(-1, keepdim=True)
    e = logits.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    total = e.sum(-1, keepdim=True)
    out = (e.reshape(n, h, g * m, t) @ vals).reshape(n, h, g, m, d) / total.clamp_min(1e-30)
    out = out.permute(0, 3, 1, 2, 4).reshape(n, m, h * g, d)
    seq = torch.repeat_interleave(torch.arange(n, device=DEV), counts,
                                  output_size=s["q"].shape[0])
    return out[seq, torch.arange(s["q"].shape[0], device=DEV) - s["cu"][seq]].to(s["q"].dtype)


def _store(x, like):
    if like.dtype == torch.int8:
        return x.round().clamp(-127, 127).to(torch.int8)
    return x.clamp(-448, 448).to(torch.float32).to(like.dtype)


def _write(s, codes, scale, x, first, seq):
    """New rows x [T, H, d] at s["pos"]; first: the page of each sequence's first
    new token and the tokens that it holds already."""
    case, peak = s["case"], CMAX[s["case"]["fmt"]]
    page = s["table"][seq, s["pos"] // case["page"]].long()  # [T]
    held, old = first
    known = torch.zeros_like(scale)
    known[held] = torch.where(old[:, None] > 0, scale[held], 0.0)
    amax = torch.zeros_like(scale).index_reduce_(0, page, x.abs().amax(-1), "amax")
    touched = torch.zeros(scale.shape[0], dtype=torch.bool, device=DEV)
    touched[page] = True
    new = torch.where(touched[:, None], torch.maximum(known, amax / peak), scale)
    # the tokens that were there already, where their scale has grown
    rows = codes[held].float()  # [n, H, page, d]
    ratio = (known[held].double() / new[held].double()).nan_to_num(0.0)
    grown = new[held] > known[held]
    keep = torch.arange(case["page"], device=DEV) < old[:, None]
    again = _store(rows.double() * ratio[..., None, None], codes)
    both = grown[:, :, None, None] & keep[:, None, :, None]
    codes[held] = torch.where(both, again.view(torch.int8),
                              codes[held].view(torch.int8)).view(codes.dtype)
    step = new[page].double()[..., None]
    row = torch.where(step > 0, x.double() / step, 0.0)
    codes.view(torch.int8)[page, :, s["pos"] % case["page"]] = _store(row, codes).view(torch.int8)
    scale.copy_(new)


def _append(s):
    case = s["case"]
    lens, counts = s["lens"].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    n, total = lens.shape[0], s["new_k"].shape[0]
    seqs = torch.arange(n, device=DEV)
    seq = torch.repeat_interleave(seqs, counts, output_size=total)
    start = lens - counts
    first = s["table"][seqs, start // case["page"]].long(), start % case["page"]
    k = s["new_k"].float()
    if s["rope"]:
        k = _turn(k, s["pos"], s["rope"], False)
    _write(s, s["k"][0], s["kscale"][0], k, first, seq)
    _write(s, s["v"][0], s["vscale"][0], s["new_v"].float(), first, seq)
    # the written pages read back
    back = (s["cu_back"][1:] - s["cu_back"][:-1]).long()
    seq = torch.repeat_interleave(seqs, back, output_size=s["total_back"])
    at = torch.arange(s["total_back"], device=DEV) - s["cu_back"][seq] + s["begin"][seq]
    page = s["table"][seq, at // case["page"]].long()
    dt = s["new_k"].dtype
    return [(c[0].view(torch.uint8)[page, :, at % case["page"]].view(c.dtype).float() *
             t[0][page][..., None]).to(dt)
            for c, t in ((s["k"], s["kscale"]), (s["v"], s["vscale"]))]


def _free_ids(refs, count):
    """The `count` lowest-numbered free pages."""
    return torch.argsort((refs != 0).to(torch.int8), stable=True)[:count]


def _pages_step(s):
    case, table, refs, lens = s["case"], s["table"], s["refs"], s["lens"]
    page, kids, n = case["page"], s["children"].long(), case["children"]
    # truncate to 0
    rows = table[kids]
    refs.index_add_(0, rows.clamp_min(0).flatten().long(), -(rows >= 0).int().flatten())
    table[kids] = -1
    lens[kids] = 0
    # fork
    rows = table[s["parents"].long()]
    refs.index_add_(0, rows.clamp_min(0).flatten().long(), (rows >= 0).int().flatten())
    table[kids] = rows
    lens[kids] = lens[s["parents"].long()]
    # reserve: shared first pages are copied, new pages taken in list order
    start = lens[kids].long()
    held = table[kids, start // page].long()
    order = torch.arange(n, device=DEV)
    earlier = ((held[:, None] == held) & (order[:, None] > order)).sum(1)
    copy = (start % page > 0) & (refs[held.clamp_min(0)] - earlier > 1)
    had, has = -(-start // page), -(-(start + case["grow"]) // page)
    need = copy.long() + has - had
    most = case["grow"] // page + 2
    free = _free_ids(refs, n * most)
    base = need.cumsum(0) - need
    dst = torch.where(copy, free[base], held.clamp_min(0))
    src = held.clamp_min(0)
    take = torch.where(copy)[0]
    for t in (s["k"], s["v"], s["kscale"], s["vscale"]):
        t = t.view(torch.int8) if t.element_size() == 1 else t
        t[:, dst[take]] = t[:, src[take]]
    refs.index_add_(0, src, -copy.int())
    refs[dst[take]] = 1
    table[kids[take], (start // page)[take]] = dst[take].int()
    step = torch.arange(most, device=DEV)
    fresh = step < (has - had)[:, None]
    at, which = torch.where(fresh)
    new = free[base[at] + copy[at].long() + which]
    refs[new] = 1
    table[kids[at], had[at] + which] = new.int()
    lens[kids] = (start + case["grow"]).int()
    return [table, refs, lens, s["k"], s["v"], s["kscale"], s["vscale"]]


def _compact(s):
    table, refs = s["table"], s["refs"]
    live = refs > 0
    ids = torch.arange(refs.shape[0], device=DEV)
    low = ids < live.sum()
    src, dst = torch.where(live & ~low)[0], torch.where(~live & low)[0]
    for t in (s["k"], s["v"], s["kscale"], s["vscale"]):
        t[:, dst] = t[:, src]
    ids[src] = dst
    refs[dst] = refs[src]
    refs[src] = 0
    table.copy_(torch.where(table >= 0, ids[table.clamp_min(0).long()].int(), table))
    return [table, refs, s["k"], s["v"], s["kscale"], s["vscale"]]


def run(s):
    case, op = s["case"], s["case"]["op"]
    if op == "attention":
        if own:
            return s["cache"].attention(0, s["q"], s["cu"], s["maxq"], causal=case["causal"],
                                        window=case["window"] if case["causal"] else 0)
        return _attention(s)
    if op == "append":
        if own:
            c = s["cache"]
            c.append(0, s["new_k"], s["new_v"], s["cu"], s["maxq"], rope=s["rope"])
            return c.read(0, s["begin"], s["cu_back"], s["total_back"], s["max_back"],
                          dtype=s["new_k"].dtype)
        return _append(s)
    if op == "rope":
        if own:
            return s["rope"].apply(s["x"], s["pos"], transpose=case["back"])
        return _turn(s["x"].float(), s["pos"], s["rope"], case["back"]).to(s["x"].dtype)
    if case["do"] == "step":
        if own:
            c = s["cache"]
            c.truncate(s["children"], s["zero"])
            c.fork(s["parents"], s["children"])
            c.reserve(s["children"], s["grow"])
            return [c.table, c.refs, c.lens, c.k, c.v, c.kscale, c.vscale]
        return _pages_step(s)
    # the fragmented tables again: a pool that is compact already moves nothing
    s["table"].copy_(s["table0"])
    s["refs"].copy_(s["refs0"])
    if own:
        c = s["cache"]
        c.compact()
        return [c.table, c.refs, c.k, c.v, c.kscale, c.vscale]
    return _compact(s)


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """The definition in 64 bits, a sequence at a time.  Pages only move whole
    numbers: None."""
    if case["op"] == "pages":
        return None
    global own
    keep, own = own, False
    s = prepare(case, seed)
    own = keep
    return {"attention": _exact_attention, "append": _exact_append,
            "rope": _exact_rope}[case["op"]](s)


def _exact_rotate(x, pos, p, back):
    r, out = p["rot"], x.clone()
    for i in range(r // 2):
        base = p["base"] * (p["factor"] ** (r / (r - 2)) if p["scaling"] == "ntk" else 1.0)
        f = base ** (-2.0 * i / r)
        if p["scaling"] == "linear":
            f /= p["factor"]
        if p["scaling"] == "parts":
            turns = p["ctx"] / (2 * math.pi / f)
            g = min(1.0, max(0.0, (turns - p["low"]) / (p["high"] - p["low"])))
            f = (1 - g) * f / p["factor"] + g * f
        a, b = (i, i + r // 2) if p["layout"] == "half" else (2 * i, 2 * i + 1)
        z = torch.polar(torch.full(pos.shape, p.get("amplitude", 1.0), dtype=torch.float64,
                                   device=DEV), (-1 if back else 1) * pos.double() * f)
        y = torch.complex(x[..., a], x[..., b]) * z[:, None]
        out[..., a], out[..., b] = y.real, y.imag
    return out


def _exact_rope(s):
    return _exact_rotate(s["x"].double(), s["pos"], s["rope"], s["case"]["back"])


def _exact_values(s, name, i, n):
    """[heads, n, d] fp64 of sequence i."""
    ids = s["table"][i, :-(-n // s["case"]["page"])].long()
    x = s[name][0][ids].double() * s[name + "scale"][0][ids].double()[..., None, None]
    return x.transpose(0, 1).flatten(1, 2)[:, :n]


def _exact_attention(s):
    case, out = s["case"], []
    lens, w = s["lens"].tolist(), s["case"]["window"]
    for i, m in enumerate(s["list"]):
        n = lens[i]
        k, v = _exact_values(s, "k", i, n), _exact_values(s, "v", i, n)
        q = s["q"][int(s["cu"][i]):][:m].double()
        pos, j = torch.arange(n - m, n, device=DEV)[:, None], torch.arange(n, device=DEV)
        hide = (j > pos) if case["causal"] else torch.zeros_like(j > pos)
        if w and case["causal"]:
            hide = hide | (j <= pos - w)
        rows = []
        for h in range(q.shape[1]):
            l = q[:, h] @ k[h // case["group"]].T / math.sqrt(case["d"])
            p = torch.softmax(l.masked_fill_(hide, -math.inf), -1)
            rows.append(p @ v[h // case["group"]])
        out.append(torch.stack(rows, 1))
    return torch.cat(out)


def _exact_append(s):
    case, page, peak = s["case"], s["case"]["page"], CMAX[s["case"]["fmt"]]
    lens, out = s["lens"].tolist(), []
    for name in "kv":
        rows = s["new_" + name].double()
        if name == "k" and s["rope"]:
            rows = _exact_rotate(rows, s["pos"], s["rope"], False)
        got = []
        for i, m in enumerate(s["list"]):
            n, x = lens[i], rows[int(s["cu"][i]):][:m]
            start = n - m
            for at in range(start // page * page, n, page):
                lo, hi = max(at, start), min(at + page, n)
                new = x[lo - start:hi - start].transpose(0, 1)  # [heads, tokens, d]
                step = new.abs().amax((1, 2)) / peak
                if lo > at:
                    p = int(s["table"][i, at // page])
                    old, was = s[name][0, p, :, :lo - at].double(), s[name + "scale"][0, p].double()
                    grown = torch.maximum(step, was)
                    again = _exact_round(old * (was / grown)[:, None, None], case)
                    old = torch.where((grown > was)[:, None, None], again, old)
                    step = grown
                new = _exact_round(new / step[:, None, None].clamp_min(1e-300), case)
                codes = torch.cat([old, new], 1) if lo > at else new
                got.append((codes * step[:, None, None]).transpose(0, 1))
        out.append(torch.cat(got))
    return out


def _exact_round(x, case):
    """To the nearest code, ties to even."""
    if case["fmt"] == "i8":
        return x.round().clamp(-127, 127)
    _, e = torch.frexp(x)
    unit = torch.ldexp(torch.ones_like(x), e.clamp_min(-5) - 4)  # 3 mantissa bits, down to 2^-9
    return ((x / unit).round() * unit).clamp(-448, 448)
