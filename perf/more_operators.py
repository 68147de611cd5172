"""The prompt-step operators next to the Q8_0 matmuls, as cases that can be timed and compared.

A prompt, or a chunk of one, goes through a layer in these steps around the matmuls of this
library: the residual's addition and the norm (q8_rms_norm, its output in bf16 or in Q8_0),
pages, slots and positions of the new tokens (q8_kv_plan), rotary positions (q8_rope; with the
write of keys and values into the paged Q8_0 cache in one, q8_rope_append), and attention of the
chunk's tokens over that cache (q8_attn_chunk).  Each has a plain form here, of elementary torch
operations in 32 bits (angles in 64), and a definition in 64 bits (`exact`).

`own` picks what `run` calls: the plain form (False) or the library's entry points (True).
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # one decode row of this library's layer width: fp32 matmul output onto an fp32 residual
        {"name": "norm_1", "op": "norm", "rows": 1, "width": 1536, "bf16": False, "res": "f32", "offset": 0.0, "q8": False},
        # a prompt chunk of odd length, bf16 onto bf16, gains stored less one, 8 bits with scales beside the bf16 rows
        {"name": "norm_4099_q8", "op": "norm", "rows": 4099, "width": 4096, "bf16": True, "res": "bf16", "offset": 1.0, "q8": True},
        # draft tokens to be checked: a quarter of each narrow head turns, pairs interleaved, far into a context
        {"name": "rope_5", "op": "rope", "tokens": 5, "heads": 40, "head_dim": 64, "rot": 16, "interleaved": True, "bf16": False,
         "far": 200000, "base": 10000.0, "yarn": 0.0},
        # a long prompt's query and key heads side by side, half layout, the whole head
        {"name": "rope_8192", "op": "rope", "tokens": 8192, "heads": 40, "head_dim": 128, "rot": 128, "interleaved": False,
         "bf16": True, "far": 0, "base": 500000.0, "yarn": 0.0},
        # one new token of one sequence: 12 heads of 128, rotated and written to the cache as a matmul leaves them
        {"name": "rope_append_1", "op": "rope_append", "tokens": 1, "q_heads": 12, "kv_heads": 12, "head_dim": 128, "rot": 128,
         "interleaved": False, "bf16": False, "page": 16, "pages": 64, "holes": False, "far": 3000, "base": 10000.0, "yarn": 0.0},
        # a prompt chunk to scattered pages, positions stretched for a long context
        {"name": "rope_append_4096", "op": "rope_append", "tokens": 4096, "q_heads": 32, "kv_heads": 8, "head_dim": 128, "rot": 128,
         "interleaved": False, "bf16": True, "page": 64, "pages": 1024, "holes": False, "far": 100000, "base": 10000.0, "yarn": 16.0},
        # a decode step's bookkeeping: 48 sequences, one new token each
        {"name": "plan_48", "op": "plan", "batch": 48, "max_new": 1, "max_len": 6000, "page": 16, "pad": 0},
        # a step that mixes prompts with single tokens: 300 sequences, some without new tokens, padded for a graph
        {"name": "plan_300", "op": "plan", "batch": 300, "max_new": 400, "max_len": 4000, "page": 32, "pad": 1000},
        # draft tokens of a serving batch: 1 to 5 new tokens each over caches of up to 6000
        {"name": "chunk_16x5", "op": "attn", "batch": 16, "q_heads": 32, "kv_heads": 8, "head_dim": 128, "page": 16, "max_new": 5,
         "max_len": 6000, "whole": False, "window": 0, "softcap": 0.0, "pad": 0},
        # a prompt by itself
        {"name": "chunk_4096", "op": "attn", "batch": 1, "q_heads": 32, "kv_heads": 8, "head_dim": 128, "page": 64, "max_new": 4096,
         "max_len": 4096, "whole": True, "window": 0, "softcap": 0.0, "pad": 0},
        # sliding window, capped scores and wide heads, 3 query heads to a key head, prompts of odd lengths, padded
        {"name": "chunk_window_cap", "op": "attn", "batch": 9, "q_heads": 12, "kv_heads": 4, "head_dim": 256, "page": 32, "max_new": 701,
         "max_len": 3001, "whole": False, "window": 1000, "softcap": 30.0, "pad": 57},
        # a chunk of 1024 deep in a context of 65,536 tokens
        {"name": "chunk_1024x65536", "op": "attn", "batch": 1, "q_heads": 32, "kv_heads": 8, "head_dim": 128, "page": 64,
         "max_new": 1024, "max_len": 65536, "whole": False, "window": 0, "softcap": 0.0, "pad": 0},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "rope", "rope_append", "plan", "attn", "attn"])
    if op == "norm":
        width = 32 * _log(rng, 2, 512)
        return {"op": op, "rows": _log(rng, 1, 4099 * 4096 // width), "width": width, "bf16": rng.random() < 0.5,
                "res": rng.choice(["none", "f32", "bf16"]), "offset": rng.choice([0.0, 1.0]), "q8": rng.random() < 0.5}
    if op in ("rope", "rope_append"):
        d = rng.choice([64, 128, 256])
        c = {"op": op, "tokens": _log(rng, 1, 4096), "head_dim": d, "rot": rng.choice([d, d, d // 2, d // 4]),
             "interleaved": rng.random() < 0.4, "bf16": rng.random() < 0.5, "far": rng.choice([0, 0, 3000, 100000, 1000000]),
             "base": rng.choice([10000.0, 500000.0]), "yarn": rng.choice([0.0, 0.0, 4.0, 32.0])}
        if op == "rope":
            c["heads"] = _log(rng, 1, 40 * 128 // d)
            return c
        kv, page = rng.randint(1, 8 * 128 // d), rng.choice([16, 32, 64, 128, 256])
        c.update(kv_heads=kv, q_heads=kv * rng.choice([1, 2, 3, 4]), page=page, pages=-(-c["tokens"] // page) + rng.randint(1, 64),
                 holes=rng.random() < 0.3)
        return c
    if op == "plan":
        batch, page = _log(rng, 1, 512), rng.choice([16, 32, 64, 128])
        return {"op": op, "batch": batch, "max_new": _log(rng, 1, min(4000, 120000 // batch)), "max_len": _log(rng, 1, 6000),
                "page": page, "pad": rng.choice([0, 0, 7, 1000])}
    hd, kv = rng.choice([64, 128, 256]), rng.randint(1, 8)
    group = rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 12, 16])
    most = 1024 * 65536 * 32 * 128 // (hd * kv * group)  # pairs of a new token and a token before it, by the largest's cost
    batch = _log(rng, 1, 32)
    new = _log(rng, 1, 2048)
    while batch * new * new > most:
        new //= 2
    # the cache holds as many values as four of the largest's at most
    length = _log(rng, 1, max(1, min(65536, most // (batch * new), 4 * 65536 * 8 * 128 // (batch * kv * hd))))
    return {"op": op, "batch": batch, "q_heads": kv * group, "kv_heads": kv, "head_dim": hd, "page": rng.choice([16, 32, 64, 128]),
            "max_new": min(new, length), "max_len": length, "whole": rng.random() < 0.3,
            "window": _log(rng, 1, 4096) if rng.random() < 0.25 else 0, "softcap": 30.0 if rng.random() < 0.25 else 0.0,
            "pad": rng.choice([0, 0, 3, 100])}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _quantised(w):
    """Q8_0 of fp32 w[..., K] for inputs: int8 codes and binary16 scales (|w| / s rounded half away from zero)."""
    b = w.reshape(*w.shape[:-1], w.shape[-1] // 32, 32)
    s = (b.abs().amax(-1) / 127.0).to(torch.float16)
    d = s.to(torch.float32).clamp_min(1e-30).unsqueeze(-1)
    q = torch.floor(b.abs().div_(d).add_(0.5)).clamp_max_(127.0).mul_(torch.sign(b))
    return q.to(torch.int8).reshape(w.shape).contiguous(), s.contiguous()


def _seqs(c):
    """New tokens of each sequence, and its tokens with them."""
    r = random.Random(c["batch"] * 1000003 + c["max_len"] * 31 + c["max_new"])
    if c["op"] == "plan":
        new = [r.randint(0, c["max_new"]) if r.random() < 0.8 else 0 for _ in range(c["batch"])]
        if c["max_new"] == 1:
            new = [1] * c["batch"]
        return new, [n + r.randint(0, c["max_len"]) for n in new]
    new = [r.randint(1, c["max_new"]) for _ in range(c["batch"])]
    new[r.randrange(c["batch"])] = c["max_new"]
    if c["whole"]:  # prompts from their first token on
        return new, list(new)
    lens = [r.randint(n, c["max_len"]) for n in new]
    lens[new.index(c["max_new"])] = c["max_len"]
    if c["batch"] > 2:  # one sequence takes no part
        at = new.index(min(new))
        if new[at] < c["max_new"]:
            new[at] = 0
    return new, lens


def _frequencies(c):
    """Radians a token for each pair of dimensions, and the factor on cosines and sines (64 bits)."""
    rot, base = c["rot"], c["base"]
    f = torch.tensor([base ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64)
    if c["yarn"] == 0.0:
        return f, 1.0
    # long contexts: pairs that turn less than once in the 4096 tokens of training are stretched, those
    # that turn more than 32 times kept, and a ramp leads from one to the other
    def pair(turns):
        return rot * math.log(4096.0 / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))
    lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), rot - 1)
    ramp = ((torch.arange(rot // 2, dtype=torch.float64) - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
    return f / c["yarn"] * ramp + f * (1.0 - ramp), 0.1 * math.log(c["yarn"]) + 1.0


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 13)

    def rn(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)

    c = dict(case)
    st = {"case": c}
    kind = torch.bfloat16 if c.get("bf16") else torch.float32
    if c["op"] == "norm":
        x = rn(c["rows"], c["width"])
        x[:, 5] *= 20.0  # a few channels stand out
        st["x"] = x.to(kind)
        st["weight"] = rn(c["width"]).mul_(0.2).add_(1.0 - c["offset"])
        if c["res"] != "none":
            st["residual"] = rn(c["rows"], c["width"]).mul_(3.0).to(torch.bfloat16 if c["res"] == "bf16" else torch.float32)
            st["residual_out"] = torch.empty_like(st["residual"])
    elif c["op"] in ("rope", "rope_append"):
        t, d = c["tokens"], c["head_dim"]
        f, st["factor"] = _frequencies(c)
        st["inv_freq"] = f.to(DEV)
        first = int(torch.randint(0, 1000, (1,), generator=g, device=DEV)) + c["far"]
        st["positions"] = torch.arange(first, first + t, device=DEV, dtype=torch.int32)
        if c["op"] == "rope":
            st["x"] = rn(t, c["heads"], d).to(kind)
        else:
            # a row of the projection: query heads, key heads, value heads
            h, kv = c["q_heads"], c["kv_heads"]
            st["qkv"] = rn(t, h + 2 * kv, d).to(kind)
            shape = (c["pages"], kv, c["page"], d)
            for name in ("k", "v"):
                st[name + "q"] = torch.zeros(shape, dtype=torch.int8, device=DEV)
                st[name + "s"] = torch.zeros(shape[:3] + (d // 32,), dtype=torch.float16, device=DEV)
            slots = torch.randperm(c["pages"] * c["page"], generator=g, device=DEV)[:t]
            if c["holes"]:
                slots[torch.rand(t, generator=g, device=DEV) < 0.2] = -1
            st["slots"] = slots.to(torch.int64)
    elif c["op"] == "plan":
        new, lens = _seqs(c)
        page, b = c["page"], c["batch"]
        width = -(-(c["max_len"] + c["max_new"]) // page)
        have = [-(-(n - m) // page) for m, n in zip(new, lens)]
        pages = sum(-(-n // page) for n in lens) + 13
        order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        h = torch.tensor(have, device=DEV)
        at = torch.arange(width, device=DEV).view(1, width)
        held = (torch.cumsum(h, 0) - h).view(b, 1) + at
        st["table"] = torch.where(at < h.view(b, 1), order[held.clamp_max(pages - 1)], torch.full((), -1, dtype=torch.int32, device=DEV))
        st["free"] = order[sum(have):].contiguous()
        st["free_count"] = torch.tensor([pages - sum(have)], dtype=torch.int32, device=DEV)
        st["pages"], st["tokens"] = pages, sum(new) + c["pad"]
        st["new"] = torch.tensor(new, dtype=torch.int32, device=DEV)
        st["lens"] = torch.tensor([n - m for m, n in zip(new, lens)], dtype=torch.int32, device=DEV)
    else:
        new, lens = _seqs(c)
        b, width = c["batch"], max(1, -(-c["max_len"] // c["page"]))
        for name in ("k", "v"):
            x = rn(b * width, c["kv_heads"], c["page"], c["head_dim"])
            if name == "k":
                x[..., 3] *= 8.0
            st[name + "q"], st[name + "s"] = _quantised(x)
            del x
        st["table"] = torch.randperm(b * width, generator=g, device=DEV).to(torch.int32).view(b, width)
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        starts = [0]
        for n in new:
            starts.append(starts[-1] + n)
        st["starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
        t = starts[-1] + c["pad"]
        st["q"] = rn(t, c["q_heads"], c["head_dim"]).mul_(1.5).to(torch.bfloat16)
        st["out"] = torch.zeros_like(st["q"])  # rows behind the last sequence stay as they were
        st["scale"] = 1.0 / math.sqrt(c["head_dim"])
    return st


# ---------------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------------
def _plain_codes(x):
    """Codes and scales of fp32 x[..., D]: d = binary16(amax / 127), the code is |x| / d rounded half away from zero."""
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    s = (b.abs().amax(-1) / 127.0).to(torch.float16)
    d = s.to(torch.float32).unsqueeze(-1)
    a = b.abs()
    k = torch.floor(a / d + 0.5)
    # the quotient's own rounding may have crossed a half: (k +- 1/2) d is exact in 32 bits
    k = torch.where((k + 0.5) * d <= a, k + 1.0, torch.where((k - 0.5) * d > a, k - 1.0, k))
    k = torch.where(d > 0.0, k.clamp(0.0, 127.0), torch.zeros_like(k))
    q = torch.where(b < 0.0, -k, k).to(torch.int8)
    return q.reshape(x.shape), s


def _values(q, s):
    return q.to(torch.float32) * s.to(torch.float32).repeat_interleave(32, -1)


def _coded_values(q, s):
    """What codes and scales stand for, in one product (binary16)."""
    return (q.unflatten(-1, (-1, 32)) * s.unsqueeze(-1)).flatten(-2)


def _plain_norm(st):
    c = st["case"]
    h = st["x"].to(torch.float32)
    out = []
    if c["res"] != "none":
        h = h + st["residual"].to(torch.float32)
        st["residual_out"].copy_(h)
        out.append(st["residual_out"])
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + 1e-6) * (st["weight"] + c["offset"])
    out.append(y.to(torch.bfloat16))
    if c["q8"]:
        out.append(_coded_values(*_plain_codes(y)))
    return out


def _plain_turned(x, st):
    """fp32 x[tokens, heads, D] with its first `rot` dimensions turned."""
    c = st["case"]
    rot = c["rot"]
    a = st["positions"].to(torch.float64).view(-1, 1, 1) * st["inv_freq"].view(1, 1, -1)
    cos, sin = (torch.cos(a) * st["factor"]).to(torch.float32), (torch.sin(a) * st["factor"]).to(torch.float32)
    if c["interleaved"]:
        x1, x2 = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        x1, x2 = x[..., :rot // 2], x[..., rot // 2:rot]
    y1, y2 = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    y = torch.stack((y1, y2), -1).flatten(-2) if c["interleaved"] else torch.cat((y1, y2), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _plain_rope(st):
    return [_plain_turned(st["x"].to(torch.float32), st).to(torch.bfloat16)]


def _plain_rope_append(st):
    c = st["case"]
    h, kv = c["q_heads"], c["kv_heads"]
    x = st["qkv"].to(torch.float32)
    turned = _plain_turned(x[:, :h + kv], st)
    rows = torch.nonzero(st["slots"] >= 0).squeeze(1)
    page, off = st["slots"][rows] // c["page"], st["slots"][rows] % c["page"]
    out = [turned[:, :h].to(torch.bfloat16)]
    kq, ks = _plain_codes(turned[:, h:])
    vq, vs = _plain_codes(x[:, h + kv:])
    st["kq"][page, :, off], st["ks"][page, :, off] = kq[rows], ks[rows]
    st["vq"][page, :, off], st["vs"][page, :, off] = vq[rows], vs[rows]
    k, v = (torch.zeros((c["tokens"], kv, c["head_dim"]), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    k[rows] = _values(st["kq"][page, :, off], st["ks"][page, :, off]).to(torch.bfloat16)
    v[rows] = _values(st["vq"][page, :, off], st["vs"][page, :, off]).to(torch.bfloat16)
    return out + [k, v]


def _plain_plan(st):
    c = st["case"]
    page, t = c["page"], st["tokens"]
    new, old = st["new"].to(torch.int64), st["lens"].to(torch.int64)
    now = old + new
    first, last = (old + page - 1) // page, (now + page - 1) // page
    taken = torch.cumsum(last - first, 0)
    at = torch.arange(st["table"].shape[1], device=DEV).view(1, -1)
    rank = (taken - last).view(-1, 1) + at  # of the pages taken: this sequence's first is the one after those before it
    fresh = (at >= first.view(-1, 1)) & (at < last.view(-1, 1))
    count = st["free_count"].to(torch.int64)
    page_of = st["free"][(count - 1 - rank).clamp(0, st["free"].shape[0] - 1)]
    st["table"].copy_(torch.where(fresh, page_of, st["table"]))
    ends = torch.cumsum(new, 0)
    token = torch.arange(t, device=DEV)
    seq = torch.searchsorted(ends, token, right=True).clamp_max(c["batch"] - 1)
    live = token < ends[-1]
    pos = token - (ends - new)[seq] + old[seq]
    pos = torch.where(live, pos, torch.zeros_like(pos))
    slot = st["table"][seq, pos // page].to(torch.int64) * page + pos % page
    slot = torch.where(live, slot, torch.full_like(slot, -1))
    starts = torch.cat((torch.zeros_like(ends[:1]), ends)).to(torch.int32)
    return [st["table"], starts, slot, pos.to(torch.int32), now.to(torch.int32), (count - taken[-1]).to(torch.int32)]


def _plain_attn(st):
    c = st["case"]
    b, hq, kv, d = c["batch"], c["q_heads"], c["kv_heads"], c["head_dim"]
    g, m = hq // kv, c["max_new"]
    at = st["table"].to(torch.int64)
    n = at.shape[1] * c["page"]
    first = st["starts"][:-1].to(torch.int64).view(b, 1)
    count = st["starts"][1:].to(torch.int64).view(b, 1) - first
    new = torch.arange(m, device=DEV).view(1, m)
    row = (first + new).clamp_max(st["q"].shape[0] - 1)  # [b, m]
    pos = (st["lens"].to(torch.int64).view(b, 1) - count + new).view(b, 1, 1, m, 1)
    k = _values(st["kq"][at], st["ks"][at]).permute(0, 2, 1, 3, 4).reshape(b, kv, n, d)
    q = st["q"][row].to(torch.float32).view(b, m, kv, g, d).permute(0, 2, 3, 1, 4)
    s = torch.matmul(q.reshape(b, kv, g * m, d), k.transpose(-1, -2)).mul_(st["scale"]).view(b, kv, g, m, n)
    del k
    if c["softcap"] > 0.0:
        s = torch.tanh(s / c["softcap"]).mul_(c["softcap"])
    t = torch.arange(n, device=DEV).view(1, 1, 1, 1, n)
    seen = t <= pos
    if c["window"] > 0:
        seen = seen & (t > pos - c["window"])
    s = s.masked_fill_(~seen, -math.inf)
    p = s.sub_(s.amax(-1, keepdim=True)).exp_()
    z = p.sum(-1, keepdim=True)
    v = _values(st["vq"][at], st["vs"][at]).permute(0, 2, 1, 3, 4).reshape(b, kv, n, d)
    o = torch.matmul(p.view(b, kv, g * m, n), v).view(b, kv, g, m, d) / z
    live = new < count
    st["out"][row[live]] = o.permute(0, 3, 1, 2, 4).reshape(b, m, hq, d)[live].to(torch.bfloat16)
    return [st["out"]]


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------
def _cache(q8, st):
    """The handle that a program makes once for its cache, of the tensors that the state has now."""
    k = st.get("cache")
    if k is None or k.kq is not st["kq"] or k.ks is not st["ks"] or k.vq is not st["vq"] or k.vs is not st["vs"]:
        k = st["cache"] = q8.KvCache(st["kq"], st["ks"], st["vq"], st["vs"])
    return k


def _turns(q8, st):
    """The table that a program makes once for its model, of the frequencies that the state has now."""
    f, made = st["inv_freq"], st.get("turns")
    if made is None or made[0] is not f or made[1] != f._version:
        made = st["turns"] = (f, f._version, q8.rope_turns(f))
    return made[2]


def _own(st):
    from block_quantized_int8_gb300 import q8
    c = st["case"]
    if c["op"] == "norm":
        y, q, s = q8.q8_rms_norm(st["x"], weight=st["weight"], offset=c["offset"], eps=1e-6, residual=st.get("residual"),
                                 residual_out=st.get("residual_out"), quantized=c["q8"])
        out = [st["residual_out"]] if c["res"] != "none" else []
        return out + ([y, _coded_values(q, s)] if c["q8"] else [y])
    if c["op"] in ("rope", "rope_append"):
        turns = _turns(q8, st)
        if c["op"] == "rope":
            return [q8.q8_rope(st["x"], st["positions"], turns, interleaved=c["interleaved"], factor=st["factor"])]
        cache = _cache(q8, st)
        h, kv = c["q_heads"], c["kv_heads"]
        x = st["qkv"]
        q = q8.q8_rope_append(x[:, :h], x[:, h:h + kv], x[:, h + kv:], cache, st["positions"], st["slots"], turns,
                              interleaved=c["interleaved"], factor=st["factor"])
        return [q, *q8.q8_kv_read(cache, st["slots"], dtype=torch.bfloat16)]
    if c["op"] == "plan":
        starts, slots, positions, lens, left = q8.q8_kv_plan(st["table"], st["lens"], st["new"], c["page"], st["pages"], st["tokens"],
                                                             free_pages=st["free"], free_count=st["free_count"])
        return [st["table"], starts, slots, positions, lens, left]
    cache = _cache(q8, st)
    if "ws" not in st:
        st["ws"] = q8.workspace(q8.q8_attn_chunk_workspace_size(c["q_heads"], c["kv_heads"], c["head_dim"]))
    out, _ = q8.q8_attn_chunk(st["q"], cache, st["table"], st["lens"], st["starts"], scale=st["scale"], softcap=c["softcap"],
                              window=c["window"], out=st["out"], ws=st["ws"])
    return [out]


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "rope": _plain_rope, "rope_append": _plain_rope_append, "plan": _plain_plan,
            "attn": _plain_attn}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------
def work(case):
    c = case
    size = 2 if c.get("bf16") else 4
    if c["op"] == "norm":
        n = c["rows"] * c["width"]
        res = {"none": 0, "f32": 8, "bf16": 4}[c["res"]]
        # the 8-bit form's values are given as binary16
        return {"bytes": n * (size + res + 2 + (2 + 2 * 1.0625 if c["q8"] else 0)) + 4 * c["width"], "flops": 6 * n}
    if c["op"] == "rope":
        n = c["tokens"] * c["heads"] * c["head_dim"]
        return {"bytes": n * (size + 2) + 4 * c["tokens"], "flops": 3 * c["tokens"] * c["heads"] * c["rot"]}
    if c["op"] == "rope_append":
        q, k = (c["tokens"] * c[h] * c["head_dim"] for h in ("q_heads", "kv_heads"))
        # rows in, queries out; codes and scales out, in again, values out
        return {"bytes": q * (size + 2) + 2 * k * (size + 2 * 1.0625 + 2) + 20 * c["tokens"],
                "flops": 3 * c["tokens"] * (c["q_heads"] + c["kv_heads"]) * c["rot"] + 8 * k}
    new, lens = _seqs(c)
    if c["op"] == "plan":
        fresh = sum(-(-n // c["page"]) - -(-(n - m) // c["page"]) for m, n in zip(new, lens))
        return {"bytes": 16 * c["batch"] + 8 * fresh + 12 * (sum(new) + c["pad"]), "flops": 4 * (sum(new) + c["pad"])}
    pairs, seen = 0, 0
    for m, n in zip(new, lens):
        if m == 0:
            continue
        w = c["window"] or n
        pairs += sum(min(p + 1, w) for p in range(n - m, n))
        seen += min(n, w + m - 1)
    rows = sum(new) * c["q_heads"] * c["head_dim"]
    return {"bytes": seen * c["kv_heads"] * c["head_dim"] * 2 * 1.0625 + rows * 4 + 4 * seen / c["page"] + 8 * c["batch"],
            "flops": 4 * pairs * c["q_heads"] * c["head_dim"]}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "plan":  # whole numbers
        return None
    c, st = case, prepare(case, seed)
    f64 = torch.float64

    def val64(q, s):
        return (q.to(f64).unflatten(-1, (-1, 32)) * s.to(f64).unsqueeze(-1)).flatten(-2)

    def coded64(x):  # what Q8_0 of x stands for
        b = x.unflatten(-1, (-1, 32))
        s = (b.abs().amax(-1).to(torch.float32) / 127.0).to(torch.float16).to(f64).unsqueeze(-1)
        return (torch.floor(b.abs() / s.clamp_min(1e-300) + 0.5).clamp_max(127.0) * torch.sign(b) * s).flatten(-2)

    if c["op"] == "norm":
        h = st["x"].to(f64)
        out = []
        if c["res"] != "none":
            h = h + st["residual"].to(f64)
            out.append(h)
        y = h / torch.sqrt((h ** 2).sum(-1, keepdim=True) / c["width"] + 1e-6) * (st["weight"].to(f64) + c["offset"])
        return out + ([y, coded64(y)] if c["q8"] else [y])
    if c["op"] in ("rope", "rope_append"):
        x = (st["x"] if c["op"] == "rope" else st["qkv"]).to(f64)
        n = c["rot"] // 2
        i = torch.arange(n, device=DEV)
        lo, hi = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + n)
        turn = torch.polar(torch.full((1, 1, n), st["factor"], dtype=f64, device=DEV),
                           st["positions"].to(f64).view(-1, 1, 1) * st["inv_freq"])
        last = x.shape[1] if c["op"] == "rope" else c["q_heads"] + c["kv_heads"]
        z = torch.complex(x[:, :last, lo], x[:, :last, hi]) * turn
        y = x.clone()
        y[:, :last, lo], y[:, :last, hi] = z.real, z.imag
        if c["op"] == "rope":
            return [y]
        live = (st["slots"] >= 0).view(-1, 1, 1)
        return [y[:, :c["q_heads"]], torch.where(live, coded64(y[:, c["q_heads"]:last]), 0.0), torch.where(live, coded64(y[:, last:]), 0.0)]
    new, lens = _seqs(c)
    g, page = c["q_heads"] // c["kv_heads"], c["page"]
    o = torch.zeros(st["q"].shape, dtype=f64, device=DEV)
    if work(c)["flops"] > 3e12:
        return None
    row = 0
    for b, (m, n) in enumerate(zip(new, lens)):
        if m == 0:
            continue
        at = st["table"][b, :-(-n // page)].to(torch.int64)
        pos = torch.arange(n - m, n, device=DEV).view(m, 1)
        t = torch.arange(n, device=DEV).view(1, n)
        hidden = (t > pos) | ((t <= pos - c["window"]) if c["window"] else (t < 0))
        for h in range(c["kv_heads"]):
            k = val64(st["kq"][at, h], st["ks"][at, h]).reshape(-1, c["head_dim"])[:n]
            v = val64(st["vq"][at, h], st["vs"][at, h]).reshape(-1, c["head_dim"])[:n]
            for j in range(h * g, (h + 1) * g):
                s = st["q"][row:row + m, j].to(f64) @ k.T * st["scale"]
                if c["softcap"] > 0.0:
                    s = c["softcap"] * torch.tanh(s / c["softcap"])
                o[row:row + m, j] = torch.softmax(s.masked_fill(hidden, -math.inf), -1) @ v
        row += m
    return [o]
