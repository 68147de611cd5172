"""The decode-step operators next to the Q8_0 matmuls, as cases that can be timed and compared.

A decode step around the matmuls of this library writes the new tokens' keys and values into a
paged Q8_0 cache (q8_kv_append; q8_kv_read gives them back), lets each new token attend to its
sequence's cache (q8_attn_decode), sends it through a mixture of Q8_0 experts (q8_moe) and draws
the next token from its logits (q8_sample).  Each has a plain form here, of elementary torch
operations in 32 bits, and a definition in 64 bits (`exact`).

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
        # one new token of one sequence: 12 heads of 128, fp32 keys and values as a matmul leaves them
        {"name": "append_1", "op": "append", "tokens": 1, "kv_heads": 12, "head_dim": 128, "page": 16, "pages": 64,
         "bf16": False, "holes": False},
        # a decode batch of odd size with padded rows (slot -1), bf16
        {"name": "append_37", "op": "append", "tokens": 37, "kv_heads": 8, "head_dim": 64, "page": 32, "pages": 300,
         "bf16": True, "holes": True},
        # a prefill chunk written to scattered pages
        {"name": "append_8192", "op": "append", "tokens": 8192, "kv_heads": 8, "head_dim": 128, "page": 64, "pages": 1024,
         "bf16": True, "holes": False},
        # the start of one conversation: every head has its own keys, latency counts
        {"name": "attn_1x200", "op": "attn", "batch": 1, "q_heads": 12, "kv_heads": 12, "head_dim": 128, "page": 16,
         "max_len": 200, "ragged": False, "window": 0, "softcap": 0.0},
        # a serving batch: 48 sequences of 0 to 6000 tokens, 4 query heads to a key head
        {"name": "attn_48_ragged", "op": "attn", "batch": 48, "q_heads": 32, "kv_heads": 8, "head_dim": 128, "page": 16,
         "max_len": 6000, "ragged": True, "window": 0, "softcap": 0.0},
        # sliding window and capped scores, wide heads, 3 query heads to a key head, 3001 tokens
        {"name": "attn_window_cap", "op": "attn", "batch": 17, "q_heads": 12, "kv_heads": 4, "head_dim": 256, "page": 32,
         "max_len": 3001, "ragged": True, "window": 1000, "softcap": 30.0},
        # one sequence of 262,144 tokens: the cache is read once, split over its whole length
        {"name": "attn_1x262144", "op": "attn", "batch": 1, "q_heads": 64, "kv_heads": 8, "head_dim": 128, "page": 64,
         "max_len": 262144, "ragged": False, "window": 0, "softcap": 0.0},
        # one token through 2 of 16 experts of this library's layer widths
        {"name": "moe_1", "op": "moe", "tokens": 1, "experts": 16, "top_k": 2, "hidden": 1536, "ffn": 4096, "renorm": True},
        # a small batch through many narrow experts, weights not normalised again
        {"name": "moe_7", "op": "moe", "tokens": 7, "experts": 64, "top_k": 6, "hidden": 2048, "ffn": 1376, "renorm": False},
        # the largest decode batch: nearly every expert is read
        {"name": "moe_32", "op": "moe", "tokens": 32, "experts": 128, "top_k": 8, "hidden": 2048, "ffn": 1024, "renorm": True},
        # one row of the 262,144-word vocabulary
        {"name": "sample_1", "op": "sample", "rows": 1, "vocab": 262144, "bf16": False, "seed_knobs": 1},
        # a batch of odd vocabulary, every row with knobs of its own, greedy rows among them
        {"name": "sample_64", "op": "sample", "rows": 64, "vocab": 131071, "bf16": False, "seed_knobs": 2},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "moe", "moe", "sample"])
    if op == "append":
        t = _log(rng, 1, 8192)
        page = rng.choice([16, 32, 64, 128, 256])
        return {"op": op, "tokens": t, "kv_heads": rng.randint(1, 12), "head_dim": rng.choice([64, 128, 256]), "page": page,
                "pages": -(-t // page) + rng.randint(1, 64), "bf16": rng.random() < 0.5, "holes": rng.random() < 0.3}
    if op == "attn":
        hd, kv = rng.choice([64, 128, 256]), rng.randint(1, 12)
        group = rng.choice([1, 1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
        top = 262144 * 8 * 128 // (hd * kv)  # tokens in all sequences of a call that costs as much as the largest
        batch = _log(rng, 1, 128)
        max_len = _log(rng, 1, min(262144, top // batch))
        return {"op": op, "batch": batch, "q_heads": kv * group, "kv_heads": kv, "head_dim": hd,
                "page": rng.choice([16, 32, 64, 128]), "max_len": max_len, "ragged": rng.random() < 0.7,
                "window": _log(rng, 1, 4096) if rng.random() < 0.25 else 0, "softcap": 30.0 if rng.random() < 0.25 else 0.0}
    if op == "moe":
        h = 32 * _log(rng, 8, 128)
        f = 32 * _log(rng, 4, 128)
        e = _log(rng, 2, 128)
        while e > 2 and e * h * f > 128 * 2048 * 1024:
            e //= 2
        return {"op": op, "tokens": _log(rng, 1, 32), "experts": e, "top_k": rng.randint(1, min(8, e)), "hidden": h, "ffn": f,
                "renorm": rng.random() < 0.5}
    return {"op": op, "rows": _log(rng, 1, 64), "vocab": _log(rng, 100, 262144), "bf16": rng.random() < 0.4,
            "seed_knobs": rng.randint(3, 1 << 20)}


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


def _lens(c):
    if not c["ragged"]:
        return [c["max_len"]] * c["batch"]
    r = random.Random(c["batch"] * 1000003 + c["max_len"])
    n = [r.randint(0, c["max_len"]) for _ in range(c["batch"])]
    n[r.randrange(c["batch"])] = c["max_len"]  # one of the longest, and (in a batch) one that is empty
    if c["batch"] > 2:
        n[n.index(min(n))] = 0
    return n


def _knobs(c):
    r = random.Random(c["seed_knobs"])
    n = c["rows"]
    t = [r.choice([0.0, 0.6, 0.7, 0.8, 1.0, 1.0, 1.3]) if n > 1 else 0.8 for _ in range(n)]
    k = [r.choice([0, 0, 20, 50, 64, 1000]) if n > 1 else 50 for _ in range(n)]
    p = [r.choice([1.0, 0.95, 0.9, 0.8, 0.5]) if n > 1 else 0.95 for _ in range(n)]
    m = [r.choice([0.0, 0.0, 0.02, 0.1]) if n > 1 else 0.01 for _ in range(n)]
    return t, k, p, m


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 13)

    def rn(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)

    c = dict(case)
    st = {"case": c}
    if c["op"] == "append":
        shape = (c["pages"], c["kv_heads"], c["page"], c["head_dim"])
        for name in ("k", "v"):
            st[name + "q"] = torch.zeros(shape, dtype=torch.int8, device=DEV)
            st[name + "s"] = torch.zeros(shape[:3] + (shape[3] // 32,), dtype=torch.float16, device=DEV)
            x = rn(c["tokens"], c["kv_heads"], c["head_dim"])
            x[..., 3] *= 8.0  # keys have a few channels that stand out
            st[name] = x.to(torch.bfloat16) if c["bf16"] else x
        slots = torch.randperm(c["pages"] * c["page"], generator=g, device=DEV)[:c["tokens"]]
        if c["holes"]:
            slots[torch.rand(c["tokens"], generator=g, device=DEV) < 0.2] = -1
        st["slots"] = slots.to(torch.int64)
    elif c["op"] == "attn":
        lens = _lens(c)
        width = max(1, -(-c["max_len"] // c["page"]))
        pages = c["batch"] * width
        for name in ("k", "v"):
            x = rn(pages, c["kv_heads"], c["page"], c["head_dim"])
            if name == "k":
                x[..., 3] *= 8.0
            st[name + "q"], st[name + "s"] = _quantised(x)
            del x
        st["table"] = torch.randperm(pages, generator=g, device=DEV).to(torch.int32).view(c["batch"], width)
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        st["q"] = rn(c["batch"], c["q_heads"], c["head_dim"]).mul_(1.5).to(torch.bfloat16)
        st["scale"] = 1.0 / math.sqrt(c["head_dim"])
    elif c["op"] == "moe":
        t, e, h, f = c["tokens"], c["experts"], c["hidden"], c["ffn"]
        q13, s13, q2, s2 = (torch.empty((e, 2 * f, h), dtype=torch.int8, device=DEV),
                            torch.empty((e, 2 * f, h // 32), dtype=torch.float16, device=DEV),
                            torch.empty((e, h, f), dtype=torch.int8, device=DEV),
                            torch.empty((e, h, f // 32), dtype=torch.float16, device=DEV))
        step = max(1, (1 << 27) // (2 * f * h))
        for i in range(0, e, step):
            n = min(step, e - i)
            q13[i:i + n], s13[i:i + n] = _quantised(rn(n, 2 * f, h).mul_(0.02))
            q2[i:i + n], s2[i:i + n] = _quantised(rn(n, h, f).mul_(0.02))
        st.update(q13=q13, s13=s13, q2=q2, s2=s2)
        st["x"] = rn(t, h).to(torch.bfloat16)
        st["logits"] = rn(t, e) * 1.5 + rn(1, e) * 0.5  # some experts are liked more than others
    else:
        n, v = c["rows"], c["vocab"]
        x = rn(n, v).mul_(2.5)
        top = torch.randint(0, v, (n, min(v, 40)), generator=g, device=DEV)  # words that fit, well above the rest
        x.scatter_add_(1, top, rn(n, top.shape[1]).abs_().mul_(6.0))
        x[:, v // 3] = -math.inf  # a forbidden word
        st["logits"] = x.to(torch.bfloat16) if c["bf16"] else x
        t, k, p, m = _knobs(c)
        st["temperature"] = torch.tensor(t, dtype=torch.float32, device=DEV)
        st["top_k"] = torch.tensor(k, dtype=torch.int32, device=DEV)
        st["top_p"] = torch.tensor(p, dtype=torch.float32, device=DEV)
        st["min_p"] = torch.tensor(m, dtype=torch.float32, device=DEV)
        st["u"] = torch.rand(n, generator=g, device=DEV, dtype=torch.float32)
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


def _plain_append(st):
    c = st["case"]
    keep = st["slots"] >= 0
    rows = torch.nonzero(keep).squeeze(1)
    page, off = st["slots"][rows] // c["page"], st["slots"][rows] % c["page"]
    out = [None, None]
    for i, name in ((0, "k"), (1, "v")):
        q, s = _plain_codes(st[name].to(torch.float32))
        st[name + "q"][page, :, off] = q[rows]
        st[name + "s"][page, :, off] = s[rows]
        got = torch.zeros(st[name].shape, dtype=torch.float32, device=DEV)
        got[rows] = _values(st[name + "q"][page, :, off], st[name + "s"][page, :, off])
        out[i] = got
    return out


def _plain_attn(st):
    c = st["case"]
    b, hq, kv, d = c["batch"], c["q_heads"], c["kv_heads"], c["head_dim"]
    at = st["table"].to(torch.int64)
    n = at.shape[1] * c["page"]
    k = _values(st["kq"][at], st["ks"][at]).permute(0, 2, 1, 3, 4).reshape(b, kv, n, d)
    q = st["q"].to(torch.float32).view(b, kv, hq // kv, d)
    s = torch.matmul(q, k.transpose(-1, -2)) * st["scale"]
    del k
    if c["softcap"] > 0.0:
        s = c["softcap"] * torch.tanh(s / c["softcap"])
    t = torch.arange(n, device=DEV).view(1, 1, 1, n)
    last = st["lens"].to(torch.int64).view(b, 1, 1, 1)
    seen = t < last
    if c["window"] > 0:
        seen = seen & (t >= last - c["window"])
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    m = s.amax(-1, keepdim=True)
    m0 = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(s - m0)
    z = p.sum(-1, keepdim=True)
    v = _values(st["vq"][at], st["vs"][at]).permute(0, 2, 1, 3, 4).reshape(b, kv, n, d)
    o = torch.matmul(p, v) / torch.where(z > 0.0, z, torch.ones_like(z))
    lse = (m0 + torch.log(z)).view(b, hq)
    return [o.reshape(b, hq, d).to(torch.bfloat16), lse]


def _plain_route(logits, top_k, renorm):
    val, ids = torch.sort(logits, dim=-1, descending=True, stable=True)
    top = val[:, :1]
    e = torch.exp(val - top)
    z = (e[:, :top_k] if renorm else e).sum(-1, keepdim=True)
    return ids[:, :top_k], e[:, :top_k] / z


def _plain_moe(st):
    c = st["case"]
    t, k = c["tokens"], c["top_k"]
    ids, w = _plain_route(st["logits"], k, c["renorm"])
    used, place = torch.unique(ids, return_inverse=True)
    x = st["x"].to(torch.float32)
    gu = torch.matmul(x, _values(st["q13"][used], st["s13"][used]).transpose(1, 2))  # [used, t, 2f]
    a, u = gu[..., :c["ffn"]], gu[..., c["ffn"]:]
    act = a / (1.0 + torch.exp(-a)) * u
    y = torch.matmul(act, _values(st["q2"][used], st["s2"][used]).transpose(1, 2))  # [used, t, h]
    tok = torch.arange(t, device=DEV).view(t, 1)
    return [(y[place, tok] * w.unsqueeze(-1)).sum(1), ids.to(torch.int32), w]


#: a word's mass is a whole number of 2^-40 parts of the likeliest word's, so that sums are exact in any order
ONE = float(1 << 40)


def _plain_sample(st):
    x = st["logits"].to(torch.float32)
    n, v = x.shape
    x = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x)
    temp = st["temperature"].view(n, 1)
    val, ids = torch.sort(x, dim=-1, descending=True, stable=True)
    top = val[:, :1]
    e = torch.where(val == top, torch.ones_like(val), torch.exp((val - top) / torch.where(temp > 0.0, temp, torch.ones_like(temp))))
    mass = (e * ONE).to(torch.int64)
    rank = torch.arange(v, device=DEV).view(1, v)
    k = st["top_k"].to(torch.int64).view(n, 1)
    k = torch.where((k <= 0) | (k > v), torch.full_like(k, v), k)
    k = torch.where(temp > 0.0, k, torch.ones_like(k))  # no temperature: the likeliest word
    mass = torch.where((rank < k) & (val > -math.inf), mass, torch.zeros_like(mass))
    total = mass.sum(-1, keepdim=True)
    p = st["top_p"].view(n, 1)
    cut = torch.ceil(p.to(torch.float64) * total.to(torch.float64)).to(torch.int64).clamp_min(1)
    cut = torch.where(p < 1.0, cut, total)
    before = torch.cumsum(mass, -1) - mass
    keep = (mass > 0) & (before < cut) & (e >= st["min_p"].view(n, 1))
    mass = torch.where(keep, mass, torch.zeros_like(mass))
    total = mass.sum(-1)
    by_word = torch.zeros_like(mass).scatter_(1, ids, mass)
    r = torch.floor(st["u"].to(torch.float64) * total.to(torch.float64)).to(torch.int64)
    r = torch.minimum(r, total - 1).clamp_min(0)
    token = (torch.cumsum(by_word, -1) <= r.view(n, 1)).sum(-1)
    got = by_word.gather(1, token.clamp_max(v - 1).view(n, 1)).squeeze(1)
    none = total == 0
    logprob = torch.log(got.to(torch.float64) / total.to(torch.float64).clamp_min(1.0)).to(torch.float32)
    return [torch.where(none, torch.full_like(token, -1), token).to(torch.int32),
            torch.where(none, torch.full_like(logprob, -math.inf), logprob), keep.sum(-1).to(torch.int32)]


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------
def _own(st):
    from block_quantized_int8_gb300 import q8
    c = st["case"]
    if c["op"] == "append":
        if "cache" not in st:  # the handle that a program makes once for its cache
            st["cache"] = q8.KvCache(st["kq"], st["ks"], st["vq"], st["vs"])
        q8.q8_kv_append(st["cache"], st["k"], st["v"], st["slots"])
        return list(q8.q8_kv_read(st["cache"], st["slots"], dtype=torch.float32))
    if c["op"] == "attn":
        if "cache" not in st:
            st["cache"] = q8.KvCache(st["kq"], st["ks"], st["vq"], st["vs"])
            st["ws"] = q8.workspace(q8.q8_attn_decode_workspace_size(c["batch"], c["q_heads"], c["kv_heads"], c["head_dim"]))
        return list(q8.q8_attn_decode(st["q"], st["cache"], st["table"], st["lens"], scale=st["scale"], softcap=c["softcap"],
                                      window=c["window"], ws=st["ws"]))
    if c["op"] == "moe":
        if "ws" not in st:
            st["ws"] = q8.workspace(q8.q8_moe_workspace_size(c["tokens"], c["experts"], c["hidden"], c["ffn"], c["top_k"]))
        return list(q8.q8_moe(st["x"], st["logits"], st["q13"], st["s13"], st["q2"], st["s2"], c["top_k"], renorm=c["renorm"],
                              ws=st["ws"]))
    return list(q8.q8_sample(st["logits"], st["u"], temperature=st["temperature"], top_k=st["top_k"], top_p=st["top_p"],
                             min_p=st["min_p"]))


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "attn": _plain_attn, "moe": _plain_moe, "sample": _plain_sample}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "append":
        n = c["tokens"] * c["kv_heads"] * c["head_dim"] * 2
        # new values in, codes and scales out, codes and scales in again, values out
        return {"bytes": n * ((2 if c["bf16"] else 4) + 2 * 1.0625 + 4) + 8 * c["tokens"], "flops": 4 * n}
    if c["op"] == "attn":
        seen = sum(min(n, c["window"]) if c["window"] else n for n in _lens(c))
        n = seen * c["kv_heads"] * c["head_dim"]
        q = c["batch"] * c["q_heads"] * c["head_dim"]
        return {"bytes": n * 2 * 1.0625 + q * 4 + c["batch"] * c["q_heads"] * 4 + 4 * seen / c["page"] + 4 * c["batch"],
                "flops": 4 * n * (c["q_heads"] // c["kv_heads"])}
    if c["op"] == "moe":
        t, e, k = c["tokens"], c["experts"], c["top_k"]
        used = e * (1.0 - (1.0 - k / e) ** t)  # of the experts, as many as t tokens choose on the average
        n = 3 * c["hidden"] * c["ffn"]
        return {"bytes": used * n * 1.0625 + t * c["hidden"] * 6 + t * e * 4 + t * k * 8, "flops": 2 * n * t * k}
    n = c["rows"] * c["vocab"]
    return {"bytes": n * (2 if c["bf16"] else 4) + c["rows"] * 32, "flops": 4 * n}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------
def exact(case, seed):
    c, st = case, prepare(case, seed)
    f64 = torch.float64

    def val64(q, s):
        return (q.to(f64).unflatten(-1, (-1, 32)) * s.to(f64).unsqueeze(-1)).flatten(-2)

    if c["op"] == "append":
        out = []
        live = (st["slots"] >= 0).view(-1, 1, 1)
        for name in ("k", "v"):
            x = st[name].to(f64).unflatten(-1, (-1, 32))
            s = (x.abs().amax(-1).to(torch.float32) / 127.0).to(torch.float16).to(f64).unsqueeze(-1)
            code = torch.floor(x.abs() / s.clamp_min(1e-300) + 0.5).clamp_max(127.0) * torch.sign(x)
            out.append(torch.where(live, (code * s).flatten(-2), torch.zeros((), dtype=f64, device=DEV)))
        return out
    if c["op"] == "attn":
        b, hq, kv, d, page = c["batch"], c["q_heads"], c["kv_heads"], c["head_dim"], c["page"]
        o = torch.zeros((b, hq, d), dtype=f64, device=DEV)
        lse = torch.full((b, hq), -math.inf, dtype=f64, device=DEV)
        for i, n in enumerate(_lens(c)):
            first = max(0, n - c["window"]) if c["window"] else 0
            if n == 0:
                continue
            at = st["table"][i, first // page:-(-n // page)].to(torch.int64)
            skip = first - first // page * page
            for h in range(kv):
                k = val64(st["kq"][at, h], st["ks"][at, h]).reshape(-1, d)[skip:skip + n - first]
                s = st["q"][i, h * (hq // kv):(h + 1) * (hq // kv)].to(f64) @ k.T * st["scale"]
                if c["softcap"] > 0.0:
                    s = c["softcap"] * torch.tanh(s / c["softcap"])
                lse[i, h * (hq // kv):(h + 1) * (hq // kv)] = torch.logsumexp(s, -1)
                v = val64(st["vq"][at, h], st["vs"][at, h]).reshape(-1, d)[skip:skip + n - first]
                o[i, h * (hq // kv):(h + 1) * (hq // kv)] = torch.softmax(s, -1) @ v
        return [o, lse]
    if c["op"] == "moe":
        t, f = c["tokens"], c["ffn"]
        lg = st["logits"].to(f64)
        prob = torch.softmax(lg, -1)
        order = torch.argsort(lg, dim=-1, descending=True, stable=True)[:, :c["top_k"]]
        w = prob.gather(1, order)
        if c["renorm"]:
            w = w / w.sum(-1, keepdim=True)
        y = torch.zeros((t, c["hidden"]), dtype=f64, device=DEV)
        for e in sorted(set(order.flatten().tolist())):
            rows, col = torch.nonzero(order == e, as_tuple=True)
            gu = st["x"][rows].to(f64) @ val64(st["q13"][e], st["s13"][e]).T
            act = gu[:, :f] * torch.sigmoid(gu[:, :f]) * gu[:, f:]
            y.index_add_(0, rows, w[rows, col].unsqueeze(1) * (act @ val64(st["q2"][e], st["s2"][e]).T))
        return [y, None, w]
    # the drawn word's probability among those that top-k, top-p and min-p leave
    out = torch.full((c["rows"],), -math.inf, dtype=f64, device=DEV)
    T, K, P, m = (a.tolist() for a in (st["temperature"], st["top_k"], st["top_p"], st["min_p"]))
    for i in range(c["rows"]):
        x = st["logits"][i].to(f64)
        if T[i] <= 0.0:
            out[i] = 0.0
            continue
        order = torch.argsort(x, descending=True, stable=True)
        n = K[i] if 0 < K[i] <= c["vocab"] else c["vocab"]
        q = torch.softmax(x[order[:n]] / T[i], 0)
        keep = q >= m[i] * q[0]
        if P[i] < 1.0:
            keep &= torch.cumsum(q, 0) - q < P[i]
        by_word = torch.zeros_like(x)
        by_word[order[:n]] = torch.where(keep, q, torch.zeros_like(q))
        total = torch.cumsum(by_word, 0)
        word = int((total <= float(st["u"][i]) * total[-1]).sum().clamp_max(c["vocab"] - 1))
        out[i] = torch.log(by_word[word] / total[-1])
    return [None, out, None]
