"""Cases of the paged-cache operators: what they compute in plain torch, and their sizes.

Two operators serve a batch of sequences whose keys and values live in pages:

* ``append``: the raw projections of new tokens get their optional per-head RMSNorm and their
  rotation (one position per token, or one per axis for images and video), the rotated queries
  come back and the keys and values are stored in the pages the table names;
* ``attend``: causal attention of the new tokens' queries over their sequence's pages, optionally
  behind a prefix of keys that all sequences share.

``run`` computes either the plain form (``own`` false) or calls the package (``own`` true).
"""
import math

import numpy as np
import torch

own = False

THETA, EPS = 1e6, 1e-6
SPARE_PAGES = 3          # pages of the pool that no sequence owns
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}


def _case(name, op, **kw):
    c = {"name": name, "op": op, "act": "f32", "kv": "bf16", "nq": 16, "nkv": 8, "hd": 128,
         "page": 16, "seqs": 1, "new": 1, "ctx": 1, "spread": "log", "prefix": 0, "pad": 0,
         "layout": 1}
    if op == "append":
        c.update(norm=True, axes=1)
    c.update(kw)
    return c


def listed():
    return [
        # one decode step of eight chats: the smallest append, where only latency counts
        _case("append_step_8", "append", kv="f32", seqs=8, ctx=4096),
        # one step of a large image-and-text batch, three position axes, two KV heads
        _case("append_step_256_axes", "append", act="bf16", nkv=2, norm=False, axes=3, seqs=256,
              ctx=8192, layout=2),
        # prompts of a mixed batch entering the cache, ragged and odd
        _case("append_prompts_24", "append", seqs=24, new=1021, ctx=4096, spread="uniform", layout=3),
        # long image-and-text prompts in bf16
        _case("append_prompts_axes", "append", act="bf16", axes=3, seqs=12, new=8192, ctx=16384,
              spread="uniform", page=64, layout=4),
        # a single chat at 4K keys with few KV heads
        _case("attend_one_4k", "attend", nkv=2, seqs=1, ctx=4096),
        # a single chat at 8K keys in an f32 cache
        _case("attend_one_8k_f32", "attend", kv="f32", seqs=1, ctx=8193),
        # a decode step of a ragged batch: a few long sequences among many short ones
        _case("attend_step_64", "attend", nkv=2, seqs=64, ctx=16384, layout=5),
        # a decode step of a full server, bf16 throughout: the largest cache read
        _case("attend_step_256", "attend", act="bf16", seqs=256, ctx=8192, spread="uniform", page=32,
              layout=6),
        # chunks of prompts among single tokens, bf16
        _case("attend_chunks_6", "attend", act="bf16", seqs=6, new=512, ctx=8192, spread="uniform",
              layout=7),
        # sixteen short chats behind one long system prompt, f32 cache
        _case("prefix_8k_16_f32", "attend", kv="f32", seqs=16, ctx=250, prefix=8192, layout=8),
        # sixty-four chats behind one prompt of odd length
        _case("prefix_4k_64", "attend", seqs=64, ctx=512, spread="uniform", prefix=4099, layout=9),
        # a large batch of samples of one 32K document, bf16 throughout
        _case("prefix_32k_256", "attend", act="bf16", nkv=2, seqs=256, ctx=1024, spread="uniform",
              prefix=32768, page=64, layout=10),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    tops = {op: [0.0, 0.0] for op in ("append", "attend")}
    for c in listed():
        w = work(c)
        tops[c["op"]] = [max(tops[c["op"]][0], w["bytes"]), max(tops[c["op"]][1], w["flops"])]
    while True:
        op = rng.choice(["append", "attend", "attend"])
        nq, nkv, hd = rng.choice([(16, 8, 128), (16, 2, 128), (4, 2, 64), (8, 8, 64), (32, 8, 128),
                                  (12, 2, 128), (14, 2, 64), (5, 1, 128)])
        act, kv = rng.choice([("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
        c = {"op": op, "act": act, "kv": kv, "nq": nq, "nkv": nkv, "hd": hd,
             "page": rng.choice([16, 32, 64, 128]), "seqs": _log(rng, 1, 256),
             "spread": rng.choice(["log", "uniform", "same"]), "pad": rng.choice([0, 0, 1, 3]),
             "layout": rng.randrange(1, 1 << 30)}
        if op == "append":
            c["new"] = _log(rng, 2, 8192) if rng.random() < 0.5 else 1
            c["prefix"] = 0
            c.update(norm=rng.random() < 0.5, axes=rng.choice([1, 3]))
        else:
            c["new"] = _log(rng, 2, 512) if rng.random() < 0.3 else 1
            c["prefix"] = _log(rng, 1, 32768) if rng.random() < 0.4 else 0
        c["ctx"] = max(c["new"], _log(rng, 1, 16384))
        w = work(c)
        # the plain form's padded keys and scores have to fit beside three states
        padded = 8 * c["seqs"] * c["ctx"] * nkv * hd
        scores = 4 * nq * c["seqs"] * c["new"] * (c["ctx"] + c["prefix"])
        if (w["bytes"] <= tops[op][0] and w["flops"] <= tops[op][1]
                and (op == "append" or padded + 2 * scores <= 24e9)):
            return c


# ------------------------------------------------------------------------- lengths and sizes
def _lengths(c):
    """(new tokens, cached keys with them) of each sequence; the first has the longest of both."""
    r = np.random.RandomState(c["layout"])
    n = c["seqs"]

    def spread(hi, lo):
        lo = np.minimum(np.asarray(lo, dtype=np.float64), hi)
        if c["spread"] == "same":
            v = np.full(n, hi, dtype=np.float64)
        elif c["spread"] == "uniform":
            v = lo + r.random_sample(n) * (hi - lo)
        else:
            v = np.exp(np.log(lo) + r.random_sample(n) * (math.log(hi) - np.log(lo)))
        return np.clip(np.rint(v), lo, hi).astype(np.int64)

    new = spread(c["new"], np.ones(n))
    new[0] = c["new"]
    ctx = spread(c["ctx"], np.maximum(new, 1))
    ctx[0] = c["ctx"]
    return new, ctx


def work(c):
    new, ctx = _lengths(c)
    tokens, nq, nkv, hd = int(new.sum()), c["nq"], c["nkv"], c["hd"]
    a, k = BYTES[c["act"]], BYTES[c["kv"]]
    if c["op"] == "append":
        heads = (nq + 2 * nkv) * hd
        rot = 3 * hd * (nq + nkv) + (4 * hd * (nq + nkv) if c["norm"] else 0)
        return {"bytes": tokens * (heads * a + nq * hd * a + 2 * nkv * hd * k + 4 * c["axes"] + 4),
                "flops": tokens * rot}
    seen = int((new * ctx - new * (new - 1) // 2).sum()) + tokens * c["prefix"]
    keys = int(ctx.sum()) + c["prefix"]
    return {"bytes": 2 * tokens * nq * hd * a + keys * 2 * nkv * hd * k + 4 * (keys // c["page"]),
            "flops": 4 * seen * nq * hd}


# ------------------------------------------------------------------------- inputs
def prepare(case, seed):
    c = case
    new, ctx = _lengths(c)
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    act, kv = DTYPES[c["act"]], DTYPES[c["kv"]]
    page, nkv, hd, nq = c["page"], c["nkv"], c["hd"], c["nq"]

    def normal(*shape, dtype=torch.float32, scale=1.0):
        t = torch.randn(*shape, generator=g, device="cuda", dtype=dtype)
        return t.mul_(scale) if scale != 1.0 else t

    pages = (ctx + page - 1) // page
    n_prefix = -(-c["prefix"] // page)
    n_pages = int(pages.sum()) + n_prefix + SPARE_PAGES
    # pages lie in the pool in no order; entries behind a sequence's last page name none
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    pages_d = torch.from_numpy(pages).cuda()
    col = torch.arange(int(pages.max()), device="cuda")
    first = torch.cumsum(pages_d, 0) - pages_d
    at = (first[:, None] + col[None]).clamp(max=n_pages - 1)
    table = torch.where(col[None] < pages_d[:, None], order[at], -1).to(torch.int32).contiguous()
    tokens = int(new.sum())
    start = np.concatenate([[0], np.cumsum(new)])
    s = {"case": c, "tokens": tokens, "rows": tokens + c["pad"], "max_new": int(c["new"]),
         "k_pages": normal(n_pages, nkv, page, hd, dtype=kv),
         "v_pages": normal(n_pages, nkv, page, hd, dtype=kv),
         "table": table,
         "kv_len": torch.from_numpy(ctx.astype(np.int32)).cuda(),
         "q_start": torch.from_numpy(start.astype(np.int32)).cuda(),
         "prefix_pages": order[int(pages.sum()):int(pages.sum()) + n_prefix].contiguous()}
    if c["op"] == "append":
        s["qkv"] = normal(s["rows"], (nq + 2 * nkv) * hd, dtype=act)
        s["q_norm"] = s["k_norm"] = None
        if c["norm"]:
            s["q_norm"] = normal(hd, scale=0.1).add_(1).to(torch.bfloat16)
            s["k_norm"] = normal(hd, scale=0.1).add_(1).to(torch.bfloat16)
        s["positions"] = s["sections"] = None
        if c["axes"] > 1:  # time advances with the token, height and width walk over a frame
            half = hd // 2
            s["sections"] = (half // 4, half // 4 + half // 8, half - half // 4 - half // 4 - half // 8)
            t = torch.arange(s["rows"], device="cuda")
            jump = torch.randint(0, 4096, (3,), generator=g, device="cuda")
            s["positions"] = torch.stack([t // 64 + jump[0], t // 8 % 32 + jump[1], t % 32 + jump[2]],
                                         1).to(torch.int32).contiguous()
        s["out"] = torch.zeros(s["rows"], nq, hd, dtype=act, device="cuda")
    else:
        s["q"] = normal(s["rows"], nq, hd, dtype=act, scale=1.5)
        s["out"] = torch.zeros(s["rows"], nq, hd, dtype=act, device="cuda")
    return s


# ------------------------------------------------------------------------- plain forms
def _rows(s):
    """Sequence, index in the sequence's new tokens and cache row of every new token."""
    i = torch.arange(s["tokens"], device="cuda")
    starts = s["q_start"].long()
    seq = torch.searchsorted(starts[1:], i, right=True)
    at = i - starts[seq]
    new = starts[1:] - starts[:-1]
    return seq, at, s["kv_len"].long()[seq] - new[seq] + at


def _plain_append(s):
    c = s["case"]
    nq, nkv, hd, page, n = c["nq"], c["nkv"], c["hd"], c["page"], s["tokens"]
    half = hd // 2
    seq, _, row = _rows(s)
    x = s["qkv"][:n].float().view(n, nq + 2 * nkv, hd)
    q, k, v = x[:, :nq], x[:, nq:nq + nkv], x[:, nq + nkv:]
    if s["q_norm"] is not None:
        q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + EPS) * s["q_norm"].float()
        k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + EPS) * s["k_norm"].float()
    j = torch.arange(half, device="cuda", dtype=torch.float64)
    inv = THETA ** (-2.0 * j / hd)
    if s["positions"] is None:
        pos = (row + c["prefix"]).double()[:, None].expand(n, half)
    else:
        axis = torch.repeat_interleave(torch.arange(3, device="cuda"),
                                       torch.tensor(s["sections"], device="cuda"), output_size=half)
        pos = s["positions"][:n].double()[:, axis]
    ang = pos * inv
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]

    def rotate(t):
        a, b = t[..., :half], t[..., half:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    s["out"][:n] = rotate(q).to(s["out"].dtype)
    at = s["table"].long()[seq, row // page]
    s["k_pages"][at, :, row % page] = rotate(k).to(s["k_pages"].dtype)
    s["v_pages"][at, :, row % page] = v.to(s["v_pages"].dtype)
    return {"q": s["out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _padded(pages, table):
    """Pages of a table [B, n] as f32 rows [B, nkv, n * page, hd]."""
    b, n = table.shape
    _, nkv, page, hd = pages.shape
    t = pages[table.long().clamp(min=0)]
    return t.permute(0, 2, 1, 3, 4).reshape(b, nkv, n * page, hd).float()


def _plain_attend(s):
    c = s["case"]
    nq, nkv, hd, n = c["nq"], c["nkv"], c["hd"], s["tokens"]
    grp, b, most = nq // nkv, c["seqs"], s["max_new"]
    seq, at, row = _rows(s)
    qf = s["q"][:n].float() / math.sqrt(hd)
    # the sequences' own keys, every sequence padded to the longest
    q = torch.zeros(b, most, nq, hd, device="cuda")
    q[seq, at] = qf
    last = torch.full((b, most), -1, device="cuda")
    last[seq, at] = row
    q = q.view(b, most, nkv, grp, hd).permute(0, 2, 1, 3, 4).reshape(b, nkv, most * grp, hd)
    keys = _padded(s["k_pages"], s["table"])
    scores = q @ keys.transpose(-1, -2)
    hide = (torch.arange(keys.shape[2], device="cuda") > last[..., None])[:, None, :, None]
    scores = scores.view(b, nkv, most, grp, -1).masked_fill_(hide, -math.inf)
    del keys
    top = scores.amax(-1, keepdim=True).clamp(min=-1e30)
    p = scores.sub_(top).exp_()
    den = p.sum(-1, keepdim=True)
    # pages past a sequence's end hold whatever they held: their weight is 0
    num = (p.view(b, nkv, most * grp, -1) @ _padded(s["v_pages"], s["table"])).view(b, nkv, most, grp, hd)
    del p, scores

    def by_token(t):
        return t.permute(0, 2, 1, 3, 4)[seq, at]     # [tokens, nkv, grp, ...]

    top, den, num = by_token(top), by_token(den), by_token(num)
    if c["prefix"]:
        keys = _padded(s["k_pages"], s["prefix_pages"][None])[0, :, :c["prefix"]]
        vals = _padded(s["v_pages"], s["prefix_pages"][None])[0, :, :c["prefix"]]
        q = qf.view(n, nkv, grp, hd).permute(1, 0, 2, 3).reshape(nkv, n * grp, hd)
        scores = q @ keys.transpose(-1, -2)
        ptop = scores.amax(-1, keepdim=True)
        p = scores.sub_(ptop).exp_()
        pden = p.sum(-1, keepdim=True)
        pnum = p @ vals
        ptop, pden, pnum = (t.view(nkv, n, grp, -1).permute(1, 0, 2, 3) for t in (ptop, pden, pnum))
        m = torch.maximum(top, ptop)
        f, pf = (top - m).exp(), (ptop - m).exp()
        num, den = num * f + pnum * pf, den * f + pden * pf
    s["out"][:n] = (num / den).reshape(n, nq, hd).to(s["out"].dtype)
    return s["out"]


def _cache(s):
    """The package's handle of the state's cache, made once as a server would keep it."""
    if "cache" not in s:
        from sequence_decode_step_gb300 import PagedKV
        s["cache"] = PagedKV(s["k_pages"], s["v_pages"], s["table"], s["kv_len"], s["q_start"],
                             prefix_pages=s["prefix_pages"], prefix_len=s["case"]["prefix"])
    return s["cache"]


def run(state):
    s = state
    if s["case"]["op"] == "append":
        if own:
            _cache(s).append(s["qkv"], s["case"]["nq"], q_norm=s["q_norm"], k_norm=s["k_norm"],
                             eps=EPS, rope_theta=THETA, positions=s["positions"],
                             sections=s["sections"], out=s["out"])
            return {"q": s["out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
        return _plain_append(s)
    if own:
        return _cache(s).attend(s["q"], max_new=s["max_new"], out=s["out"])
    return _plain_attend(s)


# ------------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    c = case
    s = prepare(c, seed)
    nq, nkv, hd, page = c["nq"], c["nkv"], c["hd"], c["page"]
    new, ctx = _lengths(c)
    table = s["table"].cpu().numpy()
    out = s["out"].double()
    if c["op"] == "append":
        kp, vp = s["k_pages"].double(), s["v_pages"].double()
        freq = torch.tensor([THETA ** (-2.0 * j / hd) for j in range(hd // 2)], dtype=torch.float64,
                            device="cuda")
        lo = 0
        for b in range(c["seqs"]):
            n = int(new[b])
            rows = np.arange(int(ctx[b]) - n, int(ctx[b]))
            x = s["qkv"][lo:lo + n].double().reshape(n, nq + 2 * nkv, hd)
            if s["positions"] is None:
                pos = torch.from_numpy(rows + c["prefix"]).cuda().double()[:, None] * torch.ones_like(freq)
            else:
                parts = [s["positions"][lo:lo + n, i:i + 1].double().repeat(1, w)
                         for i, w in enumerate(s["sections"])]
                pos = torch.cat(parts, 1)
            # the pair (x_j, x_{j + hd/2}) as a complex number, turned by its angle
            turn = torch.polar(torch.ones_like(pos), pos * freq)[:, None]

            def turned(t, gain):
                if gain is not None:
                    t = t / (t.pow(2).sum(-1, keepdim=True) / hd + EPS).sqrt() * gain.double()
                z = torch.complex(t[..., :hd // 2], t[..., hd // 2:]) * turn
                return torch.cat([z.real, z.imag], -1)

            out[lo:lo + n] = turned(x[:, :nq], s["q_norm"])
            at = torch.from_numpy(table[b, rows // page].astype(np.int64)).cuda()
            slot = torch.from_numpy(rows % page).cuda()
            kp[at, :, slot] = turned(x[:, nq:nq + nkv], s["k_norm"])
            vp[at, :, slot] = x[:, nq + nkv:]
            lo += n
        return {"q": out, "k_pages": kp, "v_pages": vp}
    if work(c)["flops"] > 6e11:
        return None
    pre = s["prefix_pages"].long()
    lo = 0
    for b in range(c["seqs"]):
        n, length = int(new[b]), int(ctx[b])
        mine = torch.from_numpy(table[b, :-(-length // page)].astype(np.int64)).cuda()
        for h in range(nkv):
            def rows_of(pool):
                parts = [pool[pre, h].reshape(-1, hd)[:c["prefix"]], pool[mine, h].reshape(-1, hd)[:length]]
                return torch.cat(parts).double()

            k, v = rows_of(s["k_pages"]), rows_of(s["v_pages"])
            grp = nq // nkv
            q = s["q"][lo:lo + n, h * grp:(h + 1) * grp].double()
            sc = torch.einsum("ngd,kd->ngk", q, k) / math.sqrt(hd)
            see = torch.arange(k.shape[0], device="cuda")[None] <= (
                torch.arange(n, device="cuda")[:, None] + c["prefix"] + length - n)
            w = torch.softmax(sc.masked_fill(~see[:, None], -math.inf), -1)
            out[lo:lo + n, h * grp:(h + 1) * grp] = torch.einsum("ngk,kd->ngd", w, v)
        lo += n
    return out
