"""Cases of the operators that put a model's attention in front of the constrained decode step.

A tool-pointer decoder reads a prompt, then emits a few pointers out of a
catalog.  In front of the output head stands a model whose keys and values lie
in a paged cache.  Four operators serve it:

- "append": the norms of queries and keys for each head, the rotation of
  positions, and the write of keys and values into the cache, from the packed
  output of the query-key-value projection;
- "prompt": causal attention of packed sequences of different lengths over the
  cache (a whole prompt, or a chunk of one behind what is cached already);
- "tree": attention of a tree of drafted tokens (branches of the catalog's
  trie below the current node) over the cache; one drafted token is the single
  token of a plain decode step;
- "pages": copies of whole pages (a fork of a sequence) and the compaction of
  an accepted branch, in every layer of a cache.

Cache: [layers, pages, 2 (keys, values), kv_heads, page, head_dim].  Token t of
a sequence that has `ctx` tokens cached lies in slot ctx + t of its pages.

`own` false: elementary torch operations in 32 bits, rounded once at the end.
`own` true: the calls of the framework.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6
THETA = 1e6


# ------------------------------------------------------------------ the cases

def _case(op, name=None, **kw):
    c = {"op": op, "dtype": "bf16", "batch": 1, "q_heads": 32, "kv_heads": 8, "head_dim": 128, "page": 64,
         "t_lo": 1, "t_hi": 1, "c_lo": 0, "c_hi": 0, "lens": 1}
    if op == "append":
        c.update(norm=True, interleaved=False)
    if op == "pages":
        c.update(layers=4, copies=0)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # One new token of one sequence, hidden size 2048: the call's latency.
        _case("append", "append_one", q_heads=16, kv_heads=4, c_lo=777, c_hi=777, lens=11),
        # A batch of prompts of different lengths, 16k tokens together.
        _case("append", "append_prompts", dtype="f16", batch=16, t_lo=37, t_hi=2011, lens=12, interleaved=True),
        # Tool calls with short questions: sixteen prompts, each shorter than a
        # few tiles, every other one behind a cached preamble.
        _case("prompt", "prompt_short", batch=16, t_lo=5, t_hi=261, c_lo=0, c_hi=300, lens=21),
        # Chunks of long prompts behind cached context, narrow heads.
        _case("prompt", "prompt_chunks", dtype="f16", batch=4, head_dim=64, page=32, t_lo=1111, t_hi=2048,
              c_lo=1500, c_hi=6001, lens=22),
        # One long prompt, hidden size 4096.
        _case("prompt", "prompt_long", t_lo=8192, t_hi=8192, lens=23),
        # A decode step of one sequence, hidden size 2048: latency.
        _case("tree", "tree_one", q_heads=16, kv_heads=4, c_lo=1499, c_hi=1499, lens=31),
        # A decode step of a batch of 64 with contexts of different lengths.
        _case("tree", "tree_decode", batch=64, c_lo=97, c_hi=8011, lens=32),
        # Drafted branches of a catalog (42 names: up to 37 nodes), sixteen
        # sequences, no head shared.
        _case("tree", "tree_draft", dtype="f16", batch=16, q_heads=16, kv_heads=16, page=16, t_lo=9, t_hi=37,
              c_lo=800, c_hi=4097, lens=33),
        # A short draft over one very long cache.
        _case("tree", "tree_long", t_lo=7, t_hi=7, c_lo=131001, c_hi=131001, page=128, lens=34),
        # Drafts of the whole batch of 256.
        _case("tree", "tree_batch", batch=256, t_lo=3, t_hi=16, c_lo=201, c_hi=4001, lens=35),
        # Forks of 61 sequences: each child gets a copy of the last page.
        _case("pages", "pages_fork", layers=16, copies=61, lens=41),
        # The accepted branches of 64 sequences move together.
        _case("pages", "pages_compact", layers=16, batch=64, t_lo=12, t_hi=37, c_lo=300, c_hi=700, lens=42),
    ]


HEADS = [(16, 16), (16, 4), (32, 8), (32, 32), (28, 4), (16, 2), (12, 4), (8, 1)]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["append", "prompt", "prompt", "tree", "tree", "tree", "pages"])
    hq, hkv = rng.choice(HEADS)
    c = _case(op, dtype=rng.choice(["bf16", "f16"]), q_heads=hq, kv_heads=hkv, head_dim=rng.choice([64, 128]),
              page=rng.choice([16, 32, 64, 128]), lens=rng.randrange(1 << 30))
    if op == "append":
        c["norm"] = rng.random() < 0.8
        c["interleaved"] = rng.random() < 0.5
        c["batch"] = _spread(rng, 1, 64)
        c["t_hi"] = _spread(rng, 1, max(1, 16384 // c["batch"]))
        c["c_hi"] = rng.choice([0, _spread(rng, 1, 2000)])
        c["t_lo"], c["c_lo"] = (c["t_hi"] + 1) // 2, c["c_hi"] // 2
    elif op == "prompt":
        c["batch"] = _spread(rng, 1, 16)
        c["t_hi"] = _spread(rng, 3, 8192 // c["batch"])
        c["c_hi"] = rng.choice([0, _spread(rng, 1, 3000)])
        c["t_lo"], c["c_lo"] = (c["t_hi"] + 2) // 3, c["c_hi"] // 3
    elif op == "tree":
        c["batch"] = _spread(rng, 1, 256)
        c["t_hi"] = rng.choice([1, _spread(rng, 1, 64)])
        c["c_hi"] = _spread(rng, 1, min(131072, 2000000 // (c["batch"] * hkv)))
        c["t_lo"], c["c_lo"] = (c["t_hi"] + 1) // 2, c["c_hi"] // 4
    else:
        c["layers"] = rng.randrange(1, 17)
        if rng.random() < 0.5:
            c["copies"] = _spread(rng, 1, max(1, min(128, 250000000 // (c["layers"] * hkv * c["page"] * c["head_dim"]))))
        else:
            c["batch"] = _spread(rng, 1, 64)
            c["t_lo"], c["t_hi"] = 9, _spread(rng, 10, 64)
            c["c_lo"], c["c_hi"] = 1, _spread(rng, 2, 500)
            held = c["batch"] * hkv * c["head_dim"] * (c["t_hi"] + c["c_hi"] + c["page"])
            c["layers"] = max(1, min(c["layers"], 500000000 // held))
    return c


# ------------------------------------------- lengths and trees of a case (host)

def _lengths(case):
    """(drafted or prompt tokens, cached tokens) of each sequence: both ends of the ranges occur."""
    r = random.Random(case["lens"])
    n = case["batch"]
    t = [r.randint(case["t_lo"], case["t_hi"]) for _ in range(n)]
    c = [r.randint(case["c_lo"], case["c_hi"]) for _ in range(n)]
    t[-1], c[0] = case["t_hi"], case["c_hi"]
    return t, c


def _parents(case):
    """Parents of each sequence's drafted tokens (-1: the last cached token), in topological order."""
    r = random.Random(case["lens"] + 1)
    t, _ = _lengths(case)
    return [[-1 if i == 0 or r.random() < 0.1 else i - 1 if r.random() < 0.4 else r.randrange(max(0, i - 9), i)
             for i in range(n)] for n in t]


def _ancestors(parents):
    """Bit j of a token's word: it attends drafted token j (its ancestors and itself)."""
    words = []
    for i, p in enumerate(parents):
        words.append((words[p] if p >= 0 else 0) | 1 << i)
    return words


def _paths(case):
    """The accepted branch of each sequence: ascending draft indices, past the slots they move to."""
    r = random.Random(case["lens"] + 2)
    t, _ = _lengths(case)
    got = []
    for n in t:
        k = r.randint(1, max(1, min(8, n // 2)))
        same = r.randint(0, 1)
        got.append(list(range(same)) + sorted(r.sample(range(k, n), k - same)))
    return got


# --------------------------------------------------------------------- inputs

def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    hq, hkv, d, page, b = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"], case["batch"]
    op = case["op"]
    t, c = _lengths(case)
    if op == "pages" and case["copies"]:
        n = case["copies"]
        pool = torch.randn((case["layers"], 2 * n + 3, 2, hkv, page, d), generator=g, device="cuda", dtype=dt)
        order = torch.randperm(2 * n + 3, generator=g, device="cuda").to(torch.int32)
        return {"case": case, "pool": pool, "src": order[:n].contiguous(), "dst": order[n:2 * n].contiguous()}
    need = [-(-(x + y) // page) for x, y in zip(t, c)]
    pages, width = sum(need), max(need)
    layers = case.get("layers", 1)
    pool = torch.randn((layers, pages + 1, 2, hkv, page, d), generator=g, device="cuda", dtype=dt)
    # a sequence's pages lie anywhere in the pool; entries past its last page are never read
    order = torch.randperm(pages + 1, generator=g, device="cuda").to(torch.int32)
    first = [sum(need[:i]) for i in range(b)]
    at = _ints(first, torch.int64)[:, None] + torch.arange(width, device="cuda")
    held = torch.arange(width, device="cuda") < _ints(need)[:, None]
    table = torch.where(held, order[at.clamp(max=pages)], -1).to(torch.int32).contiguous()
    s = {"case": case, "pool": pool, "table": table, "ctx": _ints(c), "max_tokens": max(t), "scale": d ** -0.5}
    if op == "pages":
        paths = _paths(case)
        wide = max(len(p) for p in paths)
        s["path"] = _ints([p + [-1] * (wide - len(p)) for p in paths])
        s["n_path"] = _ints([len(p) for p in paths])
        s["lens_out"] = torch.empty_like(s["ctx"])
        return s
    cu = [0]
    for x in t:
        cu.append(cu[-1] + x)
    s["cu"] = _ints(cu)
    n = cu[-1]
    if op == "append":
        s["qkv"] = torch.randn((n, (hq + 2 * hkv) * d), generator=g, device="cuda", dtype=dt)
        if case["norm"]:
            s["q_weight"] = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(dt)
            s["k_weight"] = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(dt)
        depth = [i for x in t for i in range(x)]
        base = [y for x, y in zip(t, c) for _ in range(x)]
        s["positions"] = _ints([x + y for x, y in zip(depth, base)])
        top = max(x + y for x, y in zip(t, c))
        angle = torch.arange(top, device="cuda", dtype=torch.float64)[:, None] * (
            THETA ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d))
        s["rope"] = torch.stack((angle.cos(), angle.sin()), -1).float().contiguous()
        s["q"] = torch.empty((n, hq, d), dtype=dt, device="cuda")
        return s
    # queries as the append leaves them: normed per head, some heads sharper than others
    q = torch.randn((n, hq, d), generator=g, device="cuda")
    s["q"] = (q * (0.5 + torch.rand((1, hq, 1), generator=g, device="cuda") * 2)).to(dt)
    s["out"] = torch.empty((n, hq, d), dtype=dt, device="cuda")
    if op == "tree":
        words = -(-max(t) // 64)
        rows = [w for p in _parents(case) for w in _ancestors(p)]
        cut = [[(w >> 64 * k) & (1 << 64) - 1 for k in range(words)] for w in rows]
        s["tree"] = _ints([[x - (1 << 64) if x >> 63 else x for x in w] for w in cut], torch.int64)
    return s


# ----------------------------------------------------------- the framework's calls

def _cache(state):
    """The cache's handle, made once as a program does."""
    if "cache" not in state:
        from trie_constrained_decoding_gb300 import binding as tcd
        state["cache"] = tcd.KvCache(state["pool"])
    return state["cache"]


def _run_own(s):
    c, op = s["case"], s["case"]["op"]
    cache = _cache(s)
    if op == "append":
        cache.append(0, s["qkv"], s["cu"], s["ctx"], s["table"], s["q"], q_weight=s.get("q_weight"),
                     k_weight=s.get("k_weight"), eps=EPS, rope=s["rope"], positions=s["positions"],
                     interleaved=c["interleaved"])
        return {"q": s["q"], "cache": s["pool"]}
    if op in ("prompt", "tree"):
        cache.attend(0, s["q"], s["cu"], s["ctx"], s["table"], s["out"], s["max_tokens"], scale=s["scale"],
                     tree=s.get("tree"))
        return s["out"]
    if c["copies"]:
        cache.copy_pages(s["src"], s["dst"])
        return s["pool"]
    cache.compact(s["table"], s["ctx"], s["path"], s["n_path"], s["lens_out"])
    return {"cache": s["pool"], "lens": s["lens_out"]}


# ------------------------------------------------------------------ plain forms

def _tokens(s, n):
    """Sequence and index within the call of each packed token."""
    i = torch.arange(n, device="cuda")
    seq = torch.searchsorted(s["cu"][1:].long(), i, right=True)
    return seq, i - s["cu"].long()[seq]


def _plain_append(s):
    c = s["case"]
    hq, hkv, d, page = c["q_heads"], c["kv_heads"], c["head_dim"], c["page"]
    n = s["qkv"].shape[0]
    x = s["qkv"].float().view(n, hq + 2 * hkv, d)
    v = x[:, hq + hkv:]
    x = x[:, :hq + hkv]
    if c["norm"]:
        w = torch.cat((s["q_weight"].float().expand(hq, d), s["k_weight"].float().expand(hkv, d)))
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    rot = s["rope"][s["positions"].long()][:, None]
    cos, sin = rot[..., 0], rot[..., 1]
    if c["interleaved"]:
        a, b = x[..., 0::2], x[..., 1::2]
        x = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).reshape(x.shape)
    else:
        a, b = x[..., :d // 2], x[..., d // 2:]
        x = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    x = x.to(s["q"].dtype)
    s["q"].copy_(x[:, :hq])
    seq, t = _tokens(s, n)
    slot = s["ctx"].long()[seq] + t
    where = s["table"].long()[seq, slot // page]
    s["pool"][0][where, 0, :, slot % page] = x[:, hq:]
    s["pool"][0][where, 1, :, slot % page] = v.to(s["q"].dtype)
    return {"q": s["q"], "cache": s["pool"]}


def _plain_attend(s):
    c = s["case"]
    hq, hkv, d, b = c["q_heads"], c["kv_heads"], c["head_dim"], c["batch"]
    grp, tm, n = hq // hkv, s["max_tokens"], s["q"].shape[0]
    kv = s["pool"][0][s["table"].long().clamp(min=0)]         # [b, width, 2, hkv, page, d]
    kv = kv.permute(2, 0, 3, 1, 4, 5).reshape(2, b, hkv, -1, d).float()
    length = kv.shape[3]
    at = (s["cu"].long()[:-1, None] + torch.arange(tm, device="cuda")).clamp(max=n - 1)
    q = s["q"][at].float().view(b, tm, hkv, grp, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, tm * grp, d)
    w = torch.matmul(q, kv[0].transpose(-1, -2)).mul_(s["scale"])
    j = torch.arange(length, device="cuda") - s["ctx"].long()[:, None]    # slot's index within the call's tokens
    t = torch.arange(tm, device="cuda")
    if "tree" in s:
        words = s["tree"][at]
        k = j.clamp(min=0, max=64 * words.shape[-1] - 1)[:, None].expand(b, tm, length)
        bit = words.gather(2, k // 64) >> (k % 64) & 1
        seen = (j < 0)[:, None] | (bit != 0) & (j < 64 * words.shape[-1])[:, None]
    else:
        seen = j[:, None] <= t[:, None]
    seen = seen[:, None, :, None].expand(b, 1, tm, grp, length).reshape(b, 1, tm * grp, length)
    w.masked_fill_(~seen, -math.inf)
    top = w.amax(-1, keepdim=True)
    w.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w, kv[1]) / torch.where(total == 0, 1.0, total)
    o = o.view(b, hkv, tm, grp, d).permute(0, 2, 1, 3, 4).reshape(b, tm, hq, d)
    s["out"].copy_(o[_tokens(s, n)])
    return s["out"]


def _plain_copy(s):
    s["pool"][:, s["dst"].long()] = s["pool"][:, s["src"].long()]
    return s["pool"]


def _plain_compact(s):
    page = s["case"]["page"]
    last = s["n_path"].long()[:, None] - 1
    i = torch.arange(s["path"].shape[1], device="cuda").minimum(last)     # past the branch: its last move again
    to = s["ctx"].long()[:, None] + i
    frm = s["ctx"].long()[:, None] + s["path"].long().gather(1, i)
    rows = s["pool"].permute(1, 4, 0, 2, 3, 5)                            # [pages, page, layers, 2, hkv, d]
    table = s["table"].long()
    rows[table.gather(1, to // page), to % page] = rows[table.gather(1, frm // page), frm % page]
    s["lens_out"].copy_(s["ctx"] + s["n_path"])
    return {"cache": s["pool"], "lens": s["lens_out"]}


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "append":
        return _plain_append(state)
    if op in ("prompt", "tree"):
        return _plain_attend(state)
    return _plain_copy(state) if state["case"]["copies"] else _plain_compact(state)


# ------------------------------------------------------------------------ work

def work(case):
    """Each input read once, each output written once; products and sums of what the masks keep."""
    hq, hkv, d, op = case["q_heads"], case["kv_heads"], case["head_dim"], case["op"]
    t, c = _lengths(case)
    n = sum(t)
    if op == "pages" and case["copies"]:
        return {"bytes": 2 * 2 * case["copies"] * case["layers"] * 2 * hkv * case["page"] * d, "flops": 0}
    if op == "pages":
        moved = sum(i != x for p in _paths(case) for i, x in enumerate(p))
        return {"bytes": 2 * 2 * moved * case["layers"] * 2 * hkv * d + 16 * case["batch"], "flops": 0}
    if op == "append":
        angles = len({x + i for y, x in zip(t, c) for i in range(y)})
        return {"bytes": 2 * 2 * n * (hq + 2 * hkv) * d + 4 * angles * d + 4 * n,
                "flops": n * (hq + hkv) * d * (7 if case["norm"] else 3)}
    if op == "prompt":
        pairs = sum(x * y + x * (x + 1) // 2 for x, y in zip(t, c))
    else:
        pairs = sum(x * y for x, y in zip(t, c))
        pairs += sum(bin(w).count("1") for p in _parents(case) for w in _ancestors(p))
    kept = sum(x + y for x, y in zip(t, c))
    return {"bytes": 2 * 2 * n * hq * d + 2 * 2 * kept * hkv * d + 4 * sum(-(-(x + y) // case["page"]) for x, y in zip(t, c)),
            "flops": 4 * pairs * hq * d}


# --------------------------------------------------- the definition, in 64 bits

def _exact_append(s):
    c = s["case"]
    hq, hkv, d, page = c["q_heads"], c["kv_heads"], c["head_dim"], c["page"]
    cu, ctx, table = s["cu"].tolist(), s["ctx"].tolist(), s["table"].tolist()
    pool = s["pool"].double()
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    pair = (torch.arange(d // 2, device="cuda") * 2, torch.arange(d // 2, device="cuda") * 2 + 1) if c["interleaved"] else (
        torch.arange(d // 2, device="cuda"), torch.arange(d // 2, device="cuda") + d // 2)
    for b in range(c["batch"]):
        rows = s["qkv"][cu[b]:cu[b + 1]].double().unflatten(1, (-1, d))
        rot = s["rope"].double()[s["positions"][cu[b]:cu[b + 1]].long()]
        z = torch.complex(rot[..., 0], rot[..., 1])[:, None]

        def turned(x, weight):
            if c["norm"]:
                x = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * s[weight].double()
            y = torch.complex(x[..., pair[0]], x[..., pair[1]]) * z
            x = x.clone()
            x[..., pair[0]], x[..., pair[1]] = y.real, y.imag
            return x

        out[cu[b]:cu[b + 1]] = turned(rows[:, :hq], "q_weight")
        k, v = turned(rows[:, hq:hq + hkv], "k_weight"), rows[:, hq + hkv:]
        done = 0
        while done < k.shape[0]:
            slot = ctx[b] + done
            m = min(page - slot % page, k.shape[0] - done)
            p = pool[0, table[b][slot // page]]
            p[0, :, slot % page:slot % page + m] = k[done:done + m].transpose(0, 1)
            p[1, :, slot % page:slot % page + m] = v[done:done + m].transpose(0, 1)
            done += m
    return {"q": out, "cache": pool}


def _exact_attend(s):
    c = s["case"]
    hq, hkv, d, page = c["q_heads"], c["kv_heads"], c["head_dim"], c["page"]
    cu, ctx = s["cu"].tolist(), s["ctx"].tolist()
    grp = hq // hkv
    trees = _parents(c) if c["op"] == "tree" else None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b in range(c["batch"]):
        n = cu[b + 1] - cu[b]
        length = ctx[b] + n
        pages = s["table"][b, :-(-length // page)].long()
        k, v = (s["pool"][0, pages, i].transpose(0, 1).reshape(hkv, -1, d)[:, :length].double() for i in (0, 1))
        hidden = torch.ones(n, n, dtype=torch.bool)
        for i in range(n if trees else 0):
            hidden[i, i] = False
            p = trees[b][i]
            if p >= 0:
                hidden[i] &= hidden[p]
        hidden = (hidden if trees else hidden.triu(1)).cuda()
        for t0 in range(0, n, 2048):
            q = s["q"][cu[b] + t0:cu[b] + min(n, t0 + 2048)].double()
            for h in range(hq):
                x = q[:, h] @ k[h // grp].T * s["scale"]
                x[:, ctx[b]:][hidden[t0:t0 + 2048]] = -math.inf
                out[cu[b] + t0:cu[b] + min(n, t0 + 2048), h] = torch.softmax(x, -1) @ v[h // grp]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] in ("prompt", "tree"):
        return _exact_attend(s)
    # copies: the values themselves, moved one by one
    pool = s["pool"]
    if case["copies"]:
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            pool[:, b] = pool[:, a]
        return pool.double()
    page, table, ctx = case["page"], s["table"].tolist(), s["ctx"].tolist()
    for b, p in enumerate(_paths(case)):
        for i, x in enumerate(p):
            to, frm = ctx[b] + i, ctx[b] + x
            pool[:, table[b][to // page], :, :, to % page] = pool[:, table[b][frm // page], :, :, frm % page]
    lens = torch.tensor([x + len(p) for x, p in zip(ctx, _paths(case))], dtype=torch.int32)
    return {"cache": pool.double(), "lens": lens}
