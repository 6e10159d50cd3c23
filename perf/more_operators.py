"""Cases of the operators of a layer's step over sequences that share a prompt.

A tool-pointer decoder puts the same preamble (instructions and the catalog's
descriptions) in front of every question: its pages are read once and forked.
A layer of the model in front of the constrained step is then

- "linear": a projection, with bias, activation and residual in one pass
  (queries, keys and values; the attention's output; the way back from the
  feed-forward block);
- "gated": the first half of a gated feed-forward block, two projections, the
  activation of one and their product;
- "shared": attention of new tokens (one, or a drafted tree) over a cache whose
  first pages belong to a whole group of sequences and are read once for all of
  them.

  linear   y = act(x W^T + bias) + residual
  gated    y = act(x V^T + gate_bias) * (x W^T + bias)
  shared   out = sum_j p_j v_j / sum_j p_j over the slots that a token sees

`own` false: elementary torch operations in 32 bits, rounded once at the end.
`own` true: the calls of the framework.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


# ------------------------------------------------------------------ the cases

def _product(op, tokens, k, out, name=None, **kw):
    c = {"op": op, "dtype": "bf16", "tokens": tokens, "in": k, "out": out, "bias": False, "residual": False,
         "act": "none" if op == "linear" else "silu", "gap": 0}
    c.update(kw)
    if name:
        c["name"] = name
    return c


def _shared(name=None, **kw):
    c = {"op": "shared", "dtype": "bf16", "groups": 1, "batch": 4, "q_heads": 32, "kv_heads": 8, "head_dim": 128,
         "page": 64, "t_lo": 1, "t_hi": 1, "p_lo": 0, "p_hi": 0, "c_lo": 0, "c_hi": 0, "lens": 1}
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # The attention's output of one token, hidden size 2048, onto the residual: the call's latency.
        _product("linear", 1, 2048, 2048, "linear_one", residual=True),
        # Queries, keys and values (32 + 2 x 8 heads of 128) of a decode step of 64 sequences.
        _product("linear", 64, 4096, 6144, "linear_qkv", bias=True),
        # Back from the feed-forward block, the drafts of a batch together.
        _product("linear", 253, 14336, 4096, "linear_drafts", dtype="f16", residual=True),
        # Odd sizes, rows that are slices of wider ones.
        _product("linear", 1111, 1000, 2731, "linear_odd", dtype="f16", bias=True, act="gelu", gap=24),
        # Back from the feed-forward block, prompts of 8192 tokens together.
        _product("linear", 8192, 14336, 4096, "linear_prompt", residual=True),
        # One token, hidden size 2048.
        _product("gated", 1, 2048, 8192, "gated_one", dtype="f16"),
        # A decode step of 64 sequences, hidden size 4096.
        _product("gated", 64, 4096, 14336, "gated_step"),
        # Odd sizes, both biases.
        _product("gated", 777, 1000, 2731, "gated_odd", bias=True, act="gelu_tanh", gap=8),
        # Prompts of 4096 tokens together.
        _product("gated", 4096, 4096, 14336, "gated_prompt"),
        # Four sequences behind a short common prompt: latency.
        _shared("shared_few", q_heads=8, kv_heads=2, head_dim=64, page=16, p_lo=37, p_hi=37, c_lo=3, c_hi=21, lens=11),
        # A decode step of 64 sequences behind one catalog, a question each.
        _shared("shared_step", batch=64, p_lo=8003, p_hi=8003, c_lo=20, c_hi=300, lens=12),
        # Drafts of 256 sequences that use three catalogs.
        _shared("shared_drafts", dtype="f16", groups=3, batch=256, page=32, t_lo=3, t_hi=16, p_lo=1001, p_hi=4001,
                c_lo=50, c_hi=500, lens=13),
    ]


HEADS = [(16, 16), (16, 4), (32, 8), (28, 4), (16, 2), (12, 4), (8, 1)]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "gated", "gated", "shared", "shared"])
    dtype = rng.choice(["bf16", "f16"])
    if op != "shared":
        k = 8 * _spread(rng, 32, 1792)
        out = _spread(rng, 64, 14336)
        most = 8192 * 14336 * 4096 // (1 if op == "linear" else 2)
        tokens = _spread(rng, 1, max(1, min(8192, most // (k * out))))
        return _product(op, tokens, k, out, dtype=dtype, bias=rng.random() < 0.5, residual=rng.random() < 0.5,
                        act=rng.choice(ACTS if op == "linear" else ACTS[1:]), gap=rng.choice([0, 0, 8, 56]))
    hq, hkv = rng.choice(HEADS)
    c = _shared(dtype=dtype, q_heads=hq, kv_heads=hkv, head_dim=rng.choice([64, 128]),
                page=rng.choice([16, 32, 64, 128]), lens=rng.randrange(1 << 30))
    c["batch"] = _spread(rng, 2, 256)
    c["groups"] = rng.randrange(1, 1 + min(4, c["batch"] // 2))
    c["t_hi"] = rng.choice([1, _spread(rng, 1, 16)])
    c["t_lo"] = (c["t_hi"] + 2) // 3
    c["p_hi"] = _spread(rng, 16, min(32000, 1000000 // c["batch"]))
    c["p_lo"] = c["p_hi"] // 3
    c["c_hi"] = _spread(rng, 1, min(600, 80000 // c["batch"]))
    c["c_lo"] = c["c_hi"] // 8
    return c


# ------------------------------------------- lengths and trees of a case (host)

def _lengths(case):
    """Per sequence: new tokens, slots behind the prefix, group; per group: the prefix.  Both ends of the ranges occur."""
    r = random.Random(case["lens"])
    n, groups = case["batch"], case["groups"]
    t = [r.randint(case["t_lo"], case["t_hi"]) for _ in range(n)]
    c = [r.randint(case["c_lo"], case["c_hi"]) for _ in range(n)]
    t[-1], c[0] = case["t_hi"], case["c_hi"]
    cuts = sorted(r.sample(range(1, n), groups - 1))
    first = [0] + cuts + [n]
    p = [r.randint(case["p_lo"], case["p_hi"]) for _ in range(groups)]
    p[0] = case["p_hi"]
    return t, c, first, p


def _parents(case):
    """Parents of each sequence's drafted tokens (-1: the last cached token), in topological order."""
    r = random.Random(case["lens"] + 1)
    return [[-1 if i == 0 or r.random() < 0.1 else i - 1 if r.random() < 0.4 else r.randrange(max(0, i - 9), i)
             for i in range(n)] for n in _lengths(case)[0]]


def _ancestors(parents):
    """Bit j of a token's word: it attends drafted token j (its ancestors and itself)."""
    words = []
    for i, p in enumerate(parents):
        words.append((words[p] if p >= 0 else 0) | 1 << i)
    return words


# --------------------------------------------------------------------- inputs

def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype).cuda()


def _prepare_product(case, g):
    dt, n, k, out = DTYPES[case["dtype"]], case["tokens"], case["in"], case["out"]

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dt)

    s = {"case": case, "x": normal(n, k + case["gap"])[:, :k], "w": normal(out, k, scale=k ** -0.5),
         "y": torch.empty((n, out), dtype=dt, device="cuda")}
    if case["op"] == "gated":
        s["gate"] = normal(out, k, scale=1.5 * k ** -0.5)
    if case["bias"]:
        s["bias"] = normal(out, scale=0.3)
        if case["op"] == "gated":
            s["gate_bias"] = normal(out, scale=0.3)
    if case["residual"]:
        s["residual"] = normal(n, out, scale=2.0)
    return s


def _prepare_shared(case, g):
    dt = DTYPES[case["dtype"]]
    hq, hkv, d, page, b = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"], case["batch"]
    t, c, first, p = _lengths(case)
    of = [j for j in range(case["groups"]) for _ in range(first[j + 1] - first[j])]
    whole = [x // page for x in p]                                       # pages that a group shares
    ctx = [p[of[i]] + c[i] for i in range(b)]
    need = [-(-(x + y) // page) for x, y in zip(t, ctx)]
    pages = sum(whole) + sum(need[i] - whole[of[i]] for i in range(b))
    pool = torch.randn((1, pages + 1, 2, hkv, page, d), generator=g, device="cuda", dtype=dt)
    # pages lie anywhere in the pool; entries past a sequence's last page are never read
    order = torch.randperm(pages + 1, generator=g, device="cuda").to(torch.int32)
    width, at, start = max(need), sum(whole), []
    for i in range(b):
        start.append(at - whole[of[i]])
        at += need[i] - whole[of[i]]
    j = torch.arange(width, device="cuda")
    in_prefix = j < _ints([whole[x] for x in of])[:, None]
    index = torch.where(in_prefix, _ints([sum(whole[:x]) for x in of], torch.int64)[:, None] + j,
                        _ints(start, torch.int64)[:, None] + j)
    table = torch.where(j < _ints(need)[:, None], order[index.clamp(max=pages)], -1).to(torch.int32).contiguous()
    cu = [0]
    for x in t:
        cu.append(cu[-1] + x)
    # queries as the append leaves them: normed per head, some heads sharper than others
    q = torch.randn((cu[-1], hq, d), generator=g, device="cuda")
    q = (q * (0.5 + torch.rand((1, hq, 1), generator=g, device="cuda") * 2)).to(dt)
    # the most tokens of a group, pages of a prefix, and pages that a sequence has for itself
    sizes = (max(sum(t[x:y]) for x, y in zip(first, first[1:])), max(max(whole), 1),
             max(x - whole[y] for x, y in zip(need, of)))
    return {"case": case, "sizes": sizes, "pool": pool, "table": table, "ctx": _ints(ctx), "cu": _ints(cu), "cu_seqs": _ints(first),
            "shared": _ints(p), "max_tokens": max(t), "scale": d ** -0.5, "q": q, "out": torch.empty_like(q),
            "tree": _ints([[w] for x in _parents(case) for w in _ancestors(x)], torch.int64)}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return _prepare_shared(case, g) if case["op"] == "shared" else _prepare_product(case, g)


# ----------------------------------------------------------- the framework's calls

def _run_own(s):
    from trie_constrained_decoding_gb300 import binding as tcd
    if s["case"]["op"] == "shared":
        if "cache" not in s:                 # the cache's handle, made once as a program does
            s["cache"] = tcd.KvCache(s["pool"])
        s["cache"].attend_shared(0, s["q"], s["cu"], s["ctx"], s["table"], s["out"], s["max_tokens"], s["cu_seqs"],
                                 s["shared"], scale=s["scale"], tree=s["tree"])
        return s["out"]
    if "linear" not in s:                    # the layer's weights, the same
        act = getattr(tcd, "ACT_" + s["case"]["act"].upper())
        s["linear"] = tcd.Linear(s["w"], bias=s.get("bias"), gate=s.get("gate"), gate_bias=s.get("gate_bias"), act=act)
    s["linear"].apply(s["x"], s["y"], residual=s.get("residual"))
    return s["y"]


# ------------------------------------------------------------------ plain forms

def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z / (1 + (-z).exp())
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 2 ** -0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))
    return z


def _plain_product(s):
    x = s["x"].float()
    y = torch.matmul(x, s["w"].float().T)
    if "bias" in s:
        y = y + s["bias"].float()
    if "gate" in s:
        g = torch.matmul(x, s["gate"].float().T)
        if "gate_bias" in s:
            g = g + s["gate_bias"].float()
        y = _act(g, s["case"]["act"]) * y
    else:
        y = _act(y, s["case"]["act"])
    if "residual" in s:
        y = y + s["residual"].float()
    s["y"].copy_(y)
    return s["y"]


def _softmax_part(q, k, v, seen, scale):
    """Unnormalised output, largest score and sum of the weights of the slots seen."""
    w = torch.matmul(q, k.transpose(-1, -2)).mul_(scale).masked_fill_(~seen, -math.inf)
    top = w.amax(-1, keepdim=True)
    w.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    return torch.matmul(w, v), top, w.sum(-1, keepdim=True)


def _plain_shared(s):
    c = s["case"]
    hq, hkv, d, b, page = c["q_heads"], c["kv_heads"], c["head_dim"], c["batch"], c["page"]
    grp, tm, n = hq // hkv, s["max_tokens"], s["q"].shape[0]
    most, prefix_pages, wide = s["sizes"]
    cu, table = s["cu"].long(), s["table"].long().clamp(min=0)
    i = torch.arange(n, device="cuda")
    seq = torch.searchsorted(cu[1:], i, right=True)
    cu_seqs = s["cu_seqs"].long()
    group = torch.searchsorted(cu_seqs[1:], torch.arange(b, device="cuda"), right=True)
    whole = s["shared"].long() // page

    def heads(at):      # rows of packed tokens at [x, rows] -> [x, kv heads, rows x heads of a group, d]
        x, rows = at.shape
        return s["q"][at].float().view(x, rows, hkv, grp, d).permute(0, 2, 1, 3, 4).reshape(x, hkv, rows * grp, d)

    def tokens(o, x, at):     # back to packed tokens
        e = o.shape[-1]
        return o.view(o.shape[0], hkv, -1, grp, e).permute(0, 2, 1, 3, 4)[x, at].reshape(n, hq, e)

    def cached(rows):         # [x, pages] -> keys and values [x, kv heads, slots, d]
        kv = s["pool"][0][rows].permute(2, 0, 3, 1, 4, 5)
        return kv.reshape(2, rows.shape[0], hkv, -1, d).float()

    # the prefixes, for all rows of a group
    begin = cu[cu_seqs[:-1]]
    k, v = cached(table[cu_seqs[:-1], :prefix_pages])
    at = (begin[:, None] + torch.arange(most, device="cuda")).clamp(max=n - 1)
    seen = torch.arange(k.shape[2], device="cuda") < (whole * page)[:, None]
    part = _softmax_part(heads(at), k, v, seen[:, None, None], s["scale"])
    o1, m1, l1 = (tokens(x, group[seq], i - begin[group[seq]]) for x in part)
    # what each sequence has for itself
    pages = whole[group][:, None] + torch.arange(wide, device="cuda")
    k, v = cached(table.gather(1, pages.clamp(max=table.shape[1] - 1)))
    at = (cu[:-1, None] + torch.arange(tm, device="cuda")).clamp(max=n - 1)
    slot = (whole[group] * page)[:, None] + torch.arange(wide * page, device="cuda")
    j = slot - s["ctx"].long()[:, None]                        # slot's index within the call's tokens
    bit = s["tree"][at][..., 0][..., None] >> j.clamp(min=0, max=63)[:, None] & 1
    seen = (j < 0)[:, None] | (bit != 0) & (j < 64)[:, None]
    seen = seen[:, None, :, None].expand(b, 1, tm, grp, wide * page).reshape(b, 1, tm * grp, wide * page)
    part = _softmax_part(heads(at), k, v, seen, s["scale"])
    o2, m2, l2 = (tokens(x, seq, i - cu[seq]) for x in part)
    top = torch.maximum(m1, m2)
    f1, f2 = (m1 - top).exp(), (m2 - top).exp()
    s["out"].copy_((o1 * f1 + o2 * f2) / (l1 * f1 + l2 * f2))
    return s["out"]


def run(state):
    if own:
        return _run_own(state)
    return _plain_shared(state) if state["case"]["op"] == "shared" else _plain_product(state)


# ------------------------------------------------------------------------ work

def work(case):
    """Each input read once, each output written once; products of what the masks keep."""
    if case["op"] != "shared":
        n, k, out = case["tokens"], case["in"], case["out"]
        w = 1 if case["op"] == "linear" else 2
        return {"bytes": 2 * (n * k + w * out * k + (2 if case["residual"] else 1) * n * out +
                              (w * out if case["bias"] else 0)),
                "flops": 2 * w * n * k * out}
    hq, hkv, d, page = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"]
    t, c, first, p = _lengths(case)
    of = [j for j in range(case["groups"]) for _ in range(first[j + 1] - first[j])]
    pairs = sum(x * (y + p[g]) for x, y, g in zip(t, c, of))
    pairs += sum(bin(w).count("1") for x in _parents(case) for w in _ancestors(x))
    kept = sum(x // page * page for x in p) + sum(x + y + p[g] % page for x, y, g in zip(t, c, of))
    return {"bytes": 2 * 2 * sum(t) * hq * d + 2 * 2 * kept * hkv * d + 8 * sum(t), "flops": 4 * pairs * hq * d}


# --------------------------------------------------- the definition, in 64 bits

def _exact_product(s):
    act = s["case"]["act"]
    out = torch.empty(s["y"].shape, dtype=torch.float64, device="cuda")
    w = s["w"].double()
    gate = s["gate"].double() if "gate" in s else None

    def turn(z):
        if act == "none":
            return z
        if act == "relu":
            return torch.where(z > 0, z, torch.zeros_like(z))
        if act == "silu":
            return z * torch.sigmoid(z)
        if act == "gelu":
            return z * torch.special.ndtr(z)
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))

    for i in range(0, out.shape[0], 1024):
        x = s["x"][i:i + 1024].double()
        z = x @ w.T + (s["bias"].double() if "bias" in s else 0)
        if gate is None:
            z = turn(z)
        else:
            z = turn(x @ gate.T + (s["gate_bias"].double() if "gate_bias" in s else 0)) * z
        out[i:i + 1024] = z + (s["residual"][i:i + 1024].double() if "residual" in s else 0)
    return out


def _exact_shared(s):
    c = s["case"]
    hq, hkv, d, page = c["q_heads"], c["kv_heads"], c["head_dim"], c["page"]
    cu, ctx = s["cu"].tolist(), s["ctx"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, parents in enumerate(_parents(c)):
        n = cu[b + 1] - cu[b]
        length = ctx[b] + n
        pages = s["table"][b, :-(-length // page)].long()
        k, v = (s["pool"][0, pages, i].transpose(0, 1).reshape(hkv, -1, d)[:, :length].double() for i in (0, 1))
        hidden = torch.ones(n, n, dtype=torch.bool)
        for i, p in enumerate(parents):
            hidden[i, i] = False
            if p >= 0:
                hidden[i] &= hidden[p]
        q = s["q"][cu[b]:cu[b + 1]].double().transpose(0, 1).reshape(hkv, hq // hkv, n, d)
        x = torch.einsum("hgnd,hld->hgnl", q, k) * s["scale"]
        x[..., ctx[b]:][:, :, hidden.cuda()] = -math.inf
        o = torch.einsum("hgnl,hld->hgnd", torch.softmax(x, -1), v)
        out[cu[b]:cu[b + 1]] = o.reshape(hq, n, d).transpose(0, 1)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_shared(s) if case["op"] == "shared" else _exact_product(s)
