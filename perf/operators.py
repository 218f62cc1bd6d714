"""Workloads of the 8-bit KV cache: its writes, the tree attention over it, and its eviction.

Four operators, each over a cache of rows [B][Hkv][cap][d] (or pages of it):

  attn     branch-aware attention of a draft tree over an 8-bit prefix cache
  write    rows appended to an 8-bit cache (a prefill, or a commit of the accepted path)
  weights  attention weight that every cached token received from the accepted rows
  evict    the cache cut to a budget by those weights

The 8-bit cache holds e4m3 codes and one exponent byte e for each 64 tokens of a
head: a value is code * 2^(e - 127).

``own`` selects the framework's calls; otherwise ``run`` computes the same with
elementary torch operations in 32 bits.
"""

import math
import random

import torch

own = False

BLOCK = 64                    # tokens that share an exponent
E_MIN, E_MAX = 10, 246        # exponents that a write gives
DEV = "cuda" if torch.cuda.is_available() else "cpu"   # the plain forms run on either


# ------------------------------------------------------------------ cases --

def listed():
    gqa = dict(Hq=32, Hkv=8, dk=128, dv=128, dtype="bf16", page=0)
    return [
        # one request, one token at a time: the smallest call, all latency
        dict(name="attn token", op="attn", B=1, R=1, P=2048, P_min=2048, **gqa),
        # one request, a 16-node tree: an interactive user
        dict(name="attn tree", op="attn", B=1, R=17, P=2048, P_min=2048, **gqa),
        # a served batch of ragged requests with 32-node trees over a paged cache
        dict(name="attn batch", op="attn", B=32, R=33, P=4096, P_min=1024, **{**gqa, "page": 256}),
        # long documents, the largest tree
        dict(name="attn long tree", op="attn", B=8, R=65, P=32768, P_min=32768, **gqa),
        # long documents, plain decoding: every byte of the cache is read for four rows a head
        dict(name="attn long token", op="attn", B=16, R=1, P=32768, P_min=20001, **gqa),
        # latent heads: 128 query heads of a small tree over one compressed row a token
        dict(name="attn latent", op="attn", B=64, R=9, P=8192, P_min=8192, Hq=128, Hkv=1, dk=576, dv=512,
             dtype="bf16", page=0),
        # the accepted paths of a served batch
        dict(name="write path", op="write", B=32, R=33, S=7, T=0, P=4096, P_min=1024, **gqa),
        # prompts of ragged length, behind a cached system prompt that ends inside a block
        dict(name="write prompt", op="write", B=4, R=1, S=0, T=8192, P=200, P_min=1, **gqa),
        # weights of a long document in a 16-bit cache
        dict(name="weights 16-bit", op="weights", q8=False, B=4, R=33, S=8, P=32768, P_min=30001, **gqa),
        # weights of a served batch in the 8-bit cache
        dict(name="weights 8-bit", op="weights", q8=True, B=32, R=33, S=7, P=4096, P_min=1024, **gqa),
        # a long document cut to half its length in one go
        dict(name="evict to half", op="evict", q8=False, B=4, P=32768, P_min=32768, keep=16384, sink=4, recent=512,
             **gqa),
        # a served batch held at a budget: a few rows leave in each round
        dict(name="evict a few", op="evict", q8=True, B=32, P=4104, P_min=4090, keep=4096, sink=4, recent=256, **gqa),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "write", "weights", "evict"])
    kind = rng.choice(["gqa", "gqa", "gqa", "wide", "narrow", "single", "latent"])
    dtype = "f32" if rng.random() < 0.12 else "bf16"
    c = {"gqa": dict(Hq=32, Hkv=8, dk=128, dv=128), "wide": dict(Hq=64, Hkv=8, dk=128, dv=128),
         "narrow": dict(Hq=14, Hkv=2, dk=64, dv=64), "single": dict(Hq=8, Hkv=8, dk=128, dv=128),
         "latent": dict(Hq=128, Hkv=1, dk=576, dv=512)}[kind]
    c = dict(op=op, dtype=dtype, page=rng.choice([0, 0, 128, 256]), B=_log(rng, 1, 32), P=_log(rng, 1, 32768), **c)
    # a drawn case reads no more cache, and computes no more, than the largest listed ones
    while c["B"] * c["P"] > (8192 if dtype == "f32" else 262144):
        c["B"], c["P"] = max(1, c["B"] // 2), c["P"] if c["B"] > 1 else c["P"] // 2
    if op == "attn":
        c["R"] = rng.choice([1, 1, 2, rng.randint(3, 65)])
        while c["R"] > 1 and c["B"] * c["R"] * c["P"] * c["Hq"] * (c["dk"] + c["dv"]) > (3e9 if dtype == "f32" else 2e11):
            c["R"] = c["R"] // 2
    elif op == "write":
        c["R"], c["S"] = rng.randint(17, 65), rng.randint(1, 16)
        c["T"] = 0 if rng.random() < 0.5 else _log(rng, 1, 8192)
        if c["T"]:
            c.update(P=rng.randint(1, 300), B=max(1, min(c["B"], 32768 // c["T"])))
    elif op == "weights":
        c.update(q8=rng.random() < 0.5, R=rng.randint(17, 65), S=rng.randint(1, 16))
        while c["B"] * c["P"] * c["Hq"] * c["dk"] * (1 + c["S"]) > 1e11:
            c["P"] = c["P"] // 2
    else:
        c.update(q8=rng.random() < 0.6, P=max(c["P"], 8))
        c["keep"] = max(3, int(c["P"] * rng.choice([0.25, 0.5, 0.9, 0.999])))
        c["sink"], c["recent"] = rng.randint(0, c["keep"] // 3), rng.randint(0, c["keep"] // 3)
    c["P_min"] = max(1, int(c["P"] * rng.uniform(0.3, 1.0)))
    return c


# ----------------------------------------------------------------- inputs --

def _cap(c):
    n = c["P"] + 1 + max(c.get("S", 0), c.get("T", 0))
    return n if not c["page"] else -(-n // c["page"]) * c["page"]


def _tree_masks(rnd, B, R):
    """Ancestor-or-self masks of random trees: bit j - 1 for row j >= 1."""
    out = []
    for _ in range(B):
        m = [0]
        for r in range(1, R):
            v = m[rnd.randrange(max(0, r - 6), r)] | (1 << (r - 1))
            m.append(v)
        out.append([v - (1 << 64) if v >> 63 else v for v in m])
    return torch.tensor(out, dtype=torch.int64, device=DEV)


def prepare(case, seed):
    c = case
    rnd = random.Random(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    B, Hq, Hkv, dk, dv = c["B"], c["Hq"], c["Hkv"], c["dk"], c["dv"]
    latent = dk != dv
    dt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    cap = _cap(c)
    op = c["op"]
    q8 = c.get("q8", True)

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)

    lens = [rnd.randint(c["P_min"], c["P"]) for _ in range(B)]
    lens[rnd.randrange(B)] = c["P"]
    s = dict(case=dict(c), op=op, q8=q8, latent=latent, dt=dt, cap=cap, scale=1.0 / math.sqrt(dk), kept={})
    s["plen"] = torch.tensor(lens, dtype=torch.int32, device=DEV)

    # the cache: [B][Hkv][cap][d], or pages [pages][Hkv][page][d] in a shuffled order with a few unused ones
    if c["page"]:
        per = cap // c["page"]
        pages = B * per + 3
        order = rnd.sample(range(pages), B * per)
        s["table"] = torch.tensor(order, dtype=torch.int32, device=DEV).view(B, per)
        lead, rows = (pages, Hkv), c["page"]
    else:
        s["table"] = None
        lead, rows = (B, Hkv), cap

    def cache(d):
        if not q8:
            return normal(*lead, rows, d)
        return (torch.randn(*lead, rows, d, generator=g, device=DEV) * 110).clamp_(-448, 448).to(torch.float8_e4m3fn)

    def exps():
        return torch.randint(118, 122, (*lead, -(-rows // BLOCK)), generator=g, device=DEV, dtype=torch.uint8)

    s["k"], s["v"] = cache(dk), None if latent else cache(dv)
    if q8:
        s["ke"], s["ve"] = exps(), None if latent else exps()

    if op in ("attn", "weights"):
        s["q"] = normal(B, c["R"], Hq, dk)
        s["kt"], s["vt"] = normal(B, c["R"], Hkv, dk), None if latent else normal(B, c["R"], Hkv, dv)
    if op == "attn":
        s["mask"] = _tree_masks(rnd, B, c["R"])
    if op in ("write", "weights"):
        S = c["S"]
        if c.get("T"):
            s["x"] = normal(B, c["T"], Hkv, dk)
            s["y"] = None if latent else normal(B, c["T"], Hkv, dv)
            n = [rnd.randint(max(1, c["T"] // 2), c["T"]) for _ in range(B)]
            s["n"] = torch.tensor(n, dtype=torch.int32, device=DEV)
        else:
            ls, paths = [], []
            for _ in range(B):
                L = rnd.randint(0, min(S, c["R"] - 1))
                ls.append(L)
                paths.append([0] + sorted(rnd.sample(range(1, c["R"]), L)) + [-1] * (S - L))
            s["alen"] = torch.tensor(ls, dtype=torch.int32, device=DEV)
            s["arows"] = torch.tensor(paths, dtype=torch.int32, device=DEV)
            if op == "write":
                s["kt"] = normal(B, c["R"], Hkv, dk)
                s["vt"] = None if latent else normal(B, c["R"], Hkv, dv)
        s["plen0"] = s["plen"].clone()
    if op in ("weights", "evict"):
        # weights so far: a few tokens hold most of the attention
        s["acc"] = torch.rand(B, Hkv, cap, generator=g, device=DEV).pow_(6).mul_(20)
        # earlier evictions left the rows in any order; 100 tokens of each request are gone
        inside = (torch.arange(cap, device=DEV) < s["plen"][:, None])[:, None]
        order = torch.rand(B, Hkv, cap, generator=g, device=DEV).masked_fill_(~inside, 2.0).argsort(-1)
        rank = torch.empty_like(order).scatter_(-1, order, torch.arange(cap, device=DEV).expand_as(order))
        s["pos"] = torch.where(inside, rank + 100 * (rank >= 4), torch.full_like(rank, -1)).int()
        s["seen"] = (s["plen"][:, None] + 100).expand(B, Hkv).contiguous()
    if op == "weights":
        # the log-sum-exp that the attention of the same rows left
        q = _path_rows(s["q"], s["arows"])
        sc = _scores(q, _values(s, "k", "ke"), Hkv) * s["scale"]
        sc.masked_fill_(torch.arange(cap, device=DEV) >= s["plen"][:, None, None, None, None], -math.inf)
        st = _scores(q, _path_rows(s["kt"], s["arows"]).permute(0, 2, 1, 3).float(), Hkv) * s["scale"]
        i = torch.arange(st.shape[2], device=DEV)
        st.masked_fill_(i[None, :] > i[:, None, None], -math.inf)
        lse = torch.logsumexp(torch.cat([sc, st], -1), -1).permute(0, 2, 1, 3).reshape(B, -1, Hq)
        i = torch.where(s["arows"] < 0, c["R"], s["arows"]).long()
        s["lse"] = torch.zeros(B, c["R"] + 1, Hq, device=DEV)
        s["lse"] = s["lse"].scatter_(1, i[:, :, None].expand(-1, -1, Hq), lse)[:, :-1].contiguous()
        s["decay"] = 0.75
    if op == "evict":
        s["plen0"], s["acc0"], s["pos0"] = s["plen"].clone(), s["acc"].clone(), s["pos"].clone()
    return s


def _path_rows(x, arows):
    """Rows of x [B][R][..] that the path names (row 0 in the place of the -1 behind its end)."""
    i = arows.long().clamp(min=0)
    return x.gather(1, i.view(*i.shape, *([1] * (x.dim() - 2))).expand(-1, -1, *x.shape[2:]))


def _scores(q, k, Hkv):
    """q [B][n][Hq][d], k [B][Hkv][keys][d] fp32 -> [B][Hkv][n][group][keys]."""
    B, n, Hq, d = q.shape
    q = q.float().view(B, n, Hkv, Hq // Hkv, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, d)
    return torch.matmul(q, k.transpose(-1, -2)).view(B, Hkv, n, Hq // Hkv, -1)


def _gathered(s, x):
    """A paged array [pages][Hkv][rows][..] as [B][Hkv][cap rows][..]; a contiguous one as it is."""
    if s["table"] is None:
        return x
    B, per = s["table"].shape
    x = x[s["table"].long()].transpose(1, 2)
    return x.reshape(B, x.shape[1], per * x.shape[3], *x.shape[4:])


def _put(s, x, new):
    """The reverse of _gathered: `new` into x."""
    if s["table"] is None:
        x.copy_(new)
        return
    B, per = s["table"].shape
    new = new.reshape(B, new.shape[1], per, x.shape[2], *x.shape[3:]).transpose(1, 2)
    x[s["table"].long().view(-1)] = new.reshape(B * per, *x.shape[1:])


def _power(e):
    """2^e for whole e in [-126, 127], by its bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _values(s, name, ename):
    """The cache's values in 32 bits, [B][Hkv][cap][d]."""
    x = _gathered(s, s[name].view(torch.uint8)).view(torch.float8_e4m3fn).float() if s["q8"] else \
        _gathered(s, s[name]).float()
    if s["q8"]:
        e = _gathered(s, s[ename]).int()
        x *= _power(e - 127).repeat_interleave(BLOCK, 2)[:, :, : x.shape[2], None]
    return x


# ------------------------------------------------------------ plain forms --

def _plain_attn(s):
    c = s["case"]
    B, R, Hq, Hkv, dv = c["B"], c["R"], c["Hq"], c["Hkv"], c["dv"]
    k = torch.cat([_values(s, "k", "ke"), s["kt"].float().transpose(1, 2)], 2)
    v = k[..., :dv] if s["latent"] else torch.cat([_values(s, "v", "ve"), s["vt"].float().transpose(1, 2)], 2)
    sc = _scores(s["q"], k, Hkv)
    sc *= s["scale"]
    j = torch.arange(R, device=DEV)
    seen = (s["mask"][:, :, None] >> (j - 1).clamp(min=0)) & 1                    # [B][R][R]
    seen = torch.where(j[None, :, None] == 0, torch.zeros_like(seen), seen).bool() | (j == 0)
    prefix = torch.arange(s["cap"], device=DEV) < s["plen"][:, None]
    seen = torch.cat([prefix[:, None, :].expand(-1, R, -1), seen], 2)             # [B][R][cap + R]
    sc.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = sc.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(B, Hkv, -1, p.shape[-1]), v).view(B, Hkv, R, Hq // Hkv, dv) / total
    out = out.permute(0, 2, 1, 3, 4).reshape(B, R, Hq, dv).to(s["dt"])
    lse = (total.log() + m).permute(0, 2, 1, 3, 4).reshape(B, R, Hq)
    return {"out": out, "lse": lse}


def _plain_write_rows(s, name, ename, x, n):
    """x [B][T][Hkv][d]: n[b] rows of it behind the first plen[b] ones of the cache."""
    codes = _gathered(s, s[name].view(torch.uint8)).view(torch.float8_e4m3fn).float()
    e_old = _gathered(s, s[ename]).int()
    B, Hkv, cap, d = codes.shape
    nb = e_old.shape[2]
    at = torch.arange(cap, device=DEV)
    p = s["plen"].long()[:, None]
    t = at - p
    new = (t >= 0) & (t < n.long()[:, None])                                      # [B][cap]
    rows = x.float().gather(1, t.clamp(0, x.shape[1] - 1)[:, :, None, None].expand(-1, -1, Hkv, d)).transpose(1, 2)
    mag = torch.where(new[:, None, :, None] & rows.isfinite(), rows.abs(), torch.zeros_like(rows)).amax(-1)
    mag = torch.nn.functional.pad(mag, (0, nb * BLOCK - cap)).view(B, Hkv, nb, BLOCK).amax(-1)
    part, ex = torch.frexp(mag)
    need = torch.where(mag == 0, torch.full_like(ex, E_MIN), ex - 9 + (part > 0.875).int() + 127).clamp(E_MIN, E_MAX)
    first = torch.arange(nb, device=DEV) * BLOCK
    touched = ((first < p + n.long()[:, None]) & (first + BLOCK > p) & (n[:, None] > 0))[:, None]
    e = torch.where(touched, torch.where((first < p)[:, None], torch.maximum(need, e_old), need), e_old)

    def wide(a):
        return a.repeat_interleave(BLOCK, 2)[:, :, :cap, None]

    kept = codes * wide(_power((e_old - e).clamp(-100, 100)))
    made = rows * wide(_power(127 - e.clamp(E_MIN, E_MAX)))
    change = touched & (first < p)[:, None] & (e != e_old)
    old = wide(change) & (at < p)[:, None, :, None]
    out = torch.where(new[:, None, :, None], made.clamp(-448, 448), torch.where(old, kept, codes))
    _put(s, s[name].view(torch.uint8), out.to(torch.float8_e4m3fn).view(torch.uint8))
    _put(s, s[ename], e.to(torch.uint8))


def _plain_write(s):
    s["plen"].copy_(s["plen0"])
    if "x" in s:
        x, y, n = s["x"], s["y"], s["n"]
    else:
        x, n = _path_rows(s["kt"], s["arows"]), s["alen"] + 1
        y = None if s["latent"] else _path_rows(s["vt"], s["arows"])
    _plain_write_rows(s, "k", "ke", x, n)
    if y is not None:
        _plain_write_rows(s, "v", "ve", y, n)
    s["plen"] += n
    return _written(s)


def _written(s):
    out = {"k": s["k"], "ke": s["ke"], "plen": s["plen"]}
    return out if s["latent"] else {**out, "v": s["v"], "ve": s["ve"]}


def _plain_weights(s):
    c = s["case"]
    Hkv, n = c["Hkv"], c["S"] + 1
    q = _path_rows(s["q"], s["arows"])
    lse = _path_rows(s["lse"], s["arows"]).view(c["B"], n, Hkv, -1).permute(0, 2, 1, 3)[..., None]
    live = (torch.arange(n, device=DEV) <= s["alen"][:, None])[:, None, :, None, None]

    def received(k, seen):
        p = torch.exp(_scores(q, k, Hkv) * s["scale"] - lse)
        return torch.where(live & seen, p, torch.zeros_like(p)).sum((2, 3))       # [B][Hkv][keys]

    at = torch.arange(s["cap"], device=DEV)
    prefix = (at < s["plen"][:, None])[:, None]
    got = received(_values(s, "k", "ke"), prefix[:, :, None, None, :])
    acc = torch.where(prefix, s["acc"] * s["decay"] + got, s["acc"])
    i = torch.arange(n, device=DEV)
    path = received(_path_rows(s["kt"], s["arows"]).float().transpose(1, 2), i[:, None, None] >= i)
    j = at - s["plen"][:, None]
    fresh = ((j >= 0) & (j <= s["alen"][:, None]))[:, None]
    jj = j.clamp(0, n - 1)[:, None].expand(-1, Hkv, -1)
    s["acc"].copy_(torch.where(fresh, path.gather(2, jj), acc))
    s["pos"].copy_(torch.where(fresh, (s["seen"][:, :, None] + jj).int(), s["pos"]))
    s["seen"] += s["alen"][:, None] + 1
    return {"acc": s["acc"], "pos": s["pos"], "seen": s["seen"]}


def _plain_evict(s):
    c = s["case"]
    keep, cap = c["keep"], s["cap"]
    _refill(s)
    at = torch.arange(cap, device=DEV)
    inside = (at < s["plen"][:, None])[:, None]
    safe = (s["pos"] < c["sink"]) | (s["pos"] >= s["seen"][:, :, None] - c["recent"])
    key = torch.where(inside, torch.where(safe, torch.full_like(s["acc"], math.inf), s["acc"]),
                      torch.full_like(s["acc"], -math.inf))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    kept = torch.zeros_like(inside.expand_as(key)).scatter(-1, order[..., :keep], True) & inside
    full = (s["plen"] > keep)[:, None, None]
    hole, mover = ~kept & (at < keep) & full, kept & (at >= keep) & full
    # the i-th mover goes to the i-th hole
    place = torch.where(mover, mover.cumsum(-1) - 1, torch.full_like(order, cap))
    by_rank = torch.zeros(*key.shape[:2], cap + 1, dtype=torch.int64, device=DEV).scatter_(-1, place, at.expand_as(place))
    src = torch.where(hole, by_rank.gather(-1, (hole.cumsum(-1) - 1).clamp(min=0)), at)

    def moved(x):
        return x.gather(2, src.view(*src.shape, *([1] * (x.dim() - 3))).expand_as(x))

    def cut(name, ename):
        x = _gathered(s, s[name].view(torch.uint8) if s["q8"] else s[name])
        if not s["q8"]:
            _put(s, s[name], moved(x))
            return
        e_old = _gathered(s, s[ename]).int()
        nb = e_old.shape[2]
        e_row = e_old.gather(2, src // BLOCK)
        live = torch.where(full & (at < keep), e_row, torch.zeros_like(e_row))
        e = torch.nn.functional.pad(live, (0, nb * BLOCK - cap)).view(*e_old.shape, BLOCK).amax(-1)
        e = torch.where(full & (torch.arange(nb, device=DEV) * BLOCK < keep), e, e_old)
        shift = torch.where(live > 0, e_row - e.gather(2, (at // BLOCK).expand_as(src)), torch.zeros_like(e_row))
        new = moved(x.view(torch.uint8)).view(torch.float8_e4m3fn).float() * _power(shift.clamp(min=-100))[..., None]
        _put(s, s[name].view(torch.uint8), new.to(torch.float8_e4m3fn).view(torch.uint8))
        _put(s, s[ename], e.to(torch.uint8))

    cut("k", "ke")
    if not s["latent"]:
        cut("v", "ve")
    s["acc"].copy_(moved(s["acc"]))
    s["pos"].copy_(moved(s["pos"]))
    s["plen"].clamp_(max=keep)
    return _evicted(s)


def _refill(s):
    """The weights, positions and lengths as they were before the first pass: the rows a pass moves are then the same."""
    s["acc"].copy_(s["acc0"])
    s["pos"].copy_(s["pos0"])
    s["plen"].copy_(s["plen0"])


def _evicted(s):
    out = {n: s[n] for n in ("k", "acc", "pos", "plen")}
    out.update({} if s["latent"] else {"v": s["v"]})
    out.update({n: s[n] for n in ("ke", "ve") if s.get(n) is not None})
    return out


# -------------------------------------------------- the framework's calls --

def _kept(s, T):
    """What a serving loop keeps between calls: descriptor, outputs, workspace, error word."""
    w = s["kept"]
    if not w:
        c = s["case"]
        w["desc"] = T.make_desc(c["B"], c.get("R", 1), c["Hq"], c["Hkv"], c["dk"], c["dv"], s["cap"], s["dt"],
                                s["latent"], s["scale"])
        w["err"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        if s["op"] == "attn":
            w["out"] = torch.empty(c["B"], c["R"], c["Hq"], c["dv"], dtype=s["dt"], device=DEV)
            w["lse"] = torch.empty(c["B"], c["R"], c["Hq"], device=DEV)
            w["ws"] = T.workspace(T.tsd_verify_q8_workspace_size(w["desc"]))
        elif s["op"] == "evict":
            w["ws"] = T.workspace(T.tsd_cache_evict_workspace_size(w["desc"]))
        w["paging"] = dict(page_table=s["table"], page_size=c["page"])
    return w


def _own(s):
    import tree_speculative_decoding_tsd_gb300 as T
    c, w = s["case"], _kept(s, T)
    if s["op"] == "attn":
        T.tsd_tree_verify_attn_q8(w["desc"], s["q"], s["k"], s["v"], s["ke"], s["ve"], s["plen"], s["kt"], s["vt"],
                                  s["mask"], w["out"], w["lse"], w["ws"], w["err"], **w["paging"])
        return {"out": w["out"], "lse": w["lse"]}
    if s["op"] == "write":
        s["plen"].copy_(s["plen0"])
        cache = (s["k"], s["v"], s["ke"], s["ve"], s["plen"], w["err"])
        if "x" in s:
            T.tsd_cache_write_q8(w["desc"], s["x"], s["y"], s["n"], *cache, **w["paging"])
        else:
            T.tsd_commit_path_q8(w["desc"], c["S"], s["kt"], s["vt"], s["arows"], s["alen"], *cache, **w["paging"])
        return _written(s)
    if s["op"] == "weights":
        if s["q8"]:
            T.tsd_cache_weights_q8(w["desc"], c["S"], s["q"], s["k"], s["ke"], s["plen"], s["kt"], s["arows"],
                                   s["alen"], s["lse"], s["decay"], s["acc"], s["pos"], s["seen"], w["err"],
                                   **w["paging"])
        else:
            T.tsd_cache_weights(w["desc"], c["S"], s["q"], s["k"], s["plen"], s["kt"], s["arows"], s["alen"],
                                s["lse"], s["decay"], s["acc"], s["pos"], s["seen"], w["err"], **w["paging"])
        return {"acc": s["acc"], "pos": s["pos"], "seen": s["seen"]}
    _refill(s)
    if s["q8"]:
        T.tsd_cache_evict_q8(w["desc"], c["keep"], c["sink"], c["recent"], s["acc"], s["pos"], s["seen"], s["k"],
                             s["v"], s["ke"], s["ve"], s["plen"], w["ws"], w["err"], **w["paging"])
    else:
        T.tsd_cache_evict(w["desc"], c["keep"], c["sink"], c["recent"], s["acc"], s["pos"], s["seen"], s["k"],
                          s["v"], s["plen"], w["ws"], w["err"], **w["paging"])
    return _evicted(s)


def run(state):
    if own:
        return _own(state)
    return {"attn": _plain_attn, "write": _plain_write, "weights": _plain_weights, "evict": _plain_evict}[
        state["op"]](state)


# ------------------------------------------------------------------- work --

def work(case):
    c = case
    B, Hkv, Hq, dk, dv = c["B"], c["Hkv"], c["Hq"], c["dk"], c["dv"]
    es = 4 if c["dtype"] == "f32" else 2
    keys = B * (c["P"] + c["P_min"]) / 2                 # cached tokens, on average
    row = dk if dk != dv else dk + dv                    # values of a cached token and head
    if c["op"] == "attn":
        rows = B * c["R"]
        tree = rows * Hkv * row * es
        return {"bytes": keys * Hkv * row * (1 + 1 / BLOCK / dk) + tree + rows * Hq * ((dk + dv) * es + 4),
                "flops": 2.0 * (dk + dv) * Hq * c["R"] * (keys + rows)}
    if c["op"] == "write":
        n = B * 0.75 * c["T"] if c["T"] else B * (1 + c["S"] / 2)
        return {"bytes": n * Hkv * row * (es + 1), "flops": 2.0 * n * Hkv * row}
    if c["op"] == "weights":
        rows = B * (1 + c["S"] / 2)
        return {"bytes": keys * Hkv * (dk * (1 if c["q8"] else es) + 8) + rows * (Hq * (dk * es + 4) + Hkv * dk * es),
                "flops": 2.0 * dk * Hq * (1 + c["S"] / 2) * keys}
    cut = max(0.0, keys - B * c["keep"])                 # rows that leave; as many of the kept ones lie behind the budget
    moved = cut * min(1.0, B * c["keep"] / max(1.0, keys)) * Hkv
    return {"bytes": keys * Hkv * 8 + moved * 2 * (row * (1 if c["q8"] else es) + 8), "flops": keys * Hkv}


# ------------------------------------------------------------------ exact --

def _exact_rows(s, name, ename, b, h):
    """Head h of request b in 64 bits, [cap][d], and its exponents."""
    pages = [b] if s["table"] is None else s["table"][b].tolist()
    x = torch.cat([s[name][p, h] for p in pages]) if not s["q8"] else \
        torch.cat([s[name].view(torch.uint8)[p, h] for p in pages]).view(torch.float8_e4m3fn)
    e = torch.cat([s[ename][p, h] for p in pages]).long() if s["q8"] else None
    return x.double(), e


def _exact_values(s, name, ename, b, h):
    x, e = _exact_rows(s, name, ename, b, h)
    if e is None:
        return x
    return x * torch.exp2((e - 127).double()).repeat_interleave(BLOCK)[: x.shape[0], None]


def _exact_attn(s):
    c = s["case"]
    B, R, Hq, Hkv, dv = c["B"], c["R"], c["Hq"], c["Hkv"], c["dv"]
    grp = Hq // Hkv
    out = torch.empty(B, R, Hq, dv, dtype=torch.float64, device=DEV)
    lse = torch.empty(B, R, Hq, dtype=torch.float64, device=DEV)
    masks = s["mask"].tolist()
    for b in range(B):
        P = int(s["plen"][b])
        sees = torch.tensor([[j == 0 or (i > 0 and (masks[b][i] >> (j - 1)) & 1 == 1) for j in range(R)]
                             for i in range(R)], device=DEV)
        hidden = torch.cat([torch.zeros(R, P, dtype=torch.bool, device=DEV), ~sees], 1)
        for h in range(Hkv):
            k = torch.cat([_exact_values(s, "k", "ke", b, h)[:P], s["kt"][b, :, h].double()])
            v = k[:, :dv] if s["latent"] else \
                torch.cat([_exact_values(s, "v", "ve", b, h)[:P], s["vt"][b, :, h].double()])
            q = s["q"][b, :, h * grp:(h + 1) * grp].double()
            a = torch.einsum("rgd,kd->rgk", q, k) * s["scale"]
            a = a.masked_fill(hidden[:, None], -math.inf)
            l = torch.logsumexp(a, -1)
            out[b, :, h * grp:(h + 1) * grp] = torch.einsum("rgk,kd->rgd", torch.exp(a - l[..., None]), v)
            lse[b, :, h * grp:(h + 1) * grp] = l
    return {"out": out, "lse": lse}


def _exact_put(s, x, b, h, rows):
    """Rows [cap][..] of head h of request b into the array x, laid out as the cache is."""
    pages = [b] if s["table"] is None else s["table"][b].tolist()
    n = rows.shape[0] // len(pages)
    for i, p in enumerate(pages):
        x[p, h] = rows[i * n:(i + 1) * n]


def _to_e4m3(x):
    """The nearest e4m3 value, ties to even, in 64 bits (|x| up to 448)."""
    ex = torch.frexp(x).exponent.clamp(min=-5) - 4
    step = torch.exp2(ex.double())
    return torch.round(x / step) * step


def _exact_write(s):
    B, Hkv = s["case"]["B"], s["case"]["Hkv"]
    out = {"plen": None, "ke": None, "ve": None}
    for name, ename, new in (("k", "ke", "x"), ("v", "ve", "y")):
        if s[name] is None:
            continue
        out[name] = s[name].double()
        src = s[new] if "x" in s else s[name + "t"]
        for b in range(B):
            P = int(s["plen"][b])
            rows = src[b, : int(s["n"][b])] if "x" in s else src[b, s["arows"][b, : int(s["alen"][b]) + 1].long()]
            end = P + rows.shape[0]
            for h in range(Hkv):
                codes, e = _exact_rows(s, name, ename, b, h)
                codes[P:end] = 0
                x = torch.zeros_like(codes)
                x[P:end] = rows[:, h].double()
                first, last = P // BLOCK, -(-end // BLOCK)
                pad = torch.zeros(last * BLOCK - first * BLOCK, codes.shape[1], dtype=torch.float64, device=DEV)
                top = min(last * BLOCK, codes.shape[0]) - first * BLOCK
                pad[:top] = x[first * BLOCK: first * BLOCK + top]
                need = torch.ceil(torch.log2(pad.abs().view(last - first, -1).amax(1) / 448)).long() + 127
                need = need.clamp(E_MIN, E_MAX)
                if P % BLOCK:
                    need[0] = max(int(need[0]), int(e[first]))
                old = e[first:last]
                grown = torch.exp2((old - need).double()).repeat_interleave(BLOCK)[:top, None]
                made = torch.exp2((127 - need).double()).repeat_interleave(BLOCK)[:top, None]
                at = slice(first * BLOCK, first * BLOCK + top)
                head = slice(first * BLOCK, P)
                was, scaled = codes[head].clone(), _to_e4m3(codes[at] * grown)
                codes[P:end] = _to_e4m3(x[at] * made)[P - first * BLOCK: end - first * BLOCK]
                if P % BLOCK and int(need[0]) != int(old[0]):
                    codes[head] = scaled[: P - first * BLOCK]
                else:
                    codes[head] = was
                keep, _ = _exact_rows(s, name, ename, b, h)
                keep[first * BLOCK:end] = codes[first * BLOCK:end]
                _exact_put(s, out[name], b, h, keep)
    return {n: v for n, v in out.items() if n in s and s[n] is not None}


def _exact_weights(s):
    c = s["case"]
    B, Hkv, grp = c["B"], c["Hkv"], c["Hq"] // c["Hkv"]
    acc = s["acc"].double()
    for b in range(B):
        P, L = int(s["plen"][b]), int(s["alen"][b])
        rows = s["arows"][b, : L + 1].long()
        for h in range(Hkv):
            heads = slice(h * grp, (h + 1) * grp)
            q, l = s["q"][b, rows, heads].double(), s["lse"][b, rows, heads].double()[..., None]
            k = _exact_values(s, "k", "ke", b, h)[:P]
            acc[b, h, :P] = s["decay"] * acc[b, h, :P] + \
                torch.exp(torch.einsum("igd,kd->igk", q, k) * s["scale"] - l).sum((0, 1))
            t = torch.exp(torch.einsum("igd,kd->igk", q, s["kt"][b, rows, h].double()) * s["scale"] - l).sum(1)
            acc[b, h, P: P + L + 1] = torch.tril(t).sum(0)
    return {"acc": acc, "pos": None, "seen": None}


def _exact_evict(s):
    c = s["case"]
    keep = c["keep"]
    out = {n: s[n].double() for n in ("k", "v", "acc") if s[n] is not None}
    for b in range(c["B"]):
        P = int(s["plen"][b])
        if P <= keep:
            continue
        for h in range(c["Hkv"]):
            pos, acc = s["pos"][b, h, :P].tolist(), s["acc"][b, h, :P].tolist()
            last = int(s["seen"][b, h]) - c["recent"]
            order = sorted(range(P), key=lambda i: (not (pos[i] < c["sink"] or pos[i] >= last), -acc[i], i))
            kept = set(order[:keep])
            holes = torch.tensor([i for i in range(keep) if i not in kept], dtype=torch.long, device=DEV)
            movers = torch.tensor([i for i in range(keep, P) if i in kept], dtype=torch.long, device=DEV)
            src = torch.arange(keep, device=DEV)
            src[holes] = movers
            out["acc"][b, h, :keep] = s["acc"][b, h].double()[src]
            for name, ename in (("k", "ke"), ("v", "ve")):
                if s[name] is None:
                    continue
                rows, e = _exact_rows(s, name, ename, b, h)
                new = rows[src]
                if e is not None:
                    e_row = e[src // BLOCK]
                    for j in range(0, keep, BLOCK):
                        part = e_row[j:j + BLOCK]
                        new[j:j + BLOCK] = _to_e4m3(new[j:j + BLOCK] * torch.exp2((part - part.max()).double())[:, None])
                rows[:keep] = new
                _exact_put(s, out[name], b, h, rows)
    return {**{n: None for n in _evicted(s)}, **out}


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "evict" and case["B"] * case["Hkv"] * case["P"] > 3e6:
        return None                   # the rows are ranked one by one here
    return {"attn": _exact_attn, "write": _exact_write, "weights": _exact_weights, "evict": _exact_evict}[s["op"]](s)
