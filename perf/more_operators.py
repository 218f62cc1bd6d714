"""Workloads of the 4-bit KV cache and of what makes its rows: rotation, writes, reads, attention.

Four operators:

  rope   RMS norm of every head's query and key, and the position rotation, of a draft
         tree's rows or a prompt's, from the projections [B][T][(Hq + 2 Hkv) d]
  write  rows appended to a 4-bit cache (a prompt, or a commit of the accepted path),
         and the end of the cache read back
  read   rows of a 4-bit cache as 16- or 32-bit rows
  attn   branch-aware attention of a draft tree over a 4-bit prefix cache

A row of the 4-bit cache has d codes c in 0..15 and a bf16 scale s for each 32 dims: a value
is (c - 8) s.  A 32-bit word holds the codes of dims 8w .. 8w + 7, the even ones in its
low half, the odd ones in its high half, from the lowest bits up.

``own`` selects the framework's calls; otherwise ``run`` computes the same with
elementary torch operations in 32 bits.
"""

import math
import random

import torch

own = False

GROUP = 32                    # dims that share a scale
TINY = 2.0 ** -90             # groups whose largest magnitude is below it are zeros
DEV = "cuda" if torch.cuda.is_available() else "cpu"   # the plain forms run on either


# ------------------------------------------------------------------ cases --

def listed():
    gqa = dict(Hq=32, Hkv=8, d=128, dtype="bf16", page=0)
    return [
        # one request, one token at a time: the smallest attention, all latency
        dict(name="attn token", op="attn", B=1, R=1, P=2048, P_min=2048, **gqa),
        # one request, a 16-node tree: an interactive user
        dict(name="attn tree", op="attn", B=1, R=17, P=2048, P_min=2048, **gqa),
        # a served batch of ragged requests with 32-node trees over a paged cache
        dict(name="attn batch", op="attn", B=32, R=33, P=4096, P_min=1024, **{**gqa, "page": 256}),
        # long documents, the largest tree
        dict(name="attn long tree", op="attn", B=8, R=65, P=32768, P_min=32768, **gqa),
        # long documents, plain decoding: every byte of the cache is read for four rows a head
        dict(name="attn long token", op="attn", B=16, R=1, P=32768, P_min=20001, **gqa),
        # the accepted paths of a served batch
        dict(name="write path", op="write", B=32, R=33, S=7, T=0, P=4096, P_min=1024, **gqa),
        # prompts of ragged length behind a cached system prompt
        dict(name="write prompt", op="write", B=4, R=1, S=0, T=8192, P=200, P_min=1, **gqa),
        # the last few hundred tokens of one request, for a window in 16 bits
        dict(name="read window", op="read", B=1, T=301, P=2048, P_min=2048, **gqa),
        # a paged batch handed to a 16-bit cache
        dict(name="read batch", op="read", B=32, T=4096, P=4096, P_min=1024, **{**gqa, "page": 256}),
        # rows of one 16-node tree: the smallest rotation
        dict(name="rope tree", op="rope", B=1, T=17, tree=True, axes=1, rot=128, pairs="halves", far=2048, **gqa),
        # 32-node trees of a served batch
        dict(name="rope batch", op="rope", B=32, T=33, tree=True, axes=1, rot=128, pairs="halves", far=4096, **gqa),
        # prompts of ragged length with images in them: time, height and width
        dict(name="rope prompt", op="rope", B=4, T=8192, tree=False, axes=3, rot=128, pairs="halves", far=200, **gqa),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "write", "read", "rope"])
    kind = rng.choice(["gqa", "gqa", "wide", "narrow", "single"])
    dtype = "f32" if rng.random() < 0.12 else "bf16"
    c = {"gqa": dict(Hq=32, Hkv=8, d=128), "wide": dict(Hq=64, Hkv=8, d=128), "narrow": dict(Hq=14, Hkv=2, d=64),
         "single": dict(Hq=8, Hkv=8, d=128)}[kind]
    c = dict(op=op, dtype=dtype, page=rng.choice([0, 0, 128, 256]), B=_log(rng, 1, 32), P=_log(rng, 1, 32768), **c)
    # a drawn case reads no more cache, and computes no more, than the largest listed ones
    while c["B"] * c["P"] > (8192 if dtype == "f32" and op == "attn" else 262144):
        c["B"], c["P"] = max(1, c["B"] // 2), c["P"] if c["B"] > 1 else c["P"] // 2
    if op == "attn":
        c["R"] = rng.choice([1, 1, 2, rng.randint(3, 65)])
        while c["R"] > 1 and c["B"] * c["R"] * c["P"] * c["Hq"] * 2 * c["d"] > (3e9 if dtype == "f32" else 2e11):
            c["R"] = c["R"] // 2
    elif op == "write":
        c["R"], c["S"] = rng.randint(17, 65), rng.randint(1, 16)
        c["T"] = 0 if rng.random() < 0.5 else _log(rng, 1, 8192)
        if c["T"]:
            c.update(P=rng.randint(1, 300), B=max(1, min(c["B"], 32768 // c["T"])))
    elif op == "read":
        c["P"] = max(1, min(c["P"], 131072 // c["B"]))
        c["T"] = _log(rng, 1, c["P"])
    else:
        c["tree"] = rng.random() < 0.5
        c["T"] = rng.randint(1, 65) if c["tree"] else _log(rng, 1, 8192)
        c["B"] = max(1, min(c["B"], 32768 // c["T"]))
        c.update(axes=rng.choice([1, 1, 2, 3]), rot=c["d"] if rng.random() < 0.7 else c["d"] // 2, page=0,
                 pairs=rng.choice(["halves", "neighbours"]), far=_log(rng, 1, 1000000))
    c["P_min"] = max(1, int(c["P"] * rng.uniform(0.3, 1.0)))
    return c


# ----------------------------------------------------------------- inputs --

def _cap(c):
    n = c["P"] + 1 + max(c.get("S", 0), c["T"] if c["op"] == "write" else 0)
    return n if not c["page"] else -(-n // c["page"]) * c["page"]


def _tree(rnd, B, R):
    """Random trees: ancestor-or-self masks (bit j - 1 for row j >= 1), and depths."""
    masks, depths = [], []
    for _ in range(B):
        m, d = [0], [0]
        for r in range(1, R):
            p = rnd.randrange(max(0, r - 6), r)
            m.append(m[p] | (1 << (r - 1)))
            d.append(d[p] + 1)
        masks.append([v - (1 << 64) if v >> 63 else v for v in m])
        depths.append(d)
    return (torch.tensor(masks, dtype=torch.int64, device=DEV), torch.tensor(depths, dtype=torch.int32, device=DEV))


def _frequencies(c):
    """Radians per position [axes][rot / 2]; with several axes each pair turns with one of them."""
    n = c["rot"] // 2
    f = 1000000.0 ** (-torch.arange(n, dtype=torch.float64) / n)
    if c["axes"] == 1:
        return f[None]
    cut = [n * a // c["axes"] for a in range(c["axes"] + 1)]
    out = torch.zeros(c["axes"], n, dtype=torch.float64)
    for a in range(c["axes"]):
        out[a, cut[a]:cut[a + 1]] = f[cut[a]:cut[a + 1]]
    return out


def _image_positions(rnd, axes, B, T):
    """Offsets [axes][B][T] of prompts that mix text (all axes step together) with images (a grid)."""
    out = torch.empty(axes, B, T, dtype=torch.int32)
    for b in range(B):
        t, at = 0, 0
        while t < T:
            n = min(T - t, rnd.randint(1, 200))
            out[:, b, t:t + n] = torch.arange(at, at + n, dtype=torch.int32)
            t, at = t + n, at + n
            h, w = rnd.randint(2, 24), rnd.randint(2, 24)
            n = min(T - t, h * w)
            i = torch.arange(n, dtype=torch.int32)
            for a in range(axes):
                out[a, b, t:t + n] = at + (0 * i if a == 0 else i // w if a == 1 else i % w)
            t, at = t + n, at + max(h, w)
    return out.to(DEV)


def prepare(case, seed):
    c = case
    rnd = random.Random(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    B, Hq, Hkv, d, op = c["B"], c["Hq"], c["Hkv"], c["d"], c["op"]
    dt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    s = dict(case=dict(c), op=op, dt=dt, scale=1.0 / math.sqrt(d), kept={})

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=DEV)

    if op == "rope":
        T = c["T"]
        # the projections of a row beside one another
        s["qkv"] = normal(B, T, (Hq + 2 * Hkv) * d)
        s["wq"], s["wk"] = (1 + normal(d, std=0.1, dtype=torch.float32)).to(dt), (1 + normal(d, std=0.1)).to(dt)
        s["freq"] = _frequencies(c).to(DEV)
        s["start"] = ints([rnd.randint(max(1, c["far"] // 2), c["far"]) for _ in range(B)])
        if c["tree"]:
            s["at"] = _tree(rnd, B, T)[1][None].expand(c["axes"], B, T).contiguous()
            s["n"] = None
        else:
            s["at"] = _image_positions(rnd, c["axes"], B, T) if c["axes"] > 1 else None
            n = [rnd.randint(max(1, T // 2), T) for _ in range(B)]
            n[rnd.randrange(B)] = T
            s["n"] = ints(n)
        return s

    s["cap"] = cap = _cap(c)
    lens = [rnd.randint(c["P_min"], c["P"]) for _ in range(B)]
    lens[rnd.randrange(B)] = c["P"]
    s["plen"] = ints(lens)

    # the cache: [B][Hkv][cap][..], or pages [pages][Hkv][page][..] in a shuffled order with a few unused ones
    if c["page"]:
        per = cap // c["page"]
        pages = B * per + 3
        s["table"] = ints(rnd.sample(range(pages), B * per)).view(B, per)
        lead, rows = (pages, Hkv), c["page"]
    else:
        s["table"] = None
        lead, rows = (B, Hkv), cap

    def codes():
        # two values a byte, each a code of a row of normal numbers
        x = torch.randn(2, *lead, rows, d // 2, generator=g, device=DEV).mul_(2.8).round_().clamp_(-8, 7).add_(8)
        return (x[0] + 16 * x[1]).to(torch.uint8)

    def scales():
        x = torch.rand(*lead, rows, d // GROUP, generator=g, device=DEV)
        return ((x * 0.2 + 0.25) * torch.where(x * 64 % 1 < 0.5, 1.0, -1.0)).to(torch.bfloat16)

    s["k"], s["ks"], s["v"], s["vs"] = codes(), scales(), codes(), scales()
    if op == "attn":
        s["q"] = normal(B, c["R"], Hq, d)
        s["kt"], s["vt"] = normal(B, c["R"], Hkv, d), normal(B, c["R"], Hkv, d)
        s["mask"] = _tree(rnd, B, c["R"])[0]
    if op == "write":
        S = c["S"]
        if c["T"]:
            s["x"], s["y"] = normal(B, c["T"], Hkv, d), normal(B, c["T"], Hkv, d)
            new = [rnd.randint(max(1, c["T"] // 2), c["T"]) for _ in range(B)]
            s["n"] = ints(new)
        else:
            ls, paths = [], []
            for _ in range(B):
                L = rnd.randint(0, min(S, c["R"] - 1))
                ls.append(L)
                paths.append([0] + sorted(rnd.sample(range(1, c["R"]), L)) + [-1] * (S - L))
            s["alen"], s["arows"] = ints(ls), ints(paths)
            s["kt"], s["vt"] = normal(B, c["R"], Hkv, d), normal(B, c["R"], Hkv, d)
            new = [L + 1 for L in ls]
        s["plen0"] = s["plen"].clone()
        # read back: the new rows and up to 32 before them
        s["first"] = ints([max(0, p - 32) for p in lens])
        s["count"] = ints([min(p, 32) + n for p, n in zip(lens, new)])
        s["room"] = 32 + (c["T"] or S + 1)
    if op == "read":
        n = [rnd.randint(max(1, min(c["T"], p) // 2), min(c["T"], p)) for p in lens]
        s["first"], s["count"] = ints([p - x for p, x in zip(lens, n)]), ints(n)
        s["room"] = c["T"]
    return s


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


# ------------------------------------------------------------ plain forms --

def _codes(x):
    """Packed codes [..][d / 2] as [..][d]."""
    nib = torch.stack([x & 15, x >> 4], -1).view(*x.shape[:-1], -1, 2, 4)
    return nib.transpose(-1, -2).reshape(*x.shape[:-1], -1)


def _packed(c):
    """The reverse: codes [..][d] (uint8) as [..][d / 2]."""
    nib = c.view(*c.shape[:-1], -1, 4, 2).transpose(-1, -2).reshape(*c.shape[:-1], -1, 2)
    return nib[..., 0] | (nib[..., 1] << 4)


def _values(s, name, sname):
    """The cache's values in 32 bits, [B][Hkv][cap][d]."""
    x = _codes(_gathered(s, s[name])).float() - 8
    x.view(*x.shape[:-1], -1, GROUP).mul_(_gathered(s, s[sname]).float()[..., None])
    return x


def _quantised(x):
    """Rows [..][d] as (codes [..][d] uint8, scales [..][d / 32] bf16)."""
    x = x.float().view(*x.shape[:-1], -1, GROUP)
    hi, lo = x.amax(-1), x.amin(-1)
    top = torch.where(hi >= -lo, hi, lo)
    scale = (top * -0.125).bfloat16()
    scale = torch.where(top.abs() < TINY, torch.zeros_like(scale), scale)
    inv = 1.0 / scale.float()
    c = (x.double() * inv.double()[..., None]).round().clamp(-8, 7) + 8
    c = torch.where((scale == 0)[..., None], torch.full_like(c, 8), c)
    return c.to(torch.uint8).flatten(-2), scale


def _plain_attn(s):
    c = s["case"]
    B, R, Hq, Hkv, d = c["B"], c["R"], c["Hq"], c["Hkv"], c["d"]
    k = torch.cat([_values(s, "k", "ks"), s["kt"].float().transpose(1, 2)], 2)
    q = s["q"].float().view(B, R, Hkv, Hq // Hkv, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, d)
    sc = torch.matmul(q, k.transpose(-1, -2)).view(B, Hkv, R, Hq // Hkv, -1)
    del k
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
    v = torch.cat([_values(s, "v", "vs"), s["vt"].float().transpose(1, 2)], 2)
    out = torch.matmul(p.view(B, Hkv, -1, p.shape[-1]), v).view(B, Hkv, R, Hq // Hkv, d) / total
    out = out.permute(0, 2, 1, 3, 4).reshape(B, R, Hq, d).to(s["dt"])
    lse = (total.log() + m).permute(0, 2, 1, 3, 4).reshape(B, R, Hq)
    return {"out": out, "lse": lse}


def _plain_read(s):
    out = {"plen": s["plen"]}
    i = torch.arange(s["room"], device=DEV)
    at = (s["first"].long()[:, None] + i).clamp(max=s["cap"] - 1)
    live = (i < s["count"][:, None])[:, :, None, None]
    for name, sname in (("k", "ks"), ("v", "vs")):
        x = _values(s, name, sname).transpose(1, 2)
        x = x.gather(1, at[:, :, None, None].expand(-1, -1, *x.shape[2:]))
        out[name] = torch.where(live, x, torch.zeros_like(x)).to(s["dt"])
    return out


def _plain_write(s):
    s["plen"].copy_(s["plen0"])
    cap = s["cap"]
    if "x" in s:
        new, n = (s["x"], s["y"]), s["n"]
    else:
        i = s["arows"].long().clamp(min=0)[:, :, None, None].expand(-1, -1, *s["kt"].shape[2:])
        new, n = (s["kt"].gather(1, i), s["vt"].gather(1, i)), s["alen"] + 1
    t = torch.arange(cap, device=DEV) - s["plen"].long()[:, None]
    fresh = ((t >= 0) & (t < n[:, None]))[:, None, :, None]
    for name, sname, rows in (("k", "ks", new[0]), ("v", "vs", new[1])):
        code, scale = _quantised(rows)
        code = _packed(code)
        for array, made in ((s[name], code), (s[sname], scale)):
            made = made.gather(1, t.clamp(0, made.shape[1] - 1)[:, :, None, None].expand(-1, -1, *made.shape[2:]))
            _put(s, array, torch.where(fresh, made.transpose(1, 2), _gathered(s, array)))
    s["plen"] += n
    return _plain_read(s)


def _plain_rope(s):
    c = s["case"]
    B, T, Hq, Hkv, d, n = c["B"], c["T"], c["Hq"], c["Hkv"], c["d"], c["rot"] // 2
    at = s["at"] if s["at"] is not None else torch.arange(T, device=DEV).expand(c["axes"], B, T)
    at = (at + s["start"][:, None]).double()
    angle = torch.einsum("abt,ai->bti", at, s["freq"])              # (positions reach far: 64 bits)
    cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]
    live = torch.ones(B, T, 1, 1, dtype=torch.bool, device=DEV) if s["n"] is None else \
        (torch.arange(T, device=DEV) < s["n"][:, None])[:, :, None, None]
    q, k, v = s["qkv"].view(B, T, -1, d).split([Hq, Hkv, Hkv], 2)

    def turned(x, w):
        x = x.float()
        x = x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w.float()
        r = x[..., : 2 * n]
        a, b = (r[..., :n], r[..., n:]) if c["pairs"] == "halves" else (r[..., 0::2], r[..., 1::2])
        a, b = a * cos - b * sin, a * sin + b * cos
        r = torch.cat([a, b], -1) if c["pairs"] == "halves" else torch.stack([a, b], -1).flatten(-2)
        x = torch.cat([r, x[..., 2 * n:]], -1)
        return torch.where(live, x, torch.zeros_like(x)).to(s["dt"])

    return {"q": turned(q, s["wq"]), "k": turned(k, s["wk"]), "v": torch.where(live, v, torch.zeros_like(v))}


# -------------------------------------------------- the framework's calls --

def _kept(s, T):
    """What a serving loop keeps between calls: descriptor, outputs, workspace, error word."""
    w = s["kept"]
    if w:
        return w
    c = s["case"]
    B, Hq, Hkv, d = c["B"], c["Hq"], c["Hkv"], c["d"]

    def zeros(*shape):
        return torch.zeros(shape, dtype=s["dt"], device=DEV)

    if s["op"] == "rope":
        w["desc"] = T.make_rope_desc(B, c["T"], Hq, Hkv, d, s["dt"], rot=c["rot"], axes=c["axes"],
                                     neighbours=c["pairs"] == "neighbours", norm=True, eps=1e-6)
        w["turns"] = T.rope_turns(s["freq"])
        w["out"] = zeros(B, c["T"], Hq, d), zeros(B, c["T"], Hkv, d), zeros(B, c["T"], Hkv, d)
        return w
    w["desc"] = T.make_desc(B, c.get("R", 1), Hq, Hkv, d, d, s["cap"], s["dt"], False, s["scale"])
    w["err"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    w["paging"] = dict(page_table=s["table"], page_size=c["page"])
    if s["op"] == "attn":
        w["out"] = zeros(B, c["R"], Hq, d)
        w["lse"] = torch.empty(B, c["R"], Hq, device=DEV)
        w["ws"] = T.workspace(T.tsd_verify_q4_workspace_size(w["desc"]))
    else:
        w["back"] = zeros(B, s["room"], Hkv, d), zeros(B, s["room"], Hkv, d)
    return w


def _own(s):
    import tree_speculative_decoding_tsd_gb300 as T
    c, w = s["case"], _kept(s, T)
    if s["op"] == "rope":
        q, k, v = s["qkv"].view(c["B"], c["T"], -1, c["d"]).split([c["Hq"], c["Hkv"], c["Hkv"]], 2)
        T.tsd_qk_norm_rope(w["desc"], q, k, v, w["turns"], *w["out"], q_weight=s["wq"], k_weight=s["wk"],
                           start=s["start"], offset=s["at"], count=s["n"])
        return dict(zip("qkv", w["out"]))
    cache = (s["k"], s["v"], s["ks"], s["vs"], s["plen"])
    if s["op"] == "attn":
        T.tsd_tree_verify_attn_q4(w["desc"], s["q"], *cache, s["kt"], s["vt"], s["mask"], w["out"], w["lse"], w["ws"],
                                  w["err"], **w["paging"])
        return {"out": w["out"], "lse": w["lse"]}
    if s["op"] == "write":
        s["plen"].copy_(s["plen0"])
        if "x" in s:
            T.tsd_cache_write_q4(w["desc"], s["x"], s["y"], s["n"], *cache, w["err"], **w["paging"])
        else:
            T.tsd_commit_path_q4(w["desc"], c["S"], s["kt"], s["vt"], s["arows"], s["alen"], *cache, w["err"],
                                 **w["paging"])
    T.tsd_cache_read_q4(w["desc"], *cache, s["first"], s["count"], *w["back"], w["err"], **w["paging"])
    return {"plen": s["plen"], "k": w["back"][0], "v": w["back"][1]}


def run(state):
    if own:
        return _own(state)
    return {"attn": _plain_attn, "write": _plain_write, "read": _plain_read, "rope": _plain_rope}[state["op"]](state)


# ------------------------------------------------------------------- work --

def work(case):
    c = case
    B, Hkv, Hq, d = c["B"], c["Hkv"], c["Hq"], c["d"]
    es = 4 if c["dtype"] == "f32" else 2
    held = 0.5 + 2 / GROUP                               # bytes of a cached value
    if c["op"] == "rope":
        rows = B * c["T"] * (1.0 if c["tree"] else 0.75)
        return {"bytes": rows * ((Hq + 2 * Hkv) * d * 2 * es + 4 * c["axes"]), "flops": rows * (Hq + Hkv) * d * 8.0}
    if c["op"] == "write":
        n = B * 0.75 * c["T"] if c["T"] else B * (1 + c["S"] / 2)
        back = n + B * min(32, c["P"])                   # rows read back
        return {"bytes": 2 * Hkv * d * (n * (es + held) + back * es + (back - n) * held), "flops": 4.0 * back * Hkv * d}
    if c["op"] == "read":
        n = 0.75 * B * min(c["T"], (c["P"] + c["P_min"]) / 2)
        return {"bytes": n * 2 * Hkv * d * (es + held), "flops": n * 2 * Hkv * d}
    keys = B * (c["P"] + c["P_min"]) / 2                 # cached tokens, on average
    rows = B * c["R"]
    return {"bytes": keys * Hkv * 2 * d * held + rows * (2 * Hkv * d * es + Hq * (2 * d * es + 4)),
            "flops": 4.0 * d * Hq * c["R"] * (keys + rows / B)}


# ------------------------------------------------------------------ exact --

DIMS = [0, 2, 4, 6, 1, 3, 5, 7]                          # a word's dims, from the lowest bits up


def _exact_values(s, name, sname, b, h):
    """Head h of request b in 64 bits, [cap][d]."""
    pages = [b] if s["table"] is None else s["table"][b].tolist()
    x = torch.cat([s[name][p, h] for p in pages]).long()
    f = torch.cat([s[sname][p, h] for p in pages]).double()
    word = (x.view(x.shape[0], -1, 4) << torch.arange(0, 32, 8, device=DEV)).sum(-1)
    out = torch.empty(*word.shape, 8, dtype=torch.float64, device=DEV)
    for i, dim in enumerate(DIMS):
        out[..., dim] = ((word >> (4 * i)) % 16 - 8).double()
    return out.flatten(1) * f.repeat_interleave(GROUP, 1)


def _exact_attn(s):
    c = s["case"]
    B, R, Hq, Hkv, d = c["B"], c["R"], c["Hq"], c["Hkv"], c["d"]
    grp = Hq // Hkv
    out = torch.empty(B, R, Hq, d, dtype=torch.float64, device=DEV)
    lse = torch.empty(B, R, Hq, dtype=torch.float64, device=DEV)
    masks = s["mask"].tolist()
    for b in range(B):
        P = int(s["plen"][b])
        sees = torch.tensor([[j == 0 or (i > 0 and (masks[b][i] >> (j - 1)) & 1 == 1) for j in range(R)]
                             for i in range(R)], device=DEV)
        hidden = torch.cat([torch.zeros(R, P, dtype=torch.bool, device=DEV), ~sees], 1)
        for h in range(Hkv):
            k = torch.cat([_exact_values(s, "k", "ks", b, h)[:P], s["kt"][b, :, h].double()])
            v = torch.cat([_exact_values(s, "v", "vs", b, h)[:P], s["vt"][b, :, h].double()])
            q = s["q"][b, :, h * grp:(h + 1) * grp].double()
            a = torch.einsum("rgd,kd->rgk", q, k) * s["scale"]
            a = a.masked_fill(hidden[:, None], -math.inf)
            l = torch.logsumexp(a, -1)
            out[b, :, h * grp:(h + 1) * grp] = torch.einsum("rgk,kd->rgd", torch.exp(a - l[..., None]), v)
            lse[b, :, h * grp:(h + 1) * grp] = l
    return {"out": out, "lse": lse}


def _exact_rows(x):
    """What the cache holds of rows [n][d] (64 bits)."""
    x = x.view(x.shape[0], -1, GROUP)
    big = x.abs().amax(-1)
    top = torch.where(x.amax(-1) == big, big, -big)
    scale = (top / -8).float().bfloat16().double()                    # (both steps are exact but for the last)
    scale[big < TINY] = 0
    inv = torch.where(scale == 0, torch.zeros_like(scale), 1 / scale).float().double()
    return (torch.round(x * inv[..., None]).clamp(-8, 7) * scale[..., None]).flatten(1)


def _exact_cache(s):
    """Values read back, from the cache or from the new rows."""
    c = s["case"]
    out = {"plen": None}
    for name, sname, new in (("k", "ks", "x"), ("v", "vs", "y")):
        out[name] = torch.zeros(c["B"], s["room"], c["Hkv"], c["d"], dtype=torch.float64, device=DEV)
        for b in range(c["B"]):
            first, n = int(s["first"][b]), int(s["count"][b])
            old = n
            if s["op"] == "write":
                P = int(s["plen"][b])
                old = P - first
                rows = s[new][b, : int(s["n"][b])] if "x" in s else \
                    s[name + "t"][b, s["arows"][b, : int(s["alen"][b]) + 1].long()]
            for h in range(c["Hkv"]):
                out[name][b, :old, h] = _exact_values(s, name, sname, b, h)[first:first + old]
                if old < n:
                    out[name][b, old:n, h] = _exact_rows(rows[:, h].double())
    return out


def _exact_rope(s):
    c = s["case"]
    B, T, Hq, Hkv, d, n = c["B"], c["T"], c["Hq"], c["Hkv"], c["d"], c["rot"] // 2
    x = s["qkv"].double().view(B, T, -1, d)
    out = torch.zeros(B, T, Hq + 2 * Hkv, d, dtype=torch.float64, device=DEV)
    first = torch.arange(n, device=DEV) * (1 if c["pairs"] == "halves" else 2)
    second = first + (n if c["pairs"] == "halves" else 1)
    for b in range(B):
        live = T if s["n"] is None else int(s["n"][b])
        angle = torch.zeros(live, n, dtype=torch.float64, device=DEV)
        for a in range(c["axes"]):
            at = torch.arange(T, device=DEV) if s["at"] is None else s["at"][a, b]
            angle += (at[:live].double() + float(s["start"][b]))[:, None] * s["freq"][a]
        turn = torch.polar(torch.ones_like(angle), angle)[:, None]
        for h0, h1, w in ((0, Hq, s["wq"]), (Hq, Hq + Hkv, s["wk"])):
            y = x[b, :live, h0:h1]
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / d + 1e-6) * w.double()
            z = torch.complex(y[..., first], y[..., second]) * turn
            y[..., first], y[..., second] = z.real, z.imag
            out[b, :live, h0:h1] = y
        out[b, :live, Hq + Hkv:] = x[b, :live, Hq + Hkv:]
    q, k, v = out.split([Hq, Hkv, Hkv], 2)
    return {"q": q, "k": k, "v": v}


def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attn, "write": _exact_cache, "read": _exact_cache, "rope": _exact_rope}[s["op"]](s)
