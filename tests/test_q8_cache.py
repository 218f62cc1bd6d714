"""The 8-bit KV cache, its attention weights and its eviction against plain 64-bit code.

The plain forms here work per request and head in float64 (or on whole
numbers).  Codes, exponents, ranks and moved rows have to be equal; what the
kernels compute is held to bounds derived beside each check.
"""

import ctypes
import math
import random
import threading
import time

import pytest
import torch

import tree_speculative_decoding_tsd_gb300 as T

DEV = "cuda:0"
NAN, INF = float("nan"), float("inf")
BLOCK = T.TSD_Q8_BLOCK


# ------------------------------------------------------------ plain forms --

def nearest_code(x):
    """x (float64) to the nearest e4m3 value, ties to even, saturating, NaN kept."""
    step = torch.exp2((torch.frexp(x).exponent.clamp(min=-5) - 4).double())
    y = (torch.round(x / step) * step).clamp(-448, 448)
    y = torch.where(x.abs() == INF, torch.sign(x) * 448, y)
    return torch.where(x.isnan(), x, y)


def need_of(rows):
    """The smallest exponent byte that holds the finite values of rows."""
    a = rows[rows.isfinite()].abs()
    a = float(a.max()) if a.numel() else 0.0
    e = 10
    while a > 448 * 2.0 ** (e - 127) and e < 246:
        e += 1
    return e


def codes_of(t):
    return t.view(torch.float8_e4m3fn).double()


class Cache:
    """A contiguous or paged cache of one array (K or V): values by (request, head)."""

    def __init__(self, x, e, table):
        self.x, self.e, self.table = x, e, table

    def pages(self, b):
        return [b] if self.table is None else self.table[b].tolist()

    def rows(self, b, h):
        x = self.x.view(torch.uint8) if self.e is not None else self.x
        x = torch.cat([x[p, h] for p in self.pages(b)])
        return codes_of(x) if self.e is not None else x.double()

    def exps(self, b, h):
        return torch.cat([self.e[p, h] for p in self.pages(b)]).long()

    def values(self, b, h):
        x = self.rows(b, h)
        if self.e is None:
            return x
        f = torch.exp2((self.exps(b, h) - 127).double()).repeat_interleave(BLOCK)
        return x * f[: x.shape[0], None]


def plain_write(cache, b, h, P, new):
    """(codes, exponents) of the head after rows `new` (float64) went to P.. ."""
    codes, e = cache.rows(b, h), cache.exps(b, h)
    for j in range(P // BLOCK, -(-(P + len(new)) // BLOCK)):
        lo, hi = max(P, j * BLOCK), min(P + len(new), (j + 1) * BLOCK)
        x = new[lo - P: hi - P]
        e1 = need_of(x)
        if j * BLOCK < P:
            e1 = max(e1, int(e[j]))
            if e1 != int(e[j]):
                old = slice(j * BLOCK, P)
                codes[old] = nearest_code(codes[old] * 2.0 ** (int(e[j]) - e1))
        codes[lo:hi] = nearest_code(x * 2.0 ** (127 - e1))
        e[j] = e1
    return codes, e


def plain_attn(q, k, v, sees, scale):
    """q [n][d], k [m][d], v [m][dv], sees [n][m] -> out, lse, and what the bounds need:
    the weighted mean of |v| and the largest scale * sum |q_d k_d|."""
    s = (q @ k.T * scale).masked_fill(~sees, -INF)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[:, None])
    big = (q.abs() @ k.abs().T * scale).masked_fill(~sees, 0).amax(-1)
    return p @ v, lse, p @ v.abs(), big


def plain_evict(P, keep, sink, recent, acc, pos, seen):
    """(holes, movers) of one head."""
    key = [(not (pos[i] < sink or pos[i] >= seen - recent), -acc[i], i) for i in range(P)]
    kept = set(sorted(range(P), key=lambda i: key[i])[:keep])
    return ([i for i in range(keep) if i not in kept], [i for i in range(keep, P) if i in kept])


# ----------------------------------------------------------------- inputs --

KINDS = {"gqa": (32, 8, 128, 128), "narrow": (14, 2, 64, 64), "one": (2, 2, 128, 128),
         "wide": (16, 1, 128, 128), "latent": (128, 1, 576, 512), "latent-few": (16, 1, 576, 512)}


class Setup:
    """Random cache, scratch pad, tree and lengths for one configuration."""

    def __init__(self, kind, B, R, lens, extra=8, dtype=torch.bfloat16, page=0, q8=True, seed=0,
                 spread=3):
        self.Hq, self.Hkv, self.dk, self.dv = KINDS[kind]
        self.B, self.R, self.dt, self.q8, self.page = B, R, dtype, q8, page
        self.latent = self.dk != self.dv
        self.g = torch.Generator(device=DEV).manual_seed(seed * 1000 + 7)
        self.rnd = random.Random(seed)
        self.lens = [lens[b % len(lens)] for b in range(B)]
        cap = max(self.lens) + extra
        if page:
            cap = -(-cap // page) * page
        self.cap = cap
        self.scale = float(torch.tensor(1 / math.sqrt(self.dk), dtype=torch.float32))
        self.table = None
        lead, rows = (B, self.Hkv), cap
        if page:
            per = cap // page
            order = self.rnd.sample(range(B * per + 2), B * per)
            self.table = torch.tensor(order, dtype=torch.int32, device=DEV).view(B, per)
            lead, rows = (B * per + 2, self.Hkv), page
        self.lead, self.rows = lead, rows

        def arr(d):
            x = torch.randn(*lead, rows, d, generator=self.g, device=DEV)
            return (x * 110).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if q8 \
                else x.to(dtype)

        def exps():
            return torch.randint(121 - spread, 122, (*lead, -(-rows // BLOCK)), generator=self.g,
                                 device=DEV, dtype=torch.uint8) if q8 else None

        self.k, self.ke = arr(self.dk), exps()
        self.v, self.ve = (None, None) if self.latent else (arr(self.dv), exps())
        self.plen = torch.tensor(self.lens, dtype=torch.int32, device=DEV)
        self.q = self.normal(B, R, self.Hq, self.dk)
        self.kt = self.normal(B, R, self.Hkv, self.dk)
        self.vt = None if self.latent else self.normal(B, R, self.Hkv, self.dv)
        masks = []
        for _ in range(B):
            m = [0]
            for r in range(1, R):
                m.append(m[self.rnd.randrange(max(0, r - 5), r)] | (1 << (r - 1)))
            masks.append(m)
        self.set_masks(masks)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.desc = T.make_desc(B, R, self.Hq, self.Hkv, self.dk, self.dv, cap, dtype, self.latent,
                                self.scale)
        self.paging = dict(page_table=self.table, page_size=page)

    def normal(self, *shape, std=1.0):
        return (torch.randn(*shape, generator=self.g, device=DEV) * std).to(self.dt)

    def set_masks(self, masks):
        self.masks = masks
        self.mask = torch.tensor([[v - (1 << 64) if v >> 63 else v for v in m] for m in masks],
                                 dtype=torch.int64, device=DEV)

    def cache(self, which):
        return Cache(self.k, self.ke, self.table) if which == "k" else Cache(self.v, self.ve,
                                                                            self.table)

    def attn(self, stream=None):
        out = torch.full((self.B, self.R, self.Hq, self.dv), 7.0, dtype=self.dt, device=DEV)
        lse = torch.full((self.B, self.R, self.Hq), 7.0, device=DEV)
        ws = T.workspace(T.tsd_verify_q8_workspace_size(self.desc))
        self.attn_into(out, lse, ws, stream)
        torch.cuda.synchronize()
        return out, lse

    def attn_into(self, out, lse, ws, stream=None):
        T.tsd_tree_verify_attn_q8(self.desc, self.q, self.k, self.v, self.ke, self.ve, self.plen,
                                  self.kt, self.vt, self.mask, out, lse, ws, self.err, stream,
                                  **self.paging)

    def sees(self, b):
        R = self.R
        return torch.tensor([[j == 0 or (i > 0 and self.masks[b][i] >> (j - 1) & 1 == 1)
                              for j in range(R)] for i in range(R)], device=DEV)

    def check_attn(self, out, lse, requests=None, heads=None):
        """Bounds.  A score is a product of dk terms summed in fp32, in any order and
        possibly truncated: off by at most (dk + 8) 2^-23 S with S = scale sum |q k|.
        A probability is then off by that, relatively, plus 2^-20 for the exponential
        and the sums' last bits (fp32 sums of n terms: n 2^-24 more), and 2^-12 where
        it is rounded to fp16; a split's output is rounded to fp16 (2^-12) once
        more.  Means of v move by those shares of A = the weighted mean of |v|.  bf16 outputs are
        rounded once: 2^-8 of the value (fp32: 2^-24).
        fp16 has a smallest step, 2^-24, and a probability p is held as p 2^(u - U + 7), u the
        exponent of its value row and U the largest one: half a step is 2^-25, worth 2^-25
        2^(U - 7) |code| <= 2^-32 2^U 512 of the sum over p v, whose divisor is at least 1 (the
        running maximum is at most the largest score).  So n keys add at most n 2^-32 top, with
        top = 512 * 2^U, or twice the largest scratch value; a split's output over 2^U, rounded
        to at least 2^-25, stays below one key's share."""
        g = self.Hq // self.Hkv
        for b in requests if requests is not None else range(self.B):
            P = min(self.lens[b], self.cap)
            sees = torch.cat([torch.ones(self.R, P, dtype=torch.bool, device=DEV), self.sees(b)], 1)
            live = sees.any(0)
            for h in heads if heads is not None else range(self.Hkv):
                k = torch.cat([self.cache("k").values(b, h)[:P], self.kt[b, :, h].double()])
                v = k[:, : self.dv] if self.latent else torch.cat(
                    [self.cache("v").values(b, h)[:P], self.vt[b, :, h].double()])
                k, v = k[live], v[live]
                hs = slice(h * g, (h + 1) * g)
                q = self.q[b, :, hs].double().reshape(-1, self.dk)
                o, l, A, S = plain_attn(q, k, v, sees[:, live].repeat_interleave(g, 0), self.scale)
                n = k.shape[0]
                ds = (self.dk + 8) * 2.0 ** -23 * S
                rel = 2 * ds + 2.0 ** -20 + n * 2.0 ** -24
                got = out[b, :, hs].double().reshape(-1, self.dv)
                fine = o.isfinite().all(-1)
                low = 2.0 ** -8 if self.dt == torch.bfloat16 else 2.0 ** -24
                p16 = 2.0 ** -11 if self.dt == torch.bfloat16 else 0.0
                which = "k" if self.latent else "v"
                vt = (self.kt if self.latent else self.vt)[b, :, h, : self.dv].double()
                top = 2 * float(vt[vt.isfinite()].abs().max()) if p16 else 0.0
                if p16 and P:
                    e = self.cache(which).exps(b, h)[: -(-P // BLOCK)]
                    top = max(top, 512 * 2.0 ** (int(e.max()) - 127))
                tol = low * o.abs() + (rel + p16)[:, None] * A * 1.01 + n * 2.0 ** -32 * top + 1e-37
                assert not got[fine].isnan().any()
                bad = ((got - o).abs() > tol)[fine]
                assert not bad.any(), (b, h, float(((got - o).abs() / tol)[fine].max()))
                assert not got[~fine].isfinite().all(-1).any()
                gl = lse[b, :, hs].double().reshape(-1)
                tl = rel + 2.0 ** -22 * l.abs() + 2.0 ** -20
                assert ((gl - l).abs() <= tl)[l.isfinite()].all(), (b, h)


gpu = pytest.mark.gpu


# ------------------------------------------------- refusals (on the host) --

A, U, N = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10004), None


def _desc(**kw):
    base = dict(B=2, R=5, Hq=4, Hkv=2, dk=128, dv=128, cap=256, dtype=T.TSD_BF16, v_aliases_k=0,
                scale=0.088)
    base.update(kw)
    return T.tsd_attn_desc(**base)


def _calls(d, table=N, mp=0, ps=0, npg=0, x=A, S=3, rows=4, ws=1 << 40, decay=1.0, keep=8, sink=1,
           recent=2):
    r, pg, L = ctypes.byref(d), (table, mp, ps, npg), T.lib
    return {
        "write": lambda: L.tsd_cache_write_q8(r, rows, x, A, A, A, A, A, A, *pg, A, N, N),
        "commit": lambda: L.tsd_commit_path_q8(r, S, x, A, A, A, A, A, A, A, *pg, A, N, N),
        "attn": lambda: L.tsd_tree_verify_attn_q8(r, x, A, A, A, A, *pg, A, A, A, A, A, A, A, ws,
                                                  N, N),
        "weights": lambda: L.tsd_cache_weights(r, S, x, A, *pg, A, A, A, A, A, decay, A, A, A, N, N),
        "weights_q8": lambda: L.tsd_cache_weights_q8(r, S, x, A, A, *pg, A, A, A, A, A, decay, A, A,
                                                     A, N, N),
        "evict": lambda: L.tsd_cache_evict(r, keep, sink, recent, x, A, A, A, A, *pg, A, A, ws, N,
                                           N),
        "evict_q8": lambda: L.tsd_cache_evict_q8(r, keep, sink, recent, x, A, A, A, A, A, A, *pg, A,
                                                 A, ws, N, N)}


ALL = list(_calls(_desc()))


@pytest.mark.parametrize("name", ALL)
@pytest.mark.parametrize("kw", [dict(B=0), dict(B=65536), dict(R=0), dict(R=66), dict(Hq=3),
                                dict(Hkv=0), dict(dk=96, dv=96), dict(dk=128, dv=64), dict(dtype=7),
                                dict(cap=0), dict(v_aliases_k=1)])
def test_calls_reject_bad_descriptors(name, kw):
    assert _calls(_desc(**kw))[name]() == T.TSD_ERR_INVALID_ARG


@pytest.mark.parametrize("name", ALL)
@pytest.mark.parametrize("kw", [dict(x=N), dict(x=U), dict(ps=-1), dict(ps=64, table=A, mp=4, npg=8),
                                dict(ps=128, table=A, mp=3, npg=8), dict(ps=128, table=N, mp=2, npg=8),
                                dict(ps=128, table=U, mp=2, npg=8), dict(ps=128, table=A, mp=2)])
def test_calls_reject_bad_pointers_and_pages(name, kw):
    assert _calls(_desc(), **kw)[name]() == T.TSD_ERR_INVALID_ARG


@pytest.mark.parametrize("name,kw", [("commit", dict(S=0)), ("commit", dict(S=17)),
                                     ("write", dict(rows=0)), ("weights", dict(S=17)),
                                     ("weights_q8", dict(S=0)), ("weights", dict(decay=-0.5)),
                                     ("weights", dict(decay=1.5)), ("weights_q8", dict(decay=NAN)),
                                     ("evict", dict(keep=0)), ("evict", dict(sink=-1)),
                                     ("evict", dict(recent=-1)), ("evict_q8", dict(sink=7)),
                                     ("evict", dict(ws=16)), ("evict_q8", dict(ws=16))])
def test_calls_reject_bad_numbers(name, kw):
    assert _calls(_desc(), **kw)[name]() == T.TSD_ERR_INVALID_ARG


@pytest.mark.parametrize("name", ["attn", "weights", "weights_q8"])
@pytest.mark.parametrize("scale", [0.0, -1.0, NAN, INF])
def test_attention_calls_reject_bad_scales(name, scale):
    assert _calls(_desc(scale=scale))[name]() == T.TSD_ERR_INVALID_ARG


def test_attention_rejects_a_short_workspace():
    d = _desc(B=1, R=9, Hq=8, Hkv=1, cap=8192)
    need = T.tsd_verify_q8_workspace_size(d)
    assert need > 0
    assert _calls(d, ws=need - 1)["attn"]() == T.TSD_ERR_INVALID_ARG


def test_plain_rounding_is_that_of_the_type():
    x = torch.linspace(-500, 500, 20011, dtype=torch.float64)
    x = torch.cat([x, x / 1000, x / 30000])
    ref = x.clamp(-448, 448).float().to(torch.float8_e4m3fn).double()
    assert torch.equal(nearest_code(x.float().double()), ref)


@gpu
def test_binding_rejects_types_shapes_and_pages():
    s = Setup("one", 2, 3, [40])
    out = torch.empty(2, 3, 2, 128, dtype=s.dt, device=DEV)
    lse = torch.empty(2, 3, 2, device=DEV)
    ws = T.workspace(T.tsd_verify_q8_workspace_size(s.desc))

    def call(**kw):
        a = dict(q=s.q, kq=s.k, vq=s.v, kexp=s.ke, vexp=s.ve, prefix_len=s.plen, ktree=s.kt,
                 vtree=s.vt, mask=s.mask, out=out, lse=lse, ws=ws)
        a.update(kw)
        T.tsd_tree_verify_attn_q8(s.desc, **a)

    call()
    call(kq=s.k.view(torch.float8_e4m3fn), vq=s.v.view(torch.float8_e4m3fn))
    for bad in (dict(kq=s.k.half()), dict(kexp=s.ke.int()), dict(q=s.q.float())):
        with pytest.raises(TypeError):
            call(**bad)
    for bad in (dict(kq=s.k[:, :, :-1].contiguous()), dict(vexp=s.ve[:1]), dict(page_size=128),
                dict(kq=s.k.transpose(0, 1)), dict(mask=s.mask.cpu())):
        with pytest.raises(ValueError):
            call(**bad)


# ----------------------------------------------------------------- writes --

def _write(s, new, vnew, n, commit=None):
    before = {w: [[(s.cache(w).rows(b, h), s.cache(w).exps(b, h)) for h in range(s.Hkv)]
                  for b in range(s.B)] for w in ("k", "v") if not (s.latent and w == "v")}
    cache = (s.k, s.v, s.ke, s.ve, s.plen, s.err)
    if commit is None:
        T.tsd_cache_write_q8(s.desc, new, vnew, n, *cache, **s.paging)
    else:
        rows, length, S = commit
        T.tsd_commit_path_q8(s.desc, S, new, vnew, rows, length, *cache, **s.paging)
    torch.cuda.synchronize()
    return before


def _same(a, b):
    return torch.equal(a.nan_to_num(777.0), b.nan_to_num(777.0))


def _check_write(s, before, pick):
    """pick(b, h, which): the float64 rows that request b appends (None: skipped)."""
    for w, was in before.items():
        old = s.cache(w)
        for b in range(s.B):
            for h in range(s.Hkv):
                codes, e = was[b][h]

                class Old:
                    rows = staticmethod(lambda *_: codes.clone())
                    exps = staticmethod(lambda *_: e.clone())

                new = pick(b, h, w)
                if new is not None and len(new):
                    codes, e = plain_write(Old, b, h, s.lens[b], new)
                assert torch.equal(old.exps(b, h), e), (w, b, h)
                assert _same(old.rows(b, h), codes), (w, b, h)
    for b in range(s.B):
        new = pick(b, 0, "k")
        assert int(s.plen[b]) == s.lens[b] + (0 if new is None else len(new))


@gpu
@pytest.mark.parametrize("kind,dtype,page", [("gqa", torch.bfloat16, 0), ("narrow", torch.float32, 128),
                                             ("latent", torch.bfloat16, 256), ("one", torch.float32, 0),
                                             ("latent-few", torch.float32, 0),
                                             ("narrow", torch.bfloat16, 0)])
def test_write_appends_rows_of_every_length(kind, dtype, page):
    """Old lengths at, before and behind block borders; 0, 1 and many new rows; magnitudes
    that grow the last block's exponent, and some that do not; zero rows."""
    Tn = 200
    s = Setup(kind, 6, 1, [0, 1, 63, 64, 100, 129], extra=Tn + 3, dtype=dtype, page=page, seed=3)
    x, y = s.normal(6, Tn, s.Hkv, s.dk), None if s.latent else s.normal(6, Tn, s.Hkv, s.dv)
    x[1] *= 100.0
    x[2] *= 1e-6
    x[3, :, 0] = 0.0
    n = torch.tensor([200, 64, 1, 130, 0, 63], dtype=torch.int32, device=DEV)
    before = _write(s, x, y, n)
    assert int(s.err) == 0
    _check_write(s, before, lambda b, h, w: (x if w == "k" else y)[b, : int(n[b]), h].double())


@gpu
@pytest.mark.parametrize("kind,page", [("gqa", 0), ("narrow", 128), ("latent", 0), ("wide", 256)])
def test_commit_writes_the_accepted_rows(kind, page):
    s = Setup(kind, 5, 40, [0, 60, 63, 64, 250], extra=17, page=page, seed=5)
    S = 16
    s.kt[2] *= 50.0
    paths = [[0] + sorted(s.rnd.sample(range(1, 40), L)) for L in (0, 16, 7, 3, 16)]
    rows = torch.tensor([p + [-1] * (17 - len(p)) for p in paths], dtype=torch.int32, device=DEV)
    length = torch.tensor([len(p) - 1 for p in paths], dtype=torch.int32, device=DEV)
    before = _write(s, s.kt, s.vt, None, (rows, length, S))
    assert int(s.err) == 0
    _check_write(s, before, lambda b, h, w: (s.kt if w == "k" else s.vt)[b, paths[b], h].double())


@gpu
def test_write_takes_values_at_the_ends_of_the_format():
    """Magnitudes on both sides of every border of the exponent rule, the largest and
    smallest bf16, infinities, NaN and zero."""
    s = Setup("one", 4, 1, [0], extra=256, seed=1)
    x = s.normal(4, 256, 2, 128)
    x[0, :64] = 0.0
    x[0, 0, 0, 0] = 448.0
    x[0, 64:128] = 0.0
    x[0, 64, 0, 0] = 450.0
    x[0, 128:192] *= 1e30
    x[0, 192:] *= 1e-36
    x[1, 5, 0, 3], x[1, 6, 0, 4], x[1, 7, 1, 5] = NAN, INF, -INF
    x[2, :64] = torch.finfo(torch.bfloat16).max
    x[2, 64:128] = torch.finfo(torch.bfloat16).tiny
    x[2, 128:] = INF
    x[3, 17] = -0.0
    n = torch.full((4,), 256, dtype=torch.int32, device=DEV)
    before = _write(s, x, x.clone(), n)
    _check_write(s, before, lambda b, h, w: x[b, :, h].double())


@gpu
def test_write_and_commit_skip_requests_with_errors():
    s = Setup("one", 4, 5, [10, 20, 30, 40], extra=4, page=128, seed=2)
    s.plen[1] = s.cap - 1                     # no room for two rows
    s.lens[1] = s.cap - 1
    s.table[2, 0] = 99                        # a page outside the pool
    x = s.normal(4, 8, 2, 128)
    n = torch.tensor([2, 2, 2, 9], dtype=torch.int32, device=DEV)
    k0, e0 = s.k.clone(), s.ke.clone()
    table = s.table.clone()
    _write_ok = T.tsd_cache_write_q8
    _write_ok(s.desc, x, x, n, s.k, s.v, s.ke, s.ve, s.plen, s.err, **s.paging)
    torch.cuda.synchronize()
    assert int(s.err) != 0 and int(s.err) & T.TSD_DEV_ERR_MASK in (T.TSD_DEV_ERR_CAPACITY,
                                                                   T.TSD_DEV_ERR_BAD_PAGE)
    assert s.plen.tolist() == [12, s.cap - 1, 30, 40]
    used = int(table[0, 0])
    others = [p for p in range(s.k.shape[0]) if p != used]
    assert torch.equal(s.k[others], k0[others]) and torch.equal(s.ke[others], e0[others])
    s.err.zero_()
    rows = torch.tensor([[0, 9, -1], [0, 1, 2], [0, 1, -1], [0, -1, -1]], dtype=torch.int32, device=DEV)
    length = torch.tensor([1, 2, 1, 3], dtype=torch.int32, device=DEV)
    k1 = s.k.clone()
    T.tsd_commit_path_q8(s.desc, 2, s.kt, s.vt, rows, length, s.k, s.v, s.ke, s.ve, s.plen, s.err,
                         **s.paging)
    torch.cuda.synchronize()
    assert torch.equal(s.k, k1) and s.plen.tolist() == [12, s.cap - 1, 30, 40]
    assert int(s.err) != 0


# -------------------------------------------------------------- attention --

ATTN = [("gqa", 1, 1, [2048], {}), ("gqa", 3, 17, [700, 1, 129], {}), ("gqa", 2, 33, [1300, 64], dict(page=128)),
        ("gqa", 2, 65, [515], {}), ("narrow", 3, 9, [300, 128, 5], {}), ("narrow", 2, 40, [1000], dict(page=256)),
        ("one", 4, 1, [3, 127, 128, 129], {}), ("wide", 1, 65, [900], {}), ("wide", 2, 2, [4000], dict(page=128)),
        ("latent", 2, 1, [300, 1000], {}), ("latent", 1, 9, [515], dict(page=128)), ("latent-few", 2, 3, [200], {}),
        ("gqa", 2, 5, [777], dict(dtype=torch.float32)), ("narrow", 2, 3, [90], dict(dtype=torch.float32, page=128)),
        ("latent-few", 1, 2, [333], dict(dtype=torch.float32)), ("gqa", 40, 2, [500, 90, 1], {}),
        ("gqa", 3, 4, [130, 2500, 1], {}), ("gqa", 3, 5, [130, 2500, 1], dict(page=128)), ("gqa", 2, 8, [400], {}),
        ("narrow", 2, 3, [777, 64], {}), ("gqa", 24, 9, [300, 1, 130], dict(page=128)),
        ("latent", 10, 9, [300, 10, 129], {})]


@gpu
@pytest.mark.parametrize("kind,B,R,lens,kw", ATTN)
def test_attention_matches_plain(kind, B, R, lens, kw):
    s = Setup(kind, B, R, lens, seed=B + R, **kw)
    out, lse = s.attn()
    assert int(s.err) == 0
    s.check_attn(out, lse)


@gpu
@pytest.mark.parametrize("kind,dtype", [("gqa", torch.bfloat16), ("latent", torch.bfloat16),
                                        ("narrow", torch.float32), ("narrow", torch.bfloat16)])
def test_attention_of_empty_and_tiny_prefixes(kind, dtype):
    s = Setup(kind, 5, 7, [0, 1, 2, 64, 65], dtype=dtype, seed=9)
    out, lse = s.attn()
    s.check_attn(out, lse)


@gpu
@pytest.mark.parametrize("kind", ["gqa", "latent", "latent-few"])
def test_attention_keeps_small_values_beside_large_ones(kind):
    """Blocks whose scales differ by 2^12 (K) and 2^8 (V), growing and shrinking along the
    prefix, and rows of q whose magnitudes differ by 2^60."""
    s = Setup(kind, 2, 6, [1000, 700], seed=4, spread=0)
    nb = s.ke.shape[-1]
    s.ke.copy_((114 + torch.arange(nb, device=DEV) * 5 % 13).to(torch.uint8).expand_as(s.ke))
    if s.ve is not None:
        s.ve.copy_((121 - torch.arange(nb, device=DEV) * 3 % 9).to(torch.uint8).expand_as(s.ve))
    s.q[:, 1] *= 2.0 ** -40
    s.q[:, 2] *= 2.0 ** 20
    s.q[:, 3] = 0.0
    out, lse = s.attn()
    s.check_attn(out, lse)


@gpu
@pytest.mark.parametrize("kind,R", [("gqa", 2), ("gqa", 20), ("narrow", 3), ("latent", 2)])
@pytest.mark.parametrize("tree", [False, True])
def test_attention_of_values_far_below_the_largest(kind, R, tree):
    """Value blocks (or one scratch row that one row sees) up to 2^24 times the others: what
    the small ones lose stays within the documented bound."""
    s = Setup(kind, 2, R, [1500, 300], seed=18, spread=0)
    if tree:
        s.set_masks([[0] + [1 << (r - 1) for r in range(1, R)]] * 2)
        (s.kt if s.latent else s.vt)[:, -1, :, : s.dv] *= 2.0 ** (2 if s.latent else 24)
    elif s.latent:
        s.ke[..., ::5] += 6
    else:
        s.ve[..., ::3] += 24
    if s.latent:
        s.q.mul_(2.0 ** -6)
    out, lse = s.attn()
    s.check_attn(out, lse)


@gpu
@pytest.mark.parametrize("kind,dtype", [("gqa", torch.bfloat16), ("latent", torch.bfloat16),
                                        ("gqa", torch.float32), ("latent-few", torch.bfloat16)])
def test_attention_leaves_out_what_no_row_sees(kind, dtype):
    """NaN codes and exponents behind the prefix, NaN and infinity in scratch rows that no
    row sees: the same output as with zeros there."""
    s = Setup(kind, 3, 12, [130, 64, 0], dtype=dtype, extra=200, seed=6)
    m = [list(x) for x in s.masks]
    for b in range(3):                            # rows 9..11 are padding: nobody's ancestors
        m[b][9:] = [0, 0, 0]
        for r in range(9):
            m[b][r] &= (1 << 8) - 1
    s.set_masks(m)
    for b in range(3):
        end = s.lens[b]
        s.k[b, :, end:] = 0
        s.ke[b, :, -(-end // BLOCK):] = 127
        if not s.latent:
            s.v[b, :, end:] = 0
            s.ve[b, :, -(-end // BLOCK):] = 127
    s.kt[:, 9:] = 0
    if not s.latent:
        s.vt[:, 9:] = 0
    ref = s.attn()
    for b in range(3):
        end = s.lens[b]
        s.k[b, :, end:] = 0x7F
        s.ke[b, :, -(-end // BLOCK):] = 255
        if not s.latent:
            s.v[b, :, end:] = 0x7F
            s.ve[b, :, -(-end // BLOCK):] = 255
    s.kt[:, 9], s.kt[:, 10], s.kt[:, 11] = NAN, INF, -3e38
    if not s.latent:
        s.vt[:, 9], s.vt[:, 10], s.vt[:, 11] = INF, NAN, 3e38
    got = s.attn()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    s.check_attn(*got)


@gpu
@pytest.mark.parametrize("kind,dtype", [("gqa", torch.bfloat16), ("latent", torch.bfloat16),
                                        ("gqa", torch.float32), ("latent-few", torch.bfloat16)])
def test_attention_keeps_nan_to_the_rows_that_see_it(kind, dtype):
    s = Setup(kind, 1, 8, [200], dtype=dtype, seed=8)
    s.set_masks([[0, 1, 2, 4 | 1, 8 | 2, 16 | 2, 32, 64]])
    ref = s.attn()
    (s.kt if s.latent else s.vt)[0, 2, 0, 5] = NAN            # row 2 (bit 1): rows 2, 4, 5 see it
    got, _ = s.attn()
    g = s.Hq // s.Hkv
    sick = torch.zeros(8, s.Hq, dtype=torch.bool, device=DEV)
    sick[[2, 4, 5], :g] = True
    assert got[0].isnan().any(-1)[sick].all()
    assert torch.equal(got[0][~sick], ref[0][0][~sick])
    s.vt = s.vt if s.latent else s.vt.nan_to_num(0.0)
    s.kt = s.kt.nan_to_num(0.0)
    clean, _ = s.attn()
    s.q[0, 3, 1] = INF                                        # one query row
    bad, _ = s.attn()
    assert bad[0, 3, 1].isnan().any()
    keep = torch.ones(8, s.Hq, dtype=torch.bool, device=DEV)
    keep[3, 1] = False
    assert torch.equal(bad[0][keep], clean[0][keep])


@gpu
@pytest.mark.parametrize("kind", ["gqa", "latent", "narrow"])
def test_attention_with_late_large_scores(kind):
    """Scores that keep growing along the prefix: every tile passes the running maximum."""
    s = Setup(kind, 1, 4, [1500], seed=11, spread=0)
    s.ke.copy_((113 + torch.arange(s.ke.shape[-1], device=DEV) * 2 // 3).clamp(max=124).to(torch.uint8)
               .expand_as(s.ke))
    s.q.mul_(4)
    out, lse = s.attn()
    s.check_attn(out, lse)


@gpu
@pytest.mark.parametrize("kind,R,page", [("gqa", 1, 0), ("gqa", 20, 128), ("narrow", 2, 128),
                                         ("narrow", 20, 0), ("latent", 3, 0), ("latent-few", 2, 128)])
def test_attention_waits_give_up_at_the_budget(kind, R, page):
    """A budget of a few clock cycles: the softmax's first wait on a product gives up, every
    role stops, and the kernel ends at once with a code in err.  The next call is as ever."""
    s = Setup(kind, 3, R, [2500, 700, 0], page=page, seed=19)
    want = s.attn()
    with T.wait_budget(16):
        s.attn()                                      # (loads the kernel)
        start = time.monotonic()
        s.attn()
    assert time.monotonic() - start < 0.9             # (no wait of the default budget ran out)
    e = int(s.err)
    assert e & T.TSD_DEV_ERR_MASK == T.TSD_DEV_ERR_TIMEOUT and e & 0xFFFFFF < 3, hex(e)
    assert T.tsd_set_wait_budget(0) == 0              # the context manager restored it
    s.err.zero_()
    got = s.attn()
    assert int(s.err) == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    s.check_attn(*got)


@gpu
@pytest.mark.parametrize("kind,page", [("gqa", 128), ("latent", 128), ("one", 256)])
def test_attention_reports_a_page_outside_the_pool(kind, page):
    s = Setup(kind, 2, 3, [600, 500], page=page, seed=12)
    s.table[0, 1] = s.k.shape[0] + 5
    out, lse = s.attn()
    assert int(s.err) == T.TSD_DEV_ERR_BAD_PAGE | 0
    s.check_attn(out, lse, requests=[1])


@gpu
def test_attention_clamps_lengths_to_the_cache():
    s = Setup("gqa", 2, 3, [90, 100], extra=0, seed=13)
    s.plen[0], s.plen[1] = 100000, -5
    s.lens = [s.cap, 0]
    out, lse = s.attn()
    s.check_attn(out, lse)


@gpu
@pytest.mark.parametrize("kind", ["gqa", "latent"])
def test_attention_on_a_stream_and_in_a_graph(kind):
    """A captured call replays on new contents of its tensors, also beside another
    stream's call with a workspace of its own."""
    s, other = Setup(kind, 2, 5, [900, 400], seed=14), Setup(kind, 2, 5, [900, 400], seed=15)
    out, lse = s.attn()
    st = torch.cuda.Stream()
    o = [torch.empty_like(out) for _ in range(2)]
    l = [torch.empty_like(lse) for _ in range(2)]
    ws = [T.workspace(T.tsd_verify_q8_workspace_size(s.desc)) for _ in range(2)]
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        s.attn_into(o[0], l[0], ws[0], st)
    for name in ("q", "k", "v", "ke", "ve", "kt", "vt", "mask"):
        if getattr(s, name) is not None:
            getattr(s, name).copy_(getattr(other, name))
    s.masks = other.masks
    torch.cuda.synchronize()
    graph.replay()
    with torch.cuda.stream(st):
        other.attn_into(o[1], l[1], ws[1], st)
    torch.cuda.synchronize()
    assert torch.equal(o[0], o[1]) and torch.equal(l[0], l[1])
    s.check_attn(o[0], l[0])


@gpu
@pytest.mark.parametrize("kinds", [("gqa", "latent"), ("gqa", "gqa"), ("narrow", "one")])
def test_two_streams_at_once(kinds):
    """Attention, then eviction, on two streams with state and workspaces of their own: the
    results of one at a time."""
    sets = [Setup(k, 6, 5 + i, [900, 40, 333], extra=16, seed=60 + i) for i, k in enumerate(kinds)]
    for s in sets:
        _evict_state(s)
        s.out = torch.empty(s.B, s.R, s.Hq, s.dv, dtype=s.dt, device=DEV)
        s.ws = T.workspace(T.tsd_verify_q8_workspace_size(s.desc))
        s.ws_evict = T.workspace(T.tsd_cache_evict_workspace_size(s.desc))
        s.lse = torch.empty(s.B, s.R, s.Hq, device=DEV)
        s.state = [t for t in (s.k, s.v, s.ke, s.ve, s.acc, s.pos, s.plen) if t is not None]
        s.before = [t.clone() for t in s.state]

    def round_of(s):
        for t, b in zip(s.state, s.before):
            t.copy_(b)
        s.attn_into(s.out, s.lse, s.ws)
        T.tsd_cache_evict_q8(s.desc, 200, 2, 20, s.acc, s.pos, s.seen, s.k, s.v, s.ke, s.ve, s.plen,
                             s.ws_evict, s.err)

    want = []
    for s in sets:
        round_of(s)
        torch.cuda.synchronize()
        want.append([t.clone() for t in [s.out, s.lse] + s.state])
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        for s, stream in zip(sets, streams):
            with torch.cuda.stream(stream):
                round_of(s)
    torch.cuda.synchronize()
    for s, w in zip(sets, want):
        assert all(torch.equal(t, x) for t, x in zip([s.out, s.lse] + s.state, w))
        assert int(s.err) == 0


@gpu
def test_attention_is_the_same_twice_and_for_any_rows_of_a_tree():
    s = Setup("gqa", 3, 33, [1000, 700, 65], seed=16)
    a, b = s.attn(), s.attn()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@gpu
def test_attention_past_32_bit_offsets():
    """A cache of more than 2^32 codes: its last request and head, paged and not."""
    for page in (0, 4096):
        s = Setup.__new__(Setup)
        cap, B, Hkv = 1 << 20, 5, 8
        s.Hq, s.Hkv, s.dk, s.dv, s.B, s.R, s.dt, s.q8, s.page = 32, Hkv, 128, 128, B, 2, torch.bfloat16, True, page
        s.latent, s.cap, s.scale = False, cap, float(torch.tensor(1 / math.sqrt(128), dtype=torch.float32))
        s.g, s.rnd, s.lens = torch.Generator(device=DEV).manual_seed(1), random.Random(1), [3, 3, 3, 3, 40000]
        s.table = None if not page else torch.arange(B * cap // page, dtype=torch.int32, device=DEV).flip(0).view(
            B, cap // page).contiguous()
        lead, rows = ((B, Hkv), cap) if not page else ((B * cap // page, Hkv), page)
        s.k = torch.randint(0, 120, (*lead, rows, 128), generator=s.g, device=DEV, dtype=torch.uint8)
        s.v = torch.randint(0, 120, (*lead, rows, 128), generator=s.g, device=DEV, dtype=torch.uint8)
        s.ke = torch.full((*lead, rows // BLOCK), 118, device=DEV, dtype=torch.uint8)
        s.ve = torch.full((*lead, rows // BLOCK), 119, device=DEV, dtype=torch.uint8)
        s.plen = torch.tensor(s.lens, dtype=torch.int32, device=DEV)
        s.q, s.kt, s.vt = s.normal(B, 2, 32, 128, std=0.2), s.normal(B, 2, Hkv, 128), s.normal(B, 2, Hkv, 128)
        s.set_masks([[0, 1]] * B)
        s.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        s.desc = T.make_desc(B, 2, 32, Hkv, 128, 128, cap, s.dt, False, s.scale)
        s.paging = dict(page_table=s.table, page_size=page)
        out, lse = s.attn()
        assert int(s.err) == 0
        s.check_attn(out, lse, requests=[0, 4], heads=[0, 7])


# ---------------------------------------------------------------- weights --

def _weights_state(s, S, lens=None):
    L = lens or [s.rnd.randint(0, min(S, s.R - 1)) for _ in range(s.B)]
    paths = [[0] + sorted(s.rnd.sample(range(1, s.R), n)) for n in L]
    s.paths = paths
    s.path = torch.tensor([p + [-1] * (S + 1 - len(p)) for p in paths], dtype=torch.int32, device=DEV)
    s.plength = torch.tensor(L, dtype=torch.int32, device=DEV)
    s.acc = torch.rand(s.B, s.Hkv, s.cap, generator=s.g, device=DEV) * 3
    s.pos = torch.randint(0, 1000, (s.B, s.Hkv, s.cap), generator=s.g, device=DEV, dtype=torch.int32)
    s.seen = torch.tensor([[n + 50] * s.Hkv for n in s.lens], dtype=torch.int32, device=DEV)
    s.lse = torch.rand(s.B, s.R, s.Hq, generator=s.g, device=DEV) + 5.0


def _weights(s, S, decay):
    cache = (s.k, s.ke) if s.q8 else (s.k,)
    f = T.tsd_cache_weights_q8 if s.q8 else T.tsd_cache_weights
    f(s.desc, S, s.q, *cache, s.plen, s.kt, s.path, s.plength, s.lse, decay, s.acc, s.pos, s.seen,
      s.err, **s.paging)


def _check_weights(s, acc0, pos0, seen0, decay):
    """A term exp(x) is off by its score's error, (dk + 8) 2^-23 S with S the largest
    scale sum |q k|, plus 2^-20 for the exponential and lse's products (|lse| < 16); n
    positive terms summed in fp32 add n 2^-24; the decayed value one rounding."""
    g = s.Hq // s.Hkv
    for b in range(s.B):
        P, path = s.lens[b], s.paths[b]
        for h in range(s.Hkv):
            hs = slice(h * g, (h + 1) * g)
            q, l = s.q[b, path, hs].double(), s.lse[b, path, hs].double()
            k = s.cache("k").values(b, h)[:P]
            t = s.kt[b, path, h].double()
            both = torch.cat([k, t])
            x = torch.einsum("igd,kd->igk", q, both) * s.scale
            S1 = float((torch.einsum("igd,kd->igk", q.abs(), both.abs()) * s.scale).max())
            p = torch.exp(x - l[..., None])
            ref = p[..., :P].sum((0, 1)) + decay * acc0[b, h, :P].double()
            new = torch.tril(p[..., P:].sum(1)).sum(0)
            n = len(path) * g
            rel = (s.dk + 8) * 2.0 ** -23 * S1 + 2.0 ** -20 + (n + 2) * 2.0 ** -24
            got = s.acc[b, h].double()
            end = P + len(path)
            assert ((got[:P] - ref).abs() <= rel * ref + 1e-37).all(), (b, h)
            assert ((got[P:end] - new).abs() <= rel * new + 1e-37).all(), (b, h)
            assert torch.equal(s.acc[b, h, end:], acc0[b, h, end:])
            want = pos0[b, h].clone()
            want[P:end] = int(seen0[b, h]) + torch.arange(len(path), device=DEV)
            assert torch.equal(s.pos[b, h], want)
        assert torch.equal(s.seen[b], seen0[b] + len(path))


WEIGHTS = [("gqa", 3, 20, [700, 1, 128], 8, {}), ("gqa", 2, 65, [300, 0], 16, dict(page=128)),
           ("narrow", 3, 9, [130, 63, 900], 5, {}), ("wide", 2, 33, [257], 16, dict(page=256)),
           ("one", 4, 2, [5, 127, 128, 129], 1, {}), ("latent", 2, 4, [150, 300], 3, {}),
           ("latent", 1, 20, [515], 16, dict(page=128)),
           ("latent-few", 2, 12, [200, 64], 6, {}), ("latent", 2, 5, [129], 2, dict(dtype=torch.float32)),
           ("gqa", 2, 7, [200], 3, dict(dtype=torch.float32)), ("gqa", 33, 5, [300, 20], 4, {})]


@gpu
@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("kind,B,R,lens,S,kw", WEIGHTS)
def test_weights_match_plain(kind, B, R, lens, S, kw, q8):
    s = Setup(kind, B, R, lens, extra=20, seed=B * R, q8=q8, **kw)
    _weights_state(s, S)
    for decay in (1.0, 0.25, 0.0):
        acc0, pos0, seen0 = s.acc.clone(), s.pos.clone(), s.seen.clone()
        _weights(s, S, decay)
        torch.cuda.synchronize()
        assert int(s.err) == 0
        _check_weights(s, acc0, pos0, seen0, decay)


@gpu
@pytest.mark.parametrize("q8", [True, False])
def test_weights_of_an_attention_call_sum_to_its_rows(q8):
    """The weights of one row over all keys it sees add up to 1: over all rows and heads of
    a path, to (L + 1) x group.  (Up to the terms' bounds, as in _check_weights.)"""
    s = Setup("gqa", 2, 6, [500, 77], extra=20, seed=21, q8=True)
    s.set_masks([[0, 1, 3, 7, 15, 31]] * 2)
    _, lse = s.attn()
    if not q8:          # the same values held in bf16 (4 significant bits: exact)
        s.k = torch.stack([torch.stack([s.cache("k").values(b, h) for h in range(s.Hkv)])
                           for b in range(2)]).to(torch.bfloat16)
        s.ke, s.q8 = None, False
    _weights_state(s, 5, [5, 2])
    s.paths = [list(range(6)), [0, 1, 2]]
    s.path = torch.tensor([[0, 1, 2, 3, 4, 5], [0, 1, 2, -1, -1, -1]], dtype=torch.int32, device=DEV)
    s.lse = lse
    s.acc.zero_()
    _weights(s, 5, 1.0)
    torch.cuda.synchronize()
    for b, n in ((0, 6), (1, 3)):
        total = s.acc[b, :, : s.lens[b] + n].double().sum(-1)
        assert (total - 4 * n).abs().max() <= 4 * n * 2.0 ** -14


@gpu
@pytest.mark.parametrize("q8", [True, False])
def test_weights_skip_requests_with_errors(q8):
    s = Setup("gqa", 5, 4, [100], extra=100, page=128, seed=22, q8=q8)
    _weights_state(s, 3, [1, 1, 1, 1, 1])
    s.plen[0] = s.cap - 1
    s.plength[1] = 4
    s.path[2, 1] = 4
    s.table[3, 0] = -1
    acc0, pos0, seen0 = s.acc.clone(), s.pos.clone(), s.seen.clone()
    _weights(s, 3, 0.5)
    torch.cuda.synchronize()
    assert int(s.err) != 0
    assert torch.equal(s.acc[:4], acc0[:4]) and torch.equal(s.pos[:4], pos0[:4])
    assert torch.equal(s.seen[:4], seen0[:4])
    assert torch.equal(s.seen[4], seen0[4] + 2)


@gpu
@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("kind", ["gqa", "latent"])
def test_weights_skip_a_request_whose_commit_has_no_page(kind, q8):
    s = Setup(kind, 2, 4, [126], extra=100, page=128, seed=27, q8=q8)
    _weights_state(s, 3, [3, 3])
    s.table[0, 1] = s.k.shape[0]                  # positions 126..129 need page 1
    acc0, seen0 = s.acc.clone(), s.seen.clone()
    _weights(s, 3, 0.5)
    torch.cuda.synchronize()
    assert int(s.err) & T.TSD_DEV_ERR_MASK == T.TSD_DEV_ERR_BAD_PAGE
    assert torch.equal(s.acc[0], acc0[0]) and torch.equal(s.seen[0], seen0[0])
    assert torch.equal(s.seen[1], seen0[1] + 4)


@gpu
@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("kind,dtype", [("gqa", torch.bfloat16), ("latent", torch.bfloat16),
                                        ("one", torch.float32)])
def test_weights_and_commit_take_the_same_requests(kind, dtype, q8):
    """A page missing early in the prefix does not stop the commit, so the new rows get their
    positions, and weight 0; the request's other weights stay as they were.  The rest of the
    batch is as without that page missing."""
    def one(bad):
        s = Setup(kind, 3, 4, [300], extra=84, page=128, dtype=dtype, seed=28, q8=q8)
        _weights_state(s, 3, [2, 1, 3])
        if bad:
            s.table[1, 0] = bad
        before = [t.clone() for t in (s.acc, s.pos, s.seen)]
        _weights(s, 3, 0.5)
        if q8:
            T.tsd_commit_path_q8(s.desc, 3, s.kt, s.vt, s.path, s.plength, s.k, s.v, s.ke, s.ve,
                                 s.plen, s.err, **s.paging)
        else:
            T.tsd_commit_path_paged(s.desc, 3, s.kt, s.vt, s.path, s.plength, s.k, s.v, s.table,
                                    s.page, s.plen, s.err)
        torch.cuda.synchronize()
        return s, before

    good, _ = one(0)
    assert int(good.err) == 0
    for bad in (-1, 10 ** 6):
        s, (acc0, pos0, seen0) = one(bad)
        assert int(s.err) == T.TSD_DEV_ERR_BAD_PAGE | 1
        assert s.plen.tolist() == [303, 302, 304] == good.plen.tolist()
        assert torch.equal(s.seen, good.seen) and torch.equal(s.pos, good.pos)
        assert torch.equal(s.acc[[0, 2]], good.acc[[0, 2]])
        want = acc0[1].clone()
        want[:, 300:302] = 0.0
        assert torch.equal(s.acc[1], want)


@gpu
@pytest.mark.parametrize("kind,S", [("wide", (1, 7)), ("narrow", (1, 15)), ("wide", (9, 16))])
def test_weights_from_two_host_threads(kind, S):
    """Calls of different column counts, which take different amounts of shared memory, from
    two host threads with streams and state of their own."""
    sets = []
    for i, n in enumerate(S):
        s = Setup(kind, 1, 17, [200], extra=20, seed=70 + i)
        _weights_state(s, n, [n])
        s.S, s.stream, s.bad = n, torch.cuda.Stream(), []
        s.state = (s.acc.clone(), s.pos.clone(), s.seen.clone())
        sets.append(s)
    torch.cuda.synchronize()

    def run(s):
        def p(t):
            return ctypes.c_void_p(t.data_ptr())

        args = (ctypes.byref(s.desc), s.S, p(s.q), p(s.k), p(s.ke), None, 0, 0, 0, p(s.plen), p(s.kt),
                p(s.path), p(s.plength), p(s.lse), 0.0, p(s.acc), p(s.pos), p(s.seen), p(s.err),
                ctypes.c_void_p(s.stream.cuda_stream))
        for _ in range(6000):
            status = T.lib.tsd_cache_weights_q8(*args)
            if status != T.TSD_OK:
                s.bad.append(status)

    threads = [threading.Thread(target=run, args=(s,)) for s in sets]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert [len(s.bad) for s in sets] == [0, 0]
    for s in sets:
        assert int(s.err) == 0
        acc0, pos0, seen0 = s.state
        seen0 += 5999 * (s.S + 1)                 # (the last call's positions; decay 0)
        _check_weights(s, acc0, pos0, seen0, 0.0)


@gpu
@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("kind,S", [("gqa", 3), ("wide", 9), ("narrow", 4)])
def test_weights_waits_give_up_at_the_budget(kind, S, q8):
    """As the attention's; the tokens seen stay as they were, and a call on the state of before
    is exact."""
    s = Setup(kind, 2, 10, [2500, 700], extra=20, seed=30, q8=q8)
    _weights_state(s, S, [S, 1])
    state = (s.acc, s.pos, s.seen)
    before = [t.clone() for t in state]
    with T.wait_budget(16):
        for _ in range(2):                            # (the first loads the kernel)
            torch.cuda.synchronize()
            start = time.monotonic()
            _weights(s, S, 0.5)
            torch.cuda.synchronize()
    assert time.monotonic() - start < 0.9
    e = int(s.err)
    assert e & T.TSD_DEV_ERR_MASK == T.TSD_DEV_ERR_TIMEOUT and e & 0xFFFFFF < 2, hex(e)
    assert torch.equal(s.seen[e & 1], before[2][e & 1])
    s.err.zero_()
    for t, b in zip(state, before):
        t.copy_(b)
    _weights(s, S, 0.5)
    torch.cuda.synchronize()
    assert int(s.err) == 0
    _check_weights(s, *before, 0.5)


@gpu
@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("kind,S", [("latent", 3), ("latent", 9), ("latent-few", 9)])
def test_latent_weights_waits_give_up_at_the_budget(kind, S, q8):
    """Whatever piece of Q the loading warp gives up at, no wait for a copy that was never
    requested: the kernel ends within the budget and the copies' time."""
    test_weights_waits_give_up_at_the_budget(kind, S, q8)


@gpu
@pytest.mark.parametrize("q8", [True, False])
def test_weights_ignore_what_lies_behind_the_prefix(q8):
    s = Setup("gqa", 2, 5, [130, 64], extra=200, seed=23, q8=q8)
    _weights_state(s, 4, [2, 4])
    for b in range(2):
        if q8:
            s.k[b, :, s.lens[b]:] = 0x7F
            s.ke[b, :, -(-s.lens[b] // BLOCK):] = 255
        else:
            s.k[b, :, s.lens[b]:] = NAN
    off = [r for r in range(5) if r not in s.paths[0]]
    s.kt[0, off] = NAN
    s.q[0, off] = INF
    acc0, pos0, seen0 = s.acc.clone(), s.pos.clone(), s.seen.clone()
    _weights(s, 4, 1.0)
    torch.cuda.synchronize()
    _check_weights(s, acc0, pos0, seen0, 1.0)


def as_two_codes(x):
    """bf16 rows [..][d] as the sums of two e4m3 numbers that the products take, by their
    definition: the largest element scaled into [2^7, 2^8), the nearest code, and the nearest
    code of what is left.  Off by at most half of e4m3's smallest step, 2^-10, where the
    largest is at least 2^7: 2^-17 of it."""
    y = x.double()
    top = y.abs().amax(-1, keepdim=True)
    f = torch.exp2(8.0 - torch.frexp(top).exponent.double())
    hi = nearest_code(y * f)
    z = (hi + nearest_code(y * f - hi)) / f
    assert ((z - y).abs() <= 2.0 ** -17 * top).all()
    assert torch.equal(z.to(x.dtype).double(), z)          # (no more bits than before)
    return z.to(x.dtype)


def _dominant(s, by):
    """Each row of q (of ktree, unless it is also a value) gets one element `by` times its
    others, where every key (query) is zero: the others alone make the scores.  Then the rows
    as the products take them."""
    s.q[..., 3] = by
    s.k[..., 3] = 0
    s.kt[..., 3] = 0
    if s.latent:
        return as_two_codes(s.q), s.kt
    s.q[..., -1] = 0
    s.kt[..., -1] = by
    return as_two_codes(s.q), as_two_codes(s.kt)


@gpu
@pytest.mark.parametrize("kind,R", [("gqa", 2), ("gqa", 20), ("narrow", 2), ("narrow", 9), ("latent", 2),
                                    ("latent-few", 3)])
@pytest.mark.parametrize("by", [2.0 ** 8, 2.0 ** 12, 2.0 ** 15])
def test_attention_of_rows_with_a_dominant_element(kind, R, by):
    """The small elements are rounded as documented, and by nothing else: the outputs are
    within the bounds of the rounded rows."""
    s = Setup(kind, 2, R, [400, 90], seed=17)
    q, kt = _dominant(s, by)
    assert not torch.equal(q, s.q)
    got = s.attn()
    s.q, s.kt = q, kt
    s.check_attn(*got)


@gpu
@pytest.mark.parametrize("kind", ["gqa", "narrow", "wide"])
def test_weights_of_rows_with_a_dominant_element(kind):
    s = Setup(kind, 2, 9, [300, 64], extra=20, seed=29)
    _weights_state(s, 4, [4, 2])
    rounded = _dominant(s, 2.0 ** 12)
    acc0, pos0, seen0 = s.acc.clone(), s.pos.clone(), s.seen.clone()
    _weights(s, 4, 0.5)
    torch.cuda.synchronize()
    s.q, s.kt = rounded
    _check_weights(s, acc0, pos0, seen0, 0.5)


# --------------------------------------------------------------- eviction --

def _evict_state(s, sharp=True):
    s.acc = torch.rand(s.B, s.Hkv, s.cap, generator=s.g, device=DEV) ** (6 if sharp else 1)
    s.pos = torch.full((s.B, s.Hkv, s.cap), -1, dtype=torch.int32, device=DEV)
    for b, n in enumerate(s.lens):
        for h in range(s.Hkv):
            s.pos[b, h, :n] = torch.randperm(n, generator=s.g, device=DEV).int() * 2
    s.seen = torch.tensor([[2 * n] * s.Hkv for n in s.lens], dtype=torch.int32, device=DEV)


def _evict(s, keep, sink, recent, ws=None):
    ws = T.workspace(T.tsd_cache_evict_workspace_size(s.desc)) if ws is None else ws
    state = (s.acc, s.pos, s.seen)
    if s.q8:
        T.tsd_cache_evict_q8(s.desc, keep, sink, recent, *state, s.k, s.v, s.ke, s.ve, s.plen, ws,
                             s.err, **s.paging)
    else:
        T.tsd_cache_evict(s.desc, keep, sink, recent, *state, s.k, s.v, s.plen, ws, s.err, **s.paging)
    torch.cuda.synchronize()


def _snapshot(s):
    snap = {"acc": s.acc.clone(), "pos": s.pos.clone()}
    for w in ("k",) if s.latent else ("k", "v"):
        snap[w] = [[(s.cache(w).rows(b, h), s.cache(w).exps(b, h) if s.q8 else None)
                    for h in range(s.Hkv)] for b in range(s.B)]
    return snap


def _check_evict(s, snap, keep, sink, recent):
    for b in range(s.B):
        P = s.lens[b]
        assert int(s.plen[b]) == min(P, keep)
        for h in range(s.Hkv):
            acc, pos = snap["acc"][b, h], snap["pos"][b, h]
            src = torch.arange(s.cap, device=DEV)
            if P > keep:
                holes, movers = plain_evict(P, keep, sink, recent, acc[:P].tolist(), pos[:P].tolist(),
                                            int(s.seen[b, h]))
                assert len(holes) == len(movers)
                src[holes] = torch.tensor(movers, dtype=torch.long, device=DEV)
            assert torch.equal(s.acc[b, h].view(torch.int32), acc[src].view(torch.int32)), (b, h)
            assert torch.equal(s.pos[b, h], pos[src])
            for w in ("k",) if s.latent else ("k", "v"):
                rows, e = snap[w][b][h]
                want, we = rows[src], None if e is None else e.clone()
                if e is not None and P > keep:
                    er = e[src // BLOCK]
                    for j in range(-(-keep // BLOCK)):
                        part = slice(j * BLOCK, min((j + 1) * BLOCK, keep))
                        we[j] = er[part].max()
                        want[part] = nearest_code(want[part] * torch.exp2(
                            (er[part] - we[j]).double())[:, None])
                    assert torch.equal(s.cache(w).exps(b, h), we), (w, b, h)
                assert _same(s.cache(w).rows(b, h), want), (w, b, h)


EVICT = [("gqa", 3, [700, 200, 256], 256, 4, 64, {}), ("one", 4, [5000, 4999, 4096, 9000], 4096, 0, 0, {}),
         ("narrow", 2, [300, 70], 65, 0, 65, dict(page=128)), ("latent", 2, [400, 130], 129, 3, 10, {}),
         ("one", 2, [1000, 3], 1, 1, 0, {}), ("one", 1, [40000], 30000, 10, 500, {}),
         ("wide", 2, [600, 601], 600, 0, 100, dict(page=256)), ("gqa", 2, [900], 100, 0, 0, dict(dtype=torch.float32)),
         ("one", 1, [70000], 33000, 0, 7, dict(page=128)), ("one", 2, [9000, 12000], 8500, 2, 2, {})]


@gpu
@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("kind,B,lens,keep,sink,recent,kw", EVICT)
def test_evict_matches_plain(kind, B, lens, keep, sink, recent, kw, q8):
    s = Setup(kind, B, 1, lens, seed=keep, q8=q8, spread=6, **kw)
    _evict_state(s)
    snap = _snapshot(s)
    _evict(s, keep, sink, recent)
    assert int(s.err) == 0
    _check_evict(s, snap, keep, sink, recent)


@gpu
@pytest.mark.parametrize("values", [[1.0], [0.0, -0.0], [0.0, 1.0], [INF, 1.0, 0.0, -INF, -1.0],
                                    [1.0, 1.0 + 2 ** -23]])
def test_evict_ranks_ties_by_index(values):
    s = Setup("one", 2, 1, [777, 130], seed=31)
    _evict_state(s)
    pick = torch.randint(0, len(values), s.acc.shape, generator=s.g, device=DEV)
    s.acc = torch.tensor(values, device=DEV)[pick].contiguous()
    snap = _snapshot(s)
    _evict(s, 128, 5, 20)
    _check_evict(s, snap, 128, 5, 20)


@gpu
def test_evict_keeps_nan_weights_and_all_protected_rows():
    """NaN ranks above infinity; more protected rows than places (positions that repeat): the
    first of them stay."""
    s = Setup("one", 2, 1, [300, 300], seed=32)
    _evict_state(s)
    s.acc[0, :, 290] = NAN
    s.acc[0, :, 100:200] = INF
    s.pos[1] = 0
    k0 = s.k.clone()
    _evict(s, 101, 1, 0)
    first = s.acc[0, :, :101]
    assert first.isnan().any(-1).all()
    # head by head: the protected row (position 0), the NaN, then infinities by index
    assert (first.isinf().sum(-1) >= 98).all()
    assert torch.equal(s.k[1, :, :101], k0[1, :, :101])


NAN_BITS = [0x7FFFFFFF, -1, 0x7FC00000, -0x400000, 0x7F800001]   # (0xffffffff, 0xffc00000)


def plain_evict_any(P, keep, sink, recent, acc, pos, seen):
    """plain_evict with NaN weights: behind the protected rows, before infinity, by index; and
    with more protected rows than places, the first of which stay."""
    def key(i):
        if pos[i] < sink or pos[i] >= seen - recent:
            return (0, 0.0, i)
        return (1, -INF, i) if acc[i] != acc[i] else (2, -acc[i], i)

    kept = set(sorted(range(P), key=key)[:keep])
    return ([i for i in range(keep) if i not in kept], [i for i in range(keep, P) if i in kept])


@gpu
@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("bits", [[b] for b in NAN_BITS] + [NAN_BITS])
def test_evict_keeps_protected_rows_beside_any_nan(bits, q8):
    """NaN weights of either sign and any payload (0x7fffffff is what the device's arithmetic
    gives), more of them than places, the protected rows at the highest indexes: the protected
    stay, then NaN by index, then infinities."""
    s = Setup("one", 3, 1, [300, 300, 200], seed=36, q8=q8)
    _evict_state(s)
    s.acc[0] = INF
    some = torch.tensor(bits, dtype=torch.int32, device=DEV)
    for b, n in enumerate((260, 40, 90)):         # more than places, fewer, nearly all of them
        at = torch.randperm(s.lens[b] - 20, generator=s.g, device=DEV)[:n]
        pick = torch.randint(0, len(bits), (s.Hkv, n), generator=s.g, device=DEV)
        s.acc[b].view(torch.int32)[:, at] = some[pick]
    s.pos.copy_(torch.arange(s.cap, device=DEV).int().expand_as(s.pos))
    s.seen.copy_(torch.tensor(s.lens, device=DEV).int()[:, None].expand_as(s.seen))
    snap = _snapshot(s)
    _evict(s, 100, 3, 20)
    assert int(s.err) == 0 and s.plen.tolist() == [100, 100, 100]
    for b, P in enumerate(s.lens):
        for h in range(s.Hkv):
            acc, pos = snap["acc"][b, h], snap["pos"][b, h]
            holes, movers = plain_evict_any(P, 100, 3, 20, acc[:P].tolist(), pos[:P].tolist(), P)
            src = torch.arange(s.cap, device=DEV)
            src[holes] = torch.tensor(movers, dtype=torch.long, device=DEV)
            assert torch.equal(s.pos[b, h], pos[src]), (b, h)
            assert torch.equal(s.acc[b, h].view(torch.int32), acc[src].view(torch.int32))
            have = set(s.pos[b, h, :100].tolist())
            assert {0, 1, 2} | set(range(P - 20, P)) <= have
            if not q8:
                assert torch.equal(s.cache("k").rows(b, h), snap["k"][b][h][0][src])


@gpu
@pytest.mark.parametrize("kind,dtype", [("gqa", torch.bfloat16), ("latent", torch.bfloat16),
                                        ("one", torch.float32)])
def test_evict_after_the_weights_of_an_infinite_query(kind, dtype):
    """One accepted query row is infinite: every weight of its KV head is NaN from then
    on.  Rounds of weights, commit and eviction go on taking in the newest rows."""
    s = Setup(kind, 1, 4, [120], extra=8, dtype=dtype, seed=37)
    _weights_state(s, 3, [3])
    s.acc.zero_()
    s.pos.copy_(torch.arange(s.cap, device=DEV).int().expand_as(s.pos))
    s.seen.fill_(120)
    s.q[0, 0, 0] = INF                        # row 0 is on every path
    for step in range(3):
        _weights(s, 3, 0.5)
        T.tsd_commit_path_q8(s.desc, 3, s.kt, s.vt, s.path, s.plength, s.k, s.v, s.ke, s.ve, s.plen,
                             s.err, **s.paging)
        torch.cuda.synchronize()
        P, n = int(s.plen), int(s.seen[0, 0])
        assert s.acc[0, 0, :P].isnan().sum() >= P - 3      # (row 0 weighs nothing behind itself)
        _evict(s, 100, 2, 16)
        for h in range(s.Hkv):
            have = s.pos[0, h, :100].tolist()
            assert len(set(have)) == 100
            assert {0, 1} | set(range(n - 16, n)) <= set(have), (step, h)
    assert int(s.err) == 0 and int(s.plen) == 100


@gpu
@pytest.mark.parametrize("q8", [True, False])
def test_evict_again_and_again_at_a_budget(q8):
    """Rounds that append rows and cut back to the budget: the newest and the first tokens are
    always there, and no token is there twice."""
    s = Setup("one", 2, 1, [64, 64], extra=10, seed=33, q8=q8)
    _evict_state(s)
    s.pos[:, :, :64] = torch.arange(64, device=DEV).int()
    s.seen.fill_(64)
    for step in range(12):
        for b in range(2):
            n = 1 + (step + b) % 8
            P = s.lens[b] = 64
            s.plen[b] = P + n
            s.lens[b] = P + n
            s.acc[b, :, P:P + n] = torch.rand(2, n, generator=s.g, device=DEV)
            s.pos[b, :, P:P + n] = (s.seen[b, 0] + torch.arange(n, device=DEV)).int()
            s.seen[b] += n
        snap = _snapshot(s)
        _evict(s, 64, 2, 16)
        _check_evict(s, snap, 64, 2, 16)
        for b in range(2):
            for h in range(2):
                have = s.pos[b, h, :64].tolist()
                assert len(set(have)) == 64
                assert {0, 1} <= set(have)
                assert set(range(int(s.seen[b, h]) - 16, int(s.seen[b, h]))) <= set(have)


@gpu
@pytest.mark.parametrize("q8", [True, False])
def test_evict_skips_requests_with_errors(q8):
    s = Setup("one", 3, 1, [300, 300, 300], page=128, seed=34, q8=q8)
    _evict_state(s)
    s.plen[0] = s.cap + 1
    s.table[1, 2] = -7
    snap_acc, k0 = s.acc.clone(), s.k.clone()
    t = s.table.clone()
    _evict(s, 100, 0, 0)
    assert int(s.err) != 0
    assert s.plen.tolist() == [s.cap + 1, 300, 100]
    assert torch.equal(s.acc[:2], snap_acc[:2])
    mine = t[2].tolist()
    others = [p for p in range(s.k.shape[0]) if p not in mine]
    assert torch.equal(s.k[others], k0[others])


@gpu
def test_evict_with_room_to_spare_does_nothing():
    s = Setup("one", 2, 1, [100, 90], seed=35)
    _evict_state(s)
    snap = _snapshot(s)
    for keep in (100, s.cap, s.cap + 50):
        _evict(s, keep, 0, 0)
        _check_evict(s, snap, 100, 0, 0)


# groups of query heads that take other paths, or other splits of them, than KINDS
GROUPS = {"mqa32": (32, 1, 128, 128), "mqa71": (71, 1, 64, 64), "mha": (40, 40, 64, 64),
          "latent24": (24, 1, 576, 512), "latent4": (4, 1, 576, 512), "latent-two": (32, 2, 576, 512)}


@gpu
@pytest.mark.parametrize("kind,B,R,lens,S,kw", [("mqa32", 2, 12, [300, 64], 9, {}), ("mqa71", 1, 9, [130], 5, dict(page=128)),
                                                ("mha", 2, 3, [200, 1], 2, {}), ("latent24", 2, 5, [140, 64], 3, {}),
                                                ("latent4", 2, 6, [129, 0], 4, dict(page=128)),
                                                ("latent-two", 1, 4, [200], 3, {})])
def test_other_groups_of_heads(kind, B, R, lens, S, kw, monkeypatch):
    """Attention, weights (of more columns than the tensor memory takes, and of latent groups
    that are no run of 64: the CUDA cores), commit and eviction (of rows whose positions
    repeat, so that many are protected)."""
    monkeypatch.setitem(KINDS, kind, GROUPS[kind])
    monkeypatch.setitem(globals(), "plain_evict", plain_evict_any)
    for q8 in (True, False):
        s = Setup(kind, B, R, lens, extra=20, seed=40 + R, q8=q8, **kw)
        _weights_state(s, S)
        if q8:
            out, s.lse = s.attn()
            s.check_attn(out, s.lse)
        acc0, pos0, seen0 = s.acc.clone(), s.pos.clone(), s.seen.clone()
        _weights(s, S, 0.5)
        torch.cuda.synchronize()
        assert int(s.err) == 0
        _check_weights(s, acc0, pos0, seen0, 0.5)
        if q8:
            before = _write(s, s.kt, s.vt, None, (s.path, s.plength, S))
            _check_write(s, before, lambda b, h, w: (s.kt if w == "k" else s.vt)[b, s.paths[b], h].double())
            s.lens = s.plen.tolist()
        snap = _snapshot(s)
        _evict(s, 100, 2, 20)
        _check_evict(s, snap, 100, 2, 20)


@gpu
@pytest.mark.parametrize("kind,page", [("gqa", 0), ("narrow", 128), ("latent-few", 0)])
def test_commit_of_fp32_rows(kind, page):
    s = Setup(kind, 3, 40, [0, 60, 250], extra=17, page=page, dtype=torch.float32, seed=6)
    s.kt[1] *= 50.0
    s.kt[2, 3, 0, 5] = INF
    paths = [[0], [0] + list(range(2, 18)), [0, 3, 9]]
    rows = torch.tensor([p + [-1] * (17 - len(p)) for p in paths], dtype=torch.int32, device=DEV)
    length = torch.tensor([len(p) - 1 for p in paths], dtype=torch.int32, device=DEV)
    before = _write(s, s.kt, s.vt, None, (rows, length, 16))
    assert int(s.err) == 0
    _check_write(s, before, lambda b, h, w: (s.kt if w == "k" else s.vt)[b, paths[b], h].double())


@gpu
@pytest.mark.parametrize("kind,page", [("gqa", 128), ("narrow", 0), ("latent-few", 128)])
def test_a_row_is_the_same_wherever_it_stands_in_its_tree(kind, page):
    """The rows of a tree in another order (parents before children): each row's output is
    within the bounds in both."""
    s = Setup(kind, 2, 30, [700, 65], page=page, seed=20)
    s.check_attn(*s.attn())
    order = [0]
    while len(order) < 30:                # any row whose ancestors, in both trees, are there
        there = sum(1 << (r - 1) for r in order[1:])
        order.append(s.rnd.choice([r for r in range(1, 30) if r not in order and all(
            m[r] & ~there == 1 << (r - 1) for m in s.masks)]))
    assert order != sorted(order)
    place = {r: i for i, r in enumerate(order)}

    def moved(v):
        return sum(1 << (place[j] - 1) for j in range(1, 30) if v >> (j - 1) & 1)

    s.set_masks([[moved(m[r]) for r in order] for m in s.masks])
    at = torch.tensor(order, device=DEV)
    s.q, s.kt = s.q[:, at].contiguous(), s.kt[:, at].contiguous()
    s.vt = None if s.latent else s.vt[:, at].contiguous()
    s.check_attn(*s.attn())


# ------------------------------------------------------------ all together --

@gpu
@pytest.mark.parametrize("kind,page", [("gqa", 0), ("latent", 128), ("narrow", 0)])
def test_rounds_of_the_whole_set(kind, page):
    """Prefill, then rounds of verify, weights, commit and eviction, every call checked
    against its plain form on what the call before left; also with one captured round."""
    budget, S, R = 192, 4, 9
    s = Setup(kind, 2, R, [0, 0], extra=budget + 40 + S, page=page, seed=41)
    x = s.normal(2, 200, s.Hkv, s.dk)
    y = None if s.latent else s.normal(2, 200, s.Hkv, s.dv)
    n = torch.tensor([200, 150], dtype=torch.int32, device=DEV)
    before = _write(s, x, y, n)
    _check_write(s, before, lambda b, h, w: (x if w == "k" else y)[b, : int(n[b]), h].double())
    s.lens = n.tolist()
    _weights_state(s, S)
    s.acc.zero_()
    s.pos.copy_(torch.arange(s.cap, device=DEV).int().expand_as(s.pos))
    s.seen.copy_(n[:, None].expand_as(s.seen))
    ws = T.workspace(T.tsd_cache_evict_workspace_size(s.desc))
    for step in range(4):
        s.q.copy_(s.normal(*s.q.shape))
        s.kt.copy_(s.normal(*s.kt.shape))
        acc, pos, seen = s.acc, s.pos, s.seen
        _weights_state(s, S)
        s.acc, s.pos, s.seen = acc, pos, seen
        out, lse = s.attn()
        s.check_attn(out, lse)
        s.lse = lse
        acc0, pos0, seen0 = acc.clone(), pos.clone(), seen.clone()
        _weights(s, S, 0.9)
        torch.cuda.synchronize()
        _check_weights(s, acc0, pos0, seen0, 0.9)
        before = _write(s, s.kt, s.vt, None, (s.path, s.plength, S))
        _check_write(s, before, lambda b, h, w: (s.kt if w == "k" else s.vt)[b, s.paths[b], h].double())
        s.lens = [a + len(p) for a, p in zip(s.lens, s.paths)]
        snap = _snapshot(s)
        _evict(s, budget, 4, 32, ws)
        _check_evict(s, snap, budget, 4, 32)
        s.lens = [min(a, budget) for a in s.lens]
        assert int(s.err) == 0
