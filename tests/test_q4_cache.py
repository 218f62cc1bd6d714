"""The 4-bit KV cache (writes, commits, reads, tree attention) against plain 64-bit code.

The plain forms here work per request and head in float64.  Codes and scales have to be
equal; what the kernels compute is held to bounds derived beside each check.
"""

import ctypes
import math
import random

import pytest
import torch

import tree_speculative_decoding_tsd_gb300 as T

DEV = "cuda:0"
NAN, INF = float("nan"), float("inf")
G = T.TSD_Q4_GROUP
gpu = pytest.mark.gpu


# ------------------------------------------------------------ plain forms --

def unpack(x):
    """Packed codes [..][d / 2] (uint8) as whole numbers [..][d]."""
    word = sum(x[..., i::4].long() << (8 * i) for i in range(4))
    out = torch.empty(*word.shape, 8, dtype=torch.int64, device=x.device)
    for i in range(4):
        out[..., 2 * i] = (word >> (4 * i)) & 15
        out[..., 2 * i + 1] = (word >> (16 + 4 * i)) & 15
    return out.flatten(-2)


def quantise(x):
    """Rows [n][d] (float64, each an element of the input type) as codes [n][d], scales [n][d / 32]."""
    x = x.view(x.shape[0], -1, G)
    bad = ~x.isfinite().all(-1)
    y = torch.where(bad[..., None], torch.zeros_like(x), x)
    hi, lo = y.amax(-1), y.amin(-1)
    top = torch.where(hi >= -lo, hi, lo)
    s = (top / -8).float().bfloat16().double()        # (an element over 8 is exact in fp32)
    s[top.abs() < 2.0 ** -90] = 0
    inv = torch.where(s == 0, torch.zeros_like(s), 1 / s).float().double()
    c = (y * inv[..., None]).round().clamp(-8, 7).long() + 8
    c[bad | (s == 0)] = 8
    s[bad] = NAN
    return c.flatten(1), s


class Cache:
    """A contiguous or paged cache of one array (K or V): rows by (request, head)."""

    def __init__(self, x, s, table):
        self.x, self.s, self.table = x, s, table

    def pages(self, b):
        return [b] if self.table is None else self.table[b].tolist()

    def codes(self, b, h):
        return unpack(torch.cat([self.x[p, h] for p in self.pages(b)]))

    def scales(self, b, h):
        return torch.cat([self.s[p, h] for p in self.pages(b)]).double()

    def values(self, b, h):
        return (self.codes(b, h) - 8).double() * self.scales(b, h).repeat_interleave(G, 1)


def plain_attn(q, k, v, sees, scale):
    """q [n][d], k [m][d], v [m][d], sees [n][m] -> out, lse, weights, the weighted mean of
    |v| and the largest scale * sum |q_d k_d| (what the bounds need)."""
    s = (q @ k.T * scale).masked_fill(~sees, -INF)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[:, None])
    big = (q.abs() @ k.abs().T * scale).masked_fill(~sees, 0).amax(-1)
    return p @ v, lse, p @ v.abs(), big


# ----------------------------------------------------------------- inputs --

KINDS = {"gqa": (32, 8, 128), "narrow": (14, 2, 64), "one": (2, 2, 128), "wide": (16, 1, 128),
         "wide64": (24, 2, 64), "odd": (3, 1, 64), "eight": (64, 8, 128)}


class Setup:
    """Random cache, scratch pad, tree and lengths for one configuration."""

    def __init__(self, kind, B, R, lens, extra=8, dtype=torch.bfloat16, page=0, seed=0, spread=2):
        self.Hq, self.Hkv, self.d = KINDS[kind]
        self.B, self.R, self.dt, self.page = B, R, dtype, page
        self.g = torch.Generator(device=DEV).manual_seed(seed * 1000 + 11)
        self.rnd = random.Random(seed)
        self.lens = [lens[b % len(lens)] for b in range(B)]
        cap = max(max(self.lens) + extra, 1)
        if page:
            cap = -(-cap // page) * page
        self.cap = cap
        self.scale = float(torch.tensor(1 / math.sqrt(self.d), dtype=torch.float32))
        self.table = None
        lead, rows = (B, self.Hkv), cap
        if page:
            per = cap // page
            order = self.rnd.sample(range(B * per + 2), B * per)
            self.table = torch.tensor(order, dtype=torch.int32, device=DEV).view(B, per)
            lead, rows = (B * per + 2, self.Hkv), page
        self.lead, self.rows = lead, rows

        def codes():
            return torch.randint(0, 256, (*lead, rows, self.d // 2), generator=self.g, device=DEV,
                                 dtype=torch.uint8)

        def scales():
            shape = (*lead, rows, self.d // G)
            x = torch.rand(shape, generator=self.g, device=DEV) * 0.2 + 0.1
            e = torch.randint(-spread, 1, shape, generator=self.g, device=DEV)
            sign = torch.randint(0, 2, shape, generator=self.g, device=DEV) * 2 - 1
            return (x * sign * torch.exp2(e.float())).bfloat16()

        self.k, self.ks, self.v, self.vs = codes(), scales(), codes(), scales()
        self.plen = torch.tensor(self.lens, dtype=torch.int32, device=DEV)
        self.q = self.normal(B, R, self.Hq, self.d)
        self.kt, self.vt = self.normal(B, R, self.Hkv, self.d), self.normal(B, R, self.Hkv, self.d)
        masks = []
        for _ in range(B):
            m = [0]
            for r in range(1, R):
                m.append(m[self.rnd.randrange(max(0, r - 5), r)] | (1 << (r - 1)))
            masks.append(m)
        self.set_masks(masks)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.desc = T.make_desc(B, R, self.Hq, self.Hkv, self.d, self.d, cap, dtype, False, self.scale)
        self.paging = dict(page_table=self.table, page_size=page)

    def normal(self, *shape, std=1.0):
        return (torch.randn(*shape, generator=self.g, device=DEV) * std).to(self.dt)

    def set_masks(self, masks):
        self.masks = masks
        self.mask = torch.tensor([[v - (1 << 64) if v >> 63 else v for v in m] for m in masks],
                                 dtype=torch.int64, device=DEV)

    def cache(self, which):
        return Cache(self.k, self.ks, self.table) if which == "k" else Cache(self.v, self.vs, self.table)

    def arrays(self):
        return self.k, self.v, self.ks, self.vs

    def attn(self, stream=None):
        out = torch.full((self.B, self.R, self.Hq, self.d), 7.0, dtype=self.dt, device=DEV)
        lse = torch.full((self.B, self.R, self.Hq), 7.0, device=DEV)
        ws = T.workspace(T.tsd_verify_q4_workspace_size(self.desc))
        self.attn_into(out, lse, ws, stream)
        torch.cuda.synchronize()
        return out, lse

    def attn_into(self, out, lse, ws, stream=None):
        T.tsd_tree_verify_attn_q4(self.desc, self.q, *self.arrays(), self.plen, self.kt, self.vt,
                                  self.mask, out, lse, ws, self.err, stream, **self.paging)

    def sees(self, b):
        R = self.R
        return torch.tensor([[j == 0 or (i > 0 and self.masks[b][i] >> (j - 1) & 1 == 1)
                              for j in range(R)] for i in range(R)], device=DEV)

    def check_attn(self, out, lse, requests=None, heads=None):
        """Bounds.  fp32 arithmetic: a score is a sum of d products, in any order and possibly
        truncated, of codes 0..15 from which 8 times the sum of q is taken (whose terms are at
        most 15 / 8 of |c - 8| at their largest: S below takes 16 |s| for every |c - 8| |s|): off
        by at most (d + 16) 2^-23 S, S = scale sum |q| 16 |s|.  A probability is then off by that,
        relatively, plus 2^-20 for the exponential and the sums' last bits (n terms: n 2^-24
        more).
        bf16 inputs: tensor-core paths round keys (c - 8) s to fp16 (2^-12 of each: 2^-12 of
        scale sum |q k|), values (2^-12) and probabilities (2^-12), and a split's output (2^-12).
        fp16's smallest step is 2^-24: a key or value of a tile of at most 128 rows is held over
        2^E with |s| 2^-E < 1 for the tile's largest scale, as (c - 8) s 2^-E 2^-9 or more, so it is
        off by at most 2^-25 2^9 2^E = 2^-16 2^E, which is at most 2^-15 of the largest |s| of
        the tile; scratch rows of the last one by 2^-24 of the largest element.  A
        probability times 2^E is held relative to the largest such product met so far times
        2^-8 .. 1, in steps of 2^-24, off by at most 2^-25 2^8 of it: n 2^-17 of a weight 1 over
        the keys times ... - only products 2^-16 below the largest are touched; the sum of n of
        them is off by at most n 2^-25 top, top = the largest |v| of any tile times its weight,
        of which the denominator holds at least the weight.
        """
        g = self.Hq // self.Hkv
        f32 = self.dt == torch.float32
        for b in requests if requests is not None else range(self.B):
            P = min(self.lens[b], self.cap)
            sees = torch.cat([torch.ones(self.R, P, dtype=torch.bool, device=DEV), self.sees(b)], 1)
            live = sees.any(0)
            for h in heads if heads is not None else range(self.Hkv):
                ck, cv = self.cache("k"), self.cache("v")
                kt, vt = self.kt[b, :, h].double(), self.vt[b, :, h].double()
                k, v = torch.cat([ck.values(b, h)[:P], kt]), torch.cat([cv.values(b, h)[:P], vt])
                wide = torch.cat([16 * ck.scales(b, h)[:P].abs().repeat_interleave(G, 1), kt.abs()])
                k, v, wide = k[live], v[live], wide[live]
                seen = sees[:, live].repeat_interleave(g, 0)
                hs = slice(h * g, (h + 1) * g)
                q = self.q[b, :, hs].double().reshape(-1, self.d)
                o, l, A, S = plain_attn(q, k, v, seen, self.scale)
                n = k.shape[0]
                W = (q.abs() @ wide.T * self.scale).masked_fill(~seen, 0).nan_to_num(0).amax(-1)
                ds = (self.d + 16) * 2.0 ** -23 * W
                p16 = 0.0
                low_k = low_v = torch.zeros((), dtype=torch.float64, device=DEV)
                if not f32:
                    p16 = 3 * 2.0 ** -12
                    big_k = ck.scales(b, h)[:P].abs().nan_to_num(0)
                    big_v = cv.scales(b, h)[:P].abs().nan_to_num(0)
                    top_k = max(float(big_k.max()) if P else 0.0, float(kt[kt.isfinite()].abs().max()))
                    top_v = max(float(big_v.max()) if P else 0.0, float(vt[vt.isfinite()].abs().max()))
                    ds = ds + 2.0 ** -12 * S + 2.0 ** -15 * top_k * self.scale * q.abs().sum(-1)
                    low_v = 2.0 ** -15 * top_v + n * 2.0 ** -25 * 16 * top_v
                rel = 2 * ds + 2.0 ** -20 + n * 2.0 ** -24
                got = out[b, :, hs].double().reshape(-1, self.d)
                fine = o.isfinite().all(-1)
                low = 2.0 ** -24 if f32 else 2.0 ** -8
                tol = low * o.abs() + (rel + p16)[:, None] * A * 1.01 + low_v + 1e-37
                assert not got[fine].isnan().any()
                bad = ((got - o).abs() > tol)[fine]
                assert not bad.any(), (b, h, float(((got - o).abs() / tol)[fine].max()))
                assert not got[~fine].isfinite().all(-1).any()
                gl = lse[b, :, hs].double().reshape(-1)
                tl = rel + 2.0 ** -22 * l.abs() + 2.0 ** -20
                assert ((gl - l).abs() <= tl)[l.isfinite()].all(), (b, h)


# ------------------------------------------------- refusals (on the host) --

A, U, N = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10004), None


def _desc(**kw):
    base = dict(B=2, R=5, Hq=4, Hkv=2, dk=128, dv=128, cap=256, dtype=T.TSD_BF16, v_aliases_k=0,
                scale=0.088)
    base.update(kw)
    return T.tsd_attn_desc(**base)


def _calls(d, table=N, mp=0, ps=0, npg=0, x=A, y=A, S=3, rows=4, ws=1 << 40):
    r, pg, L = ctypes.byref(d), (table, mp, ps, npg), T.lib
    return {
        "write": lambda: L.tsd_cache_write_q4(r, rows, x, A, A, A, A, A, y, *pg, A, N, N),
        "commit": lambda: L.tsd_commit_path_q4(r, S, x, A, A, A, A, A, A, y, *pg, A, N, N),
        "read": lambda: L.tsd_cache_read_q4(r, rows, x, A, A, A, *pg, A, A, A, A, y, N, N),
        "attn": lambda: L.tsd_tree_verify_attn_q4(r, x, A, A, A, y, *pg, A, A, A, A, A, A, A, ws, N, N)}


ALL = list(_calls(_desc()))


@pytest.mark.parametrize("name", ALL)
@pytest.mark.parametrize("kw", [dict(B=0), dict(B=65536), dict(R=0), dict(R=66), dict(Hq=3),
                                dict(Hkv=0), dict(dk=96, dv=96), dict(dk=128, dv=64), dict(dtype=7),
                                dict(cap=0), dict(v_aliases_k=1)])
def test_calls_reject_bad_descriptors(name, kw):
    assert _calls(_desc(**kw))[name]() == T.TSD_ERR_INVALID_ARG


@pytest.mark.parametrize("name", ALL)
def test_calls_do_not_take_latent_heads(name):
    d = _desc(dk=576, dv=512, v_aliases_k=1)
    assert _calls(d)[name]() == T.TSD_ERR_UNSUPPORTED
    assert T.tsd_verify_q4_workspace_size(d) == 0


@pytest.mark.parametrize("name", ALL)
@pytest.mark.parametrize("kw", [dict(x=N), dict(x=U), dict(y=N), dict(y=U), dict(ps=-1),
                                dict(ps=64, table=A, mp=4, npg=8), dict(ps=128, table=A, mp=3, npg=8),
                                dict(ps=128, table=N, mp=2, npg=8), dict(ps=128, table=U, mp=2, npg=8),
                                dict(ps=128, table=A, mp=2)])
def test_calls_reject_bad_pointers_and_pages(name, kw):
    assert _calls(_desc(), **kw)[name]() == T.TSD_ERR_INVALID_ARG


@pytest.mark.parametrize("name,kw", [("commit", dict(S=0)), ("commit", dict(S=17)), ("write", dict(rows=0)),
                                     ("read", dict(rows=0))])
def test_calls_reject_bad_numbers(name, kw):
    assert _calls(_desc(), **kw)[name]() == T.TSD_ERR_INVALID_ARG


@pytest.mark.parametrize("scale", [0.0, -1.0, NAN, INF])
def test_attention_rejects_bad_scales(scale):
    assert _calls(_desc(scale=scale))["attn"]() == T.TSD_ERR_INVALID_ARG


def test_attention_rejects_a_short_workspace():
    d = _desc(B=1, R=9, Hq=8, Hkv=1, cap=8192)
    need = T.tsd_verify_q4_workspace_size(d)
    assert need > 0
    assert _calls(d, ws=need - 1)["attn"]() == T.TSD_ERR_INVALID_ARG


@gpu
def test_binding_rejects_types_shapes_and_pages():
    s = Setup("one", 2, 3, [40])
    out = torch.empty(2, 3, 2, 128, dtype=s.dt, device=DEV)
    lse = torch.empty(2, 3, 2, device=DEV)
    ws = T.workspace(T.tsd_verify_q4_workspace_size(s.desc))

    def call(**kw):
        a = dict(q=s.q, kq=s.k, vq=s.v, kscale=s.ks, vscale=s.vs, prefix_len=s.plen, ktree=s.kt,
                 vtree=s.vt, mask=s.mask, out=out, lse=lse, ws=ws)
        a.update(kw)
        T.tsd_tree_verify_attn_q4(s.desc, **a)

    call()
    for kw in (dict(q=s.q.float()), dict(kq=s.k.float()), dict(kscale=s.ks.float()),
               dict(prefix_len=s.plen.long())):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(q=s.q[:, :2]), dict(kq=s.k[:, :, :-1]), dict(vscale=s.vs[..., :2]),
               dict(vscale=s.vs.cpu()), dict(lse=lse[:, :, :1]), dict(page_size=128),
               dict(kq=s.k.transpose(0, 1)), dict(ws=ws.cpu())):
        with pytest.raises(ValueError):
            call(**kw)
    torch.cuda.synchronize()


# ---------------------------------------------------------- writes, reads --

def _append(s, new, vnew, n, commit=None):
    before = [t.clone() for t in s.arrays()]
    p0 = s.plen.clone()
    if commit is None:
        T.tsd_cache_write_q4(s.desc, new, vnew, n, *s.arrays(), s.plen, s.err, **s.paging)
    else:
        T.tsd_commit_path_q4(s.desc, commit.shape[1] - 1, new, vnew, commit, n, *s.arrays(), s.plen,
                             s.err, **s.paging)
    torch.cuda.synchronize()
    return before, p0


def _check_append(s, before, p0, rows_of):
    """rows_of(b) -> (K rows, V rows) [n][Hkv][d] in order, or None for a skipped request.
    Every array against the plain form, whole."""
    want = [t.clone() for t in before]
    for b in range(s.B):
        rows = rows_of(b)
        P = int(p0[b])
        if rows is None:
            assert int(s.plen[b]) == P
            continue
        assert int(s.plen[b]) == P + rows[0].shape[0]
        for part in range(2):
            for i in range(rows[part].shape[0]):
                c, f = quantise(rows[part][i].double())
                pg, at = (b, P + i) if s.table is None else \
                    (int(s.table[b, (P + i) // s.page]), (P + i) % s.page)
                got = unpack((s.k, s.v)[part][pg, :, at])
                assert torch.equal(got, c), (b, part, i)
                assert torch.equal((s.ks, s.vs)[part][pg, :, at].double().nan_to_num(9.0), f.nan_to_num(9.0))
                want[part][pg, :, at] = (s.k, s.v)[part][pg, :, at]
                want[2 + part][pg, :, at] = (s.ks, s.vs)[part][pg, :, at]
    for x, y in zip(s.arrays(), want):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@gpu
@pytest.mark.parametrize("kind,dtype,page", [("gqa", torch.bfloat16, 0), ("narrow", torch.float32, 128),
                                             ("one", torch.float32, 0), ("odd", torch.bfloat16, 256)])
@pytest.mark.parametrize("Tn", [1, 17, 18, 67, 131])
def test_write_appends_rows_of_every_length(kind, dtype, page, Tn):
    lens = [0, 1, 63, 127, 128, 130, 255]
    s = Setup(kind, 7, 1, lens, extra=Tn, dtype=dtype, page=page, seed=Tn)
    x, y = s.normal(7, Tn, s.Hkv, s.d), s.normal(7, Tn, s.Hkv, s.d, std=3)
    n = torch.tensor([Tn, 0, Tn, 1, max(Tn - 1, 0), Tn // 2, Tn], dtype=torch.int32, device=DEV)
    before, p0 = _append(s, x, y, n)
    _check_append(s, before, p0, lambda b: (x[b, : int(n[b])], y[b, : int(n[b])]))
    assert int(s.err) == 0


@gpu
@pytest.mark.parametrize("kind,dtype,page", [("gqa", torch.bfloat16, 0), ("narrow", torch.bfloat16, 128),
                                             ("wide", torch.float32, 256)])
def test_commit_writes_the_accepted_rows(kind, dtype, page):
    s = Setup(kind, 4, 20, [0, 60, 120, 250], extra=20, dtype=dtype, page=page, seed=3)
    S = 9
    path = torch.full((4, S + 1), -1, dtype=torch.int32)
    lens = [0, 9, 4, 7]
    for b, L in enumerate(lens):
        path[b, : L + 1] = torch.tensor([0] + sorted(s.rnd.sample(range(1, 20), L)))
    L = torch.tensor(lens, dtype=torch.int32, device=DEV)
    before, p0 = _append(s, s.kt, s.vt, L, path.to(DEV))
    _check_append(s, before, p0, lambda b: (s.kt[b, path[b, : lens[b] + 1].long()],
                                            s.vt[b, path[b, : lens[b] + 1].long()]))
    assert int(s.err) == 0


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("Tn", [4, 40])
def test_write_takes_values_at_the_ends_of_the_format(dtype, Tn):
    s = Setup("one", 1, 1, [5], extra=Tn, dtype=dtype)
    x = s.normal(1, Tn, 2, 128)
    top = float(torch.finfo(dtype).max)
    r = x[0, :, 0]
    r[0, :32] = 0                                  # zeros
    r[0, 32:64] = torch.where(r[0, 32:64] > 0, 2.0 ** -91, -2.0 ** -91)
    r[0, 64:96] = 2.0 ** -90                       # the smallest group that is held
    r[0, 96:] = -0.0
    r[1, :32] = top
    r[1, 32:64] *= 1e38
    r[1, 64] = INF                                 # NaN groups, beside others
    r[1, 100] = NAN
    r[2, :32] = 3.0                                # ties of the largest magnitude, both signs
    r[2, 5] = -3.0
    r[2, 32:64] = torch.arange(32, device=DEV) / 4 - 4.0    # ties between two codes
    r[2, 64] = -INF
    r[2, 96:] = torch.arange(32, device=DEV).to(dtype) / -4 + 4.0
    r[3] *= 2.0 ** -88
    y = s.normal(1, Tn, 2, 128)
    n = torch.tensor([Tn], dtype=torch.int32, device=DEV)
    before, p0 = _append(s, x, y, n)
    _check_append(s, before, p0, lambda b: (x[b], y[b]))
    assert s.ks[0, 0, 6, 2].isnan() and s.ks[0, 0, 6, 3].isnan() and not s.ks[0, 0, 6, :2].isnan().any()


@gpu
@pytest.mark.parametrize("Tn", [6, 30])
def test_append_skips_requests_with_errors(Tn):
    s = Setup("gqa", 5, 9, [100, 120, 30, 128, 3], extra=0, page=128, seed=2)
    cap = s.cap
    x, y = s.normal(5, Tn, s.Hkv, s.d), s.normal(5, Tn, s.Hkv, s.d)
    s.plen[3] = cap - Tn + 1                        # passes the cache
    s.table[2, 0] = s.k.shape[0]                    # a page outside the pool
    for n in ([Tn, -1, Tn, Tn, Tn + 1], [0, Tn, -5, Tn, 2]):
        s.err.zero_()
        before, p0 = _append(s, x, y, torch.tensor(n, dtype=torch.int32, device=DEV))
        assert int(s.err) != 0
        bad = [b for b in range(5) if not 0 <= n[b] <= Tn or b == 2 or int(p0[b]) + n[b] > cap]
        table = s.table
        s.table = torch.where(s.table >= s.k.shape[0], 0, s.table)
        _check_append(s, before, p0, lambda b: None if b in bad else (x[b, : n[b]], y[b, : n[b]]))
        s.table = table
    path = torch.tensor([[0, 3, 9, -1], [0, 1, 2, 3], [0, -1, -1, -1], [0, 1, 2, 3], [0, 5, -1, -1]],
                        dtype=torch.int32, device=DEV)
    L = torch.tensor([2, 4, 0, 3, 1], dtype=torch.int32, device=DEV)
    s.plen[3] = cap - 3
    s.err.zero_()
    before, p0 = _append(s, s.kt, s.vt, L, path)
    s.table[2, 0] = 0
    _check_append(s, before, p0, lambda b: (s.kt[b, [0, 5]], s.vt[b, [0, 5]]) if b == 4 else None)
    assert int(s.err) & T.TSD_DEV_ERR_MASK in (T.TSD_DEV_ERR_BAD_TREE, T.TSD_DEV_ERR_CAPACITY,
                                               T.TSD_DEV_ERR_BAD_PAGE)


def _read(s, first, count, Tn):
    out = [torch.full((s.B, Tn, s.Hkv, s.d), 7.0, dtype=s.dt, device=DEV) for _ in range(2)]
    i32 = dict(dtype=torch.int32, device=DEV)
    T.tsd_cache_read_q4(s.desc, *s.arrays(), s.plen, torch.tensor(first, **i32),
                        torch.tensor(count, **i32), *out, s.err, **s.paging)
    torch.cuda.synchronize()
    return out


@gpu
@pytest.mark.parametrize("kind,dtype,page", [("gqa", torch.bfloat16, 0), ("narrow", torch.float32, 128),
                                             ("one", torch.float32, 0), ("odd", torch.bfloat16, 256)])
def test_read_gives_the_values(kind, dtype, page):
    s = Setup(kind, 5, 1, [0, 1, 130, 255, 300], dtype=dtype, page=page, seed=4)
    first, count = [0, 0, 129, 0, 37], [0, 1, 1, 255, 200]
    s.ks[tuple(0 for _ in s.ks.shape)] = NAN
    for Tn in (255, 256, 300):
        out = _read(s, first, count, Tn)
        for b in range(5):
            n = count[b]
            assert (out[0][b, n:] == 7).all() and (out[1][b, n:] == 7).all()
            for h in range(s.Hkv):
                for which, got in zip("kv", out):
                    want = s.cache(which).values(b, h)[first[b]: first[b] + n].to(dtype)
                    assert torch.equal(got[b, :n, h].nan_to_num(9.5), want.nan_to_num(9.5)), (b, h, which)
    assert int(s.err) == 0


@gpu
@pytest.mark.parametrize("bad", [(-1, 3), (5, -1), (5, 33), (90, 11), (2 ** 31 - 1, 2), (0, 2 ** 31 - 1)])
def test_read_skips_requests_with_errors(bad):
    s = Setup("one", 3, 1, [100], seed=5)
    out = _read(s, [0, bad[0], 70], [32, bad[1], 30], 32)
    assert int(s.err) == T.TSD_DEV_ERR_CAPACITY | 1
    assert (out[0][1] == 7).all() and (out[1][1] == 7).all()
    assert torch.equal(out[0][2, :30, 1].double(), s.cache("k").values(2, 1)[70:100].to(s.dt).double())


@gpu
def test_read_reports_pages_outside_the_pool_that_it_needs():
    s = Setup("one", 2, 1, [300], page=128, seed=6)
    s.table[0, 0] = -1
    s.table[1, 2] = s.k.shape[0]
    out = _read(s, [128, 0], [100, 256], 256)
    assert int(s.err) == 0 and not (out[1] == 7).all()
    out = _read(s, [100, 0], [100, 256], 256)
    assert int(s.err) == T.TSD_DEV_ERR_BAD_PAGE | 0 and (out[0][0] == 7).all()
    s.plen[1] = s.cap + 1
    s.err.zero_()
    _read(s, [128, 0], [100, 256], 256)
    assert int(s.err) == T.TSD_DEV_ERR_CAPACITY | 1


@gpu
@pytest.mark.parametrize("kind", ["gqa", "narrow"])
def test_rows_written_are_read_back(kind):
    """With a the group's largest magnitude, s = a / 8 but for its rounding, 2^-8 of it.  An
    element next to a on the side where the codes end at 7 is held as 7 s: off by at most
    a - 7 a / 8 (1 - 2^-8) = a / 8 (1 + 7 2^-8).  The others are off by half a step, or, at the
    codes' end 8 s, by 2^-8 a: less than that."""
    s = Setup(kind, 2, 1, [7], extra=100, dtype=torch.float32)
    x, y = s.normal(2, 100, s.Hkv, s.d), s.normal(2, 100, s.Hkv, s.d)
    _append(s, x, y, torch.tensor([100, 50], dtype=torch.int32, device=DEV))
    out = _read(s, [7, 7], [100, 50], 100)
    for b, n in ((0, 100), (1, 50)):
        for got, new in zip(out, (x, y)):
            g, w = (t[b, :n].double().view(n, s.Hkv, -1, G) for t in (got, new))
            big = w.abs().amax(-1, keepdim=True)
            assert ((g - w).abs() <= big / 8 * (1 + 7 * 2.0 ** -8) + 1e-30).all()
            assert ((g - w).square().mean().sqrt() < 0.12 * w.square().mean().sqrt())


@gpu
def test_writes_and_reads_on_streams_and_in_graphs():
    """A write and the read of its rows, on two streams at once, then captured and replayed."""
    sets = [Setup("gqa", 3, 1, [5, 0, 260], extra=400, page=128, seed=50),
            Setup("narrow", 2, 1, [129, 70], extra=400, dtype=torch.float32, seed=51)]
    Tn = 37
    streams = [torch.cuda.Stream() for _ in sets]
    work = []
    for s in sets:
        n = torch.tensor([Tn, 9, 20][:s.B], dtype=torch.int32, device=DEV)
        work.append((s.normal(s.B, Tn, s.Hkv, s.d), s.normal(s.B, Tn, s.Hkv, s.d), n, torch.empty_like(n),
                     [torch.zeros(s.B, Tn, s.Hkv, s.d, dtype=s.dt, device=DEV) for _ in range(2)]))

    def turn(s, x, y, n, first, out, stream=None):
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            first.copy_(s.plen)
            T.tsd_cache_write_q4(s.desc, x, y, n, *s.arrays(), s.plen, s.err, stream, **s.paging)
            T.tsd_cache_read_q4(s.desc, *s.arrays(), s.plen, first, n, *out, s.err, stream, **s.paging)

    def check(s, x, y, n, first, out):
        assert int(s.err) == 0
        for b in range(s.B):
            for got, new in zip(out, (x, y)):
                c, f = quantise(new[b, :int(n[b])].double())
                want = ((c - 8).double() * f.repeat_interleave(G, -1)).to(s.dt)
                assert torch.equal(got[b, :int(n[b])], want.view(-1, s.Hkv, s.d))

    torch.cuda.synchronize()
    for _ in range(4):
        for s, w, st in zip(sets, work, streams):
            turn(s, *w, st)
    torch.cuda.synchronize()
    for s, w in zip(sets, work):
        check(s, *w)
        assert s.plen.tolist() == [p + 4 * int(k) for p, k in zip(s.lens, w[2])]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            turn(s, *w)
        for _ in range(3):
            w[0].copy_(s.normal(*w[0].shape))
            w[1].copy_(s.normal(*w[1].shape))
            graph.replay()
            torch.cuda.synchronize()
            check(s, *w)
        assert s.plen.tolist() == [p + 7 * int(k) for p, k in zip(s.lens, w[2])]


# -------------------------------------------------------------- attention --

ATTN = [("gqa", 3, 1, [2048, 700, 5], {}), ("gqa", 2, 1, [4100], {}), ("gqa", 2, 4, [1300, 129], {}),
        ("gqa", 1, 17, [2048], {}), ("gqa", 4, 33, [1024, 257, 130, 900], dict(page=128)),
        ("gqa", 2, 65, [3000, 128], {}), ("narrow", 3, 1, [1999, 64, 2], {}),
        ("narrow", 2, 9, [700, 1025], dict(page=256)), ("narrow", 2, 33, [600, 50], {}),
        ("one", 5, 1, [127, 128, 129, 1, 3], {}), ("one", 2, 16, [500], {}), ("one", 2, 17, [500], {}),
        ("wide", 2, 1, [5000, 33], dict(page=128)), ("wide", 2, 8, [900], {}), ("wide", 1, 65, [400], {}),
        ("wide64", 2, 1, [640, 15], {}), ("wide64", 3, 11, [640, 15, 16], {}), ("odd", 3, 5, [77, 0, 401], {}),
        ("odd", 2, 6, [333], {}), ("gqa", 33, 2, [65, 200, 511, 1, 90], dict(page=128)),
        ("gqa", 70, 1, [100, 40], {}),
        ("gqa", 2, 5, [900, 100], dict(dtype=torch.float32)), ("narrow", 2, 3, [500, 64], dict(dtype=torch.float32)),
        ("wide", 2, 1, [900, 100], dict(dtype=torch.float32, page=128))]


@gpu
@pytest.mark.parametrize("kind,B,R,lens,kw", ATTN)
def test_attention_matches_plain(kind, B, R, lens, kw):
    s = Setup(kind, B, R, lens, seed=len(lens) + R, **kw)
    s.check_attn(*s.attn())
    assert int(s.err) == 0


@gpu
@pytest.mark.parametrize("kind,B,R,lens,page", [
    ("gqa", 3, 33, [700, 129, 64], 128), ("gqa", 1, 65, [1000], 0), ("narrow", 2, 65, [333, 1], 0),
    ("narrow", 2, 9, [2000, 65], 256), ("wide", 1, 65, [500], 128), ("wide", 2, 2, [63, 900], 0),
    ("one", 2, 65, [300, 0], 0), ("one", 2, 17, [130, 64], 128), ("one", 3, 1, [5000, 1, 64], 0),
    ("odd", 2, 6, [333, 20], 0), ("wide64", 2, 4, [640, 15], 0), ("gqa", 60, 1, [65, 200, 511, 1, 90], 128)])
def test_attention_of_fp32_matches_plain(kind, B, R, lens, page):
    """In the bounds of check_attn, q and scratch keys off by 2^-22 each are four of the 16 spare
    steps of 2^-23 of a score; the exponential's 2^-22, a weight's 2^-23 and a scratch value's
    2^-22 lie within 2^-20."""
    s = Setup(kind, B, R, lens, page=page, dtype=torch.float32, seed=60 + R)
    s.check_attn(*s.attn())
    assert int(s.err) == 0


@gpu
@pytest.mark.parametrize("kind,R,lens", [("gqa", 5, [700, 333]), ("gqa", 1, [8000, 5000]), ("gqa", 20, [900]),
                                         ("narrow", 30, [4000, 333]), ("one", 9, [6000])])
def test_attention_of_fp32_is_as_good_as_plain_fp32(kind, R, lens):
    """The root mean square of the error, against that of the same sums in PyTorch's fp32, whose
    roundings are as many: no more than twice it."""
    s = Setup(kind, len(lens), R, lens, dtype=torch.float32, seed=68)
    out, _ = s.attn()
    got = plain = 0.0
    for b, P in enumerate(s.lens):
        for h in range(s.Hkv):
            k = torch.cat([s.cache("k").values(b, h)[:P], s.kt[b, :, h].double()])
            v = torch.cat([s.cache("v").values(b, h)[:P], s.vt[b, :, h].double()])
            g = s.Hq // s.Hkv
            sees = torch.cat([torch.ones(R, P, dtype=torch.bool, device=DEV), s.sees(b)], 1).repeat_interleave(g, 0)
            q = s.q[b, :, h * g:(h + 1) * g].reshape(-1, s.d)
            o = plain_attn(q.double(), k, v, sees, s.scale)[0]
            p = torch.softmax((q @ k.float().T * s.scale).masked_fill(~sees, -INF), -1) @ v.float()
            got += float((out[b, :, h * g:(h + 1) * g].double().reshape(-1, s.d) - o).square().sum())
            plain += float((p.double() - o).square().sum())
    assert got <= 4 * plain


@gpu
@pytest.mark.parametrize("kind,R", [("gqa", 1), ("gqa", 5), ("gqa", 17), ("narrow", 4), ("one", 65)])
@pytest.mark.parametrize("power", [-112, -70, -40, 40, 80])
def test_attention_of_very_small_and_large_fp32_values(kind, R, power):
    s = Setup(kind, 2, R, [700, 40], dtype=torch.float32, seed=61)
    f = 2.0 ** power
    if power > -100:
        s.vs *= f
        s.vt *= f
        s.check_attn(*s.attn())
    s = Setup(kind, 2, R, [700, 40], dtype=torch.float32, seed=62)
    s.ks /= f
    s.kt /= f
    s.q *= f
    s.check_attn(*s.attn())
    s = Setup(kind, 2, R, [700, 40], dtype=torch.float32, seed=63, spread=40)
    s.check_attn(*s.attn())


@gpu
@pytest.mark.parametrize("kind,R", [("gqa", 1), ("gqa", 4), ("gqa", 20), ("narrow", 2), ("narrow", 12)])
def test_attention_of_fp32_with_late_large_scores(kind, R):
    s = Setup(kind, 2, R, [1500, 333], dtype=torch.float32, seed=64)
    ramp = torch.exp2(torch.linspace(-3, 5, s.rows, device=DEV)).bfloat16()
    s.ks *= ramp[:, None]
    s.vs *= ramp.flip(0)[:, None]
    s.check_attn(*s.attn())


@gpu
@pytest.mark.parametrize("kind,R,page", [("gqa", 1, 0), ("gqa", 4, 128), ("narrow", 9, 0), ("gqa", 20, 128),
                                         ("one", 65, 0)])
def test_attention_of_fp32_leaves_out_what_no_row_sees(kind, R, page):
    s = Setup(kind, 4, R, [0, 100, 129, 240], page=page, dtype=torch.float32, seed=65)
    for b in range(4):
        for p in range(s.lens[b], s.cap):
            pg, at = (b, p) if s.table is None else (int(s.table[b, p // page]), p % page)
            s.ks[pg, :, at], s.vs[pg, :, at] = NAN, INF
    if R > 2:
        s.set_masks([[m & ~1 for m in row] for row in s.masks])
        s.kt[:, 1], s.vt[:, 1] = NAN, INF
    out, lse = s.attn()
    assert out.isfinite().all() and lse.isfinite().all()
    s.check_attn(out, lse)


@gpu
@pytest.mark.parametrize("R", [1, 5, 20])
def test_attention_of_fp32_reports_pages_and_replays(R):
    s = Setup("gqa", 3, R, [300, 500, 200], page=128, dtype=torch.float32, seed=66)
    want, _ = s.attn()
    good = s.table.clone()
    s.table[1, 2] = s.k.shape[0]
    s.table[0, 3] = -1                              # not needed
    out, lse = s.attn()
    assert int(s.err) == T.TSD_DEV_ERR_BAD_PAGE | 1
    s.check_attn(out, lse, requests=[0, 2])
    s.table.copy_(good)
    s.err.zero_()
    ws = T.workspace(T.tsd_verify_q4_workspace_size(s.desc))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.attn_into(out, lse, ws)
    out.fill_(7)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and int(s.err) == 0
    s.plen.copy_(torch.tensor([128, 0, 1], dtype=torch.int32))
    s.lens = [128, 0, 1]
    graph.replay()
    torch.cuda.synchronize()
    s.check_attn(out, lse)


BESIDE = [("gqa", 32, 33, [300, 0, 1000, 129, 1, 64, 127, 700, 2000], 2100, 0),
          ("gqa", 16, 65, [1000, 129, 0, 300], 3200, 128), ("gqa", 2, 33, [32700, 400], 60, 128),
          ("gqa", 4, 65, [20000, 0, 129, 5], 100, 0), ("wide", 128, 17, [400, 64, 0, 129], 3800, 128)]


@gpu
@pytest.mark.parametrize("kind,B,R,lens,extra,page", BESIDE)
def test_attention_with_the_last_row_on_its_own(kind, B, R, lens, extra, page):
    """Large batches and long caches, of trees that leave 4 or 8 packed rows behind groups of 128."""
    s = Setup(kind, B, R, lens, extra=extra, page=page, seed=70)
    out, lse = s.attn()
    assert int(s.err) == 0
    s.check_attn(out, lse, requests=sorted({0, 1, min(3, B - 1), B // 2, B - 1}), heads=[0, s.Hkv - 1])
    assert not (out == 7).all(-1).any() and not (lse == 7).any()
    s.kt[0, R - 1], s.mask[0, 5] = NAN, 0           # seen by the last row alone, and no longer by row 5
    s.masks[0] = [m & ~(1 << (R - 2)) for m in s.masks[0][:-1]] + s.masks[0][-1:]
    s.masks[0][5] = 0
    s.set_masks(s.masks)
    again, _ = s.attn()
    assert again[0, R - 1].isnan().all() and again[0, :R - 1].isfinite().all()
    assert torch.equal(again[1:], out[1:])


@gpu
@pytest.mark.parametrize("kind,B,R,lens,extra,page", BESIDE[:2])
def test_attention_with_the_last_row_on_its_own_in_a_round(kind, B, R, lens, extra, page):
    """Between an append that it waits for and one that waits for it, in a graph."""
    s = Setup(kind, B, R, lens, extra=extra, page=page, seed=71)
    x, y = s.normal(B, 20, s.Hkv, s.d), s.normal(B, 20, s.Hkv, s.d)
    n = torch.tensor([(3 * b) % 21 for b in range(B)], dtype=torch.int32, device=DEV)
    out, lse = torch.empty_like(s.q), torch.empty(B, R, s.Hq, device=DEV)
    ws = T.workspace(T.tsd_verify_q4_workspace_size(s.desc))
    kept = [t.clone() for t in s.arrays()] + [s.plen.clone()]

    def turn():
        T.tsd_cache_write_q4(s.desc, x, y, n, *s.arrays(), s.plen, s.err, **s.paging)
        s.attn_into(out, lse, ws)
        T.tsd_cache_write_q4(s.desc, y, x, n, *s.arrays(), s.plen, s.err, **s.paging)

    def restore():
        for t, old in zip((*s.arrays(), s.plen), kept):
            t.copy_(old)
        out.fill_(7)
        torch.cuda.synchronize()

    T.tsd_cache_write_q4(s.desc, x, y, n, *s.arrays(), s.plen, s.err, **s.paging)
    torch.cuda.synchronize()
    s.attn_into(out, lse, ws)
    torch.cuda.synchronize()
    want = out.clone()
    restore()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        turn()
    for _ in range(10):
        restore()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        restore()
        turn()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert int(s.err) == 0


@gpu
@pytest.mark.parametrize("kind,B,R,page", [("gqa", 200, 1, 0), ("gqa", 150, 4, 128), ("gqa", 64, 4, 0),
                                           ("gqa", 64, 1, 128), ("narrow", 400, 1, 128), ("narrow", 400, 2, 0),
                                           ("gqa", 150, 33, 128)])
def test_attention_of_many_short_requests(kind, B, R, page):
    s = Setup(kind, B, R, [300, 0, 127, 1, 260, 33, 64, 129, 17], page=page, seed=40)
    some = [0, 1, 2, 3, 4, 5, 6, 7, 8, B // 2, B - 2, B - 1]
    s.check_attn(*s.attn(), requests=some, heads=[0, s.Hkv - 1])
    assert int(s.err) == 0


@gpu
@pytest.mark.parametrize("kind,R", [("gqa", 1), ("gqa", 4), ("gqa", 20), ("narrow", 2), ("narrow", 30)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attention_of_empty_and_tiny_prefixes(kind, R, dtype):
    s = Setup(kind, 7, R, [0, 1, 2, 15, 16, 17, 31], dtype=dtype, seed=8)
    s.check_attn(*s.attn())
    assert int(s.err) == 0


@gpu
@pytest.mark.parametrize("kind,R,page", [("gqa", 1, 0), ("gqa", 4, 128), ("narrow", 2, 0), ("gqa", 20, 128),
                                         ("narrow", 20, 0)])
def test_attention_leaves_out_what_no_row_sees(kind, R, page):
    """NaN scales and any codes behind the prefix, and NaN in scratch rows that nobody sees."""
    s = Setup(kind, 4, R, [0, 100, 129, 240], page=page, seed=21)
    for b in range(4):
        for p in range(s.lens[b], s.cap):
            pg, at = (b, p) if s.table is None else (int(s.table[b, p // page]), p % page)
            s.ks[pg, :, at], s.vs[pg, :, at] = NAN, INF
    if R > 2:
        masks = [[m & ~1 for m in row] for row in s.masks]      # row 1 is seen by no row
        s.set_masks(masks)
        s.kt[:, 1], s.vt[:, 1] = NAN, INF
    out, lse = s.attn()
    assert out.isfinite().all() and lse.isfinite().all()
    s.check_attn(out, lse)


@gpu
@pytest.mark.parametrize("kind,R,dtype", [("gqa", 1, torch.bfloat16), ("gqa", 3, torch.bfloat16),
                                          ("narrow", 2, torch.bfloat16), ("gqa", 20, torch.bfloat16),
                                          ("gqa", 3, torch.float32)])
def test_attention_keeps_nan_to_the_rows_that_see_it(kind, R, dtype):
    s = Setup(kind, 3, R, [200, 300, 50], dtype=dtype, seed=22)
    s.ks[0, 1, 77, 0] = NAN                         # a key: every row of its head
    s.vs[0, 0, 5, 1] = NAN                          # a value: its group's dims
    s.q[1, 0, 3, 9] = NAN
    s.q[1, R - 1, 5, 0] = INF
    if R > 1:
        s.kt[2, R - 1, 0, 3] = NAN
    out, lse = s.attn()
    g = s.Hq // s.Hkv
    assert out[0, :, g: 2 * g].isnan().all() and lse[0, :, g: 2 * g].isnan().all()
    assert out[0, :, :g, 32:64].isnan().all() and out[0, :, :g, :32].isfinite().all()
    assert lse[0, :, :g].isfinite().all()
    assert out[1, 0, 3].isnan().all() and out[1, R - 1, 5].isnan().all()
    sees = s.sees(2)[:, R - 1] if R > 1 else torch.zeros(1, dtype=torch.bool, device=DEV)
    assert out[2, sees][:, :g].isnan().all() and out[2, ~sees].isfinite().all()
    s.check_attn(out, lse)


@gpu
@pytest.mark.parametrize("kind,R", [("gqa", 1), ("gqa", 4), ("gqa", 20), ("narrow", 2), ("narrow", 12)])
def test_attention_with_late_large_scores(kind, R):
    """Scores that grow along the cache by far more than the running bound's headroom."""
    s = Setup(kind, 2, R, [1500, 333], seed=23)
    ramp = torch.exp2(torch.linspace(-3, 5, s.rows, device=DEV)).bfloat16()
    s.ks *= ramp[:, None]
    s.vs *= ramp.flip(0)[:, None]
    s.check_attn(*s.attn())


@gpu
@pytest.mark.parametrize("kind,R", [("gqa", 1), ("gqa", 3), ("gqa", 20), ("narrow", 2), ("narrow", 12)])
@pytest.mark.parametrize("power", [-80, -40, 40, 80])
def test_attention_of_very_small_and_large_values(kind, R, power):
    s = Setup(kind, 2, R, [700, 40], seed=24)
    f = 2.0 ** power
    s.vs *= f
    s.vt *= f
    s.check_attn(*s.attn())
    s = Setup(kind, 2, R, [700, 40], seed=25)
    s.ks *= f
    s.kt *= f
    s.q /= f
    s.check_attn(*s.attn())


@gpu
def test_attention_of_zero_rows():
    for R in (1, 20):
        s = Setup("gqa", 2, R, [300, 20], seed=26)
        s.vs[:, :, 10:200] = 0
        s.ks[:, 0] = 0
        s.q[0, 0, 0] = 0
        s.check_attn(*s.attn())
        s.vs.zero_()
        s.vt.zero_()
        out, lse = s.attn()
        assert (out == 0).all() and lse.isfinite().all()


@gpu
@pytest.mark.parametrize("R", [1, 4, 20])
def test_attention_of_very_large_rows_of_q(R):
    s = Setup("gqa", 2, R, [200, 30], seed=27)
    s.q[0, R - 1, 2, 7] = 2.0 ** 117                # a row that one key of its own settles
    s.q[1, 0, 1] *= 2.0 ** 85
    s.q[1, R - 1, 5] *= 2.0 ** 124
    s.ks[1] *= 2.0 ** -85
    s.kt[1] *= 2.0 ** -85
    out, lse = s.attn()
    assert out.isfinite().all() and lse.isfinite().all()
    s.check_attn(out, lse, requests=[1], heads=[0])


@gpu
@pytest.mark.parametrize("kind,R", [("gqa", 1), ("gqa", 4), ("one", 30), ("gqa", 20)])
def test_attention_reports_a_page_outside_the_pool(kind, R):
    s = Setup(kind, 3, R, [300, 500, 200], page=128, seed=28)
    s.table[1, 2] = s.k.shape[0]
    s.table[0, 3] = -1                              # not needed
    out, lse = s.attn()
    assert int(s.err) == T.TSD_DEV_ERR_BAD_PAGE | 1
    s.check_attn(out, lse, requests=[0, 2])


@gpu
def test_attention_clamps_lengths_to_the_cache():
    for R in (1, 20):
        s = Setup("gqa", 2, R, [140, 140], extra=0, seed=29)
        s.plen.copy_(torch.tensor([1000, -5], dtype=torch.int32))
        s.lens = [140, 0]
        s.check_attn(*s.attn())


@gpu
@pytest.mark.parametrize("R", [1, 3, 20])
def test_attention_on_streams_and_in_graphs(R):
    a, b = Setup("gqa", 3, R, [2000, 700, 5], seed=30), Setup("narrow", 2, R, [900, 1500], seed=31)
    want = [x.attn() for x in (a, b)]
    bufs = [(torch.zeros_like(o), torch.zeros_like(l), T.workspace(T.tsd_verify_q4_workspace_size(x.desc)))
            for x, (o, l) in zip((a, b), want)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, buf, st in zip((a, b), bufs, streams):
            x.attn_into(*buf, st)
    torch.cuda.synchronize()
    for buf, w in zip(bufs, want):
        assert torch.equal(buf[0], w[0]) and torch.equal(buf[1], w[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.attn_into(*bufs[0])
    a.q.copy_(a.normal(*a.q.shape))
    a.plen.copy_(torch.tensor([1500, 1, 0], dtype=torch.int32))
    a.lens = [1500, 1, 0]
    graph.replay()
    torch.cuda.synchronize()
    a.check_attn(*bufs[0][:2])


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R", [1, 4, 20])
def test_attention_over_a_table_of_many_pages(R, dtype):
    """A capacity of 2^27 positions, of which a request holds 300."""
    s = Setup("gqa", 1, R, [300], page=128, dtype=dtype, seed=67)
    table = torch.full((1, 1 << 20), -1, dtype=torch.int32, device=DEV)
    table[:, :s.table.shape[1]] = s.table
    s.paging["page_table"] = table
    s.desc = T.make_desc(1, R, s.Hq, s.Hkv, s.d, s.d, 1 << 27, dtype, False, s.scale)
    s.check_attn(*s.attn())
    assert int(s.err) == 0


def test_workspaces_of_the_largest_caches():
    for dtype in (torch.bfloat16, torch.float32):
        for R in (1, 4, 65):
            d = T.make_desc(40, R, 32, 8, 128, 128, 2 ** 31 - 128, dtype, False, 0.1)
            size = T.tsd_verify_q4_workspace_size(d)      # (a split has at most 2^21 positions)
            assert size >= (2 ** 31 // (1 << 21) - 1) * 40 * 32 * R * (128 * 2 + 8)


@gpu
def test_attention_past_32_bit_offsets():
    """A pool whose codes pass 2^32 bytes, the request's pages at its end."""
    pages = (1 << 32) // (8 * 128 * 64) + 40
    for R in (1, 20):
        s = Setup("gqa", 1, R, [300], page=128, seed=32)
        k, v = (torch.zeros(pages, 8, 128, 64, dtype=torch.uint8, device=DEV) for _ in range(2))
        ks, vs = (torch.zeros(pages, 8, 128, 4, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        new = s.table.long() + pages - s.k.shape[0]
        for big, small in ((k, s.k), (v, s.v), (ks, s.ks), (vs, s.vs)):
            big[new[0]] = small[s.table[0].long()]
        s.k, s.v, s.ks, s.vs, s.table = k, v, ks, vs, new.int()
        s.paging["page_table"] = s.table
        s.check_attn(*s.attn(), heads=[0, 7])
        x, y = s.normal(1, R, 8, 128), s.normal(1, R, 8, 128)
        n = torch.tensor([R], dtype=torch.int32, device=DEV)
        T.tsd_cache_write_q4(s.desc, x, y, n, *s.arrays(), s.plen, s.err, **s.paging) if R < 8 else \
            T.tsd_cache_write_q4(s.desc, x[:, :8].contiguous(), y[:, :8].contiguous(), n.clamp(max=8), *s.arrays(),
                                 s.plen, s.err, **s.paging)
        out = _read(s, [299], [2], 2)
        c, f = quantise(x[0, 0].double())
        want = ((c - 8).double() * f.repeat_interleave(G, 1)).to(s.dt)
        assert torch.equal(out[0][0, 1], want) and int(s.err) == 0
        del k, v, ks, vs


@gpu
@pytest.mark.parametrize("kind,R,page", [("gqa", 20, 128), ("narrow", 20, 0), ("gqa", 5, 0)])
def test_attention_waits_give_up_at_the_budget(kind, R, page):
    """A budget of a few cycles: every wait that is not met at once gives up, the error word
    says so, the call ends soon, and the next call is exact."""
    s = Setup(kind, 2, R, [900, 300], page=page, seed=33)
    with T.wait_budget(4):
        s.attn()
        assert int(s.err) & T.TSD_DEV_ERR_MASK == T.TSD_DEV_ERR_TIMEOUT
    s.err.zero_()
    s.check_attn(*s.attn())
    assert int(s.err) == 0


# 64 heads over 8 leave 8 packed rows behind groups of 128 for one tree row, 32 over 8 for two
LAST = [("eight", 32, 17, [300, 0, 1000, 129], 1100, 0), ("eight", 32, 33, [700, 64, 2000, 1], 100, 128),
        ("eight", 3, 17, [22000, 129, 0], 100, 128), ("gqa", 32, 34, [1000, 129, 0, 300], 1100, 0),
        ("gqa", 2, 34, [32700, 400], 60, 128), ("gqa", 40, 65, [64, 1800, 127], 300, 0)]


@gpu
@pytest.mark.parametrize("kind,B,R,lens,extra,page", LAST)
def test_attention_with_the_last_rows_on_their_own(kind, B, R, lens, extra, page):
    """One row of eight heads, two rows of four, over one split and over several."""
    s = Setup(kind, B, R, lens, extra=extra, page=page, seed=80)
    out, lse = s.attn()
    assert int(s.err) == 0
    s.check_attn(out, lse, requests=sorted({0, 1, min(2, B - 1), B // 2, B - 1}), heads=[0, s.Hkv - 1])
    assert not (out == 7).all(-1).any() and not (lse == 7).any()
    s.kt[1, R - 1] = NAN                            # seen by the last row alone
    again, _ = s.attn()
    assert again[1, R - 1].isnan().all() and again[1, :R - 1].isfinite().all()
    assert torch.equal(again[0], out[0]) and torch.equal(again[2:], out[2:])


@gpu
@pytest.mark.parametrize("kind,B,R,lens,extra,page", [
    ("gqa", 16, 33, [4000, 300, 0, 129], 96, 0), ("gqa", 32, 33, [2000, 300, 0, 129], 96, 0),
    ("gqa", 34, 34, [2000, 1, 700], 96, 128), ("eight", 16, 17, [4000, 64, 2000], 96, 0),
    ("eight", 32, 17, [2000, 64], 96, 0), ("gqa", 2, 33, [32700, 20000], 68, 128)])
def test_attention_of_rows_rewritten_right_before(kind, B, R, lens, extra, page):
    """Queries, scratch rows and masks that change right before every call: each launch of a call
    has to see what was written before it, on SMs that an earlier launch of the call left empty, too
    (16 requests: fewer CTAs than SMs)."""
    s = Setup(kind, B, R, lens, extra=extra, page=page, seed=81)
    masks = [s.mask.clone()]
    for _ in range(2):
        m = [[0] for _ in range(B)]
        for row in m:
            for r in range(1, R):
                row.append(row[s.rnd.randrange(max(0, r - 4), r)] | (1 << (r - 1)))
        s.set_masks(m)
        masks.append(s.mask)
    last = s.masks
    s.mask = masks[0].clone()
    rows = [[s.normal(B, R, h, s.d) for h in (s.Hq, s.Hkv, s.Hkv)] for _ in range(3)]
    starts = [torch.full((B,), n, dtype=torch.int32, device=DEV) for n in (5, 300, 7000)]
    start = starts[0].clone()
    freq = 1e4 ** (-torch.arange(s.d // 2, dtype=torch.float64) / (s.d // 2))
    rope, turns = T.make_rope_desc(B, R, s.Hq, s.Hkv, s.d, s.dt), T.rope_turns(freq, DEV)
    out, lse = torch.empty_like(s.q), torch.empty(B, R, s.Hq, device=DEV)
    ws = T.workspace(T.tsd_verify_q4_workspace_size(s.desc))

    def turn(i, wait=lambda: None):
        start.copy_(starts[i])
        s.mask.copy_(masks[i])
        wait()
        T.tsd_qk_norm_rope(rope, *rows[i], turns, s.q, s.kt, s.vt, start=start)
        wait()
        s.attn_into(out, lse, ws)
        wait()

    want = []
    for i in range(3):
        turn(i, torch.cuda.synchronize)
        want.append((out.clone(), lse.clone()))
    s.masks = last
    s.check_attn(out, lse, requests=[0, B - 1], heads=[0, s.Hkv - 1])
    kept = [(torch.empty_like(out), torch.empty_like(lse)) for _ in range(24)]
    for n, (o, l) in enumerate(kept):
        turn(n % 3)
        o.copy_(out)
        l.copy_(lse)
    torch.cuda.synchronize()
    for n, (o, l) in enumerate(kept):
        assert torch.equal(o, want[n % 3][0]) and torch.equal(l, want[n % 3][1]), n
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for n in range(6):
            turn(n % 3)
            kept[n][0].copy_(out)
            kept[n][1].copy_(lse)
    for _ in range(5):
        for o, _ in kept:
            o.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        for n in range(6):
            assert torch.equal(kept[n][0], want[n % 3][0]) and torch.equal(kept[n][1], want[n % 3][1]), n
    assert int(s.err) == 0


def check_tight(s, out, lse, requests=None, heads=None):
    """The bounds of check_attn for bf16 inputs, with each error at its own weight.  A run is 128 cached
    rows from a multiple of 128 (a scratch row is one of its own), S_k the largest |scale| of the run of
    key k (the largest element of the scratch row), p_k the key's probability.  A value is held to
    2^-12 and 2^-15 S_k, which costs sum_k p_k 2^-15 S_k.  A probability is held to 2^-12 and half a
    step 2^-24 where the largest p_k 2^E_k (2^E_k <= 2 S_k) is 1 or more: with |v| < 8 2^E_k, a cached key
    adds 8 2^-25 2 max_k p_k S_k at most.  A scratch row's value is held over 2^-18 of its largest element
    or less, relative to 2^E: its weight's half step is worth 2^-14 2 max_k p_k S_k."""
    g = s.Hq // s.Hkv
    for b in requests if requests is not None else range(s.B):
        P = min(s.lens[b], s.cap)
        sees = torch.cat([torch.ones(s.R, P, dtype=torch.bool, device=DEV), s.sees(b)], 1).repeat_interleave(g, 0)
        for h in heads if heads is not None else range(s.Hkv):
            ck, cv = s.cache("k"), s.cache("v")
            kt, vt = s.kt[b, :, h].double(), s.vt[b, :, h].double()
            k, v = torch.cat([ck.values(b, h)[:P], kt]), torch.cat([cv.values(b, h)[:P], vt])

            def by_run(x):
                x = x[:P].abs().amax(-1)
                x = torch.cat([x, x.new_zeros(-P % 128)]).view(-1, 128).amax(-1)
                return x.repeat_interleave(128)[:P]

            Sk = torch.cat([by_run(ck.scales(b, h)), kt.abs().amax(-1)])
            Sv = torch.cat([by_run(cv.scales(b, h)), vt.abs().amax(-1)])
            wide = torch.cat([16 * ck.scales(b, h)[:P].abs().repeat_interleave(G, 1), kt.abs()])
            q = s.q[b, :, h * g:(h + 1) * g].double().reshape(-1, s.d)
            x = (q @ k.T * s.scale).masked_fill(~sees, -INF)
            l = torch.logsumexp(x, -1)
            p = torch.exp(x - l[:, None])
            n = k.shape[0]
            # scores, each weighted by its key: off by ds_k, so a mean of v by at most twice sum_k p_k ds_k |v_k|
            qa = q.abs()
            ds = (s.d + 16) * 2.0 ** -23 * s.scale * (qa @ wide.T) + s.scale * (
                2.0 ** -12 * (qa @ k.abs().T) + 2.0 ** -15 * qa.sum(-1, keepdim=True) * Sk)
            mean = (p * ds).sum(-1, keepdim=True)
            o, A = p @ v, p @ v.abs()
            top = (p * Sv).amax(-1, keepdim=True)
            tol = 2.0 ** -8 * o.abs() + 1.1 * ((p * ds) @ v.abs() + mean * A) + \
                (3 * 2.0 ** -12 + 2.0 ** -19 + n * 2.0 ** -23) * A + 2.0 ** -15 * (p @ Sv)[:, None] + \
                (n * 2.0 ** -21 + s.R * 2.0 ** -13) * top + 1e-37
            got = out[b, :, h * g:(h + 1) * g].double().reshape(-1, s.d)
            far = (got - o).abs() / tol
            assert not got.isnan().any() and (far <= 1).all(), (b, h, float(far.max()))
            gl = lse[b, :, h * g:(h + 1) * g].double().reshape(-1)
            tl = 1.1 * mean[:, 0] + 2.0 ** -19 + n * 2.0 ** -23 + 2.0 ** -22 * l.abs()
            far = (gl - l).abs() / tl
            assert (far <= 1).all(), (b, h, float(far.max()))


def _blocks(s, powers, run):
    """Runs of value scales times 2^power, in turn along the cache (None: zeros)."""
    f = torch.tensor([0.0 if p is None else 2.0 ** p for p in powers], dtype=torch.float64, device=DEV)
    at = torch.arange(s.cap, device=DEV) // run % len(powers)
    for b in range(s.B):
        for pos in range(0, s.cap, run):
            pg, row = (b, pos) if s.table is None else (int(s.table[b, pos // s.page]), pos % s.page)
            part = s.vs[pg, :, row:row + run]
            part.copy_((part.double() * f[at[pos]]).bfloat16())


SPREAD = {"zeros beside 2^30": ([None, 30], 32), "zeros beside 2^100": ([None, 100], 128),
          "2^100 and zeros": ([100, None, None], 32), "80 apart": ([-40, 40, 0], 32),
          "160 apart": ([-80, 80], 128), "rising": ([-90, -30, 30, 90], 128), "falling": ([90, 20, -50, -90], 128)}


@gpu
@pytest.mark.parametrize("kind,R,page", [("gqa", 1, 0), ("gqa", 4, 128), ("narrow", 2, 0), ("gqa", 20, 128),
                                         ("one", 65, 0), ("narrow", 12, 256)])
@pytest.mark.parametrize("name", SPREAD)
def test_attention_counts_keys_whatever_their_values_size(kind, R, page, name):
    """Runs of values that are zero or 2^80 and more apart: every key counts in the sum of weights."""
    for tree in (1.0, 0.0, 2.0 ** 100):
        s = Setup(kind, 3, R, [700, 130, 33], page=page, seed=82)
        _blocks(s, *SPREAD[name])
        s.vt *= tree
        s.check_attn(*s.attn())
        check_tight(s, *s.attn())
    assert int(s.err) == 0


@gpu
@pytest.mark.parametrize("kind,R", [("gqa", 1), ("gqa", 4), ("narrow", 2), ("narrow", 12), ("gqa", 20)])
def test_attention_counts_keys_of_large_scores_beside_large_values(kind, R):
    """Scores that rise and fall by a hundred while the values' size does the opposite, over several splits."""
    s = Setup(kind, 2, R, [6000, 900], seed=83)
    ramp = torch.exp2(3 * torch.sin(torch.arange(s.rows, device=DEV) / 150.0)).bfloat16()
    s.ks *= ramp[:, None]
    _blocks(s, [100, 60, 20, -20, -60, -90, None, 0], 64)
    s.check_attn(*s.attn())
    check_tight(s, *s.attn())


def _shunned(s, pos, power):
    """A run of 128 cached rows whose weight is nothing (scores below -150) and whose values are 2^power."""
    s.q[..., 0] = 8.0
    for b in range(s.B):
        if s.lens[b] < pos + 128:
            continue
        pg, row = (b, pos) if s.table is None else (int(s.table[b, pos // s.page]), pos % s.page)
        s.ks[pg, :, row:row + 128, 0] = 64.0
        s.k[pg, :, row:row + 128, 1:16] = 0x88
        s.k[pg, :, row:row + 128, 0] = 0x80     # dim 0: code 0, -8 s; the other dims of the group: 0
        s.vs[pg, :, row:row + 128] = 2.0 ** power


@gpu
@pytest.mark.parametrize("kind,R,page,lens", [("gqa", 20, 128, [5000, 700]), ("one", 30, 0, [4000]),
                                              ("narrow", 12, 0, [6000, 400]), ("gqa", 65, 128, [20000, 300]),
                                              ("gqa", 4, 0, [5000]), ("narrow", 1, 128, [6000])])
@pytest.mark.parametrize("power", [16, 22, 30, 100])
def test_attention_keeps_small_values_beside_large_ones_of_no_weight(kind, R, page, lens, power):
    """Also where the large ones are in the same split."""
    s = Setup(kind, len(lens), R, lens, page=page, seed=84)
    _shunned(s, 256, power)
    check_tight(s, *s.attn())
    assert int(s.err) == 0


@gpu
@pytest.mark.parametrize("kind,R,dtype", [("gqa", 2, torch.bfloat16), ("gqa", 4, torch.bfloat16),
                                          ("narrow", 2, torch.bfloat16), ("gqa", 20, torch.bfloat16),
                                          ("gqa", 3, torch.float32), ("gqa", 20, torch.float32)])
@pytest.mark.parametrize("lens", [[200, 40, 0, 90], [6000, 5000, 4000, 3000]])
def test_attention_passes_infinite_scratch_rows_on(kind, R, dtype, lens):
    """To the rows that see them, and to no others, whatever their scores: of both signs, and in a value
    whose weight is nothing."""
    s = Setup(kind, 4, R, lens, dtype=dtype, seed=85)
    masks = [list(m) for m in s.masks]
    for m in masks:
        m[R - 1] = 1 << (R - 2)                     # the last row is seen by itself alone
    s.set_masks(masks)
    s.q[..., 0] = s.q[..., 0].abs() + 1
    s.kt[0, R - 1, :, 0] = -INF
    s.kt[1, R - 1, :, 0] = INF
    s.kt[2, R - 1, :, 0] = -20000.0
    s.vt[2, R - 1, :, 5] = -INF
    s.kt[3, R - 1, :, 0] = -INF
    s.vt[3, R - 1, :, 3] = INF
    out, lse = s.attn()
    assert out[:, :R - 1].isfinite().all() and lse[:, :R - 1].isfinite().all()
    assert not out[:, R - 1].isfinite().all(-1).any()
    assert out[[0, 1, 3], R - 1].isnan().all()


@gpu
@pytest.mark.parametrize("R,dtype", [(1, torch.bfloat16), (5, torch.bfloat16), (20, torch.bfloat16),
                                     (1, torch.float32), (20, torch.float32)])
def test_attention_over_prefixes_near_two_to_the_31(R, dtype):
    """A request of 2^31 - 228 positions: one page again and again, and another as the last one, whose
    scores are large enough for it to count.  The sums have up to 2^15 + 2^11 terms one after the other,
    each rounded to 2^-24: off by 2^-8, relatively.  Probabilities in the last split (2^15 keys) are held
    to half a step 2^-24 of the largest product: 2^15 2^-25 16 max_k p_k S_k."""
    s = Setup("odd", 1, R, [156], page=128, dtype=dtype, seed=86)
    pages = (1 << 24) - 1
    first, end = s.table[0, :2].tolist()
    s.ks[end] *= 16
    s.plen.fill_(pages * 128 - 100)
    table = torch.full((1, pages), first, dtype=torch.int32, device=DEV)
    table[0, -1] = end
    s.paging["page_table"] = table
    s.desc = T.make_desc(1, R, s.Hq, s.Hkv, s.d, s.d, pages * 128, dtype, False, s.scale)
    out, lse = s.attn()
    assert int(s.err) == 0
    ck, cv = s.cache("k"), s.cache("v")                   # (its positions 0..155 are the two pages' rows)
    k = torch.cat([ck.values(0, 0)[:156], s.kt[0, :, 0].double()])
    v = torch.cat([cv.values(0, 0)[:156], s.vt[0, :, 0].double()])
    times = torch.ones(156 + R, dtype=torch.float64, device=DEV)
    times[:128] = pages - 1
    sees = torch.cat([torch.ones(R, 156, dtype=torch.bool, device=DEV), s.sees(0)], 1).repeat_interleave(s.Hq, 0)
    q = s.q[0].double().reshape(-1, s.d)
    x = (q @ k.T * s.scale + times.log()).masked_fill(~sees, -INF)
    l = torch.logsumexp(x, -1)
    p = torch.exp(x - l[:, None])
    o, A = p @ v, p @ v.abs()
    wide = torch.cat([16 * ck.scales(0, 0)[:156].abs().repeat_interleave(G, 1), s.kt[0, :, 0].double().abs()])
    ds = s.scale * (s.d + 16) * 2.0 ** -23 * (q.abs() @ wide.T).masked_fill(~sees, 0).amax(-1, keepdim=True)
    low, p16, top = 2.0 ** -24, 0.0, torch.zeros_like(ds)
    if dtype == torch.bfloat16:
        low, p16 = 2.0 ** -8, 3 * 2.0 ** -12
        S = torch.cat([cv.scales(0, 0)[:156].abs().amax(-1), s.vt[0, :, 0].double().abs().amax(-1)])
        Sk = torch.cat([ck.scales(0, 0)[:156].abs().amax(-1), s.kt[0, :, 0].double().abs().amax(-1)])
        ds = ds + s.scale * (2.0 ** -12 * q.abs() @ k.abs().T + 2.0 ** -15 * q.abs().sum(-1, keepdim=True) * Sk.max()
                             ).masked_fill(~sees, 0).amax(-1, keepdim=True)
        top = 2.0 ** -15 * S.max() + 2.0 ** (15 - 25 + 4) * (p / times * S).amax(-1, keepdim=True)
    tol = low * o.abs() + (2.2 * ds + 2 * 2.0 ** -8 + p16) * A + top
    far = (out[0].double().reshape(-1, s.d) - o).abs() / tol
    assert (far <= 1).all(), float(far.max())
    far = (lse[0].double().reshape(-1) - l).abs() / (1.1 * ds[:, 0] + 2.0 ** -8 + 2.0 ** -22 * l.abs())
    assert (far <= 1).all(), float(far.max())
    # an append ends at the last position
    x, y = s.normal(1, 100, 1, s.d), s.normal(1, 100, 1, s.d)
    n = torch.tensor([100], dtype=torch.int32, device=DEV)
    T.tsd_cache_write_q4(s.desc, x, y, n, *s.arrays(), s.plen, s.err, **s.paging)
    back = _read(s, [pages * 128 - 1], [1], 1)
    c, f = quantise(x[0, 99].double())
    assert torch.equal(back[0][0, 0], ((c - 8).double() * f.repeat_interleave(G, 1)).to(dtype))
    assert int(s.plen) == pages * 128 and int(s.err) == 0


def test_workspaces_of_the_largest_caches_by_type():
    """At most 2^15 positions a split of bf16 inputs, 2^21 of fp32 ones."""
    for dtype, most, size in ((torch.bfloat16, 1 << 15, 2), (torch.float32, 1 << 21, 4)):
        for R in (1, 4, 65):
            d = T.make_desc(40, R, 32, 8, 128, 128, 2 ** 31 - 128, dtype, False, 0.1)
            assert T.tsd_verify_q4_workspace_size(d) >= 2 ** 31 // most * 40 * 32 * R * (128 * size + 8)


@pytest.mark.parametrize("R,dtype", [(1, T.TSD_BF16), (20, T.TSD_BF16), (20, T.TSD_F32)])
def test_attention_checks_the_largest_caches_as_others(R, dtype):
    """A capacity of 2^31 - 128 positions is refused for its workspace alone."""
    d = _desc(B=1, R=R, cap=2 ** 31 - 128, dtype=dtype)
    need = T.tsd_verify_q4_workspace_size(d)
    assert need > 0 and _calls(d, ws=need - 1)["attn"]() == T.TSD_ERR_INVALID_ARG


@gpu
@pytest.mark.parametrize("kind,R,dtype", [("gqa", 1, torch.bfloat16), ("gqa", 20, torch.bfloat16),
                                          ("gqa", 1, torch.float32), ("gqa", 3, torch.float32),
                                          ("gqa", 20, torch.float32), ("narrow", 4, torch.float32)])
@pytest.mark.parametrize("lens", [[200, 0], [5000, 300]])
def test_attention_of_rows_of_q_that_are_not_finite_is_nan(kind, R, dtype, lens):
    """Also where every score is -inf, and whatever the NaN's bits."""
    s = Setup(kind, 2, R, lens, dtype=dtype, seed=87)
    s.k[..., 0] = (s.k[..., 0] & 0xf0) | 0xc            # dim 0 of every cached key: 4 s, s > 0
    s.ks[..., 0] = s.ks[..., 0].abs()
    s.kt[..., 0] = s.kt[..., 0].abs() + 1
    s.q[0, 0, 0, 0] = -INF
    s.q[0, R - 1, 3, 0] = INF
    s.q[1, R - 1, 1, 0] = NAN
    if dtype == torch.float32:
        s.q.view(torch.int32)[1, 0, 2, 9] = 0x7f800001
    else:
        s.q.view(torch.int16)[1, 0, 2, 9] = 0x7f81
    bad = torch.zeros(2, R, s.Hq, dtype=torch.bool, device=DEV)
    bad[0, 0, 0] = bad[0, R - 1, 3] = bad[1, R - 1, 1] = bad[1, 0, 2] = True
    out, lse = s.attn()
    assert out[bad].isnan().all() and lse[bad].isnan().all()
    assert out[~bad].isfinite().all() and lse[~bad].isfinite().all()


@gpu
@pytest.mark.parametrize("kind,R", [("gqa", 1), ("gqa", 4), ("narrow", 2), ("gqa", 20)])
@pytest.mark.parametrize("lens", [[0, 5], [300, 5000]])
def test_attention_of_the_largest_scratch_values(kind, R, lens):
    """A mean of values next to bf16's largest is finite, though their sum is not in fp32."""
    s = Setup(kind, 2, R, lens, seed=88)
    s.vt = torch.where(s.vt > 0, 1.0, -1.0).to(s.dt) * (s.normal(*s.vt.shape).abs().clamp(max=1) * 0.5 + 0.5) * 3.3e38
    out, lse = s.attn()
    assert out.isfinite().all() and lse.isfinite().all()
    check_tight(s, out, lse)


@pytest.mark.parametrize("dtype", [T.TSD_BF16, T.TSD_F32])
def test_workspace_of_a_call_that_is_refused_is_none(dtype):
    """More KV heads than a grid has rows."""
    for R, Hkv in ((1, 65536), (65, 65536), (1, 65535)):
        d = _desc(B=1, R=R, Hq=Hkv, Hkv=Hkv, cap=1 << 24, dtype=dtype)
        refused = Hkv > 65535
        assert (T.tsd_verify_q4_workspace_size(d) == 0) == refused
        assert not refused or _calls(d)["attn"]() == T.TSD_ERR_INVALID_ARG
