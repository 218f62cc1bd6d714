"""Norm and rotation of queries and keys against plain 64-bit code."""

import ctypes
import math
import random
from fractions import Fraction

import pytest
import torch

import tree_speculative_decoding_tsd_gb300 as T

DEV = "cuda:0"
NAN, INF = float("nan"), float("inf")
gpu = pytest.mark.gpu


# ------------------------------------------------------------ plain forms --

def angles(freq, pos):
    """freq [axes][n] radians, pos [axes][B][T] -> [B][T][n], in exact arithmetic up to the end:
    whole turns (of a double's 2 pi, whose error 2^-53 times the angle is below 1e-9 for the
    tests' angles) are not taken off."""
    return torch.einsum("abt,an->btn", pos.double(), freq.double())


def plain(x, w, angle, rot, near, norm, eps, amplitude):
    """x [B][T][H][d] (float64) normed and turned; also the scale of its errors, the largest
    magnitude of the pair before it is turned."""
    if norm:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        if w is not None:
            x = x * w.double()
    n = rot // 2
    i = torch.arange(n, device=x.device) * (2 if near else 1)
    j = i + (1 if near else n)
    u, v = x[..., i], x[..., j]
    c, s = torch.cos(angle)[:, :, None], torch.sin(angle)[:, :, None]
    y, size = x.clone(), x.abs()
    y[..., i], y[..., j] = amplitude * (u * c - v * s), amplitude * (u * s + v * c)
    big = abs(amplitude) * torch.hypot(u, v)
    size[..., i], size[..., j] = big, big
    return y, size


class Setup:
    def __init__(self, B, Tn, Hq, Hkv, d, dtype=torch.bfloat16, rot=None, axes=1, near=False, norm=True,
                 eps=1e-6, amplitude=1.0, seed=0, far=4096, fused=True, start=True, offset=True,
                 count=None, weights=True):
        self.g = torch.Generator(device=DEV).manual_seed(seed + 77)
        self.rnd = random.Random(seed)
        self.shape = B, Tn, Hq, Hkv, d
        self.dt, self.rot, self.near, self.norm = dtype, d if rot is None else rot, near, norm
        self.eps, self.amplitude = float(torch.tensor(eps)), float(torch.tensor(amplitude))
        heads = (Hq, Hkv, Hkv)
        if fused:
            self.qkv = self.normal(B, Tn, sum(heads) * d + 64)   # (a gap between the rows)
            self.rows = [t.view(B, Tn, -1, d) for t in
                         self.qkv[..., : sum(heads) * d].split([h * d for h in heads], -1)]
        else:
            self.rows = [self.normal(B, Tn, h, d) for h in heads]
        self.w = [(1 + 0.2 * self.normal(d)).to(dtype) for _ in range(2)] if weights and norm else [None] * 2
        n = self.rot // 2
        base = 10000.0 ** (-torch.arange(max(n, 1), dtype=torch.float64)[:n] / max(n, 1))
        self.freq = torch.zeros(axes, n, dtype=torch.float64)
        for i in range(n):
            self.freq[i % axes, i] = base[i]
        self.turns = T.rope_turns(self.freq, DEV) if n else None
        i32 = dict(dtype=torch.int32, device=DEV)
        self.start = torch.tensor([self.rnd.randint(0, far) for _ in range(B)], **i32) if start else None
        self.offset = torch.tensor([[[self.rnd.randint(0, far) for _ in range(Tn)] for _ in range(B)]
                                    for _ in range(axes)], **i32) if offset else None
        self.count = None if count is None else torch.tensor(count, **i32)
        self.out = [torch.full((B, Tn, h, d), 7.0, dtype=dtype, device=DEV) for h in heads]
        self.desc = T.make_rope_desc(B, Tn, Hq, Hkv, d, dtype, self.rot, axes, near, norm, eps, amplitude)

    def normal(self, *shape):
        return torch.randn(*shape, generator=self.g, device=DEV).to(self.dt)

    def call(self, v=True, out=None, stream=None):
        out = out or self.out
        rows = self.rows
        T.tsd_qk_norm_rope(self.desc, rows[0], rows[1], rows[2] if v else None, self.turns, out[0], out[1],
                           out[2] if v else None, *self.w, self.start, self.offset, self.count, stream)
        torch.cuda.synchronize()

    def check(self, rows=None, out=None, v=True):
        """Bounds.  fp32: the mean is a sum of d squares in any order, off by d 2^-24 relatively at
        most (half of that in its root), the reciprocal root and three products 2^-22 more; an
        angle by 2^-32 turns, a float's rounding of it (2^-24 of at most pi) and the functions'
        own 2 units, below 2^-21 together; each product and sum of the turn 2^-24.  Together
        below (d/2 + 16) 2^-24 of the pair's length; the result is rounded once (bf16: 2^-8,
        fp32: 2^-24)."""
        B, Tn, Hq, Hkv, d = self.shape
        out = out or self.out
        rows = rows or self.rows
        at = self.offset if self.offset is not None else \
            torch.arange(Tn, device=DEV).expand(self.freq.shape[0], B, Tn)
        pos = at.long() + (0 if self.start is None else self.start.long()[:, None])
        a = angles(self.freq.to(DEV), pos)
        live = torch.ones(B, Tn, dtype=torch.bool, device=DEV) if self.count is None else \
            torch.arange(Tn, device=DEV) < self.count[:, None]
        low = 2.0 ** -8 if self.dt == torch.bfloat16 else 2.0 ** -24
        for i in range(2):
            y, size = plain(rows[i].double(), self.w[i], a, self.rot, self.near, self.norm, self.eps,
                            self.amplitude)
            tol = low * y.abs() + (d / 2 + 16) * 2.0 ** -24 * size + 1e-37
            got = out[i].double()
            assert ((got - y).abs() <= tol)[live].all(), (i, float(((got - y).abs() / tol)[live].max()))
            assert (got[~live] == 7).all()
        if v:
            assert torch.equal(out[2][live], rows[2][live]) and (out[2][~live] == 7).all()


# ------------------------------------------------- refusals (on the host) --

A, U, N = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008), None


def _call(q=A, qs=512, k=A, ks=256, v=A, vs=256, qw=A, kw=A, turns=A, start=A, offset=A, oa=1, count=A,
          qo=A, ko=A, vo=A, **kw_desc):
    base = dict(B=2, T=3, Hq=4, Hkv=2, d=128, dtype=T.TSD_BF16, rot=128, neighbours=0, axes=1, norm=1,
                eps=1e-6, amplitude=1.0)
    base.update(kw_desc)
    return T.lib.tsd_qk_norm_rope(ctypes.byref(T.tsd_rope_desc(**base)), q, qs, k, ks, v, vs, qw, kw, turns,
                                  start, offset, oa, count, qo, ko, vo, N)


@pytest.mark.parametrize("kw", [
    dict(B=0), dict(T=0), dict(Hq=0), dict(Hkv=0), dict(d=96), dict(d=256), dict(dtype=5), dict(rot=-8),
    dict(rot=136), dict(rot=12), dict(axes=0), dict(axes=5), dict(eps=-1.0), dict(eps=NAN), dict(eps=INF),
    dict(amplitude=NAN), dict(amplitude=INF), dict(q=N), dict(k=N), dict(q=U), dict(k=U), dict(v=U), dict(vo=N),
    dict(v=N), dict(qo=N), dict(ko=U), dict(qw=U), dict(kw=U), dict(turns=N), dict(turns=U), dict(start=U),
    dict(offset=U), dict(count=U), dict(norm=0), dict(norm=0, qw=N), dict(qs=504), dict(qs=516), dict(ks=128),
    dict(ks=-256), dict(vs=0), dict(vs=257), dict(oa=0), dict(oa=2), dict(oa=2, axes=3),
    dict(B=2 ** 31 - 1, T=2 ** 31 - 1)])
def test_call_rejects_bad_arguments(kw):
    assert _call(**kw) == T.TSD_ERR_INVALID_ARG


def test_call_rejects_no_descriptor():
    assert T.lib.tsd_qk_norm_rope(N, *[A, 512] * 3, *[A] * 5, 1, *[A] * 4, N) == T.TSD_ERR_INVALID_ARG


def test_turns_are_fractions_of_a_turn():
    pi = Fraction(math.pi) + Fraction(1.2246467991473532e-16)     # (pi to 2^-105)
    freq = torch.tensor([[0.0, 1.0, 1e-6, 3.0, 7.5], [1e4, -1.0, 2.0 ** -40, -0.25, math.pi]], dtype=torch.float64)
    got = T.rope_turns(freq)
    assert got.dtype == torch.int64 and got.shape == (2, 5)
    for f, bits in zip(freq.flatten().tolist(), got.flatten().tolist()):
        want = Fraction(f) / (2 * pi) * 2 ** 64
        off = (Fraction(bits) - want) % 2 ** 64
        assert min(off, 2 ** 64 - off) < 2
    assert T.rope_turns([0.5, 0.25]).shape == (1, 2)
    for bad in (NAN, INF, 2.0 ** 20, -1e30):
        with pytest.raises(ValueError):
            T.rope_turns([0.5, bad])
    for f in (2.0 ** 20 - 1, -5e-324, 2.0 ** -300, 1e5 / 3):
        want, bits = Fraction(f) / (2 * pi) * 2 ** 64, int(T.rope_turns([f])[0, 0])
        off = (Fraction(bits) - want) % 2 ** 64
        assert min(off, 2 ** 64 - off) < 2


# ---------------------------------------------------------------- results --

CASES = [dict(B=1, Tn=17, Hq=32, Hkv=8, d=128), dict(B=3, Tn=33, Hq=32, Hkv=8, d=128, offset=False),
         dict(B=2, Tn=1, Hq=14, Hkv=2, d=64, start=False), dict(B=2, Tn=5, Hq=14, Hkv=2, d=64, near=True),
         dict(B=1, Tn=1, Hq=1, Hkv=1, d=64), dict(B=2, Tn=3, Hq=3, Hkv=1, d=128, rot=64, near=True),
         dict(B=2, Tn=7, Hq=5, Hkv=1, d=64, rot=24), dict(B=2, Tn=9, Hq=7, Hkv=7, d=128, rot=0),
         dict(B=2, Tn=9, Hq=8, Hkv=2, d=128, rot=8, norm=False), dict(B=2, Tn=40, Hq=8, Hkv=2, d=128, axes=3),
         dict(B=1, Tn=65, Hq=8, Hkv=1, d=64, axes=4, near=True, amplitude=1.25),
         dict(B=2, Tn=12, Hq=8, Hkv=8, d=128, axes=2, amplitude=-0.5, eps=0.0),
         dict(B=3, Tn=50, Hq=8, Hkv=2, d=128, count=[0, 50, 23]), dict(B=2, Tn=6, Hq=8, Hkv=2, d=128, weights=False),
         dict(B=2, Tn=6, Hq=8, Hkv=2, d=128, norm=False, rot=64), dict(B=2, Tn=300, Hq=16, Hkv=1, d=128, eps=0.5),
         dict(B=5, Tn=2000, Hq=4, Hkv=1, d=64, count=[2000, 1, 3, 1999, 0], offset=False)]


@gpu
@pytest.mark.parametrize("kw", CASES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_match_plain(kw, dtype):
    for fused in (True, False):
        s = Setup(**kw, dtype=dtype, fused=fused, seed=len(kw))
        s.call()
        s.check()


@gpu
@pytest.mark.parametrize("far", [1 << 20, 2 ** 31 - 1])
def test_far_positions_keep_their_angle(far):
    """The turn of a far position against exact arithmetic on whole numbers: the fp32 rows of
    an unnormed (1, 0) pair are its cosine and sine, to 2^-20 (a few units of the functions)
    and the 2^-33 turns that a frequency's 64 bits leave times the position."""
    s = Setup(2, 9, 2, 1, 64, dtype=torch.float32, norm=False, far=1, seed=far % 97)
    s.start = torch.tensor([far, far - 12345], dtype=torch.int32, device=DEV)
    s.offset = torch.arange(9, dtype=torch.int32, device=DEV).expand(1, 2, 9).contiguous()
    if far == 2 ** 31 - 1:
        s.offset[0, 1] = -far                      # (sums pass 32 bits on the one side, 0 on the other)
    s.rows[0][..., :32], s.rows[0][..., 32:] = 1.0, 0.0
    s.call(v=False)
    pi = Fraction("3.14159265358979323846264338327950288419716939937510582097")
    for b in range(2):
        for t in range(9):
            pos = int(s.start[b]) + int(s.offset[0, b, t])
            for i in range(32):
                turn = float(Fraction(float(s.freq[0, i])) * pos / (2 * pi) % 1)
                tol = 2.0 ** -20 + abs(pos) * 2.0 ** -62
                assert abs(float(s.out[0][b, t, 1, i]) - math.cos(2 * math.pi * turn)) < tol
                assert abs(float(s.out[0][b, t, 1, 32 + i]) - math.sin(2 * math.pi * turn)) < tol


@gpu
def test_one_offset_serves_all_axes():
    s = Setup(2, 33, 8, 2, 128, axes=3)
    s.offset = s.offset[:1].contiguous()
    s.call()
    s.offset = s.offset.expand(3, -1, -1).contiguous()
    s.check()


@gpu
def test_rows_may_be_their_own_outputs():
    s = Setup(2, 70, 14, 2, 128, fused=False)
    before = [t.clone() for t in s.rows]
    s.call(out=s.rows)
    s.check(rows=before, out=s.rows)


@gpu
def test_nan_and_infinity_stay_in_their_row():
    s = Setup(1, 4, 4, 2, 128)
    s.rows[0][0, 1, 2, 5] = NAN
    s.rows[1][0, 2, 0, 9] = INF
    s.rows[0][0, 3, 0] = 0
    s.call()
    q, k = s.out[0].float(), s.out[1].float()
    assert q[0, 1, 2].isnan().all() and q.isnan().sum() == 128
    assert not k[0, 2, 0].isfinite().all() and k[0, 2, 1].isfinite().all() and k[0, :2].isfinite().all()
    assert (q[0, 3, 0] == 0).all()
    s.call(v=False)


@gpu
def test_call_on_a_stream_and_in_a_graph():
    s = Setup(2, 33, 32, 8, 128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s.call(stream=side)
    s.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        T.tsd_qk_norm_rope(s.desc, *s.rows, s.turns, *s.out, *s.w, s.start, s.offset, s.count)
    s.qkv.copy_(s.normal(*s.qkv.shape))
    s.start.add_(100)
    graph.replay()
    torch.cuda.synchronize()
    s.check()


@gpu
def test_binding_rejects_types_shapes_and_strides():
    s = Setup(2, 5, 4, 2, 128)
    q, k, v = s.rows

    def call(desc=s.desc, q=q, k=k, v=v, turns=s.turns, out=s.out, **kw):
        T.tsd_qk_norm_rope(desc, q, k, v, turns, *out, **kw)

    call()
    for kw in (dict(q=q.float()), dict(turns=s.turns.double()), dict(start=s.start.long()),
               dict(q_weight=s.w[0].float())):
        with pytest.raises(TypeError):
            call(**kw)
    wide = s.normal(2, 5, 8, 128)
    for kw in (dict(q=q[:, :4]), dict(q=wide[:, :, ::2]), dict(q=s.normal(5, 2, 4, 128).transpose(0, 1)),
               dict(k=s.normal(2, 10, 2, 128)[:, :5]), dict(q=q.cpu()), dict(turns=s.turns[:, :32]),
               dict(out=[s.out[0][:, :, :3], *s.out[1:]]), dict(offset=s.offset[0]), dict(count=s.start[:1])):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(T.TsdError):
        call(v=None)
    torch.cuda.synchronize()
