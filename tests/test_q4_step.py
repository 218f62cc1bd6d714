"""The step over a 4-bit cache: rounds against the calls they are made of and plain 64-bit
code, eager and captured.  (The calls have their own checks.)"""

import pytest
import torch

import tree_speculative_decoding_tsd_gb300 as T
from test_q4_cache import DEV, G, Setup, quantise, unpack
from test_rope import angles, plain
from tree_speculative_decoding_tsd_gb300.step import Q4Cache, Q4TreeVerifyStep, Rope, TreeVerifyStep

gpu = pytest.mark.gpu
S, D, V = 4, 8, 1000


@pytest.mark.parametrize("heads", [(128, 1, 576, 512, True), (8, 2, 128, 64, False), (8, 2, 96, 96, False)])
def test_step_rejects_heads(heads):
    Hq, Hkv, dk, dv, alias = heads
    with pytest.raises(ValueError):
        Q4TreeVerifyStep(2, S, V, 4, D, Hq, Hkv, dk, dv, 256, torch.bfloat16, alias, 0.1)


def _prepare(kind, page, axes, near=False):
    """A step, its state behind a prompt that went through the rotation, and logits that accept
    a few tree rows."""
    s = Setup(kind, 2, D + 1, [0, 0], extra=200, page=page, seed=5)
    n = s.d // 2
    freq = torch.zeros(axes, n, dtype=torch.float64)
    for i in range(n):
        freq[i % axes, i] = 10000.0 ** (-i / n)
    rope = Rope(T.rope_turns(freq, DEV), (1 + 0.1 * s.normal(s.d)).to(s.dt), (1 + 0.1 * s.normal(s.d)).to(s.dt),
                neighbours=near)
    step = Q4TreeVerifyStep(2, S, V, 4, D, s.Hq, s.Hkv, s.d, s.d, s.cap, s.dt, False, s.scale, DEV, rope)
    cache = Q4Cache(*s.arrays(), s.table, page) if page else step.new_cache()
    count = torch.tensor([150, 61], dtype=torch.int32, device=DEV)
    qkv = s.normal(2, 150, s.Hq + 2 * s.Hkv, s.d).split([s.Hq, s.Hkv, s.Hkv], 2)
    start = torch.zeros(2, dtype=torch.int32, device=DEV)
    _, k, v = step.rotate(rope, *qkv, start, count=count)
    step.append(k, v, count, cache, s.plen)
    probs = torch.softmax(torch.randn(2, S, V, generator=s.g, device=DEV) * 3, -1)
    root = torch.tensor([5, 9], dtype=torch.int32, device=DEV)
    step.build(probs, root)
    logits = torch.randn(2, D + 1, V, generator=s.g, device=DEV)
    for b in range(2):
        for r in range(1, D + 1):
            logits[b, int(step.tree.parent[b, r]), int(step.tree.token[b, r])] = 50.0
    proj = s.normal(2, D + 1, s.Hq + 2 * s.Hkv, s.d)
    return s, step, cache, rope, freq.to(DEV), probs, root, logits, proj


def _state(cache, plen):
    return [*cache.arrays(), plen]


@gpu
@pytest.mark.parametrize("kind,page,axes,near", [("gqa", 0, 1, False), ("narrow", 128, 3, True), ("one", 256, 2, False)])
def test_step_rounds_are_their_calls(kind, page, axes, near):
    s, step, cache, rope, freq, probs, root, logits, proj = _prepare(kind, page, axes, near)
    parts = proj.split([s.Hq, s.Hkv, s.Hkv], 2)
    for _ in range(3):
        proj.copy_(s.normal(*proj.shape))
        before = [t.clone() for t in _state(cache, s.plen)]
        lens = s.plen.tolist()
        step.run(probs, root, parts[0], cache, s.plen, parts[1], parts[2], logits)
        torch.cuda.synchronize()
        # the rotation against its plain form at prefix + depth
        pos = (before[4][:, None] + step.tree.depth).expand(axes, 2, D + 1)
        a = angles(freq, pos)
        for got, x, w in ((step.q, parts[0], rope.q_weight), (step.ktree, parts[1], rope.k_weight)):
            y, size = plain(x.double(), w, a, s.d, near, True, float(torch.tensor(1e-6)), 1.0)
            assert ((got.double() - y).abs() <= 2.0 ** -8 * y.abs() + (s.d / 2 + 16) * 2.0 ** -24 * size).all()
        assert torch.equal(step.vtree, parts[2])
        # the attention against its plain form on the state before
        s.k, s.v, s.ks, s.vs = before[:4]
        s.q, s.kt, s.vt, s.lens = step.q, step.ktree, step.vtree, lens
        s.set_masks([[v & ((1 << 64) - 1) for v in m] for m in step.tree.mask.tolist()])
        s.check_attn(step.out, step.lse)
        # the commit against its plain form
        accepted = step.walk.accept_len.tolist()
        assert all(0 < x <= S for x in accepted)
        assert s.plen.tolist() == [n + x + 1 for n, x in zip(lens, accepted)]
        for b in range(2):
            rows = step.walk.accept_rows[b, : accepted[b] + 1].tolist()
            for i, r in enumerate(rows):
                pg, at = (b, lens[b] + i) if not page else \
                    (int(cache.page_table[b, (lens[b] + i) // page]), (lens[b] + i) % page)
                for x, codes, scales in ((step.ktree, cache.kq, cache.kscale), (step.vtree, cache.vq, cache.vscale)):
                    c, f = quantise(x[b, r].double())
                    assert torch.equal(unpack(codes[pg, :, at]), c) and torch.equal(scales[pg, :, at].double(), f)
        # and read back
        first, count = before[4], step.walk.accept_len + 1
        out = [torch.zeros(2, S + 1, s.Hkv, s.d, dtype=s.dt, device=DEV) for _ in range(2)]
        step.read(cache, s.plen, first, count, *out)
        c, f = quantise(step.vtree[1, 0].double())
        assert torch.equal(out[1][1, 0], ((c - 8).double() * f.repeat_interleave(G, 1)).to(s.dt))
    assert int(step.err[0]) == 0


@gpu
@pytest.mark.parametrize("kind,axes", [("gqa", 1), ("narrow", 3)])
def test_step_captured_is_eager(kind, axes):
    s, step, cache, rope, freq, probs, root, logits, proj = _prepare(kind, 0, axes)
    q, k, v = proj.split([s.Hq, s.Hkv, s.Hkv], 2)
    start = [t.clone() for t in _state(cache, s.plen)]
    args = (probs, root, q, cache, s.plen, k, v, logits)
    eager = []
    for _ in range(3):
        step.run(*args)
        eager.append([t.clone() for t in [step.out, step.lse] + _state(cache, s.plen)])
    graph = step.capture(*args)
    torch.cuda.synchronize()
    for t, u in zip(_state(cache, s.plen), start):
        t.copy_(u)
    torch.cuda.synchronize()
    for want in eager:
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip([step.out, step.lse] + _state(cache, s.plen), want))
    assert int(step.err[0]) == 0


@gpu
def test_step_without_a_rope_takes_rows_as_they_are():
    s, roped, cache, rope, freq, probs, root, logits, proj = _prepare("gqa", 0, 1)
    step = Q4TreeVerifyStep(2, S, V, 4, D, s.Hq, s.Hkv, s.d, s.d, s.cap, s.dt, False, s.scale, DEV)
    lens = s.plen.tolist()
    step.run(probs, root, s.q, cache, s.plen, s.kt, s.vt, logits)
    assert s.plen.tolist() == [n + a + 1 for n, a in zip(lens, step.walk.accept_len.tolist())]
    with pytest.raises(ValueError):
        step.run(probs, root, s.q, cache, s.plen, s.kt, s.vt, logits, start=s.plen)
    with pytest.raises(NotImplementedError):
        step.accept_commit()
    assert int(step.err[0]) == 0


@gpu
def test_rotate_tree_serves_the_16_bit_step():
    """The tree that was built last gives the offsets."""
    s, _, _, rope, freq, probs, root, logits, proj = _prepare("gqa", 0, 1)
    step = TreeVerifyStep(2, S, V, 4, D, s.Hq, s.Hkv, s.d, s.d, s.cap, s.dt, False, s.scale, DEV)
    step.build(probs, root)
    q, k, v = step.rotate_tree(rope, *proj.split([s.Hq, s.Hkv, s.Hkv], 2), s.plen)
    torch.cuda.synchronize()
    a = angles(freq, (s.plen[:, None] + step.tree.depth)[None])
    y, size = plain(proj[:, :, : s.Hq].double(), rope.q_weight, a, s.d, False, True, float(torch.tensor(1e-6)), 1.0)
    assert ((q.double() - y).abs() <= 2.0 ** -8 * y.abs() + (s.d / 2 + 16) * 2.0 ** -24 * size).all()
    assert torch.equal(v, proj[:, :, s.Hq + s.Hkv:])


@gpu
def test_rotate_takes_a_raw_stream_handle():
    """As the calls around it do, also without buffers for the result; they belong to that stream."""
    s, step, cache, rope, freq, probs, root, logits, proj = _prepare("gqa", 0, 1)
    parts = proj.split([s.Hq, s.Hkv, s.Hkv], 2)
    want = [t.clone() for t in step.rotate_tree(rope, *parts, s.plen)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side.cuda_stream, side, torch.cuda.current_stream().cuda_stream):
        got = step.rotate_tree(rope, *parts, s.plen, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
