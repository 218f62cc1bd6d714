"""The step over an 8-bit cache: rounds against the calls they are made of, eager and
captured.  (The calls have their own checks against plain 64-bit code.)"""

import pytest
import torch

import tree_speculative_decoding_tsd_gb300 as T
from test_q8_cache import DEV, Setup
from tree_speculative_decoding_tsd_gb300.step import Q8Cache, Q8TreeVerifyStep, RowWeights

gpu = pytest.mark.gpu
SHAPE = (2, 4, 1000, 4, 8, 8, 2, 128, 128, 256, torch.bfloat16, False, 0.088)


@pytest.mark.parametrize("held", [dict(keep=252), dict(keep=-1), dict(keep=100, sink=-1),
                                  dict(keep=100, sink=60, recent=41), dict(keep=100, recent=-1),
                                  dict(keep=100, decay=1.5), dict(keep=100, decay=float("nan"))])
def test_step_rejects_budgets(held):
    with pytest.raises(ValueError):
        Q8TreeVerifyStep(*SHAPE, **held)


def _prepare(kind, page, keep):
    """A step, its state behind a prompt, and logits that accept a few tree rows."""
    S, D, V = 4, 8, 1000
    s = Setup(kind, 2, D + 1, [0, 0], extra=keep + S + 1, page=page, seed=5)
    step = Q8TreeVerifyStep(2, S, V, 4, D, s.Hq, s.Hkv, s.dk, s.dv, s.cap, s.dt, s.latent, s.scale,
                            DEV, keep=keep, sink=2, recent=8, decay=0.5)
    cache, weights = step.new_cache()
    if page:
        cache = Q8Cache(s.k, s.v, s.ke, s.ve, s.table, page)
    n = torch.tensor([keep - 3, keep // 2], dtype=torch.int32, device=DEV)
    x = s.normal(2, keep, s.Hkv, s.dk)
    y = None if s.latent else s.normal(2, keep, s.Hkv, s.dv)
    step.append(x, y, n, cache, s.plen)
    weights.pos.copy_(torch.arange(s.cap, device=DEV).int().expand_as(weights.pos))
    weights.seen.copy_(n[:, None].expand_as(weights.seen))
    probs = torch.softmax(torch.randn(2, S, V, generator=s.g, device=DEV) * 3, -1)
    root = torch.tensor([5, 9], dtype=torch.int32, device=DEV)
    step.build(probs, root)
    logits = torch.randn(2, D + 1, V, generator=s.g, device=DEV)
    for b in range(2):
        for r in range(1, D + 1):
            logits[b, int(step.tree.parent[b, r]), int(step.tree.token[b, r])] = 50.0
    return s, step, cache, weights, probs, root, logits


def _state(cache, weights, plen):
    return [t for t in (cache.kq, cache.vq, cache.kexp, cache.vexp, weights.acc, weights.pos,
                        weights.seen, plen) if t is not None]


def _same(got, want):
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@gpu
@pytest.mark.parametrize("kind,page", [("gqa", 0), ("latent", 128), ("narrow", 0)])
def test_step_rounds_are_their_calls(kind, page):
    keep = 150
    s, step, cache, weights, probs, root, logits = _prepare(kind, page, keep)
    lens = s.plen.tolist()
    for _ in range(3):
        for t in (s.q, s.kt, s.vt):
            if t is not None:
                t.copy_(s.normal(*t.shape))
        mine = [t.clone() for t in _state(cache, weights, s.plen)]
        s.k, s.v, s.ke, s.ve = mine[:4] if not s.latent else (mine[0], None, mine[1], None)
        acc, pos, seen, plen = mine[-4:]
        step.run(probs, root, s.q, cache, s.plen, s.kt, s.vt, logits, weights)
        torch.cuda.synchronize()
        # the attention against its plain form on the state before
        s.lens = plen.tolist()
        s.set_masks([[v & ((1 << 64) - 1) for v in m] for m in step.tree.mask.tolist()])
        s.check_attn(step.out, step.lse)
        # the rest against the calls in order
        w, page_args = step.walk, dict(page_table=cache.page_table, page_size=page)
        accepted = w.accept_len.tolist()
        assert all(0 < a <= 4 for a in accepted)
        T.tsd_cache_weights_q8(step.desc, 4, s.q, s.k, s.ke, plen, s.kt, w.accept_rows, w.accept_len,
                               step.lse, 0.5, acc, pos, seen, s.err, **page_args)
        T.tsd_commit_path_q8(step.desc, 4, s.kt, s.vt, w.accept_rows, w.accept_len, s.k, s.v, s.ke,
                             s.ve, plen, s.err, **page_args)
        T.tsd_cache_evict_q8(step.desc, keep, 2, 8, acc, pos, seen, s.k, s.v, s.ke, s.ve, plen,
                             T.workspace(T.tsd_cache_evict_workspace_size(step.desc)), s.err,
                             **page_args)
        _same(_state(cache, weights, s.plen), mine)
        lens = [min(n + a + 1, keep) for n, a in zip(lens, accepted)]
        assert s.plen.tolist() == lens
    assert int(step.err[0]) == 0 and int(s.err) == 0


@gpu
@pytest.mark.parametrize("kind", ["gqa", "latent"])
def test_step_captured_is_eager(kind):
    keep = 150
    s, step, cache, weights, probs, root, logits = _prepare(kind, 0, keep)
    start = [t.clone() for t in _state(cache, weights, s.plen)]
    args = (probs, root, s.q, cache, s.plen, s.kt, s.vt, logits, weights)
    eager = []
    for _ in range(3):
        step.run(*args)
        eager.append([t.clone() for t in [step.out, step.lse] + _state(cache, weights, s.plen)])
    graph = step.capture(*args)
    torch.cuda.synchronize()
    for t, u in zip(_state(cache, weights, s.plen), start):
        t.copy_(u)
    torch.cuda.synchronize()
    for want in eager:
        graph.replay()
        _same([step.out, step.lse] + _state(cache, weights, s.plen), want)
    assert int(step.err[0]) == 0


@gpu
def test_step_without_a_budget_grows_and_takes_no_weights():
    s, held, _, weights, probs, root, logits = _prepare("gqa", 0, 40)
    step = Q8TreeVerifyStep(2, 4, 1000, 4, 8, s.Hq, s.Hkv, s.dk, s.dv, s.cap, s.dt, False, s.scale, DEV)
    cache, none = step.new_cache()
    assert none is None and isinstance(weights, RowWeights)
    s.plen.zero_()
    step.run(probs, root, s.q, cache, s.plen, s.kt, s.vt, logits)
    assert s.plen.tolist() == [a + 1 for a in step.walk.accept_len.tolist()]
    with pytest.raises(ValueError):
        step.run(probs, root, s.q, cache, s.plen, s.kt, s.vt, logits, weights)
    with pytest.raises(ValueError):
        held.run(probs, root, s.q, cache, s.plen, s.kt, s.vt, logits)
    with pytest.raises(NotImplementedError):
        step.accept_commit()
    assert int(step.err[0]) == 0
