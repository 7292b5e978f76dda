"""GPU tests of kvq_reorder: the bytes of every sequence afterwards are those of the oracle's cache for the history that it took
over, and what the call does not move is left alone."""
import numpy as np
import pytest
import torch

from oracle import operators_oracle as oo
from tests import kvq_testlib as tl

pytestmark = pytest.mark.gpu


def _hist(rng, lens, hkv, d):
    return [[rng.standard_normal((n, hkv, d)).astype(np.float16) for n in lens] for _ in range(2)]


def _cache(lens, kb=4, vb=2, G=32, d=64, hkv=2, max_tokens=512, seed=0, **kw):
    spec = tl.kvq().CacheSpec(kb, vb, G, d, 2 * hkv, hkv, len(lens), max_tokens, **kw)
    cache = tl.kvq().KVQCache(spec)
    ks, vs = _hist(np.random.default_rng(seed), lens, hkv, d)
    tl.append_chunks(cache, ks, vs, "fp16")
    return cache, ks, vs


MAPS = [[1, 0, 2, 3, 4, 5], [0, 0, 0, 0, 0, 0], [5, 0, 1, 2, 3, 4], [1, 2, 3, 4, 5, 0], [0, 1, 2, 3, 4, 5], [2, 2, 2, 5, 5, 3],
        [1, 1, 1], [3, 4, 0, 0, 0, 0]]


@pytest.mark.parametrize("parent", MAPS, ids=str)
@pytest.mark.parametrize("kw", [dict(), dict(kb=2, vb=4, G=64, d=128), dict(window=48, sink=5), dict(G=64, window=16, sink=33)],
                         ids=str)
def test_bytes_after_a_reordering(parent, kw):
    lens = [200, 33, 1, 470, 64, 100]
    cache, ks, vs = _cache(lens, **kw)
    cache.reorder(parent)
    torch.cuda.synchronize()
    tl.check_cache_against_oracle(cache, oo.reorder(ks, parent), oo.reorder(vs, parent))
    # and again, and the sequences go on from there
    cache.reorder(parent)
    ks, vs = (oo.reorder(oo.reorder(x, parent), parent) for x in (ks, vs))
    more = _hist(np.random.default_rng(1), [7] * 6, ks[0].shape[1], ks[0].shape[2])
    tl.append_chunks(cache, more[0], more[1], "fp16")
    torch.cuda.synchronize()
    tl.check_cache_against_oracle(cache, [np.concatenate(p) for p in zip(ks, more[0])],
                                  [np.concatenate(p) for p in zip(vs, more[1])])


@pytest.mark.parametrize("n", [9, 20, 70])
@pytest.mark.parametrize("kind", ["cycle", "random"])
def test_long_chains(n, kind):
    rng = np.random.default_rng(n)
    lens = [int(x) for x in rng.integers(0, 130, n)]
    cache, ks, vs = _cache(lens, max_tokens=128 + 2)
    order = rng.permutation(n)
    parent = [0] * n
    for i in range(n):
        parent[order[i]] = int(order[(i + 1) % n]) if kind == "cycle" else int(rng.integers(n))
    cache.reorder(parent)
    torch.cuda.synchronize()
    tl.check_cache_against_oracle(cache, oo.reorder(ks, parent), oo.reorder(vs, parent))


def test_many_sequences_take_several_launches():
    n = 1200
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(0, 40, n)]
    cache, ks, vs = _cache(lens, hkv=1, max_tokens=40)
    order = [int(x) for x in rng.permutation(n)]
    parent = [0] * n
    for i in range(n):
        parent[order[i]] = order[(i + 1) % n]
    cache.reorder(parent)
    torch.cuda.synchronize()
    check = [0, 1, 2, 511, 512, 600, 1023, 1024, 1199] + order[:20] + order[500:520]
    tl.check_cache_against_oracle(cache, oo.reorder(ks, parent), oo.reorder(vs, parent), seqs=check)
    assert cache.device_lengths().tolist() == oo.reorder(lens, parent) == cache.lengths()


def test_empty_sequences():
    cache, ks, vs = _cache([0, 50, 0])
    cache.reorder([1, 0, 2])
    torch.cuda.synchronize()
    assert cache.lengths() == [50, 0, 0] == cache.device_lengths().tolist()
    tl.check_cache_against_oracle(cache, [ks[1], ks[0], ks[2]], [vs[1], vs[0], vs[2]])


@pytest.mark.parametrize("window,sink", [(0, 0), (64, 0), (0, 40), (32, 7)])
def test_shared_tokens(window, sink):
    """A prompt forked, different tokens appended, and beams that follow others: with the prompt declared shared."""
    prompt, beams, G = 150, 4, 32
    cache, ks, vs = _cache([prompt] + [0] * (beams - 1), window=window, sink=sink)
    cache.reorder([0] * beams)
    ks, vs = [ks[0]] * beams, [vs[0]] * beams
    rng = np.random.default_rng(2)
    for step, parent in enumerate([[1, 1, 0, 3], [0, 0, 0, 0], [3, 2, 1, 0], [0, 2, 2, 1], [1, 2, 3, 0]]):
        more = _hist(rng, [9 + step] * beams, 2, 64)
        tl.append_chunks(cache, more[0], more[1], "fp16")
        ks, vs = ([np.concatenate(p) for p in zip(x, m)] for x, m in ((ks, more[0]), (vs, more[1])))
        before = cache.buffer.clone()
        cache.reorder(parent, shared=prompt)
        torch.cuda.synchronize()
        ks, vs = oo.reorder(ks, parent), oo.reorder(vs, parent)
        tl.check_cache_against_oracle(cache, ks, vs)
        L = cache.layout                        # the shared groups are not touched
        kept = max(0, prompt - sink - window) // G * L["block_bytes"]
        for b in range(beams):
            for h in range(2):
                at = L["blocks_offset"] + (b * 2 + h) * L["max_groups"] * L["block_bytes"]
                assert torch.equal(before[at:at + kept], cache.buffer[at:at + kept])


def test_shared_tokens_that_one_side_holds_in_fp16():
    """The shorter sequence still has in its fp16 tail what the longer one has quantized."""
    G, R, shared = 32, 64, 128
    rng = np.random.default_rng(4)
    ks, vs = _hist(rng, [140, 400], 2, 64)
    for x in (ks, vs):
        x[1][:shared] = x[0][:shared]
    for parent in ([1, 1], [0, 0], [1, 0]):
        cache = tl.kvq().KVQCache(tl.kvq().CacheSpec(4, 2, G, 64, 4, 2, 2, 512, window=R))
        tl.append_chunks(cache, ks, vs, "fp16")
        cache.reorder(parent, shared=shared)
        torch.cuda.synchronize()
        tl.check_cache_against_oracle(cache, oo.reorder(ks, parent), oo.reorder(vs, parent))


def test_position_adaptive_widths():
    """Groups at both widths move with their sequence; nothing is shared between sequences of different lengths."""
    from tests.test_gpu_akvq import _append_schedule, _check_bytes, _hist as hist
    spec = tl.kvq().CacheSpec(4, 2, 32, 64, 4, 2, 3, 1024, akvq_delta=64)
    cache = tl.kvq().KVQCache(spec)
    ks, vs = hist(np.random.default_rng(5), [500, 333, 333], 2, 64)
    chunks = _append_schedule(cache, ks, vs, [[400, 100], [300, 33], [40, 293]])
    for k in (ks, vs):
        k[1][:32] = k[1][:32]
    cache.reorder([1, 2, 0])
    torch.cuda.synchronize()
    ks, vs, chunks = (oo.reorder(x, [1, 2, 0]) for x in (ks, vs, chunks))
    for b in range(3):
        _check_bytes(cache, tl.oracle_cfg(spec), ks[b], vs[b], chunks[b], b)


def test_nothing_else_is_written():
    lens = [100, 200, 50, 70]
    cache, _, _ = _cache(lens, max_tokens=256, window=16, sink=4)
    before = cache.buffer.clone()
    cache.reorder([2, 1, 2, 3])
    torch.cuda.synchronize()
    L, H = cache.layout, 2
    same = before == cache.buffer
    same[L["lens_offset"]:L["lens_offset"] + 4] = True
    for h in range(H):
        at = L["blocks_offset"] + h * L["max_groups"] * L["block_bytes"]
        same[at:at + (50 - 4 - 16) // 32 * L["block_bytes"]] = True
        for name in ("tail", "sink"):
            at = L[name + "s_offset"] + h * L[name + "_bytes"]
            same[at:at + L[name + "_bytes"]] = True
    assert same.all()


def test_captured_reordering_follows_the_lengths():
    cache, ks, vs = _cache([40, 70], max_tokens=256)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        cache.reorder([1, 0])
    cache.sync_lengths()
    assert cache.lengths() == [40, 70]
    more = _hist(np.random.default_rng(6), [100, 3], 2, 64)
    tl.append_chunks(cache, more[0], more[1], "fp16")
    ks, vs = ([np.concatenate(p) for p in zip(x, m)] for x, m in ((ks, more[0]), (vs, more[1])))
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        cache.sync_lengths()
        ks, vs = ks[::-1], vs[::-1]
        tl.check_cache_against_oracle(cache, ks, vs)


def test_a_beam_search_step_by_step():
    """The operators together as a program runs them: the projection's rows normed and rotated at the cache's positions,
    appended, attended with capped scores, and the beams reordered; the outputs against float64 all the way."""
    K = tl.kvq()
    d, hq, hkv, beams, prompt = 64, 4, 2, 3, 70
    spec = K.CacheSpec(4, 2, 32, d, hq, hkv, beams, 256)
    cache = K.KVQCache(spec)
    inv = (10000.0 ** (-np.arange(32) / 32)).astype(np.float32)
    f = torch.from_numpy(inv).cuda()
    g = torch.Generator("cuda").manual_seed(11)
    w = (torch.rand(d, generator=g, device="cuda") + 0.5).half()
    hk, hv = [np.zeros((0, hkv, d), np.float16)] * beams, [np.zeros((0, hkv, d), np.float16)] * beams
    for step, (n_new, parent) in enumerate([([prompt, 0, 0], [0, 0, 0]), ([1] * 3, [1, 1, 2]), ([1] * 3, [2, 0, 1]),
                                            ([2] * 3, [0, 0, 1]), ([40] * 3, [2, 2, 2])]):
        x = torch.randn((sum(n_new), hq + 2 * hkv, d), generator=g, device="cuda").half()
        q, k, v = cache.norm_rotary(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], n_new, f, q_weight=w, k_weight=w)
        cache.append(k, v, n_new)
        out = cache.attend(q, n_new, cap=20.0, window=60, prefix=torch.full((3,), 8, dtype=torch.int32, device="cuda"))
        cache.reorder(parent, shared=prompt if step else 0)
        torch.cuda.synchronize()
        row = 0
        for b, m in enumerate(n_new):
            sl = slice(row, row + m)
            pos = (hk[b].shape[0] + np.arange(m))[None]
            for got, part, y in ((q, x[sl, :hq], None), (k, x[sl, hq:hq + hkv], None)):
                want = oo.norm_rotary(part.double().cpu().numpy(), pos, inv, weight=w.double().cpu().numpy(), eps=1e-6)
                assert np.abs(got[sl].double().cpu().numpy() - want).max() <= 2.0 ** -11 * np.abs(want).max() + 2.0 ** -15 if m else True
            hk[b] = np.concatenate([hk[b], k[sl].cpu().numpy()])
            hv[b] = np.concatenate([hv[b], v[sl].cpu().numpy()])
            if m:
                want, tol = oo.attend(tl.oracle_cfg(spec), hk[b], hv[b], q[sl].float().cpu().numpy(), cap=20.0, window=60, prefix=8)
                assert (np.abs(out[sl].double().cpu().numpy() - want) <= tol).all(), (step, b)
            row += m
        hk, hv = oo.reorder(hk, parent), oo.reorder(hv, parent)
        tl.check_cache_against_oracle(cache, hk, hv)


def test_python_refusals():
    K = tl.kvq()
    cache, _, _ = _cache([10, 20])
    for bad in (lambda: cache.reorder([2, 0]), lambda: cache.reorder([1, 0], shared=11), lambda: cache.reorder([0, 0, 0])):
        with pytest.raises(K.KvqError):
            bad()
    assert cache.lengths() == [10, 20] == cache.device_lengths().tolist()


@pytest.mark.parametrize("n,parent", [(333, [1, 1, 2]), (333, [1, 0, 0]), (500, [1, 1, 2]), (500, [1, 0, 0])])
def test_shared_groups_of_adaptive_widths(n, parent):
    """A prefix of 300 tokens by the same appends.  Sequences of one length hold its groups in the same bytes, which stay where
    they are; sequences of different lengths hold some of them at different widths, and take over the other's."""
    from tests.test_gpu_akvq import _append_schedule, _check_bytes, _hist as hist
    G, shared = 32, 300
    spec = tl.kvq().CacheSpec(4, 2, G, 64, 4, 2, 3, 1024, akvq_delta=64)
    cfg, cache = tl.oracle_cfg(spec), tl.kvq().KVQCache(spec)
    ks, vs = hist(np.random.default_rng(n), [333, n, 333], 2, 64)
    for x in (ks, vs):
        x[1][:shared] = x[2][:shared] = x[0][:shared]
    chunks = _append_schedule(cache, ks, vs, [[shared, 33], [shared, n - shared], [shared, 20, 13]])
    from oracle import kvq_oracle as o
    bits = [o.akvq_cache_image(cfg, k, v, c)["bits"] for k, v, c in zip(ks, vs, chunks)]
    assert (n == 333) == (bits[0][:shared // G] == bits[1][:shared // G]) and {2, 4} <= set(bits[1][:shared // G])
    # a mark in group 1 of sequence 1: equal lengths leave the others' group alone, different ones take it over with the rest
    mark = cache.block_bytes(1, 0, 2)[1]
    was = mark[:16].clone()
    mark[:16] ^= 255
    cache.reorder(parent, shared=shared)
    torch.cuda.synchronize()
    if n == 333:
        assert torch.equal(cache.block_bytes(0, 0, 2)[1][:16], was)
        mark[:16] = was
    else:
        assert torch.equal(cache.block_bytes(0, 0, 2)[1][:16], was ^ 255)
        for b in range(3):
            if parent[b] == 1:
                cache.block_bytes(b, 0, 2)[1][:16] = was
    ks, vs, chunks = (oo.reorder(x, parent) for x in (ks, vs, chunks))
    for b in range(3):
        _check_bytes(cache, cfg, ks[b], vs[b], chunks[b], b)
    assert cache.lengths() == [len(k) for k in ks] == cache.device_lengths().tolist()
