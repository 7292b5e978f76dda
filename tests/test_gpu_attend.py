"""GPU parity of kvq_attend against float64 attention over the oracle's dequantized cache, within the tolerance that
``operators_oracle.attend`` derives for every element."""
import numpy as np
import pytest
import torch

from asymmetric_kv_cache_b200 import inputs
from oracle import operators_oracle as oo
from tests import kvq_testlib as tl

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["registers", "tensor cores"], autouse=True)
def kernel(request, monkeypatch):
    """Every test runs with either kernel taking every sequence (the library's choice: test_the_librarys_choice)."""
    monkeypatch.setenv("KVQ_ATTEND_TC", "1" if request.param == "tensor cores" else "0")


def _hist(rng, lens, hkv, d):
    ks = [inputs.keys_channel_outliers(rng, n, hkv, d).astype(np.float16) for n in lens]
    vs = [(inputs.values_token_norms(rng, n, hkv, d) * 3 + 0.1).astype(np.float16) for n in lens]
    return ks, vs


def _queries(rng, n_q, hq, d, dtype):
    q = rng.standard_normal((sum(n_q), hq, d)).astype(np.float32)
    return q.astype(np.float16).astype(np.float32) if dtype == "fp16" else tl.bf16_values(q) if dtype == "bf16" else q


def _filled(spec, ks, vs, chunks=None):
    """A cache holding the histories, appended in `chunks` (the same sizes for every sequence) or at once."""
    cache = tl.kvq().KVQCache(spec)
    if chunks is None:
        tl.append_chunks(cache, ks, vs, "fp16")
    else:
        at = 0
        for c in chunks:
            tl.append_chunks(cache, [k[at:at + c] for k in ks], [v[at:at + c] for v in vs], "fp16")
            at += c
    return cache


def _check(cache, spec, ks, vs, q, n_q, dtype="fp16", out=None, chunks=None, prefix=None, **kw):
    slopes = kw.get("slopes")
    dev = dict(kw)
    if slopes is not None:
        dev["slopes"] = torch.tensor(slopes, dtype=torch.float32, device="cuda")
    if prefix is not None:
        dev["prefix"] = torch.tensor(prefix, dtype=torch.int32, device="cuda")
    if out is None:
        out = cache.attend(tl.to_device(q, dtype), n_q, **dev)
    torch.cuda.synchronize()
    assert cache.workspace_status() == 0
    got = out.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    cfg, row = tl.oracle_cfg(spec), 0
    for b, m in enumerate(n_q):
        if m == 0:
            continue
        want, tol = oo.attend(cfg, ks[b], vs[b], q[row:row + m], prefix=prefix[b] if prefix is not None else 0,
                              chunks=chunks, **kw)
        off = np.abs(got[row:row + m] - want)
        worst = (off / tol).max()
        assert worst <= 1.0, (b, m, ks[b].shape[0], worst, off.max(), np.unravel_index((off / tol).argmax(), off.shape))
        row += m
    return out


@pytest.mark.parametrize("kb,vb", [(4, 2), (2, 2), (4, 4), (2, 4)])
@pytest.mark.parametrize("d,G", [(64, 32), (64, 64), (128, 32), (128, 64)])
def test_every_layout(kb, vb, d, G):
    """One, some and many tokens over sequences from a single token to several groups, in one call."""
    hkv, gqa = 2, 4
    lens = [1, 7, G, G + 1, 3 * G + 5, 2 * G, 9 * G + 31]
    n_q = [1, 7, 3, 0, 1, 2 * G, 40]
    spec = tl.kvq().CacheSpec(kb, vb, G, d, hkv * gqa, hkv, len(lens), 1024)
    rng = np.random.default_rng(1000 * kb + 100 * vb + d + G)
    ks, vs = _hist(rng, lens, hkv, d)
    _check(_filled(spec, ks, vs), spec, ks, vs, _queries(rng, n_q, hkv * gqa, d, "fp16"), n_q)


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("hkv,gqa", [(1, 1), (3, 5), (2, 8), (1, 12), (1, 20)])
def test_head_counts_and_types(hkv, gqa, dtype):
    lens, n_q = [70, 3, 200], [5, 3, 1]
    spec = tl.kvq().CacheSpec(4, 2, 32, 128, hkv * gqa, hkv, 3, 256)
    rng = np.random.default_rng(hkv * 100 + gqa)
    ks, vs = _hist(rng, lens, hkv, 128)
    _check(_filled(spec, ks, vs), spec, ks, vs, _queries(rng, n_q, hkv * gqa, 128, dtype), n_q, dtype)


SCORES = [dict(cap=30.0), dict(cap=2.0), dict(window=1), dict(window=37), dict(window=64, prefix=[0, 4, 200, 70, 1]),
          dict(prefix=[1, 1000, 64, -5, 33]), dict(slopes=True), dict(slopes=True, cap=20.0, window=50, prefix=[3, 0, 7, 0, 90]),
          dict(scale=0.01), dict(scale=0.5, cap=10.0)]


@pytest.mark.parametrize("kw", SCORES, ids=str)
@pytest.mark.parametrize("d,G,R,S", [(128, 32, 0, 0), (64, 64, 48, 5), (128, 64, 16, 33)])
def test_scores(kw, d, G, R, S):
    hkv, gqa = 2, 4
    lens, n_q = [1, 60, 333, 200, 500], [1, 60, 5, 150, 2]
    kw = dict(kw)
    if kw.pop("slopes", False):
        kw["slopes"] = [2.0 ** -(i + 1) * (-1 if i == 5 else 1) for i in range(8)]
    spec = tl.kvq().CacheSpec(4, 2, G, d, hkv * gqa, hkv, 5, 512, window=R, sink=S)
    rng = np.random.default_rng(d + G + R)
    ks, vs = _hist(rng, lens, hkv, d)
    _check(_filled(spec, ks, vs), spec, ks, vs, _queries(rng, n_q, hkv * gqa, d, "fp16"), n_q, **kw)


@pytest.mark.parametrize("R,S", [(16, 0), (128, 0), (1024, 0), (0, 4), (0, 40), (64, 33)])
@pytest.mark.parametrize("G", [32, 64])
def test_recent_and_first_tokens(R, S, G):
    hkv, gqa, d = 2, 2, 128
    W = R + G
    lens = [1, max(1, S - 1), S + 1, S + R + 1, S + W - 1, S + W, S + W + 3 * G + 5]
    n_q = [1, 1, min(S + 1, 3), 1, 9, 12, W + G]
    spec = tl.kvq().CacheSpec(4, 2, G, d, hkv * gqa, hkv, len(lens), 2048, window=R, sink=S)
    rng = np.random.default_rng(R + S + G)
    ks, vs = _hist(rng, lens, hkv, d)
    n_q = [min(a, b) for a, b in zip(n_q, lens)]
    _check(_filled(spec, ks, vs), spec, ks, vs, _queries(rng, n_q, hkv * gqa, d, "bf16"), n_q, "bf16")


@pytest.mark.parametrize("d", [64, 128])
def test_rotating_cache(d):
    hkv, gqa = 2, 4
    lens, n_q = [5, 100, 260], [5, 1, 70]
    spec = tl.kvq().CacheSpec(4, 2, 32, d, hkv * gqa, hkv, 3, 512, rotate=1, sink=4)
    rng = np.random.default_rng(d)
    ks, vs = _hist(rng, lens, hkv, d)
    _check(_filled(spec, ks, vs), spec, ks, vs, _queries(rng, n_q, hkv * gqa, d, "fp16"), n_q, cap=30.0)


@pytest.mark.parametrize("d,G,vb", [(128, 32, 2), (64, 64, 4)])
def test_position_adaptive_widths(d, G, vb):
    hkv, gqa, delta = 2, 4, 2 * G
    chunks = [3 * G + 7, G, 5, 2 * G, 9 * G + 1]
    n = sum(chunks)
    spec = tl.kvq().CacheSpec(4, vb, G, d, hkv * gqa, hkv, 2, 2048, akvq_delta=delta)
    rng = np.random.default_rng(G)
    ks, vs = _hist(rng, [n, n], hkv, d)
    n_q = [1, 50]
    _check(_filled(spec, ks, vs, chunks), spec, ks, vs, _queries(rng, n_q, hkv * gqa, d, "fp16"), n_q, chunks=chunks)


@pytest.mark.parametrize("n,n_q,kw", [(20000, 1, {}), (20000, 3, dict(cap=30.0)), (9000, 1, dict(window=5000, prefix=[4])),
                                      (6000, 130, dict(window=300))])
def test_long_sequences_are_split_and_merged(n, n_q, kw):
    hkv, gqa, d = 2, 4, 128
    spec = tl.kvq().CacheSpec(2, 2, 32, d, hkv * gqa, hkv, 1, 20480, window=32)
    rng = np.random.default_rng(n + n_q)
    ks, vs = _hist(rng, [n], hkv, d)
    _check(_filled(spec, ks, vs), spec, ks, vs, _queries(rng, [n_q], hkv * gqa, d, "fp16"), [n_q], **kw)


def test_many_ragged_sequences():
    """More units than resident blocks, and more sequences than one launch takes."""
    hkv, gqa, d = 4, 2, 64
    rng = np.random.default_rng(4)
    lens = [int(x) for x in rng.integers(1, 90, size=600)]
    n_q = [int(rng.integers(0, min(n, 4) + 1)) for n in lens]
    spec = tl.kvq().CacheSpec(4, 2, 32, d, hkv * gqa, hkv, len(lens), 96)
    ks, vs = _hist(rng, lens, hkv, d)
    _check(_filled(spec, ks, vs), spec, ks, vs, _queries(rng, n_q, hkv * gqa, d, "fp16"), n_q)


@pytest.mark.parametrize("lens,n_q", [([3000, 70, 900], [300, 1, 20]), ([2500] * 3, [64, 130, 1])])
def test_the_librarys_choice(lens, n_q, monkeypatch):
    """Sequences of one call on either kernel, by the rows and keys that they have."""
    monkeypatch.delenv("KVQ_ATTEND_TC")
    hkv, gqa, d = 8, 4, 128
    spec = tl.kvq().CacheSpec(4, 2, 32, d, hkv * gqa, hkv, 3, 3200)
    rng = np.random.default_rng(len(lens) + n_q[0])
    ks, vs = _hist(rng, lens, hkv, d)
    _check(_filled(spec, ks, vs), spec, ks, vs, _queries(rng, n_q, hkv * gqa, d, "bf16"), n_q, "bf16", cap=50.0)


def test_agrees_with_decode():
    hkv, gqa, d = 8, 4, 128
    lens = [300, 4000, 31, 1025]
    spec = tl.kvq().CacheSpec(4, 2, 32, d, hkv * gqa, hkv, 4, 4096)
    rng = np.random.default_rng(9)
    ks, vs = _hist(rng, lens, hkv, d)
    cache = _filled(spec, ks, vs)
    q = tl.to_device(_queries(rng, [1] * 4, hkv * gqa, d, "fp16"), "fp16")
    a, b = cache.attend(q, [1] * 4), cache.decode(q)
    assert (a.float() - b.float()).abs().max().item() <= tl.DECODE_TOL      # each is within it of the exact result's half


def test_large_scores_and_equal_keys():
    """Scores of some hundreds (one key takes all), and keys all alike (the mean of the values)."""
    hkv, d, n = 1, 128, 150
    spec = tl.kvq().CacheSpec(4, 2, 32, d, 4, hkv, 2, 256)
    rng = np.random.default_rng(5)
    ks, vs = _hist(rng, [n, n], hkv, d)
    ks[0] = (ks[0].astype(np.float32) * 8).astype(np.float16)
    ks[1][:] = ks[1][:1]
    _check(_filled(spec, ks, vs), spec, ks, vs, _queries(rng, [4, 4], 4, d, "fp16"), [4, 4])


def test_rows_past_the_input_are_left_alone_and_zero_counts_skip():
    spec = tl.kvq().CacheSpec(4, 2, 32, 64, 4, 1, 3, 128)
    rng = np.random.default_rng(6)
    ks, vs = _hist(rng, [40, 50, 60], 1, 64)
    cache = _filled(spec, ks, vs)
    n_q = [3, 0, 10]
    q = _queries(rng, n_q, 4, 64, "fp16")
    buf = torch.full((20, 4, 64), 7.0, dtype=torch.float16, device="cuda")
    out = cache.attend(tl.to_device(q, "fp16"), n_q, out=buf[:13])
    _check(cache, spec, ks, vs, q, n_q, out=out)
    assert (buf[13:] == 7.0).all()
    assert cache.attend(torch.empty((0, 4, 64), dtype=torch.float16, device="cuda"), [0, 0, 0]).shape == (0, 4, 64)


def test_unused_tail_slots_may_hold_anything():
    """NaN in the slots that no token has reached."""
    spec = tl.kvq().CacheSpec(4, 2, 32, 64, 4, 1, 1, 128, window=32, sink=20)
    rng = np.random.default_rng(7)
    for n in (1, 19, 30, 81):
        cache = tl.kvq().KVQCache(spec)
        L = cache.layout
        cache.buffer[L["blocks_offset"]:].view(torch.float16).fill_(float("nan"))
        torch.cuda.synchronize()
        ks, vs = _hist(rng, [n], 1, 64)
        tl.append_chunks(cache, ks, vs, "fp16")
        m = min(n, 12)
        _check(cache, spec, ks, vs, _queries(rng, [m], 4, 64, "fp16"), [m])


def test_captured_call_follows_the_lengths():
    """append + attend captured once and replayed: out is of the newest tokens, across a group's end."""
    hkv, gqa, d, n0, m = 2, 4, 128, 61, 3
    spec = tl.kvq().CacheSpec(4, 2, 32, d, hkv * gqa, hkv, 2, 256)
    rng = np.random.default_rng(8)
    steps = 5
    ks, vs = _hist(rng, [n0 + m * (steps + 1)] * 2, hkv, d)
    cache = _filled(spec, [k[:n0] for k in ks], [v[:n0] for v in vs])
    prefix = torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    q = torch.zeros((2 * m, hkv * gqa, d), dtype=torch.float16, device="cuda")
    kin, vin = (torch.zeros((2 * m, hkv, d), dtype=torch.float16, device="cuda") for _ in range(2))
    out = torch.zeros_like(q)
    feed = lambda i: [tl.to_device(np.concatenate([x[b][n0 + i * m:n0 + (i + 1) * m] for b in range(2)]), "fp16")  # noqa: E731
                      for x in (ks, vs)]

    def step():
        cache.append(kin, vin, [m, m])
        cache.attend(q, [m, m], window=40, prefix=prefix, out=out)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):               # a first, eager step
        kin.copy_(feed(0)[0]), vin.copy_(feed(0)[1])
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for i in range(1, steps + 1):
        x = _queries(rng, [m, m], hkv * gqa, d, "fp16")
        q.copy_(tl.to_device(x, "fp16"))
        kin.copy_(feed(i)[0]), vin.copy_(feed(i)[1])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        n = n0 + (i + 1) * m
        got = out.clone()
        _check(cache, spec, [k[:n] for k in ks], [v[:n] for v in vs], x, [m, m], out=got, window=40, prefix=[2, 0])


def test_python_refusals():
    K = tl.kvq()
    cache = K.KVQCache(K.CacheSpec(4, 2, 32, 64, 4, 1, 2, 64))
    cache.append(*(torch.zeros((5, 1, 64), dtype=torch.float16, device="cuda") for _ in range(2)), [5])
    q = torch.zeros((2, 4, 64), dtype=torch.float16, device="cuda")
    f, i = (torch.zeros(4, dtype=t, device="cuda") for t in (torch.float32, torch.int32))
    for bad in (lambda: cache.attend(q.double(), [2]), lambda: cache.attend(q, [1]), lambda: cache.attend(q.cpu(), [2]),
                lambda: cache.attend(q.transpose(0, 1).contiguous().transpose(0, 1), [2]),
                lambda: cache.attend(q, [2], slopes=f[:3]), lambda: cache.attend(q, [2], slopes=f.half()),
                lambda: cache.attend(q, [2], prefix=i), lambda: cache.attend(q, [2], prefix=i[:1].long()),
                lambda: cache.attend(q, [2], out=q.float()), lambda: cache.attend(q, [2], out=q[:1]),
                lambda: cache.attend(q, [2], prefix=i[:1].cpu())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: cache.attend(q, [2], cap=-1.0), lambda: cache.attend(q, [1, 1]), lambda: cache.attend(q, [2], window=-3)):
        with pytest.raises(K.KvqError):
            bad()


@pytest.mark.parametrize("gqa,n_q,R", [(8, 1, 0), (4, 5, 0), (8, 40, 64), (2, 1, 32)])
def test_values_all_alike(gqa, n_q, R):
    """Rows whose values are all the number 2040 / 1024 are that number: the weights that the values meet and the weights that
    they are divided by are the same ones, as rounded.  (fp16 steps by 2^-10 there: a sum that is off by 2^-12 of itself moves
    the result; fp32 sums of the 700 same weights are off by 700 2^-24 = 2^-14.5 at most.)"""
    hkv, d, lens = 2, 128, [700, 70, 45]
    spec = tl.kvq().CacheSpec(4, 4, 32, d, hkv * gqa, hkv, 3, 1024, window=R)
    rng = np.random.default_rng(gqa + n_q)
    ks, vs = _hist(rng, lens, hkv, d)
    for k, v in zip(ks, vs):
        # one key takes weight 1, the others some weight between 0 and 1, the same for all of them
        k[:] = k[:1]
        k[len(k) // 2] = k[0] + rng.standard_normal(k[0].shape).astype(np.float16)
        v[:] = 2040 / 1024
    counts = [min(n, n_q) for n in lens]
    cache = _filled(spec, ks, vs)
    for _ in range(4):
        out = cache.attend(tl.to_device(_queries(rng, counts, hkv * gqa, d, "fp16"), "fp16"), counts)
        assert (out == 2040 / 1024).all(), (out != 2040 / 1024).float().mean().item()


def _wide(rng, lens, hkv, d, most):
    """Histories of which every third channel's keys and every fifth's values reach over most to -most in every group."""
    ks, vs = _hist(rng, lens, hkv, d)
    for x, step in ((ks, 3), (vs, 5)):
        for h in x:
            h[:, :, ::step] = rng.uniform(-most, most, h[:, :, ::step].shape).astype(np.float16)
            h[::7, :, ::step], h[3::7, :, ::step] = most, -most
    return ks, vs


@pytest.mark.parametrize("d,G", [(128, 32), (64, 64)])
@pytest.mark.parametrize("kb,vb,delta", [(4, 2, 0), (2, 4, 0), (4, 4, 64)])
@pytest.mark.parametrize("most", [40000, 65440])
def test_keys_and_values_over_all_of_fp16(kb, vb, delta, d, G, most):
    """Groups whose keys or values spread over more than 65504: 15 steps of the scale are no fp16 number then, the keys are."""
    hkv, gqa = 2, 4
    lens, n_q = [5 * G + 9, 9 * G, 40], [50, 1, 7]
    kw = dict(akvq_delta=delta) if delta else dict(window=16, sink=5)
    spec = tl.kvq().CacheSpec(kb, vb, G, d, hkv * gqa, hkv, 3, 1024, **kw)
    rng = np.random.default_rng(kb * 10 + vb + d + most)
    ks, vs = _wide(rng, lens, hkv, d, most)
    q = _queries(rng, n_q, hkv * gqa, d, "fp16") * 0.25
    cache = _filled(spec, ks, vs)
    for x in (dict(scale=2e-5), dict(scale=2e-5, cap=3.0, window=100)):
        for b in range(3):                      # (an adaptive cache's bytes are those of its own append)
            m = [n if i == b else 0 for i, n in enumerate(n_q)]
            part = q[sum(n_q[:b]):sum(n_q[:b + 1])]
            _check(cache, spec, ks, vs, part, m, chunks=[lens[b]] if delta else None, **x)


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("kb,vb,kw", [(2, 2, {}), (4, 2, dict(sink=4)), (4, 4, dict(akvq_delta=64)), (4, 2, dict(rotate=1))], ids=str)
@pytest.mark.parametrize("size,most", [(400.0, 300.0), (20000.0, 30.0), (60000.0, 40000.0)])
def test_large_queries_over_wide_keys(size, most, kb, vb, kw, dtype):
    """Queries of some hundreds to 60000 against channels whose quantization steps are large: query times step is no fp16 number,
    the score (with a scale that leaves it at a few units) is an ordinary one."""
    hkv, gqa, d = 2, 4, 128
    if kw.get("rotate"):
        size, most = size / 32, most / 16       # (a rotated row must still be fp16 numbers)
    lens, n_q = [200, 77, 130], [40, 1, 3]
    spec = tl.kvq().CacheSpec(kb, vb, 32, d, hkv * gqa, hkv, 3, 256, **kw)
    rng = np.random.default_rng(int(size) + kb)
    ks, _ = _wide(rng, lens, hkv, d, most)
    _, vs = _hist(rng, lens, hkv, d)
    q = rng.uniform(-size, size, (sum(n_q), hkv * gqa, d)).astype(np.float32)
    q[::3] /= 1000                              # and rows of ordinary size beside them
    q = q.astype(np.float16).astype(np.float32) if dtype == "fp16" else tl.bf16_values(q) if dtype == "bf16" else q
    cache = _filled(spec, ks, vs)
    for x in (dict(scale=1.0 / (size * most)), dict(scale=4.0 / (size * most), cap=2.0)):
        for b in range(3):
            m = [n if i == b else 0 for i, n in enumerate(n_q)]
            part = q[sum(n_q[:b]):sum(n_q[:b + 1])]
            _check(cache, spec, ks, vs, part, m, dtype, chunks=[lens[b]] if kw.get("akvq_delta") else None, **x)


def test_results_do_not_follow_what_unused_slots_hold():
    """The same tokens beside zeros, large numbers and NaN in the slots that no token has reached: the same bits."""
    spec = tl.kvq().CacheSpec(4, 2, 32, 64, 4, 1, 1, 128, window=32, sink=20)
    rng = np.random.default_rng(12)
    for n in (1, 5, 30, 81):
        ks, vs = _hist(rng, [n], 1, 64)
        q = tl.to_device(_queries(rng, [min(n, 3)], 4, 64, "fp16"), "fp16")
        outs = []
        for held in (0.0, 30000.0, float("nan")):
            cache = tl.kvq().KVQCache(spec)
            cache.buffer[cache.layout["blocks_offset"]:].view(torch.float16).fill_(held)
            torch.cuda.synchronize()
            tl.append_chunks(cache, ks, vs, "fp16")
            outs.append([cache.attend(q, [min(n, 3)], cap=cap).clone() for cap in (0.0, 50.0, 12.0)])
        for other in outs[1:]:
            assert all(torch.equal(a, b) for a, b in zip(outs[0], other)), n


def test_a_workspace_that_was_not_zeroed_is_reported(monkeypatch):
    """Tickets left over from something else: no block knows that it is the last one, so out is not written.  The call records
    it, and zeroing the workspace mends it."""
    monkeypatch.setenv("KVQ_ATTEND_TC", "0")
    hkv, gqa, d, n = 1, 4, 128, 2000
    spec = tl.kvq().CacheSpec(4, 2, 32, d, hkv * gqa, hkv, 1, 2048)
    rng = np.random.default_rng(13)
    ks, vs = _hist(rng, [n], hkv, d)
    cache = _filled(spec, ks, vs)
    x = _queries(rng, [1], hkv * gqa, d, "fp16")
    q = tl.to_device(x, "fp16")
    torch.cuda.synchronize()
    for held in (0.37, -2.5, 1e-40):
        cache.workspace[256:].view(torch.float32).fill_(held)
        cache.attend(q, [1])
        torch.cuda.synchronize()
        assert cache.workspace_status() == 10         # KVQ_ERR_DEVICE
        assert tl.kvq().kvq_last_error()
        cache.workspace.zero_()
        _check(cache, spec, ks, vs, x, [1])


@pytest.mark.parametrize("size", [1e3, 1e6, 2e7, 4e9])
@pytest.mark.parametrize("gqa,n_q", [(2, 1), (8, 1), (4, 40)])
def test_scores_of_any_size(size, gqa, n_q):
    """One key wins by far, by scores of some thousands to some billions, of either sign: its value is the result."""
    hkv, d, n = 1, 128, 300
    spec = tl.kvq().CacheSpec(4, 4, 32, d, hkv * gqa, hkv, 1, 320)
    rng = np.random.default_rng(int(size) % 1000 + gqa)
    ks = [np.full((n, hkv, d), -1.0, np.float16)]
    vs = [np.tile(rng.integers(-8, 8, (n, hkv, 1)), (1, 1, d)).astype(np.float16)]
    ks[0][200] = -0.5
    q = np.full((n_q, gqa, d), 1.0, np.float32)
    for sign in (1.0, -1.0):
        # (the other sign: all keys but one at the top would tie; the row of the one is turned round)
        k = [sign * ks[0] if sign > 0 else np.where(np.arange(n)[:, None, None] == 200, 1.0, 0.5) * np.ones((n, hkv, d))]
        k = [x.astype(np.float16) for x in k]
        cache = _filled(spec, k, vs)
        out = cache.attend(tl.to_device(q, "fp16"), [n_q], scale=size / d)
        torch.cuda.synchronize()
        late = n - n_q + np.arange(n_q) >= 200
        assert late.all() and (out.float().cpu().numpy() == float(vs[0][200, 0, 0])).all(), (sign, out.flatten()[:4])


@pytest.mark.parametrize("gqa,n_q", [(2, 1), (8, 1), (4, 40)])
def test_many_small_weights(gqa, n_q):
    """One key takes a weight of 1 and 2999 others between 2^-16 and 2^-25 each, and only those have a value.  A weight is fp16
    relative to 2^15 times the largest (tensor cores: to at least 2^7 times): off by 2^-11 of itself or by 2^-25 2^-15 (2^-7).
    The result is rounded (2^-11 of itself, 2^-25), and a score of up to 17.4 is off by 2^-17 times 3 times itself, twice in
    the result."""
    import os
    hkv, d, n = 1, 128, 3000
    spec = tl.kvq().CacheSpec(4, 2, 32, d, hkv * gqa, hkv, 1, 3008)
    ks, vs = [np.zeros((n, hkv, d), np.float16)], [np.full((n, hkv, d), 64.0, np.float16)]
    ks[0][n // 3, :, 0], vs[0][n // 3] = 8.0, 0.0
    cache = _filled(spec, ks, vs)
    q = np.zeros((n_q, gqa, d), np.float32)
    q[..., 0] = np.float16(np.linspace(11.0, 17.3, n_q * gqa).reshape(n_q, gqa) / 8.0)
    out = cache.attend(tl.to_device(q, "fp16"), [n_q], scale=1.0)
    want, _ = oo.attend(tl.oracle_cfg(spec), ks[0], vs[0], q, scale=1.0)
    least = 2.0 ** (-25 - (7 if os.environ["KVQ_ATTEND_TC"] == "1" else 15))
    off = np.abs(out.double().cpu().numpy() - want)
    tol = want * (2 * 2.0 ** -11 + 2 * 3 * 17.4 * 2.0 ** -17) + n * least * 64 + 2.0 ** -25
    assert (off <= tol).all(), ((off / tol).max(), (off / want).max())


def test_outputs_on_another_stream():
    """A call on a stream of its own, while the current one still reads memory that a tensor has given back: the new output is not
    put there."""
    hkv, gqa, d, n = 1, 4, 128, 40
    spec = tl.kvq().CacheSpec(4, 2, 32, d, hkv * gqa, hkv, 1, 64)
    rng = np.random.default_rng(14)
    ks, vs = _hist(rng, [n], hkv, d)
    cache = _filled(spec, ks, vs)
    x = _queries(rng, [n], hkv * gqa, d, "fp16")
    q = tl.to_device(x, "fp16")
    kept = torch.empty_like(q)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        held = torch.full_like(q, 3.0)
        torch.cuda._sleep(50_000_000)           # (some 30 ms of the current stream)
        kept.copy_(held)
        del held
        out = cache.attend(q, [n], stream=side)
        torch.cuda.synchronize()
        assert (kept == 3.0).all()
        _check(cache, spec, ks, vs, x, [n], out=out)
