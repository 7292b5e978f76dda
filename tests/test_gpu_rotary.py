"""GPU parity of kvq_norm_rotary against its definition in float64.

Tolerance per element: half a step of the output type relative to the value, plus 2^-17 of the pair's length: the sum of 128
squares in fp32 is off by at most 128 2^-24, its root by half of that, the four products and sums by 2^-24 each, and the angle
(fp64, reduced to a turn, then fp32) by 2^-25 turns, sincospi by a few 2^-24; plus the types' smallest step.
"""
import numpy as np
import pytest
import torch

from oracle import operators_oracle as oo
from tests import kvq_testlib as tl

pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def _cache(d, hq, hkv, lens, max_tokens=1 << 20):
    K = tl.kvq()
    # a cache of the smallest blocks: only its lengths are used
    cache = K.KVQCache(K.CacheSpec(2, 2, 64, d, hq, hkv, len(lens), max(max(lens) + 64, 64) if max_tokens is None else max_tokens))
    cache.device_lengths().copy_(torch.tensor(lens, dtype=torch.int32))
    cache.sync_lengths()
    return cache


def _inv_freq(pairs, base=10000.0):
    return (base ** (-np.arange(pairs) / pairs)).astype(np.float32)


def _values(t):
    return t.double().cpu().numpy()


def _compare(got, want, x_norm, out_dtype):
    t = TYPES[out_dtype]
    tol = torch.finfo(t).eps / 2 * np.abs(want) + 2.0 ** -17 * x_norm + torch.finfo(t).smallest_normal * torch.finfo(t).eps
    off = np.abs(_values(got) - want)
    assert (off <= tol).all(), ((off / tol).max(), np.argwhere(off > tol)[:3])


def _check(cache, qkv, hq, hkv, n_new, lens, inv_freq, qw=None, kw=None, eps=1e-6, positions=None, sections=None,
           interleaved=False, out_dtype="fp16", got=None):
    x = qkv.view(qkv.shape[0], hq + 2 * hkv, -1)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if got is None:
        got = cache.norm_rotary(q, k, v, n_new, torch.from_numpy(inv_freq).cuda(), q_weight=qw, k_weight=kw, eps=eps,
                                positions=positions, sections=sections, interleaved=interleaved, out_dtype=TYPES[out_dtype])
    torch.cuda.synchronize()
    if positions is None:
        pos = np.concatenate([lens[b] + np.arange(m) for b, m in enumerate(n_new)] or [np.zeros(0)])[None]
    else:
        pos = positions.cpu().numpy().reshape(-1, x.shape[0])
    P = len(inv_freq)
    for t, y, w in ((got[0], q, qw), (got[1], k, kw)):
        w = None if w is None else _values(w)
        want = oo.norm_rotary(_values(y), pos, inv_freq, sections, w, eps, interleaved)
        sq = want ** 2
        if interleaved:
            sq[..., :2 * P] = np.repeat(sq[..., :2 * P:2] + sq[..., 1:2 * P:2], 2, -1)
        else:
            sq[..., :P] += sq[..., P:2 * P]
            sq[..., P:2 * P] = sq[..., :P]
        assert t.is_contiguous() and t.dtype == TYPES[out_dtype]
        _compare(t, want, np.sqrt(sq), out_dtype)
    assert torch.equal(got[2], v.to(TYPES[out_dtype]))
    return got


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("out", ["fp16", "bf16", "fp32"])
def test_types(d, dt, out):
    hq, hkv, lens, n_new = 6, 2, [0, 5, 70000, 1000], [1, 0, 3, 9]
    g = torch.Generator("cuda").manual_seed(1)
    qkv = torch.randn((13, (hq + 2 * hkv) * d), generator=g, device="cuda").to(TYPES[dt])
    qw, kw = ((1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(TYPES[dt]) for _ in range(2))
    _check(_cache(d, hq, hkv, lens), qkv, hq, hkv, n_new, lens, _inv_freq(d // 2), qw, kw, out_dtype=out)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("pairs", [1, 3, 8, 12, 16, 31, 32, 64])
@pytest.mark.parametrize("norm", [False, True])
def test_parts_of_a_head(pairs, interleaved, norm):
    d, hq, hkv, lens, n_new = (128 if pairs > 32 else 64), 3, 1, [17, 999999], [5, 2]
    g = torch.Generator("cuda").manual_seed(pairs)
    qkv = torch.randn((7, (hq + 2 * hkv) * d), generator=g, device="cuda").half()
    w = (torch.rand(d, generator=g, device="cuda") + 0.5).half() if norm else None
    _check(_cache(d, hq, hkv, lens), qkv, hq, hkv, n_new, lens, _inv_freq(pairs), w, None, interleaved=interleaved)


@pytest.mark.parametrize("sections", [[64], [16, 24, 24], [0, 40, 24], [64, 0, 0], [1, 2, 60, 1]])
def test_axes(sections):
    d, hq, hkv, n = 128, 5, 5, 11
    g = torch.Generator("cuda").manual_seed(len(sections))
    qkv = torch.randn((n, (hq + 2 * hkv) * d), generator=g, device="cuda").bfloat16()
    pos = torch.randint(-5, 1 << 20, (len(sections), n), generator=g, device="cuda", dtype=torch.int32)
    pos[0, 0] = 2 ** 31 - 1
    _check(_cache(d, hq, hkv, [3]), qkv, hq, hkv, [n], [3], _inv_freq(64), positions=pos, sections=sections)


@pytest.mark.parametrize("rows", [1, 148, 1023, 1024, 5000])
def test_row_counts(rows):
    """Both sides of the rule that spreads a row's heads over several blocks."""
    d, hq, hkv = 128, 32, 8
    g = torch.Generator("cuda").manual_seed(rows)
    qkv = torch.randn((rows, (hq + 2 * hkv) * d), generator=g, device="cuda").half()
    w = (torch.rand(d, generator=g, device="cuda") + 0.5).half()
    n_new = [rows // 3, rows - rows // 3]
    _check(_cache(d, hq, hkv, [100, 7]), qkv, hq, hkv, n_new, [100, 7], _inv_freq(64, 500000.0), w, w)


def test_many_sequences():
    d, hq, hkv = 64, 2, 1
    rng = np.random.default_rng(2)
    lens, n_new = [int(x) for x in rng.integers(0, 5000, 1100)], [int(x) for x in rng.integers(0, 3, 1100)]
    qkv = torch.randn((sum(n_new), 4 * d), device="cuda").half()
    _check(_cache(d, hq, hkv, lens, None), qkv, hq, hkv, n_new, lens, _inv_freq(32))


def test_separate_arrays_strides_and_no_values():
    d, hq, hkv, n = 64, 4, 2, 6
    cache = _cache(d, hq, hkv, [9])
    big = torch.randn((n, 1024), device="cuda").half()
    q, k = big[:, 64:64 + hq * d].view(n, hq, d), torch.randn((2 * n, hkv, d), device="cuda").half()[::2]
    f = torch.from_numpy(_inv_freq(32)).cuda()
    got = cache.norm_rotary(q, k, None, [n], f)
    assert got[2] is None
    qkv = torch.cat([q.reshape(n, -1), k.reshape(n, -1), k.reshape(n, -1)], 1)
    _check(cache, qkv, hq, hkv, [n], [9], _inv_freq(32), got=(got[0], got[1], k))
    out = [torch.full((n + 2, h, d), 5.0, dtype=torch.float16, device="cuda") for h in (hq, hkv, hkv)]
    cache.norm_rotary(q, k, k, [n], f, out=[t[:n] for t in out])
    assert torch.equal(out[0][:n], got[0]) and all((t[n:] == 5.0).all() for t in out)


def test_zero_rows_and_special_values():
    d, hq, hkv = 64, 2, 1
    cache = _cache(d, hq, hkv, [4])
    f = torch.from_numpy(_inv_freq(32)).cuda()
    x = torch.zeros((3, 4, d), device="cuda")
    x[1, 0, 3], x[2, 1, 40] = float("inf"), float("nan")
    q, k, _ = cache.norm_rotary(x[:, :2], x[:, 2:3], None, [3], f, out_dtype=torch.float32)
    assert (q[0] == 0).all() and (k == 0).all()
    bad = ~torch.isfinite(q)
    assert bad[1, 0, 3] and bad[1, 0, 35] and bad[2, 1, 8] and bad[2, 1, 40] and bad.sum() == 4
    w = torch.ones(d, device="cuda")
    assert (cache.norm_rotary(x[:1, :2], x[:1, 2:3], None, [1], f, q_weight=w, out_dtype=torch.float32)[0] == 0).all()
    e = torch.empty((0, 4, d), device="cuda")
    assert cache.norm_rotary(e[:, :2], e[:, 2:3], e[:, 3:], [0], f)[0].shape == (0, 2, d)


def test_python_refusals():
    K = tl.kvq()
    cache = _cache(64, 2, 1, [4], 64)
    f = torch.ones(32, device="cuda")
    x = torch.zeros((3, 4, 64), device="cuda").half()
    q, k, v = x[:, :2], x[:, 2:3], x[:, 3:]
    p = torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    for bad in (lambda: cache.norm_rotary(q, k.float(), v, [3], f), lambda: cache.norm_rotary(q, k, v, [2], f),
                lambda: cache.norm_rotary(q.double(), k.double(), v.double(), [3], f),
                lambda: cache.norm_rotary(q, k, v, [3], f.half()), lambda: cache.norm_rotary(q, k, v, [3], f[None]),
                lambda: cache.norm_rotary(q, k, v, [3], f, q_weight=f[:5].half()),
                lambda: cache.norm_rotary(q, k, v, [3], f, k_weight=torch.ones(64, device="cuda")),
                lambda: cache.norm_rotary(q, k, v, [3], f, positions=p), lambda: cache.norm_rotary(q, k, v, [3], f, sections=[32]),
                lambda: cache.norm_rotary(q, k, v, [3], f, positions=p[:, :2], sections=[16, 16]),
                lambda: cache.norm_rotary(q, k, v, [3], f, positions=p.long(), sections=[16, 16]),
                lambda: cache.norm_rotary(x.view(3, 2, 2, 64)[:, :, 0], k, v, [3], f),
                lambda: cache.norm_rotary(q, k, v, [3], f, out=[torch.empty_like(q), None, torch.empty_like(v)]),
                lambda: cache.norm_rotary(q.cpu(), k, v, [3], f)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: cache.norm_rotary(q, k, v, [3], f, positions=p, sections=[16, 15]),
                lambda: cache.norm_rotary(q, k, v, [3], f, eps=-1.0),
                lambda: cache.norm_rotary(x.view(-1)[4:4 + 512].view(2, 4, 64)[:, :2], k[:2], v[:2], [2], f)):
        with pytest.raises(K.KvqError):
            bad()


def test_captured_call_follows_the_lengths():
    d, hq, hkv, n = 128, 4, 2, 2
    K = tl.kvq()
    cache = K.KVQCache(K.CacheSpec(4, 2, 32, d, hq, hkv, 1, 256))
    qkv = torch.randn((n, (hq + 2 * hkv) * d), device="cuda").half()
    x = qkv.view(n, hq + 2 * hkv, d)
    inv = _inv_freq(64)
    f = torch.from_numpy(inv).cuda()
    out = [torch.zeros((n, h, d), dtype=torch.float16, device="cuda") for h in (hq, hkv, hkv)]

    def step():
        cache.norm_rotary(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], [n], f, out=out)
        cache.append(out[1], out[2], [n])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for i in range(1, 20):
        graph.replay()
        torch.cuda.synchronize()
        _check(cache, qkv, hq, hkv, [n], [n * i], inv, got=out)


def _guarded(cache, qkv, hq, hkv, n_new, lens, inv_freq, out_dtype, **kw):
    """_check into outputs with two rows behind the last, which stay as they were."""
    n, d = qkv.shape[0], cache.spec.head_dim
    x = qkv.view(n, hq + 2 * hkv, d)
    out = [torch.full((n + 2, h, d), 5.0, dtype=TYPES[out_dtype], device="cuda") for h in (hq, hkv, hkv)]
    names = dict(qw="q_weight", kw="k_weight")
    got = cache.norm_rotary(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], n_new, torch.from_numpy(inv_freq).cuda(),
                            out_dtype=TYPES[out_dtype], out=[t[:n] for t in out], **{names.get(k, k): v for k, v in kw.items()})
    _check(cache, qkv, hq, hkv, n_new, lens, inv_freq, out_dtype=out_dtype, got=got, **kw)
    assert all((t[n:] == 5.0).all() for t in out)


# kinds of call, each over rows on both sides of the rule that gives a block several rows (148 blocks of 8 rows of 16-bit types, of
# 4 rows of fp32) and over last blocks of every fill
KINDS = [dict(d=128, P=64), dict(d=64, P=32, interleaved=True), dict(d=64, P=31), dict(d=128, P=24, sections=[8, 10, 6]),
         dict(d=128, P=37, sections=[12, 25], norm=False), dict(d=128, P=20, interleaved=True, sections=[3, 17])]


@pytest.mark.parametrize("kind", KINDS, ids=str)
@pytest.mark.parametrize("dt,rows", [("fp16", 1183), ("bf16", 1184), ("fp16", 1185), ("bf16", 1191), ("fp16", 2006), ("fp32", 591),
                                     ("fp32", 592), ("fp32", 593), ("fp32", 595), ("fp32", 1202)])
def test_blocks_of_several_rows(dt, rows, kind):
    d, P = kind["d"], kind["P"]
    hq, hkv = (30, 5) if d == 64 else (12, 3)    # (40 and 18 heads: two passes of 32 and 16, the second not full)
    g = torch.Generator("cuda").manual_seed(rows + P)
    qkv = torch.randn((rows, (hq + 2 * hkv) * d), generator=g, device="cuda").to(TYPES[dt])
    qw, kw = ((torch.rand(d, generator=g, device="cuda") + 0.5).to(TYPES[dt]) if kind.get("norm", True) else None for _ in range(2))
    # short sequences, several to a block, and empty ones
    rng = np.random.default_rng(rows)
    n_new = []
    while sum(n_new) < rows:
        n_new.append(min(int(rng.choice([0, 1, 2, 3, 7, 60])), rows - sum(n_new)))
    lens = [int(x) for x in rng.integers(0, 20000, len(n_new))]
    pos = None
    if "sections" in kind:
        pos = torch.randint(0, 1 << 20, (len(kind["sections"]), rows), generator=g, device="cuda", dtype=torch.int32)
    for out in ("fp16", "fp32"):
        _guarded(_cache(d, hq, hkv, lens, None), qkv, hq, hkv, n_new, lens, _inv_freq(P), out, qw=qw, kw=kw, positions=pos,
                 sections=kind.get("sections"), interleaved=kind.get("interleaved", False))


def test_outputs_on_another_stream():
    """A call on a stream of its own, while the current one still reads memory that tensors have given back: the new outputs are
    not put there."""
    d, hq, hkv, n = 64, 4, 4, 30
    cache = _cache(d, hq, hkv, [9])
    qkv = torch.randn((n, 12 * d), device="cuda").half()
    x, f = qkv.view(n, 12, d), torch.from_numpy(_inv_freq(32)).cuda()
    kept, side = torch.empty((12, n, hq, d), dtype=torch.float16, device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        held = [torch.full_like(kept[0], 3.0) for _ in range(12)]
        torch.cuda._sleep(50_000_000)           # (some 30 ms of the current stream)
        for i in range(12):
            kept[i].copy_(held[i])
        del held
        got = cache.norm_rotary(x[:, :hq], x[:, hq:2 * hq], x[:, 2 * hq:], [n], f, stream=side)
        torch.cuda.synchronize()
        assert (kept == 3.0).all()
        _check(cache, qkv, hq, hkv, [n], [9], _inv_freq(32), got=got)
