"""attend, norm_rotary and reorder without a GPU: every refusal, the plans of their launches and the host mirror, on the
library's own host code with the launches recorded; and pins of the oracle's definitions."""
import ctypes
import itertools
import random

import numpy as np
import pytest

from oracle import kvq_oracle as o
from oracle import operators_oracle as oo
from tests import operators_testlib as ot


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    from asymmetric_kv_cache_b200 import build
    build.build()
    from asymmetric_kv_cache_b200 import kvq
    return ot.Host(ot.host_library(tmp_path_factory.mktemp("host")), kvq)


# ---------------------------------------------------------------- attend
OUT = ot.Host.PTR + (1 << 40)


def _attend(host, h, n_q, q=ot.Host.PTR, dt=0, out=OUT, ws=ot.Host.PTR, ws_bytes=None, n_seq=None, **sc):
    scores = host.kvq.KvqScores(**sc)
    return host.lib.kvq_attend(h, ctypes.c_void_p(q), dt, host.ints(n_q) if n_q is not None else None,
                               len(n_q or []) if n_seq is None else n_seq, ctypes.byref(scores), ctypes.c_void_p(out),
                               ctypes.c_void_p(ws), ctypes.c_size_t(host.ws if ws_bytes is None else ws_bytes), None)


def test_attend_refusals(host):
    h = host.cache([100, 1, 0, 300])
    H = host
    host.log()
    cases = [
        (dict(n_q=[1], q=0), H.NULL), (dict(n_q=[1], out=0), H.NULL), (dict(n_q=[1], ws=0), H.NULL),
        (dict(n_q=None, n_seq=1), H.NULL), (dict(n_q=[1], n_seq=-1), H.ARG), (dict(n_q=[1] * 9), H.CAPACITY),
        (dict(n_q=[-1]), H.ARG), (dict(n_q=[101]), H.ARG), (dict(n_q=[1, 1, 1]), H.EMPTY), (dict(n_q=[1], dt=3), H.DTYPE),
        (dict(n_q=[1], q=H.PTR + 8), H.ALIGN), (dict(n_q=[1], out=H.PTR + 2), H.ALIGN), (dict(n_q=[1], ws=H.PTR + 16), H.ALIGN),
        (dict(n_q=[1], slopes=H.PTR + 2), H.ALIGN), (dict(n_q=[1], prefix=H.PTR + 1), H.ALIGN),
        (dict(n_q=[1], ws_bytes=host.ws - 1), H.SMALL), (dict(n_q=[1], scale=-1.0), H.ARG),
        (dict(n_q=[1], scale=float("nan")), H.ARG), (dict(n_q=[1], cap=-2.0), H.ARG),
        (dict(n_q=[1], cap=float("inf")), H.ARG), (dict(n_q=[1], window=-1), H.ARG),
        (dict(n_q=[1], out=H.PTR), H.ARG), (dict(n_q=[2], out=H.PTR + 256), H.ARG),
        (dict(n_q=[1], scale=3e38), H.ARG), (dict(n_q=[1], cap=2e38), H.ARG), (dict(n_q=[1], scale=1.0, cap=1e-39), H.ARG),
    ]
    for kw, want in cases:
        assert _attend(host, h, **kw) == want, kw
        assert host.error()
    assert host.lib.kvq_attend(None, None, 0, None, 0, None, None, None, ctypes.c_size_t(0), None) == H.NULL
    assert not host.log()                       # nothing was launched
    assert _attend(host, h, n_q=[0, 0, 0], q=0, out=0, ws=0) == 0 and not host.log()
    assert _attend(host, h, n_q=[100, 1, 0, 300]) == 0 and host.log()


def test_out_beside_q(host):
    """out may start where q ends (n_q rows of 32 heads of 128) and end where q starts, and share no byte."""
    h, P, row = host.cache([100]), ot.Host.PTR, 32 * 128 * 2
    assert _attend(host, h, n_q=[3], out=P + 3 * row) == 0 and _attend(host, h, n_q=[3], q=P + 3 * row, out=P) == 0
    assert _attend(host, h, n_q=[3], dt=2, out=P + 3 * row) == ot.Host.ARG
    assert _attend(host, h, n_q=[3], dt=2, out=P + 6 * row) == 0
    assert _attend(host, h, n_q=[3], out=P + 3 * row - 16) == ot.Host.ARG


@pytest.mark.parametrize("values", [[2 ** 32], [1, 2 ** 31], [-2 ** 31 - 1], [0, 2 ** 32 + 1]])
def test_integers_keep_their_upper_bits(host, values):
    with pytest.raises(ValueError, match="parent"):
        host.kvq._int32s(values, "parent")
    assert list(host.kvq._int32s([-2 ** 31, 0, 2 ** 31 - 1], "parent")) == [-2 ** 31, 0, 2 ** 31 - 1]


@pytest.mark.parametrize("dt", [0, 2])
@pytest.mark.parametrize("seed", range(8))
def test_attend_plan(host, seed, dt):
    """Rows and pieces of every launch: every sequence in exactly one kernel's launch, rows in the call's order, every unit of a
    sequence in the same number of pieces, and no more partial rows than the workspace has where units are cut."""
    r = random.Random(seed)
    seqs = r.choice([1, 3, 8, 70, 700])
    hkv = r.choice([1, 2, 8])
    gqa = r.choice([1, 3, 4, 8])
    lens = [r.choice([1, 40, 1000, 4000]) for _ in range(seqs)]
    n_q = [r.choice([0, 1, 1, min(n, r.randint(1, 50)), n if n < 50 else 7, n]) for n in lens]
    window = r.choice([0, 64])
    h = host.cache(lens, max_seqs=seqs, n_kv_heads=hkv, n_q_heads=hkv * gqa)
    host.log()
    assert _attend(host, h, n_q=n_q, window=window, dt=dt) == 0
    first = [sum(n_q[:b]) for b in range(seqs)]
    log, seen = host.log(), {}
    keys = lambda b: min(lens[b], window + n_q[b]) if window else lens[b]  # noqa: E731
    steps = sum(hkv * -(-n_q[b] * gqa // 8) * (keys(b) // 32 + 1) for b in range(seqs) if n_q[b] * gqa >= 33)
    while log:
        kind, n, seq0, split, pieces, unit, slot, residual = log[:8]
        assert kind == 1 and residual == (dt == 2) and unit in ((8, 128) if residual else (8, 256))
        body, log = log[8:8 + 3 * n], log[8 + 3 * n:]
        offs = body[2::3] + [pieces]
        cut = False
        for i in range(n):
            b = seq0 + i
            assert body[3 * i:3 * i + 2] == [first[b], n_q[b]]
            rows, got = n_q[b] * gqa, offs[i + 1] - offs[i]
            if got == 0:
                continue
            assert b not in seen and (unit > 8) == (rows >= 33 and steps >= 16384)
            seen[b] = True
            units = hkv * -(-rows // unit)
            assert got % units == 0 and got >= units
            if got > units:
                cut = True
                assert got // units <= (lens[b] // (64 if unit > 8 else 32) + 4) // 4 and slot >= min(rows, unit)
        assert cut == bool(split)
        assert not split or pieces * slot * (128 + 4) * 4 <= host.ws - 4 * 4096 - 512
    assert sorted(seen) == [b for b in range(seqs) if n_q[b]]


@pytest.mark.parametrize("force", ["0", "1"])
def test_attend_kernel_forced(host, force, monkeypatch):
    monkeypatch.setenv("KVQ_ATTEND_TC", force)
    h = host.cache([4000, 1, 300])
    host.log()
    assert _attend(host, h, n_q=[4000, 1, 7]) == 0
    log = host.log()
    assert log[5] == (256 if force == "1" else 8) and log[1] == 3 and len(log) == 8 + 9


# ---------------------------------------------------------------- norm_rotary
def _rotary(host, h, n_new, q=ot.Host.PTR, k=ot.Host.PTR + (1 << 26), v=ot.Host.PTR + (2 << 26), qs=4096, ks=1024, vs=1024, dt=0,
            odt=0, qo=ot.Host.PTR + (3 << 26), ko=ot.Host.PTR + (4 << 26), vo=ot.Host.PTR + (5 << 26), n_seq=None, rot=True, **kw):
    base = dict(inv_freq=ot.Host.PTR, n_pairs=64, interleaved=0, eps=1e-6)
    sections = kw.pop("sections", None)
    base.update(kw)
    p = host.kvq.KvqRotary(**base)
    if sections:
        p.sections[:len(sections)] = sections
    c = ctypes.c_void_p
    i64 = ctypes.c_int64
    return host.lib.kvq_norm_rotary(h, c(q), i64(qs), c(k), i64(ks), c(v), i64(vs), dt,
                                    host.ints(n_new) if n_new is not None else None,
                                    len(n_new or []) if n_seq is None else n_seq, ctypes.byref(p) if rot else None, c(qo), c(ko),
                                    c(vo), odt, None)


def test_norm_rotary_refusals(host):
    h = host.cache([100, 1])
    H, P = host, ot.Host.PTR
    host.log()
    cases = [
        (dict(rot=False), H.NULL), (dict(q=0), H.NULL), (dict(k=0), H.NULL), (dict(qo=0), H.NULL), (dict(ko=0), H.NULL),
        (dict(vo=0), H.NULL), (dict(v=0), H.NULL), (dict(inv_freq=0), H.NULL), (dict(n_new=None, n_seq=1), H.NULL),
        (dict(n_seq=-1), H.ARG), (dict(n_new=[1] * 9), H.CAPACITY), (dict(n_new=[-1]), H.ARG), (dict(dt=5), H.DTYPE),
        (dict(odt=3), H.DTYPE), (dict(n_pairs=0), H.ARG), (dict(n_pairs=65), H.ARG), (dict(interleaved=2), H.ARG),
        (dict(eps=-1e-6), H.ARG), (dict(eps=float("nan")), H.ARG), (dict(qs=4095), H.ARG), (dict(ks=1023), H.ARG),
        (dict(vs=8), H.ARG), (dict(qs=1 << 32), H.ARG), (dict(q=P + 8), H.ALIGN), (dict(k=P + (1 << 26) + 2), H.ALIGN),
        (dict(qs=4100), H.ALIGN), (dict(vs=1028), H.ALIGN), (dict(qo=P + (3 << 26) + 8), H.ALIGN), (dict(q_weight=P + 4), H.ALIGN),
        (dict(k_weight=P + 2), H.ALIGN), (dict(inv_freq=P + 2), H.ALIGN), (dict(positions=P + 2, n_axes=1, sections=[64]), H.ALIGN),
        (dict(positions=P, n_axes=0), H.ARG), (dict(positions=P, n_axes=5), H.ARG),
        (dict(positions=P, n_axes=2, sections=[32, 31]), H.ARG), (dict(positions=P, n_axes=2, sections=[65, -1]), H.ARG),
        (dict(qo=P), H.ARG), (dict(ko=P + 4096), H.ARG), (dict(vo=P + (3 << 26) + 16), H.ARG), (dict(qo=P + 2 * 4096 * 9), H.ARG),
    ]
    for kw, want in cases:
        kw = {"n_new": [5, 5], **kw}
        assert _rotary(host, h, **kw) == want, kw
        assert host.error()
    assert not host.log()
    assert _rotary(host, h, n_new=[0, 0], q=0, k=0, v=0, qo=0, ko=0, vo=0, inv_freq=0) == 0 and not host.log()
    assert _rotary(host, h, n_new=[5, 5], v=0, vo=0, qo=P + 2 * 4096 * 10) == 0 and host.log()
    assert _rotary(host, h, n_new=[5, 5], positions=P, n_axes=3, sections=[0, 40, 24], dt=2, odt=1) == 0 and host.log()


def test_norm_rotary_launches(host):
    r = random.Random(3)
    n_new = [r.choice([0, 1, 17]) for _ in range(1100)]
    h = host.cache([1], max_seqs=1100)
    host.log()
    assert _rotary(host, h, n_new=n_new, qo=1 << 40, ko=2 << 40, vo=3 << 40, k=4 << 40, v=5 << 40) == 0
    log, row, b = host.log(), 0, 0
    while log:
        kind, n, seq0, row0, rows = log[:5]
        assert (kind, seq0, row0) == (3, b, row)
        offs, log = log[5:5 + n], log[5 + n:]
        for i in range(n):
            assert offs[i] == row - row0
            row += n_new[b]
            b += 1
        assert rows == row - row0
    assert row == sum(n_new) and b == 1100


# ---------------------------------------------------------------- reorder
def _reorder(host, h, parent, shared=0, n_seq=None):
    return host.lib.kvq_reorder(h, host.ints(parent) if parent is not None else None, len(parent or []) if n_seq is None else n_seq,
                                shared, None)


def _replay(log, n_all, lens):
    """What the recorded launches do: contents and device lengths, unit by unit as a thread of the kernel moves them, the chains
    of a launch in any order.  Checks that a launch's lengths are those of the contents that the moves carry."""
    held, lens = list(range(n_all)), list(lens)
    most = 0
    while log:
        kind, chains, n, shared, size = log[:5]
        assert kind == 2 and size >= 0
        start, log = log[5:6 + chains], log[6 + chains:]
        moves, log = [log[6 * i:6 * i + 6] for i in range(n)], log[6 * n:]
        most = max(most, n)
        begin, lens0 = list(held), list(lens)
        tickets = [moves[start[c]][1] for c in range(chains)]
        assert len(set(tickets)) == chains
        touched = [{s for m in moves[start[c]:start[c + 1]] for s in m[:2]} for c in range(chains)]
        for x, y in itertools.combinations(range(min(chains, 40)), 2):
            assert not touched[x] & touched[y]
        for c in reversed(range(chains)):
            i = start[c]
            while i < start[c + 1]:
                j = i
                while j < start[c + 1] and moves[j][4] == moves[i][4]:
                    j += 1
                assert j - i <= 8
                for s, d, sw, dw, _, _ in moves[i:j]:
                    assert held[s] == begin[sw] and held[d] == begin[dw]
                read = [held[m[0]] for m in moves[i:j]]
                assert len({m[1] for m in moves[i:j]}) == j - i
                for m, x in zip(moves[i:j], read):
                    held[m[1]] = x
                i = j
            final = {}
            for m in moves[start[c]:start[c + 1]]:
                if m[5]:
                    assert m[1] not in final
                    final[m[1]] = lens0[m[2]]
            assert set(final) == {m[1] for m in moves[start[c]:start[c + 1]]}
            for d, x in final.items():
                lens[d] = x
    assert most <= 512
    return held, lens


def test_reorder_refusals(host):
    h = host.cache([100, 90, 0, 300])
    H = host
    host.log()
    for kw, want in [(dict(parent=None, n_seq=2), H.NULL), (dict(parent=[0], n_seq=-1), H.ARG), (dict(parent=[0] * 9), H.CAPACITY),
                     (dict(parent=[8]), H.ARG), (dict(parent=[-1]), H.ARG), (dict(parent=[1, 0], shared=91), H.ARG),
                     (dict(parent=[0, 0], shared=-1), H.ARG), (dict(parent=[0, 1, 0], shared=1), H.ARG)]:
        assert _reorder(host, h, **kw) == want, kw
        assert host.error() and host.lengths(h, 4) == [100, 90, 0, 300]
    assert host.lib.kvq_reorder(None, None, 0, 0, None) == H.NULL
    assert not host.log()
    assert _reorder(host, h, [0, 1, 2], shared=1000) == 0 and not host.log()      # nothing moves
    assert _reorder(host, h, []) == 0 and not host.log()
    assert _reorder(host, h, [1, 0], shared=90) == 0 and host.lengths(h, 4) == [90, 100, 0, 300]


@pytest.mark.parametrize("n", [1, 2, 3, 4])
def test_reorder_every_small_map(host, n):
    lens = [10 * (i + 1) for i in range(n)]
    for parent in itertools.product(range(n), repeat=n):
        h = host.cache(lens, max_seqs=n)
        host.log()
        assert _reorder(host, h, list(parent)) == 0
        held, after = _replay(host.log(), n, lens)
        assert held == list(parent)
        want = oo.reorder(lens, parent)
        assert after == want and host.lengths(h, n) == want
        host.lib.kvq_cache_destroy(h)


@pytest.mark.parametrize("kind", ["random", "one cycle", "shift", "star", "pairs", "beams", "identity tail"])
@pytest.mark.parametrize("n", [9, 16, 300, 1500])
def test_reorder_large_maps(host, kind, n):
    r = random.Random(n)
    order = list(range(n))
    r.shuffle(order)
    parent = {
        "random": [r.randrange(n) for _ in range(n)],
        "one cycle": [dict(zip(order, order[1:] + order[:1]))[b] for b in range(n)],
        "shift": [max(0, b - 1) for b in range(n)],
        "star": [n // 2] * n,
        "pairs": [b ^ 1 if b ^ 1 < n else b for b in range(n)],
        "beams": [b // 4 * 4 + r.randrange(min(4, n - b // 4 * 4)) for b in range(n)],
        "identity tail": [r.randrange(n) for _ in range(n // 3)],
    }[kind]
    lens = [r.randrange(0, 4000) for _ in range(n)]
    h = host.cache(lens, max_seqs=n)
    host.log()
    assert _reorder(host, h, parent) == 0
    held, after = _replay(host.log(), n, lens)
    assert held == oo.reorder(list(range(n)), parent)
    assert after == oo.reorder(lens, parent) == host.lengths(h, n)


# ---------------------------------------------------------------- the oracle's definitions
def test_visible_by_hand():
    got = oo.visible(5, 3, window=2, prefix=1).astype(int).tolist()
    assert got == [[1, 1, 1, 0, 0], [1, 0, 1, 1, 0], [1, 0, 0, 1, 1]]
    assert oo.visible(3, 1, prefix=3).all() and oo.visible(3, 3, prefix=3).all()


def test_attend_oracle_is_the_decode_oracle_for_plain_scores():
    cfg = o.Config(4, 2, 32, 64, 4, 2)
    rng = np.random.default_rng(1)
    k, v = (rng.standard_normal((77, 2, 64)).astype(np.float16) for _ in range(2))
    q = rng.standard_normal((3, 4, 64))
    out, tol = oo.attend(cfg, k, v, q)
    assert np.abs(out[-1] - o.decode(cfg, k, v, q[-1])).max() < 1e-12
    kh, vh = o.dequantized_cache(cfg, k, v)
    assert np.abs(out[0] - o.attention(q[0], kh[:75], vh[:75], 2)).max() < 1e-12
    assert (tol > 0).all()


def test_scores_by_hand():
    q = np.array([[[2.0, 0.0]], [[0.0, 1.0]]])
    k = np.array([[[1.0, 3.0]], [[-1.0, 0.5]], [[4.0, 1.0]]])
    s = oo.scores(q, k, 3, 0.5, cap=2.0, slopes=[0.25])
    want = [[2 * np.tanh(0.5) - 0.25, 2 * np.tanh(-0.5), 2 * np.tanh(2.0) - 0.25],
            [2 * np.tanh(0.75) - 0.5, 2 * np.tanh(0.125) - 0.25, 2 * np.tanh(0.25)]]
    assert np.allclose(s[0], want, atol=1e-15)


def test_rotary_oracle_turns_pairs():
    x = np.zeros((2, 1, 8))
    x[:, 0, 1], x[:, 0, 5], x[:, 0, 7] = 1.0, 2.0, 9.0
    out = oo.norm_rotary(x, np.array([[0, 3]]), [0.1, np.pi / 6, 0.3, 0.5])
    assert np.allclose(out[0], x[0]) and np.allclose(out[1, 0, [1, 5]], [-2.0, 1.0])     # a quarter turn
    y = oo.norm_rotary(x, np.array([[1, 1], [0, 2]]), [0.5, np.pi / 4], sections=[1, 1], interleaved=True)
    assert np.allclose(y[1, 0, :2], [np.cos(0.5) * 0 - np.sin(0.5), np.cos(0.5)]) and np.allclose(y[..., 4:], x[..., 4:])
    w = oo.norm_rotary(x, np.array([[0, 0]]), [1.0], weight=np.full(8, 2.0), eps=0.0)
    assert np.allclose((w ** 2).mean(-1), 4.0)
