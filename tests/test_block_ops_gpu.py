"""GPU tests of the rotary, append and block-scaled cache calls against plain
64-bit forms.

Tolerances, element by element.

Rotated values: the table entry (A cos, A sin) comes from a phase that is exact to
32 bits of a half turn (2^-24 of at most pi: under 2^-22), a sine and cosine within
2 ulp of at most 1 (2^-23) and one product, so within A 2^-21; two products and a sum
in 32 bits add 3 roundings of 2^-24.  A rotated value is within A 2^-20 (|a| + |b|)
of the exact one, then off by one rounding: bf16 2^-8 of itself, e4m3 2^-4 of itself
or half its smallest step, 2^-10.

Attention: the weights y are kept as three e4m3 terms, 12 bits (2^-12 of each), and
2^-24 of the row's reference at the lower end; the row's sum takes them unrounded.
The reference is at most the largest weight w = p vs of the row, so that end costs
2^-24 max w sum |code|.  Scores: D <= 256 products of two terms summed in 32 bits, off
by at most 512 2^-23 sum |q||k| s, for the N(0, 1)-like rows used here (sum |q||k| s
<= 16) under 2^-10; 2^-10 A with A = sum p |v|.  The output's rounding: 2^-8 |o|.
Integers, copies, scales and the codes of values are equal.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F64 = torch.bfloat16, torch.float64
E4M3 = torch.float8_e4m3fn
TOP = 448.0


@pytest.fixture(scope="module")
def vsk():
    import speculative_decode_verify_prefix_gb300 as m

    m.build()
    return m


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=BF16)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def indptr(lens):
    return ints([0] + torch.tensor(lens, dtype=torch.int64).cumsum(0).tolist())


def value(codes):
    return codes.view(torch.uint8).view(E4M3).to(F64)


def frequencies(rot):
    return torch.tensor([10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float32, device=DEV)


def turned64(x, pos, freq, inter, size):
    """Rotated rows in 64 bits and, for each element, |a| + |b| of its pair (0 where it is copied)."""
    x = x.to(F64)
    rot = 2 * len(freq)
    t = pos.to(F64)[:, None, None] * freq.to(F64)
    cos, sin = size * t.cos(), size * t.sin()
    first = slice(0, rot, 2) if inter else slice(0, rot // 2)
    second = slice(1, rot, 2) if inter else slice(rot // 2, rot)
    a, b = x[..., first], x[..., second]
    y, w = x.clone(), torch.zeros_like(x)
    y[..., first], y[..., second] = a * cos - b * sin, b * cos + a * sin
    w[..., first] = w[..., second] = a.abs() + b.abs()
    return y, w


def check_rotated(got, want, pair, size, step=2.0 ** -8, least=2.0 ** -133, unit=1.0):
    """`got` stands for got * unit; step and least: half a step relative to the value, and of the smallest values."""
    near = size * 2.0 ** -20 * pair
    tol = near + step * (want.abs() + near) + least * unit
    bad = ~((got.to(F64) * unit - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float(((got.to(F64) * unit - want).abs() / tol).nan_to_num(9e9).max()))


# ---------------------------------------------------------------- rope_fwd

ROPES = [
    # (rows, h_q, h_kv, d, rot, interleaved, factor, positions)
    (1, 1, 1, 64, 16, False, 1.0, "zero"), (1, 32, 8, 128, 128, False, 1.0, "near"), (3, 5, 3, 64, 64, True, 1.2, "near"),
    (7, 4, 1, 256, 256, False, 1.0, "far"), (5, 3, 1, 256, 64, True, 1.0, "far"), (17, 14, 2, 128, 48, False, 0.5, "below"),
    (33, 8, 2, 128, 48, True, 1.0, "near"), (160, 8, 8, 64, 32, False, 1.0, "near"), (641, 2, 1, 256, 128, True, 1.0, "far"),
    (2500, 32, 8, 128, 128, False, 1.3, "far"), (9733, 6, 2, 128, 128, True, 1.0, "near"), (2, 300, 100, 64, 64, False, 1.0, "near"),
    (12161, 1, 1, 64, 64, False, 1.0, "near"),
]


def positions(g, n, kind, wide=True):
    p = {"zero": torch.zeros(n, device=DEV), "near": torch.arange(n, device=DEV) + 3,
         "far": torch.randint(1 << 20, (1 << 31) - 1, (n,), generator=g, device=DEV),
         "below": -torch.randint(0, 1 << 24, (n,), generator=g, device=DEV)}[kind].long()
    return p if wide else p.int()


@pytest.mark.parametrize("case", ROPES, ids=lambda c: f"n{c[0]}h{c[1]}x{c[2]}d{c[3]}r{c[4]}{'i' if c[5] else 's'}{c[7]}")
@pytest.mark.parametrize("wide", [True, False])
def test_rope_against_64_bits(vsk, case, wide):
    n, hq, hk, d, rot, inter, size, kind = case
    g = gen(n + d)
    qkv = normal(g, n, hq + 2 * hk, d)
    q, k = qkv[:, :hq], qkv[:, hq:hq + hk]
    pos, freq = positions(g, n, kind, wide), frequencies(rot)
    qo, ko = torch.full((n + 1, hq, d), 7.0, dtype=BF16, device=DEV), torch.empty(n, hk, 2 * d, dtype=BF16, device=DEV)[..., d:]
    vsk.rope_fwd(q, k, qo[:n], ko, pos, freq, interleaved=inter, attention_factor=size)
    for x, y in ((q, qo[:n]), (k, ko)):
        want, pair = turned64(x, pos, freq, inter, size)
        check_rotated(y, want, pair, size)
        assert torch.equal(y[..., rot:], x[..., rot:])
    assert bool((qo[n] == 7.0).all())
    # in place, and keys alone
    a, b = qkv.clone(), qkv.clone()
    vsk.rope_fwd(a[:, :hq], a[:, hq:hq + hk], a[:, :hq], a[:, hq:hq + hk], pos, freq, inter, size)
    assert torch.equal(a[:, :hq], qo[:n]) and torch.equal(a[:, hq:hq + hk], ko) and torch.equal(a[:, hq + hk:], qkv[:, hq + hk:])
    vsk.rope_fwd(None, b[:, hq:hq + hk], None, b[:, hq:hq + hk], pos, freq, inter, size)
    assert torch.equal(b[:, hq:hq + hk], ko) and torch.equal(b[:, :hq], q)


def test_rope_position_zero_copies(vsk):
    g = gen(3)
    q, k = normal(g, 20, 4, 128), normal(g, 20, 2, 128)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    vsk.rope_fwd(q, k, qo, ko, ints([0] * 20), frequencies(128))
    assert torch.equal(qo, q) and torch.equal(ko, k)


def test_rope_turns_there_and_back(vsk):
    """The inverse turn: positions and their negatives."""
    g = gen(4)
    q, k = normal(g, 50, 4, 64), normal(g, 50, 2, 64)
    pos, f = positions(g, 50, "far"), frequencies(64)
    a, b = torch.empty_like(q), torch.empty_like(k)
    vsk.rope_fwd(q, k, a, b, pos, f)
    vsk.rope_fwd(a, b, a, b, -pos, f)
    pair = (q[..., :32].to(F64).abs() + q[..., 32:].to(F64).abs()).repeat(1, 1, 2)
    # two turns, each off by 2^-20 of the pair and rounded by 2^-8 of itself (both of the pair come back)
    assert bool(((a.to(F64) - q.to(F64)).abs() <= 2.0 ** -7 * 1.02 * 2 ** 0.5 * pair).all())


def test_rope_values_that_are_no_numbers(vsk):
    q = torch.ones(4, 1, 64, dtype=BF16, device=DEV)
    q[0, 0, 3], q[1, 0, 5], q[2, 0, 50] = math.nan, math.inf, -math.inf
    f = frequencies(32)
    f[9] = math.nan
    qo, k = torch.empty_like(q), torch.ones_like(q)
    vsk.rope_fwd(q, k, qo, torch.empty_like(k), ints([1, 2, 3, 4]), f)
    bad = torch.zeros(4, 64, dtype=torch.bool, device=DEV)
    bad[:, [9, 25]] = True  # the pair of the frequency that is no number
    bad[0, [3, 19]] = True
    assert torch.equal(qo[:, 0].isnan(), bad)
    assert bool(qo[1, 0, [5, 21]].isinf().all()) and float(qo[2, 0, 50]) == -math.inf
    assert int((~qo.isfinite()).sum()) == 8 + 2 + 2 + 1


def test_rope_graph_and_other_stream(vsk):
    g = gen(5)
    q, k = normal(g, 300, 8, 128), normal(g, 300, 2, 128)
    pos, f = positions(g, 300, "near"), frequencies(128)
    want = [torch.empty_like(q), torch.empty_like(k)]
    vsk.rope_fwd(q, k, *want, pos, f)
    outs = [torch.empty_like(q), torch.empty_like(k)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vsk.rope_fwd(q, k, *outs, pos, f)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    side = torch.cuda.Stream()
    again = [torch.zeros_like(q), torch.zeros_like(k)]
    side.wait_stream(torch.cuda.current_stream())
    vsk.rope_fwd(q, k, *again, pos, f, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, want))


# ---------------------------------------------------------------- rope_append_fwd

APPENDS = [
    # (rows, h_q, h_kv, d, rot, interleaved, e4m3, scales)
    (1, 1, 1, 64, 64, False, False, (1.0, 1.0)), (1, 32, 8, 128, 128, False, True, (0.5, 0.25)), (6, 6, 2, 256, 64, True, True, (0.03, 0.7)),
    (37, 4, 4, 128, 48, False, True, (0.002, 1.0)), (65, 8, 1, 64, 32, True, False, (0.75, 3.0)), (700, 14, 2, 128, 128, False, False, (1.0, 1.0)),
    (2433, 16, 2, 256, 256, False, True, (0.5, 0.25)), (5001, 0, 3, 64, 64, False, True, (1.0, 0.125)),
]


@pytest.mark.parametrize("case", APPENDS, ids=lambda c: f"n{c[0]}h{c[1]}x{c[2]}d{c[3]}r{c[4]}{'i' if c[5] else 's'}{'e4m3' if c[6] else 'bf16'}")
@pytest.mark.parametrize("keep", [True, False])
def test_append_against_64_bits(vsk, case, keep):
    n, hq, hk, d, rot, inter, fp8, (ks, vs) = case
    g = gen(n)
    qkv = normal(g, n, hq + 2 * hk, d)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    pos, freq = positions(g, n, "near"), frequencies(rot)
    pool = n + 50
    old = normal(g, pool, 2 * hk, d).to(E4M3 if fp8 else BF16)
    cache = old.clone()
    kb, vb = cache[:, :hk], cache[:, hk:]
    loc = torch.randperm(pool, generator=g, device=DEV)[:n]
    if n > 4:
        loc[2] = -1  # a row without a place
    qo, ko = (torch.empty_like(q) if hq else None), (torch.empty(n, hk, d, dtype=BF16, device=DEV) if keep else None)
    vsk.rope_append_fwd(q if hq else None, k, v, qo, ko, kb, vb, loc if n % 2 else loc.int(), pos, freq, ks, vs, inter, 1.1)
    assert vsk.read_error_flags() == 0
    if hq:
        check_rotated(qo, *turned64(q, pos, freq, inter, 1.1), 1.1)
    want, pair = turned64(k, pos, freq, inter, 1.1)
    if keep:
        check_rotated(ko, want, pair, 1.1)
    there = loc >= 0
    rows = loc[there]
    if fp8:
        lim = TOP * ks
        got = value(kb)[rows]
        inside = want[there].clamp(-lim, lim)
        check_rotated(got, inside, pair[there], 1.1, 2.0 ** -4, 2.0 ** -10, ks)
        codes = (v.float() / vs).clamp(-TOP, TOP).to(E4M3)
        assert torch.equal(vb.view(torch.uint8)[rows], codes.view(torch.uint8)[there])
    else:
        check_rotated(kb[rows], want[there] , pair[there], 1.1, 2.0 ** -8, 2.0 ** -133, ks)
        assert torch.equal(vb[rows], (v.float() / vs).to(BF16)[there])
    rest = torch.ones(pool, dtype=torch.bool, device=DEV)
    rest[rows] = False
    as_bytes = torch.uint8 if fp8 else torch.int16
    assert torch.equal(cache.view(as_bytes)[rest], old.view(as_bytes)[rest])


def test_append_places_outside_the_pool(vsk):
    g = gen(1)
    n = 9
    q, k, v = normal(g, n, 2, 64), normal(g, n, 2, 64), normal(g, n, 2, 64)
    pos, f = positions(g, n, "near"), frequencies(64)
    for bad in (-2, 12, 1 << 40, -(1 << 40)):
        kb, vb = torch.zeros(12, 2, 64, dtype=BF16, device=DEV), torch.zeros(12, 2, 64, dtype=BF16, device=DEV)
        loc = torch.arange(n, device=DEV)
        loc[4] = bad
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        vsk.rope_append_fwd(q, k, v, qo, ko, kb, vb, loc, pos, f)
        assert vsk.read_error_flags() == 1
        keep = torch.arange(n, device=DEV) != 4
        assert torch.equal(vb[:n][keep], v[keep]) and torch.equal(kb[:n][keep], ko[keep])
        assert not vb[4].any() and not kb[4].any() and not vb[n:].any()


def test_append_values_that_are_no_numbers(vsk):
    v = torch.ones(3, 1, 64, dtype=BF16, device=DEV)
    v[0, 0, 5], v[1, 0, 6], v[2, 0, 7] = math.nan, math.inf, -math.inf
    kb, vb = (torch.zeros(3, 1, 64, dtype=torch.uint8, device=DEV).view(E4M3) for _ in "kv")
    vsk.rope_append_fwd(None, v.clone(), v, None, None, kb, vb, ints([0, 1, 2]), ints([0, 0, 0]), frequencies(16))
    x = value(vb)
    assert bool(x[0, 0, 5].isnan()) and float(x[1, 0, 6]) == TOP and float(x[2, 0, 7]) == -TOP and int(x.isnan().sum()) == 1
    x = value(kb)  # 0 times an infinite partner is none
    assert bool(x[0, 0, [5, 13]].isnan().all()) and int((x == 1).sum()) == 3 * 64 - 6


# ---------------------------------------------------------------- rope_append_block_fwd

def need64(top):
    if not top > 0:
        return 2.0 ** -40
    e = math.ceil(math.log2(top / TOP))
    assert abs(math.log2(top / TOP) - round(math.log2(top / TOP))) > 1e-5 or top / TOP == 2.0 ** round(math.log2(top / TOP))
    return 2.0 ** max(-40, min(40, e))


def block_cache(g, blocks, size, hk, d, lo=-9, hi=-5):
    kc, vc = ((normal(g, blocks * size, hk, d) * 100).clamp(-TOP, TOP).to(E4M3) for _ in "kv")
    ks, vs = (torch.exp2(torch.randint(lo, hi, (blocks, hk), generator=g, device=DEV).float()) for _ in "kv")
    return kc, vc, ks, vs


def table_of(g, held, size, blocks, cols=None):
    """Block ids of sequences that hold `held` rows, drawn without repeating."""
    n = [-(-x // size) for x in held]
    order = torch.randperm(blocks, generator=g, device=DEV).tolist()
    cols = cols or max(1, max(n))
    t = torch.full((len(held), cols), -7, dtype=torch.int32)
    at = 0
    for b, x in enumerate(n):
        t[b, :x] = torch.tensor(order[at:at + x], dtype=torch.int32)
        at += x
    return t.to(DEV)


def check_block_append(k, v, kc, vc, ks, vs, old, table, lens, new, size, pos, freq, inter, factor, skip=()):
    """The caches after a call against block after block of the definition; old: before it."""
    hk = k.shape[1]
    want, pair = turned64(k, pos, freq, inter, factor)
    okc, ovc, oks, ovs = (x.clone() for x in old)
    eks, evs = oks.clone(), ovs.clone()
    ekc, evc = okc.view(torch.uint8).clone(), ovc.view(torch.uint8).clone()
    t, at = table.tolist(), 0
    for b, (p, n) in enumerate(zip(lens, new)):
        done = 0
        while done < n:
            col, off = divmod(p + done, size)
            here = min(n - done, size - off)
            page = t[b][col]
            src = slice(at + done, at + done + here)
            done += here
            if b in skip or not 0 <= page < ks.shape[0]:
                continue
            rows = slice(page * size + off, page * size + off + here)
            olds = slice(page * size, page * size + off)
            for h in range(hk):
                for x, codes, scales, before, is_v in ((want, ekc, eks, okc, False), (v.to(F64), evc, evs, ovc, True)):
                    y = x[src, h]
                    s = need64(float(y.abs()[y.isfinite()].max()) if y.isfinite().any() else 0.0)
                    was = float(scales[page, h])
                    if off:
                        s = max(s, was)
                    scales[page, h] = s
                    if off and s != was:
                        again = (before.view(torch.uint8)[olds, h].view(E4M3).float() * (was / s)).to(E4M3)
                        codes[olds, h] = again.view(torch.uint8)
                    if is_v:
                        codes[rows, h] = (v[src, h].float() / s).clamp(-TOP, TOP).to(E4M3).view(torch.uint8)
                    else:
                        got = kc[rows, h]
                        ok = y.isfinite()
                        check_rotated(torch.where(ok, value(got), 0.0), torch.where(ok, y, 0.0), pair[src, h].nan_to_num(0, 0, 0), factor,
                                      2.0 ** -4, 2.0 ** -10, s)
                        codes[rows, h] = got.view(torch.uint8)
        at += n
    assert torch.equal(ks, eks) and torch.equal(vs, evs)
    assert torch.equal(kc.view(torch.uint8), ekc) and torch.equal(vc.view(torch.uint8), evc)


BLOCK_APPENDS = [
    # (rows before, new rows, block, h_q, h_kv, d, rot, interleaved)
    ((0,), (1,), 16, 1, 1, 64, 64, False), ((0, 5, 16, 31), (1, 1, 1, 1), 16, 32, 8, 128, 128, False),
    ((3, 0, 64, 60), (4, 4, 4, 4), 64, 8, 2, 128, 128, True), ((0,), (16,), 16, 4, 1, 64, 32, False), ((15,), (17,), 16, 4, 1, 64, 32, True),
    ((47,), (98,), 48, 6, 2, 256, 64, False), ((0, 100, 7), (129, 0, 250), 128, 4, 2, 256, 256, False),
    ((63, 64, 65, 1), (1, 64, 127, 0), 64, 0, 3, 64, 48, False), ((0, 2000), (1000, 333), 32, 7, 1, 128, 128, False),
    (tuple(range(0, 90, 3)), tuple(range(30)), 16, 2, 2, 64, 16, True), ((1,) * 300, (1,) * 300, 16, 2, 1, 64, 64, False),
    ((40,), (2100,), 112, 10, 5, 128, 96, False),
]


@pytest.mark.parametrize("case", BLOCK_APPENDS, ids=lambda c: f"b{len(c[0])}n{sum(c[1])}s{c[2]}h{c[3]}x{c[4]}d{c[5]}r{c[6]}{'i' if c[7] else 's'}")
@pytest.mark.parametrize("wide", [1.0, 40.0])  # 40: most blocks that hold rows need a larger scale
def test_block_append_against_64_bits(vsk, case, wide):
    lens, new, size, hq, hk, d, rot, inter = case
    n = sum(new)
    g = gen(n + size)
    qkv = normal(g, n + 3, hq + 2 * hk, d) * wide
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    held = [a + x for a, x in zip(lens, new)]
    blocks = sum(-(-x // size) for x in held) + 2
    table = table_of(g, held, size, blocks)
    old = block_cache(g, blocks, size, hk, d)
    cache = [x.clone() for x in old]
    pos, freq = positions(g, n + 3, "near"), frequencies(rot)
    qo, ko = (torch.full_like(q, 7.0) if hq else None), torch.full_like(k, 7.0)
    vsk.rope_append_block_fwd(q if hq else None, k, v, qo, ko, *cache, indptr(new), table, ints(lens), size, pos, freq, inter, 0.9)
    assert vsk.read_error_flags() == 0
    for x, y in ((q, qo), (k, ko)):
        if y is not None:
            check_rotated(y[:n], *turned64(x[:n], pos[:n], freq, inter, 0.9), 0.9)
            assert bool((y[n:] == 7.0).all())  # rows behind the last sequence
    check_block_append(k[:n], v[:n], *cache, old, table, lens, new, size, pos[:n], freq, inter, 0.9)
    # the keys go to the cache alone, and what is there already changes nothing
    again = [x.clone() for x in old]
    vsk.rope_append_block_fwd(None, k, v, None, None, *again, indptr(new), table, ints(lens), size, pos.int(), freq, inter, 0.9)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(again, cache))


@pytest.mark.parametrize("case", [
    # (sequences, new rows of each at least, block, h_q, h_kv, d, rot, interleaved): enough blocks that a CTA
    # takes several heads of one, of keys and values where they do not divide evenly
    (60, 200, 32, 8, 8, 64, 64, False), (40, 640, 64, 2, 32, 128, 96, True), (30, 850, 128, 4, 4, 128, 128, False),
    (80, 100, 16, 3, 1, 64, 16, False), (60, 350, 64, 0, 2, 256, 256, True),
], ids=lambda c: f"b{c[0]}n{c[1]}s{c[2]}h{c[3]}x{c[4]}d{c[5]}r{c[6]}")
def test_block_append_of_many_is_that_of_each(vsk, case):
    b, least, size, hq, hk, d, rot, inter = case
    g = gen(least)
    lens, new = [(13 * i) % 97 for i in range(b)], [least + (29 * i) % 83 for i in range(b)]
    n = sum(new)
    q, k, v = (normal(g, n, h, d) * 40 if h else None for h in (hq, hk, hk))
    held = [x + y for x, y in zip(lens, new)]
    blocks = sum(-(-x // size) for x in held) + 2
    table = table_of(g, held, size, blocks)
    old = block_cache(g, blocks, size, hk, d)
    pos, freq = positions(g, n, "near"), frequencies(rot)
    many, each = [x.clone() for x in old], [x.clone() for x in old]
    outs = [(torch.full_like(q, 7.0) if hq else None, torch.full_like(k, 7.0)) for _ in range(2)]
    vsk.rope_append_block_fwd(q, k, v, *outs[0], *many, indptr(new), table, ints(lens), size, pos, freq, inter, 1.1)
    at = 0
    for i, m in enumerate(new):
        r = slice(at, at + m)
        vsk.rope_append_block_fwd(q[r] if hq else None, k[r], v[r], outs[1][0][r] if hq else None, outs[1][1][r], *each,
                                  indptr([m]), table[i:i + 1], ints(lens[i:i + 1]), size, pos[r], freq, inter, 1.1)
        at += m
    assert vsk.read_error_flags() == 0
    for x, y in zip([*many, *outs[0]], [*each, *outs[1]]):
        assert x is None or torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))


def test_block_append_extremes(vsk):
    """Rows of zeros, of the largest and smallest numbers, infinities and NaN."""
    g = gen(8)
    size, d = 16, 64
    v = torch.zeros(7, 1, d, dtype=BF16, device=DEV)
    v[1] = 3e38
    v[2] = 1e-38
    v[3, 0, 0] = TOP
    v[4, 0, 0] = 450.0
    v[5] = normal(g, 1, d)
    v[5, 0, 1], v[5, 0, 2], v[5, 0, 3] = math.inf, -math.inf, math.nan
    v[6] = math.nan
    kc, vc, ks, vs = block_cache(g, 7, size, 1, d)
    pos = ints([0] * 7)
    vsk.rope_append_block_fwd(None, v, v, None, None, kc, vc, ks, vs, indptr([1] * 7), ints([[i] for i in range(7)]), ints([0] * 7),
                              size, pos, frequencies(16))
    assert vsk.read_error_flags() == 0
    want = [2.0 ** -40, 2.0 ** 40, 2.0 ** -40, 1.0, 2.0, need64(float(v[5][v[5].isfinite()].abs().max())), 2.0 ** -40]
    assert vs[:, 0].tolist() == want
    x = value(vc.view(7, size, d)[:, 0])
    assert not x[0].any() and bool((x[1] == TOP).all()) and not x[2].any() and float(x[3, 0]) == TOP and float(x[4, 0]) == 224.0
    assert float(x[5, 1]) == TOP and float(x[5, 2]) == -TOP and bool(x[5, 3].isnan()) and bool(x[6].isnan().all())
    assert int(x.isnan().sum()) == 1 + d


def test_block_append_bad_tables_and_lengths(vsk):
    g = gen(9)
    size, hk, d = 16, 2, 64
    new = [3, 20, 2, 5, 1]
    lens = [0, 10, -1, 30, 4]
    n = sum(new)
    q, k, v = normal(g, n, 2, d), normal(g, n, hk, d), normal(g, n, hk, d)
    old = block_cache(g, 8, size, hk, d)
    # sequence 1: its second block lies outside; 2: a negative length; 3: beyond the columns (30 + 5 > 32); 4: id 8 of 8
    table = ints([[0, 0], [1, -1], [2, 3], [4, 5], [8, 6]])
    cache = [x.clone() for x in old]
    pos, f = positions(g, n, "near"), frequencies(64)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    vsk.rope_append_block_fwd(q, k, v, qo, ko, *cache, indptr(new), table, ints(lens), size, pos, f)
    assert vsk.read_error_flags() == 1 | 2
    check_rotated(qo, *turned64(q, pos, f, False, 1.0), 1.0)
    check_rotated(ko, *turned64(k, pos, f, False, 1.0), 1.0)
    check_block_append(k, v, *cache, old, table, [0, 10, 0, 0, 4], new, size, pos, f, False, 1.0, skip=(2, 3))


def test_block_append_bad_qo_indptr(vsk):
    g = gen(10)
    k = normal(g, 6, 1, 64)
    old = block_cache(g, 4, 16, 1, 64)
    cache = [x.clone() for x in old]
    ko = torch.full_like(k, 7.0)
    # the second pair falls, the third leaves the rows
    vsk.rope_append_block_fwd(None, k, k, None, ko, *cache, ints([0, 2, 1, 9]), ints([[0], [1], [2]]), ints([0, 0, 0]), 16,
                              positions(g, 6, "zero"), frequencies(64))
    assert vsk.read_error_flags() == 4
    assert torch.equal(ko[:2], k[:2]) and bool((ko[2:] == 7.0).all())
    check_block_append(k[:2], k[:2], *cache, old, ints([[0]]), [0], [2], 16, torch.zeros(2, device=DEV), frequencies(64), False, 1.0)


# ---------------------------------------------------------------- verify_splitkv_block_fwd

def attend64(q, keys, vals, seen, weight, scale):
    """One KV head's rows in 64 bits: q [r, d], keys and vals [n, d], seen [r, n]; weight [n]: the keys' V scales (0:
    drafts).  Returns o and its tolerance."""
    x = (q @ keys.T) * scale
    x = x.masked_fill(~seen, -math.inf)
    some = seen.any(1, keepdim=True)
    p = torch.softmax(torch.where(some, x, torch.zeros_like(x)), 1) * some
    o, a = p @ vals, p @ vals.abs()
    w = (p * weight).amax(1, keepdim=True) if len(weight) else torch.zeros_like(some, dtype=F64)
    codes = torch.where(weight[:, None] > 0, vals.abs() / weight.clamp_min(1e-300)[:, None], torch.zeros_like(vals)).sum(0, keepdim=True)
    return o, 2.0 ** -8 * o.abs() * (1 + 2.0 ** -8) + (2.0 ** -12 + 2.0 ** -10) * a + 2.0 ** -24 * w * codes + 1e-37


def block_want(q, ke, ve, kc, vc, ks, vs, table, lens, size, l_ext, scale, mask=None):
    """Output and tolerance of the whole call."""
    hk = ke.shape[1]
    gq = q.shape[1] // hk
    o, tol = torch.zeros(q.shape, dtype=F64, device=DEV), torch.zeros(q.shape, dtype=F64, device=DEV)
    for b, n in enumerate(lens):
        r = slice(b * l_ext, (b + 1) * l_ext)
        pages = table[b, :-(-n // size)].long()
        rows = (pages[:, None] * size + torch.arange(size, device=DEV)).flatten()[:n]
        page = pages.repeat_interleave(size)[:n]
        seen = torch.ones(l_ext, n + l_ext, dtype=torch.bool, device=DEV).tril(n) if mask is None else torch.cat(
            [torch.ones(l_ext, n, dtype=torch.bool, device=DEV), mask[b]], 1)
        seen = seen.repeat_interleave(gq, 0)
        for h in range(hk):
            keys = torch.cat([value(kc[rows, h]) * ks[page, h].to(F64)[:, None], ke[r, h].to(F64)])
            vals = torch.cat([value(vc[rows, h]) * vs[page, h].to(F64)[:, None], ve[r, h].to(F64)])
            weight = torch.cat([vs[page, h].to(F64), torch.zeros(l_ext, dtype=F64, device=DEV)])
            x = q[r, h * gq:(h + 1) * gq].to(F64).reshape(l_ext * gq, -1)
            y, t = attend64(x, keys, vals, seen, weight, scale)
            o[r, h * gq:(h + 1) * gq], tol[r, h * gq:(h + 1) * gq] = y.view(l_ext, gq, -1), t.view(l_ext, gq, -1)
    return o, tol


def check_block(got, want, tol):
    bad = ~((got.to(F64) - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float(((got.to(F64) - want).abs() / tol).nan_to_num(9e9).max()))


def block_case(lens, size, hq, hk, d, l_ext, seed=0, spare=True):
    """A cache whose places beyond the prefixes, spare blocks and their scales hold NaN."""
    g = gen(seed)
    b = len(lens)
    blocks = sum(-(-x // size) for x in lens) + 3
    table = table_of(g, lens, size, blocks, cols=max(1, max(-(-x // size) for x in lens)) + 1)
    kc, vc, ks, vs = block_cache(g, blocks, size, hk, d, -9, -5)
    if spare:
        live = torch.zeros(blocks * size, dtype=torch.bool, device=DEV)
        for i, n in enumerate(lens):
            pages = table[i, :-(-n // size)].long()
            live[(pages[:, None] * size + torch.arange(size, device=DEV)).flatten()[:n]] = True
        for c in (kc, vc):
            c.view(torch.uint8)[~live] = 0x7F
        used = live.view(blocks, size).any(1)
        ks[~used] = math.nan
        vs[~used] = math.nan
    rows = b * l_ext
    return dict(q=normal(g, rows, hq, d), ke=normal(g, rows, hk, d), ve=normal(g, rows, hk, d), kc=kc, vc=vc, ks=ks, vs=vs,
                qo=indptr([l_ext] * b), table=table, lens=ints(lens))


def run_block(vsk, c, size, l_ext, **kw):
    o = torch.full_like(c["q"], 7.0)
    vsk.verify_splitkv_block_fwd(c["q"], c["ke"], c["ve"], o, c["kc"], c["vc"], c["ks"], c["vs"], c["qo"], c["table"], c["lens"],
                                 size, l_ext, **kw)
    return o


BLOCKS = [
    # (prefix lengths, block, h_q, h_kv, d, drafts)
    ((1,), 16, 1, 1, 64, 1), ((0,), 16, 4, 1, 128, 3), ((0, 0, 7), 16, 2, 2, 256, 2), ((15, 16, 17), 16, 4, 2, 64, 4),
    ((127, 128, 129, 255), 16, 8, 2, 128, 4), ((63, 64, 65), 64, 16, 2, 256, 4), ((1000, 3, 0, 130), 48, 14, 2, 128, 2),
    ((4097,), 128, 32, 8, 128, 1), ((5000, 4999), 32, 8, 1, 64, 4), ((300,), 16, 33, 1, 64, 1), ((777, 40), 64, 8, 1, 128, 16),
    ((900,), 128, 64, 1, 256, 2), ((2500, 10), 80, 7, 7, 256, 5), ((513, 511), 16, 40, 8, 128, 1), (tuple(range(0, 90, 2)), 16, 4, 1, 64, 2),
    ((20011,), 64, 5, 1, 128, 3), ((3,) * 400, 16, 2, 2, 64, 1), ((640, 640), 112, 24, 8, 64, 8),
]


@pytest.mark.parametrize("case", BLOCKS, ids=lambda c: f"b{len(c[0])}n{sum(c[0])}s{c[1]}h{c[2]}x{c[3]}d{c[4]}l{c[5]}")
def test_block_against_64_bits(vsk, case):
    lens, size, hq, hk, d, l_ext = case
    c = block_case(lens, size, hq, hk, d, l_ext, seed=sum(lens))
    o = run_block(vsk, c, size, l_ext)
    assert vsk.read_error_flags() == 0
    want, tol = block_want(c["q"], c["ke"], c["ve"], c["kc"], c["vc"], c["ks"], c["vs"], c["table"], lens, size, l_ext, d ** -0.5)
    check_block(o, want, tol)
    assert torch.equal(run_block(vsk, c, size, l_ext), o)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_block_strided_views(vsk, d):
    """q, k, v of one projection, outputs inside a wider buffer, caches side by side, a table with room."""
    lens, size, hq, hk, l_ext = [200, 77], 16, 6, 2, 3
    c = block_case(lens, size, hq, hk, d, l_ext, seed=5)
    x = torch.cat([c["q"], c["ke"], c["ve"]], 1)
    both = torch.stack([c["kc"].view(torch.uint8), c["vc"].view(torch.uint8)], 1).view(E4M3)  # [rows, 2, h_kv, d]
    wide = torch.zeros(c["table"].shape[0], 2 * c["table"].shape[1], dtype=torch.int32, device=DEV)
    wide[:, :c["table"].shape[1]] = c["table"]
    o = torch.full((2 * l_ext, hq + 1, d + 2), 7.0, dtype=BF16, device=DEV)
    vsk.verify_splitkv_block_fwd(x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], o[:, :hq, :d], both[:, 0], both[:, 1], c["ks"], c["vs"],
                                 c["qo"], wide[:, :c["table"].shape[1]], c["lens"], size, l_ext, sm_scale=0.2)
    want, tol = block_want(c["q"], c["ke"], c["ve"], c["kc"], c["vc"], c["ks"], c["vs"], c["table"], lens, size, l_ext, 0.2)
    check_block(o[:, :hq, :d], want, tol)
    assert bool((o[:, hq:] == 7.0).all()) and bool((o[:, :, d:] == 7.0).all())


@pytest.mark.parametrize("d,l_ext", [(64, 2), (128, 4), (256, 1)])
def test_block_scales_of_any_size(vsk, d, l_ext):
    """Scales over their whole range, no powers of two among them; each kind alone and both."""
    lens, size, hq, hk = [600, 333, 50], 16, 4, 2
    for which in ("v", "k", "both"):
        c = block_case(lens, size, hq, hk, d, l_ext, seed=d, spare=False)
        g = gen(77)
        n = c["ks"].shape
        if which in ("v", "both"):
            c["vs"] = torch.exp2(torch.rand(n, generator=g, device=DEV) * 79.9 - 39.95)
        if which in ("k", "both"):
            # scores stay those of keys of size 1 and below: their spread is the test's, not their height
            c["ks"] = 0.01 * torch.exp2(-torch.rand(n, generator=g, device=DEV) * 33)
        o = run_block(vsk, c, size, l_ext)
        assert vsk.read_error_flags() == 0
        want, tol = block_want(c["q"], c["ke"], c["ve"], c["kc"], c["vc"], c["ks"], c["vs"], c["table"], lens, size, l_ext, d ** -0.5)
        check_block(o, want, tol)


@pytest.mark.parametrize("bad", [0.0, -1.0, math.nan, math.inf, 2.0 ** -41, 2.0 ** 41])
@pytest.mark.parametrize("is_v", [False, True])
def test_block_scales_that_are_none(vsk, bad, is_v):
    lens, size, hq, hk, d, l_ext = [100, 60], 16, 4, 2, 64, 2
    c = block_case(lens, size, hq, hk, d, l_ext, seed=2, spare=False)
    clean = run_block(vsk, c, size, l_ext)
    c["vs" if is_v else "ks"][int(c["table"][0, 3]), 1] = bad
    o = run_block(vsk, c, size, l_ext)
    assert vsk.read_error_flags() == 64
    assert bool(o[:2, 2:].isnan().all())  # sequence 0, KV head 1
    o[:2, 2:] = clean[:2, 2:]
    assert torch.equal(o, clean)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_block_counts_every_key(vsk, d):
    """Queries of zero weigh all keys alike: with one-hot values the output is each column's share of the keys."""
    lens, size, l_ext = [1, 130, 2049, 999], 16, 1
    c = block_case(lens, size, 2, 1, d, l_ext, seed=3)
    c["q"].zero_()
    c["ve"].zero_()
    c["vs"].fill_(0.5)
    c["ks"].fill_(1.0)
    want = torch.zeros(len(lens), d, dtype=F64, device=DEV)
    for b, n in enumerate(lens):
        t = torch.arange(n, device=DEV)
        rows = c["table"][b].long()[t // size] * size + t % size
        c["vc"].view(torch.uint8)[rows] = 0
        c["vc"].view(torch.uint8)[rows, 0, (t * 7) % d] = 0x40  # 2.0, under the scale 1.0
        want[b] = torch.bincount((t * 7) % d, minlength=d).to(F64) / (n + 1)
    o = run_block(vsk, c, size, l_ext)
    for h in range(2):
        assert bool(((o[:, h].to(F64) - want).abs() <= 2.0 ** -8 * want).all())


def test_block_weights_far_below_the_largest(vsk):
    """One key 14 above the rest in natural units, 30,000 others: together they weigh a fortieth of it."""
    n, size, d = 30000, 16, 64
    c = block_case([n], size, 1, 1, d, 1, seed=4)
    c["q"].zero_()
    c["q"][0, 0, 0] = 8.0
    c["ke"].zero_()
    c["ke"][0, 0, 0] = -60.0
    c["ks"].fill_(1.0)
    c["vs"].fill_(1.0)
    t = torch.arange(n, device=DEV)
    rows = c["table"][0].long()[t // size] * size + t % size
    for name in ("kc", "vc"):
        c[name].view(torch.uint8)[rows] = 0
    c["kc"].view(torch.uint8)[rows[5], 0, 0] = torch.tensor([14.0], device=DEV).to(E4M3).view(torch.uint8)[0]
    c["vc"].view(torch.uint8)[rows, 0, 1] = 0x38  # 1.0 for all
    c["vc"].view(torch.uint8)[rows[5], 0, 1] = 0
    o = run_block(vsk, c, size, 1, sm_scale=0.125)
    rest = (n - 1) * math.exp(-14.0)
    want = rest / (1 + rest)
    # each weight within 2^-12 of itself and 2^-24 of the largest, times 29,999 keys; the output's rounding
    tol = want * 2.0 ** -8 + want * 2.0 ** -11 + (n - 1) * 2.0 ** -24 / (1 + rest)
    assert abs(float(o[0, 0, 1]) - want) <= tol and tol < want / 10


def test_block_rising_scores_rescale(vsk):
    """Every tile's scores lie above all before it."""
    for d in (64, 128, 256):
        n, size, hq = 3000, 16, 3
        c = block_case([n], size, hq, 1, d, 1, seed=6)
        c["q"].zero_()
        c["q"][..., 0] = 1.0
        c["kc"].view(torch.uint8)[:] = 0
        c["ks"].fill_(1.0)
        t = torch.arange(n, device=DEV)
        rows = c["table"][0].long()[t // size] * size + t % size
        steps = (t // 40).float() * 4
        c["kc"].view(torch.uint8)[rows, 0, 0] = steps.to(E4M3).view(torch.uint8)
        o = run_block(vsk, c, size, 1, sm_scale=0.25)
        want, tol = block_want(c["q"], c["ke"], c["ve"], c["kc"], c["vc"], c["ks"], c["vs"], c["table"], [n], size, 1, 0.25)
        # the scores are exact here, up to 75 of them in base e: 2^-24 of 110 in base 2 moves a weight by 2^-17
        check_block(o, want, tol)


def test_block_numbers_that_are_none_reach_their_rows_only(vsk):
    lens, size, hq, hk, d, l_ext = [70, 200], 16, 4, 2, 64, 3
    base = block_case(lens, size, hq, hk, d, l_ext, seed=7)
    clean = run_block(vsk, base, size, l_ext)

    def changed(fn):
        c = {k: x.clone() for k, x in base.items()}
        fn(c)
        return run_block(vsk, c, size, l_ext)

    def expect(o, rows, heads):
        hit = torch.zeros(o.shape[:2], dtype=torch.bool, device=DEV)
        hit[rows, heads] = True
        assert bool(o[hit].isnan().any(-1).all()) and torch.equal(o[~hit], clean[~hit])

    row = int(base["table"][1, 4]) * size + 3
    for x in (math.nan, math.inf, -math.inf):
        expect(changed(lambda c: c["q"][1, 2].fill_(x)), 1, 2)
    expect(changed(lambda c: c["q"][4, 0, 3:4].fill_(math.nan)), 4, 0)
    expect(changed(lambda c: c["kc"].view(torch.uint8)[row, 1, 5:6].fill_(0x7F)), slice(3, 6), slice(2, 4))
    expect(changed(lambda c: c["vc"].view(torch.uint8)[row, 0].fill_(0xFF)), slice(3, 6), slice(0, 2))
    # drafts: the rows before do not see them
    expect(changed(lambda c: c["ve"][4, 1].fill_(math.nan)), slice(4, 6), slice(2, 4))
    expect(changed(lambda c: c["ke"][5, 0].fill_(math.nan)), slice(5, 6), slice(0, 2))


def test_block_tree(vsk):
    lens, size, hq, hk, d, l_ext = [33, 0, 100], 16, 6, 2, 128, 5
    c = block_case(lens, size, hq, hk, d, l_ext, seed=9)
    g = gen(1)
    mask = [torch.rand(l_ext, l_ext, generator=g, device=DEV) < 0.5 for _ in lens]
    mask[1][2] = False  # an empty prefix and no draft: nothing to see
    full = [torch.cat([torch.rand(l_ext, n, generator=g, device=DEV) < 0.5, m], 1) for n, m in zip(lens, mask)]  # prefix part: not read
    flat = torch.cat([f.flatten() for f in full])
    at = [0] + torch.tensor([f.numel() for f in full]).cumsum(0).tolist()
    want, tol = block_want(c["q"], c["ke"], c["ve"], c["kc"], c["vc"], c["ks"], c["vs"], c["table"], lens, size, l_ext, d ** -0.5, mask)
    for dtype in (torch.int32, torch.int64):
        o = run_block(vsk, c, size, l_ext, custom_mask=flat, mask_indptr=torch.tensor(at, dtype=dtype, device=DEV))
        assert vsk.read_error_flags() == 0
        check_block(o, want, tol)
        assert not o[l_ext + 2].any()
    # a causal mask is the causal call; offsets outside the mask fall back to it
    low = torch.ones(l_ext, l_ext, dtype=torch.bool, device=DEV).tril()
    flat = torch.cat([torch.cat([torch.zeros(l_ext, n, dtype=torch.bool, device=DEV), low], 1).flatten() for n in lens])
    causal = run_block(vsk, c, size, l_ext)
    assert torch.equal(run_block(vsk, c, size, l_ext, custom_mask=flat, mask_indptr=ints(at)), causal)
    assert torch.equal(run_block(vsk, c, size, l_ext, custom_mask=flat[:-1], mask_indptr=ints([-1, at[1], at[2], 0])), causal)
    assert vsk.read_error_flags() == 16


def test_block_bad_tables_and_lengths(vsk):
    lens, size, hq, hk, d, l_ext = [70, 40, 64], 16, 4, 2, 64, 2
    c = block_case(lens, size, hq, hk, d, l_ext, seed=11, spare=False)
    for bad in (-1, c["ks"].shape[0], 2 ** 31 - 1, -2 ** 31):
        t = c["table"].clone()
        t[0, 1] = bad  # keys 16 .. 31 of sequence 0 are left out
        o = run_block(vsk, {**c, "table": t}, size, l_ext)
        assert vsk.read_error_flags() == 1
        # the same as a sequence without that block
        t2 = t.clone()
        t2[0, 1:-1] = t[0, 2:]
        l2 = [54, 40, 64]
        want, tol = block_want(c["q"], c["ke"], c["ve"], c["kc"], c["vc"], c["ks"], c["vs"], t2, l2, size, l_ext, d ** -0.5)
        check_block(o, want, tol)
    everything = {**c, "table": torch.full_like(c["table"], -1)}
    want, tol = block_want(c["q"], c["ke"], c["ve"], c["kc"], c["vc"], c["ks"], c["vs"], c["table"], [0, 0, 0], size, l_ext, d ** -0.5)
    check_block(run_block(vsk, everything, size, l_ext), want, tol)
    assert vsk.read_error_flags() == 1
    cols = c["table"].shape[1]
    o = run_block(vsk, {**c, "lens": ints([-5, cols * size + 1, 64])}, size, l_ext)
    assert vsk.read_error_flags() == 2
    want, tol = block_want(c["q"], c["ke"], c["ve"], c["kc"], c["vc"], c["ks"], c["vs"], c["table"], [0, 0, 64], size, l_ext, d ** -0.5)
    check_block(o, want, tol)
    o = run_block(vsk, {**c, "qo": ints([0, 3, 4, 6])}, size, l_ext)
    assert vsk.read_error_flags() == 4
    check_block(o, *block_want(c["q"], c["ke"], c["ve"], c["kc"], c["vc"], c["ks"], c["vs"], c["table"], lens, size, l_ext, d ** -0.5))


def test_block_without_a_cache(vsk):
    """No block at all: every prefix is empty, or its blocks are missed."""
    g = gen(12)
    q, ke, ve = normal(g, 4, 2, 64), normal(g, 4, 1, 64), normal(g, 4, 1, 64)
    none = torch.zeros(0, 1, 64, dtype=torch.uint8, device=DEV).view(E4M3)
    c = dict(q=q, ke=ke, ve=ve, kc=none, vc=none, ks=torch.zeros(0, 1, device=DEV), vs=torch.zeros(0, 1, device=DEV), qo=indptr([2, 2]),
             table=ints([[0], [0]]), lens=ints([0, 0]))
    o = run_block(vsk, c, 16, 2)
    assert vsk.read_error_flags() == 0
    check_block(o, *block_want(q, ke, ve, none, none, c["ks"], c["vs"], c["table"], [0, 0], 16, 2, 64 ** -0.5))
    assert torch.equal(run_block(vsk, {**c, "lens": ints([0, 5])}, 16, 2), o)
    assert vsk.read_error_flags() == 1


def test_block_one_workspace_for_calls_of_all_shapes(vsk):
    shapes = [([300, 20], 16, 8, 2, 128, 4), ([5000], 64, 16, 2, 256, 4), ([10] * 50, 32, 4, 1, 64, 2), ([2000], 16, 128, 1, 64, 1)]
    cases = [(block_case(*s, seed=i), s) for i, s in enumerate(shapes)]
    need = max(vsk.block_workspace_size(len(s[0]), s[2], s[3], s[4], s[5]) for s in shapes)
    alone = [run_block(vsk, c, s[1], s[5]) for c, s in cases]
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    for _ in range(2):
        for (c, s), want in zip(cases, alone):
            assert torch.equal(run_block(vsk, c, s[1], s[5], workspace=ws), want)
    # the counters that other calls keep at the end of a buffer stay as they are
    assert not ws[-65536:].any() and not ws[:256].any()
    with pytest.raises(ValueError, match="smaller than"):
        run_block(vsk, cases[1][0], 64, 4, workspace=ws[:4096])


def test_block_graphs_streams_and_threads(vsk):
    import threading

    lens, size, hq, hk, d, l_ext = [700, 90, 1500], 16, 8, 2, 128, 4
    cases = [block_case(lens, size, hq, hk, d, l_ext, seed=s) for s in range(3)]
    want = [run_block(vsk, c, size, l_ext) for c in cases]
    need = vsk.block_workspace_size(3, hq, hk, d, l_ext)
    # captured, then replayed over other contents of the same tensors
    c = {k: x.clone() for k, x in cases[0].items()}
    ws, o = torch.zeros(need, dtype=torch.uint8, device=DEV), torch.empty_like(c["q"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vsk.verify_splitkv_block_fwd(c["q"], c["ke"], c["ve"], o, c["kc"], c["vc"], c["ks"], c["vs"], c["qo"], c["table"], c["lens"],
                                     size, l_ext, workspace=ws)
    for src, w in zip(cases, want):
        for k, x in c.items():
            x.view(torch.uint8).copy_(src[k].view(torch.uint8))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, w)
    with pytest.raises(ValueError, match="pass workspace"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            run_block(vsk, c, size, l_ext)
    torch.cuda.synchronize()
    # host threads, each with a stream of its own; then all on one
    for shared in (False, True):
        got, errors, one = [None] * 3, [], torch.cuda.Stream()

        def work(i):
            try:
                s = one if shared else torch.cuda.Stream()
                with torch.cuda.stream(s):
                    for _ in range(5):
                        got[i] = run_block(vsk, cases[i], size, l_ext)
                s.synchronize()
            except Exception as e:  # noqa: BLE001
                errors.append(e)

        torch.cuda.synchronize()
        ts = [threading.Thread(target=work, args=(i,)) for i in range(3)]
        [t.start() for t in ts]
        [t.join() for t in ts]
        assert not errors and all(torch.equal(a, b) for a, b in zip(got, want))


def test_block_head_major_caches(vsk):
    """[h_kv, rows, D] storage seen as [rows, h_kv, D]; a row's heads far apart."""
    lens, size, hq, hk, d, l_ext = [500, 77, 1], 32, 8, 4, 64, 3
    c = block_case(lens, size, hq, hk, d, l_ext, seed=21)
    want = run_block(vsk, c, size, l_ext)
    for x in ("kc", "vc"):
        c[x] = c[x].view(torch.uint8).transpose(0, 1).contiguous().transpose(0, 1).view(E4M3)
        assert c[x].stride(1) > c[x].stride(0)
    assert torch.equal(run_block(vsk, c, size, l_ext), want)


def test_block_queries_with_an_outlier(vsk):
    """One element of a query 64 times the others: those below 2^-10 of it are off by 2^-17 of it at most."""
    lens, size, hq, hk, d, l_ext = [700], 16, 4, 1, 128, 2
    c = block_case(lens, size, hq, hk, d, l_ext, seed=22)
    c["q"][..., 5] = 64.0
    c["kc"].view(torch.uint8)[:, :, 5] &= 0x80  # (its keys are zero there: the rest decides)
    o = run_block(vsk, c, size, l_ext)
    want, tol = block_want(c["q"], c["ke"], c["ve"], c["kc"], c["vc"], c["ks"], c["vs"], c["table"], lens, size, l_ext, d ** -0.5)
    pages = c["table"][0, :-(-lens[0] // size)].long().repeat_interleave(size)[:lens[0]]
    rows = c["table"][0].long()[torch.arange(lens[0], device=DEV) // size] * size + torch.arange(lens[0], device=DEV) % size
    sums = (value(c["kc"][rows, 0]).abs().sum(1) * c["ks"][pages, 0].to(F64)).max()
    # every score off by at most delta: a weight and the sum by e^delta - 1 each, of A = sum p |v|
    delta = float(64.0 * 2.0 ** -17 * sums * d ** -0.5)
    assert delta < 0.05
    size_of, _ = block_want(c["q"], c["ke"], c["ve"].abs(), c["kc"], (c["vc"].view(torch.uint8) & 0x7F).view(E4M3), c["ks"], c["vs"], c["table"],
                            lens, size, l_ext, d ** -0.5)
    check_block(o, want, tol + 2.1 * delta * size_of)


def test_offsets_beyond_32_bits(vsk):
    """A cache of more than 2^32 bytes whose last blocks are used, and rows 2^31 elements apart."""
    g = gen(23)
    size, hk, d, hq, l_ext = 64, 8, 128, 8, 2
    blocks = 68000  # 68000 * 64 * 1024 bytes
    kc, vc = (torch.empty(blocks * size, hk, d, dtype=torch.uint8, device=DEV).view(E4M3) for _ in "kv")
    ks, vs = torch.ones(blocks, hk, device=DEV), torch.ones(blocks, hk, device=DEV)
    n = 200
    table = ints([[blocks - 1, blocks - 3, 66000, blocks - 2]])
    k, v = normal(g, n, hk, d), normal(g, n, hk, d)
    pos, f = positions(g, n, "near"), frequencies(d)
    vsk.rope_append_block_fwd(None, k, v, None, None, kc, vc, ks, vs, indptr([n]), table, ints([0]), size, pos, f)
    assert vsk.read_error_flags() == 0
    t = torch.arange(n, device=DEV)
    rows = table[0].long()[t // size] * size + t % size
    page = table[0].long()[t // size]
    codes = (v.float() / vs[page][..., None]).clamp(-TOP, TOP).to(E4M3).view(torch.uint8)
    assert torch.equal(vc.view(torch.uint8)[rows], codes)
    q, ke, ve = normal(g, l_ext, hq, d), normal(g, l_ext, hk, d), normal(g, l_ext, hk, d)
    c = dict(q=q, ke=ke, ve=ve, kc=kc, vc=vc, ks=ks, vs=vs, qo=indptr([l_ext]), table=table, lens=ints([n]))
    o = run_block(vsk, c, size, l_ext)
    assert vsk.read_error_flags() == 0
    check_block(o, *block_want(q, ke, ve, kc, vc, ks, vs, table, [n], size, l_ext, d ** -0.5))
    del kc, vc, c
    torch.cuda.empty_cache()
    base = torch.zeros((1 << 31) + 4096, dtype=BF16, device=DEV)
    x = base.as_strided((2, 3, 64), (1 << 31, 64, 1))
    x.copy_(normal(g, 2, 3, 64))
    out, kk = torch.empty(2, 3, 64, dtype=BF16, device=DEV), normal(g, 2, 1, 64)
    vsk.rope_fwd(x, kk, out, torch.empty_like(kk), ints([7, 9]), frequencies(64))
    check_rotated(out, *turned64(x, ints([7, 9]), frequencies(64), False, 1.0), 1.0)
    vsk.rope_fwd(out, kk, x, torch.empty_like(kk), ints([0, 0]), frequencies(64))
    assert torch.equal(x, out)


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("d,inter", [(64, False), (128, True), (256, False)])
def test_prompt_append_and_verify_over_blocks(vsk, d, inter):
    """A prompt and two rounds of drafts, as a server runs them."""
    g = gen(d)
    size, hq, hk, l_ext = 16, 8, 2, 3
    prompt, rot = [100, 1, 37], d // 2
    freq, factor = vsk.rope_frequencies(rot, 10000.0, "ramp", 4.0, 4096)
    kc, vc, ks, vs = block_cache(g, 40, size, hk, d)
    table = table_of(g, [x + 40 for x in prompt], size, 40)

    def project(n):
        x = normal(g, n, hq + 2 * hk, d)
        return x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]

    # the prompt: rotated in place, appended, attended
    n = sum(prompt)
    q, k, v = project(n)
    raw_q, raw_k = q.clone(), k.clone()
    pos = torch.cat([torch.arange(x, device=DEV) for x in prompt])
    vsk.rope_append_block_fwd(q, k, v, q, k, kc, vc, ks, vs, indptr(prompt), table, ints([0] * 3), size, pos, freq, inter, factor)
    check_rotated(q, *turned64(raw_q, pos, freq, inter, factor), factor)
    check_rotated(k, *turned64(raw_k, pos, freq, inter, factor), factor)
    o = torch.empty_like(raw_q)
    vsk.prompt_attn_fwd(q, k, v, o, indptr(prompt))
    at = 0
    for x in prompt:
        qq, kk, vv = (t[at:at + x].to(F64) for t in (q, k, v))
        s = torch.einsum("ihd,jhd->hij", qq, kk.repeat_interleave(hq // hk, 1)) * d ** -0.5
        s = s.masked_fill(~torch.ones(x, x, dtype=torch.bool, device=DEV).tril(), -math.inf)
        want = torch.einsum("hij,jhd->ihd", torch.softmax(s, 2), vv.repeat_interleave(hq // hk, 1))
        assert float((o[at:at + x].to(F64) - want).abs().max()) < 0.05
        at += x
    held = list(prompt)
    for taken in ([3, 1, 2], [0, 3, 1]):  # drafts accepted a round
        q, k, v = project(3 * l_ext)
        pos = torch.cat([torch.arange(x, x + l_ext, device=DEV) for x in held])
        qr, kr = torch.empty_like(raw_q[:9]), torch.empty_like(raw_k[:9])
        vsk.rope_fwd(q, k, qr, kr, pos, freq, inter, factor)
        o = torch.empty_like(qr)
        vsk.verify_splitkv_block_fwd(qr, kr, v, o, kc, vc, ks, vs, indptr([l_ext] * 3), table, ints(held), size, l_ext)
        check_block(o, *block_want(qr, kr, v, kc, vc, ks, vs, table, held, size, l_ext, d ** -0.5))
        # the accepted ones into the cache
        keep = torch.cat([torch.arange(b * l_ext, b * l_ext + t, device=DEV) for b, t in enumerate(taken)])
        old = [x.clone() for x in (kc, vc, ks, vs)]
        vsk.rope_append_block_fwd(None, k[keep], v[keep], None, None, kc, vc, ks, vs, indptr(taken), table, ints(held), size, pos[keep],
                                  freq, inter, factor)
        check_block_append(k[keep], v[keep], kc, vc, ks, vs, old, table, held, taken, size, pos[keep], freq, inter, factor)
        held = [a + b for a, b in zip(held, taken)]
    assert vsk.read_error_flags() == 0


def test_append_and_verify_over_a_pool(vsk):
    """The pool form: the rows that rope_append_fwd stores are the prefix of verify_splitkv_fwd."""
    g = gen(2)
    hq, hk, d, l_ext, n = 8, 2, 128, 4, 300
    x = normal(g, n, hq + 2 * hk, d)
    kb, vb = torch.zeros(400, hk, d, dtype=BF16, device=DEV), torch.zeros(400, hk, d, dtype=BF16, device=DEV)
    loc = torch.randperm(400, generator=g, device=DEV)[:n]
    freq = frequencies(d)
    vsk.rope_append_fwd(None, x[:, hq:hq + hk], x[:, hq + hk:], None, None, kb, vb, loc, torch.arange(n, device=DEV), freq)
    y = normal(g, l_ext, hq + 2 * hk, d)
    q, k, v = (t.contiguous() for t in (y[:, :hq], y[:, hq:hq + hk], y[:, hq + hk:]))
    vsk.rope_fwd(q, k, q, k, torch.arange(n, n + l_ext, device=DEV), freq)
    o = torch.empty_like(q)
    assert vsk.verify_splitkv_fwd(q, k, v, o, kb, vb, ints([0, l_ext]), ints([0, n]), loc, None, True, None, l_ext, 1.0, 1.0)
    keys, vals = torch.cat([kb[loc], k]).to(F64), torch.cat([vb[loc], v]).to(F64)
    s = torch.einsum("ihd,jhd->hij", q.to(F64), keys.repeat_interleave(hq // hk, 1)) * d ** -0.5
    s = s.masked_fill(~torch.ones(l_ext, n + l_ext, dtype=torch.bool, device=DEV).tril(n), -math.inf)
    want = torch.einsum("hij,jhd->ihd", torch.softmax(s, 2), vals.repeat_interleave(hq // hk, 1))
    assert float((o.to(F64) - want).abs().max()) < 0.02


# ---------------------------------------------------------------- the binding

def test_binding_names_what_is_no_dense_cuda_tensor(vsk):
    q, k = (torch.zeros(2, 1, 64, dtype=BF16, device=DEV) for _ in "qk")
    pos, f = ints([0, 1]), frequencies(64)
    with pytest.raises(ValueError, match="k must be a CUDA tensor"):
        vsk.rope_fwd(q, k.cpu(), q, k, pos, f)
    with pytest.raises(ValueError, match="positions must be a CUDA tensor"):
        vsk.rope_fwd(q, k, q, k, [0, 1], f)
    with pytest.raises(ValueError, match="strided"):
        vsk.rope_fwd(q, k, q, k, pos.to_sparse(), f)
    with pytest.raises(ValueError, match="inv_freq must be float32"):
        vsk.rope_fwd(q, k, q, k, pos, f.double())
    with pytest.raises(ValueError, match="3-d"):
        vsk.rope_fwd(q[None], k, q, k, pos, f)
    # a scalar, an empty and a five-dimensional tensor are told apart from what is wanted
    for bad in (torch.zeros((), device=DEV, dtype=BF16), torch.zeros(0, device=DEV, dtype=BF16), q[None, None]):
        with pytest.raises(ValueError, match="3-d"):
            vsk.rope_fwd(bad, k, q, k, pos, f)
