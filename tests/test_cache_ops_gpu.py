"""GPU tests of the calls around the verify call against plain 64-bit forms.

Tolerances, element by element.  Attention: the kernels round the softmax
weights P to bf16 (each off by at most eps/2 = 2^-8 of itself) and the output
to bf16 (2^-8 of itself); the sums are 32-bit.  With A = sum_j p_j |v_j| the
output is therefore within 2^-8 (A + |o| (1 + 2^-8)) of the exact one, plus
what 32-bit scores leave in the weights: D <= 256 products summed in 32 bits
are off by at most D 2^-24 sum |q||k| sm_scale, for the N(0, 1) rows used here
(sum |q||k| sm_scale <= 16) under 256 * 16 * 2^-24 = 2^-12, so 2^-12 A.
Integers are equal.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F64 = torch.bfloat16, torch.float64
E4M3 = torch.float8_e4m3fn


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


def indptr(lens):
    return torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device=DEV)


def attend64(q, k, v, visible, scale, v_abs=False):
    """q [n, h, d], k and v [m, h_kv, d] in 64 bits, visible [n, m]: (o, A)."""
    g = q.shape[1] // k.shape[1]
    o, a = torch.empty_like(q), torch.empty_like(q)
    for h in range(q.shape[1]):
        x = (q[:, h] @ k[:, h // g].T) * scale
        x = x.masked_fill(~visible, -math.inf)
        p = torch.softmax(x, 1)
        vh = v[:, h // g]
        o[:, h] = p @ vh
        a[:, h] = p @ vh.abs()
    return o, a


def check_attention(got, want, a):
    got = got.to(F64)
    tol = 2.0 ** -8 * (a + want.abs() * (1 + 2.0 ** -8)) + 2.0 ** -12 * a + 1e-30
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float(((got - want).abs() / tol).nan_to_num(9e9).max()))


# ---------------------------------------------------------------- prompts

def prompt_case(lens, hq, hk, d, seed=0, extra=0, fused=False):
    g = gen(seed)
    n = sum(lens) + extra
    if fused:
        x = normal(g, n, hq + 2 * hk, d)
        q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    else:
        q, k, v = normal(g, n, hq, d), normal(g, n, hk, d), normal(g, n, hk, d)
    return q, k, v, indptr(lens)


def prompt_want(q, k, v, lens, scale):
    o, a, at = torch.zeros(q.shape, dtype=F64, device=DEV), torch.zeros(q.shape, dtype=F64, device=DEV), 0
    for n in lens:
        s = slice(at, at + n)
        vis = torch.ones(n, n, dtype=torch.bool, device=DEV).tril()
        o[s], a[s] = attend64(q[s].to(F64), k[s].to(F64), v[s].to(F64), vis, scale)
        at += n
    return o, a


PROMPTS = [
    # (lengths, h_q, h_kv, d)
    ((1,), 1, 1, 64), ((1,), 32, 8, 128), ((1, 1, 1), 8, 1, 256), ((2, 0, 3), 4, 2, 128), ((0, 0, 5, 0), 3, 1, 64),
    ((127, 128, 129), 2, 2, 128), ((63, 64, 65), 4, 1, 128), ((31, 32, 33, 255, 256, 257), 8, 2, 64),
    ((200,), 5, 1, 128), ((333, 17), 14, 2, 256), ((77, 191), 6, 2, 64), ((129,), 16, 1, 128), ((40,), 128, 1, 64),
    ((9, 70), 100, 1, 128), ((1025, 511), 16, 2, 256), ((4097,), 4, 1, 128), ((2300, 1, 700), 7, 7, 64),
    (tuple(range(0, 90)), 4, 2, 128),
]


@pytest.mark.parametrize("case", PROMPTS, ids=lambda c: f"b{len(c[0])}n{sum(c[0])}h{c[1]}x{c[2]}d{c[3]}")
def test_prompt_against_64_bits(vsk, case):
    lens, hq, hk, d = case
    q, k, v, ptr = prompt_case(lens, hq, hk, d, extra=5)
    o = torch.full_like(q, 7.0)
    vsk.prompt_attn_fwd(q, k, v, o, ptr)
    n = sum(lens)
    want, a = prompt_want(q, k, v, lens, d ** -0.5)
    check_attention(o[:n], want[:n], a[:n])
    assert bool((o[n:] == 7.0).all())  # rows behind the last sequence
    assert vsk.read_error_flags() == 0


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompt_strided_rows_and_scale(vsk, d):
    lens = (150, 3, 260)
    q, k, v, ptr = prompt_case(lens, 6, 3, d, seed=3, fused=True)
    big = torch.zeros(sum(lens), 8, d, dtype=BF16, device=DEV)
    o = big[:, 1:7]
    vsk.prompt_attn_fwd(q, k, v, o, ptr, sm_scale=0.3 * d ** -0.5)
    want, a = prompt_want(q, k, v, lens, 0.3 * d ** -0.5)
    check_attention(o, want, a)
    assert bool((big[:, 0] == 0).all()) and bool((big[:, 7] == 0).all())


@pytest.mark.parametrize("d", [64, 256])
def test_prompt_head_major_and_single_head_layouts(vsk, d):
    lens = (140, 33)
    g = gen(4)
    q, k, v = (normal(g, h, sum(lens), d).transpose(0, 1) for h in (4, 2, 2))
    o = torch.zeros(4, sum(lens), d, dtype=BF16, device=DEV).transpose(0, 1)
    vsk.prompt_attn_fwd(q, k, v, o, indptr(lens))
    check_attention(o, *prompt_want(q, k, v, lens, d ** -0.5))
    # one KV head behind every query head: an expanded view
    k1, v1 = k[:, :1].expand(-1, 2, -1), v[:, :1].expand(-1, 2, -1)
    vsk.prompt_attn_fwd(q, k1, v1, o, indptr(lens))
    check_attention(o, *prompt_want(q, k1, v1, lens, d ** -0.5))


def test_prompt_many_sequences_and_a_vanishing_scale(vsk):
    lens = (3, 0, 1, 2) * 700
    q, k, v, ptr = prompt_case(lens, 4, 2, 64, seed=6)
    o = torch.zeros_like(q)
    vsk.prompt_attn_fwd(q, k, v, o, ptr, sm_scale=1e-45)  # all scores alike: means
    want, a = prompt_want(q, k, v, lens, 0.0)
    check_attention(o, want, a)
    vsk.prompt_attn_fwd(q, k, v, o, ptr)
    check_attention(o, *prompt_want(q, k, v, lens, 0.125))


def test_shared_head_major_pool(vsk):
    c = shared_case(700, (40, 0, 99), 4, 8, 2, 128, seed=25)
    c["kb"], c["vb"] = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (c["kb"], c["vb"]))
    check_attention(run_shared(vsk, c), *shared_want(c, 128 ** -0.5))


def test_prompt_rows_of_four_byte_alignment(vsk):
    lens, hq, d = (100, 45), 4, 128
    g = gen(5)
    flat = normal(g, sum(lens) * hq * d + 2)
    q = flat[2:].view(sum(lens), hq, d)
    oflat = torch.zeros_like(flat)
    o = oflat[2:].view_as(q)
    k, v = normal(g, sum(lens), 2, d), normal(g, sum(lens), 2, d)
    vsk.prompt_attn_fwd(q, k, v, o, indptr(lens))
    check_attention(o, *prompt_want(q, k, v, lens, d ** -0.5))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_prompt_hidden_values_stay_hidden(vsk, d, bad):
    """K and V of a later token, of the next sequence and of rows outside every sequence hold no number."""
    lens = (170, 60)
    q, k, v, ptr = prompt_case(lens, 4, 2, d, seed=11, extra=9)
    want, a = prompt_want(q, k, v, lens, d ** -0.5)
    k[230:], v[230:] = bad, bad
    k[150], v[150, :, 3] = bad, bad        # seen by rows 150.. of the first sequence
    k[170 + 59], v[170 + 59] = bad, bad    # seen by the last row of the second
    o = torch.zeros_like(q)
    vsk.prompt_attn_fwd(q, k, v, o, ptr)
    keep = torch.ones(239, dtype=torch.bool, device=DEV)
    keep[150:170] = False
    keep[229:] = False
    check_attention(o[keep], want[keep], a[keep])
    assert not o[150:170].isfinite().any() and not o[229].isfinite().any()


def test_prompt_values_not_finite_reach_the_rows_that_see_them(vsk):
    lens, d = (300,), 128
    q, k, v, ptr = prompt_case(lens, 4, 2, d, seed=12)
    want, a = prompt_want(q, k, v, lens, d ** -0.5)
    v[200, 0, 5] = float("inf")
    v[290, 1, 7] = float("-inf")
    o = torch.zeros_like(q)
    vsk.prompt_attn_fwd(q, k, v, o, ptr)
    seen = torch.zeros(o.shape, dtype=torch.bool, device=DEV)
    seen[200:, :2, 5] = True
    seen[290:, 2:, 7] = True
    assert bool((o[200:, :2, 5] == math.inf).all()) and bool((o[290:, 2:, 7] == -math.inf).all())
    check_attention(o[~seen], want[~seen], a[~seen])


def test_prompt_large_scores_raise_the_reference(vsk):
    """Scores that grow along the keys by far more than the headroom, so the running reference moves often."""
    lens, d = (700,), 128
    q, k, v, ptr = prompt_case(lens, 2, 1, d, seed=13)
    k = (k.float() * torch.linspace(0.1, 6.0, 700, device=DEV)[:, None, None]).to(BF16)
    o = torch.zeros_like(q)
    vsk.prompt_attn_fwd(q, k, v, o, ptr)
    want, a = prompt_want(q, k, v, lens, d ** -0.5)
    # scores up to 6 times as large: 6 * 2^-12 A of the header's last term
    check_attention(o, want, a * (1 + 6 * 2.0 ** -4))


def test_prompt_bad_indptr_is_flagged(vsk):
    q, k, v, _ = prompt_case((60,), 4, 2, 64, seed=14)
    ptr = torch.tensor([0, 20, 10, 40, 99], dtype=torch.int32, device=DEV)  # the second and the last pair are wrong
    o = torch.full_like(q, 7.0)
    vsk.prompt_attn_fwd(q, k, v, o, ptr)
    assert vsk.read_error_flags() == 4
    want, a = prompt_want(q[:20], k[:20], v[:20], (20,), 0.125)
    check_attention(o[:10], want[:10], a[:10])
    assert bool((o[40:] == 7.0).all())


# ---------------------------------------------------------------- a shared prefix

def shared_case(s, own, l, hq, hk, d, pool="bf16", seed=0, extra=0):
    g = gen(seed)
    t, b = sum(own), len(own)
    n = s + t + extra
    dt = E4M3 if pool == "e4m3" else BF16
    perm = torch.randperm(n, generator=g, device=DEV)
    return {
        "q": normal(g, b * l, hq, d), "ke": normal(g, b * l, hk, d), "ve": normal(g, b * l, hk, d),
        "kb": normal(g, n, hk, d).to(dt), "vb": normal(g, n, hk, d).to(dt), "sh": perm[:s].clone(),
        "kvi": perm[s:s + t].clone(), "kvp": indptr(own), "qo": indptr([l] * b), "l": l, "own": own,
    }


def rows64(pool, loc):
    return pool.float()[loc].to(F64) if pool.dtype == E4M3 else pool[loc].to(F64)


def shared_want(c, scale, ks=1.0, vs=1.0):
    l, at = c["l"], 0
    o, a = torch.empty(c["q"].shape, dtype=F64, device=DEV), torch.empty(c["q"].shape, dtype=F64, device=DEV)
    for b, n in enumerate(c["own"]):
        r = slice(b * l, (b + 1) * l)
        loc = torch.cat([c["sh"], c["kvi"][at:at + n]]).long()
        k = torch.cat([rows64(c["kb"], loc) * ks, c["ke"][r].to(F64)])
        v = torch.cat([rows64(c["vb"], loc) * vs, c["ve"][r].to(F64)])
        vis = torch.ones(l, len(loc) + l, dtype=torch.bool, device=DEV).tril(len(loc))
        o[r], a[r] = attend64(c["q"][r].to(F64), k, v, vis, scale)
        at += n
    return o, a


def run_shared(vsk, c, **kw):
    o = torch.full_like(c["q"], float("nan"))
    vsk.verify_splitkv_shared_fwd(c["q"], c["ke"], c["ve"], o, c["kb"], c["vb"], c["qo"], c["kvp"], c["kvi"], c["sh"],
                                  c["l"], **kw)
    return o


SHARED = [
    # (shared keys, own lengths, drafts, h_q, h_kv, d, pool)
    (1, (0,), 1, 1, 1, 64, "bf16"), (0, (5, 70), 4, 4, 2, 64, "bf16"), (0, (0, 0), 3, 4, 2, 128, "bf16"),
    (127, (1, 0, 33), 2, 6, 2, 128, "bf16"), (128, (64, 96), 4, 4, 1, 64, "bf16"), (129, (7,), 8, 16, 1, 128, "bf16"),
    (1000, (0, 0, 0, 0, 0), 1, 8, 8, 128, "bf16"), (513, tuple(range(40)), 4, 16, 4, 128, "bf16"),
    (5000, (300, 200), 5, 15, 3, 64, "bf16"), (3001, (17, 900, 0), 4, 16, 2, 256, "bf16"),
    (700, (30,) * 9, 7, 14, 2, 256, "bf16"), (260, (0, 9), 128, 2, 2, 128, "bf16"), (260, (3, 9), 1, 128, 1, 64, "bf16"),
    (1, (0, 2), 2, 4, 2, 256, "e4m3"), (385, (60, 0, 5), 4, 8, 2, 64, "e4m3"), (2049, (100, 33), 3, 9, 3, 128, "e4m3"),
    (4000, (0, 512, 100), 4, 16, 2, 256, "e4m3"), (8192, (0, 100, 512, 3, 40, 500, 10, 0), 4, 16, 2, 256, "e4m3"),
    (40000, (0, 7, 0), 4, 16, 2, 256, "e4m3"), (40000, (0, 7, 0), 4, 16, 2, 256, "bf16"), (40000, (9,), 4, 16, 2, 128, "e4m3"), (9000, (10,) * 70, 4, 8, 1, 128, "e4m3"),
]


@pytest.mark.parametrize("case", SHARED, ids=lambda c: f"s{c[0]}b{len(c[1])}l{c[2]}h{c[3]}x{c[4]}d{c[5]}{c[6]}")
def test_shared_against_64_bits(vsk, case):
    c = shared_case(*case, seed=21, extra=3)
    unused = torch.ones(c["kb"].shape[0], dtype=torch.bool, device=DEV)
    unused[c["sh"]] = False
    unused[c["kvi"]] = False
    for pool in (c["kb"], c["vb"]):  # rows no sequence refers to hold no number
        pool.view(torch.uint8 if pool.dtype == E4M3 else torch.int16)[unused] = 0x7F if pool.dtype == E4M3 else 0x7FC0
    o = run_shared(vsk, c)
    check_attention(o, *shared_want(c, case[5] ** -0.5))
    assert vsk.read_error_flags() == 0


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("d,hq,hk", [(64, 4, 1), (128, 8, 2), (256, 16, 2)])
@pytest.mark.parametrize("own", [(0, 1) * 20, (0,) * 30 + (1500,) + (2,) * 9, (3, 17, 0, 64, 30, 5) * 6],
                         ids=["none or one", "one long", "short"])
def test_shared_with_short_own_prefixes(vsk, own, d, hq, hk, pool):
    c = shared_case(200, own, 4, hq, hk, d, pool, seed=27)
    check_attention(run_shared(vsk, c), *shared_want(c, d ** -0.5))
    assert vsk.read_error_flags() == 0


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("ks,vs", [(0.5, 0.25), (-0.7, 2.0), (0.0, 1.0)])
def test_shared_scales(vsk, pool, ks, vs):
    c = shared_case(300, (20, 0, 150), 4, 8, 2, 128, pool, seed=22)
    c["sh"], c["kvi"] = c["sh"].int(), c["kvi"].int()
    o = run_shared(vsk, c, k_scale=ks, v_scale=vs, sm_scale=0.1)
    check_attention(o, *shared_want(c, 0.1, ks, vs))


def test_shared_equals_the_verify_call_on_joined_indices(vsk):
    c = shared_case(777, (50, 0, 301), 4, 16, 4, 128, seed=23)
    parts, at = [], 0
    for n in c["own"]:
        parts += [c["sh"], c["kvi"][at:at + n]]
        at += n
    o2 = torch.empty_like(c["q"])
    assert vsk.verify_splitkv_fwd(c["q"], c["ke"], c["ve"], o2, c["kb"], c["vb"], c["qo"],
                                  indptr([777 + n for n in c["own"]]), torch.cat(parts), None, True, None, c["l"], 1.0, 1.0)
    _, a = shared_want(c, 128 ** -0.5)
    # both are within the header's bound of the exact value
    check_attention(run_shared(vsk, c), o2.to(F64), 2 * a)


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_shared_bad_indices_are_left_out_and_flagged(vsk, pool):
    c = shared_case(400, (30, 8), 4, 8, 2, 128, pool, seed=24)
    good = dict(c)
    keep = torch.ones(400, dtype=torch.bool, device=DEV)
    keep[[3, 129, 399]] = False
    good["sh"] = c["sh"][keep]
    c["sh"][3], c["sh"][129], c["sh"][399] = -1, c["kb"].shape[0], 1 << 40
    o = run_shared(vsk, c)
    check_attention(o, *shared_want(good, 128 ** -0.5))
    assert vsk.read_error_flags() == 1
    c["sh"][:] = -5  # no shared key is left
    good["sh"] = c["sh"][:0]
    check_attention(run_shared(vsk, c), *shared_want(good, 128 ** -0.5))
    assert vsk.read_error_flags() == 1


# ---------------------------------------------------------------- attention weight of the keys

def mass_want(c, scale, ks=1.0):
    hk, l, at = c["ke"].shape[1], c["l"], 0
    g = c["q"].shape[1] // hk
    w = torch.zeros(hk, len(c["kvi"]), dtype=F64, device=DEV)
    for b, n in enumerate(c["own"]):
        r = slice(b * l, (b + 1) * l)
        k = torch.cat([rows64(c["kb"], c["kvi"][at:at + n].long()) * ks, c["ke"][r].to(F64)])
        vis = torch.ones(l, n + l, dtype=torch.bool, device=DEV).tril(n)
        for h in range(c["q"].shape[1]):
            x = (c["q"][r, h].to(F64) @ k[:, h // g].T) * scale
            p = torch.softmax(x.masked_fill(~vis, -math.inf), 1)
            w[h // g, at:at + n] += p[:, :n].sum(0)
        at += n
    return w


def check_mass(got, w, before=0.0):
    # weights: both the score (2^-12, the header) and the row's sum; then 32-bit sums of up to 130 terms
    tol = 2.0 ** -11 * w + 2.0 ** -17 * (w + before) + 1e-30
    bad = ~((got.to(F64) - (before + w)).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float(((got.to(F64) - before - w).abs() / tol).max()))


def run_mass(vsk, c, mass, **kw):
    vsk.verify_splitkv_mass(c["q"], c["ke"], c["kb"], c["qo"], c["kvp"], c["kvi"], mass, c["l"], **kw)
    return mass


MASSES = [
    # (own lengths, drafts, h_q, h_kv, d, pool)
    ((1,), 1, 1, 1, 64, "bf16"), ((0, 5, 70), 4, 4, 2, 64, "bf16"), ((64, 96), 4, 4, 1, 64, "bf16"),
    ((31, 32, 33), 2, 6, 2, 128, "bf16"), ((257, 0, 1000), 4, 16, 4, 128, "bf16"), ((5000, 4000), 4, 32, 8, 128, "bf16"),
    ((700,), 5, 15, 3, 128, "bf16"), ((300, 129), 4, 16, 2, 256, "bf16"), ((999,), 128, 2, 2, 128, "bf16"),
    ((3000, 10), 1, 128, 1, 64, "bf16"), ((40000,), 4, 8, 2, 128, "bf16"), ((9000,), 16, 16, 2, 128, "bf16"),
    ((3,), 2, 4, 2, 256, "e4m3"), ((60, 0, 5), 4, 8, 2, 64, "e4m3"), ((2000, 33), 3, 9, 3, 128, "e4m3"),
    ((4096, 8000), 4, 16, 2, 256, "e4m3"), ((17,) * 100, 4, 8, 1, 128, "e4m3"), ((2500,), 8, 64, 8, 128, "e4m3"),
]


@pytest.mark.parametrize("case", MASSES, ids=lambda c: f"b{len(c[0])}n{sum(c[0])}l{c[1]}h{c[2]}x{c[3]}d{c[4]}{c[5]}")
def test_mass_against_64_bits(vsk, case):
    c = shared_case(0, *case, seed=31, extra=2)
    c["kb"].view(torch.uint8 if case[5] == "e4m3" else torch.int16)[
        torch.ones(len(c["kb"]), dtype=torch.bool, device=DEV).index_fill_(0, c["kvi"], False)] = (
        0x7F if case[5] == "e4m3" else 0x7FC0)  # rows no sequence refers to hold no number
    t, hk = len(c["kvi"]), case[3]
    w = mass_want(c, case[4] ** -0.5)
    check_mass(run_mass(vsk, c, torch.full((hk, t), float("nan"), device=DEV)), w)
    # added to what was there, in place and as a strided view
    big = torch.rand(hk, t + 3, generator=gen(1), device=DEV)
    before = big.to(F64)
    m = big[:, 1:1 + t]
    run_mass(vsk, c, m, mass_in=m)
    check_mass(m, w, before[:, 1:1 + t])
    assert bool((big[:, 0] == before[:, 0].float()).all()) and bool((big[:, 1 + t:] == before[:, 1 + t:].float()).all())
    assert vsk.read_error_flags() == 0


def test_mass_sums_to_the_prefix_share_and_repeats_bit_for_bit(vsk):
    c = shared_case(0, (900, 40, 3000), 4, 16, 4, 128, seed=32)
    t = len(c["kvi"])
    a = run_mass(vsk, c, torch.empty(4, t, device=DEV))
    b = run_mass(vsk, c, torch.empty(4, t, device=DEV))
    assert torch.equal(a, b)
    # 16 rows a KV head, every row's weights over prefix and drafts sum to 1
    rows = a.split(c["own"], 1)
    for x in rows:
        assert bool((x.sum(1) < 16.0).all()) and bool((x.sum(1) > 12.0).all())


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("ks,qs", [(0.5, 1.0), (-0.7, 1e-4), (0.0, 1.0), (1.0, 30.0)])
def test_mass_scales(vsk, pool, ks, qs):
    c = shared_case(0, (300, 0, 77), 4, 8, 2, 128, pool, seed=33)
    c["q"] = (c["q"].float() * qs).to(BF16)
    c["kvi"] = c["kvi"].int()
    sm = 0.1 / max(qs, 1.0)  # the header's bound on the scores holds
    check_mass(run_mass(vsk, c, torch.empty(2, 377, device=DEV), k_scale=ks, sm_scale=sm), mass_want(c, sm, ks))


def test_mass_bad_indices(vsk):
    c = shared_case(0, (50, 70), 2, 4, 2, 64, seed=34)
    keep = torch.ones(120, dtype=torch.bool, device=DEV)
    keep[[7, 119]] = False
    good = dict(c, kvi=c["kvi"][keep], own=(49, 69))
    c["kvi"][7], c["kvi"][119] = -1, 120
    m = run_mass(vsk, c, torch.empty(2, 120, device=DEV))
    check_mass(m[:, keep], mass_want(good, 0.125))
    assert bool((m[:, ~keep] == 0).all())
    assert vsk.read_error_flags() == 1
    ptr = c["kvp"].clone()
    ptr[2] = 121  # past kv_indices: the second sequence is empty
    c["kvi"][7], c["kvi"][119] = 0, 1
    m = torch.full((2, 120), 7.0, device=DEV)
    run_mass(vsk, dict(c, kvp=ptr), m)
    assert vsk.read_error_flags() == 2
    assert bool((m[:, 50:] == 7.0).all()) and not bool((m[:, :50] == 7.0).any())


# ---------------------------------------------------------------- eviction

def evict_want(mass, kvi, lens, budget, recent):
    total = mass[0].clone()
    for row in mass[1:]:
        total = total + row
    total, at, ptr, keep = total.cpu(), 0, [0], []
    for n in lens:
        if n <= budget:
            k = list(range(n))
        else:
            x = total[at:at + n - recent]
            order = sorted(range(n - recent), key=lambda j: (not math.isnan(x[j]), 0.0 if math.isnan(x[j]) else -x[j].item(), j))
            k = sorted(order[:budget - recent]) + list(range(n - recent, n))
        keep += [at + j for j in k]
        ptr.append(len(keep))
        at += n
    keep = torch.tensor(keep, dtype=torch.long)
    gone = torch.ones(at, dtype=torch.bool).index_fill_(0, keep, False).nonzero()[:, 0]
    return torch.tensor(ptr, dtype=torch.int32), kvi.cpu()[keep], mass.cpu()[:, keep], kvi.cpu()[gone]


def run_evict(vsk, mass, lens, kvi, budget, recent, m=None):
    m = min(len(kvi), len(lens) * budget) if m is None else m
    out = [torch.full((len(lens) + 1,), -7, dtype=torch.int32, device=DEV), torch.full((m,), -7, dtype=kvi.dtype, device=DEV),
           torch.full((mass.shape[0], m), -7.0, device=DEV), torch.full((len(kvi),), -7, dtype=kvi.dtype, device=DEV)]
    vsk.kv_evict(mass, indptr(lens), kvi, budget, recent, *out)
    return [x.cpu() for x in out]


def check_evict(got, want):
    n, f = len(want[1]), len(want[3])
    assert torch.equal(got[0], want[0])
    assert torch.equal(got[1][:n], want[1]) and bool((got[1][n:] == -7).all())
    assert torch.equal(got[2][:, :n].nan_to_num(5e5), want[2].nan_to_num(5e5)) and bool((got[2][:, n:] == -7).all())
    assert torch.equal(got[3][:f], want[3]) and bool((got[3][f:] == -7).all())


def masses(g, h, t, kind):
    m = torch.exp(2 * torch.randn(h, t, generator=g, device=DEV))
    if kind == "ties":
        m = torch.randint(0, 3, (h, t), generator=g, device=DEV).float()
    if kind == "zero":
        m = torch.where(torch.rand(h, t, generator=g, device=DEV) < 0.5, -0.0, 0.0)
    if kind == "signed":
        m = torch.randn(h, t, generator=g, device=DEV)
        m[:, ::7] = math.inf
        m[:, 3::11] = -math.inf
        m[:, 5::13] = math.nan
    return m


EVICTS = [
    # (lengths, h_kv, budget, recent)
    ((1,), 1, 1, 0), ((0, 0), 2, 3, 1), ((5,), 1, 1, 1), ((5, 0, 9), 3, 4, 0), ((5, 4, 3), 2, 4, 4), ((700, 256, 257, 0, 1), 2, 256, 32),
    ((513, 1200), 8, 100, 99), ((2048, 2049, 5000), 4, 1000, 7), ((30000,), 2, 4096, 512), ((70000, 3), 1, 50, 1),
    (tuple(range(0, 600, 3)), 2, 64, 16), ((40000, 33), 3, 39999, 12345),
]


@pytest.mark.parametrize("kind", ["heavy", "ties", "zero", "signed"])
@pytest.mark.parametrize("case", EVICTS, ids=lambda c: f"b{len(c[0])}n{sum(c[0])}h{c[1]}k{c[2]}r{c[3]}")
def test_evict_is_exact(vsk, case, kind):
    lens, h, budget, recent = case
    g = gen(41)
    t = sum(lens)
    mass, kvi = masses(g, h, t, kind), torch.randperm(t + 9, generator=g, device=DEV)[:t].clone()
    check_evict(run_evict(vsk, mass, lens, kvi, budget, recent), evict_want(mass, kvi, lens, budget, recent))
    assert vsk.read_error_flags() == 0


def test_evict_strided_rows_and_int32(vsk):
    g = gen(42)
    lens = (300, 50, 411)
    mass = masses(g, 4, 800, "heavy")[1:4, 5:766]
    kvi = torch.randperm(761, generator=g, device=DEV).int()
    check_evict(run_evict(vsk, mass, lens, kvi, 128, 16), evict_want(mass, kvi, lens, 128, 16))


def test_evict_of_one_very_long_sequence(vsk):
    """More keys a CTA than shared memory holds."""
    g = gen(43)
    t = 500_000
    mass, kvi = masses(g, 2, t, "ties"), torch.randperm(t, generator=g, device=DEV)
    total = mass[0] + mass[1]
    k, rec = 123_457, 1000
    got = run_evict(vsk, mass, (t,), kvi, k, rec)
    order = torch.sort(total[:t - rec], descending=True, stable=True).indices[:k - rec]
    keep = torch.cat([order.sort().values, torch.arange(t - rec, t, device=DEV)])
    gone = torch.ones(t, dtype=torch.bool, device=DEV).index_fill_(0, keep, False)
    check_evict(got, (torch.tensor([0, k], dtype=torch.int32), kvi[keep].cpu(), mass[:, keep].cpu(), kvi[gone].cpu()))


@pytest.mark.parametrize("lens", [(60000,) + (500,) * 31, (3,) * 100 + (60000,) + (700,) * 100, (9000,) * 20])
def test_evict_of_uneven_lengths(vsk, lens):
    g = gen(45)
    t = sum(lens)
    mass, kvi = masses(g, 2, t, "ties"), torch.randperm(t, generator=g, device=DEV)
    check_evict(run_evict(vsk, mass, lens, kvi, 600, 30), evict_want(mass, kvi, lens, 600, 30))


def test_evict_flags_bad_indptr_and_short_outputs(vsk):
    g = gen(44)
    mass, kvi = masses(g, 2, 100, "heavy"), torch.arange(100, device=DEV)
    out = [torch.full((4,), -7, dtype=torch.int32, device=DEV), torch.full((100,), -7, device=DEV),
           torch.full((2, 100), -7.0, device=DEV), torch.full((100,), -7, device=DEV)]
    ptr = torch.tensor([0, 40, 30, 101], dtype=torch.int32, device=DEV)
    vsk.kv_evict(mass, ptr, kvi, 10, 2, *out)
    assert vsk.read_error_flags() == 2
    assert out[0].tolist() == [0, 10, 10, 10] and bool((out[1][10:] == -7).all())
    big = [torch.full((20,), -7, device=DEV), torch.full((2, 20), -7.0, device=DEV), torch.full((20,), -7, device=DEV)]
    short = [big[0][:12], big[1][:, :12], big[2][:15]]
    vsk.kv_evict(mass, indptr((50, 50)), kvi, 10, 2, out[0][:3], *short)
    assert vsk.read_error_flags() == 32
    want = evict_want(mass, kvi, (50, 50), 10, 2)
    assert torch.equal(short[0].cpu(), want[1][:12]) and torch.equal(short[2].cpu(), want[3][:15])
    assert bool((big[0][12:] == -7).all()) and bool((big[1][:, 12:] == -7).all()) and bool((big[2][15:] == -7).all())


# ---------------------------------------------------------------- together, streams, graphs

def test_a_run_of_all_four(vsk):
    """Prompts fill the cache; a batch behind the first prompt's rows is verified; the keys' weights decide what stays;
    the next verify call reads the cut-down index."""
    g, hq, hk, d, l = gen(51), 8, 2, 128, 4
    lens = (300, 120, 77)
    q, k, v, ptr = prompt_case(lens, hq, hk, d, seed=52)
    n = sum(lens)
    o = torch.empty_like(q)
    vsk.prompt_attn_fwd(q, k, v, o, ptr)
    want, a = prompt_want(q, k, v, lens, d ** -0.5)
    check_attention(o, want, a)
    slots = torch.randperm(n + 40, generator=g, device=DEV)[:n].clone()
    kb, vb = normal(g, n + 40, hk, d), normal(g, n + 40, hk, d)
    kb[slots], vb[slots] = k, v
    own = (120, 77)
    c = {"q": normal(g, 2 * l, hq, d), "ke": normal(g, 2 * l, hk, d), "ve": normal(g, 2 * l, hk, d), "kb": kb, "vb": vb,
         "sh": slots[:300], "kvi": slots[300:], "kvp": indptr(own), "qo": indptr([l] * 2), "l": l, "own": own}
    check_attention(run_shared(vsk, c), *shared_want(c, d ** -0.5))
    m = run_mass(vsk, c, torch.empty(hk, 197, device=DEV))
    check_mass(m, mass_want(c, d ** -0.5))
    out = [torch.empty(3, dtype=torch.int32, device=DEV), torch.empty(197, dtype=torch.long, device=DEV),
           torch.empty(hk, 197, device=DEV), torch.empty(197, dtype=torch.long, device=DEV)]
    vsk.kv_evict(m, c["kvp"], c["kvi"], 64, 16, *out)
    w = evict_want(m, c["kvi"], own, 64, 16)
    assert out[0].tolist() == [0, 64, 128] and torch.equal(out[1][:128].cpu(), w[1]) and torch.equal(out[3][:69].cpu(), w[3])
    c2 = dict(c, kvi=out[1][:128].clone(), kvp=out[0], own=(64, 64))
    check_attention(run_shared(vsk, c2), *shared_want(c2, d ** -0.5))


def test_on_another_stream_and_replayed_from_a_graph(vsk):
    """Each call on a side stream and captured into one graph, replayed on changed inputs."""
    lens, d = (200, 55), 128
    q, k, v, ptr = prompt_case(lens, 8, 2, d, seed=61)
    c = shared_case(300, (40, 90), 4, 8, 2, d, seed=62)
    t = 130
    o, os = torch.zeros_like(q), torch.zeros_like(c["q"])
    m = torch.zeros(2, t, device=DEV)
    out = [torch.zeros(3, dtype=torch.int32, device=DEV), torch.zeros(t, dtype=torch.long, device=DEV),
           torch.zeros(2, t, device=DEV), torch.zeros(t, dtype=torch.long, device=DEV)]
    ws = torch.zeros(vsk.shared_workspace_size(2, 8, 2, d, 4), dtype=torch.uint8, device=DEV)

    def calls(**kw):
        vsk.prompt_attn_fwd(q, k, v, o, ptr, **kw)
        vsk.verify_splitkv_shared_fwd(c["q"], c["ke"], c["ve"], os, c["kb"], c["vb"], c["qo"], c["kvp"], c["kvi"],
                                      c["sh"], 4, **kw)
        run_mass(vsk, c, m, **kw)
        vsk.kv_evict(m, c["kvp"], c["kvi"], 32, 8, *out, **kw)

    def check():
        check_attention(o, *prompt_want(q, k, v, lens, d ** -0.5))
        check_attention(os, *shared_want(c, d ** -0.5))
        check_mass(m, mass_want(c, d ** -0.5))
        w = evict_want(m, c["kvi"], c["own"], 32, 8)
        assert torch.equal(out[1][:64].cpu(), w[1]) and torch.equal(out[3][:66].cpu(), w[3])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    side.synchronize()
    check()
    calls(stream=side)
    side.synchronize()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ValueError, match="workspace"):
            vsk.prompt_attn_fwd(q, k, v, o, ptr)
        calls(workspace=ws)
    for seed in (63, 64):
        g = gen(seed)
        for x in (q, k, v, c["q"], c["ke"], c["ve"], c["kb"], c["vb"]):
            x.copy_(normal(g, *x.shape))
        graph.replay()
        torch.cuda.synchronize()
        check()
    flags = vsk.read_error_flags(ws)
    assert flags == 0


def test_many_calls_in_flight_on_two_streams(vsk):
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    cases = [shared_case(500 + 100 * i, (60 * i, 33), 4, 8, 2, 128, seed=70 + i) for i in range(4)]
    outs = []
    torch.cuda.synchronize()
    for i in range(16):
        with torch.cuda.stream((a, b)[i % 2]):
            outs.append(run_shared(vsk, cases[i % 4]))
    torch.cuda.synchronize()
    for i in range(16):
        assert torch.equal(outs[i], outs[i % 4])
    for i in range(4):
        check_attention(outs[i], *shared_want(cases[i], 128 ** -0.5))
