"""GPU tests of the calls around the verify call at their edges: host threads,
values and sizes that the tests of their formulas do not reach."""
import math
import threading

import pytest
import torch

import test_cache_ops_gpu as base
from test_cache_ops_gpu import (BF16, DEV, E4M3, F64, check_attention, gen, indptr, normal, run_mass, run_shared,  # noqa: F401
                                shared_case, shared_want, vsk)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- host threads

@pytest.mark.parametrize("form", ["shared prefix", "stream and combine"])
def test_threads_on_one_stream_keep_their_partials(vsk, form):
    """Calls of several launches from four host threads on one stream: the threads have one workspace, in which the
    launches of a call hand partials on, so no other call's launches may come between them."""
    d, l = 128, 4
    cases = [shared_case(700, (150, 40, 333, 90), l, 8, 2, d, seed=90 + i) for i in range(4)]
    assert vsk.call_form(4, 8, 2, d, d, l, 613) == "stream_only" and vsk.launches_per_call(4, 8, 2, d, l, 613) == 2

    def run(c, o):
        if form == "shared prefix":
            vsk.verify_splitkv_shared_fwd(c["q"], c["ke"], c["ve"], o, c["kb"], c["vb"], c["qo"], c["kvp"], c["kvi"],
                                          c["sh"], l)
        else:
            assert vsk.verify_splitkv_fwd(c["q"], c["ke"], c["ve"], o, c["kb"], c["vb"], c["qo"], c["kvp"], c["kvi"], None,
                                          True, None, l, 1.0, 1.0)

    alone = []
    for c in cases:
        alone.append(torch.empty_like(c["q"]))
        run(c, alone[-1])
    if form == "shared prefix":
        for c, o in zip(cases, alone):
            check_attention(o, *shared_want(c, d ** -0.5))
    calls, outs, failed, start = 100, [[] for _ in cases], [], threading.Barrier(len(cases))
    for i, c in enumerate(cases):
        outs[i] = [torch.full_like(c["q"], float("nan")) for _ in range(calls)]
    torch.cuda.synchronize()

    def work(i):
        try:
            start.wait(30)
            for o in outs[i]:
                run(cases[i], o)
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not failed, failed
    torch.cuda.synchronize()
    wrong = [sum(not torch.equal(o, alone[i]) for o in outs[i]) for i in range(len(cases))]
    assert wrong == [0] * len(cases), f"calls of {calls} with another call's partials: {wrong}"
    assert vsk.read_error_flags() == 0


def test_threads_and_the_library_owned_workspace(vsk):
    """Calls without a workspace from four threads on one stream, of sizes that make the library's buffer grow: it is not
    replaced between its choice and a launch."""
    import ctypes

    from speculative_decode_verify_prefix_gb300 import _native

    d, l = 128, 4
    cases = [shared_case(500, (90,) * b, l, 8, 2, d, seed=95 + b) for b in (1, 3, 9, 40)]
    alone = [run_shared(vsk, c) for c in cases]
    outs = [[torch.full_like(c["q"], float("nan")) for _ in range(25)] for c in cases]
    ref, failed, start = vsk.api._ref, [], threading.Barrier(len(cases))
    stream = torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()

    def work(i):
        try:
            c = cases[i]
            start.wait(30)
            for o in outs[i]:
                t = (c["q"], c["ke"], c["ve"], o, c["kb"], c["vb"], c["qo"], c["kvp"], c["kvi"], c["sh"])
                if not _native.lib().verify_splitkv_shared_fwd(*[ref(x) for x in t], l, 1.0, 1.0, 0.0, None, 0, ctypes.c_void_p(stream)):
                    failed.append(vsk.last_error())
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    torch.cuda.synchronize()
    assert not failed, failed
    for i, c in enumerate(cases):
        assert all(torch.equal(o, alone[i]) for o in outs[i])


# ---------------------------------------------------------------- sizes

def test_shared_workspace_size_of_shapes_that_no_call_takes(vsk):
    assert vsk.shared_workspace_size(2, 8, 2, 128, 4) > 0
    for shape in ((2, 0, 2, 128, 4), (2, -4, 2, 128, 4), (2, 8, 0, 128, 4), (0, 8, 2, 128, 4), (2, 8, 2, 96, 4),
                  (2, 8, 2, 128, 0), (2, 7, 2, 128, 4)):
        assert vsk.shared_workspace_size(*shape) == 0, shape


# ---------------------------------------------------------------- e4m3 pools behind a shared prefix
#
# Softmax weights of e4m3 pools are held in f16, as in the verify call: 2^-11 of
# themselves, so 2^-11 A in the output for the header's 2^-8 A of bf16 ones, and
# below f16's normal range an absolute 2^-25 of the row's largest weight (2^-32
# for shared rows) a key.


def check_f16_weights(got, want, a, c, vs=1.0):
    top = float(c["vb"].float().nan_to_num(0.0).abs().max()) * abs(vs)
    small = (max(c["own"]) * 2.0 ** -25 + len(c["sh"]) * 2.0 ** -32) * top
    tol = (2.0 ** -11 + 2.0 ** -12) * a + small + 2.0 ** -8 * want.abs() * (1 + 2.0 ** -8)
    off = ((got.to(F64) - want).abs() / tol).max()
    assert bool(off <= 1), float(off)


@pytest.mark.parametrize("d,hq,hk", [(64, 4, 2), (128, 8, 2), (256, 16, 2)])
def test_shared_e4m3_weights_have_the_bits_of_f16(vsk, d, hq, hk):
    """Every other key has a weight half a step of bf16 above 0.5 (not quite: bf16 would take it to 0.5, f16 to 2^-12 of
    itself), and values that cancel: the output is what the weights' rounding leaves."""
    n = 1024
    c = shared_case(n, (0, 0), 4, hq, hk, d, "e4m3", seed=81)
    low = torch.zeros(n, dtype=torch.bool, device=DEV)
    low[c["sh"][1::2]] = True
    c["q"].zero_()
    c["q"][:, :, 0] = 1
    c["ke"].zero_()
    c["ve"].zero_()
    kb = torch.zeros(n, hk, d, device=DEV)
    kb[low, :, 0] = -1
    c["kb"] = kb.to(E4M3)
    c["vb"] = torch.where(low, -2.0, 1.0)[:, None, None].expand(n, hk, d).contiguous().to(E4M3)
    sm = -math.log(0.5 + 2.0 ** -9 - 2.0 ** -14)
    check_f16_weights(run_shared(vsk, c, sm_scale=sm), *shared_want(c, sm), c)


@pytest.mark.parametrize("case", [c for c in base.SHARED if c[6] == "e4m3"], ids=lambda c: f"s{c[0]}b{len(c[1])}d{c[5]}")
def test_shared_e4m3_within_the_bound_of_f16_weights(vsk, case):
    c = shared_case(*case, seed=86)
    check_f16_weights(run_shared(vsk, c, k_scale=0.5, v_scale=0.25), *shared_want(c, case[5] ** -0.5, 0.5, 0.25), c, 0.25)


@pytest.mark.parametrize("d", [128, 256])
def test_shared_e4m3_scores_far_apart(vsk, d):
    """Weights from 1 down to 2^-30 of the largest, which comes late in the row: the reference moves, f16 keeps its range."""
    c = shared_case(2000, (40, 0), 4, 8, 2, d, "e4m3", seed=87)
    c["q"].zero_()
    c["q"][:, :, 0] = 1
    kb = c["kb"].float()
    kb[:, :, 0] = 0
    order = torch.cat([c["sh"], c["kvi"]])
    kb[order, :, 0] = torch.linspace(-15, 15, 2040, device=DEV)[:, None]
    c["kb"] = kb.to(E4M3)
    sm = math.log(2.0)
    check_f16_weights(run_shared(vsk, c, sm_scale=sm), *shared_want(c, sm), c)


# ---------------------------------------------------------------- bad shared indices

@pytest.mark.parametrize("pool,d", [("bf16", 128), ("e4m3", 128), ("bf16", 256), ("e4m3", 256)])
@pytest.mark.parametrize("bad", [-1, -2, -3, -(1 << 31), -(1 << 63), (1 << 63) - 1, (1 << 32)])
def test_every_bad_shared_index_is_flagged(vsk, pool, d, bad):
    c = shared_case(300, (30, 8), 4, 8, 2, d, pool, seed=82)
    run_shared(vsk, c)
    assert vsk.read_error_flags() == 0  # (300 indices end inside a tile)
    good = dict(c)
    keep = torch.ones(300, dtype=torch.bool, device=DEV)
    keep[[5, 299]] = False
    good["sh"] = c["sh"][keep]
    c["sh"][5] = c["sh"][299] = bad
    check_attention(run_shared(vsk, c), *shared_want(good, d ** -0.5))
    assert vsk.read_error_flags() == 1
    if abs(bad) < 1 << 31 or bad == -(1 << 31):
        c["sh"], c["kvi"] = c["sh"].int(), c["kvi"].int()
        check_attention(run_shared(vsk, c), *shared_want(good, d ** -0.5))
        assert vsk.read_error_flags() == 1


# ---------------------------------------------------------------- windows of one buffer

def test_windows_of_one_buffer_that_do_not_meet_are_taken(vsk):
    """mass beside mass_in, and out_mass beside mass, as column windows of the same rows."""
    c = shared_case(0, (300, 80), 4, 8, 2, 128, seed=88)
    t = 380
    big = torch.rand(2, 2 * t + 100, generator=gen(2), device=DEV)
    before = big.clone()
    run_mass(vsk, c, big[:, t:2 * t], mass_in=big[:, :t])
    base.check_mass(big[:, t:2 * t], base.mass_want(c, 128 ** -0.5), before[:, :t].to(F64))
    assert torch.equal(big[:, :t], before[:, :t]) and torch.equal(big[:, 2 * t:], before[:, 2 * t:])
    mass = big[:, :t].clone()
    out = [torch.zeros(3, dtype=torch.int32, device=DEV), torch.zeros(100, dtype=torch.long, device=DEV),
           big[:, 2 * t:], torch.zeros(t, dtype=torch.long, device=DEV)]
    vsk.kv_evict(big[:, :t], c["kvp"], c["kvi"], 50, 5, *out)
    want = base.evict_want(mass, c["kvi"], (300, 80), 50, 5)
    assert torch.equal(out[1].cpu(), want[1]) and torch.equal(out[2].cpu(), want[2]) and torch.equal(out[3][:280].cpu(), want[3])


# ---------------------------------------------------------------- tuning

def test_workspaces_follow_the_tuned_grid(vsk):
    """More CTAs than the workspace of an earlier call was sized for: the size is asked again."""
    c = shared_case(300, (300, 80), 4, 8, 2, 128, seed=83)
    o = torch.empty_like(c["q"])

    def verify():
        vsk.verify_splitkv_fwd(c["q"], c["ke"], c["ve"], o, c["kb"], c["vb"], c["qo"], c["kvp"], c["kvi"], None, True, None,
                               4, 1.0, 1.0)
        return o

    own = dict(c, sh=c["sh"][:0])
    stream = torch.cuda.Stream()  # a workspace of its own, not grown by other tests
    with torch.cuda.stream(stream):
        stream.wait_stream(torch.cuda.default_stream())
        run_shared(vsk, c)
        verify()
        vsk.set_tuning(num_ctas=40 * torch.cuda.get_device_properties(0).multi_processor_count)
        try:
            check_attention(verify(), *shared_want(own, 128 ** -0.5))
            check_attention(run_shared(vsk, c), *shared_want(c, 128 ** -0.5))
        finally:
            vsk.set_tuning()
        check_attention(run_shared(vsk, c), *shared_want(c, 128 ** -0.5))
        assert vsk.read_error_flags() == 0


# ---------------------------------------------------------------- prompts at once

def test_prompts_that_draw_their_work_on_two_streams_and_from_two_graphs(vsk):
    """Several items a CTA, so that the counters in the workspace are drawn from, in calls that overlap: on two streams
    and replayed from two graphs, each with its workspace."""
    d, hq, hk, lens = 64, 16, 8, [((700,) * 12, 300, 64), ((33, 900, 5) * 9, 500, 1)]
    cases = []
    for i, (a, b, c) in enumerate(lens):
        n = [*a, b, c]
        assert sum(-(-x // 128) for x in n) * hk > 2 * torch.cuda.get_device_properties(0).multi_processor_count
        q, k, v, p = base.prompt_case(n, hq, hk, d, seed=71 + i)
        want = torch.full_like(q, float("nan"))
        vsk.prompt_attn_fwd(q, k, v, want, p)
        check_attention(want, *base.prompt_want(q, k, v, n, d ** -0.5))
        cases.append((q, k, v, p, want))
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (q, k, v, p, _w) in zip(streams, cases):
            with torch.cuda.stream(s):
                outs.append(torch.full_like(q, float("nan")))
                vsk.prompt_attn_fwd(q, k, v, outs[-1], p)
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, cases[i % 2][4]), i
    graphs, graph_outs, spaces = [], [], [torch.zeros(256, dtype=torch.uint8, device=DEV) for _ in cases]
    for (q, k, v, p, _w), ws in zip(cases, spaces):
        o = torch.full_like(q, float("nan"))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            vsk.prompt_attn_fwd(q, k, v, o, p, workspace=ws)
        graphs.append(g)
        graph_outs.append(o)
    for _ in range(10):
        for o in graph_outs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, c[4]) for o, c in zip(graph_outs, cases))
    assert all(int(ws.sum()) == 0 for ws in spaces)  # no error, the counters back at zero


# ---------------------------------------------------------------- every key counts
#
# With queries of zero all n visible keys weigh the same.  Key t has the value 1
# in one place of (KV head, column), t mod (h_kv D), and 0 elsewhere, so every
# output is count / n with its own count of keys: exact sums (P is a power of
# two), then 1 / n and the product in 32 bits, joined pieces a few more (2^-18
# of itself is ample), and the rounding to bf16.  Where at most 64 keys share a
# place a key left out or taken twice moves the output by 1.5 % or more, further
# than bf16 steps are apart (2^-7).


def markers(t, hk, d, dtype):
    v = torch.zeros(len(t), hk * d, device=DEV)
    v[torch.arange(len(t), device=DEV), t % (hk * d)] = 1
    return v.view(len(t), hk, d).to(dtype)


def check_counts(got, count, n):
    """got [rows, h, d] bf16 against count / n, [rows, h, d] and [rows]."""
    x = count.to(F64) / n.to(F64)[:, None, None]
    lo, hi = (x * (1 - 2.0 ** -18)).to(BF16), (x * (1 + 2.0 ** -18)).to(BF16)
    bad = ~((got >= lo) & (got <= hi))
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:3].tolist())


def counts_upto(rows, hk, d, start=0):
    """[rows, hk * d]: how many of keys start .. start + i are in each place, for i < rows."""
    c = torch.zeros(rows, hk * d, dtype=torch.int32, device=DEV)
    c[torch.arange(rows, device=DEV), (start + torch.arange(rows, device=DEV)) % (hk * d)] = 1
    return c.cumsum(0)


@pytest.mark.parametrize("lens,hq,hk,d", [((4097,), 4, 1, 128), ((127, 128, 129, 255, 256, 257, 1, 2), 2, 2, 64), ((2500, 1), 6, 2, 256),
                                          ((3000, 700), 4, 4, 64), ((1025,), 16, 1, 256), ((1300,), 5, 5, 128)])
def test_prompt_counts_every_key(vsk, lens, hq, hk, d):
    n = sum(lens)
    q, k = torch.zeros(n, hq, d, dtype=BF16, device=DEV), normal(gen(3), n, hk, d)
    t = torch.cat([torch.arange(x, device=DEV) for x in lens])
    assert max(lens) <= 64 * hk * d
    o = torch.full_like(q, float("nan"))
    vsk.prompt_attn_fwd(q, k, markers(t, hk, d, BF16), o, indptr(lens))
    count = torch.cat([counts_upto(x, hk, d) for x in lens]).view(n, hk, 1, d).expand(n, hk, hq // hk, d).reshape(n, hq, d)
    check_counts(o, count, t + 1)
    assert vsk.read_error_flags() == 0


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("s,own,l,hq,hk,d", [
    (40000, (0, 7, 0), 4, 16, 4, 256), (40000, (900, 0, 33), 4, 32, 8, 128), (20000, (5,) * 9, 3, 8, 8, 64), (0, (5000, 1, 128), 4, 16, 2, 256),
    (129, (300, 64, 65, 0), 2, 8, 2, 128), (8191, (0,) * 70, 4, 8, 2, 128), (6000, (0, 1) * 20, 4, 16, 1, 256), (255, (0,), 1, 1, 1, 64),
])
def test_shared_counts_every_key(vsk, s, own, l, hq, hk, d, pool):
    c = shared_case(s, own, l, hq, hk, d, pool, seed=89)
    assert s + max(own) + l <= 64 * hk * d
    c["q"].zero_()
    # a key's place goes by its position behind the shared prefix: keys, then drafts
    place = torch.empty(len(c["kb"]), dtype=torch.long, device=DEV)
    place[c["sh"]] = torch.arange(s, device=DEV)
    at = 0
    for n in own:
        place[c["kvi"][at:at + n]] = s + torch.arange(n, device=DEV)
        at += n
    c["vb"] = markers(place, hk, d, c["vb"].dtype)
    t = torch.cat([s + n + torch.arange(l, device=DEV) for n in own])
    c["ve"] = markers(t, hk, d, BF16)
    count = []
    for n in own:
        total = torch.bincount(torch.arange(s + n, device=DEV) % (hk * d), minlength=hk * d)
        count.append(total + counts_upto(l, hk, d, s + n))
    count = torch.cat(count).view(-1, hk, 1, d).expand(-1, hk, hq // hk, d).reshape(-1, hq, d)
    check_counts(run_shared(vsk, c), count, t + 1)
    assert vsk.read_error_flags() == 0


# ---------------------------------------------------------------- calls the documentation allows

@pytest.mark.parametrize("hq,hk,d", [(6, 2, 64), (8, 2, 128), (16, 2, 256), (5, 5, 128)])
def test_prompt_written_over_its_queries(vsk, hq, hk, d):
    lens = (300, 1, 129, 500, 64)
    q, k, v, p = base.prompt_case(lens, hq, hk, d, seed=101, extra=4)
    want, a = base.prompt_want(q[:994], k[:994], v[:994], lens, d ** -0.5)
    tail = q[994:].clone()
    vsk.prompt_attn_fwd(q, k, v, q, p)
    check_attention(q[:994], want, a)
    assert torch.equal(q[994:], tail)


def test_prompt_sequences_with_rows_between_them(vsk):
    q, k, v, _ = base.prompt_case((400,), 4, 2, 128, seed=102)
    k[:7], v[:7] = float("nan"), float("nan")  # rows before the first sequence
    o = torch.full_like(q, 7.0)
    vsk.prompt_attn_fwd(q, k, v, o, torch.tensor([7, 7, 150, 399], dtype=torch.int32, device=DEV))
    want, a = base.prompt_want(q[7:399], k[7:399], v[7:399], (143, 249), 128 ** -0.5)
    check_attention(o[7:399], want, a)
    assert bool((o[:7] == 7.0).all()) and bool((o[399:] == 7.0).all())
    assert vsk.read_error_flags() == 0


@pytest.mark.parametrize("pool,d,hq,hk", [("bf16", 64, 6, 3), ("bf16", 128, 8, 2), ("e4m3", 128, 8, 2), ("bf16", 256, 16, 2), ("e4m3", 256, 16, 2)])
@pytest.mark.parametrize("shift", [0, 2])
def test_strided_drafts_and_pools(vsk, pool, d, hq, hk, shift):
    """Drafts as windows of one projection (4-byte aligned where shift is 2), pools as windows of wider rows."""
    c = shared_case(300, (40, 0, 99), 4, hq, hk, d, pool, seed=103)
    n = len(c["q"])
    wide = normal(gen(5), n * (hq + 2 * hk) * d + shift)[shift:].view(n, hq + 2 * hk, d)
    c["q"], c["ke"], c["ve"] = wide[:, :hq], wide[:, hq:hq + hk], wide[:, hq + hk:]
    both = torch.cat([c["kb"].float(), c["vb"].float()], 1).to(c["kb"].dtype)
    c["kb"], c["vb"] = both[:, :hk], both[:, hk:]
    space = torch.full((n * (hq + 1) * d + shift,), 7.0, dtype=BF16, device=DEV)
    o = space[shift:].view(n, hq + 1, d)[:, 1:]
    vsk.verify_splitkv_shared_fwd(c["q"], c["ke"], c["ve"], o, c["kb"], c["vb"], c["qo"], c["kvp"], c["kvi"], c["sh"], 4)
    check_attention(o, *shared_want(c, d ** -0.5))
    assert bool((space[shift:].view(n, hq + 1, d)[:, 0] == 7.0).all())
    base.check_mass(run_mass(vsk, c, torch.empty(hk, 139, device=DEV)), base.mass_want(c, d ** -0.5))
    assert vsk.read_error_flags() == 0


def test_padded_indices_are_not_looked_at(vsk):
    """kv_indices longer than the sequences, as a captured program keeps it: what lies behind is no index."""
    c = shared_case(200, (70, 0, 33), 4, 8, 2, 128, seed=104)
    padded = dict(c, kvi=torch.cat([c["kvi"], c["kvi"].new_full((400,), -9)]))
    check_attention(run_shared(vsk, padded), *shared_want(c, 128 ** -0.5))
    m = torch.full((2, 503), 7.0, device=DEV)
    run_mass(vsk, padded, m)
    base.check_mass(m[:, :103], base.mass_want(c, 128 ** -0.5))
    assert bool((m[:, 103:] == 7.0).all())
    out = [torch.full((4,), -7, dtype=torch.int32, device=DEV), torch.full((60,), -7, device=DEV), torch.full((2, 60), -7.0, device=DEV),
           torch.full((503,), -7, device=DEV)]
    vsk.kv_evict(m, c["kvp"], padded["kvi"], 20, 5, *out)
    want = base.evict_want(m[:, :103], c["kvi"], (70, 0, 33), 20, 5)
    base.check_evict([x.cpu() for x in out], want)
    assert vsk.read_error_flags() == 0


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("d,hq,hk", [(64, 4, 2), (128, 8, 2), (256, 16, 2)])
def test_queries_that_are_no_numbers_stay_with_their_sequence(vsk, pool, d, hq, hk):
    c = shared_case(500, (60, 20, 0, 9), 4, hq, hk, d, pool, seed=105)
    want, a = shared_want(c, d ** -0.5)
    w = base.mass_want(c, d ** -0.5)
    c["q"] = c["q"].clone()
    c["q"][4:6], c["q"][9, :, 3] = float("nan"), float("inf")
    rows = torch.ones(16, dtype=torch.bool, device=DEV)
    rows[[4, 5, 9]] = False
    o = run_shared(vsk, c)
    check_attention(o[rows], want[rows], a[rows])
    assert bool(o[4:6].isnan().all())
    m = run_mass(vsk, c, torch.empty(hk, 89, device=DEV))
    base.check_mass(m[:, :60], w[:, :60])
    base.check_mass(m[:, 80:], w[:, 80:])
    assert bool(m[:, 60:80].isnan().all())


def test_prompt_queries_that_are_no_numbers_stay_with_their_row(vsk):
    for d, hq, hk in ((64, 4, 2), (128, 8, 2), (256, 16, 2)):
        lens = (200, 90)
        q, k, v, p = base.prompt_case(lens, hq, hk, d, seed=106)
        want, a = base.prompt_want(q, k, v, lens, d ** -0.5)
        q[37], q[250] = float("nan"), float("inf")
        o = torch.empty_like(q)
        vsk.prompt_attn_fwd(q, k, v, o, p)
        rows = torch.ones(290, dtype=torch.bool, device=DEV)
        rows[[37, 250]] = False
        check_attention(o[rows], want[rows], a[rows])
        assert bool(o[37].isnan().all())


def test_evict_of_nothing_and_of_what_stays(vsk):
    none = torch.zeros(0, dtype=torch.long, device=DEV)
    ptr = torch.full((4,), -7, dtype=torch.int32, device=DEV)
    vsk.kv_evict(torch.zeros(2, 0, device=DEV), indptr((0, 0, 0)), none, 5, 1, ptr, none.clone(), torch.zeros(2, 0, device=DEV), none.clone())
    assert ptr.tolist() == [0, 0, 0, 0] and vsk.read_error_flags() == 0
    m, kvi = torch.rand(2, 30, device=DEV), torch.arange(30, device=DEV)
    out = [ptr, torch.zeros(30, dtype=torch.long, device=DEV), torch.zeros(2, 30, device=DEV), none.clone()]  # nothing is freed
    vsk.kv_evict(m, indptr((10, 0, 20)), kvi, 1 << 40, 1 << 33, *out)
    assert ptr.tolist() == [0, 10, 10, 30] and torch.equal(out[1], kvi) and torch.equal(out[2], m)
    assert vsk.read_error_flags() == 0


def test_lengths_that_change_under_a_captured_graph(vsk):
    """One graph of the shared call, the weights and the eviction; replayed with other indptrs over the same arrays."""
    t, b, d = 400, 3, 128
    c = shared_case(250, (t, 0, 0), 4, 8, 2, d, seed=107)
    o, m = torch.zeros_like(c["q"]), torch.zeros(2, t, device=DEV)
    out = [torch.zeros(b + 1, dtype=torch.int32, device=DEV), torch.zeros(t, dtype=torch.long, device=DEV), torch.zeros(2, t, device=DEV),
           torch.zeros(t, dtype=torch.long, device=DEV)]
    ws = torch.zeros(vsk.shared_workspace_size(b, 8, 2, d, 4), dtype=torch.uint8, device=DEV)
    run_shared(vsk, c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vsk.verify_splitkv_shared_fwd(c["q"], c["ke"], c["ve"], o, c["kb"], c["vb"], c["qo"], c["kvp"], c["kvi"], c["sh"], 4, workspace=ws)
        run_mass(vsk, c, m, workspace=ws)
        vsk.kv_evict(m, c["kvp"], c["kvi"], 64, 16, *out, workspace=ws)
    for lens in ((0, 0, 0), (1, 399, 0), (133, 134, 133), (0, 17, 300), (400, 0, 0)):
        c["kvp"].copy_(indptr(lens))
        graph.replay()
        torch.cuda.synchronize()
        n = sum(lens)
        now = dict(c, own=lens, kvi=c["kvi"][:n])
        check_attention(o, *shared_want(now, d ** -0.5))
        base.check_mass(m[:, :n], base.mass_want(now, d ** -0.5))
        want = base.evict_want(m[:, :n], c["kvi"][:n], lens, 64, 16)
        assert torch.equal(out[0].cpu(), want[0]) and torch.equal(out[1][:len(want[1])].cpu(), want[1])
        assert torch.equal(out[3][:len(want[3])].cpu(), want[3])
    assert vsk.read_error_flags(ws) == 0


FORMS = [
    # (name, tuning of the verify call, head_dims)
    ("default", {}, (64, 128, 256)), ("one launch", {"tc": 0, "colsplit": 0, "split_launch": 0}, (64, 128, 256)),
    ("stream and combine", {"tc": 0, "colsplit": 0, "split_launch": 2}, (64, 128, 256)), ("column split", {"tc": 0, "colsplit": 2}, (256,)),
    ("cluster", {"tc": 0, "cluster": 2}, (64, 128, 256)), ("keys on M", {"tc": 1}, (256,)), ("rows on M", {"tc": 2}, (256,)),
]


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("form,d", [(f, d) for f in FORMS for d in f[2]], ids=lambda x: x[0] if isinstance(x, tuple) else str(x))
def test_verify_queries_that_are_no_numbers_stay_with_their_row(vsk, form, d, pool):
    """Rows of one tile share a scale over e4m3 pools: it goes by their finite values."""
    name, tuning, _ = form
    hq, hk = (16, 2) if d == 256 else (8, 2)
    c = shared_case(0, (60, 200, 9, 0), 4, hq, hk, d, pool, seed=108)
    want, a = shared_want(c, d ** -0.5)
    c["q"] = c["q"].clone()
    c["q"][1], c["q"][4:6], c["q"][9, :, 3] = float("inf"), float("nan"), float("-inf")
    rows = torch.ones(16, dtype=torch.bool, device=DEV)
    rows[[1, 4, 5, 9]] = False
    o = torch.full_like(c["q"], 7.0)
    try:
        for k, v in tuning.items():
            getattr(vsk, "set_tuning_" + k)(v)
        assert vsk.verify_splitkv_fwd(c["q"], c["ke"], c["ve"], o, c["kb"], c["vb"], c["qo"], c["kvp"], c["kvi"], None, True, None, 4, 1.0, 1.0)
    finally:
        vsk.set_tuning_tc()
        vsk.set_tuning_colsplit()
        vsk.set_tuning_split_launch()
        vsk.set_tuning_cluster()
    check_attention(o[rows], want[rows], a[rows])
    assert bool(o[~rows].isnan().all())
    assert vsk.read_error_flags() == 0


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("d,hq,hk", [(64, 4, 2), (128, 8, 2), (256, 16, 2)])
def test_mass_of_a_row_that_sees_only_minus_infinity(vsk, pool, d, hq, hk):
    """Such a row gives no weight, like one that sees nothing, and leaves the other rows' weights alone."""
    c = shared_case(0, (500, 30), 4, hq, hk, d, pool, seed=109)
    kb = c["kb"].float()
    kb[:, :, 5] = kb[:, :, 5].abs() + 0.5
    c["kb"], c["ke"] = kb.to(c["kb"].dtype), c["ke"].clone()
    c["ke"][:, :, 5] = c["ke"][:, :, 5].abs() + 0.5
    q = c["q"].clone()
    q[2, 0, 5] = q[5, :, 5] = -math.inf
    blind = torch.zeros(8, hq, dtype=torch.bool, device=DEV)
    blind[2, 0] = blind[5] = True
    g, w, at = hq // hk, torch.zeros(hk, 530, dtype=F64, device=DEV), 0
    for b, n in enumerate(c["own"]):
        r = slice(4 * b, 4 * b + 4)
        k = torch.cat([base.rows64(c["kb"], c["kvi"][at:at + n]), c["ke"][r].to(F64)])
        vis = torch.ones(4, n + 4, dtype=torch.bool, device=DEV).tril(n)
        for h in range(hq):
            x = (c["q"][r, h].to(F64) @ k[:, h // g].T) * d ** -0.5
            p = torch.softmax(x.masked_fill(~vis, -math.inf), 1)
            w[h // g, at:at + n] += p[~blind[r, h], :n].sum(0)
        at += n
    c["q"] = q
    base.check_mass(run_mass(vsk, c, torch.empty(hk, 530, device=DEV)), w)
    assert vsk.read_error_flags() == 0


# ---------------------------------------------------------------- repeats

@pytest.mark.parametrize("d,hq,hk", [(64, 8, 2), (128, 32, 8), (256, 16, 2)])
def test_calls_repeat_bit_for_bit(vsk, d, hq, hk):
    """Which CTA takes which item, and when, plays no part in the result."""
    lens = (1500, 70, 700, 1, 333) * 3
    q, k, v, p = base.prompt_case(lens, hq, hk, d, seed=110)
    shared = [shared_case(5000, (300, 0, 45, 800) * 3, 4, hq, hk, d, pool, seed=111) for pool in ("bf16", "e4m3")]
    first = None
    for _ in range(10):
        o = torch.full_like(q, float("nan"))
        vsk.prompt_attn_fwd(q, k, v, o, p)
        got = [o] + [run_shared(vsk, c) for c in shared] + [run_mass(vsk, c, torch.empty(hk, len(c["kvi"]), device=DEV)) for c in shared]
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


# ---------------------------------------------------------------- keys and values that are no numbers
#
# One element of one KV head's key (or value) is NaN or infinite: every row that
# sees it has no finite output where the 64-bit form has none, and no other row,
# head or column changes.


def poison(c, which, bad, row):
    t = c[which].float().clone()
    t[row, 1, 3] = bad
    c[which] = t.to(c[which].dtype)


def check_poisoned(c, o, want, a, which, rows, d):
    exact, _ = shared_want(c, d ** -0.5)
    hit = torch.zeros(o.shape, dtype=torch.bool, device=DEV)
    g = o.shape[1] // c["ke"].shape[1]
    if which[0] == "k":
        hit[rows, g:] = True
    else:
        hit[rows, g:, 3] = True
    check_attention(o[~hit], want[~hit], a[~hit])
    assert not bool((o[hit].isfinite() & ~exact[hit].isfinite()).any())


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_shared_keys_that_are_no_numbers(vsk, d, pool):
    """In the shared prefix, a sequence's own (over many pieces) and the drafts."""
    hq, hk = (16, 2) if d == 256 else (8, 2)
    c0 = shared_case(600, (60, 900, 9, 0), 4, hq, hk, d, pool, seed=112)
    want, a = shared_want(c0, d ** -0.5)
    places = [("b", int(c0["sh"][333]), slice(0, 16)), ("b", int(c0["kvi"][60 + 777]), slice(4, 8)), ("e", 5, slice(5, 8))]
    for kind, row, rows in places:
        for which in ("k" + kind, "v" + kind):
            for bad in (math.nan, math.inf):
                if bad == math.inf and pool == "e4m3" and kind == "b":
                    continue  # e4m3 has none
                c = dict(c0)
                poison(c, which, bad, row)
                check_poisoned(c, run_shared(vsk, c), want, a, which, rows, d)


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("form,d", [(f, d) for f in FORMS for d in f[2]], ids=lambda x: x[0] if isinstance(x, tuple) else str(x))
def test_verify_keys_that_are_no_numbers(vsk, form, d, pool):
    _, tuning, _ = form
    hq, hk = (16, 2) if d == 256 else (8, 2)
    c0 = shared_case(0, (60, 900, 9, 0), 4, hq, hk, d, pool, seed=113)
    want, a = shared_want(c0, d ** -0.5)
    try:
        for k, v in tuning.items():
            getattr(vsk, "set_tuning_" + k)(v)
        for which, bad in [("kb", math.nan), ("vb", math.nan), ("ke", math.nan), ("ke", math.inf)] + (
                [("kb", math.inf), ("vb", math.inf)] if pool == "bf16" else []):
            c = dict(c0)
            row, rows = (int(c0["kvi"][60 + 777]), slice(4, 8)) if which[1] == "b" else (5, slice(5, 8))
            poison(c, which, bad, row)
            o = torch.full_like(c["q"], 7.0)
            assert vsk.verify_splitkv_fwd(c["q"], c["ke"], c["ve"], o, c["kb"], c["vb"], c["qo"], c["kvp"], c["kvi"], None, True, None,
                                          4, 1.0, 1.0)
            check_poisoned(c, o, want, a, which, rows, d)
    finally:
        vsk.set_tuning_tc()
        vsk.set_tuning_colsplit()
        vsk.set_tuning_split_launch()
        vsk.set_tuning_cluster()


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("d,hq,hk", [(64, 4, 2), (128, 8, 2), (256, 16, 2)])
def test_the_same_pool_row_more_than_once(vsk, pool, d, hq, hk):
    """Twice in the shared prefix, there and in a sequence's own, in two sequences: every entry is a key."""
    c = shared_case(260, (70, 5, 90), 4, hq, hk, d, pool, seed=115)
    c["sh"][7] = c["sh"][8] = c["sh"][200]
    c["kvi"][3], c["kvi"][71], c["kvi"][80:85] = c["sh"][7], c["kvi"][3], c["kvi"][0]
    check_attention(run_shared(vsk, c), *shared_want(c, d ** -0.5))
    base.check_mass(run_mass(vsk, c, torch.empty(hk, 165, device=DEV)), base.mass_want(c, d ** -0.5))
    assert vsk.read_error_flags() == 0
