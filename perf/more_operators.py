"""The rotary, cache-append and block-scaled cache operators: their cases, inputs and plain forms.

Four operators between the projections and the verify call:

``rope``          rotary positions of queries and keys (``rope_fwd``);
``append``        the same, with the keys and values stored into a pool of
                  bf16 or e4m3 rows (``rope_append_fwd``);
``append_block``  the same into an e4m3 cache of blocks with a power-of-two
                  scale for each block and KV head (``rope_append_block_fwd``);
``block``         the verify call over that cache (``verify_splitkv_block_fwd``).

``run`` computes a case in elementary torch operations in 32 bits (angles in
64), or with ``own`` set through the package's entry points.  ``exact``
computes it again from the definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

TOP = 448.0  # the largest e4m3 value
SMALL = 2.0 ** -40  # the smallest scale of a block


def _c(name, op, **kw):
    return {"name": name, "op": op, **kw}


def listed():
    return [
        # one new token of one request: what a call costs before any arithmetic
        _c("rope_one_token", "rope", batch=1, lo=1, hi=1, past=1000, h_q=32, h_kv=8, d=128, rot=128, interleaved=False, factor=1.0),
        # a few documents, the wide head size, a quarter of the head rotated, neighbours paired
        _c("rope_documents_partial", "rope", batch=3, lo=511, hi=2049, past=0, h_q=16, h_kv=2, d=256, rot=64, interleaved=True, factor=1.0),
        # chunks of long prompts at far positions, frequencies scaled for a longer context
        _c("rope_long", "rope", batch=4, lo=4001, hi=8192, past=120000, h_q=32, h_kv=8, d=128, rot=128, interleaved=False, factor=16.0),
        # the drafts of a serving batch into a bf16 pool
        _c("append_drafts", "append", batch=64, lo=4, hi=4, past=32768, h_q=32, h_kv=8, d=128, rot=128, interleaved=False, factor=1.0, pool="bf16"),
        # documents into an e4m3 pool, the wide head size
        _c("append_documents_fp8", "append", batch=3, lo=511, hi=2049, past=0, h_q=16, h_kv=2, d=256, rot=256, interleaved=False, factor=1.0, pool="e4m3"),
        # long prompts into a bf16 pool
        _c("append_long", "append", batch=4, lo=4001, hi=8192, past=0, h_q=32, h_kv=8, d=128, rot=128, interleaved=False, factor=1.0, pool="bf16"),
        # the drafts of a serving batch, in blocks that hold earlier rows
        _c("append_block_drafts", "append_block", batch=64, lo=4, hi=4, past=8192, h_q=32, h_kv=8, d=128, rot=128, interleaved=False, factor=1.0, block=64),
        # long prompts, in chunks that begin and end inside blocks
        _c("append_block_long", "append_block", batch=4, lo=4001, hi=8192, past=2000, h_q=32, h_kv=8, d=128, rot=128, interleaved=False, factor=1.0, block=64),
        # two short sequences, small heads, short blocks
        _c("block_tiny", "block", batch=2, lo=64, hi=96, l_ext=4, h_q=4, h_kv=1, d=64, block=16),
        # single tokens of a mid-size batch
        _c("block_decode", "block", batch=32, lo=1024, hi=16384, l_ext=1, h_q=32, h_kv=8, d=128, block=32),
        # two mid-size sequences, the wide head size
        _c("block_d256", "block", batch=2, lo=4096, hi=8192, l_ext=4, h_q=16, h_kv=2, d=256, block=64),
        # the serving batch
        _c("block_serving", "block", batch=64, lo=8192, hi=32768, l_ext=4, h_q=32, h_kv=8, d=128, block=64),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: any operator, sizes over the logarithm of their range, odd ones among them."""
    big = {c["op"]: work(c) for c in listed()}  # the last one of each operator is its largest
    while True:
        op = rng.choice(["rope", "append", "append_block", "block"])
        d, h_kv, g = rng.choice([64, 128, 256]), rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8])
        c = {"op": op, "batch": _log(rng, 1, 64), "h_q": g * h_kv, "h_kv": h_kv, "d": d}
        if op == "block":
            hi = _log(rng, 16, 32768)
            c.update(lo=rng.randint(0, hi), hi=hi, l_ext=min(_log(rng, 1, 16), (64 if d == 256 else 128) // g),
                     block=rng.choice([16, 32, 48, 64, 128]))
        else:
            hi = _log(rng, 1, 8192)
            c.update(lo=rng.randint(1, hi), hi=hi, past=rng.choice([0, _log(rng, 1, 32768)]),
                     rot=rng.choice([d, d, d // 2, d // 4, 48]), interleaved=rng.choice([False, True]),
                     factor=rng.choice([1.0, 1.0, 4.0, 16.0]))
            if op == "append":
                c["pool"] = rng.choice(["bf16", "e4m3"])
            if op == "append_block":
                c["block"] = rng.choice([16, 32, 48, 64, 128])
        w, top = work(c), big[op]
        held = 0 if op == "block" else c["batch"] * (c["past"] + c["hi"]) * h_kv * d  # an appended cache's values
        if w["bytes"] <= top["bytes"] and w["flops"] <= top["flops"] and sum(_lens(c)) > 0 and held <= 64 * 16384 * 1024:
            return c


def _lens(c):
    """The sequences' lengths (rows, or keys in the cache): the case's own, whatever the seed of the inputs."""
    r = random.Random(1000003 * c["batch"] + 1009 * c["lo"] + c["hi"])
    return [r.randint(c["lo"], c["hi"]) for _ in range(c["batch"])]


def _past(c):
    """Rows before the new ones, by sequence."""
    r = random.Random(7919 * c["batch"] + c["past"])
    return [r.randint(c["past"] // 2, c["past"]) for _ in range(c["batch"])]


def _blocks(c):
    """Blocks of the cache, by sequence."""
    held = _lens(c) if c["op"] == "block" else [a + n for a, n in zip(_past(c), _lens(c))]
    return [-(-x // c["block"]) for x in held]


def _scales(c):
    return (0.5, 0.25) if c["pool"] == "e4m3" else (1.0, 1.0)


def work(c):
    n = _lens(c)
    t, b, hq, hk, d = sum(n), c["batch"], c["h_q"], c["h_kv"], c["d"]
    if c["op"] == "block":
        l_ext, rows = c["l_ext"], b * c["l_ext"]
        return {"bytes": 2 * t * hk * d + sum(_blocks(c)) * (8 * hk + 4) + 4 * rows * d * (hq + hk) + 4 * (2 * b + 1),
                "flops": 4 * d * hq * (l_ext * t + b * l_ext * (l_ext + 1) // 2)}
    moved = 4 * t * (hq + hk) * d + 8 * t + 2 * c["rot"]  # queries and keys in and out, positions, frequencies
    flops = 3 * t * (hq + hk) * c["rot"]
    if c["op"] == "append":
        e = 1 if c["pool"] == "e4m3" else 2
        moved += 2 * t * hk * d + 2 * t * hk * d * e + 8 * t
    elif c["op"] == "append_block":
        new = sum(-(-(p + x) // c["block"]) - p // c["block"] for p, x in zip(_past(c), n))
        moved += 4 * t * hk * d + new * (8 * hk + 4) + 4 * (2 * b + 1)
        flops += 2 * t * hk * d
    return {"bytes": moved, "flops": flops}


def _indptr(n, dev):
    return torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32, device=dev)


def _frequencies(c):
    """Base 10000; for a longer context those that turn less than 32 times over 4,096 positions are slowed, all
    of those that turn less than once by the factor; and the size that the rotated values get with it."""
    i = np.arange(c["rot"] // 2, dtype=np.float64)
    f = 10000.0 ** (-2.0 * i / c["rot"])
    lo, hi = (c["rot"] * math.log(4096.0 / (r * 2.0 * math.pi)) / (2.0 * math.log(10000.0)) for r in (32.0, 1.0))
    slow = np.clip((i - math.floor(lo)) / max(math.ceil(hi) - math.floor(lo), 1e-3), 0.0, 1.0)
    return (f * (1.0 - slow) + f / c["factor"] * slow).astype(np.float32), 1.0 + 0.1 * math.log(c["factor"])


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    n = _lens(case)
    t, b, hq, hk, d = sum(n), case["batch"], case["h_q"], case["h_kv"], case["d"]
    s = {"case": case, "lens": n}

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.bfloat16)

    def codes(*shape):  # rows as they lie in an e4m3 cache
        return (normal(*shape) * 100).clamp_(-TOP, TOP).to(torch.float8_e4m3fn)

    def amounts(blocks):  # scales of blocks whose values differ by a few powers of two
        return torch.exp2(torch.randint(-9, -5, (blocks, hk), generator=g, device=dev).float())

    if case["op"] in ("block", "append_block"):
        held = _blocks(case)
        total = sum(held) + 3  # some blocks are nobody's
        order = torch.randperm(total, generator=g, device=dev)[:sum(held)].to(torch.int32)
        table = torch.zeros(b, max(1, max(held)), dtype=torch.int32, device=dev)
        real = torch.arange(table.shape[1], device=dev)[None, :] < torch.tensor(held, device=dev)[:, None]
        table[real] = order
        s.update(k_cache=codes(total * case["block"], hk, d), v_cache=codes(total * case["block"], hk, d),
                 k_scales=amounts(total), v_scales=amounts(total), block_table=table)
    if case["op"] == "block":
        rows = b * case["l_ext"]
        s.update(q=normal(rows, hq, d), k_ext=normal(rows, hk, d), v_ext=normal(rows, hk, d),
                 o=torch.zeros(rows, hq, d, dtype=torch.bfloat16, device=dev), sm_scale=1.0 / math.sqrt(d),
                 qo_indptr=_indptr([case["l_ext"]] * b, dev), seq_lens=torch.tensor(n, dtype=torch.int32, device=dev))
        return s
    qkv = normal(t, hq + 2 * hk, d)  # one projection's output: the three are views of it
    past = _past(case)
    pos = np.concatenate([np.arange(p, p + x) for p, x in zip(past, n)])
    freq, size = _frequencies(case)
    s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hk], v=qkv[:, hq + hk:], positions=torch.from_numpy(pos).to(dev),
             inv_freq=torch.from_numpy(freq).to(dev), size=size, q_out=torch.zeros(t, hq, d, dtype=torch.bfloat16, device=dev),
             k_out=torch.zeros(t, hk, d, dtype=torch.bfloat16, device=dev))
    if case["op"] == "append":
        cache = torch.float8_e4m3fn if case["pool"] == "e4m3" else torch.bfloat16
        rows = t + 64 + t // 4
        s.update(k_buffer=torch.zeros(rows, hk, d, dtype=cache, device=dev), v_buffer=torch.zeros(rows, hk, d, dtype=cache, device=dev),
                 loc=torch.randperm(rows, generator=g, device=dev)[:t].clone())
        s["k_scale"], s["v_scale"] = _scales(case)
    if case["op"] == "append_block":
        s.update(qo_indptr=_indptr(n, dev), cache_lens=torch.tensor(past, dtype=torch.int32, device=dev))
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        return _run_own(op, s)
    return {"rope": _rope, "append": _append, "append_block": _append_block, "block": _block}[op](s)


def _run_own(op, s):
    import speculative_decode_verify_prefix_gb300 as vsk

    if op == "block":
        vsk.verify_splitkv_block_fwd(s["q"], s["k_ext"], s["v_ext"], s["o"], s["k_cache"], s["v_cache"], s["k_scales"],
                                     s["v_scales"], s["qo_indptr"], s["block_table"], s["seq_lens"], s["case"]["block"],
                                     s["case"]["l_ext"], sm_scale=s["sm_scale"])
        return s["o"]
    how = {"interleaved": s["case"]["interleaved"], "attention_factor": s["size"]}
    if op == "rope":
        vsk.rope_fwd(s["q"], s["k"], s["q_out"], s["k_out"], s["positions"], s["inv_freq"], **how)
        return [s["q_out"], s["k_out"]]
    if op == "append":
        vsk.rope_append_fwd(s["q"], s["k"], s["v"], s["q_out"], s["k_out"], s["k_buffer"], s["v_buffer"], s["loc"],
                            s["positions"], s["inv_freq"], k_scale=s["k_scale"], v_scale=s["v_scale"], **how)
        return [s["q_out"], s["k_out"], s["k_buffer"], s["v_buffer"]]
    vsk.rope_append_block_fwd(s["q"], s["k"], s["v"], s["q_out"], s["k_out"], s["k_cache"], s["v_cache"], s["k_scales"],
                              s["v_scales"], s["qo_indptr"], s["block_table"], s["cache_lens"], s["case"]["block"],
                              s["positions"], s["inv_freq"], **how)
    return [s["q_out"], s["k_out"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"]]


# ---- plain forms, 32 bits (angles 64) ----


def _turned(s, x, cos, sin):
    """Rows x [n, h, d] rotated, in 32 bits."""
    c = s["case"]
    y, r = x.float(), c["rot"]
    if c["interleaved"]:
        a, b = y[..., :r:2], y[..., 1:r:2]
        z = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :r // 2], y[..., r // 2:r]
        z = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([z, y[..., r:]], -1)


def _both(s):
    t = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = (f(t).float()[:, None] * s["size"] for f in (torch.cos, torch.sin))
    return _turned(s, s["q"], cos, sin), _turned(s, s["k"], cos, sin)


def _rope(s):
    q, k = _both(s)
    return [q.to(torch.bfloat16), k.to(torch.bfloat16)]


def _put(pool, at, x):
    """Rows `at` of a pool; e4m3 rows are stored as bytes."""
    if pool.dtype == torch.float8_e4m3fn:
        pool.view(torch.uint8)[at] = x.clamp(-TOP, TOP).to(pool.dtype).view(torch.uint8)
    else:
        pool[at] = x.to(pool.dtype)


def _append(s):
    q, k = _both(s)
    _put(s["k_buffer"], s["loc"], k / s["k_scale"])
    _put(s["v_buffer"], s["loc"], s["v"].float() / s["v_scale"])
    return [q.to(torch.bfloat16), k.to(torch.bfloat16), s["k_buffer"], s["v_buffer"]]


def _gather(pool, at):
    """Pool rows as 32-bit values; e4m3 rows are gathered as bytes."""
    return pool.view(torch.uint8)[at].view(pool.dtype).float()


def _append_block(s):
    """The blocks touched as one batch of whole blocks: their earlier rows, then the new ones."""
    c = s["case"]
    size, hk, d = c["block"], c["h_kv"], c["d"]
    q, k = _both(s)
    ptr, past = s["qo_indptr"].long(), s["cache_lens"].long()
    t = k.shape[0]
    row = torch.arange(t, device=k.device)
    seq = torch.searchsorted(ptr[1:], row, right=True)
    at = past[seq] + row - ptr[seq]  # position in the cache
    page = s["block_table"][seq, at // size].long()
    touched, which = torch.unique(page, return_inverse=True)
    # earlier rows of the touched blocks: those before the sequence's first new one
    first = torch.zeros_like(touched)
    first[which] = torch.where(at // size == past[seq] // size, past[seq] % size, torch.zeros_like(at))
    old = torch.arange(size, device=k.device)[None, :] < first[:, None]
    inside = which * size + at % size
    rows = (touched[:, None] * size + torch.arange(size, device=k.device)).flatten()
    for x, cache, scales in ((k, s["k_cache"], s["k_scales"]), (s["v"].float(), s["v_cache"], s["v_scales"])):
        top = torch.zeros(len(touched), hk, device=k.device)
        top.index_reduce_(0, which, x.abs().amax(-1), "amax")
        need = top / TOP
        e = torch.frexp(need)
        need = torch.ldexp(torch.ones_like(need), e.exponent - (e.mantissa == 0.5).int())  # the power of two at or above it
        need = torch.where(top > 0, need, torch.zeros_like(need)).clamp_min(SMALL)
        before = scales[touched]
        now = torch.where((first > 0)[:, None], torch.maximum(before, need), need)
        was = _gather(cache, rows).view(-1, size, hk, d)
        again = (was * (before / now)[:, None, :, None])
        y = torch.where((old[:, :, None] & (now != before)[:, None, :])[..., None], again, was).view(-1, hk, d)
        y[inside] = x / now[which][:, :, None]
        _put(cache, rows, y)
        scales[touched] = now
    return [q.to(torch.bfloat16), k.to(torch.bfloat16), s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"]]


def _softmax(x):
    """Over the last dimension; a row with nothing visible (all -inf) is 0."""
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total == 0, torch.ones_like(total), total)


def _block(s):
    c = s["case"]
    b, l_ext, hk, hq, d, size = c["batch"], c["l_ext"], c["h_kv"], c["h_q"], c["d"], c["block"]
    q = s["q"].float().view(b, l_ext, hk, hq // hk, d).permute(0, 2, 1, 3, 4).reshape(b, hk, -1, d)
    ke, ve = (s[w].float().view(b, l_ext, hk, d).transpose(1, 2) for w in ("k_ext", "v_ext"))
    j = torch.arange(max(max(s["lens"]), 1), device=q.device)
    real = j[None, :] < s["seq_lens"].long()[:, None]
    page = s["block_table"].long()[:, j // size] * real
    at = page * size + j % size
    k = (_gather(s["k_cache"], at) * s["k_scales"][page][..., None]).permute(0, 2, 3, 1)
    x = torch.matmul(q, k).mul_(s["sm_scale"]).masked_fill_(~real[:, None, None, :], -math.inf)
    del k
    y = torch.matmul(q, ke.transpose(2, 3)) * s["sm_scale"]
    i = torch.arange(l_ext, device=q.device)
    y = y.masked_fill_(i[None, :] > i.repeat_interleave(hq // hk)[:, None], -math.inf)
    p = _softmax(torch.cat([x, y], -1))
    v = (_gather(s["v_cache"], at) * s["v_scales"][page][..., None]).masked_fill_(~real[:, :, None, None], 0.0).transpose(1, 2)
    o = torch.matmul(p[..., :-l_ext], v) + torch.matmul(p[..., -l_ext:], ve)
    return o.view(b, hk, l_ext, hq // hk, d).permute(0, 2, 1, 3, 4).reshape(b * l_ext, hq, d).to(torch.bfloat16)


# ---- the definition in 64 bits ----


def _exact_turned(c, s, x):
    """The rotation as a product of complex numbers."""
    z, r = x.double().clone(), c["rot"]
    turn = torch.polar(torch.full((), s["size"], dtype=torch.float64, device=z.device).expand(len(s["positions"]), r // 2),
                       torch.outer(s["positions"].double(), s["inv_freq"].double()))[:, None]
    first = slice(0, r, 2) if c["interleaved"] else slice(0, r // 2)
    second = slice(1, r, 2) if c["interleaved"] else slice(r // 2, r)
    w = torch.complex(z[..., first], z[..., second]) * turn
    z[..., first], z[..., second] = w.real, w.imag
    return z


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "block":
        return _exact_block(case, s)
    q, k = _exact_turned(case, s, s["q"]), _exact_turned(case, s, s["k"])
    if case["op"] == "rope":
        return [q, k]
    v = s["v"].double()
    if case["op"] == "append":
        pools = []
        for x, scale in ((k, s["k_scale"]), (v, s["v_scale"])):
            pool = torch.zeros(s["k_buffer"].shape, dtype=torch.float64, device=q.device)
            pool[s["loc"]] = x / scale
            pools.append(pool.clamp(-TOP, TOP) if case["pool"] == "e4m3" else pool)
        return [q, k] + pools
    return [q, k] + _exact_append_block(case, s, k, v)


def _exact_append_block(case, s, k, v):
    """Block after block, in the order of the sequences."""
    size = case["block"]
    table = s["block_table"].cpu().numpy()
    # the largest new values of a row and head
    most = [x.abs().amax(-1).cpu().numpy() for x in (k, v)]
    caches = [s[w].double() for w in ("k_cache", "v_cache")]
    scales = [s[w].cpu().numpy().astype(np.float64) for w in ("k_scales", "v_scales")]
    place, div, more = [], [[], []], [[], []]
    at = 0
    for b, (p, n) in enumerate(zip(_past(case), s["lens"])):
        done = 0
        while done < n:
            col, off = divmod(p + done, size)
            here = min(n - done, size - off)
            page = int(table[b, col])
            place.append(np.arange(page * size + off, page * size + off + here))
            for w in (0, 1):
                top = most[w][at + done:at + done + here].max(0)
                now = np.array([2.0 ** max(-40, math.ceil(math.log2(x / TOP))) if x > 0 else SMALL for x in top])
                if off:
                    was = scales[w][page].copy()
                    now = np.maximum(now, was)
                    if (now != was).any():
                        more[w].append((page * size, off, was / now))
                scales[w][page] = now
                div[w].append(np.repeat(now[None], here, 0))
            done += here
        at += n
    place = torch.from_numpy(np.concatenate(place)).to(k.device)
    for w, x in ((0, k), (1, v)):
        for row, count, by in more[w]:
            caches[w][row:row + count] *= torch.from_numpy(by).to(k.device)[None, :, None]
        caches[w][place] = x / torch.from_numpy(np.concatenate(div[w])).to(k.device)[:, :, None]
    return caches + [torch.from_numpy(x) for x in scales]


def _exact_block(case, s):
    if work(case)["flops"] > 8e12:
        return None
    l_ext, size, g = case["l_ext"], case["block"], case["h_q"] // case["h_kv"]
    low = torch.tril(torch.ones(l_ext, l_ext, dtype=torch.bool, device=s["q"].device))
    outs = []
    for i, n in enumerate(s["lens"]):
        r = slice(i * l_ext, (i + 1) * l_ext)
        pages = s["block_table"][i, :-(-n // size)].long()
        rows = (pages[:, None] * size + torch.arange(size, device=pages.device)).flatten()[:n]
        keys, vals = (torch.cat([s[c].view(torch.uint8)[rows].view(torch.float8_e4m3fn).double()
                                 * s[m].double()[pages].repeat_interleave(size, 0)[:n, :, None], s[e][r].double()])
                      for c, m, e in (("k_cache", "k_scales", "k_ext"), ("v_cache", "v_scales", "v_ext")))
        q = s["q"][r].double() * case["d"] ** -0.5
        heads = []
        for u in range(case["h_q"]):
            x = q[:, u] @ keys[:, u // g].T
            x[:, n:] = torch.where(low, x[:, n:], torch.full_like(x[:, n:], -math.inf))
            heads.append(torch.exp(x - torch.logsumexp(x, 1, keepdim=True)) @ vals[:, u // g])
        outs.append(torch.stack(heads, 1))
    return torch.cat(outs)
