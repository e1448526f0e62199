"""The prompt, shared-prefix and cache-eviction operators: their cases, inputs and plain forms.

Four operators around the verify call (``verify_splitkv_fwd``):

``prompt``  attention over whole prompts, causal, grouped heads, sequences of
            different lengths packed one after the other (``prompt_attn_fwd``);
``shared``  the verify call for a batch whose sequences share a long prefix,
            read once for all of them (``verify_splitkv_shared_fwd``);
``mass``    the attention weight every cached key receives from a verify
            call, added to what it had (``verify_splitkv_mass``);
``evict``   the cache index cut down to a budget by that weight
            (``kv_evict``).

``run`` computes a case in elementary torch operations in 32 bits, or with
``own`` set through the package's entry points.  ``exact`` computes it again
from the definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False


def _c(name, op, **kw):
    return {"name": name, "op": op, **kw}


def listed():
    return [
        # one request of one token: what a call costs before any arithmetic
        _c("prompt_one_token", "prompt", batch=1, lo=1, hi=1, h_q=32, h_kv=8, d=128),
        # a burst of short chat turns of odd lengths, small heads
        _c("prompt_short_turns_d64", "prompt", batch=16, lo=17, hi=701, h_q=8, h_kv=2, d=64),
        # a few documents, the wide head size
        _c("prompt_documents_d256", "prompt", batch=3, lo=511, hi=2049, h_q=16, h_kv=2, d=256),
        # long prompts at the serving shape
        _c("prompt_long", "prompt", batch=4, lo=4001, hi=8192, h_q=32, h_kv=8, d=128),
        # few sequences after a short common instruction
        _c("shared_small", "shared", shared=512, batch=4, lo=64, hi=96, l_ext=4, h_q=4, h_kv=1, d=64, pool="bf16"),
        # a common document in an e4m3 cache, the wide head size
        _c("shared_fp8_d256", "shared", shared=8192, batch=8, lo=0, hi=512, l_ext=4, h_q=16, h_kv=2, d=256, pool="e4m3"),
        # the serving batch behind one long system prompt
        _c("shared_serving", "shared", shared=32768, batch=64, lo=128, hi=2048, l_ext=4, h_q=32, h_kv=8, d=128, pool="bf16"),
        # two short sequences
        _c("mass_tiny", "mass", batch=2, lo=64, hi=96, l_ext=4, h_q=4, h_kv=1, d=64, pool="bf16"),
        # two mid-size sequences in an e4m3 cache, the wide head size
        _c("mass_fp8_d256", "mass", batch=2, lo=4096, hi=8192, l_ext=4, h_q=16, h_kv=2, d=256, pool="e4m3"),
        # the serving batch
        _c("mass_serving", "mass", batch=64, lo=8192, hi=32768, l_ext=4, h_q=32, h_kv=8, d=128, pool="bf16"),
        # a few sequences just past their budget
        _c("evict_small", "evict", batch=4, lo=200, hi=1001, h_kv=2, budget=256, recent=32),
        # the serving batch cut down to 4k tokens each
        _c("evict_serving", "evict", batch=64, lo=8192, hi=32768, h_kv=8, budget=4096, recent=512),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: any operator, sizes over the logarithm of their range, odd ones among them."""
    big = {c["op"]: work(c) for c in listed()}  # the last one of each operator is its largest
    while True:
        op = rng.choice(["prompt", "shared", "mass", "evict"])
        h_kv = rng.choice([1, 2, 3, 4, 8])
        if op == "evict":
            hi = _log(rng, 2, 32768)
            budget = _log(rng, 1, 8192)
            c = {"op": op, "batch": _log(rng, 1, 64), "lo": rng.randint(0, hi), "hi": hi, "h_kv": h_kv, "budget": budget,
                 "recent": rng.randint(0, budget)}
        else:
            d = rng.choice([64, 128, 256])
            g = rng.choice([1, 2, 3, 4, 5, 7, 8])
            c = {"op": op, "h_q": g * h_kv, "h_kv": h_kv, "d": d}
            if op == "prompt":
                hi = _log(rng, 1, 8192)
                c.update(batch=_log(rng, 1, 64), lo=rng.randint(1, hi), hi=hi)
            else:
                hi = _log(rng, 16, 2048 if op == "shared" else 32768)
                l_ext = min(_log(rng, 1, 16), (64 if d == 256 else 128) // g)
                c.update(batch=_log(rng, 1, 64), lo=rng.randint(0, hi), hi=hi, l_ext=l_ext,
                         pool=rng.choice(["bf16", "e4m3"]))
                if op == "shared":
                    c["shared"] = _log(rng, 33, 32768)
        w, top = work(c), big[op]
        heads = c.get("h_q", h_kv) * max(1, c.get("l_ext", 1))
        top_heads = {"prompt": 32, "shared": 128, "mass": 128, "evict": 8}[op]
        if w["bytes"] <= top["bytes"] and w["flops"] <= top["flops"] and heads <= top_heads and sum(_lens(c)) > 0:
            return c


def _lens(c):
    """The sequences' lengths: the case's own, whatever the seed of the inputs."""
    r = random.Random(1000003 * c["batch"] + 1009 * c["lo"] + c["hi"])
    return [r.randint(c["lo"], c["hi"]) for _ in range(c["batch"])]


def _scale(c):
    return 1.0 / math.sqrt(c["d"])


def _scales(c):
    return (0.5, 0.25) if c["pool"] == "e4m3" else (1.0, 1.0)


def work(c):
    n = _lens(c)
    t, b = sum(n), c["batch"]
    if c["op"] == "prompt":
        return {"bytes": 4 * t * c["d"] * (c["h_q"] + c["h_kv"]) + 4 * (b + 1),
                "flops": 4 * c["d"] * c["h_q"] * sum(x * (x + 1) // 2 for x in n)}
    if c["op"] == "evict":
        kept = sum(min(x, c["budget"]) for x in n)
        return {"bytes": 4 * c["h_kv"] * (t + kept) + 8 * 2 * t + 8 * (b + 1), "flops": t * c["h_kv"]}
    rows, e, l_ext = b * c["l_ext"], 1 if c["pool"] == "e4m3" else 2, c["l_ext"]
    drafts = b * l_ext * (l_ext + 1) // 2
    if c["op"] == "shared":
        keys = c["shared"] + t
        return {"bytes": 2 * keys * c["h_kv"] * c["d"] * e + 8 * keys + 4 * rows * c["d"] * (c["h_q"] + c["h_kv"]) + 8 * (b + 1),
                "flops": 4 * c["d"] * c["h_q"] * (rows * c["shared"] + l_ext * t + drafts)}
    return {"bytes": t * c["h_kv"] * (c["d"] * e + 8) + 8 * t + 2 * rows * c["d"] * (c["h_q"] + c["h_kv"]) + 8 * (b + 1),
            "flops": 2 * c["d"] * c["h_q"] * (l_ext * t + drafts)}


def _indptr(n, dev):
    return torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32, device=dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    n = _lens(case)
    t, b = sum(n), case["batch"]
    s = {"case": case, "lens": n, "own": own}

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.bfloat16)

    if case["op"] == "prompt":
        hq, hk, d = case["h_q"], case["h_kv"], case["d"]
        s.update(q=normal(t, hq, d), k=normal(t, hk, d), v=normal(t, hk, d), qo_indptr=_indptr(n, dev),
                 o=torch.zeros(t, hq, d, dtype=torch.bfloat16, device=dev), sm_scale=_scale(case))
        return s
    s["kv_indptr"] = _indptr(n, dev)
    if case["op"] == "evict":
        # weights of a heavy-tailed kind, as attention gives them; some keys got none at all
        mass = torch.exp(2.0 * torch.randn(case["h_kv"], t, generator=g, device=dev)) * 1e-3
        mass[:, torch.rand(t, generator=g, device=dev) < 0.05] = 0.0
        kept = sum(min(x, case["budget"]) for x in n)
        i64 = {"dtype": torch.int64, "device": dev}
        s.update(mass=mass, kv_indices=torch.randperm(t, generator=g, device=dev), out_kv_indptr=torch.zeros(b + 1, dtype=torch.int32, device=dev),
                 out_kv_indices=torch.zeros(kept, **i64), out_mass=torch.zeros(case["h_kv"], kept, device=dev),
                 freed=torch.zeros(t - kept, **i64))
        return s
    hq, hk, d, rows = case["h_q"], case["h_kv"], case["d"], b * case["l_ext"]
    sh = case.get("shared", 0)
    cache = torch.float8_e4m3fn if case["pool"] == "e4m3" else torch.bfloat16
    perm = torch.randperm(sh + t, generator=g, device=dev)
    s.update(q=normal(rows, hq, d), k_ext=normal(rows, hk, d), k_buffer=normal(sh + t, hk, d).to(cache),
             kv_indices=perm[sh:].clone(), qo_indptr=_indptr([case["l_ext"]] * b, dev), sm_scale=_scale(case))
    s["k_scale"], s["v_scale"] = _scales(case)
    if case["op"] == "shared":
        s.update(v_ext=normal(rows, hk, d), v_buffer=normal(sh + t, hk, d).to(cache), shared_indices=perm[:sh].clone(),
                 o=torch.zeros(rows, hq, d, dtype=torch.bfloat16, device=dev))
    else:
        s.update(mass_in=torch.rand(hk, t, generator=g, device=dev), mass=torch.zeros(hk, t, device=dev))
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        return _run_own(op, s)
    return {"prompt": _prompt, "shared": _shared, "mass": _mass, "evict": _evict}[op](s)


def _run_own(op, s):
    import speculative_decode_verify_prefix_gb300 as vsk

    if op == "prompt":
        vsk.prompt_attn_fwd(s["q"], s["k"], s["v"], s["o"], s["qo_indptr"], sm_scale=s["sm_scale"])
        return s["o"]
    if op == "shared":
        vsk.verify_splitkv_shared_fwd(s["q"], s["k_ext"], s["v_ext"], s["o"], s["k_buffer"], s["v_buffer"],
                                      s["qo_indptr"], s["kv_indptr"], s["kv_indices"], s["shared_indices"],
                                      s["case"]["l_ext"], s["k_scale"], s["v_scale"], sm_scale=s["sm_scale"])
        return s["o"]
    if op == "mass":
        vsk.verify_splitkv_mass(s["q"], s["k_ext"], s["k_buffer"], s["qo_indptr"], s["kv_indptr"], s["kv_indices"],
                                s["mass"], s["case"]["l_ext"], s["k_scale"], sm_scale=s["sm_scale"],
                                mass_in=s["mass_in"])
        return s["mass"]
    vsk.kv_evict(s["mass"], s["kv_indptr"], s["kv_indices"], s["case"]["budget"], s["case"]["recent"],
                 s["out_kv_indptr"], s["out_kv_indices"], s["out_mass"], s["freed"])
    return [s["out_kv_indptr"], s["out_kv_indices"], s["out_mass"], s["freed"]]


# ---- plain forms, 32 bits ----


def _softmax(x):
    """Over the last dimension; a row with nothing visible (all -inf) is 0."""
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total == 0, torch.ones_like(total), total)


def _prompt(s):
    c, o, at = s["case"], torch.empty_like(s["o"]), 0
    g, hk, d = c["h_q"] // c["h_kv"], c["h_kv"], c["d"]
    for n in s["lens"]:
        q = s["q"][at:at + n].float().view(n, hk, g, d).permute(1, 2, 0, 3).reshape(hk, g * n, d)
        k = s["k"][at:at + n].float().transpose(0, 1)
        v = s["v"][at:at + n].float().transpose(0, 1)
        x = (torch.matmul(q, k.transpose(1, 2)) * s["sm_scale"]).view(hk, g, n, n)
        pos = torch.arange(n, device=x.device)
        p = _softmax(x.masked_fill_(pos[None, :] > pos[:, None], -math.inf))
        y = torch.matmul(p.view(hk, g * n, n), v).view(hk, g, n, d)
        o[at:at + n] = y.permute(2, 0, 1, 3).reshape(n, hk * g, d).to(o.dtype)
        at += n
    return o


def _own_keys(s):
    """The sequences' own prefixes as one padded batch: positions in kv_indices and which of them are real."""
    first, last = s["kv_indptr"][:-1].long(), s["kv_indptr"][1:].long()
    j = torch.arange(max(s["lens"]), device=first.device)
    real = j[None, :] < (last - first)[:, None]
    return torch.where(real, first[:, None] + j[None, :], torch.zeros_like(first)[:, None]), real


def _grouped(s):
    """Queries as [batch, h_kv, l_ext * group, d] and draft keys as [batch, h_kv, l_ext, d]."""
    c = s["case"]
    b, l_ext, hk, d = c["batch"], c["l_ext"], c["h_kv"], c["d"]
    q = s["q"].float().view(b, l_ext, hk, c["h_q"] // hk, d).permute(0, 2, 1, 3, 4).reshape(b, hk, -1, d)
    return q, s["k_ext"].float().view(b, l_ext, hk, d).transpose(1, 2)


def _draft_scores(s, q, ke):
    c = s["case"]
    x = torch.matmul(q, ke.transpose(2, 3)) * s["sm_scale"]
    i = torch.arange(c["l_ext"], device=x.device)
    row = i.repeat_interleave(c["h_q"] // c["h_kv"])
    return x.masked_fill_(i[None, :] > row[:, None], -math.inf)


def _gather(pool, at):
    """Pool rows as 32-bit values; e4m3 rows are gathered as bytes."""
    if pool.dtype == torch.float8_e4m3fn:
        return pool.view(torch.uint8)[at].view(torch.float8_e4m3fn).float()
    return pool[at].float()


def _own_scores(s, q):
    at, real = _own_keys(s)
    loc = s["kv_indices"][at] if s["kv_indices"].numel() else at
    k = _gather(s["k_buffer"], loc).permute(0, 2, 3, 1)
    x = torch.matmul(q, k) * (s["sm_scale"] * s["k_scale"])
    return x.masked_fill_(~real[:, None, None, :], -math.inf), loc, real


def _shared(s):
    c = s["case"]
    b, l_ext, hk, hq, d, sh = c["batch"], c["l_ext"], c["h_kv"], c["h_q"], c["d"], c["shared"]
    q, ke = _grouped(s)
    m = q.shape[2]
    ks = _gather(s["k_buffer"], s["shared_indices"]).permute(1, 2, 0)
    vs = _gather(s["v_buffer"], s["shared_indices"]).transpose(0, 1)
    flat = q.transpose(0, 1).reshape(hk, b * m, d)
    x0 = (torch.matmul(flat, ks) * (s["sm_scale"] * s["k_scale"])).view(hk, b, m, sh).transpose(0, 1)
    x1, loc, real = _own_scores(s, q)
    p = _softmax(torch.cat([x0, x1, _draft_scores(s, q, ke)], -1))
    y0 = torch.matmul(p[..., :sh].transpose(0, 1).reshape(hk, b * m, sh), vs).view(hk, b, m, d).transpose(0, 1)
    vo = _gather(s["v_buffer"], loc).masked_fill_(~real[:, :, None, None], 0.0).transpose(1, 2)
    y1 = torch.matmul(p[..., sh:-l_ext], vo)
    ve = s["v_ext"].float().view(b, l_ext, hk, d).transpose(1, 2)
    y = s["v_scale"] * (y0 + y1) + torch.matmul(p[..., -l_ext:], ve)
    y = y.view(b, hk, l_ext, hq // hk, d).permute(0, 2, 1, 3, 4)
    return y.reshape(b * l_ext, hq, d).to(torch.bfloat16)


def _places(s):
    """The sequence of every entry of kv_indices, and its position there."""
    at = torch.arange(sum(s["lens"]), device=s["kv_indptr"].device)
    seq = torch.searchsorted(s["kv_indptr"][1:].long(), at, right=True)
    return seq, at - s["kv_indptr"].long()[seq]


def _mass(s):
    q, ke = _grouped(s)
    x, _, _ = _own_scores(s, q)
    n = x.shape[-1]
    w = _softmax(torch.cat([x, _draft_scores(s, q, ke)], -1))[..., :n].sum(2)
    seq, j = _places(s)
    return s["mass_in"] + w[seq, :, j].t()


def _evict(s):
    c = s["case"]
    total = s["mass"][0]
    for row in s["mass"][1:]:  # the definition's order of the sum
        total = total + row
    n = (s["kv_indptr"][1:] - s["kv_indptr"][:-1]).long()[:, None]
    at, real = _own_keys(s)
    j = torch.arange(at.shape[1], device=at.device)[None, :]
    old = j < n - c["recent"]
    x = torch.where(old, total[at], torch.full_like(total[:1], -math.inf))
    order = torch.sort(x, dim=1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, j.expand_as(order).contiguous())
    keep = (n <= c["budget"]) | ~old | (rank < c["budget"] - c["recent"])
    seq, jj = _places(s)
    keep = keep[seq, jj]
    indptr = torch.zeros_like(s["kv_indptr"])
    indptr[1:] = torch.cumsum(torch.clamp(n[:, 0], max=c["budget"]), 0)
    kept, gone = s["out_kv_indices"].numel(), s["freed"].numel()
    to = torch.cumsum(keep, 0) - 1
    to_gone = torch.cumsum(~keep, 0) - 1
    idx = s["kv_indices"].new_zeros(kept + 1)
    idx[torch.where(keep, to, torch.full_like(to, kept))] = s["kv_indices"]
    m = s["mass"].new_zeros(c["h_kv"], kept + 1)
    m[:, torch.where(keep, to, torch.full_like(to, kept))] = s["mass"]
    freed = s["kv_indices"].new_zeros(gone + 1)
    freed[torch.where(keep, torch.full_like(to, gone), to_gone)] = s["kv_indices"]
    return [indptr, idx[:kept], m[:, :kept].contiguous(), freed[:gone]]


# ---- the definition in 64 bits ----


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "evict":
        return _exact_evict(case, s)
    if work(case)["flops"] > 8e12:
        return None
    g, hk = case["h_q"] // case["h_kv"], case["h_kv"]
    if case["op"] == "prompt":
        o = torch.empty(s["o"].shape, dtype=f64, device=s["o"].device)
        at = 0
        for n in s["lens"]:
            i = torch.arange(n, device=o.device)
            for h in range(hk):
                k, v = s["k"][at:at + n, h].to(f64), s["v"][at:at + n, h].to(f64)
                for u in range(h * g, (h + 1) * g):
                    x = (s["q"][at:at + n, u].to(f64) @ k.T) * case["d"] ** -0.5
                    x = torch.where(i[:, None] >= i[None, :], x, torch.full_like(x, -math.inf))
                    o[at:at + n, u] = torch.exp(x - torch.logsumexp(x, 1, keepdim=True)) @ v
            at += n
        return o
    l_ext, b = case["l_ext"], case["batch"]
    first = [0] + list(np.cumsum(s["lens"]))
    sh = s["shared_indices"] if case["op"] == "shared" else s["kv_indices"][:0]
    group = [h // g for h in range(case["h_q"])]
    outs, mass = [], torch.empty(hk, sum(s["lens"]), dtype=f64, device=s["q"].device)

    def rows64(pool, loc):
        return pool.view(torch.uint8)[loc].view(pool.dtype).to(f64) if pool.dtype == torch.float8_e4m3fn else pool[loc].to(f64)

    # the shared rows' scores of all sequences together: they are what takes long here
    kc = rows64(s["k_buffer"], sh) * s["k_scale"]
    vc = rows64(s["v_buffer"], sh) * s["v_scale"] if case["op"] == "shared" else None
    low = torch.tril(torch.ones(l_ext, l_ext, dtype=torch.bool, device=s["q"].device))
    for i in range(b):
        r = slice(i * l_ext, (i + 1) * l_ext)
        loc = s["kv_indices"][first[i]:first[i + 1]]
        q = s["q"][r].to(f64) * case["d"] ** -0.5
        ko = rows64(s["k_buffer"], loc) * s["k_scale"]
        kd = s["k_ext"][r].to(f64)
        keys = torch.cat([kc, ko, kd])
        x = torch.stack([q[:, u] @ keys[:, group[u]].T for u in range(case["h_q"])])
        x[:, :, -l_ext:] = torch.where(low, x[:, :, -l_ext:], torch.full_like(x[:, :, -l_ext:], -math.inf))
        p = torch.exp(x - torch.logsumexp(x, 2, keepdim=True))
        if case["op"] == "shared":
            vals = torch.cat([vc, rows64(s["v_buffer"], loc) * s["v_scale"], s["v_ext"][r].to(f64)])
            outs.append(torch.stack([p[u] @ vals[:, group[u]] for u in range(case["h_q"])], 1))
        else:
            w = p[:, :, :len(loc)].sum(1).view(hk, g, len(loc)).sum(1)
            mass[:, first[i]:first[i + 1]] = w + s["mass_in"][:, first[i]:first[i + 1]].to(f64)
    return torch.cat(outs) if case["op"] == "shared" else mass


def _exact_evict(case, s):
    mass, idx = s["mass"].cpu().numpy(), s["kv_indices"].cpu().numpy()
    total = mass[0].copy()
    for h in range(1, len(mass)):
        total = (total + mass[h]).astype(np.float32)  # the definition: 32 bits, heads in ascending order
    keep, ptr, at = [], [0], 0
    for n in s["lens"]:
        old = max(0, n - case["recent"])
        if n <= case["budget"]:
            k = np.arange(n)
        else:
            best = np.lexsort((np.arange(old), -total[at:at + old].astype(np.float64)))[:case["budget"] - case["recent"]]
            k = np.concatenate([np.sort(best), np.arange(old, n)])
        keep.append(at + k)
        ptr.append(ptr[-1] + len(k))
        at += n
    keep = np.concatenate(keep).astype(np.int64)
    gone = np.setdiff1d(np.arange(at), keep)
    return [torch.tensor(ptr, dtype=torch.int32), torch.from_numpy(idx[keep]), torch.from_numpy(mass[:, keep].astype(np.float64)),
            torch.from_numpy(idx[gone])]
