"""Cases for the key-value cache of a decode step: appending new tokens to a paged cache, the attention of one
new token over it (with or without the accumulation of what each cached token was given), and eviction from it
by that accumulated weight.

`own` chooses what run() calls: the operators' plain forms in torch, or this library's entry points.
"""
import math

import numpy as np
import torch

own = False

# Head layouts (query heads, key-value heads, head size) of the models whose layer shapes the workloads use, and
# two generic ones: plain multi-head attention at a small head, one key-value head for all.
HEADS = {
    "qwen2.5-1.5b": (12, 2, 128),
    "llama3-8b": (32, 8, 128),
    "llama3-70b": (64, 8, 128),
    "llama3.1-405b": (128, 8, 128),
    "mha": (16, 16, 64),
    "mqa": (16, 1, 64),
}
STATIC_K, STATIC_V = 0.03125, 0.0234375   # calibrated FP8 scales: amax of N(0, 1) rows at about half the range


def listed():
    return [
        # One user's chat on the smallest model: a short context, where a call is all latency.
        dict(name="attend_one_short", op="attend", heads="qwen2.5-1.5b", seqs=1, lo=517, hi=517, page=16, fmt="bf16",
             window=0, weigh=False),
        # Continuous batching of short chats, among them freshly padded rows with nothing in the cache.
        dict(name="attend_batch", op="attend", heads="llama3-8b", seqs=64, lo=0, hi=2047, page=16, fmt="bf16",
             window=0, weigh=False),
        # Long documents in a large batch: the most a layer reads.
        dict(name="attend_long_batch", op="attend", heads="llama3.1-405b", seqs=16, lo=9001, hi=32768, page=64,
             fmt="bf16", window=0, weigh=False),
        # The FP8 serving path: a calibrated scale for the tensor.
        dict(name="attend_fp8_batch", op="attend", heads="llama3-70b", seqs=32, lo=100, hi=8192, page=32,
             fmt="fp8_static", window=0, weigh=False),
        # One sequence with a very long context: few rows, the cache's length has to fill the card.
        dict(name="attend_one_long", op="attend", heads="llama3-70b", seqs=1, lo=131071, hi=131071, page=128,
             fmt="fp8_dynamic", window=0, weigh=False),
        # A sliding window over a multi-head model at a small head size.
        dict(name="attend_window", op="attend", heads="mha", seqs=24, lo=700, hi=6001, page=32, fmt="bf16",
             window=1024, weigh=False),
        # Decode under an eviction policy: the weights that each cached token is given are accumulated.
        dict(name="weigh_batch", op="attend", heads="llama3-8b", seqs=16, lo=1, hi=8191, page=16, fmt="bf16",
             window=0, weigh=True),
        # A decode step's new tokens, one for each sequence, quantised on the way in.
        dict(name="append_step_fp8", op="append", heads="llama3-8b", seqs=128, lo=1, hi=255, new=1, page=16,
             fmt="fp8_dynamic"),
        # A batch of prompts of uneven length, as the prefill leaves them in the stacked projection.
        dict(name="append_prompts", op="append", heads="llama3-8b", seqs=7, lo=1300, hi=2603, new=1170, page=16,
             fmt="bf16"),
        # The same into the FP8 cache of a calibrated model.
        dict(name="append_prompts_fp8", op="append", heads="llama3-70b", seqs=16, lo=1024, hi=2048, new=1023, page=64,
             fmt="fp8_static"),
        # A batch that has run into its budget: about half of the tokens go.
        dict(name="evict_batch", op="evict", heads="llama3-8b", seqs=16, lo=1500, hi=4099, page=16, fmt="bf16",
             budget=2048, recent=256),
        # One very long context cut down to what the next steps can afford.
        dict(name="evict_one_long", op="evict", heads="llama3-70b", seqs=1, lo=131072, hi=131072, page=128,
             fmt="fp8_dynamic", budget=32768, recent=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "evict"])
    heads = rng.choice(sorted(HEADS))
    hkv, d = HEADS[heads][1:]
    case = dict(op=op, heads=heads, page=rng.choice([8, 16, 32, 64, 128]),
                fmt=rng.choice(["bf16", "fp8_static", "fp8_dynamic"]))
    per_token = 2 * hkv * d * (2 if case["fmt"] == "bf16" else 1)
    if op == "append":
        new = rng.choice([1, _log(rng, 2, 2048)])
        seqs = _log(rng, 1, max(1, min(256, 16384 // new)))
        hi = new + _log(rng, 1, 512)
        return dict(case, seqs=seqs, lo=new, hi=hi, new=new)
    hi = _log(rng, 1 if op == "attend" else 64, 131072)
    seqs = _log(rng, 1, max(1, min(128, (1 << 29) // (per_token * hi))))
    case.update(seqs=seqs, lo=rng.randint(0, hi) if seqs > 1 else hi, hi=hi)
    if op == "attend":
        return dict(case, window=rng.choice([0, 0, 0, _log(rng, 1, hi)]), weigh=rng.random() < 0.4)
    budget = max(1, int(hi * rng.uniform(0.1, 1.0)))
    return dict(case, budget=budget, recent=rng.randint(0, budget))


# ---------------------------------------------------------------------------------------------- inputs

def _lens(case):
    """The batch's lengths, evenly spread between lo and hi: the same ones for every seed, which orders them."""
    n = case["seqs"]
    return [case["hi"]] if n == 1 else [round(case["lo"] + (case["hi"] - case["lo"]) * i / (n - 1)) for i in range(n)]


def _new(case):
    """New tokens of the append cases, by sequence: one each, or uneven prompts of at most `new`."""
    n, lens = case["seqs"], _lens(case)
    if case["new"] == 1:
        return [1] * n
    return [min(lens[i], max(1, case["new"] * (n - i) // n)) for i in range(n)]


def _e4m3(x):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def prepare(case, seed):
    hq, hkv, d = HEADS[case["heads"]]
    ps, n, fmt = case["page"], case["seqs"], case["fmt"]
    g = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    # Lengths in an order of the seed's; the pages of a pool in any order, as an allocator leaves them after a while;
    # entries of the page table behind a sequence's last page hold nothing (-1).
    lens, new = _lens(case), _new(case) if case["op"] == "append" else [0] * n
    turn = np.random.RandomState(seed % (1 << 32)).permutation(n)
    lens, new = [lens[i] for i in turn], [new[i] for i in turn]
    width = max(1, -(-max(lens) // ps))
    used = [-(-x // ps) for x in lens]
    n_pages = sum(used) + 3
    free = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    column = torch.arange(width, device="cuda")
    live = column[None] < torch.tensor(used, device="cuda")[:, None]
    table[live] = free[:sum(used)]
    s = dict(case=case, hq=hq, hkv=hkv, d=d, ps=ps, seqs=n, width=width, n_pages=n_pages, table=table,
             lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), scale=1.0 / math.sqrt(d), fmt=fmt)

    shape = (n_pages, hkv, ps, d)
    s["k_scale"] = s["v_scale"] = None
    if fmt == "bf16":
        s["k"], s["v"] = normal(*shape).bfloat16(), normal(*shape).bfloat16()
    elif fmt == "fp8_static":
        s["k_scale"] = torch.full((1,), STATIC_K, device="cuda")
        s["v_scale"] = torch.full((1,), STATIC_V, device="cuda")
        s["k"], s["v"] = _e4m3(normal(*shape) / s["k_scale"]), _e4m3(normal(*shape) / s["v_scale"])
    else:
        for name in "kv":
            x = normal(*shape)
            scale = x.abs().amax(-1) / 448
            s[name], s[name + "_scale"] = _e4m3(x / scale[..., None]), scale
    # One stacked projection of the new tokens: queries, keys and values side by side in a row. Queries differ in
    # size from head to head, so that some heads look at few tokens and some at many.
    rows = sum(new) if case["op"] == "append" else n
    qkv = normal(rows, (hq + 2 * hkv) * d)
    qkv[:, :hq * d] *= torch.exp(1.5 * torch.rand(hq, generator=g, device="cuda")).repeat_interleave(d)
    qkv = qkv.bfloat16()
    s["qkv"], s["q"] = qkv, qkv[:, :hq * d]
    s["k_new"], s["v_new"] = qkv[:, hq * d:(hq + hkv) * d], qkv[:, (hq + hkv) * d:]
    if case["op"] == "append":
        s["tokens"] = rows
        s["cu"] = None if case["new"] == 1 else torch.tensor(np.concatenate([[0], np.cumsum(new)]).astype(np.int32),
                                                             device="cuda")
        return s
    # What earlier steps have accumulated: heavy-tailed, with tokens that were never looked at. Positions: those of
    # the newest half in order, the older ones shuffled by earlier evictions, which left gaps between them.
    meta = torch.empty((2,) + shape[:3], dtype=torch.int32, device="cuda")
    weight, position = meta[0].view(torch.float32), meta[1]
    w = torch.rand(*shape[:3], generator=g, device="cuda")
    weight.copy_(torch.where(w < 0.05, 0.0, 4 * w ** 6))
    if case["op"] == "attend":
        s["weight"] = weight
        s["out"] = torch.empty(n, hq * d, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(n, hq, device="cuda")
        return s
    cap = width * ps
    slot = torch.arange(cap, device="cuda")[None, None]
    half = (s["lens"].long() // 2)[:, None, None]
    order = torch.rand(n, hkv, cap, generator=g, device="cuda") + (slot >= half) * 1.0
    order = torch.where(slot < half, order, 2.0 + slot)
    rank = torch.argsort(torch.argsort(order, -1), -1)
    at = torch.where(slot < half, 2 * rank, half + rank).to(torch.int32)
    position.zero_()
    at = at.view(n, hkv, width, ps).permute(0, 2, 1, 3)
    position[table[live].long()] = at[live]
    s.update(meta=meta, meta0=meta.clone(), weight=weight, position=position,
             new_lens=torch.empty(n, dtype=torch.int32, device="cuda"))
    return s


# ---------------------------------------------------------------------------------------------- plain forms

def _gathered(s, pool):
    """[pages, heads, page, ...] of a pool as [seqs, heads, slots, ...], behind each sequence whatever is there."""
    x = pool[s["table"].clamp(min=0).long()].transpose(1, 2)
    return x.reshape((s["seqs"], s["hkv"], s["width"] * s["ps"]) + tuple(pool.shape[3:]))


def _values(s, name):
    x, scale = _gathered(s, s[name]).float(), s[name + "_scale"]
    if s["fmt"] == "fp8_static":
        x *= scale
    elif s["fmt"] == "fp8_dynamic":
        x *= _gathered(s, scale)[..., None]
    return x


def _attend(s):
    case, n, hkv, d = s["case"], s["seqs"], s["hkv"], s["d"]
    k = _values(s, "k")
    x = torch.matmul(s["q"].float().view(n, hkv, -1, d), k.transpose(2, 3)) * s["scale"]
    del k
    slot, lens = torch.arange(x.shape[-1], device="cuda")[None], s["lens"][:, None]
    seen = slot < lens
    if case["window"]:
        seen = seen & (slot >= lens - case["window"])
    x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m.masked_fill(m == -math.inf, 0))
    total = e.sum(-1, keepdim=True)
    e /= total.clamp(min=1e-30)
    v = _values(s, "v").masked_fill_(~seen[:, None, :, None], 0)
    out = torch.matmul(e, v).view(n, -1).bfloat16()
    lse = (m + torch.log(total)).view(n, -1)
    if not case["weigh"]:
        return out, lse
    w = e.sum(2).view(n, hkv, s["width"], s["ps"]).transpose(1, 2).reshape(-1, hkv, s["ps"])
    s["weight"].index_add_(0, s["table"].clamp(min=0).reshape(-1), w)
    return out, lse, s["weight"]


def _append(s):
    n, hkv, d, rows = s["seqs"], s["hkv"], s["d"], s["tokens"]
    row = torch.arange(rows, device="cuda")
    cu = torch.arange(n + 1, device="cuda") if s["cu"] is None else s["cu"].long()
    seq = torch.searchsorted(cu, row, right=True) - 1
    slot = s["lens"].long()[seq] - cu[seq + 1] + row
    page, at = s["table"][seq, slot // s["ps"]].long(), slot % s["ps"]
    for name in "kv":
        x, scale = s[name + "_new"].reshape(rows, hkv, d), s[name + "_scale"]
        if s["fmt"] == "bf16":
            s[name][page, :, at] = x
            continue
        x = x.float()
        if s["fmt"] == "fp8_dynamic":
            of_row = x.abs().amax(-1) / 448
            scale[page, :, at] = of_row
            x = torch.where(of_row[..., None] > 0, x / of_row[..., None], 0)
        else:
            x = x / scale
        s[name].view(torch.uint8)[page, :, at] = _e4m3(x).view(torch.uint8)
    return (s["k"], s["v"]) + ((s["k_scale"], s["v_scale"]) if s["fmt"] == "fp8_dynamic" else ())


def _evicted(s):
    pools = (s["k"], s["v"]) + ((s["k_scale"], s["v_scale"]) if s["fmt"] == "fp8_dynamic" else ())
    return pools + (s["weight"], s["position"], s["new_lens"])


def _evict(s):
    s["meta"].copy_(s["meta0"])
    budget, recent, ps = s["case"]["budget"], s["case"]["recent"], s["ps"]
    lens = s["lens"].long()[:, None, None]
    torch.clamp(s["lens"], max=budget, out=s["new_lens"])
    if s["width"] * ps <= budget:
        return _evicted(s)
    weight, position = _gathered(s, s["weight"]), _gathered(s, s["position"])
    slot = torch.arange(weight.shape[-1], device="cuda")[None, None]
    live = slot < lens
    newest = position.masked_fill(~live, -1).amax(-1, keepdim=True)
    rank = weight.masked_fill(position.long() > newest.long() - recent, math.inf).masked_fill(~live, -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices
    kept = torch.zeros_like(live.expand_as(rank)).scatter_(-1, order[..., :budget], True)
    over = live & (lens > budget)
    hole, mover = over & ~kept & (slot < budget), over & kept & (slot >= budget)
    to, source = torch.nonzero(hole, as_tuple=True), torch.nonzero(mover, as_tuple=True)   # in ascending order of the slots
    b, h = to[0], to[1]
    page_to, page_from = (s["table"][b, x // ps].long() for x in (to[2], source[2]))
    at_to, at_from = to[2] % ps, source[2] % ps
    for pool in _evicted(s)[:-1]:
        pool = pool.view(torch.uint8) if pool.dtype == torch.float8_e4m3fn else pool
        pool[page_to, h, at_to] = pool[page_from, h, at_from]
    return _evicted(s)


# ---------------------------------------------------------------------------------------------- one pass

def _own(s):
    import memory_bound_decoder_gb300 as mbd
    case, op = s["case"], s["case"]["op"]
    if "cache" not in s:   # the descriptor and the workspace that a program makes once, with its pools
        mode = "dynamic" if s["fmt"] == "fp8_dynamic" else "static"
        s["cache"] = mbd.kv_cache(s["k"], s["v"], s["n_pages"], s["ps"], s["hkv"], s["d"],
                                  "bf16" if s["fmt"] == "bf16" else "fp8", mode, s["k_scale"], s["v_scale"],
                                  s.get("weight"), s.get("position"))
        if op == "attend":
            nbytes = mbd.paged_attention_workspace_bytes(s["cache"], s["width"], s["seqs"], s["hq"], case["weigh"])
            s["workspace"] = torch.empty(max(1, nbytes), dtype=torch.uint8, device="cuda")
            s["workspace_bytes"] = nbytes
    if op == "attend":
        mbd.paged_attention_decode(s["out"], s["q"], s["qkv"].stride(0), s["cache"], s["table"], s["width"], s["lens"],
                                   s["seqs"], s["hq"], s["scale"], case["window"], s["lse"], case["weigh"],
                                   s["workspace"], s["workspace_bytes"])
        return (s["out"], s["lse"]) + ((s["weight"],) if case["weigh"] else ())
    if op == "append":
        mbd.kv_cache_append(s["cache"], s["k_new"], s["v_new"], s["qkv"].stride(0), s["table"], s["width"], s["lens"],
                            s["seqs"], s["tokens"], s["cu"])
        return (s["k"], s["v"]) + ((s["k_scale"], s["v_scale"]) if s["fmt"] == "fp8_dynamic" else ())
    s["meta"].copy_(s["meta0"])   # a full cache again, as each eviction of a program meets one
    mbd.kv_cache_evict(s["cache"], s["new_lens"], s["lens"], s["table"], s["width"], s["seqs"], case["budget"],
                       case["recent"])
    return _evicted(s)


def run(s):
    if own:
        return _own(s)
    return {"attend": _attend, "append": _append, "evict": _evict}[s["case"]["op"]](s)


def work(case):
    hq, hkv, d = HEADS[case["heads"]]
    size = 2 if case["fmt"] == "bf16" else 1
    row = d * size + (4 if case["fmt"] == "fp8_dynamic" else 0)   # one token's key or value of one head
    n, lens = case["seqs"], _lens(case)
    if case["op"] == "append":
        rows = sum(_new(case))
        return {"bytes": rows * 2 * hkv * (2 * d + row) + 8 * n, "flops": 0 if size == 2 else rows * 4 * hkv * d}
    pages = sum(-(-x // case["page"]) for x in lens)
    if case["op"] == "attend":
        seen = sum(min(x, case["window"] or x) for x in lens)
        moved = seen * hkv * (2 * row + (8 if case["weigh"] else 0)) + n * hq * (4 * d + 4) + 4 * pages + 4 * n
        return {"bytes": moved, "flops": 4 * seen * hq * d}
    # Eviction: every live token's weight and position, and the rows that have to move: those kept behind the budget.
    moved, read = 0.0, 0
    for x in lens:
        if x > case["budget"]:
            old = x - case["recent"]
            share = (case["budget"] - case["recent"]) / max(1, old)
            behind = x - max(case["budget"], old)
            moved += behind + share * max(0, old - case["budget"])
            read += x
    return {"bytes": 8 * read * hkv + moved * hkv * 2 * (2 * row + 8) + 8 * n + 4 * pages, "flops": 2 * read * hkv}


# ---------------------------------------------------------------------------------------------- in 64 bits

def _e4m3_exact(x):
    """The E4M3 value nearest to each 64-bit value, ties to even: steps of 2^(e-3), 2^-9 below 2^-6, at most 448."""
    _, e = torch.frexp(x.abs().clamp(min=2.0 ** -6))
    step = torch.exp2((e - 4).double())
    return (torch.round(x / step) * step).clamp(-448, 448)


def _one(s, pool, b, used):
    """Sequence b's rows of a pool, heads first."""
    x = pool[s["table"][b, :used].long()]
    return x.transpose(0, 1).reshape((s["hkv"], used * s["ps"]) + tuple(pool.shape[3:]))


def _one_double(s, name, b, used):
    x = _one(s, s[name], b, used).double()
    if s["fmt"] == "fp8_static":
        return x * s[name + "_scale"].double()
    return x if s["fmt"] == "bf16" else x * _one(s, s[name + "_scale"], b, used).double()[..., None]


def exact(case, seed):
    s = prepare(case, seed)
    hq, hkv, d, ps, n = s["hq"], s["hkv"], s["d"], s["ps"], s["seqs"]
    lens, table = s["lens"].tolist(), s["table"]
    if case["op"] == "attend":
        out = torch.zeros(n, hq, d, dtype=torch.float64, device="cuda")
        lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device="cuda")
        weight = s["weight"].double()
        for b, length in enumerate(lens):
            if not length:
                continue
            used, first = -(-length // ps), max(0, length - case["window"]) if case["window"] else 0
            q = s["q"][b].double().view(hkv, hq // hkv, d)
            k = _one_double(s, "k", b, used)[:, first:length]
            logits = torch.einsum("hgd,hld->hgl", q, k) / math.sqrt(d)
            lse[b] = torch.logsumexp(logits, -1).view(-1)
            p = torch.exp(logits - lse[b].view(hkv, -1, 1))
            out[b] = torch.einsum("hgl,hld->hgd", p, _one_double(s, "v", b, used)[:, first:length]).reshape(hq, d)
            if case["weigh"]:
                at = torch.arange(first, length, device="cuda")
                weight[table[b, at // ps].long(), :, at % ps] += p.sum(1).t()
        return (out.view(n, -1), lse) + ((weight,) if case["weigh"] else ())
    if case["op"] == "append":
        cu = list(range(n + 1)) if s["cu"] is None else s["cu"].tolist()
        got = {name: s[name].double() for name in "kv"}
        scales = {name: s[name + "_scale"].double() for name in "kv"} if s["fmt"] != "bf16" else {}
        for b, length in enumerate(lens):
            count = cu[b + 1] - cu[b]
            at = torch.arange(length - count, length, device="cuda")
            page = table[b, at // ps].long()
            for name in "kv":
                x = s[name + "_new"][cu[b]:cu[b + 1]].double().reshape(count, hkv, d)
                if s["fmt"] == "fp8_static":
                    x = _e4m3_exact(x / scales[name])
                elif s["fmt"] == "fp8_dynamic":
                    top = x.abs().amax(-1) / 448
                    scales[name][page, :, at % ps] = top
                    x = _e4m3_exact(torch.nan_to_num(x / top[..., None]))
                got[name][page, :, at % ps] = x
        return (got["k"], got["v"]) + ((scales["k"], scales["v"]) if s["fmt"] == "fp8_dynamic" else ())
    # Eviction moves values and computes none: each head's kept slots by an ordinary sort on the host.
    budget, recent = case["budget"], case["recent"]
    pools = [x.double() if x.dtype != torch.int32 else x.clone() for x in _evicted(s)[:-1]]
    for b, length in enumerate(lens):
        if length <= budget:
            continue
        used = -(-length // ps)
        weight = _one(s, s["weight"], b, used)[:, :length].cpu().numpy()
        position = _one(s, s["position"], b, used)[:, :length].cpu().numpy()
        for h in range(hkv):
            old = position[h] <= position[h].max() - recent
            best = np.lexsort((np.arange(length), -weight[h], old))[:budget]
            kept = np.zeros(length, bool)
            kept[best] = True
            to = torch.from_numpy(np.flatnonzero(~kept[:budget])).cuda()
            source = torch.from_numpy(budget + np.flatnonzero(kept[budget:])).cuda()
            for pool in pools:
                pool[table[b, to // ps].long(), h, to % ps] = pool[table[b, source // ps].long(), h, source % ps]
    return tuple(pools) + (torch.tensor([min(x, budget) for x in lens], dtype=torch.int32, device="cuda"),)
