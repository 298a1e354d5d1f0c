"""Cases for what a serving step needs around the paged key-value cache: the attention of whole prompts, rotary
positions, pages and slots handed out on the GPU, and decode attention over a cache held in 4 bits.

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
# How the frequencies of rotary positions are made: base, then what stretches them for long contexts.
ROTARY = {
    "none": dict(base=10000.0),
    "linear": dict(base=10000.0, factor=4.0),
    "ntk": dict(base=10000.0, factor=8.0),
    "llama3": dict(base=500000.0, factor=8.0, original=8192, low=1.0, high=4.0),
    "yarn": dict(base=1000000.0, factor=4.0, original=32768, beta_fast=32.0, beta_slow=1.0),
}
S_K, S_V = 0.001953125, 0.0014648438   # calibrated tensor scales of a 4-bit cache: amax / (6 * 448) of N(0, 1) rows


def listed():
    return [
        # One user's first message on the smallest model: a call is all latency.
        dict(name="prompt_one_short", op="prompt", heads="qwen2.5-1.5b", seqs=1, lo=517, hi=517, window=0),
        # A prefill batch of chats, from a single token to two thousand.
        dict(name="prompt_batch", op="prompt", heads="llama3-8b", seqs=16, lo=1, hi=2047, window=0),
        # One long document, the most a layer computes.
        dict(name="prompt_long", op="prompt", heads="llama3-70b", seqs=1, lo=16001, hi=16001, window=0),
        # A sliding window over a multi-head model at a small head size.
        dict(name="prompt_window", op="prompt", heads="mha", seqs=24, lo=700, hi=6001, window=1024),
        # A decode step's new tokens at far positions.
        dict(name="rotary_step", op="rotary", heads="llama3-8b", tokens=128, far=131071, layout="half", dim=128,
             scaling="llama3"),
        # A prefill batch's queries and keys.
        dict(name="rotary_prompts", op="rotary", heads="llama3-70b", tokens=16380, far=40000, layout="half", dim=128,
             scaling="yarn"),
        # Interleaved pairs in half of each head, as other models turn them.
        dict(name="rotary_partial", op="rotary", heads="mha", tokens=9001, far=9000, layout="interleaved", dim=32,
             scaling="none"),
        # A decode step: every sequence grows by one token, a few of them into a new page.
        dict(name="resize_step", op="resize", seqs=128, hi=8191, page=16, done=0.0, fresh=0.0, prompt=1),
        # Continuous batching: some requests end, as many prompts come in, the others grow by a token.
        dict(name="resize_batch", op="resize", seqs=256, hi=4099, page=16, done=0.2, fresh=0.2, prompt=700),
        # Decode attention over the 4-bit cache: one user's chat, where a call is all latency.
        dict(name="attend4_one_short", op="attend", heads="qwen2.5-1.5b", seqs=1, lo=517, hi=517, page=16, window=0,
             weigh=False),
        # The serving path of a large batch.
        dict(name="attend4_batch", op="attend", heads="llama3-70b", seqs=32, lo=100, hi=8192, page=32, window=0,
             weigh=False),
        # One sequence with a very long context.
        dict(name="attend4_one_long", op="attend", heads="llama3-70b", seqs=1, lo=131071, hi=131071, page=128, window=0,
             weigh=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "rotary", "resize", "attend", "attend"])
    heads = rng.choice(sorted(HEADS))
    hq, hkv, d = HEADS[heads]
    if op == "prompt":
        hi = _log(rng, 1, 16384)
        seqs = _log(rng, 1, max(1, min(64, 65536 // hi, (1 << 40) // (hq * d * hi * hi))))
        while seqs * hq * d * hi * hi > 2 ** 41 * 0.95:
            hi = hi * 7 // 10
        return dict(op=op, heads=heads, seqs=seqs, lo=rng.randint(0, hi) if seqs > 1 else hi, hi=hi,
                    window=rng.choice([0, 0, 0, _log(rng, 1, hi)]))
    if op == "rotary":
        tokens = _log(rng, 1, max(1, min(32768, (1 << 27) // ((hq + hkv) * d))))
        return dict(op=op, heads=heads, tokens=tokens, far=_log(rng, 512, 1 << 20), layout=rng.choice(["half", "interleaved"]),
                    dim=rng.choice([d, d, d // 2, d // 4]), scaling=rng.choice(sorted(ROTARY)))
    if op == "resize":
        prompt = rng.choice([1, _log(rng, 2, 2048)])
        seqs = _log(rng, 1, min(512, max(1, 262144 // prompt)))
        return dict(op=op, seqs=seqs, hi=_log(rng, 16, 8192), page=rng.choice([8, 16, 32, 64, 128]),
                    done=rng.choice([0.0, rng.uniform(0, 0.5)]), fresh=rng.choice([0.0, rng.uniform(0, 0.5)]), prompt=prompt)
    hi = _log(rng, 1, 131072)
    seqs = _log(rng, 1, max(1, min(128, (1 << 30) // (2 * hkv * d * hi))))
    return dict(op=op, heads=heads, seqs=seqs, lo=rng.randint(0, hi) if seqs > 1 else hi, hi=hi,
                page=rng.choice([8, 16, 32, 64, 128]), window=rng.choice([0, 0, 0, _log(rng, 1, hi)]),
                weigh=rng.random() < 0.3)


# ---------------------------------------------------------------------------------------------- inputs

def _lens(case):
    """The batch's lengths, evenly spread between lo and hi: the same ones for every seed, which orders them."""
    n = case["seqs"]
    return [case["hi"]] if n == 1 else [round(case["lo"] + (case["hi"] - case["lo"]) * i / (n - 1)) for i in range(n)]


def _turned(case, seed):
    return np.array(_lens(case))[np.random.RandomState(seed % (1 << 32)).permutation(case["seqs"])]


def _queries(normal, g, rows, hq, hkv, d):
    """One stacked projection of the tokens: queries, keys and values side by side in a row. Queries differ in size from
    head to head, so that some heads look at few tokens and some at many."""
    qkv = normal(rows, (hq + 2 * hkv) * d)
    qkv[:, :hq * d] *= torch.exp(1.5 * torch.rand(hq, generator=g, device="cuda")).repeat_interleave(d)
    return qkv.bfloat16()


def _frequencies(dim, scaling):
    """Radians a position, in 64 bits, and what the rotated pairs are multiplied by."""
    a = ROTARY[scaling]
    i = np.arange(0, dim, 2, dtype=np.float64) / dim
    base, factor = a["base"], a.get("factor", 1.0)
    if scaling == "ntk":
        return (base * factor ** (dim / (dim - 2))) ** -i, 1.0
    f = base ** -i
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "llama3":
        turns = a["original"] * f / (2 * math.pi)   # that the original context makes
        smooth = np.clip((turns - a["low"]) / (a["high"] - a["low"]), 0.0, 1.0)
        return (1 - smooth) * f / factor + smooth * f, 1.0
    if scaling == "yarn":
        at = [dim * math.log(a["original"] / (beta * 2 * math.pi)) / (2 * math.log(base))
              for beta in (a["beta_fast"], a["beta_slow"])]
        low, high = max(0, math.floor(at[0])), min(dim - 1, math.ceil(at[1]))
        ramp = np.clip((np.arange(dim // 2) - low) / max(high - low, 0.001), 0.0, 1.0)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    return f, 1.0


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quantised(x, tensor_scale):
    """Rows [..., d] as E2M1 codes, two a byte (the first in the low bits), and an E4M3 scale for each 16 elements."""
    y = x.unflatten(-1, (-1, 16))
    scale = (y.abs().amax(-1) / (6 * tensor_scale)).clamp(max=448).to(torch.float8_e4m3fn)
    y = y / (scale.float() * tensor_scale).clamp(min=1e-30)[..., None]
    code = torch.bucketize(y.abs(), torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")).to(torch.uint8)
    code = (code + 8 * (y < 0)).to(torch.uint8).flatten(-2).unflatten(-1, (-1, 2))
    return code[..., 0] | (code[..., 1] << 4), scale.view(torch.uint8)


def _pages(lens, page, g, spare=3, width=0):
    """A table of pages in any order, as an allocator leaves them after a while, and the pages that are left. Entries
    behind a sequence's last page hold nothing (-1)."""
    used = [-(-int(x) // page) for x in lens]
    width = max([1, width] + used)
    n_pages = sum(used) + spare
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    live = torch.arange(width, device="cuda")[None] < torch.tensor(used, device="cuda")[:, None]
    table[live] = order[:sum(used)]
    return table, order[sum(used):], n_pages


def prepare(case, seed):
    op = case["op"]
    g = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if op == "resize":
        return _prepare_resize(case, seed, g)
    hq, hkv, d = HEADS[case["heads"]]
    s = dict(case=case, hq=hq, hkv=hkv, d=d, scale=1.0 / math.sqrt(d))
    if op == "prompt":
        lens = _turned(case, seed)
        rows = int(lens.sum())
        qkv = _queries(normal, g, rows, hq, hkv, d)
        s.update(seqs=case["seqs"], rows=rows, most=max(_lens(case)), qkv=qkv, q=qkv[:, :hq * d],
                 k=qkv[:, hq * d:(hq + hkv) * d], v=qkv[:, (hq + hkv) * d:],
                 cu=torch.tensor(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32), device="cuda"),
                 out=torch.empty(rows, hq * d, dtype=torch.bfloat16, device="cuda"),
                 lse=torch.empty(rows, hq, device="cuda"))
        return s
    if op == "rotary":
        # Positions as a batch brings them: those of a decode step lie anywhere, those of a prompt follow one another.
        rows = case["tokens"]
        qkv = _queries(normal, g, rows, hq, hkv, d)
        if rows <= 512:
            positions = torch.randint(0, case["far"] + 1, (rows,), generator=g, device="cuda")
        else:
            start = torch.randint(0, max(1, case["far"] - rows) + 1, (8,), generator=g, device="cuda")
            at = torch.arange(rows, device="cuda")
            positions = start[at * 8 // rows] + at
        f, amplitude = _frequencies(case["dim"], case["scaling"])
        s.update(rows=rows, x=qkv, positions=positions.to(torch.int32), f=torch.tensor(f, device="cuda"), amplitude=amplitude,
                 out=torch.empty(rows, (hq + hkv) * d, dtype=torch.bfloat16, device="cuda"))
        return s
    n, ps = case["seqs"], case["page"]
    lens = _turned(case, seed)
    table, _, n_pages = _pages(lens, ps, g)
    s.update(seqs=n, ps=ps, width=table.shape[1], n_pages=n_pages, table=table,
             lens=torch.tensor(lens.astype(np.int32), device="cuda"), k_scale=torch.full((1,), S_K, device="cuda"),
             v_scale=torch.full((1,), S_V, device="cuda"))
    codes = n_pages, hkv * ps * d // 2
    scales = n_pages, hkv * ps * d // 16
    for name in "kv":   # a page: the codes of its heads and slots, behind them their scales
        pool = torch.empty(n_pages, codes[1] + scales[1], dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 26) // (hkv * ps * d))
        for p in range(0, n_pages, step):
            part = pool[p:p + step]
            c, f = _quantised(normal(len(part), hkv, ps, d), s[name + "_scale"])
            part[:, :codes[1]], part[:, codes[1]:] = c.flatten(1), f.flatten(1)
        s[name] = pool
    qkv = _queries(normal, g, n, hq, hkv, d)
    w = torch.rand(n_pages, hkv, ps, generator=g, device="cuda")
    s.update(qkv=qkv, q=qkv[:, :hq * d], weight=torch.where(w < 0.05, 0.0, 4 * w ** 6),
             out=torch.empty(n, hq * d, dtype=torch.bfloat16, device="cuda"), lse=torch.empty(n, hq, device="cuda"))
    return s


def _requests(case, seed=0):
    """Lengths now and wanted: of the batch `done` requests end, `fresh` rows without one get a prompt, the rest grow by one."""
    r, n = np.random.RandomState(seed % (1 << 32)), case["seqs"]
    now = np.rint(np.linspace(1, case["hi"] - 1, n) if n > 1 else np.array([case["hi"] - 1])).astype(np.int64)
    want = now + 1
    done, fresh = int(case["done"] * n), int(case["fresh"] * n)
    kind = np.arange(n) * 7919 % n   # which rows: spread over the lengths
    want[kind < done] = 0
    new = (kind >= done) & (kind < done + fresh)
    now[new] = 0
    want[new] = 1 + np.arange(int(new.sum())) * 37 % case["prompt"]
    turn = r.permutation(n)
    return now[turn], want[turn]


def _prepare_resize(case, seed, g):
    n, ps = case["seqs"], case["page"]
    now, want = _requests(case, seed)
    width = -(-int(max(now.max(), want.max())) // ps)
    need = int(np.maximum(0, -(-want // ps) - -(-now // ps)).sum())
    table, free, n_pages = _pages(now, ps, g, spare=need + 5, width=width)
    rows = int(np.maximum(0, want - now).sum())
    head = int(np.random.RandomState(seed % (1 << 32)).randint(n_pages))
    # What the call changes, in one allocation: the table, the ring of free pages with its first place and number, lengths and
    # the number of tokens that each sequence has seen (some have lost slots to an eviction).
    sizes = [table.numel(), n_pages, 2, n, n]
    state = torch.zeros(sum(sizes), dtype=torch.int32, device="cuda")
    parts = list(state.split(sizes))
    parts[0].copy_(table.view(-1))
    parts[1].fill_(-1)
    parts[1][(torch.arange(len(free), device="cuda") + head) % n_pages] = free
    parts[2].copy_(torch.tensor([head, len(free)]))
    parts[3].copy_(torch.tensor(now))
    lost = torch.randint(0, 3, (n,), generator=g, device="cuda") * 100
    parts[4].copy_(parts[3] + torch.where(parts[3] > 0, lost, 0))
    return dict(case=case, ps=ps, seqs=n, width=width, n_pages=n_pages, rows=rows, state=state, state0=state.clone(),
                table=parts[0].view(n, width), ring=parts[1], ends=parts[2], lens=parts[3], seen=parts[4],
                want=torch.tensor(want.astype(np.int32), device="cuda"),
                cu=torch.empty(n + 1, dtype=torch.int32, device="cuda"),
                positions=torch.empty(rows, dtype=torch.int32, device="cuda"),
                slots=torch.empty(rows, dtype=torch.int64, device="cuda"))


# ---------------------------------------------------------------------------------------------- plain forms

def _prompt(s):
    n, hq, hkv, d, most, window = s["seqs"], s["hq"], s["hkv"], s["d"], s["most"], s["case"]["window"]
    cu = s["cu"].long()
    at = torch.arange(most, device="cuda")
    lens = cu[1:] - cu[:-1]
    live = at[None] < lens[:, None]                                       # [n, most]
    row = (cu[:-1, None] + at[None]).clamp(max=s["rows"] - 1)

    def padded(x, heads):                                                # [n, heads, most, d]
        return x[row].float().view(n, most, heads, d).masked_fill(~live[..., None, None], 0).transpose(1, 2)

    q = padded(s["q"], hq).view(n, hkv, hq // hkv, most, d)
    k, v = padded(s["k"], hkv), padded(s["v"], hkv)
    out, lse = s["out"].view(-1, hq, d), s["lse"]
    step = max(16, (1 << 30) // (n * hq * most))                          # query rows whose logits are held at once
    for i in range(0, most, step):
        here = at[i:i + step]
        first, end = (max(0, i - window + 1) if window else 0), min(most, i + step)
        j = at[None, first:end]
        c = len(here)
        x = torch.matmul(q[:, :, :, i:i + step].reshape(n, hkv, -1, d), k[:, :, first:end].transpose(2, 3)) * s["scale"]
        x = x.view(n, hq, c, -1)
        seen = j <= here[:, None]
        if window:
            seen = seen & (j > here[:, None] - window)
        x.masked_fill_(~seen, -math.inf)
        m = x.amax(-1, keepdim=True)
        x.sub_(m).exp_()
        total = x.sum(-1, keepdim=True)
        o = torch.matmul(x.div_(total).view(n, hkv, -1, end - first), v[:, :, first:end]).view(n, hq, c, d)
        mine = live[:, i:i + step]
        to = row[:, i:i + step][mine]
        out[to] = o.transpose(1, 2)[mine].bfloat16()
        lse[to] = (m + torch.log(total)).squeeze(-1).transpose(1, 2)[mine]
    return s["out"], s["lse"]


def _rotary(s):
    rows, heads, d, dim = s["rows"], s["hq"] + s["hkv"], s["d"], s["case"]["dim"]
    angle = (s["positions"].double()[:, None] * s["f"])[:, None]          # [rows, 1, dim / 2]
    cos, sin = torch.cos(angle) * s["amplitude"], torch.sin(angle) * s["amplitude"]
    x = s["x"][:, :heads * d].view(rows, heads, d)
    out = s["out"].view(rows, heads, d)
    turned = x[..., :dim].float()
    if s["case"]["layout"] == "half":
        a, b = turned[..., :dim // 2], turned[..., dim // 2:]
    else:
        a, b = turned[..., 0::2], turned[..., 1::2]
    cos, sin = cos.float(), sin.float()
    p, q = a * cos - b * sin, b * cos + a * sin
    if s["case"]["layout"] == "half":
        out[..., :dim // 2], out[..., dim // 2:dim] = p, q
    else:
        out[..., 0:dim:2], out[..., 1:dim:2] = p, q
    out[..., dim:] = x[..., dim:]
    return s["out"]


def _resize(s):
    s["state"].copy_(s["state0"])
    ps, n_pages, rows = s["ps"], s["n_pages"], s["rows"]
    old, want = s["lens"].long(), s["want"].long()
    head, count = s["ends"][0].long(), s["ends"][1].long()
    used, then = (old + ps - 1) // ps, (want + ps - 1) // ps
    need, new = (then - used).clamp(min=0), (want - old).clamp(min=0)
    there = count + (used - then).clamp(min=0).sum()
    granted = ((need == 0) | (need.cumsum(0) <= there)) & ((new == 0) | (new.cumsum(0) <= rows))
    after = torch.where(granted, want, old)
    then = torch.where(granted, then, used)
    new = torch.where(granted, new, 0)
    column = torch.arange(s["width"], device="cuda")[None]
    given_up = ((column >= then[:, None]) & (column < used[:, None])).view(-1)
    taken = ((column >= used[:, None]) & (column < then[:, None])).view(-1)
    to = (head + count + given_up.cumsum(0) - 1) % n_pages
    table = s["table"].view(-1)
    ring = torch.cat([s["ring"], s["ring"][:1]])                          # one place more, for what is not given up
    ring[torch.where(given_up, to, n_pages)] = table
    ring = ring[:n_pages]
    table.copy_(torch.where(taken, ring[(head + taken.cumsum(0) - 1) % n_pages], torch.where(given_up, -1, table)))
    s["ring"].copy_(ring)
    popped = taken.sum()
    s["ends"][0], s["ends"][1] = (head + popped) % n_pages, count + given_up.sum() - popped
    s["cu"][0] = 0
    s["cu"][1:] = new.cumsum(0)
    at = torch.arange(rows, device="cuda")
    seq = torch.searchsorted(s["cu"][1:].long(), at, right=True)
    i = at - s["cu"].long()[seq]
    slot = old[seq] + i
    s["slots"].copy_(s["table"][seq, slot // ps].long() * ps + slot % ps)
    s["positions"].copy_(s["seen"].long()[seq] + i)
    s["seen"].copy_(torch.where(after == 0, 0, s["seen"] + new))
    s["lens"].copy_(after)
    return _resized(s)


def _resized(s):
    return s["table"], s["ring"], s["ends"], s["lens"], s["seen"], s["cu"], s["positions"], s["slots"]


def _gathered(s, pool):
    """[pages, heads, page, ...] of a pool as [seqs, heads, slots, ...], behind each sequence whatever is there."""
    x = pool[s["table"].clamp(min=0).long()].transpose(1, 2)
    return x.reshape((s["seqs"], s["hkv"], s["width"] * s["ps"]) + tuple(pool.shape[3:]))


def _values(s, name):
    hkv, ps, d = s["hkv"], s["ps"], s["d"]
    codes, scales = s[name].split([hkv * ps * d // 2, hkv * ps * d // 16], dim=1)
    codes = _gathered(s, codes.view(-1, hkv, ps, d // 2)).int()
    scales = _gathered(s, scales.view(-1, hkv, ps, d // 16)).view(torch.float8_e4m3fn).float() * s[name + "_scale"]
    value = torch.tensor(E2M1 + tuple(-x for x in E2M1), device="cuda")
    x = torch.stack([value[codes & 15], value[codes >> 4]], -1).flatten(-2)
    return (x.unflatten(-1, (-1, 16)) * scales[..., None]).flatten(-2)


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
    s["out"].copy_(torch.matmul(e, v).view(n, -1))
    s["lse"].copy_((m + torch.log(total)).view(n, -1))
    if not case["weigh"]:
        return s["out"], s["lse"]
    w = e.sum(2).view(n, hkv, s["width"], s["ps"]).transpose(1, 2).reshape(-1, hkv, s["ps"])
    s["weight"].index_add_(0, s["table"].clamp(min=0).reshape(-1), w)
    return s["out"], s["lse"], s["weight"]


# ---------------------------------------------------------------------------------------------- one pass

def _own(s):
    import memory_bound_decoder_gb300 as mbd
    case, op = s["case"], s["case"]["op"]
    if op == "prompt":
        mbd.prompt_attention(s["out"], s["q"], s["qkv"].stride(0), s["k"], s["v"], s["qkv"].stride(0), s["cu"], s["seqs"],
                             s["rows"], s["hq"], s["hkv"], s["d"], s["scale"], case["window"], s["lse"])
        return s["out"], s["lse"]
    if op == "rotary":
        if "turns" not in s:   # a model's table, made once
            table, s["amp"] = mbd.rotary_table(case["dim"], scaling=case["scaling"], **ROTARY[case["scaling"]])
            s["turns"] = torch.frombuffer(table, dtype=torch.int64).to("cuda")
        heads, d = s["hq"] + s["hkv"], s["d"]
        mbd.rotary(s["out"], heads * d, s["x"], s["x"].stride(0), s["turns"], s["amp"], s["positions"], s["rows"], heads, d,
                   case["dim"], case["layout"])
        return s["out"]
    if op == "resize":
        s["state"].copy_(s["state0"])   # the lengths and pages of before, as each step of a program meets others
        mbd.kv_cache_resize(s["table"], s["width"], s["ps"], s["n_pages"], s["ring"], s["ends"], s["lens"], s["want"],
                            s["seqs"], s["cu"], s["positions"], s["slots"], s["rows"], s["seen"])
        return _resized(s)
    if "cache" not in s:   # the descriptor and the workspace that a program makes once, with its pools
        s["cache"] = mbd.kv_cache(s["k"], s["v"], s["n_pages"], s["ps"], s["hkv"], s["d"], "nvfp4", "static", s["k_scale"],
                                  s["v_scale"], s["weight"])
        s["bytes"] = mbd.paged_attention_workspace_bytes(s["cache"], s["width"], s["seqs"], s["hq"], case["weigh"])
        s["workspace"] = torch.empty(max(1, s["bytes"]), dtype=torch.uint8, device="cuda")
    mbd.paged_attention_decode(s["out"], s["q"], s["qkv"].stride(0), s["cache"], s["table"], s["width"], s["lens"], s["seqs"],
                               s["hq"], s["scale"], case["window"], s["lse"], case["weigh"], s["workspace"], s["bytes"])
    return (s["out"], s["lse"]) + ((s["weight"],) if case["weigh"] else ())


def run(s):
    if own:
        return _own(s)
    return {"prompt": _prompt, "rotary": _rotary, "resize": _resize, "attend": _attend}[s["case"]["op"]](s)


def work(case):
    op, n = case["op"], case.get("seqs", 0)
    if op == "resize":
        now, want = _requests(case)
        pages = int(np.abs(-(-want // case["page"]) - -(-now // case["page"])).sum())
        rows = int(np.maximum(0, want - now).sum())
        return {"bytes": 12 * pages + 12 * rows + 24 * n, "flops": 0}
    hq, hkv, d = HEADS[case["heads"]]
    if op == "rotary":
        rows = case["tokens"]
        return {"bytes": rows * (4 * (hq + hkv) * d + 4), "flops": rows * (hq + hkv) * case["dim"] * 3}
    lens = _lens(case)
    if op == "prompt":
        w = case["window"]
        pairs = sum(x * (x + 1) // 2 - (max(0, x - w) * (max(0, x - w) + 1) // 2 if w else 0) for x in lens)
        return {"bytes": sum(lens) * (2 * d * (2 * hq + 2 * hkv) + 4 * hq), "flops": 4 * pairs * hq * d}
    seen = sum(min(x, case["window"] or x) for x in lens)
    pages = sum(-(-x // case["page"]) for x in lens)
    row = d * 9 // 16   # one token's key or value of one head: codes and scales
    moved = seen * hkv * (2 * row + (8 if case["weigh"] else 0)) + n * hq * (4 * d + 4) + 4 * pages + 4 * n
    return {"bytes": moved, "flops": 4 * seen * hq * d}


# ---------------------------------------------------------------------------------------------- in 64 bits

def _one_double(s, name, b, length):
    """Sequence b's first rows of a 4-bit pool, [heads, length, d]."""
    hkv, ps, d = s["hkv"], s["ps"], s["d"]
    slot = torch.arange(length, device="cuda")
    page, at = s["table"][b, slot // ps].long() * s[name].shape[1], slot % ps
    flat = s[name].view(-1)
    out = torch.empty(hkv, length, d, dtype=torch.float64, device="cuda")
    for h in range(hkv):
        code = flat[(page + (h * ps + at) * (d // 2))[:, None] + torch.arange(d // 2, device="cuda")]
        mark = flat[(page + hkv * ps * (d // 2) + (h * ps + at) * (d // 16))[:, None] + torch.arange(d // 16, device="cuda")]
        e, m = ((mark >> 3) & 15).double(), (mark & 7).double()
        scale = torch.where(e == 0, m / 512, (1 + m / 8) * torch.exp2(e - 7))
        both = torch.stack([code & 15, code >> 4], -1).flatten(1)
        e, m = ((both >> 1) & 3).double(), (both & 1).double()
        x = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e - 1)) * (1 - 2 * (both >> 3).double())
        out[h] = x * scale.repeat_interleave(16, 1) * float(s[name + "_scale"])
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "resize":
        return _exact_resize(s)
    hq, hkv, d = s["hq"], s["hkv"], s["d"]
    group = hq // hkv
    if case["op"] == "rotary":
        rows, dim, heads = s["rows"], case["dim"], hq + hkv
        out = s["x"][:, :heads * d].double().view(rows, heads, d).clone()
        z = out[..., :dim].unflatten(-1, (2, -1) if case["layout"] == "half" else (-1, 2))
        z = torch.view_as_complex((z.transpose(-1, -2) if case["layout"] == "half" else z).contiguous())
        f, amplitude = _frequencies(dim, case["scaling"])
        angle = s["positions"].double()[:, None] * torch.from_numpy(f).cuda()
        z = torch.view_as_real(z * torch.polar(torch.full_like(angle, amplitude), angle)[:, None])
        out[..., :dim] = (z.transpose(-1, -2) if case["layout"] == "half" else z).flatten(-2)
        return out.view(rows, -1)
    if case["op"] == "prompt":
        rows, window, cu = s["rows"], case["window"], s["cu"].tolist()
        out = torch.zeros(rows, hq, d, dtype=torch.float64, device="cuda")
        lse = torch.zeros(rows, hq, dtype=torch.float64, device="cuda")
        for a, b in zip(cu, cu[1:]):
            for h in range(hkv):
                q = s["q"][a:b].double().view(b - a, hq, d)[:, h * group:(h + 1) * group].transpose(0, 1) / math.sqrt(d)
                k, v = (s[name][a:b, h * d:(h + 1) * d].double() for name in "kv")
                for i in range(0, b - a, 2048):
                    end = min(b - a, i + 2048)
                    first = max(0, i - window + 1) if window else 0
                    logits = q[:, i:end] @ k[first:end].t()
                    gap = torch.arange(i, end, device="cuda")[:, None] - torch.arange(first, end, device="cuda")
                    logits.masked_fill_((gap < 0) | (gap >= (window or rows + 1)), -math.inf)
                    total = torch.logsumexp(logits, -1)
                    lse[a + i:a + end, h * group:(h + 1) * group] = total.t()
                    p = logits.sub_(total[..., None]).exp_()
                    out[a + i:a + end, h * group:(h + 1) * group] = (p @ v[first:end]).transpose(0, 1)
        return out.view(rows, -1), lse
    n, ps, lens = s["seqs"], s["ps"], s["lens"].tolist()
    out = torch.zeros(n, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device="cuda")
    weight = s["weight"].double()
    for b, length in enumerate(lens):
        if not length:
            continue
        first = max(0, length - case["window"]) if case["window"] else 0
        q = s["q"][b].double().view(hkv, group, d)
        logits = torch.einsum("hgd,hld->hgl", q, _one_double(s, "k", b, length)[:, first:]) / math.sqrt(d)
        lse[b] = torch.logsumexp(logits, -1).view(-1)
        p = torch.exp(logits - lse[b].view(hkv, -1, 1))
        out[b] = torch.einsum("hgl,hld->hgd", p, _one_double(s, "v", b, length)[:, first:]).reshape(hq, d)
        if case["weigh"]:
            at = torch.arange(first, length, device="cuda")
            weight[s["table"][b, at // ps].long(), :, at % ps] += p.sum(1).t()
    return (out.view(n, -1), lse) + ((weight,) if case["weigh"] else ())


def _exact_resize(s):
    """The same by an allocator as one writes it on the host: a queue of free pages, one sequence after another."""
    ps, n_pages, rows = s["ps"], s["n_pages"], s["rows"]
    table, ring = s["table"].tolist(), s["ring"].tolist()
    head, count = s["ends"].tolist()
    lens, seen, want = s["lens"].tolist(), s["seen"].tolist(), s["want"].tolist()
    pages = lambda length: -(-length // ps)   # noqa: E731
    for b, (old, new) in enumerate(zip(lens, want)):
        for p in range(pages(new), pages(old)):
            ring[(head + count) % n_pages] = table[b][p]
            table[b][p] = -1
            count += 1
    asked_pages = asked_rows = 0
    there, cu, positions, slots = count, [0], [], []
    for b, (old, new) in enumerate(zip(lens, want)):
        more = max(0, pages(new) - pages(old))
        asked_pages += more
        asked_rows += max(0, new - old)
        if (more and asked_pages > there) or (new > old and asked_rows > rows):
            cu.append(cu[-1])
            continue
        for p in range(pages(old), pages(new)):
            table[b][p] = ring[head]
            head, count = (head + 1) % n_pages, count - 1
        for slot in range(old, new):
            positions.append(seen[b] + slot - old)
            slots.append(table[b][slot // ps] * ps + slot % ps)
        cu.append(cu[-1] + max(0, new - old))
        lens[b], seen[b] = new, (seen[b] + max(0, new - old)) if new else 0
    whole = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (table, ring, [head, count], lens, seen, cu, positions)]
    return tuple(whole) + (torch.tensor(slots, dtype=torch.int64, device="cuda"),)
