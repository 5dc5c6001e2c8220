"""What is measured of the paged KV-cache operators: appending a step's keys
and values (per-head Q/K RMSNorm and rotary embedding applied on the way) to a
paged cache, and the grouped-query attention that reads that cache, each for a
bf16 cache and for an E4M3 one with a power-of-two scale per 16-token block and
head.

A case is one call.  `seqs` sequences bring up to `q` new tokens each, after
which the longest holds `ctx` tokens; with `ragged` the others hold less and
bring less.  The attention's causal rule lets the query at position p see the
keys at positions p - window + 1 .. p (0: all up to p); `sinks` adds a learned
logit per head to the softmax's denominator.
"""
import math
import random

import torch

own = False

D = 128          # head size
BLOCK = 16       # tokens that share a scale in the E4M3 cache
EPS = 1e-6
CODE_MAX = 448.0
EXP_MIN, EXP_MAX = -40, 40   # exponents of the block scales


def listed():
    c = dict(heads=32, kv_heads=4, page=16, theta=1e6, window=0, sinks=False, ragged=False)
    return [
        # A single user's next token: nothing but latency.
        dict(c, name="append bf16 1 token", op="append", cache="bf16", seqs=1, q=1, ctx=1000),
        # A chunk of prompts, several at once and of odd lengths.
        dict(c, name="append bf16 prompts", op="append", cache="bf16", seqs=3, q=1021, ctx=4093,
             ragged=True, page=64),
        # The next token of eight users in the middle of their contexts.
        dict(c, name="append e4m3 8 tokens", op="append", cache="e4m3", seqs=8, q=1, ctx=2000,
             ragged=True),
        # A large prompt, brought into the 8-bit cache in chunks.
        dict(c, name="append e4m3 prompts", op="append", cache="e4m3", seqs=2, q=4096, ctx=8192,
             ragged=True, page=64),
        # Eight users at 100K tokens, full attention, bf16 cache.
        dict(c, name="attend bf16 8 x 100K", op="attend", cache="bf16", seqs=8, q=1, ctx=100000),
        # A sliding-window layer with sinks, 32 users: short ranges, many of them.
        dict(c, name="attend bf16 32 window", op="attend", cache="bf16", seqs=32, q=1, ctx=4001,
             ragged=True, window=513, sinks=True),
        # A prompt's chunk of 2048 tokens over 8192: bound by arithmetic.
        dict(c, name="attend bf16 prompt", op="attend", cache="bf16", seqs=1, q=2048, ctx=8192,
             page=64),
        # A short conversation's next token: latency again.
        dict(c, name="attend e4m3 1 x 1000", op="attend", cache="e4m3", seqs=1, q=1, ctx=1000),
        # One user at 100K tokens: the long axis has to be split.
        dict(c, name="attend e4m3 1 x 100K", op="attend", cache="e4m3", seqs=1, q=1, ctx=100000,
             sinks=True),
        # 32 users up to 100K tokens, each of another length: the largest cache.
        dict(c, name="attend e4m3 32 x 100K", op="attend", cache="e4m3", seqs=32, q=1, ctx=100000,
             ragged=True, page=64),
        # Drafted tokens verified, four a user.
        dict(c, name="attend e4m3 8 x 4 drafts", op="attend", cache="e4m3", seqs=8, q=4, ctx=30011,
             ragged=True),
        # Prompt chunks in a sliding-window layer with sinks.
        dict(c, name="attend e4m3 prompts", op="attend", cache="e4m3", seqs=3, q=1000, ctx=5000,
             ragged=True, window=513, sinks=True, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    group, kv_heads = rng.choice([(8, 4), (8, 4), (8, 4), (4, 4), (8, 2), (8, 1), (2, 8), (1, 4)])
    c = dict(op=rng.choice(["append", "attend", "attend"]), cache=rng.choice(["bf16", "e4m3"]),
             heads=group * kv_heads, kv_heads=kv_heads, page=rng.choice([16, 32, 64, 128]),
             theta=rng.choice([1e6, 1e4, 0.0]), ragged=rng.random() < 0.7,
             window=rng.choice([0, 0, 513, _log(rng, 1, 4000)]), sinks=rng.random() < 0.5)
    if c["op"] == "append":
        seqs = _log(rng, 1, 128)
        q = 1 if rng.random() < 0.4 else _log(rng, 1, 8192 // seqs)
        ctx = q + _log(rng, 1, 400000 // seqs) - 1
        return dict(c, seqs=seqs, q=q, ctx=ctx, window=0, sinks=False)
    if rng.random() < 0.6:    # next tokens
        seqs = _log(rng, 1, 128)
        most = (1 if c["cache"] == "bf16" else 4) * 800000 * 4 // max(4, kv_heads)
        return dict(c, seqs=seqs, q=1, ctx=_log(rng, 1, min(100000, most // seqs)))
    seqs = _log(rng, 1, 16)   # drafts and prompt chunks
    q = _log(rng, 2, 2048 // seqs)
    ctx = min(q + _log(rng, 1, 30000) - 1, max(q, 2048 * 8192 // (seqs * q)))
    return dict(c, seqs=seqs, q=q, ctx=ctx)


def _lengths(c):
    """(new tokens, tokens after the call) of each sequence: the case's own, whatever the seed."""
    rng = random.Random("%(seqs)d %(q)d %(ctx)d" % c)
    new, total = [c["q"]], [c["ctx"]]
    for _ in range(1, c["seqs"]):
        n = rng.randint(1, c["q"]) if c["ragged"] else c["q"]
        new.append(n)
        total.append(max(n, rng.randint(max(1, c["ctx"] // 4), c["ctx"])) if c["ragged"] else c["ctx"])
    return new, total


def _visible(c):
    """(cached tokens that some query sees, query-key pairs) of a head."""
    tokens = pairs = 0
    for n, total in zip(*_lengths(c)):
        first = total - n
        lo = max(0, first - c["window"] + 1) if c["window"] else 0
        tokens += total - lo
        if c["window"]:
            w = c["window"]
            short = max(0, min(n, w - 1 - first))  # queries with fewer than w keys before them
            pairs += sum(range(first + 1, first + short + 1)) + (n - short) * w
        else:
            pairs += n * first + n * (n + 1) // 2
    return tokens, pairs


def work(c):
    new, _ = _lengths(c)
    t, h, kv = sum(new), c["heads"], c["kv_heads"]
    size = 2 if c["cache"] == "bf16" else 1 + 4.0 / (BLOCK * D)
    if c["op"] == "append":
        return {"bytes": t * (h + 2 * kv) * D * 2 + t * h * D * 2 + t * 2 * kv * D * size,
                "flops": t * (h + kv) * D * 10}
    tokens, pairs = _visible(c)
    return {"bytes": 2 * t * h * D * 2 + tokens * 2 * kv * D * size, "flops": 4 * D * h * pairs}


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(int(seed))
    h, kv, page = c["heads"], c["kv_heads"], c["page"]
    new, total = _lengths(c)
    pages = [-(-n // page) for n in total]
    n_pages = sum(pages) + 1
    order = torch.randperm(n_pages, generator=g, device=dev, dtype=torch.int64).to(torch.int32)
    table = torch.full((c["seqs"], max(pages)), -1, dtype=torch.int32, device=dev)
    at = 0
    for s, n in enumerate(pages):
        table[s, :n] = order[at:at + n]
        at += n
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    seq_of = [s for s, n in enumerate(new) for _ in range(n)]
    t = start[-1]
    st = dict(c, tokens=t, max_q=max(new), max_len=max(total), n_pages=n_pages, page_table=table,
              q_start=torch.tensor(start, dtype=torch.int32, device=dev),
              kv_len=torch.tensor(total, dtype=torch.int32, device=dev),
              seq_of=torch.tensor(seq_of, device=dev))
    gain = lambda: (1.5 + 0.1 * torch.randn(D, generator=g, device=dev)).to(torch.bfloat16)  # noqa: E731
    kc, ks = _cache(c, g, n_pages, 1.5)
    vc, vs = _cache(c, g, n_pages, 1.0)
    st.update(k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs)
    if c["op"] == "append":
        st["qkv"] = torch.randn(t, (h + 2 * kv) * D, generator=g, device=dev).to(torch.bfloat16)
        st["q_norm"], st["k_norm"] = gain(), gain()
        st["q_out"] = torch.zeros(t, h, D, dtype=torch.bfloat16, device=dev)
    else:
        st["q"] = (1.5 * torch.randn(t, h, D, generator=g, device=dev)).to(torch.bfloat16)
        st["sink"] = torch.randn(h, generator=g, device=dev) if c["sinks"] else None
        st["out"] = torch.zeros(t, h, D, dtype=torch.bfloat16, device=dev)
    if own:
        import moe_decode_sigmoid_gb300 as m
        st["dims"] = m.AttnDims(h, kv, D)
        st["batch"] = m.PagedBatch(st["q_start"], st["kv_len"], table, page, max(new))
        st["workspace"] = m.new_attn_workspace() if c["op"] == "attend" else None
    return st


def _cache(c, g, n_pages, size):
    """One cache with earlier tokens in all its rows, each of a loudness of its own."""
    dev, shape = g.device, (n_pages, c["page"], c["kv_heads"], D)
    if c["cache"] == "bf16":
        x = torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)
        loud = torch.exp(0.3 * torch.randn(shape[:3], generator=g, device=dev)) * size
        return x.mul_(loud[..., None].to(torch.bfloat16)), None
    codes = torch.empty(shape, dtype=torch.float8_e4m3fn, device=dev)
    scale = torch.empty(n_pages, c["page"] // BLOCK, c["kv_heads"], device=dev)
    step = max(1, (1 << 28) // (c["page"] * c["kv_heads"] * D))
    for i in range(0, n_pages, step):
        x = torch.randn((min(step, n_pages - i),) + shape[1:], generator=g, device=dev)
        x *= torch.exp(0.3 * torch.randn(x.shape[:3], generator=g, device=dev))[..., None] * size
        x = x.view(x.shape[0], -1, BLOCK, c["kv_heads"], D)
        s = _scale_for(x.abs().amax(dim=(2, 4)))
        scale[i:i + step] = s
        codes[i:i + step] = (x / s[:, :, None, :, None]).to(torch.float8_e4m3fn).view(-1, *shape[1:])
    return codes.view(torch.uint8), scale


def _scale_for(amax):
    """The smallest power of two whose 448-fold is at least amax, within its limits."""
    m, e = torch.frexp(amax)                       # amax = m 2^e, 448 = 0.875 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(amax > 0, e, torch.full_like(e, EXP_MIN)).clamp(EXP_MIN, EXP_MAX)
    return torch.ldexp(torch.ones_like(amax), e)


def run(st):
    if st["op"] == "append":
        outs = _append_own(st) if own else _append_plain(st)
        if st["cache"] == "bf16":
            return [st["q_out"] if own else outs, st["k_cache"], st["v_cache"]]
        return [st["q_out"] if own else outs, st["k_cache"].view(torch.float8_e4m3fn),
                st["v_cache"].view(torch.float8_e4m3fn), st["k_scale"], st["v_scale"]]
    return _attend_own(st) if own else _attend_plain(st)


def _append_own(st):
    import moe_decode_sigmoid_gb300 as m
    if st["cache"] == "bf16":
        m.flint_qk_norm_rope_kv_paged_bf16(st["qkv"], st["q_norm"], st["k_norm"], st["batch"],
                                           st["q_out"], st["k_cache"], st["v_cache"], st["theta"],
                                           EPS, dims=st["dims"])
    else:
        m.flint_qk_norm_rope_kv_paged_fp8(st["qkv"], st["q_norm"], st["k_norm"], st["batch"],
                                          st["q_out"], st["k_cache"], st["v_cache"],
                                          st["k_scale"], st["v_scale"], st["theta"], EPS,
                                          dims=st["dims"])


def _attend_own(st):
    import moe_decode_sigmoid_gb300 as m
    if st["cache"] == "bf16":
        m.flint_attn_paged_bf16(st["q"], st["k_cache"], st["v_cache"], st["batch"], st["out"],
                                st["workspace"], sinks=st["sink"], window=st["window"],
                                dims=st["dims"])
    else:
        m.flint_attn_paged_fp8(st["q"], st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"],
                               st["batch"], st["out"], st["workspace"], sinks=st["sink"],
                               window=st["window"], dims=st["dims"])
    return st["out"]


def _positions(st):
    """The position of every new token."""
    s = st["seq_of"]
    rest = st["q_start"][s + 1].long() - torch.arange(st["tokens"], device=s.device)
    return st["kv_len"][s].long() - rest


def _append_plain(st):
    h, kv, page, s = st["heads"], st["kv_heads"], st["page"], st["seq_of"]
    pos = _positions(st)
    x = st["qkv"].float().view(st["tokens"], h + 2 * kv, D)

    def turned(x, gain):
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gain.float()
        if not st["theta"]:
            return x
        freq = st["theta"] ** (-2.0 * torch.arange(D // 2, device=x.device, dtype=torch.float64) / D)
        angle = pos[:, None].double() * freq
        cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
        a, b = x[..., :D // 2], x[..., D // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    q = turned(x[:, :h], st["q_norm"]).to(torch.bfloat16)
    k, v = turned(x[:, h:h + kv], st["k_norm"]), x[:, h + kv:]
    slot = st["page_table"][s, pos // page].long() * page + pos % page
    if st["cache"] == "bf16":
        st["k_cache"].view(-1, kv, D)[slot] = k.to(torch.bfloat16)
        st["v_cache"].view(-1, kv, D)[slot] = v.to(torch.bfloat16)
        return q
    block = slot // BLOCK
    # Rows of each token's block that hold earlier tokens of its sequence.
    first = st["kv_len"][s].long() - (st["q_start"][s + 1] - st["q_start"][s]).long()
    kept = (first - (pos - pos % BLOCK)).clamp(0, BLOCK)
    _quantise(k, st["k_cache"], st["k_scale"], slot, block, kept)
    _quantise(v, st["v_cache"], st["v_scale"], slot, block, kept)
    return q


def _quantise(x, cache, scale, slot, block, kept):
    kv = x.shape[1]
    rows, scale = cache.view(torch.float8_e4m3fn).view(-1, BLOCK, kv, D), scale.view(-1, kv)
    amax = torch.zeros_like(scale).scatter_reduce(0, block[:, None].expand(-1, kv),
                                                  x.abs().amax(-1), "amax")
    old = scale[block]
    wanted = _scale_for(amax[block])
    grown = torch.where(kept[:, None] > 0, torch.maximum(old, wanted), wanted)
    codes = rows[block].float()
    again = (codes * (old / grown)[:, None, :, None]).to(torch.float8_e4m3fn)
    earlier = torch.arange(BLOCK, device=x.device) < kept[:, None]
    rows.view(torch.uint8)[block] = torch.where(earlier[..., None, None], again.view(torch.uint8),
                                                rows.view(torch.uint8)[block])
    code = (x / grown[..., None]).clamp(-CODE_MAX, CODE_MAX).to(torch.float8_e4m3fn)
    rows.view(torch.uint8).view(-1, kv, D)[slot] = code.view(torch.uint8)
    scale[block] = grown


def _attend_plain(st):
    h, kv, page, s = st["heads"], st["kv_heads"], st["page"], st["seq_of"]
    n, dev = st["seqs"], s.device
    start, length = st["q_start"].long(), st["kv_len"].long()
    count = start[1:] - start[:-1]
    i = torch.arange(st["max_q"], device=dev)
    row = (start[:-1, None] + i).clamp(max=st["tokens"] - 1)
    pos = (length - count)[:, None] + i                                     # [n, max_q]
    j = torch.arange(st["max_len"], device=dev)
    seen = (j <= pos[..., None]) & (j < length[:, None, None])              # [n, max_q, len]
    if st["window"]:
        seen &= j > pos[..., None] - st["window"]
    slot = st["page_table"][:, j // page].long().clamp(min=0) * page + j % page
    held = (j < length[:, None])[..., None, None]

    def rows(name):
        x = st[name + "_cache"]
        if st["cache"] == "bf16":
            x = x.view(-1, kv, D)[slot].float()
        else:
            x = x.view(torch.float8_e4m3fn).view(-1, kv, D)[slot].float()
            x *= st[name + "_scale"].view(-1, kv)[slot // BLOCK][..., None]
        return x.masked_fill_(~held, 0.0).transpose(1, 2)                   # [n, kv, len, D]

    q = st["q"][row].float().view(n, -1, kv, h // kv, D).permute(0, 2, 1, 3, 4)
    score = q.reshape(n, kv, -1, D) @ rows("k").transpose(2, 3) * D ** -0.5
    score = score.view(n, kv, st["max_q"], h // kv, -1)
    score.masked_fill_(~seen[:, None, :, None], -math.inf)
    most = score.amax(-1, keepdim=True)
    sink = st["sink"].view(kv, 1, h // kv, 1) if st["sinks"] else None
    if sink is not None:
        most = torch.maximum(most, sink)
    most = most.masked_fill(most == -math.inf, 0.0)
    p = score.sub_(most).exp_()
    total = p.sum(-1, keepdim=True)
    if sink is not None:
        total = total + (sink - most).exp()
    o = (p.view(n, kv, -1, st["max_len"]) @ rows("v")).view(n, kv, st["max_q"], h // kv, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o)).permute(0, 2, 1, 3, 4)
    t = torch.arange(st["tokens"], device=dev)
    return o[s, t - start[s]].reshape(st["tokens"], h, D).to(torch.bfloat16)


def exact(c, seed):
    st = prepare(c, seed)
    return _append_exact(c, st) if c["op"] == "append" else _attend_exact(c, st)


def _token_slots(c, st, s, positions):
    return [int(p) for p in (st["page_table"][s].cpu()[positions // c["page"]].long() * c["page"]
                             + positions % c["page"])]


def _append_exact(c, st):
    h, kv, half = c["heads"], c["kv_heads"], D // 2
    new, total = _lengths(c)
    where = torch.cat([torch.arange(b - a, b) for a, b in zip(new, total)]).to("cuda").double()
    x = st["qkv"].double().reshape(-1, h + 2 * kv, D)
    out = []
    for part, gain in ((x[:, :h], st["q_norm"]), (x[:, h:h + kv], st["k_norm"])):
        y = part / (part.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * gain.double()
        if c["theta"]:
            i = torch.arange(half, device="cuda", dtype=torch.float64)
            turn = torch.polar(torch.ones(len(where), half, device="cuda", dtype=torch.float64),
                               where[:, None] * c["theta"] ** (-i / half))
            z = torch.complex(y[..., :half].contiguous(), y[..., half:].contiguous()) * turn[:, None]
            y = torch.cat([z.real, z.imag], -1)
        out.append(y)
    q, k = out
    v = x[:, h + kv:]
    if c["cache"] == "bf16":
        kc, vc = st["k_cache"].double(), st["v_cache"].double()
    else:
        kc = st["k_cache"].view(torch.float8_e4m3fn).double()
        vc = st["v_cache"].view(torch.float8_e4m3fn).double()
    scales = [st["k_scale"], st["v_scale"]]
    at = 0
    for s in range(c["seqs"]):
        lo, hi = total[s] - new[s], total[s]
        slots = torch.tensor(_token_slots(c, st, s, torch.arange(lo, hi)), device="cuda")
        for i, (cache, values) in enumerate(((kc, k), (vc, v))):
            flat = cache.view(-1, kv, D)
            mine = values[at:at + new[s]]
            if c["cache"] == "bf16":
                flat[slots] = mine
                continue
            factor = scales[i].view(-1, kv)
            # The new tokens, padded to whole blocks of their sequence.
            front, back = lo % BLOCK, -hi % BLOCK
            padded = torch.zeros(front + new[s] + back, kv, D, device="cuda", dtype=torch.float64)
            padded[front:front + new[s]] = mine
            big = padded.abs().view(-1, BLOCK, kv, D).amax(dim=(1, 3))
            want = torch.exp2(torch.ceil(torch.log2(big / CODE_MAX)).clamp(EXP_MIN, EXP_MAX))
            want = torch.where(want < big / CODE_MAX, want * 2, want)     # log2's last bit
            want = torch.where(want / 2 >= big / CODE_MAX, want / 2, want).clamp(
                2.0 ** EXP_MIN, 2.0 ** EXP_MAX)
            heads = slots[::1] // BLOCK
            first = heads[0]
            if front:
                had = factor[first].double()
                want[0] = torch.maximum(want[0], had)
                flat[first * BLOCK:first * BLOCK + front] *= (had / want[0])[None, :, None]
            group = (torch.arange(new[s], device="cuda") + front) // BLOCK
            flat[slots] = mine / want[group][..., None]
            factor[heads] = want[group].float()
        at += new[s]
    if c["cache"] == "bf16":
        return [q, kc, vc]
    return [q, kc, vc, scales[0].double(), scales[1].double()]


def _attend_exact(c, st):
    h, kv = c["heads"], c["kv_heads"]
    g = h // kv
    new, total = _lengths(c)
    if sum(n * t for n, t in zip(new, total)) * h > 3e9:
        return None
    out = torch.zeros(st["tokens"], h, D, device="cuda", dtype=torch.float64)
    at = 0
    for s in range(c["seqs"]):
        lo = max(0, total[s] - new[s] - c["window"] + 1) if c["window"] else 0
        keys = torch.arange(lo, total[s])
        slots = torch.tensor(_token_slots(c, st, s, keys), device="cuda")
        keys = keys.to("cuda")
        where = torch.arange(total[s] - new[s], total[s], device="cuda")
        hide = keys[None] > where[:, None]
        if c["window"]:
            hide |= keys[None] + c["window"] <= where[:, None]
        for n in range(kv):
            def held(name):
                x = st[name + "_cache"]
                if c["cache"] == "bf16":
                    return x.view(-1, kv, D)[slots, n].double()
                x = x.view(torch.float8_e4m3fn).view(-1, kv, D)[slots, n].double()
                return x * st[name + "_scale"].view(-1, kv)[slots // BLOCK, n].double()[:, None]
            k, v = held("k"), held("v")
            for i in range(n * g, n * g + g):
                x = st["q"][at:at + new[s], i].double() @ k.T / math.sqrt(D)
                x = x.masked_fill(hide, -math.inf)
                if c["sinks"]:
                    x = torch.cat([x, st["sink"][i].double().expand(new[s], 1)], 1)
                out[at:at + new[s], i] = torch.softmax(x, 1)[:, :len(slots)] @ v
        at += new[s]
    return out
