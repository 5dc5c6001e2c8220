"""What is measured of the linear side of a prompt: a matrix product with bias,
activation and residual in its epilogue (projections around the attention, a
dense MLP, router scores), the same grouped by expert with ragged group sizes,
the selection of each token's experts with the rows' order by expert, the
weighted sum of the experts' rows, and the mixture-of-experts layer of many
tokens made of them.

A case is one call.
  linear   out = act(x w^T + bias) + residual; x [rows, n_in]; with act "swiglu"
           w holds n_out gate rows and n_out up rows and out is silu(gate) * up.
  grouped  row r of group g: act(w[g] x[index[r]] + bias[g]), rows in group order.
  select   top 6 of 256 sigmoid scores, ties to the lower index, weights
           renormalised, and a stable order of all (token, slot) pairs by expert.
  combine  residual + shared + sum of a token's 6 expert rows times their weights.
  layer    router, select, gate/up, down, shared expert and combine.
"""
import math
import random

import torch

own = False

H, E, K, I = 2048, 256, 6, 512    # the layer: hidden, experts, experts a token, expert width
ACTS = ("none", "silu", "gelu", "swiglu")
GAP = 1e-4    # the layer's tokens have router scores whose order 32 bits settle


def listed():
    lin = dict(op="linear", act="none", bias=False, residual=False, out="bf16")
    return [
        # One user's next token into query, key and value heads: latency, the weights read once.
        dict(lin, name="linear 1 token", rows=1, n_in=2048, n_out=5120),
        # Drafts of a few users back from the attention into the residual stream.
        dict(lin, name="linear 33 rows residual", rows=33, n_in=4096, n_out=2048, bias=True,
             residual=True),
        # Router scores of a prompt: few outputs, kept in 32 bits.
        dict(lin, name="linear 4001 rows f32", rows=4001, n_in=2048, n_out=256, out="f32"),
        # The gate and up projection of a dense layer over the largest chunk of a prompt.
        dict(lin, name="linear 8192 rows swiglu", rows=8192, n_in=2048, n_out=4096, act="swiglu",
             bias=True),
        # The experts' down projection for 700 tokens of a short prompt: most of all experts, few rows each.
        dict(op="grouped", name="grouped 4200 rows down", groups=E, rows=4200, n_x=4200, n_in=I,
             n_out=H, act="none", bias=False, gather=False, spread=0.5),
        # Gate and up projections of a full chunk, rows gathered from the tokens.
        dict(op="grouped", name="grouped 49152 rows gate/up", groups=E, rows=8192 * K, n_x=8192,
             n_in=H, n_out=I, act="swiglu", bias=False, gather=True, spread=0.5),
        # A few prompts' last tokens, offsets that steer the choice only.
        dict(op="select", name="select 17 tokens", tokens=17, offsets="select"),
        # A full chunk.
        dict(op="select", name="select 8192 tokens", tokens=8192, offsets="logit"),
        # A short prompt's rows back together.
        dict(op="combine", name="combine 40 tokens", tokens=40, shared=True),
        # A full chunk, one token short.
        dict(op="combine", name="combine 8191 tokens", tokens=8191, shared=True),
        # A short prompt through the layer, some experts preferred.
        dict(op="layer", name="layer 300 tokens", tokens=300, offsets="logit"),
        # A full chunk through the layer.
        dict(op="layer", name="layer 8192 tokens", tokens=8192, offsets="none"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "grouped", "grouped", "select", "combine", "layer"])
    if op == "linear":
        while True:
            c = dict(op=op, rows=_log(rng, 1, 8192), n_in=8 * _log(rng, 8, 1024),
                     n_out=16 * _log(rng, 4, 512), act=rng.choice(ACTS), bias=rng.random() < 0.5,
                     residual=rng.random() < 0.5, out="f32" if rng.random() < 0.25 else "bf16")
            if work(c)["flops"] <= 2.7e11 and work(c)["bytes"] <= 1.4e9:
                return c
    if op == "grouped":
        while True:
            rows, gather = _log(rng, 1, 49152), rng.random() < 0.5
            c = dict(op=op, groups=_log(rng, 1, 256), rows=rows, gather=gather,
                     n_x=_log(rng, 1, 8192) if gather else rows, n_in=8 * _log(rng, 8, 512),
                     n_out=16 * _log(rng, 4, 256), act=rng.choice(("none", "swiglu")),
                     bias=rng.random() < 0.3, spread=rng.choice((0.0, 0.5, 1.0)))
            if work(c)["flops"] <= 2.0e11 and work(c)["bytes"] <= 1.4e9:
                return c
    return dict(op=op, tokens=_log(rng, 1, 8192), offsets=rng.choice(("none", "logit", "select")),
                shared=rng.random() < 0.8)


def _sizes(c):
    """Rows of each group: the case's own, whatever the seed; some groups have none."""
    rng = random.Random("%(groups)d %(rows)d %(n_in)d" % c)
    share = [math.exp(rng.gauss(0, c["spread"])) for _ in range(c["groups"])]
    most = 6 * -(-c["rows"] // c["groups"])
    sizes = [min(most, int(c["rows"] * s / sum(share))) for s in share]
    while sum(sizes) < c["rows"]:
        i = rng.randrange(c["groups"])
        sizes[i] += min(c["rows"] - sum(sizes), 1 + most // 16)
    return sizes


def work(c):
    if c["op"] == "linear":
        n2 = c["n_out"] * (2 if c["act"] == "swiglu" else 1)
        size = 4 if c["out"] == "f32" else 2
        return {"bytes": 2 * (c["rows"] + n2) * c["n_in"] + 4 * n2 * c["bias"] +
                c["rows"] * c["n_out"] * size * (2 if c["residual"] else 1),
                "flops": 2 * c["rows"] * n2 * c["n_in"]}
    if c["op"] == "grouped":
        n2 = c["n_out"] * (2 if c["act"] == "swiglu" else 1)
        used = sum(1 for n in _sizes(c) if n)
        return {"bytes": 2 * used * n2 * c["n_in"] + 2 * min(c["n_x"], c["rows"]) * c["n_in"] +
                2 * c["rows"] * c["n_out"] + 4 * used * n2 * c["bias"] + 4 * c["rows"] * c["gather"],
                "flops": 2 * c["rows"] * n2 * c["n_in"]}
    t = c["tokens"]
    if c["op"] == "select":
        return {"bytes": t * E * 4 + t * K * 16 + 4 * (E + 1), "flops": t * E}
    if c["op"] == "combine":
        return {"bytes": t * H * 2 * (K + 2 + c["shared"]) + t * K * 8, "flops": 2 * t * H * (K + 1)}
    used = E * (1 - (1 - K / E) ** t)    # experts that some token chooses, on average
    return {"bytes": 2 * E * H + (used + 1) * 6 * I * H + t * H * 2 * 3 + t * K * 8,
            "flops": 2 * t * H * E + 2 * t * (K + 1) * 3 * H * I}


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(int(seed))
    randn = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    bf = lambda *s: torch.randn(s, generator=g, device=dev, dtype=torch.bfloat16)  # noqa: E731
    st = dict(c)
    op = c["op"]
    if op in ("linear", "grouped"):
        n2 = c["n_out"] * (2 if c["act"] == "swiglu" else 1)
        lead = (c["groups"],) if op == "grouped" else ()
        st["x"] = bf(c["n_x"] if op == "grouped" else c["rows"], c["n_in"])
        st["w"] = bf(*lead, n2, c["n_in"]).mul_(c["n_in"] ** -0.5)
        st["bias_v"] = 0.5 * randn(*lead, n2) if c["bias"] else None
        f32 = c.get("out") == "f32"
        st["out_v"] = torch.zeros(c["rows"], c["n_out"], device=dev,
                                  dtype=torch.float32 if f32 else torch.bfloat16)
    if op == "linear":
        st["residual_v"] = None
        if c["residual"]:
            r = randn(c["rows"], c["n_out"])
            st["residual_v"] = r if f32 else r.to(torch.bfloat16)
    elif op == "grouped":
        sizes = torch.tensor(_sizes(c), device=dev)
        st["start"] = torch.cat([sizes.new_zeros(1), sizes.cumsum(0)]).to(torch.int32)
        st["cap"] = max(_sizes(c))
        st["index"] = (torch.randint(0, c["n_x"], (c["rows"],), generator=g, device=dev,
                                     dtype=torch.int32) if c["gather"] else None)
    else:
        t = c["tokens"]
        offsets = c.get("offsets", "none")
        st["offset_v"] = 0.5 * randn(E) if offsets != "none" else None
        if op == "select":
            # scores on bf16's grid, so that some are equal
            st["logits"] = (0.9 * randn(t, E)).to(torch.bfloat16).float()
            if st["offset_v"] is not None:
                st["offset_v"] = st["offset_v"].to(torch.bfloat16).float()
            i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)  # noqa: E731
            st.update(idx=i32(t, K), weight=torch.zeros(t, K, device=dev), start=i32(E + 1),
                      row_token=i32(t * K), pair_row=i32(t, K))
        elif op == "combine":
            st["residual"], st["y"] = bf(t, H), bf(t * K, H).mul_(0.25)
            st["y_shared"] = bf(t, H).mul_(0.25) if c["shared"] else None
            w = torch.sigmoid(randn(t, K))
            st["weight"] = w / w.sum(1, keepdim=True)
            st["pair_row"] = torch.randperm(t * K, generator=g, device=dev).to(torch.int32).view(t, K)
        else:
            st["wr"] = bf(E, H).mul_(0.02)
            st["w13"], st["w2"] = bf(E, 2 * I, H).mul_(0.02), bf(E, H, I).mul_(0.02)
            st["ws13"], st["ws2"] = bf(1, 2 * I, H).mul_(0.02), bf(1, H, I).mul_(0.02)
            # tokens whose 7 highest scores lie apart, of some more than needed
            more = randn(t + t // 8 + 64, H)
            rows = more / more.square().mean(1, keepdim=True).sqrt()
            score = rows.to(torch.bfloat16).double() @ st["wr"].double().T
            if st["offset_v"] is not None:
                score = score + st["offset_v"].double()
            top = score.topk(K + 1, dim=1)
            keep = (top.values[:, :-1] - top.values[:, 1:]).amin(1) > GAP
            order = (~keep).to(torch.int8).argsort(stable=True)[:t]
            st["x"], st["residual"] = rows[order].to(torch.bfloat16), more[order].to(torch.bfloat16)
            st["cap"] = int(top.indices[order, :K].flatten().bincount(minlength=E).max())
        st["out_v"] = torch.zeros(t, H, dtype=torch.bfloat16, device=dev)
    if own:
        import moe_decode_sigmoid_gb300 as m
        st["workspace"] = m.new_prompt_workspace(c["tokens"] if op == "layer" else 0)
        st["act_v"] = {"none": m.FLINT_ACT_NONE, "silu": m.FLINT_ACT_SILU, "gelu": m.FLINT_ACT_GELU,
                       "swiglu": m.FLINT_ACT_SWIGLU}[c.get("act", "none")]
        st["dims"] = m.SELECT_DIMS if c.get("offsets") == "select" else m.FULL_DIMS
        if op == "layer":
            st["idx"] = torch.zeros(c["tokens"], K, dtype=torch.int32, device=dev)
            st["weight"] = torch.zeros(c["tokens"], K, device=dev)
    return st


def run(st):
    op = st["op"]
    if own:
        import moe_decode_sigmoid_gb300 as m
        if op == "linear":
            m.flint_linear_bf16(st["x"], st["w"], st["out_v"], st["workspace"], bias=st["bias_v"],
                                residual=st["residual_v"], act=st["act_v"])
            return st["out_v"]
        if op == "grouped":
            m.flint_grouped_linear_bf16(st["x"], st["w"], st["start"], st["out_v"], st["workspace"],
                                        row_index=st["index"], bias=st["bias_v"], act=st["act_v"])
            return st["out_v"]
        if op == "select":
            m.flint_moe_select(st["logits"], st["offset_v"], st["idx"], st["weight"], st["start"],
                               st["row_token"], st["pair_row"], st["workspace"], dims=st["dims"])
            return [st[k] for k in ("idx", "weight", "start", "row_token", "pair_row")]
        if op == "combine":
            m.flint_moe_combine_bf16(st["residual"], st["y"], st["pair_row"], st["weight"],
                                     st["y_shared"], st["out_v"])
            return st["out_v"]
        m.flint_moe_prompt_bf16(st["x"], st["residual"], st["wr"], st["offset_v"], st["w13"],
                                st["w2"], st["ws13"], st["ws2"], st["out_v"], st["workspace"],
                                st["idx"], st["weight"], dims=st["dims"])
        return [st["out_v"], st["idx"], st["weight"]]

    if op == "linear":
        y = _act(st["x"].float() @ st["w"].float().T, st["bias_v"], st["act"])
        if st["residual_v"] is not None:
            y = y + st["residual_v"].float()
        return y.to(st["out_v"].dtype)
    if op == "grouped":
        rows = st["x"].float()
        if st["index"] is not None:
            rows = rows[st["index"].long()]
        bias = None if st["bias_v"] is None else st["bias_v"][:, None]
        return _by_group(rows, st["start"].long(), st["cap"],
                         lambda x: _act(torch.bmm(x, st["w"].float().transpose(1, 2)), bias,
                                        st["act"])).to(torch.bfloat16)
    if op == "select":
        idx, weight = _choose(st["logits"], st["offset_v"], st["offsets"])
        start, row_token, pair_row = _order(idx)
        return [idx.to(torch.int32), weight, start.to(torch.int32), row_token.to(torch.int32),
                pair_row.to(torch.int32)]
    if op == "combine":
        y = st["y"].float()[st["pair_row"].long()]
        out = st["residual"].float() + (st["weight"][..., None] * y).sum(1)
        if st["y_shared"] is not None:
            out = out + st["y_shared"].float()
        return out.to(torch.bfloat16)
    x = st["x"].float()
    idx, weight = _choose(x @ st["wr"].float().T, st["offset_v"], st["offsets"])
    start, row_token, pair_row = _order(idx)
    w13, w2 = st["w13"].float().transpose(1, 2), st["w2"].float().transpose(1, 2)
    y = _by_group(x[row_token], start, st["cap"],
                  lambda r: torch.bmm(_act(torch.bmm(r, w13), None, "swiglu"), w2))
    shared = _act(x @ st["ws13"][0].float().T, None, "swiglu") @ st["ws2"][0].float().T
    out = st["residual"].float() + shared + (weight[..., None] * y[pair_row]).sum(1)
    return [out.to(torch.bfloat16), idx.to(torch.int32), weight]


def _act(y, bias, act):
    if bias is not None:
        y = y + bias
    if act == "swiglu":
        gate, up = y.chunk(2, dim=-1)
        return gate / (1 + torch.exp(-gate)) * up
    if act == "silu":
        return y / (1 + torch.exp(-y))
    if act == "gelu":
        return 0.5 * y * (1 + torch.erf(y * 0.5 ** 0.5))
    return y


def _by_group(rows, start, cap, f):
    """f of the rows in groups, each padded to `cap` rows, back in the rows' order."""
    at = start[:-1, None] + torch.arange(cap, device=rows.device)
    padded = f(rows[at.clamp(max=rows.shape[0] - 1)])
    r = torch.arange(rows.shape[0], device=rows.device)
    group = torch.searchsorted(start, r, right=True) - 1
    return padded[group, r - start[group]]


def _choose(logits, offset, mode):
    key = logits if offset is None else logits + offset
    idx = key.sort(dim=1, descending=True, stable=True).indices[:, :K]
    s = torch.sigmoid((logits if mode == "select" else key).gather(1, idx))
    return idx, s / s.sum(1, keepdim=True)


def _order(idx):
    """(first row of each expert, token of each row, row of each pair)."""
    flat = idx.flatten()
    pair = flat.argsort(stable=True)
    count = torch.zeros(E, dtype=torch.int64, device=idx.device).scatter_add_(
        0, flat, torch.ones_like(flat))
    row = torch.empty_like(pair)
    row[pair] = torch.arange(pair.numel(), device=idx.device)
    return torch.cat([count.new_zeros(1), count.cumsum(0)]), pair // K, row.view(idx.shape)


def exact(c, seed):
    st = prepare(c, seed)
    f64 = lambda k: None if st[k] is None else st[k].double()  # noqa: E731
    op = c["op"]
    if op == "linear":
        y = _value(st["x"].double().mm(st["w"].double().t()), f64("bias_v"), c["act"])
        return y if st["residual_v"] is None else y.add_(st["residual_v"].double())
    if op == "grouped":
        out = torch.empty(c["rows"], c["n_out"], dtype=torch.float64, device="cuda")
        at = 0
        for i, n in enumerate(_sizes(c)):
            x = st["x"][at:at + n] if st["index"] is None else st["x"][st["index"][at:at + n].long()]
            bias = None if st["bias_v"] is None else st["bias_v"][i].double()
            out[at:at + n] = _value(x.double().mm(st["w"][i].double().t()), bias, c["act"])
            at += n
        return out
    if op == "select":
        return [None, _weights(f64("logits"), f64("offset_v"), c["offsets"])[1], None, None, None]
    if op == "combine":
        out = f64("residual")
        for j in range(K):
            out += st["weight"][:, j:j + 1].double() * st["y"][st["pair_row"][:, j].long()].double()
        return out if st["y_shared"] is None else out + f64("y_shared")
    x = f64("x")
    idx, weight = _weights(x.mm(st["wr"].double().t()), f64("offset_v"), c["offsets"])
    out = f64("residual") + _value(x.mm(st["ws13"][0].double().t()), None, "swiglu").mm(
        st["ws2"][0].double().t())
    for e in range(E):
        tok, slot = (idx == e).nonzero(as_tuple=True)
        h = _value(x[tok].mm(st["w13"][e].double().t()), None, "swiglu")
        out.index_add_(0, tok, weight[tok, slot, None] * h.mm(st["w2"][e].double().t()))
    return [out, None, weight]


def _value(y, bias, act):
    y = y if bias is None else y + bias
    if act == "swiglu":
        n = y.shape[1] // 2
        return y[:, :n] * torch.sigmoid(y[:, :n]) * y[:, n:]
    if act == "silu":
        return y * torch.sigmoid(y)
    if act == "gelu":
        return y * torch.special.ndtr(y)
    return y


def _weights(score, offset, mode):
    key = score if offset is None else score + offset
    # Equal keys: the lower index first, by a rank of both.
    order = torch.argsort(-key, dim=1, stable=True)[:, :K]
    s = torch.sigmoid(torch.gather(score if mode == "select" else key, 1, order))
    return order, s / s.sum(1, keepdim=True)
