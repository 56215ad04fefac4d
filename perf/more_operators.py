"""What is measured of the operators around a decode step and an adapter's
training step that wht_adapters_amd.whtq has beside its cache and attention:

  append   norms of each head's queries and keys, rotary positions, then keys
           and values into the slots of a paged cache, 16-bit or INT4.
  norm     the same norms and rotation on dense rows, with their gradients.
  attend   attention of new tokens over their sequence's pages under a sliding
           window with a few first tokens that stay visible.
  logprob  log probabilities of given tokens, the entropy and the likeliest
           tokens of rows of logits; with `grad` the gradient of the logits.

`own` False computes them from elementary torch operations in 32 bits.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
DEV = "cuda"
EPS = 1e-6


def listed():
    """Head layouts: 32 or 64 query heads of 128 are the 4096- and 8192-wide
    layers of this repository's benchmark, with all or 8 key/value heads."""
    a = dict(op="append", dtype="bf16", fmt="plain", heads=32, kv_heads=8, dim=128, page=16, interleaved=False,
             per_head=False)
    n = dict(op="norm", dtype="bf16", heads=32, kv_heads=8, dim=128, interleaved=False, per_head=False)
    t = dict(op="attend", dtype="bf16", fmt="plain", heads=32, kv_heads=8, dim=128, page=16, causal=True, sinks=4,
             q_lo=1, q_hi=1)
    p = dict(op="logprob", dtype="bf16", scale=1.0, top=0, grad=False)
    return [
        # one sequence produces one token: nothing but latency
        dict(a, name="append_one", tokens=1),
        # a decode step of 61 sequences into the 4-bit cache, read back as its values
        dict(a, name="append_step_int4", tokens=61, heads=64, dtype="f16", fmt="int4", page=64),
        # a prompt of 8192 tokens into 16-bit pages
        dict(a, name="append_prompt", tokens=8192),
        # a short odd batch, fp16, small heads, pairs interleaved, a weight for every head
        dict(n, name="norm_odd", tokens=333, heads=24, kv_heads=24, dim=64, dtype="f16", interleaved=True,
             per_head=True),
        # a training batch: four sequences of 2048 tokens
        dict(n, name="norm_train", tokens=8192),
        # one token far into a stream
        dict(t, name="attend_one", seqs=1, kv_lo=50021, kv_hi=50021, window=1024),
        # a decode step of 64 streams of very different lengths
        dict(t, name="attend_step", seqs=64, kv_lo=17, kv_hi=20011, window=4096),
        # a decode step of 16 long streams held in 4 bits, a prefix of 37 tokens kept
        dict(t, name="attend_step_int4", seqs=16, heads=64, kv_lo=8000, kv_hi=65536, fmt="int4", page=64, window=16384,
             sinks=37),
        # a whole prompt of 8192 tokens
        dict(t, name="attend_prompt", seqs=1, q_lo=8192, q_hi=8192, kv_lo=8192, kv_hi=8192, page=64, window=1500),
        # one token's logits, with the alternatives a user is shown
        dict(p, name="logprob_one", rows=1, vocab=131072, top=20, scale=1.25),
        # a long text scored token by token, an odd vocabulary
        dict(p, name="logprob_text", rows=2047, vocab=100003, top=5),
        # a training step's loss with a bonus for entropy, and its gradient
        dict(p, name="logprob_grad", rows=8192, vocab=32000, grad=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kv_heads, group = rng.choice([(8, 4), (8, 8), (32, 1), (8, 3), (4, 7), (1, 16), (5, 5), (16, 2)])
    op = rng.choice(["append", "norm", "attend", "attend", "logprob", "logprob"])
    if op == "logprob":
        grad = rng.random() < 0.5
        vocab = _log(rng, 1000, 262144)
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), scale=rng.choice([1.0, 1.0, 0.7, 1.25]),
                    top=rng.choice([0, 1, 5, 20, 32]), grad=grad, vocab=vocab,
                    rows=_log(rng, 1, max(1, min(8192, 125000000 // vocab))))
    c = dict(op=op, dtype=rng.choice(["bf16", "f16"]), kv_heads=kv_heads, heads=kv_heads * group,
             dim=rng.choice([64, 128, 128]))
    if op in ("append", "norm"):
        c.update(tokens=_log(rng, 1, 8192), interleaved=rng.random() < 0.3, per_head=rng.random() < 0.3)
        return dict(c, fmt=rng.choice(["plain", "int4"]), page=rng.choice([16, 32, 64, 128])) if op == "append" else c
    c.update(fmt=rng.choice(["plain", "int4"]), page=rng.choice([16, 32, 64, 128]), causal=rng.random() < 0.85,
             window=_log(rng, 64, 16384), sinks=rng.choice([1, 4, 4, _log(rng, 2, 256)]))
    kind = rng.choice(["step", "few", "chunk"])
    if kind == "chunk":
        seqs = _log(rng, 1, 8)
        q_hi = _log(rng, 33, 4096 // seqs)
        room = int(1e11 / (4 * c["dim"] * c["heads"] * seqs * q_hi))  # no more work than the largest listed case
        kv_hi = max(q_hi, min(q_hi + _log(rng, 1, 16384), room))
    else:
        seqs = _log(rng, 1, 128)
        q_hi = 1 if kind == "step" else rng.randint(2, 9)
        kv_hi = max(q_hi + 1, _log(rng, 64, 400000 // seqs))
    q_lo = 1 if kind == "step" else rng.randint(1, q_hi)
    return dict(c, seqs=seqs, q_lo=q_lo, q_hi=q_hi, kv_lo=max(q_hi, _log(rng, max(1, kv_hi // 8), kv_hi)), kv_hi=kv_hi)


def _spread(lo, hi, n, turn):
    """n whole numbers from lo to hi, even over the logarithm, in an order of their own."""
    v = [int(round(math.exp(math.log(lo) + (math.log(hi) - math.log(lo)) * (i / max(1, n - 1))))) for i in range(n)]
    v[-1] = hi
    return [v[(i * turn + n // 3) % n] if math.gcd(turn, n) == 1 else v[i] for i in range(n)]


def lengths(case):
    """(new tokens, keys) of each sequence of an attend case."""
    n = case["seqs"]
    q = _spread(case["q_lo"], case["q_hi"], n, 5)
    kv = _spread(case["kv_lo"], case["kv_hi"], n, 7)
    return q, [max(a, b) for a, b in zip(q, kv)]


def _visible(case):
    """Pairs of a query and a key it sees, and keys that any query of their sequence sees."""
    pairs = keys = 0
    for ql, kl in zip(*lengths(case)):
        first = max(0, kl - ql - case["window"] + 1)
        keys += kl - first + min(case["sinks"], first)
        for i in range(ql):
            p = kl - ql + i
            end = p + 1 if case["causal"] else kl
            lo = max(0, p - case["window"] + 1)
            pairs += end - lo + min(case["sinks"], lo)
    return pairs, keys


def work(case):
    if case["op"] == "logprob":
        n, row = case["rows"], case["vocab"] * (4 if case["dtype"] == "f32" else 2)
        # a gradient needs the row's sum first: the logits are read in one pass and once more in the other
        return {"bytes": n * (row * (3 if case["grad"] else 1) + 8 + 12 + case["top"] * 12),
                "flops": n * case["vocab"] * (12 if case["grad"] else 6)}
    d, hk, h = case["dim"], case["kv_heads"], case["heads"]
    if case["op"] == "norm":
        n = case["tokens"]
        row = 2 * (hk + h) * d
        # forward: rows in and out; backward: rows and their gradients in, gradients out
        return {"bytes": n * (5 * row + 4 + 4 * d) + 8 * d * (hk + h if case["per_head"] else 2),
                "flops": n * (hk + h) * 20 * d}
    entry = 2 * hk * (2 * d if case["fmt"] == "plain" else d // 2 + 2)  # a token's key and value in the cache
    dense = 2 * hk * d * 2                                             # the same in 16-bit rows
    if case["op"] == "append":
        n, q = case["tokens"], 2 * h * d
        moved = n * (dense + entry + 2 * q + 8 + 4 + 4 * d)
        if case["fmt"] == "int4":
            moved += n * (entry + dense)  # read back
        return {"bytes": moved, "flops": n * (hk + h) * 7 * d}
    pairs, keys = _visible(case)
    rows = sum(lengths(case)[0]) * h * d * 2
    return {"bytes": 2 * rows + keys * entry, "flops": 4 * d * h * pairs}


# ------------------------------------------------------------------ inputs

def _rand(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _pack(c):
    """INT4 codes (whole numbers, last axis even) as bytes, the lower index in the low nibble."""
    c = c.to(torch.int32) & 15
    return (c[..., 0::2] | (c[..., 1::2] << 4)).to(torch.uint8)


def _cache(case, gen, pages):
    """Pages as earlier steps left them: normed keys with channels of different size, values without."""
    hk, p, d = case["kv_heads"], case["page"], case["dim"]
    if case["fmt"] == "plain":
        size = torch.exp(0.4 * _rand(gen, 1, hk, 1, d))
        return {"k": (_rand(gen, pages, hk, p, d) * size).to(DT[case["dtype"]]),
                "v": _rand(gen, pages, hk, p, d).to(DT[case["dtype"]])}
    c = {}
    for name in ("k", "v"):
        c[name] = _pack(torch.clamp(torch.round(_rand(gen, pages, hk, p, d) * 2.6), -7, 7))
        c[name + "_scales"] = (0.37 * torch.exp(0.2 * _rand(gen, pages, hk, p))).to(torch.float16)
    c["signs"] = torch.randint(-2 ** 31, 2 ** 31, (d // 32,), generator=gen, device=DEV, dtype=torch.int64).to(torch.int32)
    return c


def _prepare_attend(case, gen, st):
    page, d = case["page"], case["dim"]
    ql, kl = lengths(case)
    width = -(-max(kl) // page)
    pages = sum(-(-n // page) for n in kl) + 3
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.zeros((len(kl), width), dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(kl):
        table[b, :-(-n // page)] = order[at:at + -(-n // page)]
        at += -(-n // page)
    start = [0]
    for n in ql:
        start.append(start[-1] + n)
    st.update(table=table, q_start=torch.tensor(start, dtype=torch.int32, device=DEV),
              kv_len=torch.tensor(kl, dtype=torch.int32, device=DEV), max_q=max(ql), max_kv=max(kl),
              q=_rand(gen, start[-1], case["heads"], d).to(DT[case["dtype"]]), scale=d ** -0.5)
    st["cache"] = _cache(case, gen, pages)


def _prepare_rows(case, gen, st):
    n, d, h, hk, dt = case["tokens"], case["dim"], case["heads"], case["kv_heads"], DT[case["dtype"]]
    # queries, keys and values are one projection's output
    size = torch.exp(0.4 * _rand(gen, 1, h + 2 * hk, d)) * torch.exp(0.3 * _rand(gen, n, 1, 1))
    qkv = (_rand(gen, n, h + 2 * hk, d) * size).to(dt)
    st["q"], st["k"], st["v"] = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]
    for name, heads in (("q_norm", h), ("k_norm", hk)):
        st[name] = (1 + 0.3 * _rand(gen, *((heads, d) if case["per_head"] else (d,)))).to(dt)
    top = max(n, 4096)
    angle = torch.arange(top, device=DEV, dtype=torch.float64)[:, None] * 10000.0 ** (
        -torch.arange(0, d, 2, device=DEV, dtype=torch.float64) / d)
    st["cos"], st["sin"] = angle.cos().float(), angle.sin().float()
    st["positions"] = (torch.arange(n, device=DEV, dtype=torch.int32) if n > 64 else
                       torch.randint(0, top, (n,), generator=gen, device=DEV).to(torch.int32))
    if case["op"] == "norm":
        st["dq_out"], st["dk_out"] = (1e-2 * _rand(gen, n, h, d)).to(dt), (1e-2 * _rand(gen, n, hk, d)).to(dt)
        return
    page = case["page"]
    pages = -(-n // page) + 5
    st["slots"] = torch.randperm(pages * page, generator=gen, device=DEV)[:n].contiguous()
    if n > 64:  # a prompt: runs of whole pages in an order of their own
        order = torch.randperm(pages, generator=gen, device=DEV)[:-(-n // page)]
        st["slots"] = (order[:, None] * page + torch.arange(page, device=DEV)).reshape(-1)[:n].contiguous()
    st["cache"] = _cache(case, gen, pages)


def _prepare_logits(case, gen, st):
    n, v = case["rows"], case["vocab"]
    # a model's logits: a few tokens stand out, by as much as the row is sure of itself
    x = 2.0 * _rand(gen, n, v)
    likely = torch.randint(0, v, (n, 8), generator=gen, device=DEV)
    x.scatter_add_(1, likely, 4 + 8 * torch.rand(n, 8, generator=gen, device=DEV))
    x[:, v - 3:] = -math.inf  # the vocabulary's padding
    st["logits"] = x.to(DT[case["dtype"]])
    pick = torch.randint(0, 8, (n, 1), generator=gen, device=DEV)
    sure = torch.rand(n, generator=gen, device=DEV) < 0.6
    st["targets"] = torch.where(sure, likely.gather(1, pick)[:, 0],
                                torch.randint(0, v - 3, (n,), generator=gen, device=DEV)).clamp_max(v - 4)
    if n > 8:
        st["targets"][torch.rand(n, generator=gen, device=DEV) < 0.05] = -1  # padding of the batch
    if case["grad"]:
        st["dlogprob"] = torch.full((n,), -1.0 / n, device=DEV) * (st["targets"] >= 0)
        st["dentropy"] = 0.01 / n * torch.rand(n, generator=gen, device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    st = {"case": case}
    {"attend": _prepare_attend, "logprob": _prepare_logits}.get(case["op"], _prepare_rows)(case, gen, st)
    if own and "cache" in st:
        from wht_adapters_amd import whtq
        st["handle"] = whtq.KVCache(**st["cache"])
    return st


# ------------------------------------------------------------------ the plain form

def _hadamard(d, like):
    i = torch.arange(d, device=like.device)
    x = i[:, None] & i[None, :]
    for s in (8, 4, 2, 1):
        x = x ^ (x >> s)
    return (1 - 2 * (x & 1)).to(like.dtype) / math.sqrt(d)


def _signs(c, like):
    bit = torch.arange(32, device=like.device)
    return (1 - 2 * ((c["signs"][:, None] >> bit) & 1)).reshape(-1).to(like.dtype)


def _rows(case, c, name, page, offset):
    """float32 [..., kv_heads, dim]: what the cache entries at (page, offset) stand for."""
    x = c[name][page, :, offset]
    if case["fmt"] == "plain":
        return x.float()
    x = torch.stack((x & 15, x >> 4), -1).flatten(-2).to(torch.int16)
    y = ((x ^ 8) - 8).float() * c[name + "_scales"][page, :, offset].float()[..., None]
    return (y @ _hadamard(case["dim"], y)) * _signs(c, y)


def _store(case, c, name, slots, x):
    page, offset = slots // case["page"], slots % case["page"]
    if case["fmt"] == "plain":
        c[name][page, :, offset] = x.to(c[name].dtype)
        return
    y = (x * _signs(c, x)) @ _hadamard(case["dim"], x)
    s = (y.abs().amax(-1) / 7).to(torch.float16)
    inv = torch.where(s > 0, 1 / s.float(), torch.zeros_like(s, dtype=torch.float32))
    c[name][page, :, offset] = _pack(torch.clamp(torch.round(y * inv[..., None]), -7, 7))
    c[name + "_scales"][page, :, offset] = s


def _rotate(x, cos, sin, interleaved, back=False):
    h = x.shape[-1] // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :h], x[..., h:])
    cos, sin = cos[:, None], -sin[:, None] if back else sin[:, None]
    u, w = a * cos - b * sin, b * cos + a * sin
    return torch.stack((u, w), -1).flatten(-2) if interleaved else torch.cat((u, w), -1)


def _norm(x, w):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def _tables(st):
    at = st["positions"].long()
    return st["cos"][at], st["sin"][at], st["case"]["interleaved"]


def _plain_append(st):
    case, c = st["case"], st["cache"]
    table = _tables(st)
    _store(case, c, "k", st["slots"], _rotate(_norm(st["k"], st["k_norm"]), *table))
    _store(case, c, "v", st["slots"], st["v"].float())
    q = _rotate(_norm(st["q"], st["q_norm"]), *table).to(st["q"].dtype)
    if case["fmt"] == "plain":
        return [q, c["k"], c["v"]]
    page, offset = st["slots"] // case["page"], st["slots"] % case["page"]
    return [q] + [_rows(case, c, name, page, offset).to(st["q"].dtype) for name in ("k", "v")]


def _plain_norm(st):
    table = _tables(st)
    outs, grads, weights = [], [], []
    for name in ("q", "k"):
        x, w, dy = st[name].float(), st[name + "_norm"].float(), st[f"d{name}_out"].float()
        outs.append(_rotate(_norm(x, w), *table).to(st[name].dtype))
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        g = _rotate(dy, *table, back=True)
        weights.append((g * x * r).sum(0 if w.dim() == 2 else (0, 1)))
        u = g * w
        grads.append((r * (u - x * (r * r * (u * x).mean(-1, keepdim=True)))).to(st[name].dtype))
    return outs + grads + weights


def _plain_attend(st):
    case, q = st["case"], st["q"]
    hk, d, m, dev = case["kv_heads"], case["dim"], st["max_q"], q.device
    window, sinks = case["window"], case["sinks"]
    start, count = st["q_start"][:-1].long(), st["q_start"][1:].long() - st["q_start"][:-1].long()
    kv = st["kv_len"].long()
    # the first keys, and those from the first query's window on
    first = (kv - count - window + 1).clamp_min(0)[:, None]
    far = torch.arange(min(st["max_kv"], window + m - 1), device=dev)
    near = torch.arange(min(sinks, st["max_kv"]), device=dev)
    j = torch.cat((near.expand(len(kv), -1), first + far), 1)                 # [seqs, keys]
    there = j < kv[:, None]
    there[:, len(near):] &= j[:, len(near):] >= sinks                         # not twice
    page = st["table"].long().gather(1, (j // case["page"]).clamp_max(st["table"].shape[1] - 1))
    k, v = (torch.where(there[:, None, :, None], _rows(case, st["cache"], name, page, j % case["page"]).transpose(1, 2),
                        0.0) for name in ("k", "v"))                         # [seqs, kv_heads, keys, dim]
    i = torch.arange(m, device=dev)
    take = (start[:, None] + i).clamp_max(q.shape[0] - 1)
    x = q[take].float().reshape(len(start), m, hk, -1, d).permute(0, 2, 3, 1, 4)  # [seqs, kv_heads, group, m, dim]
    s = (x.flatten(2, 3) @ k.transpose(-1, -2)) * st["scale"]
    at = ((kv - count)[:, None] + i)[..., None]
    jj = j[:, None, :]
    see = there[:, None, :] & ((jj > at - window) | (jj < sinks))
    if case["causal"]:
        see = see & (jj <= at)
    s = s.unflatten(2, (-1, m)).masked_fill(~see[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).unflatten(2, (-1, m)) / torch.where(total == 0, 1.0, total)
    token = torch.arange(q.shape[0], device=dev)
    b = torch.searchsorted(st["q_start"].long(), token, right=True) - 1
    return o.permute(0, 3, 1, 2, 4)[b, token - start[b]].reshape(q.shape).to(q.dtype)


def _plain_logprob(st):
    case, t = st["case"], st["targets"]
    z = st["logits"].float() * case["scale"]
    top = z.amax(-1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(-1, keepdim=True)
    logp = z - top - torch.log(total)
    p = e / total
    entropy = -torch.where(p > 0, p * logp, 0.0).sum(-1)
    given = t >= 0
    out = [torch.where(given, logp.gather(1, t.clamp_min(0)[:, None])[:, 0], 0.0), entropy]
    if case["top"]:
        # the logits' own order (scaling rounds, and would make ties); ties: the lowest index first
        index = torch.sort(st["logits"].float(), dim=-1, descending=True, stable=True).indices[:, :case["top"]]
        out += [logp.gather(1, index), index.contiguous()]
    if case["grad"]:
        g, h = (st["dlogprob"] * given)[:, None], st["dentropy"][:, None]
        dz = torch.where(p > 0, -p * (g + h * (logp + entropy[:, None])), 0.0)
        dz.scatter_add_(1, t.clamp_min(0)[:, None], g)
        out.append((dz * case["scale"]).to(st["logits"].dtype))
    return out


def run(state):
    case = state["case"]
    if not own:
        return {"append": _plain_append, "norm": _plain_norm, "attend": _plain_attend,
                "logprob": _plain_logprob}[case["op"]](state)
    from wht_adapters_amd import whtq
    if case["op"] == "logprob":
        r = whtq.token_logprobs(state["logits"], state["targets"], top=case["top"], scale=case["scale"])
        out = [r.logprob, r.entropy] + ([r.top_logprob, r.top_id] if case["top"] else [])
        if case["grad"]:
            out.append(whtq.token_logprobs_backward(state["logits"], state["targets"], r, state["dlogprob"],
                                                    state["dentropy"], scale=case["scale"]))
        return out
    if case["op"] == "attend":
        return whtq.kv_attention(state["handle"], state["q"], state["q_start"], state["kv_len"], state["table"],
                                 max_q_len=state["max_q"], max_kv_len=state["max_kv"], scale=state["scale"],
                                 causal=case["causal"], window=case["window"], sinks=case["sinks"])
    how = dict(q_norm=state["q_norm"], k_norm=state["k_norm"], norm_eps=EPS, cos=state["cos"], sin=state["sin"],
               positions=state["positions"], interleaved=case["interleaved"])
    if case["op"] == "norm":
        out = whtq.qk_norm_rope(state["q"], state["k"], **how)
        return [*out, *whtq.qk_norm_rope_backward(state["dq_out"], state["dk_out"], state["q"], state["k"], **how)]
    cache = state["handle"]
    q = whtq.kv_append(cache, state["k"], state["v"], state["slots"], q=state["q"], **how)
    if case["fmt"] == "plain":
        return [q, cache.k, cache.v]
    return [q, *whtq.kv_gather(cache, state["slots"], dtype=DT[case["dtype"]])]


# ------------------------------------------------------------------ the definition in 64 bits

def _matrix64(d, signs):
    """Hn S as a product of 2 x 2 blocks: the Kronecker power of [[1, 1], [1, -1]], columns signed."""
    h = torch.ones(1, 1, dtype=torch.float64)
    while h.shape[0] < d:
        h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)), 0)
    words = [int(w) & 0xffffffff for w in signs.cpu()]
    s = torch.tensor([-1.0 if words[i // 32] >> (i % 32) & 1 else 1.0 for i in range(d)], dtype=torch.float64)
    return (h * s / math.sqrt(d)).to(DEV)


def _entries64(case, st, slots):
    """float64 (k, v) [slots, kv_heads, dim] of the cache as it is."""
    out = []
    for name in ("k", "v"):
        x = st["cache"][name].transpose(1, 2).flatten(0, 1)[slots]
        if case["fmt"] == "plain":
            out.append(x.double())
            continue
        low, high = (x % 16).double(), (x // 16).double()
        y = torch.empty(*x.shape[:-1], case["dim"], dtype=torch.float64, device=x.device)
        y[..., 0::2] = torch.where(low > 7, low - 16, low)
        y[..., 1::2] = torch.where(high > 7, high - 16, high)
        s = st["cache"][name + "_scales"].transpose(1, 2).flatten(0, 1)[slots].double()
        out.append((y * s[..., None]) @ _matrix64(case["dim"], st["cache"]["signs"]))
    return out


def _turn64(x, st, way):
    """Every pair turned by its token's angle (way 1) or back (way -1)."""
    d = x.shape[-1]
    at = st["positions"].long()
    cos, sin = st["cos"].double()[at][:, None, :], way * st["sin"].double()[at][:, None, :]
    first = torch.arange(d // 2, device=x.device)
    first, second = (2 * first, 2 * first + 1) if st["case"]["interleaved"] else (first, first + d // 2)
    y = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    y[..., first] = x[..., first] * cos - x[..., second] * sin
    y[..., second] = x[..., first] * sin + x[..., second] * cos
    return y


def _unit64(x):
    return x / torch.sqrt(torch.sum(x ** 2, -1, keepdim=True) / x.shape[-1] + EPS)


def _exact_norm(st):
    outs, grads, weights = [], [], []
    for name in ("q", "k"):
        x, w = st[name].double(), st[name + "_norm"].double()
        n = _unit64(x)
        outs.append(_turn64(n * w, st, 1))
        g = _turn64(st[f"d{name}_out"].double(), st, -1)
        weights.append(torch.sum(g * n, 0) if w.dim() == 2 else torch.sum(g * n, (0, 1)))
        # x = n / r, and n's gradient loses its part along n (but for eps, which n^2 < 1 carries)
        r = 1 / torch.sqrt(torch.sum(x ** 2, -1, keepdim=True) / x.shape[-1] + EPS)
        grads.append(r * (g * w - n * torch.sum(g * w * n, -1, keepdim=True) / x.shape[-1]))
    return outs + grads + weights


def _exact_append(case, st):
    new = [_turn64(_unit64(st["k"].double()) * st["k_norm"].double(), st, 1), st["v"].double()]
    q = _turn64(_unit64(st["q"].double()) * st["q_norm"].double(), st, 1)
    if case["fmt"] == "plain":
        for i, name in enumerate(("k", "v")):
            c = st["cache"][name].double()
            rows = c.transpose(1, 2).flatten(0, 1)
            rows[st["slots"]] = new[i]
            new[i] = rows.unflatten(0, (c.shape[0], c.shape[2])).transpose(1, 2)
        return [q, *new]
    m = _matrix64(case["dim"], st["cache"]["signs"])
    out = []
    for x in new:
        y = x @ m.T
        s = (y.abs().amax(-1, keepdim=True) / 7).to(torch.float16).double()
        out.append((torch.clamp(torch.round(y / s), -7, 7) * s) @ m)
    return [q, *out]


def _exact_attend(case, st):
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    group, at = case["heads"] // case["kv_heads"], 0
    for b, (ql, kl) in enumerate(zip(*lengths(case))):
        first = max(0, kl - ql - case["window"] + 1)
        j = torch.tensor([*range(min(case["sinks"], first)), *range(first, kl)], device=DEV)
        k, v = _entries64(case, st, st["table"][b].long()[j // case["page"]] * case["page"] + j % case["page"])
        p = kl - ql + torch.arange(ql, device=DEV)[:, None]
        hide = (j <= p - case["window"]) & (j >= case["sinks"])
        if case["causal"]:
            hide |= j > p
        for h in range(case["heads"]):
            s = (st["q"][at:at + ql, h].double() @ k[:, h // group].T) * st["scale"]
            out[at:at + ql, h] = torch.softmax(s.masked_fill(hide, -math.inf), -1) @ v[:, h // group]
        at += ql
    return out


def _exact_logprob(case, st):
    n, t = case["rows"], st["targets"]
    some = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device=DEV)
    logprob, entropy = some(n), some(n)
    top = some(n, case["top"])
    ids = torch.zeros(n, case["top"], dtype=torch.int64, device=DEV)
    grad = some(n, case["vocab"]) if case["grad"] else None
    for a in range(0, n, 256):
        part = slice(a, min(n, a + 256))
        z = st["logits"][part].double() * case["scale"]
        logp = z - torch.logsumexp(z, -1, keepdim=True)
        p = torch.softmax(z, -1)
        finite = torch.where(p > 0, logp, 0.0)
        entropy[part] = -torch.sum(p * finite, -1)
        row = torch.arange(z.shape[0], device=DEV)
        given = t[part] >= 0
        logprob[part] = torch.where(given, logp[row, t[part].clamp_min(0)], 0.0)
        if case["top"]:
            order = torch.argsort(z, dim=-1, descending=True, stable=True)[:, :case["top"]]
            ids[part], top[part] = order, logp.gather(1, order)
        if case["grad"]:
            g = torch.where(given, st["dlogprob"][part].double(), 0.0)[:, None]
            h = st["dentropy"][part].double()[:, None]
            d = -g * p - h * p * (finite + entropy[part][:, None])
            d[row, t[part].clamp_min(0)] += g[:, 0]
            grad[part] = d * case["scale"]
    return [logprob, entropy] + ([top, ids] if case["top"] else []) + ([grad] if case["grad"] else [])


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "logprob":
        return _exact_logprob(case, st)
    if case["op"] == "norm":
        return _exact_norm(st)
    return _exact_append(case, st) if case["op"] == "append" else _exact_attend(case, st)
