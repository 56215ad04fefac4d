"""What is measured of the paged key/value cache and its attention.

Three operators of wht_adapters_amd.whtq over one cache of pages
[pages][kv_heads][page][dim]:

  append  rotary positions on new queries and keys, then keys and values into
          their slots: as they are (16-bit pages), or as INT4 codes of the
          randomized Hadamard transform of each vector with one fp16 scale.
  gather  the keys and values that given slots stand for, as dense rows.
  attend  attention of new tokens (a chunk, or one token) over their
          sequence's pages, with grouped heads, causal or windowed.

`own` False computes them from elementary torch operations in 32 bits.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
DEV = "cuda"


def listed():
    """Head layouts: 32 or 64 query heads of 128 are the 4096- and 8192-wide
    layers of this repository's benchmark, with all or 8 key/value heads."""
    a = dict(op="append", dtype="bf16", fmt="plain", heads=32, kv_heads=8, dim=128, page=16, interleaved=False)
    g = dict(op="gather", dtype="bf16", fmt="int4", kv_heads=8, dim=128, page=16)
    t = dict(op="attend", dtype="bf16", fmt="plain", heads=32, kv_heads=8, dim=128, page=16, causal=True, window=0,
             q_lo=1, q_hi=1)
    return [
        # one sequence produces one token: nothing but latency
        dict(a, name="append_one", tokens=1),
        # a decode step of 61 sequences into the 4-bit cache, read back as its values
        dict(a, name="append_step_int4", tokens=61, heads=64, fmt="int4", page=64),
        # a prompt of 8192 tokens into 16-bit pages
        dict(a, name="append_prompt", tokens=8192),
        # an odd prompt, fp16, small heads, pairs interleaved, into the 4-bit cache and read back
        dict(a, name="append_prompt_int4_f16", tokens=4093, heads=24, kv_heads=24, dim=64, dtype="f16", fmt="int4",
             page=32, interleaved=True),
        # a long prefix taken out of the 4-bit cache
        dict(g, name="gather_prefix_int4", tokens=30011),
        # a few hundred entries of 16-bit pages moved elsewhere
        dict(g, name="gather_some", tokens=333, fmt="plain", dtype="f16", dim=64),
        # one token over a short context: latency
        dict(t, name="attend_one", seqs=1, kv_lo=777, kv_hi=777),
        # a decode step of 64 sequences of very different lengths
        dict(t, name="attend_step", seqs=64, kv_lo=17, kv_hi=8191),
        # decode over two very long contexts held in 4 bits
        dict(t, name="attend_long_int4", seqs=2, heads=64, kv_lo=100003, kv_hi=131072, fmt="int4", page=64),
        # a whole prompt of 8192 tokens, every head its own keys
        dict(t, name="attend_prompt", seqs=1, kv_heads=32, q_lo=8192, q_hi=8192, kv_lo=8192, kv_hi=8192, page=64),
        # a chunk of 512 tokens after a long prefix held in 4 bits
        dict(t, name="attend_chunk_int4", seqs=1, heads=64, q_lo=512, q_hi=512, kv_lo=33000, kv_hi=33000, fmt="int4",
             page=32),
        # odd chunks of six sequences in fp16, small heads, three queries to a key head, a sliding window
        dict(t, name="attend_chunks_window", seqs=6, heads=24, kv_heads=8, dim=64, dtype="f16", q_lo=5, q_hi=1500,
             kv_lo=1601, kv_hi=6007, window=1000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kv_heads, group = rng.choice([(8, 4), (8, 8), (32, 1), (8, 3), (4, 7), (1, 16), (5, 5), (16, 2)])
    c = dict(op=rng.choice(["append", "gather", "attend", "attend"]), dtype=rng.choice(["bf16", "f16"]),
             fmt=rng.choice(["plain", "int4"]), kv_heads=kv_heads, dim=rng.choice([64, 128, 128]),
             page=rng.choice([16, 32, 64, 128]))
    if c["op"] == "gather":
        return dict(c, tokens=_log(rng, 1, 30000))
    c["heads"] = kv_heads * group
    if c["op"] == "append":
        return dict(c, tokens=_log(rng, 1, 8192), interleaved=rng.random() < 0.3)
    c.update(causal=rng.random() < 0.85, window=rng.choice([0, 0, 0, _log(rng, 64, 4096)]))
    kind = rng.choice(["step", "few", "chunk"])
    if kind == "chunk":
        seqs = _log(rng, 1, 8)
        q_hi = _log(rng, 33, 4096 // seqs)
        room = int(5e11 / (4 * c["dim"] * c["heads"] * seqs * q_hi))  # no more work than the largest listed case
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
        w, causal = case["window"], case["causal"]
        first = max(0, kl - ql - w + 1) if w else 0
        keys += kl - first
        if not w and not causal:
            pairs += ql * kl
        elif not w:
            pairs += ql * kl - ql * (ql - 1) // 2
        else:
            for i in range(ql):
                p = kl - ql + i
                pairs += (p + 1 if causal else kl) - max(0, p - w + 1)
    return pairs, keys


def work(case):
    d, hk = case["dim"], case["kv_heads"]
    entry = 2 * hk * (2 * d if case["fmt"] == "plain" else d // 2 + 2)  # a token's key and value in the cache
    dense = 2 * hk * d * 2                                             # the same in 16-bit rows
    if case["op"] == "gather":
        n = case["tokens"]
        return {"bytes": n * (entry + dense + 8), "flops": n * 2 * hk * d * (7 if case["fmt"] == "int4" else 0)}
    if case["op"] == "append":
        n, q = case["tokens"], 2 * case["heads"] * d
        moved = n * (dense + entry + 2 * q + 8 + 4 + 4 * d)
        if case["fmt"] == "int4":
            moved += n * (entry + dense)  # read back
        return {"bytes": moved, "flops": n * (hk + case["heads"]) * 3 * d}
    pairs, keys = _visible(case)
    rows = sum(lengths(case)[0]) * case["heads"] * d * 2
    return {"bytes": 2 * rows + keys * entry, "flops": 4 * d * case["heads"] * pairs}


# ------------------------------------------------------------------ inputs

def _rand(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _pack(c):
    """INT4 codes (whole numbers, last axis even) as bytes, the lower index in the low nibble."""
    c = c.to(torch.int32) & 15
    return (c[..., 0::2] | (c[..., 1::2] << 4)).to(torch.uint8)


def _cache(case, gen, pages):
    """Pages as earlier steps left them: keys with channels of different size, values without."""
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


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    page, d, dt = case["page"], case["dim"], DT[case["dtype"]]
    st = {"case": case}
    if case["op"] == "attend":
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
                  q=_rand(gen, start[-1], case["heads"], d).to(dt), scale=d ** -0.5)
    else:
        n = case["tokens"]
        pages = -(-n // page) + 5
        st["slots"] = torch.randperm(pages * page, generator=gen, device=DEV)[:n].contiguous()
        if n > 64:  # a prompt: runs of whole pages in an order of their own
            order = torch.randperm(pages, generator=gen, device=DEV)[:-(-n // page)]
            st["slots"] = (order[:, None] * page + torch.arange(page, device=DEV)).reshape(-1)[:n].contiguous()
        if case["op"] == "append":
            size = torch.exp(0.4 * _rand(gen, 1, case["kv_heads"], d))
            st["k"] = (_rand(gen, n, case["kv_heads"], d) * size).to(dt)
            st["v"] = _rand(gen, n, case["kv_heads"], d).to(dt)
            st["q"] = _rand(gen, n, case["heads"], d).to(dt)
            top = max(n, 4096)
            angle = torch.arange(top, device=DEV, dtype=torch.float64)[:, None] * 10000.0 ** (
                -torch.arange(0, d, 2, device=DEV, dtype=torch.float64) / d)
            st["cos"], st["sin"] = angle.cos().float(), angle.sin().float()
            st["positions"] = (torch.arange(n, device=DEV, dtype=torch.int32) if n > 64 else
                               torch.randint(0, top, (n,), generator=gen, device=DEV).to(torch.int32))
    st["cache"] = _cache(case, gen, pages)
    if own:
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


def _rotate(x, cos, sin, interleaved):
    x = x.float()
    h = x.shape[-1] // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :h], x[..., h:])
    cos, sin = cos[:, None], sin[:, None]
    u, w = a * cos - b * sin, b * cos + a * sin
    return torch.stack((u, w), -1).flatten(-2) if interleaved else torch.cat((u, w), -1)


def _plain_append(st):
    case, c = st["case"], st["cache"]
    at = st["positions"].long()
    cos, sin = st["cos"][at], st["sin"][at]
    _store(case, c, "k", st["slots"], _rotate(st["k"], cos, sin, case["interleaved"]))
    _store(case, c, "v", st["slots"], st["v"].float())
    q = _rotate(st["q"], cos, sin, case["interleaved"]).to(st["q"].dtype)
    return [q, c["k"], c["v"]] if case["fmt"] == "plain" else [q, *_plain_gather(st)]


def _plain_gather(st):
    case = st["case"]
    page, offset = st["slots"] // case["page"], st["slots"] % case["page"]
    return [_rows(case, st["cache"], name, page, offset).to(DT[case["dtype"]]) for name in ("k", "v")]


def _plain_attend(st):
    case, q = st["case"], st["q"]
    hk, d, n, m, dev = case["kv_heads"], case["dim"], st["max_kv"], st["max_q"], q.device
    j = torch.arange(n, device=dev)
    there = j < st["kv_len"][:, None]                                        # [seqs, keys]
    page = st["table"].long()[:, j // case["page"]]
    k, v = (torch.where(there[:, None, :, None], _rows(case, st["cache"], name, page, j % case["page"]).transpose(1, 2),
                        0.0) for name in ("k", "v"))                         # [seqs, kv_heads, keys, dim]
    start, count = st["q_start"][:-1].long(), st["q_start"][1:].long() - st["q_start"][:-1].long()
    i = torch.arange(m, device=dev)
    take = (start[:, None] + i).clamp_max(q.shape[0] - 1)
    x = q[take].float().reshape(len(start), m, hk, -1, d).permute(0, 2, 3, 1, 4)  # [seqs, kv_heads, group, m, dim]
    s = (x.flatten(2, 3) @ k.transpose(-1, -2)) * st["scale"]
    at = (st["kv_len"].long() - count)[:, None] + i
    see = there[:, None, :]
    if case["causal"]:
        see = see & (j <= at[..., None])
    if case["window"]:
        see = see & (j > at[..., None] - case["window"])
    s = s.unflatten(2, (-1, m)).masked_fill(~see[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).unflatten(2, (-1, m)) / torch.where(total == 0, 1.0, total)
    token = torch.arange(q.shape[0], device=dev)
    b = torch.searchsorted(st["q_start"].long(), token, right=True) - 1
    return o.permute(0, 3, 1, 2, 4)[b, token - start[b]].reshape(q.shape).to(q.dtype)


def run(state):
    case = state["case"]
    if not own:
        return {"append": _plain_append, "gather": _plain_gather, "attend": _plain_attend}[case["op"]](state)
    from wht_adapters_amd import whtq
    cache = state["handle"]
    if case["op"] == "gather":
        return list(whtq.kv_gather(cache, state["slots"], dtype=DT[case["dtype"]]))
    if case["op"] == "append":
        q = whtq.kv_append(cache, state["k"], state["v"], state["slots"], q=state["q"], cos=state["cos"],
                           sin=state["sin"], positions=state["positions"], interleaved=case["interleaved"])
        if case["fmt"] == "plain":
            return [q, cache.k, cache.v]
        return [q, *whtq.kv_gather(cache, state["slots"], dtype=DT[case["dtype"]])]
    return whtq.kv_attention(cache, state["q"], state["q_start"], state["kv_len"], state["table"],
                             max_q_len=state["max_q"], max_kv_len=state["max_kv"], scale=state["scale"],
                             causal=case["causal"], window=case["window"])


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


def _rotate64(x, st):
    d = x.shape[-1]
    at = st["positions"].long()
    cos, sin = st["cos"].double()[at][:, None, :], st["sin"].double()[at][:, None, :]
    first = torch.arange(d // 2, device=x.device)
    first, second = (2 * first, 2 * first + 1) if st["case"]["interleaved"] else (first, first + d // 2)
    y = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    y[..., first] = x.double()[..., first] * cos - x.double()[..., second] * sin
    y[..., second] = x.double()[..., first] * sin + x.double()[..., second] * cos
    return y


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "gather":
        return _entries64(case, st, st["slots"])
    if case["op"] == "append":
        new = [_rotate64(st["k"], st), st["v"].double()]
        q = _rotate64(st["q"], st)
        if case["fmt"] == "plain":
            for x, name in zip(new, ("k", "v")):
                c = st["cache"][name].double()
                rows = c.transpose(1, 2).flatten(0, 1)
                rows[st["slots"]] = x
                new[0 if name == "k" else 1] = rows.unflatten(0, (c.shape[0], c.shape[2])).transpose(1, 2)
            return [q, *new]
        m = _matrix64(case["dim"], st["cache"]["signs"])
        out = []
        for x in new:
            y = x @ m.T
            s = (y.abs().amax(-1, keepdim=True) / 7).to(torch.float16).double()
            out.append((torch.clamp(torch.round(y / s), -7, 7) * s) @ m)
        return [q, *out]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    group, at = case["heads"] // case["kv_heads"], 0
    for b, (ql, kl) in enumerate(zip(*lengths(case))):
        j = torch.arange(kl, device=DEV)
        k, v = _entries64(case, st, st["table"][b].long()[j // case["page"]] * case["page"] + j % case["page"])
        p = kl - ql + torch.arange(ql, device=DEV)[:, None]
        hide = torch.zeros(ql, kl, dtype=torch.bool, device=DEV)
        if case["causal"]:
            hide |= j > p
        if case["window"]:
            hide |= j <= p - case["window"]
        for h in range(case["heads"]):
            s = (st["q"][at:at + ql, h].double() @ k[:, h // group].T) * st["scale"]
            out[at:at + ql, h] = torch.softmax(s.masked_fill(hide, -math.inf), -1) @ v[:, h // group]
        at += ql
    return out
