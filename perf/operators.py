"""The decode step's operators around the projections, as measured calls: attention
over the K/V caches (attn_decode), eviction from them by accumulated attention
weight (kv_evict) and sampling from the head's logits (head_sample).

`run` computes an operator in plain torch operations, or through the library's
entry points where `own` is true, on the state that `prepare` makes.
"""
import math

import torch

own = False   # run the library's entry points instead of the plain forms

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}

# ------------------------------------------------------------------- cases


def listed():
    return [
        # one user, a short conversation: the launch's latency
        dict(name="attn-one-short", op="attn", rows=1, heads=32, kv_heads=8, dim=128, n_pos=4096,
             len_max=613, len_min=613, window=-1, sinks=0, kv="f32", acc=False),
        # one user, a document of 128 K tokens, the weights accumulated for an eviction
        dict(name="attn-one-long", op="attn", rows=1, heads=32, kv_heads=8, dim=128, n_pos=131072,
             len_max=130001, len_min=130001, window=-1, sinks=0, kv="bf16", acc=True),
        # a ragged batch under a sliding window with four sinks, caches as the projection writes them
        dict(name="attn-batch-window", op="attn", rows=16, heads=32, kv_heads=8, dim=128, n_pos=8192,
             len_max=8192, len_min=37, window=2048, sinks=4, kv="f32", acc=False),
        # odd sizes: seven query heads a K/V head, 64 values a head, a ragged window
        dict(name="attn-odd", op="attn", rows=5, heads=14, kv_heads=2, dim=64, n_pos=5001,
             len_max=5001, len_min=1, window=1001, sinks=3, kv="f16", acc=True),
        # a full serving batch with every token visible
        dict(name="attn-batch-full", op="attn", rows=64, heads=32, kv_heads=8, dim=128, n_pos=8192,
             len_max=8192, len_min=4100, window=-1, sinks=0, kv="bf16", acc=False),
        # one user's cache of 4096 halved
        dict(name="evict-one", op="evict", rows=1, kv_heads=8, dim=128, n_pos=4096, len_max=4096,
             len_min=4096, budget=2048, sinks=4, recent=256, kv="f32"),
        # a batch of 16 at 8192, some sequences still under the budget
        dict(name="evict-batch", op="evict", rows=16, kv_heads=8, dim=128, n_pos=8192, len_max=8192,
             len_min=2000, budget=4096, sinks=4, recent=512, kv="bf16"),
        # long caches, a quarter of each evicted
        dict(name="evict-long", op="evict", rows=4, kv_heads=8, dim=128, n_pos=32768, len_max=32768,
             len_min=32001, budget=24576, sinks=16, recent=1024, kv="f32"),
        # a small vocabulary, odd, three users
        dict(name="sample-small", op="sample", rows=3, vocab=1001, top_k=40, top_p=0.9, min_p=0.02,
             spread=2.0),
        # one user, the full head, every filter on
        dict(name="sample-one", op="sample", rows=1, vocab=128256, top_k=50, top_p=0.95, min_p=0.05,
             spread=3.0),
        # a serving batch, the nucleus alone (most tokens near its border)
        dict(name="sample-batch-nucleus", op="sample", rows=64, vocab=128256, top_k=0, top_p=0.9,
             min_p=0.0, spread=2.0),
        # the largest batch on a smaller odd vocabulary, users with different settings
        dict(name="sample-batch-mixed", op="sample", rows=256, vocab=32003, top_k=-1, top_p=-1.0,
             min_p=-1.0, spread=3.0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "evict", "sample"])
    if op == "sample":
        rows = _log_int(rng, 1, 256)
        vocab = min(_log_int(rng, 100, 200000), (64 * 128256) // rows)
        mixed = rng.random() < 0.4
        return dict(op=op, rows=rows, vocab=vocab,
                    top_k=-1 if mixed else rng.choice([0, _log_int(rng, 1, 2000)]),
                    top_p=-1.0 if mixed else rng.choice([1.0, round(rng.uniform(0.3, 0.99), 3)]),
                    min_p=-1.0 if mixed else rng.choice([0.0, round(rng.uniform(0.001, 0.2), 3)]),
                    spread=round(rng.uniform(1.0, 4.0), 2))
    rows = _log_int(rng, 1, 64)
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    dim = rng.choice([64, 80, 96, 128, 256])
    kv = rng.choice(["f32", "f16", "bf16"])
    # caches of at most 64 x 8192 x 1024 values of 16 bits, or half as many of 32
    room = (64 * 8192 * 1024 * 2 // BYTES[kv]) // (rows * kv_heads * dim)
    if op == "attn":
        group = rng.choice([1, 2, 3, 4, 6, 7, 8])
        n_pos = _log_int(rng, 64, max(65, min(131072, room // (2 if group <= 4 else 4))))
        window = -1 if rng.random() < 0.4 else _log_int(rng, 1, n_pos)
        return dict(op=op, rows=rows, heads=kv_heads * group, kv_heads=kv_heads, dim=dim, n_pos=n_pos,
                    len_max=max(1, n_pos - rng.randrange(0, 1 + n_pos // 4)),
                    len_min=_log_int(rng, 1, max(2, n_pos // 2)), window=window,
                    sinks=0 if window < 0 else rng.choice([0, 1, 4, 13]), kv=kv,
                    acc=rng.random() < 0.5)
    n_pos = _log_int(rng, 256, max(257, min(65536, room // 4)))
    budget = max(64, int(n_pos * rng.uniform(0.3, 0.9)))
    return dict(op=op, rows=rows, kv_heads=kv_heads, dim=dim, n_pos=n_pos, len_max=n_pos,
                len_min=max(1, int(n_pos * rng.uniform(0.2, 1.0))), budget=budget,
                sinks=rng.choice([0, 1, 4, 16]), recent=rng.choice([1, budget // 8, budget // 4]), kv=kv)


def _lens(case):
    """The rows' lengths: from len_max down to len_min, in an order that mixes long and short."""
    rows, hi, lo = case["rows"], max(case["len_max"], case["len_min"]), min(case["len_max"], case["len_min"])
    if rows == 1:
        return [hi]
    lens = [hi - (hi - lo) * i // (rows - 1) for i in range(rows)]
    return [lens[(i * 7) % rows] for i in range(rows)] if rows % 7 else lens


def _visible(case, n):
    if case["window"] < 0:
        return n
    return min(n, min(case["sinks"], n) + case["window"])


def work(case):
    if case["op"] == "attn":
        vis = sum(_visible(case, n) for n in _lens(case))
        kv_dim = case["kv_heads"] * case["dim"]
        nbytes = 2 * vis * kv_dim * BYTES[case["kv"]] + 8 * case["rows"] * case["heads"] * case["dim"]
        nbytes += 8 * vis * case["kv_heads"] if case["acc"] else 0
        return {"bytes": nbytes, "flops": 4 * vis * case["heads"] * case["dim"]}
    if case["op"] == "evict":
        # each kept entry behind the sinks is read and written in K and in V
        full = sum(n > case["budget"] for n in _lens(case))
        moved = full * (case["budget"] - case["sinks"]) * case["kv_heads"]
        nbytes = 4 * moved * case["dim"] * BYTES[case["kv"]]
        nbytes += 4 * case["rows"] * case["kv_heads"] * (2 * case["n_pos"] + case["budget"])
        return {"bytes": nbytes, "flops": case["rows"] * case["kv_heads"] * case["n_pos"]}
    n = case["rows"] * case["vocab"]
    return {"bytes": 4 * n, "flops": 4 * n}


# ------------------------------------------------------------------ inputs


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    rows = case["rows"]
    if case["op"] == "sample":
        # a head's logits: a bell of the given spread and a few tokens that stand out
        n = case["vocab"]
        x = torch.randn(rows, n, generator=g, device=DEV) * case["spread"]
        hot = torch.randint(0, n, (rows, 8), generator=g, device=DEV)
        lift = torch.rand(rows, n, generator=g, device=DEV) * 6
        x += lift * torch.zeros_like(x).scatter_(1, hot, 1.0)
        r = torch.rand(4, rows, generator=g, device=DEV)
        temp = 0.5 + r[0]
        top_k = torch.full((rows,), case["top_k"], dtype=torch.int32, device=DEV)
        top_p = torch.full((rows,), case["top_p"], device=DEV)
        min_p = torch.full((rows,), case["min_p"], device=DEV)
        if case["top_k"] < 0:   # users with settings of their own, some of them greedy
            i = torch.arange(rows, device=DEV)
            top_k = torch.where(i % 3 == 0, (1 + r[1] * 300).to(torch.int32), 0).to(torch.int32)
            top_p = torch.where(i % 4 < 2, 0.3 + 0.69 * r[2], 1.0)
            min_p = torch.where(i % 5 == 0, 0.1 * r[3], 0.0)
            temp = torch.where(i % 16 == 7, 0.0, temp)
        return dict(case=case, x=x, u=torch.rand(rows, generator=g, device=DEV), temp=temp, top_k=top_k,
                    top_p=top_p, min_p=min_p, tok=torch.zeros(rows, dtype=torch.int32, device=DEV),
                    prob=torch.zeros(rows, device=DEV),
                    kept=torch.zeros(rows, dtype=torch.int32, device=DEV))
    n_pos, kvh, dim, dt = case["n_pos"], case["kv_heads"], case["dim"], TYPES[case["kv"]]
    pos = torch.tensor(_lens(case), dtype=torch.int32, device=DEV) - 1
    k = torch.empty(rows, n_pos, kvh * dim, dtype=dt, device=DEV).normal_(generator=g)
    v = torch.empty(rows, n_pos, kvh * dim, dtype=dt, device=DEV).normal_(generator=g)
    # accumulated weights: a heavy tail, as attention leaves them, and some never attended
    a = torch.empty(rows, kvh, n_pos, device=DEV).normal_(generator=g).mul_(2).sub_(4).exp_()
    a.masked_fill_(a < 1e-3, 0.0)
    state = dict(case=case, k=k, v=v, pos=pos, acc=a)
    if case["op"] == "attn":
        # q is the first part of the fused QKV projection's output rows
        qkv = torch.randn(rows, (case["heads"] + 2 * kvh) * dim, generator=g, device=DEV) * 1.5
        state.update(qkv=qkv, out=torch.zeros(rows, case["heads"] * dim, device=DEV))
        if case["acc"]:
            # weights accumulated over a few steps only, so that this step's weigh in them
            a.mul_(1e-3)
    else:
        state.update(new_pos=torch.zeros_like(pos), new_acc=torch.zeros_like(a),
                     kept=torch.zeros(rows, kvh, case["budget"], dtype=torch.int32, device=DEV))
    return state


# ---------------------------------------------------------------- passes

_ws = [None]


def _workspace(nbytes):
    """One zeroed workspace for every call, as a serving program keeps it."""
    if _ws[0] is None or _ws[0].numel() < nbytes:
        _ws[0] = torch.zeros(nbytes, dtype=torch.uint8, device=DEV)
    return _ws[0]


def run(state):
    op = state["case"]["op"]
    if op == "attn":
        return _attn_own(state) if own else _attn_plain(state)
    if op == "evict":
        return _evict_own(state) if own else _evict_plain(state)
    return _sample_own(state) if own else _sample_plain(state)


def _attn_own(s):
    from q8_quantized_projection_gb300 import native
    c = s["case"]
    nbytes = native.attn_decode_workspace(c["rows"], c["heads"], c["kv_heads"], c["dim"], c["n_pos"],
                                          window=c["window"], sinks=c["sinks"], acc=c["acc"])
    native.attn_decode(s["qkv"], s["k"], s["v"], s["pos"], s["out"], _workspace(nbytes),
                       heads=c["heads"], kv_heads=c["kv_heads"], window=c["window"], sinks=c["sinks"],
                       acc=s["acc"] if c["acc"] else None)
    return [s["out"], s["acc"]] if c["acc"] else [s["out"]]


def _attn_plain(s):
    c = s["case"]
    rows, kvh, dim = c["rows"], c["kv_heads"], c["dim"]
    group = c["heads"] // kvh
    q = s["qkv"][:, :c["heads"] * dim].reshape(rows, kvh, group, dim)
    k = s["k"].view(rows, -1, kvh, dim).permute(0, 2, 3, 1).float()
    v = s["v"].view(rows, -1, kvh, dim).permute(0, 2, 1, 3).float()
    i, pos = torch.arange(c["n_pos"], device=DEV), s["pos"].long()[:, None]
    vis = i <= pos
    if c["window"] >= 0:
        vis = vis & ((i < c["sinks"]) | (i > pos - c["window"]))
    vis = vis[:, None, None, :]
    score = torch.matmul(q * (1.0 / math.sqrt(dim)), k).masked_fill(~vis, -math.inf)
    top = score.amax(-1, keepdim=True)
    w = torch.where(vis, torch.exp(score - torch.where(top == -math.inf, 0.0, top)), 0.0)
    total = w.sum(-1, keepdim=True)
    w = torch.where(total == 0, 0.0, w / total)
    out = torch.matmul(w, v).reshape(rows, c["heads"] * dim)
    if not c["acc"]:
        return [out]
    s["acc"] += w.sum(2)
    return [out, s["acc"]]


def _evict_own(s):
    from q8_quantized_projection_gb300 import native
    c = s["case"]
    ws = _workspace(native.kv_evict_workspace(c["rows"], c["kv_heads"], c["budget"]))
    native.kv_evict(s["k"], s["v"], s["pos"], s["acc"], s["new_pos"], s["new_acc"], ws,
                    kv_heads=c["kv_heads"], budget=c["budget"], sinks=c["sinks"], recent=c["recent"],
                    kept=s["kept"])
    return [s["k"], s["v"], s["new_pos"], s["new_acc"], s["kept"]]


def _evict_plain(s):
    c = s["case"]
    rows, kvh, dim, budget = c["rows"], c["kv_heads"], c["dim"], c["budget"]
    n = s["pos"].long()[:, None] + 1
    i = torch.arange(c["n_pos"], device=DEV)
    over = n > budget                                                    # [rows, 1]
    always = (i < c["sinks"]) | (i >= n - c["recent"])
    key = torch.where((i < n)[:, None], torch.where(always[:, None], math.inf, s["acc"]), -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :budget]
    src = torch.where(over[:, None], order.sort(dim=-1).values, i[:budget])   # [rows, kvh, budget]
    at = src.transpose(1, 2)[..., None].expand(rows, budget, kvh, dim)
    k, v = s["k"].view(rows, -1, kvh, dim), s["v"].view(rows, -1, kvh, dim)
    k[:, :budget] = k.gather(1, at)
    v[:, :budget] = v.gather(1, at)
    new_acc = torch.zeros_like(s["acc"])
    new_acc[..., :budget] = s["acc"].gather(2, src)
    new_acc = torch.where(over[:, None], new_acc, s["acc"])
    new_pos = torch.where(over[:, 0], budget - 1, s["pos"]).to(torch.int32)
    kept = torch.where((over | (i[:budget] < n))[:, None], src, -1).to(torch.int32)
    return [s["k"], s["v"], new_pos, new_acc, kept]


def _sample_own(s):
    from q8_quantized_projection_gb300 import native
    native.head_sample(s["x"], s["u"], s["tok"], temperature=s["temp"], top_k=s["top_k"],
                       top_p=s["top_p"], min_p=s["min_p"], prob=s["prob"], kept=s["kept"])
    return [s["tok"], s["prob"], s["kept"]]


def _sample_plain(s):
    # in 64 bits: which token a number draws, and where a nucleus ends, lie next to borders
    x = s["x"].double()
    n = x.shape[1]
    greedy = (s["temp"] == 0)[:, None]
    valid = x > -math.inf
    top = torch.where(valid, x, -math.inf).amax(1, keepdim=True)
    t = torch.where(greedy, 1.0, s["temp"].double()[:, None])
    w = torch.where(valid, torch.exp((x - top) / t), 0.0)
    order = torch.sort(torch.where(valid, x, -math.inf), dim=1, descending=True, stable=True).indices
    ws, ok, rank = w.gather(1, order), valid.gather(1, order), torch.arange(n, device=DEV)
    first = rank == 0
    k = torch.where(s["top_k"] > 0, s["top_k"].long(), n)[:, None]
    keep = ok & (rank < torch.where(greedy, 1, k))
    mass = torch.where(keep, ws, 0.0).cumsum(1)
    p = s["top_p"].double()[:, None]
    before = mass - torch.where(keep, ws, 0.0)
    keep = keep & (first | (p >= 1) | (before < p * mass[:, -1:]))
    keep = keep & (first | (ws >= s["min_p"].double()[:, None]))
    stays = torch.zeros_like(valid).scatter_(1, order, keep)
    cdf = torch.where(stays, w, 0.0).cumsum(1)
    total = cdf[:, -1:]
    tok = (cdf <= s["u"].double()[:, None] * total).sum(1, keepdim=True).clamp(max=n - 1)
    prob = (w.gather(1, tok) / total)[:, 0]
    return [tok[:, 0].to(torch.int32), prob.float(), stays.sum(1).to(torch.int32)]


# ---------------------------------------------------- the definition, 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attn":
        return _attn_exact(case, s)
    if case["op"] == "evict":
        return _evict_exact(case, s)
    return _sample_exact(case, s)


def _attn_exact(case, s):
    rows, kvh, dim = case["rows"], case["kv_heads"], case["dim"]
    group = case["heads"] // kvh
    out = torch.zeros(rows, case["heads"] * dim, dtype=torch.float64, device=DEV)
    acc = s["acc"].double()
    for m, n in enumerate(_lens(case)):
        see = list(range(min(case["sinks"], n))) if case["window"] >= 0 else []
        see += range(max(len(see), n - case["window"]) if case["window"] >= 0 else 0, n)
        if not see:
            continue
        see = torch.tensor(see, device=DEV)
        for h in range(kvh):
            cols = slice(h * dim, (h + 1) * dim)
            qh = s["qkv"][m, h * group * dim:(h + 1) * group * dim].double().view(group, dim)
            w = torch.softmax((qh @ s["k"][m, see][:, cols].double().T) / math.sqrt(dim), dim=1)
            out[m, h * group * dim:(h + 1) * group * dim] = (w @ s["v"][m, see][:, cols].double()).flatten()
            acc[m, h, see] += w.sum(0)
    return [out, acc] if case["acc"] else [out]


def _evict_exact(case, s):
    kvh, dim, budget = case["kv_heads"], case["dim"], case["budget"]
    new_pos, new_acc = s["pos"].clone(), s["acc"].double()
    kept = torch.full((case["rows"], kvh, budget), -1, dtype=torch.int32, device=DEV)
    for m, n in enumerate(_lens(case)):
        if n <= budget:
            kept[m, :, :n] = torch.arange(n, device=DEV)
            continue
        new_pos[m] = budget - 1
        lo, hi = case["sinks"], n - case["recent"]
        for h in range(kvh):
            mid = s["acc"][m, h, lo:hi].double()
            best = torch.argsort(mid, descending=True, stable=True)[:budget - lo - case["recent"]] + lo
            idx = torch.cat([torch.arange(lo, device=DEV), best.sort().values,
                             torch.arange(hi, n, device=DEV)])
            cols = slice(h * dim, (h + 1) * dim)
            s["k"][m, :budget, cols] = s["k"][m, idx][:, cols]
            s["v"][m, :budget, cols] = s["v"][m, idx][:, cols]
            new_acc[m, h] = 0
            new_acc[m, h, :budget] = s["acc"][m, h, idx].double()
            kept[m, h] = idx
    return [s["k"], s["v"], new_pos, new_acc, kept]


def _sample_exact(case, s):
    toks, probs, counts = [], [], []
    for m in range(case["rows"]):
        x, t = s["x"][m].double(), float(s["temp"][m])
        order = torch.argsort(x, descending=True, stable=True)
        if t == 0:
            order = order[:1]
        if s["top_k"][m] > 0:
            order = order[:int(s["top_k"][m])]
        w = torch.exp((x[order] - x[order[0]]) / (t or 1.0))
        if s["top_p"][m] < 1:
            # the first place whose mass, itself included, reaches the share
            cum = w.cumsum(0)
            end = int((cum >= s["top_p"][m].double() * cum[-1]).double().argmax()) + 1
            order, w = order[:end], w[:end]
        big = w >= s["min_p"][m].double()
        big[0] = True
        order, w = order[big], w[big]
        ids, at = order.sort()
        w = w[at]
        cum = w.cumsum(0)
        j = min(int((cum <= s["u"][m].double() * cum[-1]).sum()), len(ids) - 1)
        toks.append(int(ids[j]))
        probs.append(float(w[j] / cum[-1]))
        counts.append(len(ids))
    return [torch.tensor(toks, dtype=torch.int32), torch.tensor(probs, dtype=torch.float64),
            torch.tensor(counts, dtype=torch.int32)]
