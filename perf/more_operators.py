"""K/V caches held in 8 and 4 bits, as measured calls: tokens stored and read back (kvq_store,
kvq_load), entries read back (kvq_load), attention of a decode step over such a cache
(kvq_attn_decode) and eviction from it by accumulated attention weight (kvq_evict).

A head's values are cut in blocks of 32.  "i8": d = amax / 127 in binary32, codes
round_half_away(x / d) of -127 to 127.  "u4": m = binary16(min), s = binary16((max - min) / 15),
codes round_half_away((x - m) / s) of 0 to 15, the value m + s * code; two codes a byte, the
even value's below.  Codes lie [rows][kv_heads][n_pos][head_dim], the blocks' d or (s, m) beside
them [rows][kv_heads][n_pos][head_dim / 32].

`run` computes an operator in plain torch operations, or through the library's
entry points where `own` is true, on the state that `prepare` makes.
"""
import math

import torch

own = False   # run the library's entry points instead of the plain forms

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
VALUE_BYTES = {"i8": 36 / 32, "u4": 20 / 32}   # codes and blocks, a value

# ------------------------------------------------------------------- cases


def listed():
    return [
        # one user's new token behind the QKV projection: the launches' latency
        dict(name="store-token", op="store", kind="u4", rows=1, tokens=1, len_min=1, kv_heads=8, dim=128,
             n_pos=4096, src="f32"),
        # a serving batch's new tokens
        dict(name="store-batch", op="store", kind="i8", rows=64, tokens=1, len_min=1, kv_heads=8, dim=128,
             n_pos=4096, src="f32"),
        # a padded batch of prompts, computed in 16 bits
        dict(name="store-prompts", op="store", kind="u4", rows=6, tokens=6001, len_min=1200, kv_heads=8,
             dim=128, n_pos=8192, src="bf16"),
        # odd sizes: part of three short caches, in binary32
        dict(name="load-odd", op="load", kind="i8", rows=3, tokens=1001, len_min=317, kv_heads=5, dim=96,
             n_pos=1501, src="f32"),
        # a long cache read back whole, for a computation in 16 bits
        dict(name="load-long", op="load", kind="u4", rows=2, tokens=65536, len_min=65536, kv_heads=8, dim=128,
             n_pos=65536, src="bf16"),
        # one user, a short conversation: the launch's latency
        dict(name="attn-one-short", op="attn", kind="u4", rows=1, heads=32, kv_heads=8, dim=128, n_pos=4096,
             len_max=613, len_min=613, window=-1, sinks=0, acc=False),
        # one user, a document of 128 K tokens, the weights accumulated for an eviction
        dict(name="attn-one-long", op="attn", kind="u4", rows=1, heads=32, kv_heads=8, dim=128, n_pos=131072,
             len_max=130001, len_min=130001, window=-1, sinks=0, acc=True),
        # a ragged batch under a sliding window with four sinks, eight query heads a K/V head
        dict(name="attn-batch-window", op="attn", kind="i8", rows=16, heads=64, kv_heads=8, dim=128, n_pos=8192,
             len_max=8192, len_min=37, window=2048, sinks=4, acc=False),
        # odd sizes: seven query heads a K/V head, 96 values a head, a ragged window, a row of no entry
        dict(name="attn-odd", op="attn", kind="i8", rows=5, heads=14, kv_heads=2, dim=96, n_pos=5001,
             len_max=5001, len_min=0, window=1001, sinks=3, acc=True),
        # a full serving batch with every token visible
        dict(name="attn-batch-full", op="attn", kind="u4", rows=64, heads=32, kv_heads=8, dim=128, n_pos=8192,
             len_max=8192, len_min=4100, window=-1, sinks=0, acc=False),
        # a batch of 16 at 8192 halved, some sequences still under the budget
        dict(name="evict-batch", op="evict", kind="u4", rows=16, kv_heads=8, dim=128, n_pos=8192, len_max=8192,
             len_min=2000, budget=4096, sinks=4, recent=512),
        # long caches, a quarter of each evicted
        dict(name="evict-long", op="evict", kind="i8", rows=4, kv_heads=8, dim=128, n_pos=32768, len_max=32768,
             len_min=32001, budget=24576, sinks=16, recent=1024),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["store", "load", "attn", "attn", "attn", "evict"])
    kind = rng.choice(["i8", "u4"])
    rows = _log_int(rng, 1, 64)
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    dim = rng.choice([32, 64, 96, 128, 160, 256])
    # entries, by the bytes of attn-batch-full
    room = int(64 * 6146 * 1024 * VALUE_BYTES["u4"] / VALUE_BYTES[kind]) // (rows * kv_heads * dim)
    if op in ("store", "load"):
        # (a value costs the float it comes from or goes to as well)
        tokens = 1 if op == "store" and rng.random() < 0.3 else _log_int(rng, 1, max(2, min(65536, room // 16)))
        return dict(op=op, kind=kind, rows=rows, tokens=tokens, len_min=_log_int(rng, 1, tokens), kv_heads=kv_heads,
                    dim=dim, n_pos=tokens + rng.randrange(1, 300), src=rng.choice(["f32", "f16", "bf16"]))
    if op == "attn":
        group = rng.choice([1, 2, 3, 4, 5, 7, 8])
        n_pos = _log_int(rng, 64, max(65, min(131072, room // (2 if group <= 4 else 4))))
        window = -1 if rng.random() < 0.5 else _log_int(rng, 1, n_pos)
        return dict(op=op, kind=kind, rows=rows, heads=kv_heads * group, kv_heads=kv_heads, dim=dim, n_pos=n_pos,
                    len_max=max(1, n_pos - rng.randrange(0, 1 + n_pos // 4)),
                    len_min=_log_int(rng, 1, max(2, n_pos // 2)), window=window,
                    sinks=0 if window < 0 else rng.choice([0, 1, 4, 13]), acc=rng.random() < 0.5)
    n_pos = _log_int(rng, 256, max(257, min(65536, room // 4)))
    budget = max(64, int(n_pos * rng.uniform(0.3, 0.9)))
    return dict(op=op, kind=kind, rows=rows, kv_heads=kv_heads, dim=dim, n_pos=n_pos, len_max=n_pos,
                len_min=max(1, int(n_pos * rng.uniform(0.2, 1.0))), budget=budget,
                sinks=rng.choice([0, 1, 4, 16]), recent=rng.choice([1, budget // 8, budget // 4]))


def _lens(case):
    """The rows' lengths: from the longest down to len_min, in an order that mixes long and short."""
    rows, most = case["rows"], case["len_max"] if "len_max" in case else case["tokens"]
    hi, lo = max(most, case["len_min"]), min(most, case["len_min"])
    if rows == 1:
        return [hi]
    lens = [hi - (hi - lo) * i // (rows - 1) for i in range(rows)]
    return [lens[(i * 7) % rows] for i in range(rows)] if rows % 7 else lens


def _visible(case, n):
    if case["window"] < 0:
        return n
    return min(n, min(case["sinks"], n) + case["window"])


def work(case):
    kv_dim, held = case["kv_heads"] * case["dim"], VALUE_BYTES[case["kind"]]
    if case["op"] in ("store", "load"):
        n = 2 * sum(_lens(case)) * kv_dim
        floats = 2 if case["op"] == "store" else 1        # read, and written again
        return {"bytes": n * floats * (BYTES[case["src"]] + held), "flops": 4 * n * floats}
    if case["op"] == "attn":
        vis = sum(_visible(case, n) for n in _lens(case))
        nbytes = 2 * vis * kv_dim * held + 8 * case["rows"] * case["heads"] * case["dim"]
        nbytes += 8 * vis * case["kv_heads"] if case["acc"] else 0
        return {"bytes": nbytes, "flops": 4 * vis * case["heads"] * case["dim"]}
    # each kept entry behind the sinks is read and written in K and in V
    full = sum(n > case["budget"] for n in _lens(case))
    moved = full * (case["budget"] - case["sinks"]) * kv_dim
    nbytes = 4 * moved * held + 4 * case["rows"] * case["kv_heads"] * (2 * case["n_pos"] + case["budget"])
    return {"bytes": nbytes, "flops": case["rows"] * case["kv_heads"] * case["n_pos"]}


# ------------------------------------------------------- the quantised form


def _half_away(x):
    t = torch.trunc(x)
    return t + torch.sign(x) * ((x - t).abs() >= 0.5)


def _quantise(x, kind):
    """x [..., D] binary32: codes and blocks."""
    b = x.unflatten(-1, (-1, 32))
    if kind == "i8":
        d = b.abs().amax(-1) / torch.full((), 127.0, device=DEV)   # (a divisor on the host would be inverted)
        q = torch.where(d[..., None] == 0, 0.0, _half_away(b / d[..., None])).clamp(-127, 127)
        return q.flatten(-2).to(torch.int8), d
    lo = b.amin(-1)
    s = ((b.amax(-1) - lo) / torch.full((), 15.0, device=DEV)).half()
    m = lo.half()
    q = (b - m.float()[..., None]) / s.float()[..., None]
    q = torch.where((s == 0)[..., None], 0.0, _half_away(q)).clamp(0, 15).flatten(-2).to(torch.uint8)
    return q[..., 0::2] | q[..., 1::2] << 4, torch.stack((s, m), -1)


def _values(codes, blocks, kind):
    """The values [..., D] that they stand for, in binary32."""
    if kind == "i8":
        return (codes.float().unflatten(-1, (-1, 32)) * blocks[..., None]).flatten(-2)
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float().unflatten(-1, (-1, 32))
    return (q * blocks[..., 0:1].float() + blocks[..., 1:2].float()).flatten(-2)


# ------------------------------------------------------------------ inputs


def _cache(case, g, n):
    """One quantised cache, its first n entries of a bell with some channels larger than others, as keys have them."""
    rows, kvh, dim, kind = case["rows"], case["kv_heads"], case["dim"], case["kind"]
    u4 = kind == "u4"
    codes = torch.zeros(rows, kvh, case["n_pos"], dim // 2 if u4 else dim, dtype=torch.uint8 if u4 else torch.int8,
                        device=DEV)
    blocks = torch.zeros((rows, kvh, case["n_pos"], dim // 32) + ((2,) if u4 else ()),
                         dtype=torch.float16 if u4 else torch.float32, device=DEV)
    channel = torch.randn(kvh, 1, dim, generator=g, device=DEV).mul_(0.5).exp_()
    step = max(1, (1 << 26) // max(1, kvh * n * dim))
    for m in range(0, rows, step):
        x = torch.randn(min(step, rows - m), kvh, n, dim, generator=g, device=DEV).mul_(channel)
        codes[m:m + step, :, :n], blocks[m:m + step, :, :n] = _quantise(x, kind)
    return [codes, blocks]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    rows, kvh, dim = case["rows"], case["kv_heads"], case["dim"]
    kv_dim = kvh * dim
    if case["op"] in ("store", "load"):
        tokens, src = case["tokens"], TYPES[case["src"]]
        lens = torch.tensor(_lens(case), dtype=torch.int32, device=DEV)
        pos = torch.randint(0, case["n_pos"] - tokens + 1, (rows,), generator=g, device=DEV).to(torch.int32)
        stored = case["n_pos"] if case["op"] == "load" else 0
        state = dict(case=case, pos=pos, lens=lens, cache=_cache(case, g, stored) + _cache(case, g, stored),
                     k_out=torch.zeros(rows, tokens, kv_dim, dtype=src, device=DEV),
                     v_out=torch.zeros(rows, tokens, kv_dim, dtype=src, device=DEV))
        if case["op"] == "store":
            # K and V are columns of the fused QKV projection's rows (four query heads a K/V head)
            qkv = torch.randn(rows, tokens, 6 * kv_dim, generator=g, device=DEV).to(src)
            state.update(k=qkv[..., 4 * kv_dim:5 * kv_dim], v=qkv[..., 5 * kv_dim:])
        return state
    pos = torch.tensor(_lens(case), dtype=torch.int32, device=DEV) - 1
    cache = _cache(case, g, case["n_pos"]) + _cache(case, g, case["n_pos"])
    # accumulated weights: a heavy tail, as attention leaves them, and some never attended
    a = torch.empty(rows, kvh, case["n_pos"], device=DEV).normal_(generator=g).mul_(2).sub_(4).exp_()
    a.masked_fill_(a < 1e-3, 0.0)
    state = dict(case=case, cache=cache, pos=pos, acc=a)
    if case["op"] == "attn":
        # q is the first part of the fused QKV projection's output rows
        qkv = torch.randn(rows, (case["heads"] + 2 * kvh) * dim, generator=g, device=DEV)
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
    if op == "store":
        return _store_own(state) if own else _store_plain(state)
    if op == "load":
        return _load_own(state) if own else _load_plain(state)
    if op == "attn":
        return _attn_own(state) if own else _attn_plain(state)
    return _evict_own(state) if own else _evict_plain(state)


def _store_own(s):
    from q8_quantized_projection_gb300 import native
    native.kvq_store(s["k"], s["v"], s["pos"], s["cache"], lens=s["lens"])
    return _load_own(s)


def _load_own(s):
    from q8_quantized_projection_gb300 import native
    native.kvq_load(s["cache"], s["k_out"], s["v_out"], pos=s["pos"], lens=s["lens"])
    return [s["k_out"], s["v_out"]]


def _attn_own(s):
    from q8_quantized_projection_gb300 import native
    c = s["case"]
    nbytes = native.kvq_attn_decode_workspace(c["rows"], c["heads"], c["kv_heads"], c["dim"], c["n_pos"],
                                              window=c["window"], sinks=c["sinks"], acc=c["acc"])
    native.kvq_attn_decode(s["qkv"], s["cache"], s["pos"], s["out"], _workspace(nbytes), heads=c["heads"],
                           window=c["window"], sinks=c["sinks"], acc=s["acc"] if c["acc"] else None)
    return [s["out"], s["acc"]] if c["acc"] else [s["out"]]


# (eviction computes no code or block, it moves them: they come back as they are held, and are equal)

def _evict_own(s):
    from q8_quantized_projection_gb300 import native
    c = s["case"]
    ws = _workspace(native.kvq_evict_workspace(c["rows"], c["kv_heads"], c["budget"]))
    native.kvq_evict(s["cache"], s["pos"], s["acc"], s["new_pos"], s["new_acc"], ws, budget=c["budget"],
                     sinks=c["sinks"], recent=c["recent"], kept=s["kept"])
    return [s["cache"], s["new_pos"], s["new_acc"], s["kept"]]


def _slots(s):
    """Rows [rows, 1], entries [rows, tokens] and which of them the rows' lengths cover."""
    rows, tokens = s["case"]["rows"], s["case"]["tokens"]
    t = torch.arange(tokens, device=DEV)
    return torch.arange(rows, device=DEV)[:, None], s["pos"].long()[:, None] + t, t < s["lens"][:, None]


def _store_plain(s):
    c = s["case"]
    m, i, within = _slots(s)
    for x, codes, blocks in ((s["k"], *s["cache"][:2]), (s["v"], *s["cache"][2:])):
        q, b = _quantise(x.float().unflatten(-1, (c["kv_heads"], c["dim"])), c["kind"])
        codes[m, :, i] = torch.where(within[..., None, None], q, codes[m, :, i])
        within_b = within.view(within.shape + (1,) * (b.dim() - 2))
        blocks[m, :, i] = torch.where(within_b, b, blocks[m, :, i])
    return _load_plain(s)


def _load_plain(s):
    m, i, within = _slots(s)
    for out, codes, blocks in ((s["k_out"], *s["cache"][:2]), (s["v_out"], *s["cache"][2:])):
        x = _values(codes[m, :, i], blocks[m, :, i], s["case"]["kind"]).flatten(-2).to(out.dtype)
        out.copy_(torch.where(within[..., None], x, out))
    return [s["k_out"], s["v_out"]]


def _attn_plain(s):
    c = s["case"]
    rows, kvh, dim = c["rows"], c["kv_heads"], c["dim"]
    group = c["heads"] // kvh
    q = s["qkv"][:, :c["heads"] * dim].reshape(rows, kvh, group, dim)
    i, pos = torch.arange(c["n_pos"], device=DEV), s["pos"].long()[:, None]
    vis = i <= pos
    if c["window"] >= 0:
        vis = vis & ((i < c["sinks"]) | (i > pos - c["window"]))
    vis = vis[:, None, None, :]
    k = _values(*s["cache"][:2], c["kind"]).transpose(-1, -2)
    score = torch.matmul(q * (1.0 / math.sqrt(dim)), k).masked_fill(~vis, -math.inf)
    top = score.amax(-1, keepdim=True)
    w = torch.where(vis, torch.exp(score - torch.where(top == -math.inf, 0.0, top)), 0.0)
    total = w.sum(-1, keepdim=True)
    w = torch.where(total == 0, 0.0, w / total)
    out = torch.matmul(w, _values(*s["cache"][2:], c["kind"])).reshape(rows, c["heads"] * dim)
    if not c["acc"]:
        return [out]
    s["acc"] += w.sum(2)
    return [out, s["acc"]]


def _evict_plain(s):
    c = s["case"]
    budget = c["budget"]
    n = s["pos"].long()[:, None] + 1
    i = torch.arange(c["n_pos"], device=DEV)
    over = n > budget                                                    # [rows, 1]
    always = (i < c["sinks"]) | (i >= n - c["recent"])
    key = torch.where((i < n)[:, None], torch.where(always[:, None], math.inf, s["acc"]), -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :budget]
    src = torch.where(over[:, None], order.sort(dim=-1).values, i[:budget])   # [rows, kv_heads, budget]
    for x in s["cache"]:
        at = src.view(src.shape + (1,) * (x.dim() - 3)).expand(src.shape + x.shape[3:])
        x[:, :, :budget] = x.gather(2, at)
    new_acc = torch.zeros_like(s["acc"])
    new_acc[..., :budget] = s["acc"].gather(2, src)
    new_acc = torch.where(over[:, None], new_acc, s["acc"])
    new_pos = torch.where(over[:, 0], budget - 1, s["pos"]).to(torch.int32)
    kept = torch.where((over | (i[:budget] < n))[:, None], src, -1).to(torch.int32)
    return [s["cache"], new_pos, new_acc, kept]


# ---------------------------------------------------- the definition, 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("store", "load"):
        return _roundtrip_exact(case, s)
    if case["op"] == "attn":
        return _attn_exact(case, s)
    return _evict_exact(case, s)


def _exact_values(codes, blocks):
    """In 64 bits, from one row and head's codes and blocks [n, ...]."""
    n = codes.shape[0]
    if codes.dtype == torch.int8:
        return (codes.double().view(n, -1, 32) * blocks.double().view(n, -1, 1)).view(n, -1)
    q = torch.empty(n, codes.shape[1] * 2, dtype=torch.float64, device=DEV)
    q[:, 0::2], q[:, 1::2] = (codes % 16).double(), torch.div(codes, 16, rounding_mode="floor").double()
    s, m = blocks.double().unbind(-1)
    return (m[..., None] + q.view(n, -1, 32) * s[..., None]).view(n, -1)


def _exact_stored(x, kind):
    """What x [n, D] reads back as.  The definition rounds to binary32 or binary16 at these places; a
    quotient of such numbers in 64 bits, rounded, is the quotient rounded."""
    b = x.double().view(x.shape[0], -1, 32)
    to = lambda v, t: v.to(t).double()  # noqa: E731
    if kind == "i8":
        d = to(b.abs().max(-1, keepdim=True).values / 127, torch.float32)
        code = to(b / d, torch.float32)
        code = torch.where(d > 0, torch.copysign((code.abs() + 0.5).floor(), code), 0)
        return (code * d).view(x.shape)
    lo, hi = b.min(-1, keepdim=True).values, b.max(-1, keepdim=True).values
    s = to(to(to(hi - lo, torch.float32) / 15, torch.float32), torch.float16)
    m = to(lo, torch.float16)
    code = to(to(b - m, torch.float32) / s, torch.float32)
    code = torch.where(s > 0, (code + 0.5).floor().clamp(0, 15), 0)
    return (m + s * code).view(x.shape)


def _roundtrip_exact(case, s):
    got = []
    for name, at in (("k", 0), ("v", 2)):
        out = torch.zeros(s["k_out"].shape, dtype=torch.float64, device=DEV)
        for m, n in enumerate(_lens(case)):
            first = int(s["pos"][m])
            for h in range(case["kv_heads"]):
                cols = slice(h * case["dim"], (h + 1) * case["dim"])
                if case["op"] == "store":
                    out[m, :n, cols] = _exact_stored(s[name][m, :n, cols], case["kind"])
                else:
                    out[m, :n, cols] = _exact_values(s["cache"][at][m, h, first:first + n],
                                                     s["cache"][at + 1][m, h, first:first + n])
        got.append(out)
    return got


def _attn_exact(case, s):
    kvh, dim = case["kv_heads"], case["dim"]
    group = case["heads"] // kvh
    out = torch.zeros(case["rows"], case["heads"] * dim, dtype=torch.float64, device=DEV)
    acc = s["acc"].double()
    for m, n in enumerate(_lens(case)):
        see = list(range(min(case["sinks"], n))) if case["window"] >= 0 else []
        see += range(max(len(see), n - case["window"]) if case["window"] >= 0 else 0, n)
        if not see:
            continue
        see = torch.tensor(see, device=DEV)
        for h in range(kvh):
            k, v = (_exact_values(s["cache"][i][m, h, see], s["cache"][i + 1][m, h, see]) for i in (0, 2))
            qh = s["qkv"][m, h * group * dim:(h + 1) * group * dim].double().view(group, dim)
            w = torch.softmax((qh @ k.T) / math.sqrt(dim), dim=1)
            out[m, h * group * dim:(h + 1) * group * dim] = (w @ v).flatten()
            acc[m, h, see] += w.sum(0)
    return [out, acc] if case["acc"] else [out]


def _evict_exact(case, s):
    kvh, budget = case["kv_heads"], case["budget"]
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
            for x in s["cache"]:
                x[m, h, :budget] = x[m, h, idx]
            new_acc[m, h] = 0
            new_acc[m, h, :budget] = s["acc"][m, h, idx].double()
            kept[m, h] = idx
    return [s["cache"], new_pos, new_acc, kept]
