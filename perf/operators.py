"""What is measured of the operators around the KV cache: the query / key norm
with rotary positions that fills it, the decode over a prefix that a whole
batch shares, and the decode over blocks of keys that a cheap score selects.

A case names one call (or the calls of one step) at one size.  `run` computes
it in plain torch operations, or, where `own` is true, by the package's calls.
Geometry throughout: 8 query heads on one KV head of 256 dims; blocks of 64
keys.
"""
import math

import torch

own = False

HEADS, DIM, BLOCK = 8, 256, 64
MAX_POSITION = 131072
SCALE = 1.0 / 16.0
EPS = 1e-6
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# --------------------------------------------------------------------- cases

def listed():
    return [
        # One new token of one conversation: q / k / v of a decode step, normed,
        # rotated and appended.  Latency is all that counts.
        {"name": "norm_rope one token bf16", "op": "norm_rope", "rows": 1, "axes": 1, "dtype": "bf16", "kv": "bf16",
         "far": 131071, "fused": True, "norm_v": True},
        # A prefill chunk of image and text tokens: positions in time, height
        # and width, the three axes interleaved over the frequencies.
        {"name": "norm_rope chunk 768 three axes", "op": "norm_rope", "rows": 768, "axes": 3, "dtype": "bf16",
         "kv": "bf16", "far": 40000, "fused": True, "norm_v": True},
        # A whole 16K prompt at once, f32 activations into an f16 cache.
        {"name": "norm_rope 16384 rows f32 to f16", "op": "norm_rope", "rows": 16384, "axes": 1, "dtype": "f32",
         "kv": "f16", "far": 16384, "fused": False, "norm_v": False},
        # Three drafts behind a short system prompt.
        {"name": "prefix 3 x 1000 bf16", "op": "prefix", "batch": 3, "prefix": 1000, "own_keys": 77, "window": 0,
         "q": "bf16", "kv": "bf16", "device_len": False},
        # A service step: 32 conversations behind one document of 16K tokens,
        # lengths kept on the GPU as a captured step would.
        {"name": "prefix 32 x 16384 bf16", "op": "prefix", "batch": 32, "prefix": 16384, "own_keys": 1024, "window": 0,
         "q": "bf16", "kv": "bf16", "device_len": True},
        # f32 queries on an f16 cache, eight ragged continuations, a sliding
        # window that cuts the prefix at another key for each of them.
        {"name": "prefix 8 x 9001 window f32 q", "op": "prefix", "batch": 8, "prefix": 9001, "own_keys": 700,
         "window": 8192, "q": "f32", "kv": "f16", "device_len": False},
        # The largest: 256 continuations behind 120,000 shared tokens.
        {"name": "prefix 256 x 120000 f16", "op": "prefix", "batch": 256, "prefix": 120000, "own_keys": 1000,
         "window": 0, "q": "f16", "kv": "f16", "device_len": False},
        # Long-context decode of one sequence: 64 of 2,048 blocks.
        {"name": "blocks 1 x 131072 f16", "op": "blocks", "batch": 1, "ctx": 131072, "select": 64, "q": "f16",
         "kv": "f16"},
        # A ragged batch, 128 blocks each.
        {"name": "blocks 32 x 32768 bf16", "op": "blocks", "batch": 32, "ctx": 32768, "select": 128, "q": "bf16",
         "kv": "bf16"},
        # A small odd one: f32 queries, contexts that end inside a block.
        {"name": "blocks 5 x 4999 f32 q", "op": "blocks", "batch": 5, "ctx": 4999, "select": 21, "q": "f32",
         "kv": "f16"},
        # Block bounds after one decode step of 64 sequences: some of them
        # complete a block, most do not.
        {"name": "summaries step of 64", "op": "summaries", "batch": 64, "ctx": 4096, "new": 1, "kv": "f16"},
        # Block bounds of four full caches after their prefill.
        {"name": "summaries 4 x 131072 bf16", "op": "summaries", "batch": 4, "ctx": 131072, "new": 131072,
         "kv": "bf16"},
    ]


def _spread(rng, lo, hi):
    """A whole number in lo..hi, spread over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["norm_rope", "prefix", "blocks", "summaries"])
    if op == "norm_rope":
        return {"op": op, "rows": _spread(rng, 1, 16384), "axes": rng.choice([1, 1, 2, 3]),
                "dtype": rng.choice(["bf16", "f16", "f32"]), "kv": rng.choice(["bf16", "f16"]),
                "far": _spread(rng, 100, MAX_POSITION), "fused": rng.random() < 0.5, "norm_v": rng.random() < 0.5}
    q, kv = rng.choice([("bf16", "bf16"), ("f16", "f16"), ("f32", "f16")])
    if op == "prefix":
        prefix = _spread(rng, 100, 120000)
        # f32 queries take operands in two parts: a fifth of the batch for the same cost
        batch = _spread(rng, 1, max(1, min(256, 256 * 120000 // prefix) // (5 if q == "f32" else 1)))
        return {"op": op, "batch": batch, "prefix": prefix, "own_keys": _spread(rng, 1, 1000),
                "window": rng.choice([0, 0, 0, _spread(rng, 64, 60000)]), "q": q, "kv": kv,
                "device_len": rng.random() < 0.5}
    ctx = _spread(rng, 65, MAX_POSITION)
    batch = _spread(rng, 1, max(1, min(64, (1 << 20) // ctx)))
    if op == "blocks":
        return {"op": op, "batch": batch, "ctx": ctx, "select": _spread(rng, 2, 256), "q": q, "kv": kv}
    return {"op": op, "batch": batch, "ctx": ctx, "new": _spread(rng, 1, ctx), "kv": rng.choice(["bf16", "f16", "f32"])}


# -------------------------------------------------------------------- inputs

def _normal(g, shape, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std


def _inv_freq(axes):
    """Frequencies of a rotary base of 10,000 (base 1,000,000 for one axis,
    whose last eighth does not turn)."""
    i = torch.arange(DIM // 2, dtype=torch.float64)
    base = 1e6 if axes == 1 else 1e4
    f = base ** (-i / (DIM // 2))
    if axes == 1:
        f[-DIM // 16:] = 0.0
    return f.float().cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    kept = {}   # workspaces of the package's calls, made by the first of them
    if op == "norm_rope":
        n, dt = case["rows"], DTYPES[case["dtype"]]
        if case["fused"]:   # slices of one projection's output
            qkv = (_normal(g, (n, (HEADS + 2) * DIM), 1.5)).to(dt)
            q = qkv[:, :HEADS * DIM].unflatten(1, (HEADS, DIM))
            k, v = qkv[:, HEADS * DIM:(HEADS + 1) * DIM], qkv[:, (HEADS + 1) * DIM:]
        else:
            q, k, v = (_normal(g, s, 1.5).to(dt) for s in ((n, HEADS, DIM), (n, DIM), (n, DIM)))
        cache_rows = n + 100
        kc, vc = (_normal(g, (cache_rows, DIM)).to(DTYPES[case["kv"]]) for _ in range(2))
        # text rows share a position on every axis, image rows differ
        pos = torch.randint(0, case["far"] + 1, (case["axes"], n), generator=g, device="cuda")
        dst = torch.randperm(cache_rows, generator=g, device="cuda")[:n]
        wq, wk = ((1 + 0.2 * _normal(g, (DIM,))).to(dt) for _ in range(2))
        return {"case": case, "q": q, "k": k, "v": v, "k_cache": kc, "v_cache": vc, "pos": pos, "dst": dst, "wq": wq,
                "wk": wk, "inv_freq": _inv_freq(case["axes"]),
                "freq_axis": [i % case["axes"] for i in range(DIM // 2)],
                "q_out": torch.empty((n, HEADS, DIM), dtype=DTYPES[case["kv"]], device="cuda"), "kept": kept}
    batch, kvt = case["batch"], DTYPES[case["kv"]]
    if op == "prefix":
        cap = case["own_keys"] + 24
        pk, pv = (_normal(g, (case["prefix"], DIM)).to(kvt) for _ in range(2))
        kc, vc = (_normal(g, (batch, cap, DIM)).to(kvt) for _ in range(2))
        mine = torch.randint(1, case["own_keys"] + 1, (batch,), generator=g, device="cuda")
        qt = DTYPES[case["q"]]
        ctx = mine + case["prefix"]
        return {"case": case, "q": _normal(g, (batch, HEADS, DIM)).to(qt), "pk": pk, "pv": pv, "k": kc, "v": vc,
                "ctx": ctx, "ctx_host": ctx.tolist(), "out": torch.empty((batch, HEADS, DIM), dtype=qt, device="cuda"),
                "kept": kept}
    blocks = -(-case["ctx"] // BLOCK)
    cap = blocks * BLOCK
    # keys drift from block to block, as a text's do
    drift = _normal(g, (batch, blocks, 1, DIM), 0.5)
    kc = (_normal(g, (batch, blocks, BLOCK, DIM)) + drift).reshape(batch, cap, DIM).to(kvt)
    ctx = torch.randint(max(1, case["ctx"] // 2), case["ctx"] + 1, (batch,), generator=g, device="cuda")
    if op == "summaries":
        if case["new"] == 1:   # a quarter of the sequences complete a block
            ctx = torch.where(torch.arange(batch, device="cuda") % 4 == 0, ctx // BLOCK * BLOCK + BLOCK, ctx)
            ctx = ctx.clamp(max=case["ctx"])
        elif case["new"] == case["ctx"]:
            ctx = torch.full_like(ctx, case["ctx"])
        # summaries of blocks that the call does not complete stay as they were
        codes = torch.randint(-127, 128, (batch, blocks, 2, DIM), generator=g, device="cuda", dtype=torch.int8)
        return {"case": case, "k": kc, "ctx": ctx, "kept": kept, "codes": codes,
                "scales": torch.rand((batch, blocks), generator=g, device="cuda") + 0.01}
    vc = _normal(g, (batch, cap, DIM)).to(kvt)
    qt = DTYPES[case["q"]]
    codes, scales = _bounds(kc)   # what earlier steps left behind
    return {"case": case, "q": _normal(g, (batch, HEADS, DIM)).to(qt), "k": kc, "v": vc, "ctx": ctx, "codes": codes,
            "scales": scales, "out": torch.empty((batch, HEADS, DIM), dtype=qt, device="cuda"), "kept": kept,
            "blocks": torch.empty((batch, case["select"]), dtype=torch.int32, device="cuda")}


# --------------------------------------------------------------- plain forms

def _codes(x, amax):
    """int8 codes of x under amax (broadcast): round half to even of the f32
    quotient by amax * f32(1/127)."""
    s = amax * (1.0 / 127.0)
    return torch.where(s > 0, torch.round(x / s), 0.0).clamp(-127, 127), s


def _bounds(k):
    """int8 codes [batch, blocks, 2, 256] of the largest and the smallest key
    of every whole block, by dim, and their scales [batch, blocks]."""
    x = k.unflatten(1, (-1, BLOCK))
    hi_lo = torch.stack((x.amax(2), x.amin(2)), 2).float()
    codes, s = _codes(hi_lo, hi_lo.abs().amax((2, 3), keepdim=True))
    return codes.to(torch.int8), s[:, :, 0, 0].contiguous()


def _plain_norm_rope(s):
    case = s["case"]

    def norm(x, w):
        x = x.float()
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        return y if w is None else y * w.float()

    axis = torch.tensor(s["freq_axis"], device="cuda")
    angle = s["pos"].double()[axis].T * s["inv_freq"].double()   # [rows, 128]
    cos, sin = angle.cos().float(), angle.sin().float()

    def turn(x, cos, sin):
        a, b = x[..., :DIM // 2], x[..., DIM // 2:]
        return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)

    kvt = DTYPES[case["kv"]]
    s["q_out"].copy_(turn(norm(s["q"], s["wq"]), cos[:, None], sin[:, None]))
    s["k_cache"][s["dst"]] = turn(norm(s["k"], s["wk"]), cos, sin).to(kvt)
    s["v_cache"][s["dst"]] = (norm(s["v"], None) if case["norm_v"] else s["v"].float()).to(kvt)
    return s["q_out"], s["k_cache"], s["v_cache"]


def _plain_prefix(s):
    case, q = s["case"], s["q"].float()
    prefix, ctx = case["prefix"], s["ctx"]
    pos_p = torch.arange(prefix, device="cuda")
    pos_s = prefix + torch.arange(s["k"].shape[1], device="cuda")
    lo = (ctx - case["window"]).clamp(min=0)[:, None] if case["window"] > 0 else torch.zeros_like(ctx)[:, None]
    sp = q.reshape(-1, DIM) @ s["pk"].float().T * SCALE
    sp = sp.view(-1, HEADS, prefix).masked_fill((pos_p < lo)[:, None], -math.inf)
    ss = torch.matmul(q, s["k"].float().transpose(1, 2)) * SCALE
    ss = ss.masked_fill(((pos_s >= ctx[:, None]) | (pos_s < lo))[:, None], -math.inf)
    m = torch.maximum(sp.amax(-1), ss.amax(-1))[..., None]
    ep, es = (sp - m).exp(), (ss - m).exp()
    o = (ep.view(-1, prefix) @ s["pv"].float()).view_as(q) + torch.matmul(es, s["v"].float())
    s["out"].copy_(o / (ep.sum(-1) + es.sum(-1))[..., None])
    return s["out"]


def _plain_blocks(s):
    case, q, ctx = s["case"], s["q"].float(), s["ctx"]
    n, codes = s["codes"].shape[1], s["codes"].float()
    qc, sq = _codes(q, q.abs().amax(-1, keepdim=True))
    # sums of at most 256 products of whole numbers to 127: exact in f32
    dot = (torch.matmul(qc.clamp(min=0), codes[:, :, 0].transpose(1, 2))
           + torch.matmul(qc.clamp(max=0), codes[:, :, 1].transpose(1, 2)))
    score = (dot * (sq * s["scales"][:, None])).amax(1) + 0.0   # [batch, blocks]
    block = torch.arange(n, device="cuda")
    last = ((ctx - 1) // BLOCK)[:, None]
    score = torch.where((block == 0) | (block == last), math.inf, score).masked_fill(block > last, -math.inf)
    # the highest scores, ties to the lowest index; then in order, -1 behind the last
    top = torch.sort(score, dim=1, descending=True, stable=True)
    take = min(case["select"], n)
    ids = torch.where(top.values[:, :take] == -math.inf, n, top.indices[:, :take]).sort(1).values
    ids = torch.nn.functional.pad(ids, (0, case["select"] - take), value=n)
    s["blocks"].copy_(torch.where(ids == n, -1, ids))
    safe = ids.clamp(max=n - 1)
    pos = (safe[:, :, None] * BLOCK + torch.arange(BLOCK, device="cuda")).flatten(1)
    seen = (pos < ctx[:, None]) & (ids < n).repeat_interleave(BLOCK, 1)
    k, v = (torch.gather(x, 1, pos[..., None].expand(-1, -1, DIM)).float() for x in (s["k"], s["v"]))
    sc = (torch.matmul(q, k.transpose(1, 2)) * SCALE).masked_fill(~seen[:, None], -math.inf)
    e = (sc - sc.amax(-1, keepdim=True)).exp()
    s["out"].copy_(torch.matmul(e, v) / e.sum(-1, keepdim=True))
    return s["blocks"], s["out"]


def _plain_summaries(s):
    case, ctx = s["case"], s["ctx"][:, None]
    codes, scales = _bounds(s["k"])
    end = torch.arange(1, codes.shape[1] + 1, device="cuda") * BLOCK
    done = (end <= ctx) & (end > ctx - case["new"])
    s["codes"].copy_(torch.where(done[..., None, None], codes, s["codes"]))
    s["scales"].copy_(torch.where(done, scales, s["scales"]))
    return s["codes"], s["scales"]


# ----------------------------------------------------------- the package's calls

def _own_norm_rope(s):
    import kv_cache_attention_states_b200 as kca
    kca.attn_norm_rope_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["dst"], s["pos"], s["inv_freq"],
                              freq_axis=s["freq_axis"], q_weight=s["wq"], k_weight=s["wk"], eps=EPS,
                              norm_v=s["case"]["norm_v"], q_out=s["q_out"])
    return s["q_out"], s["k_cache"], s["v_cache"]


def _own_prefix(s):
    import kv_cache_attention_states_b200 as kca
    case, kept = s["case"], s["kept"]
    bound = case["prefix"] + case["own_keys"]
    if "ws" not in kept:
        kept["ws"] = kca.new_workspace(kca.attn_decode_prefix_workspace_bytes(
            kca.dtype_code(s["q"]), kca.dtype_code(s["k"]), case["prefix"], [bound] * case["batch"], case["window"]))
    return kca.attn_decode_prefix(s["q"], s["pk"], s["pv"], case["prefix"], s["k"], s["v"],
                                  s["ctx"] if case["device_len"] else s["ctx_host"], window=case["window"],
                                  ctx_bound=bound, out=s["out"], workspace=kept["ws"])


def _own_blocks(s):
    import kv_cache_attention_states_b200 as kca
    case, kept = s["case"], s["kept"]
    if "ws" not in kept:
        kept["select"] = kca.new_workspace(kca.attn_select_blocks_workspace_bytes(case["batch"], case["ctx"]))
        kept["ws"] = kca.new_workspace(kca.attn_decode_blocks_workspace_bytes(case["batch"], case["select"]))
    kca.attn_select_blocks(s["q"], s["codes"], s["scales"], s["ctx"], case["ctx"], case["select"], blocks=s["blocks"],
                           workspace=kept["select"])
    kca.attn_decode_blocks(s["q"], s["k"], s["v"], s["blocks"], s["ctx"], case["ctx"], out=s["out"],
                           workspace=kept["ws"])
    return s["blocks"], s["out"]


def _own_summaries(s):
    import kv_cache_attention_states_b200 as kca
    return kca.attn_summarize_blocks(s["k"], s["ctx"], s["case"]["new"], codes=s["codes"], scales=s["scales"])


def run(state):
    op = state["case"]["op"]
    if own:
        f = {"norm_rope": _own_norm_rope, "prefix": _own_prefix, "blocks": _own_blocks, "summaries": _own_summaries}
    else:
        f = {"norm_rope": _plain_norm_rope, "prefix": _plain_prefix, "blocks": _plain_blocks,
             "summaries": _plain_summaries}
    return f[op](state)


# ---------------------------------------------------------------------- work

def work(case):
    size = {"f32": 4, "f16": 2, "bf16": 2}
    op = case["op"]
    if op == "norm_rope":
        n = case["rows"]
        row = (HEADS + 2) * DIM
        return {"bytes": n * (row * (size[case["dtype"]] + size[case["kv"]]) + 8 * (case["axes"] + 1)),
                "flops": n * row * 8}
    kv = size[case["kv"]]
    if op == "prefix":
        b = case["batch"]
        mine = (case["own_keys"] + 1) / 2                 # lengths are even over 1..own_keys
        seen = case["prefix"] if case["window"] <= 0 else min(case["prefix"], case["window"])
        own_seen = mine if case["window"] <= 0 else min(mine, case["window"])
        bytes_ = (seen + b * own_seen) * 2 * DIM * kv + 2 * b * HEADS * DIM * size[case["q"]]
        return {"bytes": bytes_, "flops": 4 * DIM * HEADS * b * (max(0, seen - (mine if case["window"] > 0 else 0)) + own_seen)}
    b = case["batch"]
    if op == "blocks":
        ctx = 0.75 * case["ctx"]                          # lengths are even over the upper half
        blocks = ctx / BLOCK
        keys = min(ctx, case["select"] * BLOCK)
        return {"bytes": b * (blocks * (2 * DIM + 4) + keys * 2 * DIM * kv + 2 * HEADS * DIM * size[case["q"]]
                              + 4 * case["select"]),
                "flops": b * HEADS * DIM * (4 * blocks + 4 * keys)}
    ctx = case["ctx"] if case["new"] == case["ctx"] else 0.75 * case["ctx"]
    blocks = min(ctx, case["new"]) / BLOCK if case["new"] > 1 else 0.25
    return {"bytes": b * (blocks * (BLOCK * DIM * kv + 2 * DIM + 4) + 8), "flops": b * blocks * 2 * BLOCK * DIM}


# --------------------------------------------------------------------- exact

def _exact_norm_rope(s):
    f64 = torch.float64
    n = s["q"].shape[0]
    x = torch.cat((s["q"].reshape(n, HEADS, DIM), s["k"].reshape(n, 1, DIM), s["v"].reshape(n, 1, DIM)), 1).to(f64)
    y = x / (x.pow(2).sum(-1, keepdim=True) / DIM + EPS).sqrt()
    w = torch.cat((s["wq"].to(f64).expand(HEADS, DIM), s["wk"].to(f64)[None]))
    z = torch.view_as_complex((y[:, :-1] * w).unflatten(-1, (2, DIM // 2)).transpose(-1, -2).contiguous())
    freq = s["inv_freq"].to(f64)
    # angle of frequency i from the axis it belongs to
    turn = torch.stack([s["pos"][a].to(f64) * freq[i] for i, a in enumerate(s["freq_axis"])], -1)
    z = torch.view_as_real(z * torch.polar(torch.ones_like(turn), turn)[:, None]).transpose(-1, -2).flatten(-2)
    k, v = s["k_cache"].to(f64), s["v_cache"].to(f64)
    k[s["dst"]] = z[:, HEADS]
    v[s["dst"]] = y[:, -1] if s["case"]["norm_v"] else x[:, -1]
    return z[:, :HEADS], k, v


def _exact_prefix(s):
    case, f64 = s["case"], torch.float64
    prefix, out = case["prefix"], []
    pk, pv = s["pk"].to(f64), s["pv"].to(f64)
    for b, ctx in enumerate(s["ctx_host"]):
        lo = max(0, ctx - case["window"]) if case["window"] > 0 else 0
        first, mine = min(lo, prefix), max(0, lo - prefix)
        k = torch.cat((pk[first:], s["k"][b, mine:ctx - prefix].to(f64)))
        v = torch.cat((pv[first:], s["v"][b, mine:ctx - prefix].to(f64)))
        out.append(torch.softmax(s["q"][b].to(f64) @ k.T * SCALE, -1) @ v)
    return torch.stack(out)


def _exact_blocks(s):
    f64 = torch.float64
    lists, outs = [], []
    for b, ctx in enumerate(s["ctx"].tolist()):
        n = -(-ctx // BLOCK)
        q = s["q"][b].float()
        # codes and scales are f32 by definition, the sums whole numbers
        step = q.abs().max(-1).values * torch.tensor(1.0 / 127.0, dtype=torch.float32, device="cuda")
        code = (q / step[:, None]).round().to(f64)
        high, low = s["codes"][b, :n].to(f64).unbind(1)
        whole = torch.where(code[:, None] > 0, code[:, None] * high, code[:, None] * low).sum(-1)
        score = (whole.float() * (step[:, None] * s["scales"][b, :n])).max(0).values.tolist()
        forced = sorted({0, n - 1})
        rest = sorted((j for j in range(n) if j not in forced), key=lambda j: (-score[j], j))
        ids = sorted((forced + rest)[:s["case"]["select"]])
        lists.append(ids + [-1] * (s["case"]["select"] - len(ids)))
        rows = torch.cat([torch.arange(j * BLOCK, min(ctx, (j + 1) * BLOCK), device="cuda") for j in ids])
        p = torch.softmax(s["q"][b].to(f64) @ s["k"][b, rows].to(f64).T * SCALE, -1)
        outs.append(p @ s["v"][b, rows].to(f64))
    return torch.tensor(lists, dtype=torch.int32, device="cuda"), torch.stack(outs)


def _exact_summaries(s):
    codes, scales = s["codes"].clone(), s["scales"].to(torch.float64)
    third = torch.tensor(1.0 / 127.0, dtype=torch.float32, device="cuda")
    for b, ctx in enumerate(s["ctx"].tolist()):
        first, last = -(-(ctx - s["case"]["new"] + 1) // BLOCK), ctx // BLOCK   # block ends in (ctx - new, ctx]
        lo, hi = max(0, first - 1), last
        if hi <= lo:
            continue
        x = s["k"][b, lo * BLOCK:hi * BLOCK].float().view(hi - lo, BLOCK, DIM)
        both = torch.stack((x.max(1).values, x.min(1).values), 1)
        top = both.abs().flatten(1).max(1).values
        codes[b, lo:hi] = (both / (top * third)[:, None, None]).round().to(torch.int8)
        scales[b, lo:hi] = top.to(torch.float64) / 127
    return codes, scales


def exact(case, seed):
    state = prepare(case, seed)
    return {"norm_rope": _exact_norm_rope, "prefix": _exact_prefix, "blocks": _exact_blocks,
            "summaries": _exact_summaries}[case["op"]](state)
