"""The operators around a chunk of new tokens over the paged latent cache, as
cases to measure: the chunk's attention (the rows of any number of new tokens a
request, causal, over every cached row), the weight that its queries or a decode
step's give to each cached row, and the eviction of the rows that got least.

`run` computes each in its plain form (elementary torch operations) or, with
`own` set, through the framework's entry points.  `exact` is the same in 64
bits, written from the definitions.
"""
import math

import numpy as np
import torch

own = False

LATENT, ROPE = 512, 64
WIDTH = LATENT + ROPE                     # one cached row, and one absorbed query
ROW_BYTES = {"bf16": 2 * WIDTH, "fp8": WIDTH + WIDTH // 32, "fp4": WIDTH // 2 + WIDTH // 16}
SCALE = 1.0 / 16.0                        # 1 / sqrt(192 + 64), the width of an un-absorbed head
E4M3 = torch.float8_e4m3fn
E8M0 = torch.float8_e8m0fnu


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _chunk(requests, chunk, context, heads=20, cache="bf16", page=64, ragged=False, padded=0, **kw):
    """`chunk` new tokens of each request behind `context` cached ones (about
    as many where ragged); `padded` token rows that belong to no request."""
    return dict(op="chunk", requests=requests, chunk=chunk, context=context, heads=heads, cache=cache,
                page=page, ragged=ragged, padded=padded, **kw)


def _weights(requests, chunk, context, heads=20, cache="bf16", page=64, ragged=False, **kw):
    """The last `chunk` tokens' queries over everything cached."""
    return dict(op="weights", requests=requests, chunk=chunk, context=context, heads=heads, cache=cache,
                page=page, ragged=ragged, padded=0, **kw)


def _evict(requests, context, budget, sinks, recent, cache="bf16", page=64, ragged=False, again=False, **kw):
    """`context` cached rows of each request cut to `budget`; again: a cache
    whose slots are out of order from earlier evictions."""
    return dict(op="evict", requests=requests, context=context, budget=budget, sinks=sinks, recent=recent,
                cache=cache, page=page, ragged=ragged, again=again, **kw)


def listed():
    return [
        # a short follow-up in a dialogue, a small model's few heads, small pages
        _chunk(1, 5, 700, heads=4, page=16, name="chunk: 5 tokens behind 700"),
        # one chunk of a prompt in the middle of its prefill
        _chunk(1, 512, 8192, name="chunk: 512 tokens behind 8192"),
        # the last chunk of a long prompt
        _chunk(1, 2048, 14336, name="chunk: 2048 tokens behind 14336"),
        # many users' turns of uneven lengths in one batch, an FP8 cache
        _chunk(24, 101, 2600, cache="fp8", ragged=True, padded=13, name="chunk: 24 requests, FP8"),
        # two whole prompts at once, nothing cached before them, an FP4 cache
        _chunk(2, 1283, 0, heads=32, cache="fp4", page=128, ragged=True, name="chunk: whole prompts, FP4"),
        # a decode step's weights, added up step by step
        _weights(64, 1, 4608, ragged=True, name="weights: decode step of 64"),
        # the end of a long prompt looks back over all of it
        _weights(1, 64, 32768, page=128, name="weights: last 64 of 32768"),
        # a step with two drafts over an FP8 cache
        _weights(17, 2, 1500, heads=16, cache="fp8", ragged=True, name="weights: drafts, FP8"),
        # a long prompt cut to what its end looked at
        _evict(1, 32768, 4096, 4, 64, name="evict: prompt 32768 to 4096"),
        # a decode batch whose caches have grown 64 tokens over their budget
        _evict(64, 4160, 4096, 4, 256, cache="fp8", again=True, name="evict: batch of 64, FP8"),
        # short contexts, some below the budget, small pages, FP4
        _evict(5, 240, 128, 1, 17, cache="fp4", page=16, ragged=True, name="evict: short contexts, FP4"),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("chunk", "chunk", "weights", "evict"))
    cache, page = rng.choice(("bf16", "bf16", "fp8", "fp4")), rng.choice((16, 32, 64, 128))
    ragged = rng.random() < 0.6
    if op == "chunk":
        heads = rng.choice((1, 4, 8, 16, 20, 20, 32))
        requests = _log(rng, 1, 32)
        chunk = _log(rng, 1, 2048 // requests)
        # a batch is padded to its longest request in the plain form: half of the largest case's scores
        context = _log(rng, 1, min(16384, 2 * 10**8 // (requests * chunk * heads), 200000 // requests)) - 1
        return _chunk(requests, chunk, context, heads, cache, page, ragged, rng.choice((0, 0, 9)))
    if op == "weights":
        heads = rng.choice((1, 4, 8, 16, 20, 20, 32))
        requests = _log(rng, 1, 64)
        chunk = _log(rng, 1, max(1, 96 // requests))
        context = _log(rng, 1, min(32768, 250000 // requests))
        return _weights(requests, chunk, context, heads, cache, page, ragged)
    requests = _log(rng, 1, 64)
    context = _log(rng, 2, min(65536, 250000 // requests))
    budget = max(1, int(context * rng.choice((0.1, 0.25, 0.5, 0.9, 1.0))) - rng.randint(0, 3))
    recent = rng.choice((0, 1, budget // 8, budget // 2))
    return _evict(requests, context, budget, rng.choice((0, 1, 4)), recent, cache, page, ragged,
                  rng.random() < 0.5)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _spread(rng, mean, count, ragged, reach):
    """`count` lengths, their sum count * mean: where ragged, up to `reach` of
    the mean away from it."""
    n = np.full(count, mean)
    if ragged:
        d = rng.integers(0, int(mean * reach) + 1, count // 2)
        n[:len(d)] += d
        n[len(d):2 * len(d)] -= d
        rng.shuffle(n)
    return n


def _pool(kind, pool, page, g):
    """A cache pool in use: every slot holds a row of values of order one."""
    slots = pool * page
    if kind == "bf16":
        return torch.randn(pool, page, WIDTH, generator=g, device="cuda", dtype=torch.bfloat16)
    raw = torch.randint(0, 256, (slots, ROW_BYTES[kind]), generator=g, device="cuda", dtype=torch.uint8)
    codes = WIDTH if kind == "fp8" else WIDTH // 2
    if kind == "fp8":                     # magnitudes below 2 before the scale, no NaN
        raw[:, :codes] = (raw[:, :codes] & 0x80) | (raw[:, :codes] & 0x3F)
    raw[:, codes:] = 124 + raw[:, codes:] % 4
    return raw.view(pool, page * ROW_BYTES[kind])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(int(torch.randint(1 << 31, (1,), generator=g, device="cuda")))
    put = lambda a, t=np.int32: torch.from_numpy(np.ascontiguousarray(a, dtype=t)).cuda()  # noqa: E731
    rand = lambda *s, dtype=torch.bfloat16: torch.randn(*s, generator=g, device="cuda", dtype=dtype)  # noqa: E731
    B, P, evict = case["requests"], case["page"], case["op"] == "evict"
    # chunks down to none at all: a request of the batch without a new token
    new = np.zeros(B, dtype=np.int64) if evict else _spread(
        rng, case["chunk"], B, case["ragged"], 1.0 if case["op"] == "chunk" else 0.5)
    lens = new + _spread(rng, case["context"], B, case["ragged"], 0.5)
    most_new = int(new.max())
    # what the program's arrays are sized for: the most that any lengths of the case come to
    longest = case["context"] + case.get("chunk", 0)
    if case["ragged"]:
        longest = case["context"] + int(case["context"] * 0.5) + 2 * case.get("chunk", 0)
    pages = -(-lens // P)
    pool = -(-int(case["context"] + case.get("chunk", 0)) * B // P) + 2 * B + 1  # as many as any seed's requests can take
    order = rng.permutation(pool)
    table = np.zeros((B, -(-longest // P)), dtype=np.int32)
    for b, (first, k) in enumerate(zip(np.cumsum(pages) - pages, pages)):
        table[b, :k] = order[first:first + k]
    s = dict(case=case, stream=torch.cuda.current_stream(), pool=pool, longest=longest,
             most_new=most_new, cached=int(lens.sum()), lens=put(lens), block_table=put(table),
             cache=_pool(case["cache"], pool, P, g), grid=torch.tensor(E2M1, device="cuda"))
    S = longest
    if evict:
        # attention's weights: a few rows with most of it, many with none
        w = (1.5 * rand(B, S, dtype=torch.float32)).exp()
        s["weights"] = torch.where(w < 0.3, torch.zeros_like(w), w)
        place = np.broadcast_to(np.arange(S), (B, S)).copy()
        if case["again"]:                 # what was kept before stands in any order, what came since behind it
            old = max(0, min(case["budget"], int(lens.min())))
            gone = 2 * S
            for b in range(B):
                kept = np.sort(rng.choice(gone, old, replace=False))
                kept[:1] = 0
                place[b] = gone + np.arange(S)
                place[b, :old] = rng.permutation(kept)
        s["positions"] = put(place)
        s["weights_out"], s["positions_out"] = torch.zeros_like(s["weights"]), torch.zeros_like(s["positions"])
        s["lens_out"] = torch.zeros_like(s["lens"])
    else:
        H, T = case["heads"], int(new.sum()) + case["padded"]
        s["starts"] = put(np.concatenate([[0], np.cumsum(new)]))
        q = rand(T, H, WIDTH)
        q[..., :LATENT] *= 0.61           # absorbed from 192 values through weights of variance 1 / 512
        s["q"], s["live"] = q, int(new.sum())
        if case["op"] == "chunk":
            s["o"] = torch.zeros(T, H, LATENT, device="cuda", dtype=torch.bfloat16)
            s["lse"] = torch.zeros(T, H, device="cuda")
        else:                             # what the attention left: scores have a variance of about one
            mean = put(np.repeat(np.log(np.maximum(lens, 1)), new), np.float32)
            s["lse"] = mean[:, None] + 0.5 + 0.05 * rand(T, H, dtype=torch.float32)
            s["weights"] = rand(B, S, dtype=torch.float32).abs()
            s["weights_out"] = torch.zeros_like(s["weights"])
    if own:
        s["calls"] = _handles(s)
    return s


# --------------------------------------------------------------------------
# the framework's operators
# --------------------------------------------------------------------------
def _handles(s):
    """The plan and the workspace that a program keeps."""
    import head_latent_attention_paged_gb300 as m
    case = s["case"]
    kv = {"bf16": m.MLA_KV_BF16, "fp8": m.MLA_KV_FP8_E4M3_E8M0, "fp4": m.MLA_KV_FP4_E2M1_E8M0}[case["cache"]]
    problem = m.make_problem(case["requests"], 1, case.get("heads", 1), case["page"], s["pool"],
                             s["block_table"].shape[1], kv_dtype=kv, sm_scale=SCALE)
    if case["op"] == "evict":
        plan = m.mla_evict_make_plan(problem, budget=case["budget"], sinks=case["sinks"], recent=case["recent"])
    else:
        plan = m.mla_chunk_make_plan(problem, tokens=s["q"].shape[0], context_tokens=s["cached"])
    return m, plan, torch.zeros(int(plan.workspace_bytes), dtype=torch.uint8, device="cuda")


def _own_chunk(s):
    m, plan, workspace = s["calls"]
    m.mla_chunk_attend(plan, s["q"], s["starts"], s["cache"], s["block_table"], s["lens"], workspace,
                       s["o"], s["lse"], stream=s["stream"])


def _own_weights(s):
    m, plan, workspace = s["calls"]
    m.mla_cache_weights(plan, s["q"], s["lse"], s["starts"], s["cache"], s["block_table"], s["lens"], workspace,
                        s["weights_out"], weights_in=s["weights"], stride=s["longest"], stream=s["stream"])


def _own_evict(s):
    m, plan, workspace = s["calls"]
    m.mla_cache_evict(plan, s["cache"], s["block_table"], s["lens"], s["weights"], s["positions"], workspace,
                      s["lens_out"], s["weights_out"], s["positions_out"], stride=s["longest"],
                      stream=s["stream"])


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------
E2M1 = (0., .5, 1., 1.5, 2., 3., 4., 6., -0., -.5, -1., -1.5, -2., -3., -4., -6.)


def _slots(s, places):
    """The pool slots of logical slots [B, n] of each request."""
    P = s["case"]["page"]
    return s["block_table"].long().gather(1, places // P) * P + places % P


def _rows(s):
    """Every request's cached rows in 32 bits, [B, longest, 576] (a request's
    first row again behind its last), and which of them it has."""
    kind = s["case"]["cache"]
    at = torch.arange(s["longest"], device="cuda")
    live = at < s["lens"][:, None]
    slots = _slots(s, at * live)
    if kind == "bf16":
        return s["cache"].view(-1, WIDTH)[slots].float(), live
    raw = s["cache"].view(-1, ROW_BYTES[kind])[slots]
    if kind == "fp8":
        v, e = raw[..., :WIDTH].view(E4M3).float(), raw[..., WIDTH:]
    else:
        byte, e = raw[..., :WIDTH // 2], raw[..., WIDTH // 2:]
        v = s["grid"][torch.stack((byte & 15, byte >> 4), -1).flatten(-2).long()]
    v = torch.ldexp(v.unflatten(-1, (e.shape[-1], -1)), e.int()[..., None] - 127).flatten(-2)
    return v, live


def _scores(s):
    """Scores [B, new * heads, longest] of every request's padded queries (the
    masked ones -inf), the rows, the packed token of each padded one, and the
    padded place of each packed one."""
    case, starts = s["case"], s["starts"].long()
    new = starts[1:] - starts[:-1]
    j = torch.arange(s["most_new"], device="cuda")
    there = j < new[:, None]
    token = (starts[:-1, None] + j) * there
    rows, live = _rows(s)
    q = s["q"][token].float().flatten(1, 2)
    scores = torch.matmul(q, rows.transpose(1, 2)).mul_(SCALE)
    last = (s["lens"] - new)[:, None] + j                # the last row that a token sees
    at = torch.arange(s["longest"], device="cuda")
    seen = (at <= last[..., None]) & live[:, None] & there[..., None]
    view = scores.unflatten(1, (-1, case["heads"]))
    view.masked_fill_(~seen[:, :, None], -math.inf)
    packed = torch.arange(s["live"], device="cuda")
    b = torch.searchsorted(starts, packed, right=True) - 1
    return scores, rows, token, b * s["most_new"] + packed - starts[b]


def _plain_chunk(s):
    scores, rows, _, place = _scores(s)
    top = scores.amax(-1, keepdim=True).clamp_(min=-1e30)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, rows[..., :LATENT]) / total.clamp(min=1e-30)
    lse = (top + total.log()).squeeze(-1)
    heads = s["case"]["heads"]
    s["o"][:s["live"]] = o.view(-1, heads, LATENT)[place].to(torch.bfloat16)
    s["lse"][:s["live"]] = lse.view(-1, heads)[place]


def _plain_weights(s):
    scores, _, token, _ = _scores(s)
    p = scores.sub_(s["lse"][token].flatten(1)[..., None]).exp_()
    at = torch.arange(s["longest"], device="cuda")
    torch.where(at < s["lens"][:, None], s["weights"] + p.sum(1), s["weights_out"], out=s["weights_out"])


def _plain_evict(s):
    case, w, place = s["case"], s["weights"], s["positions"]
    at = torch.arange(s["longest"], device="cuda")
    live = at < s["lens"][:, None]
    newest = torch.where(live, place, -1).amax(1, keepdim=True)
    safe = (place < case["sinks"]) | (place > newest - case["recent"])
    rank = torch.where(safe, math.inf, w).masked_fill_(~live, -math.inf)
    order = torch.sort(rank, dim=1, descending=True, stable=True).indices     # ties: the lowest slot first
    left = s["lens"].clamp(max=case["budget"])[:, None]
    kept = torch.zeros_like(live).scatter_(1, order, at < left)
    hole, moved = ~kept & (at < left), kept & (at >= left)
    source = torch.argsort((~moved).byte(), dim=1, stable=True)               # moved slots, ascending, first
    origin = torch.where(hole, source.gather(1, (hole.cumsum(1) - 1).clamp(min=0)), at)
    n = min(case["budget"], s["longest"])
    inside = at[:n] < left                                                    # the others' rows stay in place
    flat = s["cache"].view(-1, WIDTH if case["cache"] == "bf16" else ROW_BYTES[case["cache"]])
    flat[_slots(s, at[:n] * inside)] = flat[_slots(s, origin[:, :n] * inside)]
    w, place = w.gather(1, origin), place.gather(1, origin)
    freed = live & (at >= left)
    w.masked_fill_(freed, 0.0)
    place.masked_fill_(freed, -1)
    torch.where(live, w, s["weights_out"], out=s["weights_out"])
    torch.where(live, place, s["positions_out"], out=s["positions_out"])
    s["lens_out"].copy_(left[:, 0])


def run(state):
    case, op = state["case"], state["case"]["op"]
    if op == "chunk":
        _own_chunk(state) if own else _plain_chunk(state)
        return {"o": state["o"], "lse": state["lse"]}
    if op == "weights":
        _own_weights(state) if own else _plain_weights(state)
        return {"weights": state["weights_out"]}
    _own_evict(state) if own else _plain_evict(state)
    got = {"lens": state["lens_out"], "weights": state["weights_out"], "positions": state["positions_out"]}
    if case["cache"] == "bf16":
        return got | {"cache": state["cache"]}
    flat = state["cache"].view(-1, ROW_BYTES[case["cache"]])
    if case["cache"] == "fp8":
        return got | {"codes": flat[:, :WIDTH].view(E4M3), "scales": flat[:, WIDTH:].view(E8M0)}
    byte = flat[:, :WIDTH // 2].int()     # the values that the 4-bit codes stand for
    return got | {"codes": state["grid"][torch.stack((byte & 15, byte >> 4), -1).flatten(1)],
                  "scales": flat[:, WIDTH // 2:].view(E8M0)}


# --------------------------------------------------------------------------
# work
# --------------------------------------------------------------------------
def work(case):
    """Each input read once, each output written once; 576 + 512 products for
    each head of a new token and each row that it sees (576 for its weight)."""
    B, row = case["requests"], ROW_BYTES[case["cache"]]
    if case["op"] == "evict":
        # of the rows below the budget, the share that is not kept is filled from behind
        n, k = case["context"], min(case["budget"], case["context"])
        moved = k * (1 - k / n)
        return {"bytes": int(B * (16 * n + 2 * row * moved)), "flops": B * n}
    new, n = case["chunk"], case["chunk"] + case["context"]
    pairs = B * case["heads"] * (new * n - new * (new - 1) // 2)
    moved = B * (n * row + new * case["heads"] * (2 * WIDTH + 4))
    if case["op"] == "chunk":
        return {"bytes": moved + B * new * case["heads"] * 2 * LATENT, "flops": pairs * 2 * (WIDTH + LATENT)}
    return {"bytes": moved + 8 * B * n, "flops": pairs * 2 * WIDTH}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def _x_row_values(s, slots):
    kind = s["case"]["cache"]
    if kind == "bf16":
        return s["cache"].view(-1, WIDTH)[slots].double()
    raw = s["cache"].view(-1, ROW_BYTES[kind])[slots]
    n = WIDTH if kind == "fp8" else WIDTH // 2
    if kind == "fp8":
        b = raw[:, :n].int()
        exp, man = (b >> 3) & 15, (b & 7).double()
        v = torch.where(exp > 0, torch.exp2((exp - 7).double()) * (1 + man / 8), man / 512)
        v = torch.where(b >= 128, -v, v)
    else:
        b = torch.stack((raw[:, :n] % 16, raw[:, :n] // 16), -1).flatten(1).int()
        exp, man = (b >> 1) & 3, (b & 1).double()
        v = torch.where(exp > 0, torch.exp2((exp - 1).double()) * (1 + man / 2), man / 2)
        v = torch.where(b >= 8, -v, v)
    groups = raw.shape[1] - n
    return (v.unflatten(-1, (groups, -1)) * torch.exp2(raw[:, n:].double() - 127)[..., None]).flatten(1)


def _x_attention(case, s):
    starts, lens = s["starts"].tolist(), s["lens"].tolist()
    H, P = case["heads"], case["page"]
    if case["op"] == "chunk":
        o, lse = s["o"].double(), s["lse"].double()
    else:
        total = s["weights_out"].double()
    for b in range(case["requests"]):
        first, end, n = starts[b], starts[b + 1], lens[b]
        t = torch.arange(n, device="cuda")
        rows = _x_row_values(s, s["block_table"][b].long()[t // P] * P + t % P)
        if case["op"] == "weights":
            total[b, :n] = s["weights"][b, :n].double()
        step = max(1, 2**27 // (H * max(n, 1)))
        for k in range(first, end, step):
            k2 = min(end, k + step)
            z = torch.einsum("jhd,td->jht", s["q"][k:k2].double(), rows) / 16
            hidden = t[None] > (torch.arange(k, k2, device="cuda") - end + n)[:, None]
            if case["op"] == "chunk":
                z = z.masked_fill(hidden[:, None], -math.inf)
                lse[k:k2] = torch.logsumexp(z, -1)
                o[k:k2] = torch.einsum("jht,td->jhd", torch.softmax(z, -1), rows[:, :LATENT])
            else:
                p = (z - s["lse"][k:k2].double()[..., None]).exp().masked_fill(hidden[:, None], 0.0)
                total[b, :n] += p.sum((0, 1))
    return {"o": o, "lse": lse} if case["op"] == "chunk" else {"weights": total}


def _x_evict(case, s):
    lens, P = s["lens"].tolist(), case["page"]
    w, place = s["weights"].double().cpu().numpy(), s["positions"].cpu().numpy()
    w_out, place_out = s["weights_out"].double().cpu().numpy(), s["positions_out"].cpu().numpy()
    left, to, fro = [], [], []
    table = s["block_table"].cpu().numpy().astype(np.int64)
    for b, n in enumerate(lens):
        k = min(n, case["budget"])
        p = place[b, :n]
        safe = (p < case["sinks"]) | (p > p.max() - case["recent"])
        best = np.lexsort((np.arange(n), np.where(safe, -np.inf, -w[b, :n])))[:k]
        take = np.zeros(n, dtype=bool)
        take[best] = True
        origin = np.arange(k)
        origin[~take[:k]] = np.flatnonzero(take[k:]) + k
        w_out[b, :k], place_out[b, :k] = w[b, origin], p[origin]
        w_out[b, k:n], place_out[b, k:n] = 0.0, -1
        left.append(k)
        moved = np.flatnonzero(origin != np.arange(k))
        to.append(table[b][moved // P] * P + moved % P)
        fro.append(table[b][origin[moved] // P] * P + origin[moved] % P)
    put = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    to, fro = put(np.concatenate(to)), put(np.concatenate(fro))
    every = torch.arange(s["pool"] * P, device="cuda")
    every[to] = fro
    got = {"lens": put(np.array(left, dtype=np.int32)), "weights": put(w_out), "positions": put(place_out)}
    if case["cache"] == "bf16":
        return got | {"cache": _x_row_values(s, every).view(s["cache"].shape)}
    raw = s["cache"].view(-1, ROW_BYTES[case["cache"]])[every]
    n = WIDTH if case["cache"] == "fp8" else WIDTH // 2
    scales = torch.exp2(raw[:, n:].double() - 127)
    if case["cache"] == "fp8":
        return got | {"codes": raw[:, :n].view(E4M3).double(), "scales": scales}
    code = torch.stack((raw[:, :n] % 16, raw[:, :n] // 16), -1).flatten(1).int()
    a = torch.where((code & 7) < 2, (code & 7) * 0.5, torch.exp2(((code >> 1) & 3).double() - 1) * (1 + (code & 1) * 0.5))
    return got | {"codes": torch.where(code >= 8, -a, a.double()), "scales": scales}


def exact(case, seed):
    global own
    own, kept = False, own
    s = prepare(case, seed)
    own = kept
    return _x_evict(case, s) if case["op"] == "evict" else _x_attention(case, s)
