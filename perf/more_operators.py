"""Cases for the operators around the linear layers of a rollout and of a training step: the residual addition with RMS
norm and quantization and its backward pass, rotary positions, the attention of samples that share a prompt, and the
page operations of the key/value cache (fork, sweep, compaction).

Definitions (shared by the plain form, `exact` and the library):
  * norm: h = bf16(x + residual), r = 1 / sqrt(mean(h^2) + eps) in fp32, y = bf16((h r) w), then y's codes in groups of
    1x128.  Its backward pass, with g = dy w: dx = r (g - h r^2 mean(g h)) + dres, dw = sum over the rows of dy h r;
  * rotary: pair i of a head's first 2 P channels, (i, P + i) or (2 i, 2 i + 1), turns by position * freqs[i];
  * cache: blocks of 64 tokens as in operators.py.  Consecutive requests with the same group id share the leading blocks
    of their tables; a unit's record in `prefix` is (first unit of its group, units, shared blocks, 0), shared blocks
    being a multiple of 8;
  * fork: request r becomes a copy of request parents[r] (-1: stays); sweep: the free list is what no live request's
    table holds, ascending; compaction: the live blocks at or above the number L of live blocks, ascending, move into the
    free ids below L, ascending.
"""
import math
import random

import torch

own = False

BLOCK = 64
SPAN = 8
EPS = 1e-5


# ------------------------------------------------------------------------------------------------ cases
def listed():
    a = dict(q_heads=32, kv_heads=8, head_dim=128)     # the heads of the repository's 4096 -> 6144 qkv linear
    b = dict(q_heads=40, kv_heads=8, head_dim=128)     # and of its 5120 -> 7168 one
    return [
        # in front of a linear layer in one decode step: latency
        dict(name="norm 32 x 5120", kind="norm", rows=32, cols=5120),
        # the same in the large training step: bandwidth
        dict(name="norm 65536 x 5120", kind="norm", rows=65536, cols=5120),
        # the backward pass of the 8 x 2048 token training step
        dict(name="norm backward 16384 x 4096", kind="norm_back", rows=16384, cols=4096),
        # queries and keys of a decode step
        dict(name="rotary 32 single tokens", kind="rotary", tokens=32, far=4096, pairs=64, interleaved=False,
             inverse=False, packed=False, **a),
        # their gradients in the training step, four sequences
        dict(name="rotary backward 65536 tokens", kind="rotary", tokens=65536, far=16384, pairs=64, interleaved=True,
             inverse=True, packed=True, **b),
        # part of narrow heads, far positions, an odd number of rows
        dict(name="rotary part of 1001 rows", kind="rotary", tokens=1001, far=1 << 20, pairs=16, interleaved=False,
             inverse=False, packed=False, q_heads=16, kv_heads=16, head_dim=64),
        # one prompt with a few samples: latency
        dict(name="8 samples of a prompt of 2000", kind="attend", prompts=1, samples=8, prompt=2000, grown=300, new=1,
             idle=0, **a),
        # a rollout batch, 16 samples of each of 16 prompts
        dict(name="16 samples of 16 prompts of 8192", kind="attend", prompts=16, samples=16, prompt=8192, grown=1024,
             new=1, idle=0, **a),
        # many samples of few prompts, several tokens at once, some samples finished, narrow heads
        dict(name="48 samples of 3 prompts, 3 tokens, some idle", kind="attend", prompts=3, samples=48, prompt=5000,
             grown=700, new=3, idle=7, q_heads=16, kv_heads=8, head_dim=64),
        # a batch's samples take over from one another (beam search, resampling), and one layer's unfinished blocks
        dict(name="fork 256 requests", kind="fork", requests=256, ctx=4096, kv_heads=8, head_dim=128),
        # requests have ended: the blocks that nobody holds any more
        dict(name="sweep 1000 requests", kind="sweep", requests=1000, ctx=8192, kv_heads=0, head_dim=0),
        # the cache is made smaller before training: tables, free list and one layer's blocks
        dict(name="compact 128 requests", kind="compact", requests=128, ctx=4096, kv_heads=8, head_dim=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "norm_back", "rotary", "rotary", "attend", "attend", "attend", "fork", "sweep", "compact"])
    heads = lambda: (lambda kv: dict(kv_heads=kv, q_heads=kv * rng.randint(1, 8), head_dim=rng.choice([64, 128, 128])))(
        rng.choice([1, 2, 4, 8, 8, 16]))
    while True:
        if kind in ("norm", "norm_back"):
            c = dict(kind=kind, rows=_log(rng, 1, 65536), cols=128 * rng.randint(1, 64))
            if c["rows"] * c["cols"] <= (65536 * 5120 if kind == "norm" else 65536 * 4096):
                return c
        elif kind == "rotary":
            c = dict(kind=kind, tokens=_log(rng, 1, 65536), far=_log(rng, 64, 1 << 20), interleaved=rng.random() < 0.5,
                     inverse=rng.random() < 0.5, packed=rng.random() < 0.5, **heads())
            c["pairs"] = 8 * rng.randint(1, c["head_dim"] // 16)
            if c["tokens"] * (c["q_heads"] + c["kv_heads"]) * c["head_dim"] <= 65536 * 48 * 128:
                return c
        elif kind == "attend":
            c = dict(kind=kind, prompts=_log(rng, 1, 32), samples=rng.randint(2, 64), prompt=_log(rng, 16, 32768),
                     grown=_log(rng, 1, 4096), new=rng.choice([1, 1, 1, rng.randint(2, 9)]),
                     idle=rng.choice([0, 0, rng.randint(2, 9)]), **heads())
            _, pairs = _requests(c)
            seen = sum(n * (x + n) for x, n in pairs)
            rows = c["prompts"] * c["samples"] * c["kv_heads"]
            if rows * (c["grown"] + c["new"] + 64) <= 1 << 22 and seen * c["q_heads"] <= 1 << 27 and \
                    c["prompts"] * c["prompt"] * c["kv_heads"] <= 1 << 20:
                return c
        else:
            c = dict(kind=kind, requests=_log(rng, 1, 1000 if kind == "sweep" else 256), ctx=_log(rng, 1, 16384), kv_heads=0,
                     head_dim=0)
            if kind != "sweep":
                c |= dict(kv_heads=rng.choice([1, 2, 4, 8]), head_dim=rng.choice([64, 128]))
            if kind == "sweep" or kind == "fork" and c["requests"] * c["kv_heads"] <= 2048 or \
                    c["requests"] * c["ctx"] * c["kv_heads"] <= 1 << 22:
                return c


def _requests(c):
    """(prompt length of each group), (tokens so far, new tokens) of each request: the prompts between half of the
    case's bound and the bound, the samples' own tokens spread evenly; every idle-th sample has no new tokens."""
    G, n = c["prompts"], c["samples"]
    R = G * n
    prompts = [c["prompt"] - i * c["prompt"] // (2 * G) for i in range(G)]
    step = next(s for s in range(R // 2 + 1, 2 * R + 2) if math.gcd(s, R) == 1)
    pairs = []
    for r in range(R):
        own_tokens = (2 * (r * step % R) + 1) * c["grown"] // (2 * R)
        pairs.append((prompts[r // n] + own_tokens, 0 if c["idle"] and r % c["idle"] == c["idle"] - 1 else c["new"]))
    return prompts, pairs


def max_units(tokens, requests):
    return min(tokens, (tokens + 62 * requests) // BLOCK + requests)


# ------------------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return {"norm": _prepare_norm, "norm_back": _prepare_norm, "rotary": _prepare_rotary, "attend": _prepare_attend,
            "fork": _prepare_pages, "sweep": _prepare_pages, "compact": _prepare_pages}[case["kind"]](case, seed, g)


def _randn(shape, g):
    return torch.randn(shape, device="cuda", generator=g)


def _prepare_norm(c, seed, g):
    R, C = c["rows"], c["cols"]
    loud = torch.where(torch.rand((C,), device="cuda", generator=g) < 0.002, 50.0, 1.0)   # outlier channels
    s = dict(kind=c["kind"], weight=(1 + 0.1 * _randn((C,), g)).to(torch.bfloat16))
    x, res = (_randn((R, C), g) * loud).to(torch.bfloat16), (4 * _randn((R, C), g) * loud).to(torch.bfloat16)
    if c["kind"] == "norm":
        return s | dict(x=x, residual=res)
    del x
    # a gradient's heavy tails
    dy = (1e-3 * _randn((R, C), g) / (0.1 + torch.rand((R, C), device="cuda", generator=g))).to(torch.bfloat16)
    dres = (1e-3 * _randn((R, C), g)).to(torch.bfloat16)
    rstd = torch.empty((R,), device="cuda")
    for i in range(0, R, 8192):
        rstd[i:i + 8192] = (1 / torch.sqrt(res[i:i + 8192].double().square().mean(1) + EPS)).float()
    return s | dict(dy=dy, h=res, dres=dres, rstd=rstd)


def _prepare_rotary(c, seed, g):
    T, H, D, P = c["tokens"], c["q_heads"] + c["kv_heads"], c["head_dim"], c["pairs"]
    # queries and keys are columns of the qkv projection's output, or (packed: gradients) a matrix of their own
    x = _randn((T, H + (0 if c["packed"] else c["kv_heads"]), D), g).to(torch.bfloat16)[:, :H]
    if c["packed"]:       # sequences of a training step, one after the other
        positions = torch.arange(T, device="cuda", dtype=torch.int32) % c["far"]
    else:
        positions = torch.randint(0, c["far"], (T,), device="cuda", generator=g, dtype=torch.int32)
    # a long context's frequencies: positions of the slow half of the pairs closer together
    i = torch.arange(P, dtype=torch.float64, device="cuda")
    freqs = 10000.0 ** (-i / P) / torch.where(i < P // 2, 1.0, 4.0)
    return dict(kind="rotary", x=x, positions=positions, freqs=freqs, interleaved=c["interleaved"], inverse=c["inverse"],
                amplitude=1.0 if c["packed"] else 1.1)


def _places(D):
    """[64, D] indices of a block's values in memory: E4M3 keys, E4M3 values, bf16 keys, bf16 values."""
    n = torch.arange(BLOCK, device="cuda")[:, None]
    d = torch.arange(D, device="cuda")[None, :]
    k8 = ((n // 16 * (D // 64) + d // 64) * 64 + d % 32 // 8 * 16 + n % 16) * 16 + d % 64 // 32 * 8 + d % 8
    k16 = ((n // 16 * (D // 32) + d // 32) * 64 + d % 32 // 8 * 16 + n % 16) * 8 + d % 8
    j = n % 32 // 16 * 4 + n % 4
    v8 = (d // 16 * 64 + n % 16 // 4 * 16 + d % 16) * 16 + n // 32 * 8 + j
    v16 = ((d // 16 * 2 + n // 32) * 64 + n % 16 // 4 * 16 + d % 16) * 8 + j
    return k8, v8, k16, v16


def _fill_cache(blocks, recents, H, D, g):
    """A layer's codes, scales and recent blocks with random keys and values; a few key channels stand out."""
    k8, _, k16, _ = _places(D)
    gain = torch.where(torch.rand((H, D), device="cuda", generator=g) < 0.02, 6.0, 1.0)
    channel = torch.arange(D, device="cuda").expand(BLOCK, D)
    at8, at16 = (torch.empty(BLOCK * D, dtype=torch.long, device="cuda").scatter_(0, p.reshape(-1), channel.reshape(-1))
                 for p in (k8, k16))
    codes = torch.empty((blocks, H, 2, BLOCK * D), dtype=torch.uint8, device="cuda")
    scales = torch.empty((blocks, H, 2), device="cuda")
    step = max(1, (1 << 28) // (2 * H * BLOCK * D))
    for b in range(0, blocks, step):
        x = _randn((min(step, blocks - b), H, 2, BLOCK * D), g)
        x[:, :, 0] *= gain[:, at8]
        sc = x.abs().amax(3) / 448
        scales[b:b + step] = sc
        codes[b:b + step] = (x / sc[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    recent = _randn((recents, H, 2, BLOCK * D), g)
    recent[:, :, 0] *= gain[:, at16]
    return codes, scales, recent.to(torch.bfloat16)


def _prepare_attend(c, seed, g):
    Hq, H, D = c["q_heads"], c["kv_heads"], c["head_dim"]
    prompts, pairs = _requests(c)
    R, n = len(pairs), c["samples"]
    T = sum(m for _, m in pairs)
    ends = [(x + m) // BLOCK for x, m in pairs]                 # complete blocks after the step
    held = [p // BLOCK for p in prompts]
    blocks = sum(held) + sum(e - held[r // n] for r, e in enumerate(ends)) + 3
    width = max(ends) + 1
    order = torch.randperm(blocks, generator=g, device="cuda").tolist()
    table = [[-1] * width for _ in range(R)]
    at = 0
    for i, h in enumerate(held):
        for r in range(i * n, i * n + n):
            table[r][:h] = order[at:at + h]
        at += h
    for r, e in enumerate(ends):
        h = held[r // n]
        table[r][h:e] = order[at:at + e - h]
        at += e - h
    units, row, middle = [], 0, 0
    for r, (x, m) in enumerate(pairs):
        first, last = x // BLOCK, (x + m - 1) // BLOCK
        for j in range(first, last + 1 if m else first):
            lo, hi = max(x, j * BLOCK), min(x + m, (j + 1) * BLOCK)
            place = 2 * r + r % 2 if j == first else 2 * r + 1 - r % 2 if j == last else 2 * R + middle
            middle += first < j < last
            units.append((r, j, place, row + lo - x, hi - lo, lo - j * BLOCK,
                          table[r][j] if (j + 1) * BLOCK <= x + m else -1, 0))
        row += m
    prefix = []
    for i in range(c["prompts"]):
        mine = [k for k, u in enumerate(units) if u[0] // n == i]
        busy = len({units[k][0] for k in mine}) > 1
        shared = held[i] // SPAN * SPAN if busy else 0
        # requests whose own first blocks are still the prompt's only: those after it differ
        prefix += [(mine[0] if shared else k, len(mine) if shared else 1, shared, 0) for k in mine]
    total = max_units(T, R)
    pad = total - len(units)
    units = torch.tensor(units + [(-1,) * 8] * pad, dtype=torch.int32, device="cuda")
    prefix = torch.tensor(prefix + [(-1, 0, 0, 0)] * pad, dtype=torch.int32, device="cuda")
    codes, scales, recent = _fill_cache(blocks, 2 * R + T // BLOCK, H, D, g)
    # queries are columns of the qkv projection's output
    q = _randn((T, (Hq + 2 * H) * D), g).to(torch.bfloat16)[:, :Hq * D].unflatten(1, (Hq, D))
    return dict(kind="attend", q=q, units=units, table=torch.tensor(table, dtype=torch.int32, device="cuda"), prefix=prefix,
                codes=codes, scales=scales, recent=recent, max_new=c["new"], max_seq=max(x + m for x, m in pairs),
                ctx=torch.tensor([x for x, _ in pairs], device="cuda"), new=torch.tensor([m for _, m in pairs], device="cuda"),
                held=torch.tensor(held, device="cuda"), samples=n, longest=held[0],
                wide=max(e - held[r // n] for r, e in enumerate(ends)) + 1)


def _prepare_pages(c, seed, g):
    """A cache in the middle of a rollout: samples that share prompts, ended requests, blocks in random places."""
    R, ctx, kind = c["requests"], c["ctx"], c["kind"]
    rng = random.Random(seed)
    lens = [(2 * i + 1) * ctx // (2 * R) for i in range(R)]
    rng.shuffle(lens)
    group = 4
    width = max(lens) // BLOCK + 2
    need = sum(x // BLOCK for x in lens)
    blocks = need + need // 4 + 5
    order = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    length = torch.tensor(lens, device="cuda")
    full = length // BLOCK
    j = torch.arange(width, device="cuda")[None]
    starts = full.cumsum(0) - full
    table = order[(starts[:, None] + j).clamp(max=blocks - 1)]
    leader = torch.arange(R, device="cuda") // group * group
    common = torch.minimum(full, full[leader]) // 2                       # half of the shorter one is the prompt
    table = torch.where(j < common[:, None], table[leader], table)
    table = torch.where(j < full[:, None], table, -1).int()
    if kind != "fork":
        ended = torch.rand((R,), device="cuda", generator=g) < 0.3
        length = torch.where(ended, 0, length)                            # their rows keep what they held
    slot = torch.randint(0, 2, (R,), device="cuda", generator=g)
    s = dict(kind=kind, state=torch.stack([length, slot], 1).int(), table=table, blocks=blocks)
    if kind == "sweep":
        return s
    H, D = c["kv_heads"], c["head_dim"]
    if kind == "fork":
        keep = torch.rand((R,), device="cuda", generator=g) < 0.4
        parents = torch.randint(0, R, (R,), device="cuda", generator=g)
        _, _, recent = _fill_cache(1, 2 * R + 4, H, D, g)
        return s | dict(parents=torch.where(keep, -1, parents).int(), recent=recent)
    codes, scales, _ = _fill_cache(blocks, 1, H, D, g)
    return s | dict(codes=codes, scales=scales)


# ------------------------------------------------------------------------------------------------ the operators
def run(state):
    s, kind = state, state["kind"]
    if own:
        import fp8_precision_rl_amd as jf
        if kind == "norm":
            codes, scales, rstd, h = jf.rmsnorm_add_quantize(s["x"], s["residual"], s["weight"], EPS)
            return {"codes": codes.view(torch.float8_e4m3fn), "scales": scales, "rstd": rstd, "h": h}
        if kind == "norm_back":
            dx, dw = jf.rmsnorm_backward(s["dy"], s["h"], s["weight"], s["rstd"], s["dres"])
            return {"dx": dx, "dw": dw}
        if kind == "rotary":
            return jf.rotary(s["x"], s["positions"], s["freqs"], interleaved=s["interleaved"], amplitude=s["amplitude"],
                             inverse=s["inverse"])
        if kind == "attend":
            return jf.attention(s["q"], s["units"], s["table"], s["codes"], s["scales"], s["recent"],
                                max_new=s["max_new"], max_seq=s["max_seq"], prefix=s["prefix"])
        if kind == "fork":
            f = jf.kv_fork(s["state"], s["table"], s["parents"])
            jf.kv_fork_recent(s["parents"], s["state"], s["recent"])
            return {"state": f.next_state, "table": f.next_table, "recent": s["recent"]}
        p = jf.kv_sweep(s["state"], s["table"], s["blocks"], compact=kind == "compact")
        out = {"free": p.free_blocks, "head": p.free_head, "live": p.live}
        if kind == "compact":
            jf.kv_move(p.moves, s["codes"], s["scales"])
            out |= {"table": p.next_table, "moves": p.moves, "codes": s["codes"].view(torch.float8_e4m3fn),
                    "scales": s["scales"]}
        return out
    return {"norm": _norm, "norm_back": _norm_back, "rotary": _rotary, "attend": _attend, "fork": _fork, "sweep": _sweep,
            "compact": _sweep}[kind](s)


def _round_e4m3(x):
    """The nearest E4M3 value, ties to the even code, largest 448 (x in 64 bits)."""
    a = x.abs().clamp(min=2.0 ** -6)
    step = a / torch.frexp(a).mantissa / 16       # an eighth of the power of two at or below |x|
    return (torch.round(x / step) * step).clamp(-448, 448)


def _norm(s):
    x, w = s["x"], s["weight"].float()
    R, C = x.shape
    codes = torch.empty((R, C), dtype=torch.float8_e4m3fn, device=x.device)
    scales = torch.empty((C // 128, R), device=x.device)
    rstd = torch.empty((R,), device=x.device)
    h = torch.empty_like(x)
    for i in range(0, R, 16384):                  # in 64 bits: bounded in memory
        k = slice(i, i + 16384)
        h[k] = x[k].float() + s["residual"][k].float()
        f = h[k].float()
        r = (1 / torch.sqrt(f.double().square().mean(1) + EPS)).float()
        y = ((f * r[:, None]) * w).to(torch.bfloat16).double().view(-1, C // 128, 128)
        sc = (y.abs().amax(2) / 448).float()
        q = torch.where(sc[..., None] > 0, _round_e4m3(y / sc.double()[..., None]), y)
        codes[k] = q.view(-1, C).float().to(torch.float8_e4m3fn)
        scales[:, k] = sc.t()
        rstd[k] = r
    return {"codes": codes, "scales": scales, "rstd": rstd, "h": h}


def _norm_back(s):
    h, dy, r = s["h"].float(), s["dy"].float(), s["rstd"][:, None]
    g = dy * s["weight"].float()
    c = (g * h).sum(1, keepdim=True) / h.shape[1]
    dx = (r * (g - h * (r * r * c)) + s["dres"].float()).to(torch.bfloat16)
    return {"dx": dx, "dw": (dy * h * r).sum(0, dtype=torch.float64).float()}


def _rotary(s):
    x, P = s["x"], len(s["freqs"])
    angle = s["positions"].double()[:, None] * s["freqs"]
    cos, sin = ((f(angle) * s["amplitude"]).float()[:, None] for f in (torch.cos, torch.sin))
    if s["inverse"]:
        sin = -sin
    f = x.float()
    rot = f[..., :2 * P]
    a, b = (rot[..., 0::2], rot[..., 1::2]) if s["interleaved"] else (rot[..., :P], rot[..., P:])
    a, b = a * cos - b * sin, b * cos + a * sin
    rot = torch.stack([a, b], -1).flatten(2) if s["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([rot, f[..., 2 * P:]], -1).to(torch.bfloat16)


def _attend(s):
    """The prompts' keys once for all queries of a group, each sample's own beside them, one softmax over both."""
    q, codes, scales, recent = s["q"], s["codes"], s["scales"], s["recent"]
    T, Hq, D = q.shape
    H, N, R, n = codes.shape[1], s["max_new"], len(s["ctx"]), s["samples"]
    G, g, dev = R // n, Hq // codes.shape[1], q.device
    k8, v8, k16, v16 = _places(D)
    ctx, new, held = s["ctx"], s["new"], s["held"]
    row = new.cumsum(0) - new
    i = torch.arange(N, device=dev)
    rows = (row[:, None] + i[None]).clamp(max=T - 1)                                       # [R, N]
    pos = ctx[:, None] + i[None]
    mine = pos // BLOCK                                                                   # a query's own block
    Q = q[rows].float().view(R, N, H, g, D).permute(0, 2, 1, 3, 4).reshape(R, H, N * g, D)

    def cached(ids):
        ids = ids.long().clamp(min=0)
        x = codes[ids].view(torch.float8_e4m3fn).float() * scales[ids][..., None]          # [A, B, H, 2, 64 D]
        x = x.transpose(1, 2)
        return (x[:, :, :, i][..., p].flatten(2, 3) for i, p in ((0, k8), (1, v8)))        # [A, H, B * 64, D]

    most = s["longest"]
    K, V = cached(s["table"][::n, :most])
    S = [torch.matmul(Q.view(G, n, H, N * g, D).transpose(1, 2).reshape(G, H, n * N * g, D), K.transpose(2, 3))]
    S[0] = S[0].view(G, H, n, N * g, most * BLOCK).transpose(1, 2).reshape(R, H, N, g, most * BLOCK)
    there = torch.arange(most * BLOCK, device=dev)[None] < held[:, None] * BLOCK           # [G, keys]
    see = [there.repeat_interleave(n, 0)[:, None].expand(R, N, -1)]
    # the sample's own complete blocks, and the block of each new token
    first = held.repeat_interleave(n)
    j = first[:, None] + torch.arange(s["wide"], device=dev)                                    # [R, wide]
    ids = torch.gather(s["table"].long(), 1, j.clamp(max=s["table"].shape[1] - 1))
    K2, V2 = cached(ids)
    key = j.repeat_interleave(BLOCK, 1)[:, None]                                            # their blocks
    see.append(key < mine[:, :, None])
    S.append(torch.matmul(Q, K2.transpose(2, 3)).view(R, H, N, g, -1))
    spans = (BLOCK + N - 2) // BLOCK + 1                                                    # blocks that new tokens lie in
    unit = (((ctx + new - 1) // BLOCK - ctx // BLOCK + 1) * (new > 0)).cumsum(0)
    unit = unit - ((ctx + new - 1) // BLOCK - ctx // BLOCK + 1) * (new > 0)
    at = s["units"][:, 2].long().clamp(min=0)[(unit[:, None] + torch.arange(spans, device=dev)).clamp(max=len(s["units"]) - 1)]
    x = recent[at].float().transpose(1, 2)
    K3, V3 = (x[:, :, :, i][..., p].flatten(2, 3) for i, p in ((0, k16), (1, v16)))
    key = ((ctx // BLOCK)[:, None] + torch.arange(spans, device=dev))[..., None] * BLOCK + torch.arange(BLOCK, device=dev)
    key = key.flatten(1)[:, None]
    see.append((key // BLOCK == mine[:, :, None]) & (key <= pos[:, :, None]))
    S.append(torch.matmul(Q, K3.transpose(2, 3)).view(R, H, N, g, -1))
    P = torch.where(torch.cat(see, 2)[:, None, :, None], torch.cat(S, 4) * D ** -0.5, -math.inf)
    P = torch.exp(P - P.amax(-1, keepdim=True))
    P = (P / P.sum(-1, keepdim=True)).view(R, H, N * g, -1)
    A, B, C = P.split([x.shape[-1] for x in S], -1)
    O = torch.matmul(A.reshape(G, n, H, N * g, most * BLOCK).transpose(1, 2).reshape(G, H, n * N * g, most * BLOCK), V)
    O = O.view(G, H, n, N * g, D).transpose(1, 2).reshape(R, H, N * g, D)
    O = (O + torch.matmul(B, V2) + torch.matmul(C, V3)).view(R, H, N, g, D).transpose(1, 2).reshape(R * N, Hq, D)
    t = torch.arange(T, device=dev)
    r = torch.searchsorted(new.cumsum(0), t, right=True)
    return O[r * N + t - row[r]].to(torch.bfloat16)


def _fork(s):
    state, table, recent = s["state"], s["table"], s["recent"]
    R, width = table.shape
    r = torch.arange(R, device=table.device)
    p = s["parents"].long()
    moved = (p >= 0) & (p != r)
    p = torch.where(moved, p, r)
    next_state = torch.stack([state[p, 0], torch.where(moved, 1 - state[:, 1], state[:, 1])], 1)
    j = torch.arange(width, device=table.device)
    next_table = torch.where(j[None] < state[p, :1] // BLOCK, table[p], -1)
    to = torch.where(moved, 2 * r + next_state[:, 1], 2 * r + state[:, 1])
    recent[to] = recent[2 * p + state[p, 1]]
    return {"state": next_state, "table": next_table, "recent": recent}


def _sweep(s):
    state, table, n = s["state"], s["table"], s["blocks"]
    dev = table.device
    j = torch.arange(table.shape[1], device=dev)
    held = (j[None] < state[:, :1] // BLOCK) & (table >= 0)
    live = torch.zeros(n + 1, dtype=torch.bool, device=dev)
    live[torch.where(held, table, n).long().flatten()] = True
    live = live[:n]
    ids = torch.arange(n, device=dev, dtype=torch.int32)
    L = live.sum()
    compact = s["kind"] == "compact"
    free = ~live if not compact else ids >= L
    at = torch.where(free, free.cumsum(0) - 1, n)
    out = torch.full((n + 1,), -1, dtype=torch.int32, device=dev)
    out[at] = torch.where(free, ids, -1)
    res = {"free": out[:n], "head": torch.zeros(1, dtype=torch.int32, device=dev), "live": L.int().reshape(1)}
    if not compact:
        return res
    source, target = live & (ids >= L), ~live & (ids < L)
    moves = torch.full((n // 2 + 2, 2), -1, dtype=torch.int32, device=dev)
    last = n // 2 + 1
    for i, which in ((0, source), (1, target)):
        moves[torch.where(which, which.cumsum(0) - 1, last), i] = torch.where(which, ids, -1)
    moves = moves[:n // 2]
    to = torch.cat([ids, ids.new_full((1,), -1)])
    there = moves[:, 0] >= 0
    to[torch.where(there, moves[:, 0], n).long()] = torch.where(there, moves[:, 1], -1)
    m = moves[:, 0].long()
    codes, scales = s["codes"], s["scales"]
    # rows without a move copy a block onto itself
    source = torch.where(there, m, L)
    target = torch.where(there, moves[:, 1].long(), L)
    codes[target] = codes[source]
    scales[target] = scales[source]
    return res | {"table": torch.where(held, to[table.long()], -1), "moves": moves,
                  "codes": codes.view(torch.float8_e4m3fn), "scales": scales}


# ------------------------------------------------------------------------------------------------ work
def work(case):
    kind = case["kind"]
    if kind in ("norm", "norm_back"):
        n, R, C = case["rows"] * case["cols"], case["rows"], case["cols"]
        if kind == "norm":      # x, residual in; h, codes, scales and rstd out
            return {"bytes": 7 * n + 4 * (n // 128) + 4 * R + 2 * C, "flops": 8 * n}
        return {"bytes": 8 * n + 4 * R + 6 * C, "flops": 10 * n}
    if kind == "rotary":
        n = case["tokens"] * (case["q_heads"] + case["kv_heads"])
        return {"bytes": 4 * n * case["head_dim"] + 4 * case["tokens"] + 8 * case["pairs"], "flops": 6 * n * case["pairs"]}
    if kind == "attend":
        Hq, H, D = case["q_heads"], case["kv_heads"], case["head_dim"]
        prompts, pairs = _requests(case)
        read = sum(2 * D * H * BLOCK * (p // BLOCK) for p in prompts)
        flops = 0
        for r, (x, m) in enumerate(pairs):
            if m:
                last, first = (x + m - 1) // BLOCK, prompts[r // case["samples"]] // BLOCK
                read += 2 * D * H * BLOCK * (last - first) + 4 * D * H * (x + m - x // BLOCK * BLOCK)
                flops += 4 * D * Hq * (m * x + m * (m + 1) // 2)
        return {"bytes": read + 4 * sum(m for _, m in pairs) * Hq * D, "flops": flops}
    R, ctx = case["requests"], case["ctx"]
    lens = [(2 * i + 1) * ctx // (2 * R) for i in range(R)]
    held = sum(x // BLOCK for x in lens)
    if kind == "fork":          # six in ten take over another's unfinished block
        fresh = 0.6 * sum(x % BLOCK for x in lens) * case["kv_heads"] * case["head_dim"]
        return {"bytes": int(8 * fresh) + 8 * held + 20 * R, "flops": 0}
    blocks = held + held // 4 + 5
    b = {"bytes": 4 * held + 8 * R + 4 * blocks, "flops": 0}
    if kind == "compact":       # about a quarter of the blocks move
        block = 2 * BLOCK * case["kv_heads"] * case["head_dim"] + 8 * case["kv_heads"]
        b["bytes"] += 4 * held + 2 * (blocks // 4) * block
    return b


# ------------------------------------------------------------------------------------------------ 64 bits
def _e4m3():
    """The 127 values of the positive codes."""
    return torch.tensor([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)],
                        dtype=torch.float64, device="cuda")


def exact(case, seed):
    kind = case["kind"]
    if kind == "sweep":
        return None                                     # whole numbers: compared as they are
    s = prepare(case, seed)
    if kind == "norm":
        return _exact_norm(s)
    if kind == "norm_back":
        return _exact_norm_back(s)
    if kind == "rotary":
        x, P = s["x"].double(), len(s["freqs"])
        out = x.clone()
        for i in range(P):
            a, b = (2 * i, 2 * i + 1) if s["interleaved"] else (i, P + i)
            turn = s["positions"].double() * s["freqs"][i] * (-1 if s["inverse"] else 1)
            z = torch.complex(x[..., a], x[..., b]) * torch.polar(torch.full_like(turn, s["amplitude"]), turn)[:, None]
            out[..., a], out[..., b] = z.real, z.imag
        return out
    if kind == "attend":
        return _exact_attend(s)
    if kind == "fork":
        recent = s["recent"].double()
        state, parents = s["state"].tolist(), s["parents"].tolist()
        for r, p in enumerate(parents):
            if p >= 0 and p != r:
                recent[2 * r + 1 - state[r][1]] = s["recent"][2 * p + state[p][1]].double()
        return {"state": None, "table": None, "recent": recent}
    codes, scales = s["codes"].view(torch.float8_e4m3fn).double(), s["scales"].double()
    table = s["table"].tolist()
    live = {b for row, (x, _) in zip(table, s["state"].tolist()) for b in row[:x // BLOCK]}
    L = len(live)
    source = sorted(b for b in live if b >= L)
    target = [b for b in range(L) if b not in live]
    if source:
        a, b = (torch.tensor(v, device="cuda") for v in (source, target))
        codes[b], scales[b] = codes[a], scales[a]
    return {"free": None, "head": None, "live": None, "table": None, "moves": None, "codes": codes, "scales": scales}


def _exact_norm(s):
    x, w = s["x"], s["weight"].double()
    R, C = x.shape
    value = _e4m3()
    halves = (value[1:] + value[:-1]) / 2
    codes = torch.empty((R, C), dtype=torch.float64, device="cuda")
    h, rstd = torch.empty_like(codes), torch.empty((R,), dtype=torch.float64, device="cuda")
    scales = torch.empty((C // 128, R), dtype=torch.float64, device="cuda")
    for k in (slice(i, i + 8192) for i in range(0, R, 8192)):
        h[k] = (x[k].double() + s["residual"][k].double()).float().to(torch.bfloat16).double()
        rstd[k] = ((h[k] * h[k]).sum(1) / C + EPS).rsqrt().float().double()
        y = ((h[k] * rstd[k][:, None]).float().double() * w).float().to(torch.bfloat16).double()
        for j in range(C // 128):
            z = y[:, 128 * j:128 * j + 128]
            sc = (z.abs().amax(1) / 448).float().double()
            a = z.abs() / torch.where(sc > 0, sc, 1.0)[:, None]
            i = torch.searchsorted(halves, a)
            tie = (i < 126) & (a == halves[i.clamp(max=125)])
            codes[k, 128 * j:128 * j + 128] = value[torch.where(tie & (i % 2 == 1), i + 1, i)] * torch.sign(z)
            scales[j, k] = sc
    return {"codes": codes, "scales": scales, "rstd": rstd, "h": h}


def _exact_norm_back(s):
    R, C = s["h"].shape
    dx = torch.empty((R, C), dtype=torch.float64, device="cuda")
    dw = torch.zeros((C,), dtype=torch.float64, device="cuda")
    w = s["weight"].double()
    for i in range(0, R, 4096):
        k = slice(i, i + 4096)
        h, dy, r = s["h"][k].double(), s["dy"][k].double(), s["rstd"][k].double()[:, None]
        n = h * r                                          # the normalized rows
        g = dy * w
        dx[k] = s["dres"][k].double() + r * (g - n * ((g * n).sum(1, keepdim=True) / C))
        dw += (dy * n).sum(0)
    return {"dx": dx, "dw": dw}


def _exact_attend(s):
    T, Hq, D = s["q"].shape
    H = s["codes"].shape[1]
    G = Hq // H
    k8, v8, k16, v16 = _places(D)
    value = _e4m3()
    nan = value.new_full((1,), math.nan)
    signed = torch.cat([value, nan, -value, nan])
    out = torch.empty((T, Hq, D), dtype=torch.float64, device="cuda")
    table = s["table"].long()
    last = (-1, -1)
    for r, j, place, row, rows, offset, _, _ in s["units"].tolist():
        if r < 0:
            continue
        if (r, j) != last and j:
            ids = table[r, :j]
            sc, c = s["scales"][ids].double(), s["codes"][ids].long()
            K0 = (signed[c[:, :, 0][:, :, k8]] * sc[:, :, 0, None, None]).transpose(0, 1).reshape(H, -1, D)
            V0 = (signed[c[:, :, 1][:, :, v8]] * sc[:, :, 1, None, None]).transpose(0, 1).reshape(H, -1, D)
            last = (r, j)
        h = offset + rows
        K, V = s["recent"][place, :, 0][:, k16[:h]].double(), s["recent"][place, :, 1][:, v16[:h]].double()
        if j:
            K, V = torch.cat([K0, K], 1), torch.cat([V0, V], 1)
        Q = s["q"][row:row + rows].double().view(rows, H, G, D).permute(1, 2, 0, 3).reshape(H, G * rows, D)
        S = (Q @ K.transpose(1, 2).contiguous() / math.sqrt(D)).view(H, G, rows, -1)
        late = torch.arange(j * BLOCK + h, device="cuda")[None] > j * BLOCK + offset + torch.arange(rows, device="cuda")[:, None]
        P = torch.softmax(S.masked_fill(late, -math.inf), -1).view(H, G * rows, -1)
        out[row:row + rows] = (P @ V).view(H, G, rows, D).permute(2, 0, 1, 3).reshape(rows, Hq, D)
    return out
