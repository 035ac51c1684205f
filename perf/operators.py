"""Cases for the operators between a new token and its attention over a paged latent cache: block
tables and slot maps, rotary positions, the 4-bit cache, attention over a selection of it, and
attention over a sliding window with first tokens that stay visible.

``run`` computes them in plain torch (own = False) or through this package (own = True); ``exact``
gives the same from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
LATENT, ROTARY = 512, 64        # a cache row: 512 latent elements, then 64 rotary ones
ROW = LATENT + ROTARY
BLOCK = 16                      # latent elements per scale of the 4-bit row
ROW4 = LATENT // 2 + LATENT // BLOCK + 2 * ROTARY   # bytes: 4-bit codes, e4m3 scales, bf16 rotary part
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
SCALE = 1.0 / math.sqrt(192.0)


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step's bookkeeping: 32 requests, one new token each
        dict(name="tables decode 32", op="tables", requests=32, page=64, length=8192, new=1, spread=0),
        # a mixed batch of a large server: chunked prefill beside decode, odd page size
        dict(name="tables mixed 1500", op="tables", requests=1500, page=48, length=40000, new=37, spread=1),
        # one decode step's queries and rows: indexer query and key, attention query and row
        dict(name="rope decode 8", op="rope", tokens=8, heads=128, rot=64, dtype="bf16", layout="interleaved",
             scaling="yarn", far=163840),
        # a prefill chunk with every head
        dict(name="rope prefill 8192", op="rope", tokens=8192, heads=64, rot=64, dtype="bf16", layout="half",
             scaling="yarn", far=163840),
        # a step's new rows into the cache
        dict(name="kv4 decode 32", op="kv4", rows=32, page=64, pages=4096),
        # a long prompt's rows
        dict(name="kv4 prefill 65537", op="kv4", rows=65537, page=64, pages=2048),
        # one request, GLM-5's head count
        dict(name="sparse4 b1 h64", op="sparse", cache="kv4", requests=1, tokens=1, heads=64, k=2048, length=8192,
             page=64, spread=0),
        # the consumer's decode shape
        dict(name="sparse4 b8 h128", op="sparse", cache="kv4", requests=8, tokens=1, heads=128, k=2048, length=32768,
             page=64, spread=0),
        # two tokens a request, one shard of the heads, odd sizes
        dict(name="sparse4 b37 h16 mtp2", op="sparse", cache="kv4", requests=37, tokens=2, heads=16, k=1000,
             length=9001, page=48, spread=1),
        # a decode step of a window layer
        dict(name="window4 decode b32", op="window", cache="kv4", requests=32, tokens=1, heads=128, window=512,
             sinks=4, length=16384, page=64, spread=1),
        # one request with its whole context in view
        dict(name="window4 long 131071", op="window", cache="kv4", requests=1, tokens=1, heads=128, window=131072,
             sinks=0, length=131071, page=64, spread=0),
        # a prefill chunk over bf16 rows
        dict(name="window16 prefill 1024", op="window", cache="bf16", requests=1, tokens=1024, heads=128, window=512,
             sinks=16, length=5000, page=64, spread=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "rope", "kv4", "sparse", "sparse", "window", "window"])
    if op == "tables":
        new = rng.choice([1, 1, _log(rng, 2, 64)])
        return dict(op=op, requests=_log(rng, 1, 1500), page=rng.choice([16, 32, 48, 64, 128]),
                    length=_log(rng, 64, 40000) + new, new=new, spread=rng.randint(0, 1))
    if op == "rope":
        tokens = _log(rng, 1, 4096)
        return dict(op=op, tokens=tokens, heads=rng.choice([8, 16, 32, 64, 128] if tokens < 2048 else [8, 16, 32]),
                    rot=rng.choice([32, 64, 128]), dtype=rng.choice(["bf16", "bf16", "fp32"]),
                    layout=rng.choice(["interleaved", "half"]), scaling=rng.choice(["none", "linear", "yarn"]),
                    far=_log(rng, 4096, 1000000))
    if op == "kv4":
        page = rng.choice([16, 48, 64, 128])
        rows = _log(rng, 1, 60000)
        return dict(op=op, rows=rows, page=page, pages=rows // page + _log(rng, 1, 1000))
    cache = rng.choice(["kv4", "kv4", "bf16"])
    page = rng.choice([1, 16, 48, 64, 128])
    heads = rng.choice([8, 16, 32, 64, 128])
    if op == "sparse":
        requests, tokens = _log(rng, 1, 32), rng.choice([1, 1, 2, 3])
        return dict(op=op, cache=cache, requests=requests, tokens=tokens, heads=heads, k=_log(rng, 64, 2048),
                    length=_log(rng, 16, 16384) + 8, page=page, spread=rng.randint(0, 1))
    if rng.random() < 0.5:
        requests, tokens = _log(rng, 1, 32), rng.choice([1, 1, 2])
        window, length = _log(rng, 1, 2048), _log(rng, 16, 16384)
    else:
        requests, tokens = rng.randint(1, 3), _log(rng, 16, 256)
        window, length = _log(rng, 16, 512), _log(rng, 300, 8192)
    return dict(op=op, cache=cache, requests=requests, tokens=tokens, heads=heads, window=window,
                sinks=rng.choice([0, 1, 4, 16, 64]), length=length + tokens, page=page, spread=rng.randint(0, 1))


def _lens(case):
    """The requests' lengths after the step: all the same, or spread down to the new tokens alone."""
    n, top, low = case["requests"], case["length"], case.get("tokens", 1)
    if not case["spread"]:
        return [top] * n
    r = random.Random(n * 1000003 + top)
    return [top if i == 0 else r.randint(min(low, top), top) for i in range(n)]


def _news(case):
    """New tokens per request: all the same, or every fourth request prefills and the others decode."""
    return [min(n, case["new"] if not case["spread"] or i % 4 == 0 else 1) for i, n in enumerate(_lens_tables(case))]


def _lens_tables(case):
    n, top = case["requests"], case["length"]
    if not case["spread"]:
        return [top - (i * 7919) % max(1, min(top - case["new"], top // 3) + 1) for i in range(n)]
    r = random.Random(n * 1000003 + top)
    return [r.randint(1, top) for _ in range(n)]


def _visible(case):
    """Positions each request's tokens see, per token."""
    t = case.get("tokens", 1)
    out = []
    for n in _lens(case):
        for i in range(t):
            p = n - t + i
            if case["op"] == "sparse":
                out.append(min(case["k"], p + 1))
            else:
                w = min(case["window"], p + 1)
                out.append(w + min(case["sinks"], p + 1 - w))
    return out


def work(case):
    op = case["op"]
    if op == "tables":
        lens, news, p = _lens_tables(case), _news(case), case["page"]
        taken = sum(-(-n // p) - (-(-(n - w) // p)) for n, w in zip(lens, news))
        return {"bytes": 12 * len(lens) + 8 * taken + 16 * sum(news) + 4, "flops": 4 * sum(news)}
    if op == "rope":
        size = 2 if case["dtype"] == "bf16" else 4
        part = case["tokens"] * (case["heads"] + 1)
        return {"bytes": 2 * part * (case["rot"] + 64) * size + 4 * case["tokens"], "flops": part * case["rot"] * 3}
    if op == "kv4":
        return {"bytes": case["rows"] * (2 * ROW * 2 + 2 * ROW4 + 16), "flops": 4 * case["rows"] * LATENT}
    row = ROW4 if case["cache"] == "kv4" else 2 * ROW
    seen, n = _visible(case), case["requests"] * case["tokens"]
    if op == "sparse":
        rows = sum(seen)
    else:  # a request's tokens share their rows
        rows = sum(min(length, case["sinks"] + case["window"] + case["tokens"] - 1) for length in _lens(case))
    return {"bytes": rows * row + n * case["heads"] * (ROW + LATENT) * 2 + (4 * sum(seen) if op == "sparse" else 0),
            "flops": 2 * case["heads"] * (ROW + LATENT) * sum(seen)}


# --------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device=DEV)


def _rows(n, g):
    """Normalised latent rows with channels of different size, and their rotary part, in bf16."""
    gain = torch.exp(0.5 * torch.randn(ROW, device=DEV, generator=g))
    return (torch.randn(n, ROW, device=DEV, generator=g) * gain).to(torch.bfloat16)


def _layers(pages, page, case, g):
    """The cache of `pages` pages in the case's format, filled with rows."""
    if case["cache"] == "bf16":
        return _rows(pages * page, g).view(pages, page, ROW)
    cache = torch.empty(pages * page, ROW4, dtype=torch.uint8, device=DEV)
    for at in range(0, pages * page, 65536):
        n = min(65536, pages * page - at)
        cache[at:at + n] = _pack4(_rows(n, g))
    return cache.view(pages, page, ROW4)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "tables":
        lens, news, p = _lens_tables(case), _news(case), case["page"]
        blocks = max(-(-n // p) for n in lens)
        total = sum(-(-n // p) for n in lens)
        pages = total + 64
        order = torch.randperm(pages, device=DEV, generator=g).to(torch.int32)
        held = _ints([-(-(n - w) // p) for n, w in zip(lens, news)], torch.int64)
        at = torch.cumsum(held, 0) - held
        j = torch.arange(blocks, device=DEV)
        table = torch.full((len(lens), blocks), -1, dtype=torch.int32, device=DEV)
        keep = j[None, :] < held[:, None]
        table[keep] = order[(at[:, None] + j[None, :])[keep]]
        s.update(seq=_ints(lens), new=_ints(news), table=table, free=order[int(held.sum()):].contiguous(),
                 pages=pages, tokens=sum(news))
    elif op == "rope":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        n, h, r = case["tokens"], case["heads"], case["rot"]
        dim = r + 64   # the rotated part stands behind 64 elements that keep their values
        s.update(q=torch.randn(n, h, dim, device=DEV, generator=g).to(dt),
                 k=torch.randn(n, dim, device=DEV, generator=g).to(dt),
                 pos=torch.randint(0, case["far"], (n,), device=DEV, generator=g, dtype=torch.int32),
                 freq=_frequencies(case), mscale=_mscale(case))
        if own:
            from sparse_attention_lightning_score_b200 import api
            s["rope"] = api.li_rope_table(r, **_scaling(case), device=DEV)
    elif op == "kv4":
        slots = torch.randperm(case["pages"] * case["page"], device=DEV, generator=g)[:case["rows"]].contiguous()
        s.update(rows=_rows(case["rows"], g), slots=slots,
                 cache=torch.zeros(case["pages"], case["page"], ROW4, dtype=torch.uint8, device=DEV))
    else:
        lens, t, p = _lens(case), case["tokens"], case["page"]
        blocks = max(-(-n // p) for n in lens)
        pages = len(lens) * blocks + 3
        table = torch.randperm(pages, device=DEV, generator=g)[:len(lens) * blocks].to(torch.int32)
        requests = torch.arange(len(lens), device=DEV, dtype=torch.int32).repeat_interleave(t)
        pos = (_ints(lens)[:, None] - t + torch.arange(t, device=DEV, dtype=torch.int32)).reshape(-1)
        gain = 0.5 + 2.0 * torch.rand(case["heads"], 1, device=DEV, generator=g)   # flat heads and sharp ones
        q = torch.randn(len(lens) * t, case["heads"], ROW, device=DEV, generator=g) * gain
        s.update(q=q.to(torch.bfloat16), cache=_layers(pages, p, case, g), table=table.view(len(lens), blocks),
                 requests=requests, pos=pos.contiguous(), max_len=max(lens))
        if op == "sparse":
            score = torch.rand(len(pos), max(lens), device=DEV, generator=g)
            score.masked_fill_(torch.arange(max(lens), device=DEV)[None, :] > pos[:, None], -1.0)
            k = min(case["k"], max(lens))
            val, idx = torch.topk(score, k, dim=1)
            idx = torch.where(val < 0, max(lens), idx).sort(dim=1).values
            sel = torch.full((len(pos), case["k"]), -1, dtype=torch.int32, device=DEV)
            sel[:, :k] = torch.where(idx == max(lens), -1, idx)
            s["sel"] = sel
    return s


# --------------------------------------------------------------------------- rotary frequencies
def _scaling(case):
    return {"none": dict(base=10000.0), "linear": dict(base=10000.0, scaling="linear", factor=8.0),
            "yarn": dict(base=10000.0, scaling="yarn", factor=40.0, original_len=4096, beta_fast=32.0,
                         beta_slow=1.0)}[case["scaling"]]


def _mscale(case):
    return 0.1 * math.log(40.0) + 1.0 if case["scaling"] == "yarn" else 1.0


def _frequencies(case):
    """Radians per position of each pair, in 64 bits."""
    r, c = case["rot"], _scaling(case)
    f = c["base"] ** (-torch.arange(0, r, 2, dtype=torch.float64, device=DEV) / r)
    if case["scaling"] == "linear":
        f = f / c["factor"]
    if case["scaling"] == "yarn":
        def turn(beta):  # the (fractional) pair that makes `beta` turns over the original length
            return r * math.log(c["original_len"] / (beta * 2 * math.pi)) / (2 * math.log(c["base"]))
        lo, hi = max(math.floor(turn(c["beta_fast"])), 0), min(math.ceil(turn(c["beta_slow"])), r - 1)
        ramp = ((torch.arange(r // 2, dtype=torch.float64, device=DEV) - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f / c["factor"] * ramp + f * (1 - ramp)
    return f


# --------------------------------------------------------------------------- plain forms
def _pack4(rows):
    """bf16 rows [n, 576] -> 4-bit rows [n, 416] bytes."""
    n = rows.shape[0]
    x = rows[:, :LATENT].float().view(n, LATENT // BLOCK, BLOCK)
    sc = (x.abs().amax(2) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = sc.float()[:, :, None]
    a = (x.abs() / torch.where(s > 0, s, torch.ones_like(s))).masked_fill(s == 0, 0.0)
    # nearest of the eight magnitudes, ties to the even code
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code + 8 * torch.signbit(x).to(torch.uint8)).view(n, LATENT // 2, 2)
    return torch.cat([code[:, :, 0] + 16 * code[:, :, 1], sc.view(torch.uint8),
                      rows[:, LATENT:].contiguous().view(torch.uint8)], dim=1)


def _unpack4(raw):
    """4-bit rows [..., 416] bytes -> fp32 rows [..., 576]."""
    value = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=raw.device)
    codes = raw[..., :LATENT // 2]
    v = value[torch.stack([codes & 15, codes >> 4], -1).long()].flatten(-2)
    s = raw[..., LATENT // 2:LATENT // 2 + LATENT // BLOCK].contiguous().view(torch.float8_e4m3fn).float()
    rope = raw[..., LATENT // 2 + LATENT // BLOCK:].contiguous().view(torch.bfloat16).float()
    return torch.cat([v * s.repeat_interleave(BLOCK, -1), rope], -1)


def _plain_tables(s):
    p = s["case"]["page"]
    seq, new = s["seq"].long(), s["new"].long()
    held, have = -((new - seq) // p), -(-seq // p)
    need = have - held
    first = torch.cumsum(need, 0) - need
    cu = torch.cat([torch.zeros_like(seq[:1]), torch.cumsum(new, 0)])
    j = torch.arange(s["table"].shape[1], device=DEV)[None, :]
    take = (j >= held[:, None]) & (j < have[:, None])
    at = (first[:, None] + j - held[:, None]).clamp(0, s["free"].numel() - 1)
    table = torch.where(take, s["free"][at], s["table"])
    req = torch.repeat_interleave(torch.arange(len(seq), device=DEV), new, output_size=s["tokens"])
    pos = torch.arange(s["tokens"], device=DEV) - cu[req] + (seq - new)[req]
    slot = table[req, pos // p].long() * p + pos % p
    return [slot, pos.int(), req.int(), cu.int(), need.sum().int().view(1), table]


def _plain_rope(s):
    r, half = s["case"]["rot"], s["case"]["layout"] == "half"
    angle = s["pos"].double()[:, None] * s["freq"][None, :]
    cos, sin = (angle.cos() * s["mscale"]).float(), (angle.sin() * s["mscale"]).float()

    def turn(x, c, n):
        rest, y = x[..., :-r], x[..., -r:].float()
        a, b = (y[..., :r // 2], y[..., r // 2:]) if half else (y[..., 0::2], y[..., 1::2])
        u, v = a * c - b * n, a * n + b * c
        y = torch.cat([u, v], -1) if half else torch.stack([u, v], -1).flatten(-2)
        return torch.cat([rest, y.to(x.dtype)], -1)

    return [turn(s["q"], cos[:, None], sin[:, None]), turn(s["k"], cos, sin)]


def _plain_kv4(s):
    flat = s["cache"].view(-1, ROW4)
    flat[s["slots"]] = _pack4(s["rows"])
    return _unpack4(flat[s["slots"]]).to(torch.bfloat16)


def _attend(s, at, valid):
    """Attention of each token over positions `at` [n, m] of its request where `valid`."""
    p = s["case"]["page"]
    at = at.clamp(min=0).long()
    slot = s["table"][s["requests"].long()[:, None], at // p].long() * p + at % p
    raw = s["cache"].flatten(0, 1)[slot]
    kv = (_unpack4(raw) if s["case"]["cache"] == "kv4" else raw.float()).masked_fill(~valid[:, :, None], 0.0)
    logit = torch.bmm(s["q"].float(), kv.transpose(1, 2)) * SCALE
    logit = logit.masked_fill(~valid[:, None, :], -math.inf)
    w = torch.exp(logit - logit.amax(2, keepdim=True))
    return (torch.bmm(w, kv[:, :, :LATENT]) / w.sum(2, keepdim=True)).to(torch.bfloat16)


def _plain_window(s):
    c, pos = s["case"], s["pos"].long()[:, None]
    window = min(c["window"], s["max_len"])
    first = torch.arange(c["sinks"], device=DEV)[None, :].expand(len(pos), -1)
    near = pos - window + 1 + torch.arange(window, device=DEV)[None, :]
    return _attend(s, torch.cat([first, near], 1), torch.cat([first <= pos - window, near >= 0], 1))


def run(s):
    op = s["case"]["op"]
    if not own:
        if op == "sparse":
            return _attend(s, s["sel"], s["sel"] >= 0)
        return {"tables": _plain_tables, "rope": _plain_rope, "kv4": _plain_kv4, "window": _plain_window}[op](s)
    from sparse_attention_lightning_score_b200 import api
    if op == "tables":
        return list(api.li_block_tables(s["seq"], s["new"], s["table"], s["free"], s["case"]["page"], s["pages"],
                                        s["tokens"])) + [s["table"]]
    if op == "rope":
        return api.li_rope([s["q"], s["k"]], s["pos"], s["rope"], layout=s["case"]["layout"], offset=64,
                           mscale=s["mscale"])
    if op == "kv4":
        api.li_kv4_write(s["rows"], s["slots"], s["cache"])
        return api.li_kv4_read(s["cache"], s["slots"])
    if op == "sparse":
        return api.li_paged_sparse_attention(s["q"], s["cache"], s["sel"], SCALE, block_table=s["table"],
                                             requests=s["requests"])
    return api.li_window_attention(s["q"], s["cache"], s["pos"], SCALE, s["case"]["window"], sinks=s["case"]["sinks"],
                                   block_table=s["table"], requests=s["requests"], max_len=s["max_len"])


# --------------------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    if case["op"] == "tables":
        return None    # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "rope":
        r = case["rot"]
        turns = torch.polar(torch.full((), s["mscale"], dtype=torch.float64, device=DEV),
                            torch.outer(s["pos"].double(), s["freq"]))
        out = []
        for x in (s["q"], s["k"]):
            y = x.double().reshape(case["tokens"], -1, x.shape[-1]).clone()
            i = torch.arange(r // 2, device=DEV)
            lo, hi = (i, i + r // 2) if case["layout"] == "half" else (2 * i, 2 * i + 1)
            z = torch.complex(y[:, :, 64 + lo], y[:, :, 64 + hi]) * turns[:, None, :]
            y[:, :, 64 + lo], y[:, :, 64 + hi] = z.real, z.imag
            out.append(y.view(x.shape))
        return out
    if case["op"] == "kv4":
        # each value by distance to all eight magnitudes times its block's scale
        x = s["rows"].double()
        b = x[:, :LATENT].view(-1, LATENT // BLOCK, BLOCK)
        sc = (b.abs().amax(2) / 6).clamp(max=448).float().to(torch.float8_e4m3fn).double()
        grid = sc[:, :, None] * torch.tensor(E2M1, dtype=torch.float64, device=DEV)
        out = torch.empty_like(b)
        for i in range(BLOCK):
            d = (b[:, :, i].abs()[:, :, None] - grid).abs()
            d = d + 1e-12 * sc[:, :, None] * torch.tensor([0., 1.] * 4, dtype=torch.float64, device=DEV)  # ties: even
            out[:, :, i] = torch.gather(grid, 2, d.argmin(2, keepdim=True))[:, :, 0] * torch.where(b[:, :, i] < 0, -1., 1.)
        return torch.cat([out.view(-1, LATENT), x[:, LATENT:]], 1)
    cache, page = s["cache"].flatten(0, 1), case["page"]
    out = torch.empty(s["q"].shape[0], case["heads"], LATENT, dtype=torch.float64, device=DEV)
    pos = s["pos"].tolist()
    for t, r in enumerate(s["requests"].tolist()):
        if case["op"] == "sparse":
            at = s["sel"][t].long()
            at = at[at >= 0]
        else:
            p = torch.arange(pos[t] + 1, device=DEV)
            at = p[(p < case["sinks"]) | (p > pos[t] - case["window"])]
        raw = cache[s["table"][r].long()[torch.div(at, page, rounding_mode="floor")] * page + at % page]
        if case["cache"] == "kv4":
            byte = raw.to(torch.int64)
            nib = torch.stack([byte[:, :256] % 16, byte[:, :256] // 16], 2).view(-1, LATENT)
            e, m = (nib // 2) % 4, nib % 2
            v = torch.where(e > 0, (1 + 0.5 * m) * 2.0 ** (e - 1).double(), 0.5 * m.double())
            v = v * torch.where(nib > 7, -1.0, 1.0)
            f, g = byte[:, 256:288] // 8, byte[:, 256:288] % 8
            sc = torch.where(f > 0, (1 + g / 8.0).double() * 2.0 ** (f - 7).double(), g.double() / 512)
            rope = raw[:, 288:].contiguous().view(torch.bfloat16).double()
            kv = torch.cat([(v.view(-1, 32, 16) * sc[:, :, None]).view(-1, LATENT), rope], 1)
        else:
            kv = raw.double()
        w = torch.softmax((s["q"][t].double() @ kv.T) * SCALE, 1)
        out[t] = w @ kv[:, :LATENT]
    return out
