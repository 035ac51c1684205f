"""GPU parity of the paged-cache operators against the plain 64-bit definitions (oracle.paged): block
tables and slot maps, rotary positions, the 4-bit cache, attention over a selection and over a window.

Attention tolerance.  Per output element, with u = 2^-8 (half a bf16 step) and mag = sum_i p_i |v_i|:
  - each weight is rounded to bf16 for the product: u * mag; the output once: u * |o|;
  - the logits are fp32 sums of 576 exact products, the running sums and the rescaling fp32:
    a relative weight error of d = 2^-23 * (600 * top + 64 + n / 16), where top bounds
    scale * sum |q_d k_d|; numerator and denominator both carry it: 2 d * mag.
"""
import numpy as np
import pytest
import torch

from oracle import paged as oracle
from sparse_attention_lightning_score_b200 import api
from sparse_attention_lightning_score_b200._lib import LI_ERR_BOUNDS, LI_OK

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -8


def _np(t):
    return t.detach().cpu().numpy()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


# --------------------------------------------------------------------------- block tables
def _tables_case(R, page, top, new_max, seed, spare=5):
    g = np.random.default_rng(seed)
    seq = g.integers(0, top + 1, R)
    new = np.minimum(seq, g.integers(0, new_max + 1, R))
    blocks = max(1, -(-top // page)) + 1
    held, have = -(-(seq - new) // page), -(-seq // page)
    pages = int(have.sum()) + spare
    perm = g.permutation(pages)
    table = np.full((R, blocks), -7)
    at = 0
    for r in range(R):
        table[r, :held[r]] = perm[at:at + held[r]]
        at += held[r]
    return seq, new, table, perm[at:], pages


def _run_tables(seq, new, table, free, page, pages, tokens, start=None, **kw):
    t = _i32(table)
    out = api.li_block_tables(_i32(seq), _i32(new), t, _i32(free), page, pages, tokens,
                              free_start=None if start is None else _i32([start]), **kw)
    return [_np(x) for x in out] + [_np(t)]


def _same_tables(got, want):
    for g, w, name in zip(got, want[:4] + (np.array([want[4]]), want[5]),
                          ["slots", "positions", "requests", "starts", "free_next", "table"]):
        assert np.array_equal(g, w), name


@pytest.mark.parametrize("R,page,top,new_max,start", [
    (1, 64, 0, 0, None), (1, 64, 1, 1, None), (3, 1, 40, 9, 0), (32, 64, 8000, 1, 3), (257, 48, 3000, 300, 2),
    (1500, 16, 500, 5, None), (9000, 128, 300, 2, 1), (16384, 64, 100, 1, None)])
def test_block_tables(R, page, top, new_max, start):
    seq, new, table, free, pages = _tables_case(R, page, top, new_max, seed=R + page)
    n = int(new.sum())
    for tokens in (n, n + 37):
        got = _run_tables(seq, new, table, free, page, pages, tokens, start)
        _same_tables(got, oracle.block_tables(seq, new, table, free, page, pages, tokens, start or 0))
        if not start:
            assert api.li_get_last_error() == LI_OK
    api.li_get_last_error()


def test_block_tables_no_requests_or_tokens():
    got = _run_tables(np.zeros(0, int), np.zeros(0, int), np.zeros((0, 3), int), [1, 2], 8, 4, 5)
    assert (got[0] == -1).all() and (got[1] == -1).all() and (got[2] == -1).all()
    assert got[3].tolist() == [0] and got[4].tolist() == [0]
    got = _run_tables([5], [0], [[3, -1]], [1], 8, 4, 0)
    assert got[3].tolist() == [0, 0] and got[5].tolist() == [[3, -1]] and api.li_get_last_error() == LI_OK


@pytest.mark.parametrize("what", ["short pool", "bad pool page", "bad held page", "negative new", "new above seq",
                                  "beyond the table", "too many tokens", "bad start", "start at the end"])
def test_block_tables_reports(what):
    seq, new, table, free, pages = _tables_case(12, 16, 200, 40, seed=5)
    tokens, start = int(new.sum()), None
    if what == "short pool":
        free = free[:2]
    elif what == "bad pool page":
        free[1] = pages
    elif what == "bad held page":
        r = int(np.argmax((seq - new) % 16 > 0) if ((seq - new) % 16 > 0).any() else 0)
        new[r] = max(new[r], 1)
        table[r, (seq[r] - new[r]) // 16] = -3 if (seq[r] - new[r]) % 16 else table[r, 0]
    elif what == "negative new":
        new[3] = -1
    elif what == "new above seq":
        new[4] = seq[4] + 1
    elif what == "beyond the table":
        seq[2] = table.shape[1] * 16 + 1
    elif what == "too many tokens":
        tokens -= 3
    elif what == "bad start":
        start = -1
    elif what == "start at the end":
        start = len(free)
    got = _run_tables(seq, new, table, free, 16, pages, tokens, start)
    if what == "bad start":     # nothing may be taken
        want = oracle.block_tables(seq, new, table, free, 16, pages, tokens, len(free))
    else:
        want = oracle.block_tables(seq, new, table, free, 16, pages, tokens, start or 0)
    assert api.li_get_last_error() == (LI_ERR_BOUNDS if want[6] or what == "bad start" else LI_OK)
    _same_tables(got, want)
    assert want[6] or what == "bad start"


def test_block_tables_steps_in_a_graph():
    """Decode steps with the pool index passed on in two buffers, captured and replayed."""
    page, R, pages = 4, 5, 60
    seq, table = _i32([0, 3, 4, 7, 8]), torch.full((R, 10), -1, dtype=torch.int32, device=DEV)
    free = torch.randperm(pages, device=DEV, dtype=torch.int32)
    have, at = [-(-s // page) for s in seq.tolist()], 0
    for r, h in enumerate(have):
        table[r, :h] = free[at:at + h]
        at += h
    free = free[at:].contiguous()
    want_table, start = _np(table).copy(), 0
    one, a, b = _i32([1] * R), _i32([0]), _i32([0])
    bufs = dict(slots=torch.empty(R, dtype=torch.int64, device=DEV), positions=_i32([0] * R), requests=_i32([0] * R),
                starts=_i32([0] * (R + 1)))
    step = lambda: (seq.add_(1), api.li_block_tables(seq, one, table, free, page, pages, R, free_start=a,  # noqa: E731
                                                     free_next=b, **bufs), a.copy_(b))
    keep = (seq.clone(), table.clone())
    step()
    torch.cuda.synchronize()
    seq.copy_(keep[0]); table.copy_(keep[1]); a.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(9):
        graph.replay()
        w = oracle.block_tables(_np(seq), [1] * R, want_table, _np(free), page, pages, R, start)
        want_table, start = w[5], w[4]
        assert np.array_equal(_np(bufs["slots"]), w[0]) and np.array_equal(_np(table), w[5]) and a.item() == start
    assert api.li_get_last_error() == LI_OK


# --------------------------------------------------------------------------- rotary positions
def _rope_tol(dtype, x, mscale):
    """One rounding of the result, and fp32 arithmetic on the pair: the angle's fraction (2^-25 turns), cosine and
    sine (2 ulp), two products and a sum: 8 units of 2^-24 of the pair's norm."""
    u = U if dtype == torch.bfloat16 else 2.0 ** -24
    return u, 8 * 2.0 ** -24 * abs(mscale) * 2 * np.abs(x).max()


def _check_rope(got, x, pos, freq, layout, offset, mscale):
    x64 = x.detach().cpu().double().numpy().reshape(x.shape[0], -1, x.shape[-1])
    want = oracle.rope(x64, pos, freq, layout, offset, mscale).reshape(x.shape)
    u, a = _rope_tol(x.dtype, x64, mscale)
    err = np.abs(got.detach().cpu().double().numpy() - want)
    live = (np.asarray(pos) >= 0).reshape((-1,) + (1,) * (x.dim() - 1))
    assert np.all((err <= u * np.abs(want) + a) | ~live), float(err.max())
    return live


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("tokens,heads,dim,rot,offset", [
    (1, 1, 64, 64, 0), (8, 64, 128, 64, 0), (3, 128, 576, 64, 512), (5, 7, 100, 36, 10), (17, 3, 130, 2, 128),
    (300, 5, 192, 128, 64), (2, 2, 33, 30, 3), (9, 4, 1024, 1024, 0)])
def test_rope(dtype, layout, tokens, heads, dim, rot, offset):
    g = torch.Generator().manual_seed(tokens + dim)
    x = torch.randn(tokens, heads, dim, generator=g).to(dtype)
    pos = torch.randint(0, 1 << 20, (tokens,), generator=g).to(torch.int32)
    pos[0] = 0
    if tokens > 2:
        pos[1], pos[2] = 2 ** 31 - 1, -1
    kw = dict(scaling="yarn", factor=40.0, original_len=4096) if rot == 64 else \
        dict(scaling="linear", factor=3.0) if rot == 128 else {}
    table = api.li_rope_table(rot, **kw)
    freq = oracle.rope_frequencies(rot, **kw)
    xd = x.to(DEV)
    out = torch.full_like(xd, 77.0)
    assert api.li_rope(xd, pos.to(DEV), table, layout=layout, offset=offset, mscale=1.25, out=out) is out
    live = _check_rope(out, x, pos.tolist(), freq, layout, offset, 1.25)
    assert torch.equal(xd.cpu(), x)
    dead = ~torch.from_numpy(live.reshape(-1))
    assert (out.cpu()[dead] == 77).all()                     # padding is left as it was
    rest = torch.cat([out.cpu()[~dead][..., :offset], out.cpu()[~dead][..., offset + rot:]], -1)
    assert torch.equal(rest, torch.cat([x[~dead][..., :offset], x[~dead][..., offset + rot:]], -1))
    api.li_rope(xd, pos.to(DEV), table, layout=layout, offset=offset, mscale=1.25, out=xd)
    assert torch.equal(xd.cpu()[~dead], out.cpu()[~dead]) and torch.equal(xd.cpu()[dead], x[dead])
    assert api.li_get_last_error() == LI_OK


def test_rope_several_tensors_and_strides():
    """An indexer's query and key, an attention query's last 64 elements inside a fused buffer, a row: one launch."""
    g = torch.Generator().manual_seed(3)
    n = 6
    iq = torch.randn(n, 64, 128, generator=g).to(torch.bfloat16)
    ik = torch.randn(n, 128, generator=g)
    fused = torch.randn(n, 16 * 576 + 576, generator=g).to(torch.bfloat16)
    pos = torch.randint(0, 100000, (n,), generator=g).to(torch.int32)
    freq, table = oracle.rope_frequencies(64), api.li_rope_table(64)
    fd, old = fused.to(DEV), fused.clone()
    q, row = fd[:, :16 * 576].view(n, 16, 576), fd[:, 16 * 576:]
    outs = [torch.empty_like(iq, device=DEV), torch.empty_like(ik, device=DEV), q, row]
    got = api.li_rope([iq.to(DEV), ik.to(DEV), q, row], pos.to(DEV), table,
                      layout=["half", "half", "interleaved", "interleaved"], offset=[0, 0, 512, 512], out=outs)
    _check_rope(got[0], iq, pos.tolist(), freq, "half", 0, 1.0)
    _check_rope(got[1], ik, pos.tolist(), freq, "half", 0, 1.0)
    _check_rope(got[2], old[:, :16 * 576].view(n, 16, 576), pos.tolist(), freq, "interleaved", 512, 1.0)
    _check_rope(got[3], old[:, 16 * 576:], pos.tolist(), freq, "interleaved", 512, 1.0)
    # heads first in memory, an odd base address
    base = torch.randn(4 * n * 66 + 1, generator=g).to(torch.bfloat16)
    x = base.to(DEV)[1:].view(4, n, 66).transpose(0, 1)
    out = torch.empty_like(x)
    api.li_rope(x, pos.to(DEV), table, layout="half", offset=1, out=out)
    _check_rope(out, base[1:].view(4, n, 66).transpose(0, 1), pos.tolist(), freq, "half", 1, 1.0)
    empty = api.li_rope(torch.empty(0, 4, 64, device=DEV), _i32([]), table)
    assert empty.shape == (0, 4, 64) and api.li_get_last_error() == LI_OK


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rope_many_tokens(dtype, layout):
    """Sizes that go by bulk copies: heads that fill several stages, one head over many tokens, padding inside
    a block of tokens; a fused buffer's rows (a token stride of their own), and the same call in place."""
    g = torch.Generator(device=DEV).manual_seed(5)
    n, table, freq = 3001, api.li_rope_table(64), oracle.rope_frequencies(64)
    pos = torch.randint(0, 200000, (n,), generator=g, device=DEV, dtype=torch.int32)
    pos[torch.tensor([0, 7, 8, 9, 100, n - 1], device=DEV)] = -1
    fused = torch.randn(n, 20 * 192 + 192, generator=g, device=DEV).to(dtype)
    xs = [fused[:, :20 * 192].view(n, 20, 192), torch.randn(n, 128, generator=g, device=DEV).to(dtype),
          torch.randn(n, 1, 64, generator=g, device=DEV).to(dtype), fused[:, 20 * 192:]]
    offsets = [128, 0, 0, 64]
    outs = [torch.full_like(x, 7.0, memory_format=torch.contiguous_format) for x in xs]
    got = api.li_rope(xs, pos, table, layout=layout, offset=offsets, mscale=0.75, out=outs)
    assert api.li_get_last_error() == LI_OK
    some = np.r_[0:24, 90:110, 1490:1510, n - 20:n]
    dead = (pos < 0).cpu()
    for x, o, off in zip(xs, got, offsets):
        assert (o.cpu()[dead] == 7).all()
        _check_rope(o.cpu()[some], x.cpu()[some], pos.cpu().numpy()[some].tolist(), freq, layout, off, 0.75)
        rest = lambda v: torch.cat([v[..., :off], v[..., off + 64:]], -1).cpu()[~dead]  # noqa: E731
        assert torch.equal(rest(o), rest(x))
    for x, o in zip(xs, got):                       # every row, against the other form
        same = x.clone()
        api.li_rope(same, pos, table, layout=layout, offset=offsets[[id(v) for v in xs].index(id(x))], mscale=0.75, out=same)
        assert torch.equal(same[~dead.to(DEV)], o[~dead.to(DEV)])


def test_rope_refusals():
    table, pos = api.li_rope_table(64), _i32([1, 2])
    x = torch.zeros(2, 4, 128, device=DEV)
    for kw in [dict(layout="both"), dict(offset=65), dict(offset=-1), dict(out=x[:, :, :64]), dict(layout=["half"] * 2),
               dict(mscale=float("nan"))]:
        with pytest.raises((ValueError, api.LiError)):
            api.li_rope(x, pos, table, **kw)
    for bad in [x.half(), x[:1], x.transpose(1, 2), x.cpu(), [x] * 5, [], [x, x]]:
        with pytest.raises((ValueError, api.LiError)):
            api.li_rope(bad, pos, table, out=bad if isinstance(bad, list) else None)
    with pytest.raises(ValueError):
        api.li_rope(x, pos.long(), table)


# --------------------------------------------------------------------------- the 4-bit cache
@pytest.mark.parametrize("n,stride", [(1, 576), (31, 576), (1000, 584), (77, 579)])
def test_kv4_write_and_read(n, stride):
    g = torch.Generator().manual_seed(n)
    buf = torch.randn(n, stride, generator=g) * torch.exp(3 * torch.randn(n, 1, generator=g))
    buf = buf.to(torch.bfloat16)
    if n > 20:
        buf[3] = 0
        buf[4, :512] = 1e-5                       # scales round to zero
        buf[5, :64] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 8)   # ties
        buf[6, 7] = float("inf")
        buf[7, 20], buf[7, 40] = float("nan"), -float("inf")
        buf[8, 100:116] = torch.linspace(-2700, 2700, 16)
        buf[9, :512] = 3e38
        buf[10, :16] = -0.0
    rows = buf[:, :576]
    pages, page = n // 5 + 3, 7
    slots = torch.randperm(pages * page, generator=g)[:n]
    if n > 20:
        slots[11] = -1
    cache = torch.randint(0, 255, (pages, page, 416), dtype=torch.uint8, generator=g)
    cd = cache.to(DEV)
    rd = buf.to(DEV)[:, :576]
    assert api.li_kv4_write(rd, slots.to(DEV), cd) is cd
    want = cache.reshape(-1, 416).numpy().copy()
    packed = oracle.kv4_pack(rows)
    live = slots.numpy() >= 0
    want[slots.numpy()[live]] = packed[live]
    got = _np(cd).reshape(-1, 416)
    nan = np.zeros((want.shape[0], 416), bool)     # the codes of a block whose scale is NaN say nothing
    nan[:, :256] = np.repeat(want[:, 256:288] == 127, 8, axis=1)
    assert np.array_equal(np.where(nan, 0, got), np.where(nan, 0, want))
    back = api.li_kv4_read(cd, slots.to(DEV))
    ref = oracle.kv4_unpack(packed)
    ref[~live] = 0
    assert np.array_equal(back.cpu().double().numpy(), ref, equal_nan=True)     # exact
    assert api.li_get_last_error() == LI_OK


def test_kv4_every_code_and_scale_reads_exactly():
    """All 16 codes under all 256 scale bytes, through the read and through attention over one position."""
    raw = np.zeros((16, 416), np.uint8)
    raw[:, :256] = np.tile(np.arange(16, dtype=np.uint8).reshape(8, 2) @ np.array([1, 16], np.uint8), (16, 32))
    sc = np.arange(256, dtype=np.uint8)
    raw[:8, 256:288] = sc.reshape(8, 32)
    raw[8:, 256:288] = sc.reshape(8, 32)[::-1]
    raw[:, 256:288][raw[:, 256:288] >= 127] = 0    # scales the write makes: positive and finite
    ref = oracle.kv4_unpack(raw)
    cache = torch.from_numpy(raw).view(4, 4, 416).to(DEV)
    back = api.li_kv4_read(cache, torch.arange(16, device=DEV))
    assert np.array_equal(back.cpu().double().numpy(), ref)
    sel = torch.arange(16, dtype=torch.int32, device=DEV).view(16, 1)
    out = api.li_paged_sparse_attention(torch.randn(16, 3, 576, device=DEV).to(torch.bfloat16), cache, sel, 0.01,
                                        block_table=_i32([[0, 1, 2, 3]]), requests=_i32([0] * 16))
    for h in range(3):     # one position: its weight is 1 and the output the row itself
        assert np.array_equal(out[:, h].cpu().double().numpy(), ref[:, :512])


def test_kv4_bad_slots():
    rows = torch.randn(4, 576, device=DEV).to(torch.bfloat16)
    cache = torch.full((2, 3, 416), 9, dtype=torch.uint8, device=DEV)
    slots = torch.tensor([5, 6, -1, 1 << 40], device=DEV)
    api.li_kv4_write(rows, slots, cache)
    assert api.li_get_last_error() == LI_ERR_BOUNDS
    assert (cache.view(-1, 416)[:5] == 9).all() and (cache.view(-1, 416)[5] != 9).any()
    back = api.li_kv4_read(cache, slots)
    assert api.li_get_last_error() == LI_ERR_BOUNDS
    assert (back[1:] == 0).all() and (back[0] != 0).any()
    empty = torch.empty(0, dtype=torch.int64, device=DEV)
    api.li_kv4_write(rows[:0], empty, cache)
    assert api.li_kv4_read(cache, empty).shape == (0, 576) and api.li_get_last_error() == LI_OK
    for bad in [lambda: api.li_kv4_write(rows[:, :575], slots, cache), lambda: api.li_kv4_write(rows.float(), slots, cache),
                lambda: api.li_kv4_write(rows, slots.int(), cache), lambda: api.li_kv4_read(cache[:, :, :400], slots),
                lambda: api.li_kv4_write(rows[:1].expand(4, 576), slots, cache)]:
        with pytest.raises((ValueError, api.LiError)):
            bad()


# --------------------------------------------------------------------------- attention
class Case:
    """R requests of different lengths in a shuffled paged cache, T query tokens each."""

    def __init__(self, R, T, H, L, page, kind, seed, scale=0.07, shape=None):
        g = torch.Generator().manual_seed(seed)
        self.scale, self.page, self.kind = scale, page, kind
        blocks = -(-L // page)
        pages = R * blocks + 2
        rows = torch.randn(pages * page, 576, generator=g)
        if shape is not None:
            rows = shape(rows)
        rows = rows.to(torch.bfloat16)
        if kind == "kv4":
            raw = oracle.kv4_pack(rows)
            self.cache = torch.from_numpy(raw).view(pages, page, 416).to(DEV)
            self.rows = oracle.kv4_unpack(raw)
        else:
            self.cache = rows.view(pages, page, 576).to(DEV)
            self.rows = rows.double().numpy()
        self.table = torch.randperm(pages, generator=g)[:R * blocks].view(R, blocks).to(torch.int32)
        self.lens = [L if r == 0 else int(torch.randint(min(T, L), L + 1, (1,), generator=g)) for r in range(R)]
        self.req = [r for r in range(R) for _ in range(T)]
        self.pos = [self.lens[r] - T + i for r in range(R) for i in range(T)]
        self.q = torch.randn(R * T, H, 576, generator=g).to(torch.bfloat16)
        self.g = g

    def select(self, k):
        sel = np.full((len(self.req), k), -1, np.int32)
        for t, p in enumerate(self.pos):
            n = min(k, max(p + 1, 0))
            sel[t, :n] = np.sort(torch.randperm(p + 1, generator=self.g)[:n].numpy()) if n else []
        return sel

    def kw(self):
        return dict(block_table=self.table.to(DEV), requests=_i32(self.req))

    def check(self, out, lists, skip=()):
        got = out.detach().cpu().double().numpy()
        q = self.q.double().numpy()
        tab = self.table.numpy()
        for t, s in enumerate(lists):
            if t in skip:
                continue
            s = np.asarray(s, np.int64)
            rows = self.rows[tab[self.req[t], s // self.page].astype(np.int64) * self.page + s % self.page]
            ref, mag, top = oracle.attention(q[t], rows, self.scale)
            d = 2.0 ** -23 * (600 * top + 64 + len(s) / 16)
            bound = U * mag + U * np.abs(ref) + 2 * d[:, None] * mag
            err = np.abs(got[t] - ref)
            assert np.all(err <= bound), (t, float((err - bound).max()), float((err / (mag + 1e-30)).max()))


def _lists(sel):
    return [row[row >= 0] for row in sel]


@pytest.mark.parametrize("kind", ["kv4", "bf16"])
@pytest.mark.parametrize("R,T,H,L,page,k", [
    (1, 1, 64, 1, 1, 1), (1, 1, 64, 300, 64, 128), (2, 1, 128, 3000, 64, 2048), (3, 2, 16, 700, 48, 129),
    (5, 3, 1, 200, 7, 64), (2, 1, 130, 900, 16, 300), (200, 1, 8, 260, 16, 256), (40, 2, 100, 400, 33, 400)])
def test_paged_sparse_attention(kind, R, T, H, L, page, k):
    c = Case(R, T, H, L, page, kind, seed=R * 7 + k)
    sel = c.select(k)
    out = api.li_paged_sparse_attention(c.q.to(DEV), c.cache, torch.from_numpy(sel).to(DEV), c.scale, **c.kw())
    c.check(out, _lists(sel))
    assert api.li_get_last_error() == LI_OK


@pytest.mark.parametrize("kind", ["kv4", "bf16"])
@pytest.mark.parametrize("R,T,H,L,page,window,sinks", [
    (1, 1, 64, 1, 1, 1, 0), (3, 1, 64, 500, 64, 1, 0), (3, 1, 64, 500, 64, 1, 3), (2, 1, 128, 3000, 64, 512, 4),
    (4, 2, 16, 1000, 48, 100, 300), (2, 1, 64, 777, 16, 10 ** 9, 0), (1, 200, 64, 400, 64, 130, 5),
    (2, 90, 72, 300, 1, 33, 64), (6, 3, 8, 150, 7, 127, 1), (1, 1, 128, 9000, 64, 9000, 9000)])
def test_window_attention(kind, R, T, H, L, page, window, sinks):
    c = Case(R, T, H, L, page, kind, seed=R * 11 + L)
    out = api.li_window_attention(c.q.to(DEV), c.cache, _i32(c.pos), c.scale, window, sinks=sinks, **c.kw())
    c.check(out, [oracle.visible(p, window, sinks) for p in c.pos])
    out = api.li_window_attention(c.q.to(DEV), c.cache, _i32(c.pos), c.scale, window, sinks=sinks, max_len=max(c.lens),
                                  **c.kw())
    c.check(out, [oracle.visible(p, window, sinks) for p in c.pos])
    assert api.li_get_last_error() == LI_OK


@pytest.mark.parametrize("kind", ["kv4", "bf16"])
def test_attention_maximum_that_keeps_rising(kind):
    """Logits that grow along the context: every tile raises the maximum and rescales what came before; and
    ones that fall, where later tiles vanish against the first."""
    def ramp(up):
        step = torch.linspace(0.1, 40.0, 2000)
        step = step if up else step.flip(0)
        return lambda x: torch.cat([x[:, :512], step.repeat(x.shape[0] // 2000)[:, None].expand(-1, 64)], 1)

    for up in (True, False):
        c = Case(1, 1, 64, 2000, 2000, kind, seed=2, scale=0.3, shape=ramp(up))
        c.table[:] = 0
        c.q = torch.cat([c.q[:, :, :512] * 0.05, c.q[:, :, 512:].abs()], 2).to(torch.bfloat16)
        out = api.li_window_attention(c.q.to(DEV), c.cache, _i32(c.pos), c.scale, 10 ** 6, **c.kw())
        c.check(out, [np.arange(2000)])


@pytest.mark.parametrize("kind", ["kv4", "bf16"])
@pytest.mark.parametrize("R,H,k", [(1, 64, 2048), (8, 128, 2048), (40, 256, 512), (20, 16, 1000), (40, 96, 500)])
def test_attention_holes_before_far_negative_logits(kind, R, H, k):
    """Every second tile of 128 list entries has nothing, the first among them, and every logit is far below zero:
    the weights are taken against the logits that are there, whatever the empty tiles left as a maximum."""
    c = Case(R, 1, H, 3000, 64, kind, seed=R + k, scale=0.3,
             shape=lambda x: torch.cat([x[:, :512], 20 + 4 * x[:, 512:].abs()], 1))
    c.q = torch.cat([c.q[:, :, :512] * 0.05, -2 - c.q[:, :, 512:].abs()], 2).to(torch.bfloat16)
    sel = c.select(k)
    for a in range(0, k, 256):
        sel[:, a:a + 128] = -1
    out = api.li_paged_sparse_attention(c.q.to(DEV), c.cache, torch.from_numpy(sel).to(DEV), c.scale, **c.kw())
    c.check(out, _lists(sel))
    assert api.li_get_last_error() == LI_OK


@pytest.mark.parametrize("R,H,k", [(1, 64, 2048), (8, 128, 2048), (40, 256, 512)])
def test_attention_nan_in_a_visible_place_is_passed_on(R, H, k):
    """Split or whole: a head whose query is NaN gives NaN, and so does every head of a token that selects a NaN row;
    the others are as they would be."""
    c = Case(R, 1, H, 3000, 64, "bf16", seed=k)
    sel = c.select(k)
    s = int(sel[0, 1])
    c.cache.view(-1, 576)[int(c.table[0, s // 64]) * 64 + s % 64] = float("nan")
    q = c.q.to(DEV)
    q[R - 1, 5] = float("nan")
    out = api.li_paged_sparse_attention(q, c.cache, torch.from_numpy(sel).to(DEV), c.scale, **c.kw())
    assert out[0].isnan().all() and out[R - 1, 5].isnan().all()
    if R > 1:
        keep = [h for h in range(H) if h != 5]
        assert not out[1:, keep].isnan().any()
        c.check(out, _lists(sel), skip=(0, R - 1))


def test_attention_masks():
    """Rows with nothing selected, holes and repeats in the list, padding tokens left as they were, NaN and
    infinities in rows that nothing selects."""
    c = Case(6, 1, 64, 1000, 16, "bf16", seed=9)
    sel = c.select(400)
    sel[0] = -1                                   # nothing: zeros
    sel[1, ::2] = -1                              # holes
    sel[2, 130:300] = -1                          # a whole tile of the list without one
    sel[3, :200] = sel[3, 0]                      # repeats
    c.req[4] = -1                                 # padding
    used = np.unique(np.concatenate([c.table.numpy()[r, s // 16].astype(np.int64) * 16 + s % 16
                                     for r, s in zip(c.req, _lists(sel)) if r >= 0]))
    poison = torch.full((c.cache.shape[0] * 16, 576), float("nan"), dtype=torch.bfloat16)
    poison[::3] = float("inf")
    flat = c.cache.view(-1, 576)
    poison[used] = flat[used].cpu()
    flat.copy_(poison.to(DEV))
    out = torch.full((6, 64, 512), 5.0, dtype=torch.bfloat16, device=DEV)
    api.li_paged_sparse_attention(c.q.to(DEV), c.cache, torch.from_numpy(sel).to(DEV), c.scale, out=out, **c.kw())
    c.check(out, _lists(sel), skip=(4,))
    assert (out[0] == 0).all() and (out[4] == 5).all()
    pos = list(c.pos)
    pos[1] = -1
    flat.copy_(torch.randn_like(flat))
    c.rows = flat.cpu().double().numpy()
    out.fill_(5.0)
    api.li_window_attention(c.q.to(DEV), c.cache, _i32(pos), c.scale, 200, sinks=2, out=out, **c.kw())
    c.check(out, [oracle.visible(max(p, 0), 200, 2) for p in pos], skip=(1, 4))
    assert (out[1] == 5).all() and (out[4] == 5).all()
    none = torch.empty(6, 0, dtype=torch.int32, device=DEV)
    out.fill_(5.0)
    api.li_paged_sparse_attention(c.q.to(DEV), c.cache, none, c.scale, out=out, **c.kw())
    assert (out[4] == 5).all() and (out[[0, 1, 2, 3, 5]] == 0).all()
    assert api.li_get_last_error() == LI_OK


@pytest.mark.parametrize("kind", ["kv4", "bf16"])
def test_attention_reports_negative_selections_other_than_none(kind):
    """-2 and the lowest integer, alone among real positions and in place of whole runs, are skipped and reported."""
    c = Case(3, 1, 64, 700, 16, kind, seed=31)
    sel = c.select(400)
    sel[0, ::3] = -2
    sel[1, 64:200] = -2
    sel[1, 300] = np.iinfo(np.int32).min
    sel[2, 399] = -3
    out = api.li_paged_sparse_attention(c.q.to(DEV), c.cache, torch.from_numpy(sel).to(DEV), c.scale, **c.kw())
    assert api.li_get_last_error() == LI_ERR_BOUNDS
    c.check(out, _lists(sel))
    sel[sel < 0] = -1
    again = api.li_paged_sparse_attention(c.q.to(DEV), c.cache, torch.from_numpy(sel).to(DEV), c.scale, **c.kw())
    assert torch.equal(out, again) and api.li_get_last_error() == LI_OK


def test_attention_dense_cache():
    """No block table: request r's positions are page r, as a dense [R, L] cache holds them."""
    c = Case(3, 1, 64, 500, 500, "bf16", seed=4)
    c.table = torch.arange(3, dtype=torch.int32).view(3, 1)
    sel = c.select(200)
    got = api.li_paged_sparse_attention(c.q.to(DEV), c.cache, torch.from_numpy(sel).to(DEV), c.scale)
    c.check(got, _lists(sel))
    ref = api.li_sparse_attention(c.q.to(DEV), c.cache[:3].contiguous(), torch.from_numpy(sel).to(DEV), c.scale)
    assert (got.float() - ref).abs().max() <= 4 * U * ref.abs().max()


@pytest.mark.parametrize("what", ["position", "page", "request", "window position"])
def test_attention_reports_what_is_out_of_range(what):
    c = Case(3, 1, 64, 300, 16, "kv4", seed=6)
    sel = c.select(200)
    lists, skip = _lists(sel), ()
    table = c.table.clone()
    out = torch.full((3, 64, 512), 5.0, dtype=torch.bfloat16, device=DEV)
    if what == "position":
        sel[1, 3] = table.shape[1] * 16
        lists[1] = np.delete(lists[1], 3)
    elif what == "page":
        b = sel[1, 5] // 16
        table[1, b] = c.cache.shape[0]
        lists[1] = lists[1][lists[1] // 16 != b]
    elif what == "request":
        c.req[2], skip = 3, (2,)
    if what == "window position":
        api.li_window_attention(c.q.to(DEV), c.cache, _i32([c.pos[0], 304, c.pos[2]]), c.scale, 50, out=out, **c.kw())
        lists, skip = [oracle.visible(p, 50, 0) for p in c.pos], (1,)
    else:
        api.li_paged_sparse_attention(c.q.to(DEV), c.cache, torch.from_numpy(sel).to(DEV), c.scale, out=out,
                                      block_table=table.to(DEV), requests=_i32(c.req))
    assert api.li_get_last_error() == LI_ERR_BOUNDS
    c.check(out, lists, skip)
    for t in skip:
        assert (out[t] == 5).all()


def test_attention_on_another_stream_and_in_a_graph():
    c = Case(4, 1, 128, 2500, 64, "kv4", seed=8)
    sel = torch.from_numpy(c.select(1500)).to(DEV)
    q, kw = c.q.to(DEV), c.kw()
    want = api.li_paged_sparse_attention(q, c.cache, sel, c.scale, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = [api.li_paged_sparse_attention(q, c.cache, sel, c.scale, stream=side if i % 2 else None, **kw)
            for i in range(6)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    out = torch.zeros_like(want)
    pos = _i32(c.pos)
    win = api.li_window_attention(q, c.cache, pos, c.scale, 700, sinks=3, **kw)
    wout = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.li_paged_sparse_attention(q, c.cache, sel, c.scale, out=out, **kw)
        api.li_window_attention(q, c.cache, pos, c.scale, 700, sinks=3, out=wout, **kw)
    for _ in range(3):
        out.zero_()
        wout.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(wout, win)
    q.mul_(-1)                                     # a replay works on the inputs' present values
    graph.replay()
    assert torch.equal(out, api.li_paged_sparse_attention(q, c.cache, sel, c.scale, **kw))
    assert api.li_get_last_error() == LI_OK


def test_attention_two_calls_at_once_with_workspaces_of_their_own():
    """Split plans on two streams: each call's parts lie in its own workspace; and a workspace that is too small is
    not used."""
    c = Case(6, 1, 64, 3000, 64, "kv4", seed=14)
    q, kw = [c.q.to(DEV), (-c.q).to(DEV)], c.kw()
    sel = torch.from_numpy(c.select(2048)).to(DEV)
    want = [api.li_paged_sparse_attention(x, c.cache, sel, c.scale, **kw) for x in q]
    ws = [api.li_paged_attention_workspace(6, 64, 2048, DEV) for _ in range(2)]
    assert ws[0].numel() > 6 * 64 * 512 * 4
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [torch.empty_like(want[0]) for _ in range(2)]
    for _ in range(20):
        for i in range(2):
            api.li_paged_sparse_attention(q[i], c.cache, sel, c.scale, out=outs[i], workspace=ws[i], stream=streams[i], **kw)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    small = torch.empty(256, dtype=torch.uint8, device=DEV)
    assert torch.equal(api.li_paged_sparse_attention(q[0], c.cache, sel, c.scale, workspace=small, **kw), want[0])
    assert api.li_get_last_error() == LI_OK


def test_out_of_memory_is_torchs_own_error():
    """A call whose output the allocator refuses raises what torch raises, and the next call works."""
    cache = api.li_kv4_cache(4, 16)
    slots = torch.zeros(1 << 21, dtype=torch.int64, device=DEV)        # (out: 2.4 GB)
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (1 << 29)) / total)
    try:
        with pytest.raises(torch.OutOfMemoryError):
            api.li_kv4_read(cache, slots)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert (api.li_kv4_read(cache, slots[:7]) == 0).all() and api.li_get_last_error() == LI_OK


def test_new_outputs_of_a_call_are_apart_and_outlive_each_other():
    """Outputs that share an allocation: any of them can be written, kept or dropped without the others."""
    g = torch.Generator().manual_seed(8)
    xs = [torch.randn(s, generator=g).to(t).to(DEV) for s, t in
          [((5, 3, 64), torch.bfloat16), ((5, 64), torch.float32), ((5, 7, 100), torch.bfloat16), ((5, 1, 66), torch.float32)]]
    pos, table = _i32([0, 9, -1, 70000, 3]), api.li_rope_table(64)
    live = [0, 1, 3, 4]
    want = [torch.zeros_like(x) for x in xs]
    api.li_rope(xs, pos, table, out=want)
    outs = api.li_rope(xs, pos, table)
    assert all(o.is_contiguous() and o.shape == x.shape and o.dtype == x.dtype for o, x in zip(outs, xs))
    assert all(torch.equal(o[live], w[live]) for o, w in zip(outs, want))
    outs[1].fill_(5)
    assert all(torch.equal(outs[i][live], want[i][live]) for i in (0, 2, 3))
    last = outs.pop()
    del outs
    torch.full((1 << 16,), 7.0, device=DEV)
    assert torch.equal(last[live], want[3][live])
    assert api.li_rope(xs[0][:0], pos[:0], table).shape == (0, 3, 64)
    tables = api.li_block_tables(_i32([5, 2]), _i32([1, 2]), _i32([[3, -1], [-1, -1]]), _i32([6, 7]), 4, 8, 3)
    got = [_np(x) for x in tables]
    tables[0].fill_(-9)
    assert all(np.array_equal(_np(x), w) for x, w in zip(tables[1:], got[1:])) and got[3].tolist() == [0, 1, 3]
    assert api.li_get_last_error() == LI_OK


@pytest.mark.parametrize("kind", ["kv4", "bf16"])
def test_attention_gives_the_same_bits_again(kind):
    """No sum depends on the order in which CTAs run."""
    c = Case(9, 2, 40, 1500, 16, kind, seed=21)
    q, kw, pos = c.q.to(DEV), c.kw(), _i32(c.pos)
    outs = [api.li_window_attention(q, c.cache, pos, c.scale, 1100, sinks=9, **kw) for _ in range(4)]
    assert all(torch.equal(o, outs[0]) for o in outs)


def test_attention_without_pages_or_rows():
    q = torch.randn(2, 16, 576, device=DEV).to(torch.bfloat16)
    for cache in (api.li_kv4_cache(0, 16), torch.empty(0, 16, 576, dtype=torch.bfloat16, device=DEV)):
        table = torch.zeros(2, 3, dtype=torch.int32, device=DEV)
        sel = torch.full((2, 5), -1, dtype=torch.int32, device=DEV)
        assert (api.li_paged_sparse_attention(q, cache, sel, 0.1, block_table=table) == 0).all()
        assert api.li_get_last_error() == LI_OK
        sel[1, 2] = 7                              # a position whose page (0) does not exist
        assert (api.li_paged_sparse_attention(q, cache, sel, 0.1, block_table=table) == 0).all()
        assert api.li_get_last_error() == LI_ERR_BOUNDS
        assert api.li_paged_sparse_attention(q[:0], cache, sel[:0], 0.1, block_table=table[:0]).shape == (0, 16, 512)
        none = torch.empty(0, dtype=torch.int32, device=DEV)
        assert api.li_window_attention(q[:0], cache, none, 0.1, 4, block_table=table[:0]).shape == (0, 16, 512)
    assert api.li_get_last_error() == LI_OK


def test_attention_over_slots_beyond_four_gigabytes():
    """A cache of 4.6 GB: the bytes of its last rows lie past 32 bits."""
    page, pages = 64, 173000
    cache = torch.empty(pages, page, 416, dtype=torch.uint8, device=DEV)
    table = torch.tensor([[pages - 1, 0, pages - 3, pages - 2]], dtype=torch.int32)
    n = 4 * page - 5
    g = torch.Generator().manual_seed(5)
    rows = torch.randn(n, 576, generator=g).to(torch.bfloat16)
    s = np.arange(n)
    slots = torch.from_numpy(table.numpy()[0, s // page].astype(np.int64) * page + s % page).to(DEV)
    api.li_kv4_write(rows.to(DEV), slots, cache)
    held = oracle.kv4_unpack(oracle.kv4_pack(rows))
    assert np.array_equal(api.li_kv4_read(cache, slots).double().cpu().numpy(), held)
    q = torch.randn(1, 64, 576, generator=g).to(torch.bfloat16)
    out = api.li_window_attention(q.to(DEV), cache, _i32([n - 1]), 0.06, n, block_table=table.to(DEV))
    ref, mag, top = oracle.attention(q[0].double().numpy(), held, 0.06)
    d = 2.0 ** -23 * (600 * top + 64 + n / 16)
    err = np.abs(out[0].double().cpu().numpy() - ref)
    assert np.all(err <= U * mag + U * np.abs(ref) + 2 * d[:, None] * mag)
    assert api.li_get_last_error() == LI_OK


def test_attention_refusals():
    c = Case(2, 1, 64, 100, 16, "kv4", seed=1)
    q, sel, kw = c.q.to(DEV), torch.from_numpy(c.select(50)).to(DEV), c.kw()
    call = api.li_paged_sparse_attention
    for bad in [lambda: call(q.float(), c.cache, sel, 0.1, **kw), lambda: call(q[:, :, :512], c.cache, sel, 0.1, **kw),
                lambda: call(q, c.cache.float(), sel, 0.1, **kw), lambda: call(q, c.cache, sel.long(), 0.1, **kw),
                lambda: call(q, c.cache, sel[:1], 0.1, **kw), lambda: call(q, c.cache, sel, 0.0, **kw),
                lambda: call(q, c.cache, sel, 0.1, block_table=kw["block_table"], requests=_i32([0])),
                lambda: call(q, c.cache, sel, 0.1, block_table=kw["block_table"][:1]),
                lambda: call(q, c.cache, sel, 0.1, out=torch.empty(2, 64, 512, device=DEV), **kw),
                lambda: call(q.transpose(0, 1), c.cache, sel, 0.1, **kw),
                lambda: api.li_window_attention(q, c.cache, _i32([1, 2]), 0.1, 0, **kw),
                lambda: api.li_window_attention(q, c.cache, _i32([1, 2]), 0.1, 5, sinks=-1, **kw),
                lambda: api.li_window_attention(q, c.cache, _i32([1, 2]), 0.1, 5, max_len=10 ** 6, **kw),
                lambda: api.li_window_attention(q, c.cache, _i32([1]), 0.1, 5, **kw)]:
        with pytest.raises((ValueError, api.LiError)):
            bad()


# --------------------------------------------------------------------------- together
@pytest.mark.parametrize("layer", ["selection", "window"])
def test_from_lengths_to_attention(layer):
    """A prefill chunk beside decode tokens, step after step: tables and slots from the lengths, rotation of
    queries and rows in one launch, the rows into the 4-bit cache, the attention over it; against a dense record
    of every row kept on the host."""
    page, pages, R, H, blocks = 16, 80, 4, 64, 24
    g = torch.Generator().manual_seed(12)
    freq, rope = oracle.rope_frequencies(64), api.li_rope_table(64)
    cache = api.li_kv4_cache(pages, page)
    table = torch.full((R, blocks), -1, dtype=torch.int32, device=DEV)
    free = torch.randperm(pages, generator=g).to(torch.int32).to(DEV)
    start = _i32([0])
    seen = [np.zeros((0, 576)) for _ in range(R)]
    lens = np.zeros(R, int)
    for new in [(130, 1, 40, 0), (1, 1, 1, 200), (1, 1, 0, 1), (3, 3, 3, 3)]:
        lens = lens + np.array(new)
        cap = sum(new) + 5                                     # a padded batch
        slots, pos, req, starts, start = api.li_block_tables(_i32(lens), _i32(new), table, free, page, pages, cap,
                                                             free_start=start)
        q = torch.randn(cap, H, 576, generator=g).to(torch.bfloat16)
        row = torch.randn(cap, 576, generator=g).to(torch.bfloat16)
        qd, rd = q.to(DEV), row.to(DEV)
        api.li_rope([qd, rd], pos, rope, offset=512, out=[qd, rd])
        api.li_kv4_write(rd, slots, cache)
        out = torch.full((cap, H, 512), 5.0, dtype=torch.bfloat16, device=DEV)
        P, Q = pos.tolist(), req.tolist()
        for t in range(sum(new)):
            y = oracle.rope(row[t].double().numpy().reshape(1, 1, 576), [P[t]], freq, "interleaved", 512, 1.0)
            y = torch.from_numpy(y).view(1, 576)
            # the rotated row as the device holds it (its rounding is checked by the rotation's own test)
            assert (rd[t].cpu().double() - y[0]).abs().max() <= U * y.abs().max()
            seen[Q[t]] = np.concatenate([seen[Q[t]], oracle.kv4_unpack(oracle.kv4_pack(rd[t:t + 1]))])
        if layer == "window":
            api.li_window_attention(qd, cache, pos, 0.06, 50, sinks=4, block_table=table, requests=req, out=out)
            lists = [oracle.visible(P[t], 50, 4) for t in range(sum(new))]
        else:
            scores = torch.randn(cap, 256, generator=g).to(DEV)
            sel = api.li_topk(scores, 64, lens=(pos + 1).clamp(max=256))
            api.li_paged_sparse_attention(qd, cache, sel, 0.06, block_table=table, requests=req, out=out)
            lists = _lists(_np(sel))[:sum(new)]
        for t, s in enumerate(lists):
            ref, mag, top = oracle.attention(qd[t].cpu().double().numpy(), seen[Q[t]][s], 0.06)
            d = 2.0 ** -23 * (600 * top + 64 + len(s) / 16)
            err = np.abs(out[t].cpu().double().numpy() - ref)
            assert np.all(err <= U * mag + U * np.abs(ref) + 2 * d[:, None] * mag), (new, t)
        assert (out[sum(new):] == 5).all()
    assert api.li_get_last_error() == LI_OK


@pytest.mark.parametrize("L", [900, 897])          # the new token inside a page, and first of a new one
def test_decode_layers_over_a_paged_4bit_cache(L):
    """The decode step over layers, two streams, captured and replayed: each layer's output against the definition
    on the cache that the step left."""
    from sparse_attention_lightning_score_b200.schedule import DecodeLayerStack, StepGraph, mli_plan, priority_streams
    B, H, k, page = 3, 24, 256, 64
    stack = DecodeLayerStack(n_layers=3, B=B, L=L, k=k, att_heads=H, device=DEV, seed=2, page_size=page)
    step = stack.bind(mli_plan(3, lag=1))
    main, side = priority_streams()
    main.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(main):
        step.run(main, side)
    torch.cuda.synchronize()
    first = stack.out.clone()
    table = _np(stack.block_table)
    assert (np.sort(table.reshape(-1)) == np.arange(table.size)).all()
    pos, rope = _i32([L - 1] * B), api.li_rope_table(64)
    slots = table[:, (L - 1) // page] * page + (L - 1) % page
    assert np.array_equal(_np(stack.step_map["slots"]), slots)
    for layer, p in enumerate(step.plan):
        raw = _np(stack.kv[layer]).reshape(-1, 416)
        # the rotated rows and queries as the device holds them (their rounding is checked by the rotation's own tests)
        q, row = api.li_rope([stack.qa[layer], stack.row[layer]], pos, rope, offset=512)
        assert np.array_equal(raw[slots], oracle.kv4_pack(row.cpu()))
        slot = step.slots[p.attends]
        assert max(i for i, w in enumerate(step.plan) if w.runs_indexer and step.slots[i] == slot) == p.attends
        for b, s in enumerate(_lists(_np(stack.sel[slot]))):
            s = s.astype(np.int64)
            rows = oracle.kv4_unpack(raw[table[b, s // page].astype(np.int64) * page + s % page])
            ref, mag, top = oracle.attention(q[b].cpu().double().numpy(), rows, stack.scale)
            d = 2.0 ** -23 * (600 * top + 64 + len(s) / 16)
            err = np.abs(first[layer, b].cpu().double().numpy() - ref)
            assert len(s) == k and np.all(err <= U * mag + U * np.abs(ref) + 2 * d[:, None] * mag), (layer, b)
    with torch.cuda.stream(main):
        graph = StepGraph(step, main, side)
        for _ in range(2):
            stack.out.zero_()
            graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(stack.out, first)
    graph.close()
    assert api.li_get_last_error() == LI_OK
