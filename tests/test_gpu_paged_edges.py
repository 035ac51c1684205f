"""Paged-cache operators at edges: tensors that share a buffer, heads over several stages of a bulk copy, two rows a warp
into the 4-bit cache, values that all rows have in common, NaN far below the maximum.  Definitions: oracle.paged."""
import numpy as np
import pytest
import torch

from oracle import paged as oracle
from sparse_attention_lightning_score_b200 import api
from sparse_attention_lightning_score_b200._lib import LI_ERR_BOUNDS, LI_OK
from tests.test_gpu_paged import DEV, U, Case, _check_rope, _i32, _np

pytestmark = pytest.mark.gpu


def test_rope_tensors_of_a_call_that_share_a_buffer():
    """The two halves of one fused buffer, both in place, turn as they do apart; a tensor that reads or writes what
    another one writes is refused, and nothing changes."""
    g = torch.Generator().manual_seed(4)
    pos, table = _i32([3, 70000, 12]), api.li_rope_table(64)
    fused = torch.randn(3, 4 * 128, generator=g).to(torch.bfloat16).to(DEV)
    old = fused.clone()
    halves = lambda b: [b[:, :256].view(3, 2, 128), b[:, 256:].view(3, 2, 128)]  # noqa: E731
    want = [api.li_rope(h, pos, table) for h in halves(old)]
    got = api.li_rope(halves(fused), pos, table, out=halves(fused))
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and api.li_get_last_error() == LI_OK
    fused.copy_(old)
    heads = fused.view(3, 4, 128)
    for xs in [[heads[:, :2], heads[:, 1:3]], [heads[:, :2], heads[:, :2]]]:    # the first one's second head; the same
        with pytest.raises(api.LiError):
            api.li_rope(xs, pos, table, out=xs)
    with pytest.raises(api.LiError):                  # reads past its half, into what the other writes
        api.li_rope([heads[:, 2:], heads[:, :3]], pos, table, out=[heads[:, 2:], torch.empty(3, 3, 128, device=DEV,
                                                                                             dtype=torch.bfloat16)])
    assert torch.equal(fused, old)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("n,heads,dim,offset", [(301, 43, 192, 128), (301, 127, 192, 64), (67, 128, 576, 512)])
def test_rope_heads_over_several_stages(dtype, layout, n, heads, dim, offset):
    """Sizes that go by bulk copies (2 MB and more, out of place) whose tokens fill several 16 KB stages, the last of them
    shorter (43 heads of 192 in bf16: 22 and 21; 128 of 576: nine of 13 and 11), beside tensors of one stage, with
    padding: every row as the in-place form makes it, and some against the definition."""
    g = torch.Generator(device=DEV).manual_seed(heads)
    table, freq = api.li_rope_table(64), oracle.rope_frequencies(64)
    pos = torch.randint(0, 200000, (n,), generator=g, device=DEV, dtype=torch.int32)
    pos[torch.tensor([0, 7, 8, 50, n - 1], device=DEV)] = -1
    xs = [torch.randn(s, generator=g, device=DEV).to(dtype) for s in [(n, heads, dim), (n, 128), (n, 3, dim)]]
    assert sum(x.numel() * x.element_size() for x in xs) >= 2 << 20
    offsets = [offset, 32, offset]
    outs = [torch.full_like(x, 7.0) for x in xs]
    got = api.li_rope(xs, pos, table, layout=layout, offset=offsets, mscale=1.5, out=outs)
    assert api.li_get_last_error() == LI_OK
    dead, some = pos < 0, np.r_[0:10, 48:52, n - 4:n]
    for x, o, off in zip(xs, got, offsets):
        assert (o[dead] == 7).all()
        same = x.clone()
        api.li_rope(same, pos, table, layout=layout, offset=off, mscale=1.5, out=same)
        assert torch.equal(same[~dead], o[~dead])
        _check_rope(o.cpu()[some], x.cpu()[some], pos.cpu().numpy()[some].tolist(), freq, layout, off, 1.5)


# --------------------------------------------------------------------------- the 4-bit cache
@pytest.mark.parametrize("n", [16383, 16384, 16385, 20001])
@pytest.mark.parametrize("stride", [576, 584, 577])
def test_kv4_write_of_many_rows(n, stride):
    """From 16384 rows on a warp takes two (where rows are 16-byte aligned): padding and bad slots in the first and in the
    second row of a pair, an odd last row, ones that are none; byte for byte what calls of fewer rows leave."""
    g = torch.Generator(device=DEV).manual_seed(n)
    rows = torch.randn(n, stride, generator=g, device=DEV).to(torch.bfloat16)[:, :576]
    page, pages = 64, n // 64 + 3
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:n]
    for i, bad in [(10, -1), (21, -1), (30, pages * page), (41, 1 << 40), (52, -1), (53, pages * page), (n - 2, -1)]:
        slots[i] = bad
    if n % 2:
        slots[n - 1] = pages * page - 1 if (slots != pages * page - 1).all() else slots[n - 1]
    cache = torch.randint(0, 255, (pages, page, 416), dtype=torch.uint8, generator=g, device=DEV)
    want = cache.clone()
    good = ((slots >= 0) & (slots < pages * page)).nonzero()[:, 0]
    for part in good.split(5000):
        api.li_kv4_write(rows[part], slots[part], want)
    assert api.li_get_last_error() == LI_OK
    api.li_kv4_write(rows, slots, cache)
    assert api.li_get_last_error() == LI_ERR_BOUNDS
    assert torch.equal(cache, want)
    some = torch.cat([good[:30], good[40:60], good[-9:]])
    assert np.array_equal(_np(cache.view(-1, 416)[slots[some]]), oracle.kv4_pack(rows[some].cpu()))
    back = api.li_kv4_read(cache, slots)
    assert api.li_get_last_error() == LI_ERR_BOUNDS
    keep = torch.zeros(n, dtype=torch.bool, device=DEV)
    keep[good] = True
    assert (back[~keep] == 0).all()
    assert np.array_equal(back[some].cpu().double().numpy(), oracle.kv4_unpack(oracle.kv4_pack(rows[some].cpu())))


def test_kv4_range_of_the_scales():
    """Blocks around the least absmax that does not read as zeros, the least of a normal scale and the largest that does
    not saturate; and the same rows times a power of two, which the attention's scale and output undo."""
    tops = [6 * 2.0 ** -10, 6 * 2.0 ** -10 * (1 + 2.0 ** -7), 6 * 2.0 ** -6, 6 * 2.0 ** -6 * (1 - 2.0 ** -8), 2688.0, 2704.0,
            1e30, 0.0]
    x = torch.zeros(1, 576)
    for b, top in enumerate(tops):
        x[0, 16 * b:16 * b + 16] = torch.linspace(-1, 1, 16) * top
    rows = x.to(torch.bfloat16)
    cache = api.li_kv4_write(rows.to(DEV), torch.tensor([0], device=DEV), api.li_kv4_cache(1, 1))
    raw = oracle.kv4_pack(rows)
    assert np.array_equal(_np(cache).reshape(1, 416), raw)
    assert raw[0, 256:264].tolist() == [0, 1, 0x08, 0x08, 0x7e, 0x7e, 0x7e, 0]
    assert np.abs(oracle.kv4_unpack(raw))[0, 16 * 4:16 * 7].max() == 2688

    g = torch.Generator().manual_seed(17)
    small = (torch.randn(300, 576, generator=g) * 2.0 ** -12).to(torch.bfloat16)
    q, f, scale = torch.randn(1, 64, 576, generator=g).to(torch.bfloat16), 2.0 ** 12, 300.0
    held = api.li_kv4_write((small * f).to(DEV), torch.arange(300, device=DEV), api.li_kv4_cache(3, 100))
    table = _i32([[0, 1, 2]])
    got = api.li_window_attention(q.to(DEV), held, _i32([299]), scale / f, 300, block_table=table)
    ref, mag, top = oracle.attention(q[0].double().numpy(), oracle.kv4_unpack(oracle.kv4_pack(small * f)) / f, scale)
    d = 2.0 ** -23 * (600 * top + 64 + 300 / 16)     # (the bound of test_gpu_paged, and the sum's share of the weights)
    err = np.abs((got / f)[0].cpu().double().numpy() - ref)
    assert np.all(err <= 2 * U * mag + U * np.abs(ref) + 2 * d[:, None] * mag)


@pytest.mark.parametrize("kind", ["kv4", "bf16"])
@pytest.mark.parametrize("R,H,L,k", [(1, 64, 300, 300), (2, 128, 3000, 2048), (40, 256, 600, 512), (80, 16, 1100, 1000),
                                     (150, 8, 500, 400), (3, 100, 900, 900)])
def test_attention_gives_back_what_all_rows_have_in_common(kind, R, H, L, k):
    """Every row has the same latent elements and only the rotary ones differ: whatever the weights, the output is
    those elements.  They are bf16, and fp32 sums of at most 2048 terms are off by less than 2^-12 of the value, below
    the half step of 2^-9 and more at which the output's rounding would leave it."""
    c = Case(R, 1, H, L, 64, kind, seed=R + k, scale=0.3,
             shape=lambda x: torch.cat([x[:1, :512].expand(x.shape[0], -1), x[:, 512:] * 3], 1))
    sel = c.select(k)
    q = c.q.to(DEV)
    want = torch.from_numpy(c.rows[0, :512]).to(torch.bfloat16).to(DEV)
    assert np.array_equal(want.double().cpu().numpy(), c.rows[0, :512])
    out = api.li_paged_sparse_attention(q, c.cache, torch.from_numpy(sel).to(DEV), c.scale, **c.kw())
    assert (out == want).all()
    out = api.li_window_attention(q, c.cache, _i32(c.pos), c.scale, k, sinks=3, **c.kw())
    assert (out == want).all() and api.li_get_last_error() == LI_OK


@pytest.mark.parametrize("kind", ["kv4", "bf16"])
@pytest.mark.parametrize("where", [(5,), tuple(range(128)), (2047,)])
@pytest.mark.parametrize("R,H", [(1, 64), (8, 128), (40, 256)])
def test_attention_nan_far_below_the_maximum_is_passed_on(kind, where, R, H):
    """A visible NaN row, or a tile of nothing else, among logits so far below the maximum that their weights
    underflow: every head is NaN, in parts (the first two) or in one piece (the last)."""
    L = 2048
    level = torch.full((L, 1), 40.0)
    level[:128], level[1900:] = -40.0, -40.0
    c = Case(R, 1, H, L, L, kind, seed=3, scale=0.3,
             shape=lambda x: torch.cat([x[:, :512], level.repeat(x.shape[0] // L, 1).expand(-1, 64)], 1))
    c.lens, c.pos = [L] * R, [L - 1] * R
    q = torch.cat([c.q[:, :, :512] * 0.05, c.q[:, :, 512:].abs() + 0.1], 2).to(torch.bfloat16).to(DEV)
    sel = torch.arange(L, dtype=torch.int32, device=DEV).expand(R, L).contiguous()
    clean = api.li_paged_sparse_attention(q, c.cache, sel, c.scale, **c.kw())
    assert not clean.isnan().any()
    rows = c.cache[int(c.table[0, 0])]
    if kind == "bf16":
        rows[list(where)] = float("nan")
    else:
        rows[list(where), 256:288] = 127           # every scale NaN
    out = api.li_paged_sparse_attention(q, c.cache, sel, c.scale, **c.kw())
    assert out[0].isnan().all() and torch.equal(out[1:], clean[1:])
    out = api.li_window_attention(q, c.cache, _i32(c.pos), c.scale, L, **c.kw())
    assert out[0].isnan().all() and torch.equal(out[1:], clean[1:])
