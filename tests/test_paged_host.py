"""Host side of the paged-cache calls: the argument checks of the C ABI and of the binding, the rotary
table, and the oracle's own definitions by hand-computed values.  No GPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import paged as oracle
from sparse_attention_lightning_score_b200 import _lib, api

P = ctypes.c_void_p(256)
BAD, NO = _lib.LI_ERR_INVALID_ARG, _lib.LI_ERR_UNSUPPORTED


def _tables(R=4, blocks=8, page=64, pages=100, n_free=10, tokens=4, seq=P, new=P, table=P, free=P, start=None, slots=P,
            nxt=ctypes.c_void_p(512), starts=P):
    return _lib.load().li_block_tables(seq, new, R, table, blocks, page, pages, free, n_free, start, tokens, slots, P, P,
                                       starts, nxt, None)


def test_block_tables_rejects_bad_arguments():
    assert _tables(R=-1) == BAD and _tables(page=0) == BAD and _tables(blocks=-1) == BAD
    assert _tables(pages=-1) == BAD and _tables(n_free=-1) == BAD and _tables(tokens=-1) == BAD
    assert _tables(seq=None) == BAD and _tables(table=None) == BAD and _tables(free=None) == BAD
    assert _tables(slots=None) == BAD and _tables(starts=None) == BAD and _tables(nxt=None) == BAD
    assert _tables(start=P, nxt=P) == BAD                      # the next index may not overwrite the first
    assert _tables(slots=ctypes.c_void_p(260)) == BAD          # int64 alignment
    assert _tables(R=_lib.LI_BLOCK_TABLE_MAX_REQUESTS + 1) == NO


def _rope(n=1, tokens=2, rot=64, mscale=1.0, **kw):
    d = (_lib.RopeTensor * max(n, 1))()
    for i in range(max(n, 1)):
        f = dict(x=4096 + 65536 * i, out=1 << 24 | 65536 * i, x_token_stride=256, x_head_stride=128,
                 out_token_stride=256, out_head_stride=128, heads=2, dim=128, offset=0, layout=0, dtype=1)
        f.update(kw)
        for k, v in f.items():
            setattr(d[i], k, v)
    return _lib.load().li_rope(d, n, tokens, P, P, rot, mscale, None)


def test_rope_rejects_bad_arguments():
    assert _rope(n=0) == BAD and _rope(n=5) == BAD and _rope(tokens=-1) == BAD
    assert _rope(rot=63) == BAD and _rope(rot=0) == BAD and _rope(rot=130) == BAD and _rope(rot=2048) == BAD
    assert _rope(mscale=math.nan) == BAD and _rope(mscale=math.inf) == BAD
    assert _rope(heads=0) == BAD and _rope(offset=-1) == BAD and _rope(offset=65) == BAD and _rope(layout=2) == BAD
    assert _rope(dtype=_lib.LI_DTYPE_E4M3) == NO
    assert _rope(x=None) == BAD and _rope(x=4097) == BAD and _rope(x_token_stride=-1) == BAD
    assert _rope(out=4096, out_token_stride=512) == BAD        # in place with other strides
    assert _rope(out=4096 + 2) == BAD                          # out overlaps x without being it
    assert _rope(out_head_stride=64) == BAD                    # heads of out overlap
    assert _rope(out_token_stride=0) == BAD                    # tokens of out overlap
    assert _rope(tokens=0) == _lib.LI_OK


def test_rope_refuses_tensors_of_a_call_that_share_elements():
    d = (_lib.RopeTensor * 2)()
    def put(i, x, out, heads, dim, offset):
        for k, v in dict(x=x, out=out, x_token_stride=512, x_head_stride=128, out_token_stride=512, out_head_stride=128,
                         heads=heads, dim=dim, offset=offset, layout=0, dtype=1).items():
            setattr(d[i], k, v)
    run = lambda: _lib.load().li_rope(d, 2, 3, P, P, 64, 1.0, None)  # noqa: E731
    put(0, 4096, 4096, 2, 128, 0)
    put(1, 4096 + 256, 4096 + 256, 2, 128, 0)     # its first head is the other's second
    assert run() == BAD
    put(1, 4096 + 512, 4096 + 512, 2, 128, 0)     # the two halves of one fused buffer, both in place
    assert run() in (_lib.LI_ERR_CUDA, _lib.LI_OK)  # accepted: only the missing device stops it here
    put(1, 4096 + 512, 1 << 20, 3, 128, 0)        # reads past its half, into what the other writes
    assert run() == BAD


def test_rope_table_values_and_refusals():
    lib = _lib.load()
    out = (ctypes.c_uint64 * 512)()
    for rot, kw in [(64, dict()), (128, dict(scaling="linear", factor=8.0)),
                    (64, dict(scaling="yarn", factor=40.0, original_len=4096)),
                    (32, dict(scaling="yarn", factor=2.0, original_len=77, beta_fast=8.0, beta_slow=0.5)),
                    (2, dict(base=500000.0))]:
        got = api.li_rope_table(rot, device="cpu", **kw).numpy().astype(np.uint64)
        want = oracle.rope_frequencies(rot, **kw)
        # both in fp64: a few units of 2^-53 of the value, and half a step (2^-65 turns) of the fixed point
        np.testing.assert_allclose(got.astype(np.float64) * 2.0 ** -64 * 2 * math.pi, want, rtol=1e-14,
                                   atol=2.0 ** -65 * 2 * math.pi)
    ok = (64, 10000.0, 2, 40.0, 4096, 32.0, 1.0)
    assert lib.li_rope_table(*ok, out) == _lib.LI_OK
    for at, v in [(0, 63), (0, 0), (0, 1026), (1, 1.0), (1, math.nan), (2, 3), (3, 0.5), (3, math.inf), (4, 0), (5, 1.0),
                  (6, 0.0), (6, math.nan)]:
        bad = list(ok)
        bad[at] = v
        assert lib.li_rope_table(*bad, out) == BAD, (at, v)
    assert lib.li_rope_table(*ok, None) == BAD
    with pytest.raises(ValueError):
        api.li_rope_table(64, scaling="cubic", device="cpu")


def test_kv4_rejects_bad_arguments():
    w, r = _lib.load().li_kv4_write, _lib.load().li_kv4_read
    assert w(P, 576, P, -1, P, 10, None) == BAD and w(P, 575, P, 1, P, 10, None) == BAD
    assert w(None, 576, P, 1, P, 10, None) == BAD and w(P, 576, None, 1, P, 10, None) == BAD
    assert w(P, 576, P, 1, ctypes.c_void_p(264), 10, None) == BAD and w(P, 576, P, 1, P, -1, None) == BAD
    assert w(P, 576, P, 1 << 31, P, 10, None) == NO
    assert w(None, 576, None, 0, None, 10, None) == _lib.LI_OK
    assert r(P, 10, P, -1, P, None) == BAD and r(P, 10, P, 1, None, None) == BAD
    assert r(P, 10, P, 1, ctypes.c_void_p(264), None) == BAD and r(None, 0, None, 0, None, None) == _lib.LI_OK


def _desc(**kw):
    f = dict(rows=2, heads=64, requests=2, num_pages=8, page_size=16, max_blocks=4, cache_dtype=_lib.LI_DTYPE_E2M1,
             scale=0.1)
    f.update(kw)
    return _lib.AttnDesc(*[f[k] for k, _ in _lib.AttnDesc._fields_])


def _sparse(d, q=P, cache=P, table=P, req=None, sel=P, k=8, out=P, ws=P, wsb=1 << 40):
    return _lib.load().li_paged_sparse_attention(q, cache, table, req, sel, k, d, out, ws, wsb, None)


def _window(d, pos=P, window=8, sinks=1, max_len=64, req=None, ws=P, wsb=1 << 40):
    return _lib.load().li_window_attention(P, P, P, req, pos, window, sinks, max_len, d, P, ws, wsb, None)


def test_paged_attention_rejects_bad_arguments():
    for kw in [dict(rows=-1), dict(heads=0), dict(requests=-1), dict(num_pages=-1), dict(page_size=0),
               dict(max_blocks=-1), dict(scale=0.0), dict(scale=math.nan), dict(scale=math.inf),
               dict(rows=3)]:                                     # three tokens, two requests, no requests_of
        assert _sparse(_desc(**kw)) == BAD, kw
        assert _window(_desc(**kw)) == BAD, kw
    for kw in [dict(cache_dtype=_lib.LI_DTYPE_E4M3), dict(cache_dtype=_lib.LI_DTYPE_F32), dict(heads=5000)]:
        assert _sparse(_desc(**kw)) == NO, kw
    d = _desc()
    assert _sparse(d, k=-1) == BAD and _sparse(d, sel=None) == BAD and _sparse(d, q=None) == BAD
    assert _sparse(d, cache=None) == BAD and _sparse(d, out=None) == BAD and _sparse(d, out=ctypes.c_void_p(264)) == BAD
    assert _sparse(d, q=ctypes.c_void_p(264)) == BAD and _sparse(d, cache=ctypes.c_void_p(264)) == BAD
    assert _sparse(_desc(num_pages=7), table=None) == BAD          # a dense cache smaller than its requests
    assert _sparse(_desc(rows=0)) == _lib.LI_OK
    need = _lib.load().li_paged_attention_workspace(2, 64, 300)
    assert need > 0
    assert _sparse(d, k=300, wsb=need - 1) == BAD and _sparse(d, k=300, ws=None) == BAD
    assert _sparse(d, k=300, ws=ctypes.c_void_p(16)) == BAD
    assert _window(d, window=0) == BAD and _window(d, sinks=-1) == BAD and _window(d, max_len=0) == BAD
    assert _window(d, max_len=65) == BAD and _window(d, pos=None) == BAD   # longer than the block table


def test_paged_attention_limits():
    assert _sparse(_desc(), k=(1 << 28) + 1) == NO
    assert _sparse(_desc(num_pages=1 << 25, page_size=64)) == NO      # 2^31 rows
    assert _window(_desc(max_blocks=1 << 26), window=1 << 29, max_len=1 << 29) == NO


def test_paged_attention_workspace_size():
    f = _lib.load().li_paged_attention_workspace
    assert f(0, 64, 10) == 0 and f(2, 0, 10) == 0 and f(2, 64, 0) == 0
    assert f(1, 64, 128) == 0                     # one tile: nothing to split
    assert f(100000, 128, 4096) == 0              # enough tokens for every SM
    assert f(1, 64, 2048) % 256 == 0 and f(1, 64, 2048) > 0


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    i32 = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        api.li_block_tables(i32, i32, torch.zeros(2, 4, dtype=torch.int32), i32, 16, 8, 2)
    with pytest.raises(ValueError):
        api.li_rope(torch.zeros(2, 4, 64), i32, torch.zeros(32, dtype=torch.int64))
    with pytest.raises(ValueError):
        api.li_kv4_write(torch.zeros(2, 575, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int64),
                         torch.zeros(1, 4, 416, dtype=torch.uint8))
    with pytest.raises(ValueError):
        api.li_paged_sparse_attention(torch.zeros(2, 64, 576, dtype=torch.bfloat16),
                                      torch.zeros(2, 4, 416, dtype=torch.uint8), torch.zeros(2, 3, dtype=torch.int32), 0.1)


# --------------------------------------------------------------------------- the oracle, by hand
def test_oracle_block_tables_by_hand():
    # page size 4: request 0 grows 3 -> 6 (holds page 9), request 1 is idle, request 2 starts with 5
    s, p, r, st, nxt, t, bad = oracle.block_tables([6, 4, 5], [3, 0, 5], [[9, -1], [8, -1], [-1, -1]], [2, 5, 7, 1], 4, 10,
                                                   9)
    assert s.tolist() == [39, 8, 9, 20, 21, 22, 23, 28, -1]
    assert p.tolist() == [3, 4, 5, 0, 1, 2, 3, 4, -1] and r.tolist() == [0, 0, 0, 2, 2, 2, 2, 2, -1]
    assert st.tolist() == [0, 3, 3, 8] and nxt == 3 and t.tolist() == [[9, 2], [8, -1], [5, 7]] and not bad


def test_oracle_window_by_hand():
    assert oracle.visible(0, 1, 0).tolist() == [0]
    assert oracle.visible(5, 2, 1).tolist() == [0, 4, 5]
    assert oracle.visible(5, 100, 3).tolist() == [0, 1, 2, 3, 4, 5]
    assert oracle.visible(3, 2, 3).tolist() == [0, 1, 2, 3]      # window and sinks meet: nothing twice


def test_oracle_kv4_by_hand():
    x = torch.zeros(1, 576)
    x[0, :16] = torch.tensor([6.0, -6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, 0, 0.3, 0.5, 4, 5.1, -1.0])
    x[0, 512:] = torch.arange(64.)
    raw = oracle.kv4_pack(x.to(torch.bfloat16))
    assert raw.shape == (1, 416) and raw[0, 256] == 0x38          # scale 1
    back = oracle.kv4_unpack(raw)[0]
    assert back[:16].tolist() == [6, -6, 0, 1, 1, 2, 2, 4, 4, 0, 0, 0.5, 0.5, 4, 6, -1]
    assert back[512:].tolist() == list(range(64)) and np.all(back[16:512] == 0)


def test_oracle_rope_by_hand():
    x = np.zeros((1, 1, 4))
    x[0, 0] = [1.0, 2.0, 3.0, 4.0]
    f = oracle.rope_frequencies(2)
    y = oracle.rope(x, [1], f, "interleaved", 2, 1.0)[0, 0]
    assert y[:2].tolist() == [1.0, 2.0]
    assert np.allclose(y[2:], [3 * math.cos(1) - 4 * math.sin(1), 3 * math.sin(1) + 4 * math.cos(1)])
    assert np.array_equal(oracle.rope(x, [-1], f, "half", 0, 2.0), x)
