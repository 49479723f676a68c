"""Layouts and sizes that the attention calls take besides the usual ones:
keys and values of unlike strides, page tables cut out of wider ones, heads
outermost, single rows whose strides mean nothing, very wide groups."""
import numpy as np
import pytest
import torch

import precision_gemm_token_gb300 as E
from oracle import attention_oracle as AO
from precision_gemm_token_gb300 import attention as A

from .attention_util import Batch, assert_attention, ensure_lib, f64, status_buf

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def attend(b, q=None, cache=None, table=None, out=None, **kw):
    dq, start, length, dt = b.dev("q", "q_start", "kv_len", "table")
    st = status_buf()
    lse = torch.full((b.tokens, b.heads), 7.0, device="cuda")
    o = A.paged_attention(dq if q is None else q, b.cache if cache is None else cache, start, length,
                          dt if table is None else table, out=out, lse=lse, status=st, **kw)
    assert int(st.item()) == 0
    assert_attention(o, lse, *b.oracle(b.dim ** -0.5), fmt=b.fmt)
    return o


def heads_outermost(x):
    """The same rows with the heads as the outermost axis in memory."""
    return x.transpose(0, 1).contiguous().transpose(0, 1)


MIXED = [(1, 300), (1, 17), (40, 200), (3, 90)]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
def test_keys_and_values_of_unlike_strides(fmt, dim):
    """Keys in head order, values in token order and with gaps between pages."""
    b = Batch(MIXED, 8, 2, dim, fmt=fmt, page=32, seed=dim)
    pages, kv, page, _ = b.cache.v.shape
    wide = torch.zeros(pages, page + 2, kv, dim, dtype=b.cache.v.dtype, device="cuda")
    v = wide[:, :page].transpose(1, 2)
    v.copy_(b.cache.v)
    attend(b, cache=A.PagedKVCache(b.cache.k, v, b.cache.k_scale, b.cache.v_scale))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_append_to_unlike_strides(fmt):
    """An append into such a cache leaves what one into a plain cache does."""
    b = Batch(MIXED, 8, 2, 64, fmt=fmt, page=32, seed=1)
    x = torch.randn(b.tokens, 12, 64, device="cuda").to(torch.bfloat16)
    pages, kv, page, d = b.cache.v.shape
    wide = torch.zeros(pages, page + 2, kv, d, dtype=b.cache.v.dtype, device="cuda")
    v = wide[:, :page].transpose(1, 2)
    v.copy_(b.cache.v)
    odd = A.PagedKVCache(b.cache.k.clone(), v, b.cache.k_scale, b.cache.v_scale)
    _, start, length, table = b.dev("q", "q_start", "kv_len", "table")
    for cache in (b.cache, odd):
        A.kv_append(x[:, :8], x[:, 8:10], x[:, 10:], cache, start, length, table)
    torch.cuda.synchronize()
    bits = torch.int16 if fmt == "bf16" else torch.uint8
    assert torch.equal(odd.k.view(bits), b.cache.k.view(bits))
    assert torch.equal(odd.v.contiguous().view(bits), b.cache.v.contiguous().view(bits))
    assert not wide[:, page:].any()


def test_page_table_of_a_wider_table():
    """The columns of a wider table, and single rows of it."""
    b = Batch(MIXED, 8, 2, 128, seed=2)
    wide = torch.full((len(MIXED), b.table.shape[1] + 7), 1 << 30, dtype=torch.int32, device="cuda")
    table = wide[:, 3:3 + b.table.shape[1]]
    table.copy_(b.table)
    attend(b, table=table)
    x = torch.randn(b.tokens, 12, 128, device="cuda").to(torch.bfloat16)
    start, length = b.dev("q_start", "kv_len")
    st = status_buf()
    A.kv_append(x[:, :8], x[:, 8:10], x[:, 10:], b.cache, start, length, table, status=st)
    assert int(st.item()) == 0
    for (n, m), t, row in zip(MIXED, b.starts, b.table):
        for i in range(n):
            p = m - n + i
            assert torch.equal(b.cache.k[int(row[p // 16]), :, p % 16], x[t + i, 8:10])
            assert torch.equal(b.cache.v[int(row[p // 16]), :, p % 16], x[t + i, 10:])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads", [8, 14])
def test_heads_outermost(fmt, heads):
    b = Batch(MIXED, heads, 2, 128, fmt=fmt, seed=heads)
    out = heads_outermost(torch.full((b.tokens, heads, 128), 7.0, dtype=torch.bfloat16, device="cuda"))
    o = attend(b, q=heads_outermost(b.q.cuda()), out=out)
    assert o.stride() == (128, b.tokens * 128, 1)


def test_prompts_with_heads_outermost():
    lens, heads, kv_heads, dim = [70, 1, 200], 8, 2, 64
    g = torch.Generator().manual_seed(0)
    x = torch.randn(sum(lens), heads + 2 * kv_heads, dim, generator=g).to(torch.bfloat16)
    q, k, v = x[:, :heads], x[:, heads:heads + kv_heads], x[:, heads + kv_heads:]
    starts = np.r_[0, np.cumsum(lens)]
    got = A.prompt_attention(*(heads_outermost(t.cuda()) for t in (q, k, v)),
                             torch.tensor(starts, dtype=torch.int32).cuda(),
                             out=heads_outermost(torch.zeros(q.shape, dtype=torch.bfloat16, device="cuda")))
    for n, t in zip(lens, starts):
        s = slice(t, t + n)
        o, lse, spread = AO.attention_rows(f64(q[s]), f64(k[s]), f64(v[s]), np.arange(n), dim ** -0.5)
        assert_attention(got[s], None, o, lse, *spread)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("group", [128, 129, 200, 256, 300])
def test_wide_groups(fmt, group):
    """A group fills, passes or straddles a row tile."""
    check = [(1, 50), (3, 140), (2, 1), (0, 9)]
    attend(Batch(check, group, 1, 64, fmt=fmt, seed=group, tail=1))


def test_wide_groups_of_prompts():
    heads, dim, n = 200, 64, 35
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(n, h, dim, generator=g).to(torch.bfloat16) for h in (heads, 1, 1))
    got = A.prompt_attention(q.cuda(), k.cuda(), v.cuda(), torch.tensor([0, n], dtype=torch.int32).cuda())
    o, lse, spread = AO.attention_rows(f64(q), f64(k), f64(v), np.arange(n), dim ** -0.5)
    assert_attention(got, None, o, lse, *spread)


@pytest.mark.parametrize("heads", [1, 20])
def test_strides_that_reach_nothing(heads):
    """One token has no token stride and one head no head stride: 0 is taken
    there by the C entry points as any other multiple of 8 is."""
    dim = 64
    hs = 0 if heads == 1 else dim
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(1, h, dim, generator=g).to(torch.bfloat16) for h in (heads, 1, 1))
    gq, gk, gv = q.cuda(), k.cuda(), v.cuda()
    ws = A.AttentionWorkspace("cuda").get(dim)
    start = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    o, st = torch.zeros_like(gq), status_buf()
    rc = E.epilora_prompt_attention(1, 1, start, heads, 1, dim, gq, (0, hs), gk, (0, 0), gv, (0, 0), dim ** -0.5, o,
                                    (0, hs), None, ws, ws.numel(), st)
    assert rc == E.EPILORA_OK
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and torch.equal(o, gv.expand(1, heads, dim))
    b = Batch([(1, 33)], heads, 1, dim, seed=3)
    dq, start, length, table = b.dev("q", "q_start", "kv_len", "table")
    batch = E.KvBatch(1, 1, 3, table.shape[1], table.shape[1], start.data_ptr(), length.data_ptr(), table.data_ptr())
    o = torch.zeros_like(dq)
    rc = E.epilora_paged_attention(b.cache.struct, batch, heads, dq, (0, hs), dim ** -0.5, o, (0, hs), None, ws,
                                   ws.numel(), st)
    assert rc == E.EPILORA_OK
    assert int(st.item()) == 0
    assert_attention(o, None, *b.oracle(dim ** -0.5))
