"""Appending to the paged cache: bit-exact codes, keys, values and queries
against the oracle's float32 arithmetic, and nothing else written."""
import numpy as np
import pytest
import torch

import precision_gemm_token_gb300 as E
from oracle import attention_oracle as AO
from precision_gemm_token_gb300 import attention as A

from .attention_util import Batch, ensure_lib, status_buf

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def bits(x: np.ndarray):
    """bf16 bits of float32 values (round to nearest even)."""
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).view(torch.int16).numpy()


def table_of(n_pos, rot):
    t = np.arange(n_pos)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    return torch.from_numpy(np.concatenate([np.cos(t), np.sin(t)], 1).astype(np.float32))


def check(b: Batch, rot=None, interleaved=False, seed=0, in_place=False, with_table=True, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    heads, kv, dim, T = b.heads, b.kv_heads, b.dim, b.tokens
    x = (torch.randn(T, heads + 2 * kv, dim, generator=g) * spread).to(torch.bfloat16)
    rot = dim if rot is None else rot
    longest = max([m for _, m in b.seqs] + [1])
    cs = table_of(longest, rot) if with_table else None
    xg = x.cuda()
    start, length, table = b.dev("q_start", "kv_len", "table")
    before = [b.cache.k.cpu().clone(), b.cache.v.cpu().clone()]
    st = status_buf()
    q, k, v = xg[:, :heads], xg[:, heads:heads + kv], xg[:, heads + kv:]
    q_out = A.kv_append(q, k, v, b.cache, start, length, table, cs.cuda() if with_table else None, interleaved,
                        q_out=q if in_place else None, status=st)
    assert int(st.item()) == 0
    xf = x.float().numpy()
    want_q = np.zeros((T, heads, dim), np.float32)
    want = [before[0].view(torch.int16 if b.fmt == "bf16" else torch.uint8).numpy().copy(),
            before[1].view(torch.int16 if b.fmt == "bf16" else torch.uint8).numpy().copy()]
    for t, p in enumerate(b.positions()):
        if p < 0:
            continue
        seq = int(np.searchsorted(b.starts, t, side="right")) - 1
        y = xf[t]
        if with_table:
            c, s = cs[p, :rot // 2].numpy(), cs[p, rot // 2:].numpy()
            y = np.concatenate([AO.rotate_f32(y[:heads + kv], c, s, interleaved), y[heads + kv:]])
        want_q[t] = y[:heads]
        pg, row = int(b.table[seq, p // b.page]), p % b.page
        for i, part in ((0, y[heads:heads + kv]), (1, y[heads + kv:])):
            if b.fmt == "bf16":
                want[i][pg, :, row] = bits(part)
            else:
                sc = (b.k_scale if i == 0 else b.v_scale).numpy()
                want[i][pg, :, row] = np.stack([AO.cache_codes(part[h], sc[h]) for h in range(kv)])
    assert (q_out.view(torch.int16).cpu().numpy() == bits(want_q)).all()
    for i, pool in enumerate((b.cache.k, b.cache.v)):
        got = pool.cpu().view(torch.int16 if b.fmt == "bf16" else torch.uint8).numpy()
        assert (got == want[i]).all(), ("kv"[i], np.argwhere(got != want[i])[:5])
    if not in_place:
        assert torch.equal(xg.cpu().view(torch.int16), x.view(torch.int16))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("heads,kv_heads,dim,rot", [(32, 8, 128, 128), (64, 8, 128, 64), (14, 2, 64, 64),
                                                    (5, 1, 64, 16), (96, 32, 128, 48)])
def test_append(fmt, interleaved, heads, kv_heads, dim, rot):
    seqs = [(1, 1), (1, 40), (0, 9), (5, 5), (33, 70), (0, 0), (1, 17), (16, 64)]
    check(Batch(seqs, heads, kv_heads, dim, fmt=fmt, seed=heads), rot, interleaved, seed=dim)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("order", ["head", "token"])
def test_append_pages(fmt, page, order):
    check(Batch([(70, 300), (1, page), (1, page + 1)], 4, 2, 64, fmt=fmt, page=page, order=order, seed=page))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_many_tokens(fmt, interleaved):
    """Enough tokens that a block takes several: sequences that begin and end
    inside a block, a last block that is not full, padding rows."""
    seqs = [(1, 30)] * 5 + [(301, 400), (0, 3), (2, 1), (213, 213), (1, 7), (6, 90)]
    check(Batch(seqs, 12, 4, 64, fmt=fmt, seed=9, tail=2), interleaved=interleaved)
    check(Batch([(600, 611)], 6, 2, 128, fmt=fmt, page=64, order="token", seed=10), 96, interleaved)


def test_append_in_place_and_without_rotation():
    check(Batch([(9, 30), (1, 1)], 8, 2, 128, seed=1), in_place=True)
    check(Batch([(9, 30), (1, 1)], 8, 2, 128, seed=1), in_place=True, interleaved=True)
    check(Batch([(9, 30), (1, 1)], 8, 2, 128, fmt="e4m3", seed=2), with_table=False)


def test_append_extremes():
    """Values that saturate E4M3, underflow it, and infinities."""
    check(Batch([(20, 64)], 4, 2, 64, fmt="e4m3", seed=3), spread=1e4)
    check(Batch([(20, 64)], 4, 2, 64, fmt="e4m3", seed=4), spread=1e-6)


def test_append_empty_rows_and_padding():
    """Tokens at negative positions and padding rows append nothing; their
    queries come back zero."""
    check(Batch([(5, 2), (3, 0), (1, 4)], 8, 2, 64, seed=5, tail=7))
    check(Batch([], 8, 2, 64, seed=5, tail=2))


def test_append_many_sequences():
    rng = np.random.default_rng(1)
    seqs = [(int(n), int(n + m)) for n, m in zip(rng.integers(0, 4, 300), rng.integers(0, 50, 300))]
    check(Batch(seqs, 4, 2, 64, seed=6))


def test_append_keys_and_values_only():
    b = Batch([(3, 20)], 4, 2, 64, seed=7)
    T = 3
    k = torch.randn(T, 2, 64, device="cuda").to(torch.bfloat16)
    start, length, table = b.dev("q_start", "kv_len", "table")
    batch = E.KvBatch(1, T, T, table.shape[1], table.shape[1], start.data_ptr(), length.data_ptr(), table.data_ptr())
    rc = E.epilora_kv_append(b.cache.struct, batch, 4, None, (0, 0), k, (128, 64), k, (128, 64), None, 0, 0, False,
                             None, (0, 0))
    assert rc == 0
    torch.cuda.synchronize()
    for p in range(17, 20):
        pg = int(b.table[0, p // 16])
        assert torch.equal(b.cache.k[pg, :, p % 16], k[p - 17]) and torch.equal(b.cache.v[pg, :, p % 16], k[p - 17])


def test_append_device_detected_errors():
    def run(mutate, n_pos=64):
        b = Batch([(2, 40), (1, 20)], 4, 2, 64, seed=8)
        mutate(b)
        x = torch.randn(3, 8, 64, device="cuda").to(torch.bfloat16)
        start, length, table = b.dev("q_start", "kv_len", "table")
        st = status_buf()
        before = b.cache.k.clone()
        q = A.kv_append(x[:, :4], x[:, 4:6], x[:, 6:], b.cache, start, length, table, table_of(n_pos, 64).cuda(),
                        status=st)
        torch.cuda.synchronize()
        return int(st.item()), q, (before.view(torch.int16) != b.cache.k.view(torch.int16)).any().item()

    assert run(lambda b: None)[0] == 0
    for mutate in (lambda b: b.table.__setitem__((0, 2), -1), lambda b: b.table.__setitem__((0, 2), 1000),
                   lambda b: b.kv_len.__setitem__(0, 60), lambda b: b.q_start.__setitem__(0, 1)):
        code, q, _ = run(mutate)
        assert code == E.EPILORA_ERR_INVALID_ARG
        assert (q[:2] == 0).any()
    code, q, _ = run(lambda b: None, n_pos=38)          # positions 38 and 39 have no rotation row
    assert code == E.EPILORA_ERR_INVALID_ARG and (q[:2] == 0).all() and not (q[2] == 0).all()
