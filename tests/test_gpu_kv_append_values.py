"""Appending what is not finite, and nothing at all: infinities and NaN
through the rotation and the conversion to E4M3; tokens that fail a device
check leave every byte of both pools as it was and come back as zero rows."""
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


def table_of(n_pos, rot):
    t = np.arange(n_pos)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    return torch.from_numpy(np.concatenate([np.cos(t), np.sin(t)], 1).astype(np.float32))


def codes(y, scale):
    """E4M3 codes of fp32 values: infinities saturate; NaN is 0x7F here."""
    y = (y.astype(np.float32) / np.float32(scale)).astype(np.float32)
    c = AO.cache_codes(np.where(np.isnan(y), 0.0, np.clip(y, -1e30, 1e30)), 1.0)
    return np.where(np.isnan(y), 0x7F, c).astype(np.uint8)


def bits_bf16(y):
    """bf16 bits; every NaN as 0x7FC0."""
    t = torch.from_numpy(np.ascontiguousarray(y, dtype=np.float32)).to(torch.bfloat16)
    return torch.where(torch.isnan(t), torch.tensor(0x7FC0, dtype=torch.int16), t.view(torch.int16)).numpy()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_infinities_and_nan(fmt, interleaved):
    heads, kv, dim, rot = 4, 2, 64, 32
    b = Batch([(9, 30), (3, 3)], heads, kv, dim, fmt=fmt, seed=1)
    g = torch.Generator().manual_seed(2)
    x = torch.randn(b.tokens, heads + 2 * kv, dim, generator=g)
    for i, bad in enumerate((float("inf"), float("-inf"), float("nan"), 3e38, -3e38)):
        x[i::5, :, i::7] = bad             # rotated elements and copied ones, of q, k and v
    x = x.to(torch.bfloat16)
    cs = table_of(30, rot)
    xg, st = x.cuda(), status_buf()
    start, length, table = b.dev("q_start", "kv_len", "table")
    q = A.kv_append(xg[:, :heads], xg[:, heads:heads + kv], xg[:, heads + kv:], b.cache, start, length, table, cs.cuda(),
                    interleaved, status=st)
    assert int(st.item()) == 0
    got_q = bits_bf16(q.float().cpu().numpy())
    pools = [t.cpu() for t in (b.cache.k, b.cache.v)]
    xf = x.float().numpy()
    for t, p in enumerate(b.positions()):
        seq = int(np.searchsorted(b.starts, t, side="right")) - 1
        c, s = cs[p, :rot // 2].numpy(), cs[p, rot // 2:].numpy()
        with np.errstate(invalid="ignore", over="ignore"):
            y = np.concatenate([AO.rotate_f32(xf[t, :heads + kv], c, s, interleaved), xf[t, heads + kv:]])
            assert (got_q[t] == bits_bf16(y[:heads])).all()
            pg, row = int(b.table[seq, p // b.page]), p % b.page
            for i in range(2):
                for h in range(kv):
                    part, got = y[heads + i * kv + h], pools[i][pg, h, row]
                    if fmt == "bf16":
                        assert (bits_bf16(got.float().numpy()) == bits_bf16(part)).all(), (t, i, h)
                    else:
                        got = got.numpy()
                        got = np.where((got & 0x7F) == 0x7F, 0x7F, got)
                        want = codes(part, (b.k_scale if i == 0 else b.v_scale)[h].numpy())
                        assert (got == want).all(), (t, i, h)


def set_(name, at, value):
    return lambda b: getattr(b, name).__setitem__(at, value)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("mutate,n_pos", [
    (set_("table", (0, 2), -1), 64), (set_("table", (0, 2), 1000), 64), (set_("kv_len", 0, 60), 64),
    (set_("q_start", 0, 1), 64), (lambda b: None, 38)],
    ids=["page -1", "page 1000", "length 60 of 48", "q_start from 1", "no rotation row"])
def test_refused_tokens_append_nothing(fmt, mutate, n_pos):
    """Both tokens of the first sequence fail; the second sequence's token is
    appended and nothing else is written."""
    b = Batch([(2, 40), (1, 20)], 4, 2, 64, fmt=fmt, seed=8)
    mutate(b)
    g = torch.Generator().manual_seed(3)
    x = torch.randn(3, 8, 64, generator=g).to(torch.bfloat16).cuda()
    start, length, table = b.dev("q_start", "kv_len", "table")
    bits = torch.int16 if fmt == "bf16" else torch.uint8
    want = [t.cpu().view(bits).clone() for t in (b.cache.k, b.cache.v)]
    st, cs = status_buf(), table_of(n_pos, 64)
    q = A.kv_append(x[:, :4], x[:, 4:6], x[:, 6:], b.cache, start, length, table, cs.cuda(), status=st)
    assert int(st.item()) == E.EPILORA_ERR_INVALID_ARG
    assert (q[:2] == 0).all() and (q[2] != 0).any(-1).all()
    xf = x.float().cpu().numpy()
    k = AO.rotate_f32(xf[2, 4:6], cs[19, :32].numpy(), cs[19, 32:].numpy(), False)
    pg = int(b.table[1, 1])
    for i, part in enumerate((k, xf[2, 6:])):
        if fmt == "bf16":
            want[i][pg, :, 3] = torch.from_numpy(part).to(torch.bfloat16).view(bits)
        else:
            scale = (b.k_scale if i == 0 else b.v_scale).numpy()
            want[i][pg, :, 3] = torch.from_numpy(np.stack([AO.cache_codes(part[h], scale[h]) for h in range(2)]))
    for pool, w in zip((b.cache.k, b.cache.v), want):
        assert torch.equal(pool.cpu().view(bits), w)
