"""Attention over the paged cache and of packed prompts against the float64
oracle: formats, head groups, page sizes and layouts, lengths around the tile
edges, empty rows, splits of long sequences, NaN in everything masked."""
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


def check(b: Batch, scale=None, what="", **kw):
    st = status_buf()
    lse = torch.full((b.tokens, b.heads), 7.0, device="cuda")
    out = torch.full((b.tokens, b.heads, b.dim), 7.0, dtype=torch.bfloat16, device="cuda")
    o = b.attend(scale=scale, lse=lse, out=out, status=st, **kw)
    assert int(st.item()) == 0
    scale = b.dim ** -0.5 if scale is None else scale
    assert_attention(o, lse, *b.oracle(scale), what=what, fmt=b.fmt)
    return o


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(32, 8), (64, 8), (8, 8), (5, 1), (14, 2), (16, 1), (3, 3)])
def test_decode(fmt, dim, heads, kv_heads):
    """One new token a sequence; lengths around the tile and page edges."""
    seqs = [(1, n) for n in (1, 2, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 200, 511, 777)]
    check(Batch(seqs, heads, kv_heads, dim, fmt=fmt, seed=heads + dim))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("order", ["head", "token"])
def test_decode_pages(fmt, page, order):
    seqs = [(1, n) for n in (5, page, page + 1, 3 * page - 1, 700)]
    check(Batch(seqs, 8, 2, 128, fmt=fmt, page=page, order=order, seed=page, table_extra=2))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_decode_long_split(fmt):
    """One sequence alone on the GPU: split along its length and joined."""
    check(Batch([(1, 9001)], 8, 2, 128, fmt=fmt, seed=3))
    check(Batch([(1, 4099), (1, 3), (1, 0), (1, 2500)], 4, 1, 64, fmt=fmt, page=64, seed=4))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
def test_decode_long_line(fmt, dim):
    """More positions than SMs by far: every thread block goes round its ring
    many times, over several sequences and heads; repeated, since the order
    in which copies land changes from run to run."""
    seqs = [(1, 4096), (1, 17), (1, 3001), (1, 64)] + [(1, 2500 + 37 * i) for i in range(10)]
    b = Batch(seqs, 8, 8, dim, fmt=fmt, seed=dim, page=64)
    first = check(b)
    ws = A.AttentionWorkspace("cuda")
    for _ in range(50):
        assert torch.equal(b.attend(workspace=ws), first)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [2, 3, 4])
def test_few_tokens(fmt, n):
    """A few new tokens a sequence (drafted tokens), causal among themselves."""
    seqs = [(n, m) for m in (n, n + 1, 16, 64, 130, 600)]
    check(Batch(seqs, 8, 2, 128, fmt=fmt, seed=n))
    check(Batch(seqs, 32, 2, 64, fmt=fmt, page=32, seed=n))     # rows beyond one small tile


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(8, 2), (8, 8), (16, 2), (7, 1), (20, 1)])
def test_chunks(fmt, dim, heads, kv_heads):
    """Chunks of new tokens over a history, lengths off every tile edge."""
    seqs = [(37, 37), (64, 200), (33, 400), (129, 131), (1, 90), (250, 613)]
    check(Batch(seqs, heads, kv_heads, dim, fmt=fmt, seed=dim + heads))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("page,order", [(16, "token"), (32, "head"), (64, "token"), (128, "head"), (256, "token")])
def test_chunk_pages(fmt, page, order):
    seqs = [(40, 40), (65, 300), (100, 255), (17, 1000)]
    check(Batch(seqs, 8, 2, 128, fmt=fmt, page=page, order=order, seed=page))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_chunk_long_split(fmt):
    """Few rows over a long history: the history is split and joined."""
    check(Batch([(33, 5003)], 8, 1, 128, fmt=fmt, seed=9))
    check(Batch([(70, 3001), (5, 4000)], 8, 1, 64, fmt=fmt, page=32, seed=10))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_mixed(fmt):
    """Decoding sequences and prefill chunks in one call, with sequences that
    have no new token or no token at all among them, and padding rows."""
    seqs = [(1, 300), (0, 50), (1, 1), (300, 300), (0, 0), (1, 77), (130, 500), (2, 9)]
    check(Batch(seqs, 16, 2, 128, fmt=fmt, seed=21, tail=5))


def test_max_new_selects_no_results():
    b = Batch([(1, 300), (1, 40), (2, 100)], 8, 2, 128, seed=5)
    ref = b.oracle(128 ** -0.5)
    for max_new in (2, 5, 100, None):
        assert_attention(b.attend(max_new=max_new), None, *ref, what=max_new)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_full_batches(fmt):
    """As many packed tokens as the bound allows, n_seqs * max_new: chunks of
    one length, and the same sizes where rows are padding and the sequences
    shorter, single tokens and empty ones among them."""
    check(Batch([(37, 300), (37, 37), (37, 1000)], 8, 2, 128, fmt=fmt, seed=4))
    for seqs, most, dim in (([(1, 100), (0, 50), (20, 300), (2, 2)], 20, 128), ([(3, 700)], 40, 64), ([(0, 9)], 40, 64),
                            ([(1, 5), (6, 4)], 33, 128)):
        b = Batch(seqs, 8, 2, dim, fmt=fmt, seed=7, tail=len(seqs) * most - sum(n for n, _ in seqs))
        out, lse = torch.full_like(b.q, float("nan")).cuda(), torch.full((b.tokens, 8), float("nan"), device="cuda")
        st = status_buf()
        b.attend(max_new=most, out=out, lse=lse, status=st)
        assert int(st.item()) == 0
        assert_attention(out, lse, *b.oracle(dim ** -0.5), what=seqs, fmt=fmt)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_empty_rows(fmt):
    """More new tokens than positions (rows that see nothing), sequences of
    length zero, nothing but padding."""
    check(Batch([(3, 1), (1, 0), (2, 2)], 8, 2, 128, fmt=fmt, seed=1, tail=2))
    check(Batch([(60, 20), (40, 0), (1, 5)], 8, 2, 64, fmt=fmt, seed=2, tail=200))
    check(Batch([], 8, 2, 64, fmt=fmt, seed=2, tail=3))
    b = Batch([(1, 5)], 8, 2, 64, fmt=fmt)
    q = torch.empty((0, 8, 64), dtype=torch.bfloat16, device="cuda")
    start, length, table = b.dev("q_start", "kv_len", "table")
    assert A.paged_attention(q, b.cache, start, length, table).shape == (0, 8, 64)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 40])
def test_sharp_and_flat_scores(fmt, n):
    """Softmax rows that one position owns, whose maximum keeps rising, and
    flat ones."""
    for scale, k_std in ((2.0, 1.0), (0.088, 4.0), (0.0, 1.0), (-0.5, 1.0)):
        b = Batch([(n, 700), (n, 90)], 8, 2, 128, fmt=fmt, seed=7, k_std=k_std)
        check(b, scale=scale, what=(scale, k_std))


@pytest.mark.parametrize("n", [1, 3, 50])
def test_rising_maximum(n):
    """Keys that grow along the sequence: each tile raises the maximum."""
    b = Batch([(n, 640)], 8, 2, 128, seed=8)
    x = b.cache.k.double()
    for j in range(640):
        pg = int(b.table[0, j // 16])
        x[pg, :, j % 16] *= (0.05 + j / 40.0)
    b.cache.k.copy_(x.to(torch.bfloat16))
    b.rows[0][0] = f64(b.cache.k)[b.table[0, :40].numpy()].transpose(0, 2, 1, 3).reshape(-1, 2, 128)[:640]
    check(b)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,heads", [(2, 8), (4, 8), (70, 8), (200, 2)])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_masked_positions_do_not_reach_earlier_rows(fmt, n, heads, which, bad):
    """The last new token's key or value is NaN or infinite: rows before it
    are what they were."""
    m = n + 100
    b = Batch([(n, m), (1, 30)], heads, 2, 128, fmt=fmt, seed=n)
    clean = b.oracle(128 ** -0.5)
    pool = getattr(b.cache, which)
    pg, row = int(b.table[0, (m - 1) // 16]), (m - 1) % 16
    if fmt == "e4m3":
        pool[pg, :, row] = 0x7F                  # E4M3 has no infinity
    else:
        pool[pg, :, row, ::3] = float(bad)
    st = status_buf()
    o = b.attend(status=st)
    assert int(st.item()) == 0
    keep = np.r_[0:n - 1, n:n + 1]
    assert_attention(o[torch.from_numpy(keep).cuda()], None, *(x[keep] for x in clean), fmt=fmt)
    assert not torch.isfinite(o[n - 1]).all()    # the row that sees it shows it


def test_queries_of_any_size():
    """Rows scaled from 2^-100 to 2^100: scores stay what the scale makes
    them (the E4M3 path carries queries in fp16)."""
    for fmt in ("bf16", "e4m3"):
        for n in (1, 40):
            for e in (-100, 0, 100):
                b = Batch([(n, 150)], 8, 2, 128, fmt=fmt, seed=3)
                b.q = (b.q.double() * 2.0 ** e).to(torch.bfloat16)
                check(b, scale=float(np.float32(0.088 * 2.0 ** -e)), what=(fmt, n, e))


def test_strided_queries_and_outputs():
    """q as a slice of a fused projection, o into a wider buffer."""
    for n in (1, 45):
        b = Batch([(n, 200), (n, 64)], 8, 2, 128, seed=n)
        wide = torch.zeros(b.tokens, 20, 128, dtype=torch.bfloat16, device="cuda")
        wide[:, 3:11] = b.q.cuda()
        buf = torch.full((b.tokens, 8, 256), 3.0, dtype=torch.bfloat16, device="cuda")
        start, length, table = b.dev("q_start", "kv_len", "table")
        o = A.paged_attention(wide[:, 3:11], b.cache, start, length, table, out=buf[:, :, 128:])
        assert_attention(o, None, *b.oracle(128 ** -0.5))
        assert (buf[:, :, :128] == 3.0).all()


def test_deterministic_and_workspace_reuse():
    """Calls of different shapes share a workspace; each gives the same bits
    every time, also while other work shares the GPU."""
    ws = A.AttentionWorkspace("cuda")
    bs = [Batch([(1, 9000)], 8, 2, 128, seed=1), Batch([(33, 5003), (1, 100)], 8, 1, 128, seed=2),
          Batch([(1, 33), (1, 4000)], 8, 2, 128, fmt="e4m3", seed=3)]
    first = [b.attend(workspace=ws) for b in bs]
    side = torch.cuda.Stream()
    x = torch.randn(2048, 2048, device="cuda")
    with torch.cuda.stream(side):
        for _ in range(20):
            x = x @ x * 1e-3
    for _ in range(5):
        for b, f in zip(bs, first):
            assert torch.equal(b.attend(workspace=ws), f)
    torch.cuda.synchronize()


def test_on_another_stream_and_in_a_graph():
    b = Batch([(1, 700), (40, 300)], 8, 2, 128, seed=11)
    ref = b.attend()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = A.AttentionWorkspace("cuda")
    q, start, length, table = b.dev("q", "q_start", "kv_len", "table")
    torch.cuda.synchronize()
    got = A.paged_attention(q, b.cache, start, length, table, max_new=40, workspace=ws, stream=s)
    got_raw = A.paged_attention(q, b.cache, start, length, table, max_new=40, workspace=ws, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(got, ref) and torch.equal(got_raw, ref)
    out = torch.zeros_like(ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        A.paged_attention(q, b.cache, start, length, table, max_new=40, workspace=ws, out=out)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
    # the captured call follows the lengths it finds: one token less
    length -= torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    g.replay()
    torch.cuda.synchronize()
    b.seqs = [(1, 699), (40, 300)]
    b.rows = [[r[0][:699], r[1]] for r in b.rows]
    assert_attention(out, None, *b.oracle(128 ** -0.5))


def _prompt(lens, heads, kv_heads, dim, seed=0, tail=0, scale=None):
    g = torch.Generator().manual_seed(seed)
    T = sum(lens) + tail
    x = torch.randn(T, heads + 2 * kv_heads, dim, generator=g).to(torch.bfloat16)
    starts = np.r_[0, np.cumsum(lens)].astype(int)
    x[starts[-1]:, heads:] = float("nan")        # padding rows hold anything
    q, k, v = x[:, :heads], x[:, heads:heads + kv_heads], x[:, heads + kv_heads:]
    o, lse = np.zeros((T, heads, dim)), np.full((T, heads), -np.inf)
    mean_abs, mag = np.zeros((T, heads, dim)), np.zeros((T, heads))
    sc = dim ** -0.5 if scale is None else scale
    for n, t in zip(lens, starts):
        s = slice(t, t + n)
        o[s], lse[s], (mean_abs[s], mag[s]) = AO.attention_rows(f64(q[s]), f64(k[s]), f64(v[s]), np.arange(n), sc)
    xg = x.cuda()
    q, k, v = xg[:, :heads], xg[:, heads:heads + kv_heads], xg[:, heads + kv_heads:]
    return q, k, v, torch.tensor(starts, dtype=torch.int32).cuda(), (o, lse, mean_abs, mag)


def check_prompt(lens, heads, kv_heads, dim, seed=0, tail=0, scale=None):
    q, k, v, start, ref = _prompt(lens, heads, kv_heads, dim, seed, tail, scale)
    st = status_buf()
    lse = torch.full((q.shape[0], heads), 7.0, device="cuda")
    o = A.prompt_attention(q, k, v, start, scale=scale, lse=lse, status=st)
    assert int(st.item()) == 0
    assert_attention(o, lse, *ref)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(8, 2), (8, 8), (16, 2), (7, 1), (40, 1)])
def test_prompts(dim, heads, kv_heads):
    check_prompt([1, 2, 0, 15, 64, 129, 300, 33, 127, 128], heads, kv_heads, dim, seed=dim + heads, tail=3)


@pytest.mark.parametrize("n", [1, 5, 31, 32, 33, 64, 127, 128, 129, 255, 256, 257, 1000])
def test_prompt_lengths(n):
    check_prompt([n], 4, 1, 128, seed=n)
    check_prompt([n], 2, 2, 64, seed=n)


def test_many_prompts():
    rng = np.random.default_rng(0)
    check_prompt([int(n) for n in rng.integers(0, 40, 400)], 4, 2, 64, seed=1)
    check_prompt([700] + [1] * 50 + [0] * 20 + [900], 4, 2, 128, seed=2)


def test_prompt_scales_and_empty():
    for scale in (2.0, 0.0, -0.5):
        check_prompt([90, 257], 4, 2, 128, seed=4, scale=scale)
    check_prompt([], 4, 2, 64, tail=4)
    check_prompt([0, 0], 4, 2, 64, tail=40)


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_prompt_neighbours_and_later_rows_do_not_leak(which, bad):
    """A non-finite row in one prompt reaches neither its earlier rows nor
    the prompts packed beside it."""
    lens = [50, 200, 70]
    q, k, v, start, ref = _prompt(lens, 8, 2, 128, seed=5)
    (k if which == "k" else v)[180, :, ::5] = float(bad)       # row 130 of the second prompt
    o = A.prompt_attention(q, k, v, start)
    keep = np.r_[0:180, 250:320]
    assert_attention(o[torch.from_numpy(keep).cuda()], None, *(x[keep] for x in ref))
    assert not torch.isfinite(o[180]).all() and not torch.isfinite(o[249]).all()


def test_prompt_equals_paged():
    """The same prompt through the cache (append, then attention)."""
    n, heads, kv_heads, dim = 333, 8, 2, 128
    q, k, v, start, ref = _prompt([n], heads, kv_heads, dim, seed=6)
    b = Batch([(n, n)], heads, kv_heads, dim, page=64, seed=6)
    _, start2, length, table = b.dev("q", "q_start", "kv_len", "table")
    q2 = A.kv_append(q, k, v, b.cache, start2, length, table)
    assert torch.equal(q2, q)
    assert_attention(A.paged_attention(q2, b.cache, start2, length, table), None, *ref)


def test_device_detected_errors():
    """Bad metadata is recorded and stays in bounds (every index below is
    checked against its limits before it is used)."""
    def status_of(mutate, n=1):
        b = Batch([(n, 100), (n, 40)], 8, 2, 128, seed=1)
        mutate(b)
        st = status_buf()
        b.attend(status=st, max_new=b.__dict__.get("max_new", n))
        return int(st.item())

    def page_out(value):
        def f(b):
            b.table[0, 2] = value
        return f

    for n in (1, 40):
        assert status_of(lambda b: None, n) == 0
        assert status_of(page_out(-1), n) == E.EPILORA_ERR_INVALID_ARG
        assert status_of(page_out(10 ** 6), n) == E.EPILORA_ERR_INVALID_ARG
        assert status_of(lambda b: b.kv_len.__setitem__(1, 7 * 16 + 1), n) == E.EPILORA_ERR_INVALID_ARG
        assert status_of(lambda b: b.q_start.__setitem__(2, 10 ** 6), n) == E.EPILORA_ERR_INVALID_ARG
        assert status_of(lambda b: b.q_start.__setitem__(1, 10 ** 6), n) == E.EPILORA_ERR_INVALID_ARG
        assert status_of(lambda b: b.q_start.__setitem__(0, 1), n) == E.EPILORA_ERR_INVALID_ARG
    assert status_of(lambda b: b.__dict__.__setitem__("max_new", 30), 40) == E.EPILORA_ERR_INVALID_ARG
