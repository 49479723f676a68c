"""What the attention helpers refuse, with tensors on the GPU and one defect a
call: the check that a defect is meant for is the one that names it, and
nothing is launched (the outputs, the cache and the status stay as they were)."""
import pytest
import torch

import precision_gemm_token_gb300 as E
from precision_gemm_token_gb300 import attention as A

from .attention_util import ensure_lib

pytestmark = pytest.mark.gpu

T, HEADS, KV, D, PAGE, PAGES = 3, 8, 2, 64, 16, 6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def bf(*shape):
    return torch.full(shape, 0.5, dtype=torch.bfloat16, device="cuda")


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def f32(*shape):
    return torch.full(shape, 0.25, device="cuda")


class Arguments:
    """Good arguments of the three calls; a test spoils one."""

    def __init__(self):
        self.k_pages, self.v_pages = bf(PAGES, KV, PAGE, D), bf(PAGES, KV, PAGE, D)
        self.ws = A.AttentionWorkspace("cuda")
        self.a = dict(q=bf(T, HEADS, D), k=bf(T, KV, D), v=bf(T, KV, D), cache=A.PagedKVCache(self.k_pages, self.v_pages),
                      q_start=i32(0, 1, 3), kv_len=i32(20, 30), page_table=i32([0, 1], [2, 3]), cos_sin=f32(40, D),
                      out=torch.full((T, HEADS, D), 7.0, dtype=torch.bfloat16, device="cuda"),
                      lse=torch.full((T, HEADS), 7.0, device="cuda"), status=i32(0), workspace=self.ws, max_new=2,
                      scale=0.125)

    def call(self, which):
        a = self.a
        if which == "append":
            return A.kv_append(a["q"], a["k"], a["v"], a["cache"], a["q_start"], a["kv_len"], a["page_table"],
                               a["cos_sin"], q_out=a["out"], status=a["status"])
        if which == "paged":
            return A.paged_attention(a["q"], a["cache"], a["q_start"], a["kv_len"], a["page_table"], a["max_new"],
                                     a["scale"], a["out"], a["lse"], a["workspace"], a["status"])
        return A.prompt_attention(a["q"], a["k"], a["v"], a["q_start"], a["scale"], a["out"], a["lse"], a["workspace"],
                                  a["status"])


ALL, CACHED, KV_ROWS, ATTENTION = ("append", "paged", "prompt"), ("append", "paged"), ("append", "prompt"), \
    ("paged", "prompt")
_cache64 = lambda: A.PagedKVCache(bf(PAGES, KV, PAGE, 128), bf(PAGES, KV, PAGE, 128))       # noqa: E731
_cache_cpu = lambda: A.PagedKVCache(bf(PAGES, KV, PAGE, D).cpu(), bf(PAGES, KV, PAGE, D).cpu())  # noqa: E731
_strided = lambda *s: bf(*s[:-1], 2 * s[-1])[..., ::2]                                      # noqa: E731

# calls, argument, its spoilt value, the start of the message
DEFECTS = [
    (ALL, "q", lambda: bf(T, HEADS * D), "q: "), (ALL, "q", lambda: bf(T, HEADS, D).float(), "q: bf16"),
    (ALL, "q", lambda: bf(T, HEADS, D).cpu(), "tensors on the current CUDA device"),
    (ALL, "q", lambda: _strided(T, HEADS, D), "q: the elements of a head"),
    (CACHED, "cache", _cache64, "disagree in head_dim"), (CACHED, "cache", _cache_cpu, "disagree in head_dim or device"),
    (KV_ROWS, "k", lambda: bf(T - 1, KV, D), "k: bf16"), (KV_ROWS, "k", lambda: bf(T, KV, D + 8), "k: bf16"),
    (("append",), "k", lambda: bf(T, KV + 1, D), "k: bf16"), (("prompt",), "k", lambda: bf(T, KV * D), "k: "),
    (KV_ROWS, "k", lambda: bf(T, KV, D).half(), "k: bf16"), (KV_ROWS, "k", lambda: bf(T, KV, D).cpu(), "k: bf16"),
    (KV_ROWS, "k", lambda: _strided(T, KV, D), "k: the elements of a head"),
    (KV_ROWS, "v", lambda: bf(T + 1, KV, D), "v: bf16"), (KV_ROWS, "v", lambda: bf(T, KV + 1, D), "v: bf16"),
    (KV_ROWS, "v", lambda: bf(T, KV, D).float(), "v: bf16"), (KV_ROWS, "v", lambda: bf(T, KV, D).cpu(), "v: bf16"),
    (KV_ROWS, "v", lambda: _strided(T, KV, D), "v: the elements of a head"),
    (ALL, "q_start", lambda: i32(0, 1, 3).long(), "q_start: contiguous int32"),
    (ALL, "q_start", lambda: i32(0, 1, 3).cpu(), "q_start: contiguous int32"),
    (ALL, "q_start", lambda: i32(0, 9, 1, 9, 3)[::2], "q_start: contiguous int32"),
    (ALL, "q_start", lambda: i32([0, 1, 3]), "q_start: contiguous int32"),
    (ALL, "q_start", lambda: i32(), "q_start: \\[sequences"),
    (CACHED, "kv_len", lambda: i32(20), "kv_len: contiguous int32"),
    (CACHED, "kv_len", lambda: i32(20, 30).long(), "kv_len: contiguous int32"),
    (CACHED, "kv_len", lambda: i32(20, 30).cpu(), "kv_len: contiguous int32"),
    (CACHED, "kv_len", lambda: i32(20, 0, 30)[::2], "kv_len: contiguous int32"),
    (CACHED, "page_table", lambda: i32(0, 1, 2, 3), "page_table: int32"),
    (CACHED, "page_table", lambda: i32([0, 1], [2, 3]).long(), "page_table: int32"),
    (CACHED, "page_table", lambda: i32([0, 1], [2, 3]).cpu(), "page_table: int32"),
    (CACHED, "page_table", lambda: i32([0, 1]), "page_table: \\[2"),
    (CACHED, "page_table", lambda: i32([0, 2], [1, 3]).T, "page_table: \\[2, pages\\] with contiguous rows"),
    (CACHED, "page_table", lambda: i32([0, 1]).expand(2, 2), "page_table: \\[2, pages\\] with contiguous rows"),
    (("append",), "cos_sin", lambda: f32(40, D).double(), "cos_sin: contiguous fp32"),
    (("append",), "cos_sin", lambda: f32(40, D).cpu(), "cos_sin: contiguous fp32"),
    (("append",), "cos_sin", lambda: f32(40 * D), "cos_sin: contiguous fp32"),
    (("append",), "cos_sin", lambda: f32(D, 40).T, "cos_sin: contiguous fp32"),
    (("append",), "cos_sin", lambda: f32(0, D), "cos_sin: "), (("append",), "cos_sin", lambda: f32(40, 0), "cos_sin: "),
    (("append",), "cos_sin", lambda: f32(40, 24), "kv_append"), (("append",), "cos_sin", lambda: f32(40, 80), "kv_append"),
    (ATTENTION, "lse", lambda: f32(T, HEADS + 1), "lse: contiguous fp32"),
    (ATTENTION, "lse", lambda: f32(T, HEADS).bfloat16(), "lse: contiguous fp32"),
    (ATTENTION, "lse", lambda: f32(HEADS, T).T, "lse: contiguous fp32"),
    (ATTENTION, "lse", lambda: f32(T, HEADS).cpu(), "lse: contiguous fp32"),
    (ALL, "status", lambda: i32(0).long(), "status: int32"), (ALL, "status", lambda: i32(0).cpu(), "status: int32"),
    (ALL, "status", lambda: i32(), "status: int32"),
    (("paged",), "max_new", lambda: -1, "paged_attention"), (ATTENTION, "scale", lambda: float("nan"), "_attention"),
    (ATTENTION, "scale", lambda: float("inf"), "_attention"),
]
# the written rows: q_out of an append, out of the attention calls
for bad, message in ((lambda: bf(T, HEADS, D + 8), "bf16"), (lambda: bf(T + 1, HEADS, D), "bf16"),
                     (lambda: bf(T, HEADS - 1, D), "bf16"), (lambda: bf(T, HEADS, D).half(), "bf16"),
                     (lambda: bf(T, HEADS, D).cpu(), "bf16"), (lambda: _strided(T, HEADS, D), "the elements of a head")):
    DEFECTS += [(("append",), "out", bad, "q_out: " + message), (ATTENTION, "out", bad, "out: " + message)]
CASES = [(call, *d[1:]) for d in DEFECTS for call in d[0]]


@pytest.mark.parametrize("call,name,bad,message", CASES, ids=[f"{c[0]}-{c[1]}-{i}" for i, c in enumerate(CASES)])
def test_refused(call, name, bad, message):
    good = Arguments()
    kept = {n: good.a[n] for n in ("out", "lse", "status")}
    before = {n: t.clone() for n, t in kept.items()}
    pools = good.k_pages.clone(), good.v_pages.clone()
    good.a[name] = bad()
    with pytest.raises(E.EpiloraError, match=message):
        good.call(call)
    torch.cuda.synchronize()
    assert all(torch.equal(kept[n], before[n]) for n in kept)
    assert torch.equal(good.k_pages, pools[0]) and torch.equal(good.v_pages, pools[1])


@pytest.mark.parametrize("call", ALL)
def test_good_arguments_are_taken(call):
    good = Arguments()
    o = good.call(call)
    torch.cuda.synchronize()
    assert o is good.a["out"] and int(good.a["status"].item()) == 0 and bool(torch.isfinite(o).all())
    assert not (o == 7.0).any()


@pytest.mark.parametrize("heads,want", [(HEADS, True), (7, False), (1, False)])
def test_head_counts(heads, want):
    """Query heads that are no multiple of the key/value heads are refused."""
    good = Arguments()
    good.a.update(q=bf(T, heads, D), out=bf(T, heads, D), lse=f32(T, heads))
    for call in ALL:
        if want:
            good.call(call)
        else:
            with pytest.raises(E.EpiloraError):
                good.call(call)


@pytest.mark.parametrize("make", [
    lambda k, v, s: A.PagedKVCache(k, v.cpu()), lambda k, v, s: A.PagedKVCache(k.byte(), v.byte(), s.cpu(), s),
    lambda k, v, s: A.PagedKVCache(k.byte(), v.byte(), s, s[:1]),
    lambda k, v, s: A.PagedKVCache(k.byte(), v.byte(), s, s.double()), lambda k, v, s: A.PagedKVCache(k.byte(), v.byte(), s),
    lambda k, v, s: A.PagedKVCache(k, v, s, s), lambda k, v, s: A.PagedKVCache(k, v[..., :32]),
    lambda k, v, s: A.PagedKVCache(k, v.byte()), lambda k, v, s: A.PagedKVCache(k[0], v[0]),
    lambda k, v, s: A.PagedKVCache(k.transpose(2, 3), v.transpose(2, 3))])
def test_cache_refused(make):
    with pytest.raises(E.EpiloraError, match="cache: "):
        make(bf(PAGES, KV, PAGE, D), bf(PAGES, KV, PAGE, D), f32(KV))


@pytest.mark.parametrize("shape,status", [((PAGES, KV, 8, D), "UNSUPPORTED"), ((PAGES, KV, 48, D), "UNSUPPORTED"),
                                          ((PAGES, KV, 16, 96), "UNSUPPORTED")])
def test_cache_sizes_refused_by_the_calls(shape, status):
    """Sizes that the kernels do not take are named by the status of the call."""
    good = Arguments()
    d = shape[-1]
    good.a.update(cache=A.PagedKVCache(bf(*shape), bf(*shape)), q=bf(T, HEADS, d), k=bf(T, KV, d), v=bf(T, KV, d),
                  out=bf(T, HEADS, d), cos_sin=f32(40, d))
    for call in CACHED:
        with pytest.raises(E.EpiloraError, match=status):
            good.call(call)
