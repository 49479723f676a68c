"""Host-side argument checks of the attention entry points: every call below
is refused before anything is enqueued (fake, never dereferenced addresses;
only where no device exists to launch on), and the oracle's own pins."""
import numpy as np
import pytest
import torch

import precision_gemm_token_gb300 as E
from oracle import attention_oracle as AO
from precision_gemm_token_gb300 import attention as A

FAKE = 0x10000
INVALID, UNSUP, WS = E.EPILORA_ERR_INVALID_ARG, E.EPILORA_ERR_UNSUPPORTED, E.EPILORA_ERR_WORKSPACE
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer checks run only where nothing can launch")


@pytest.fixture(scope="module", autouse=True)
def lib():
    E.build()
    return E.load()


def cache(**kw):
    a = dict(kv_fmt=E.KV_BF16, kv_heads=2, head_dim=128, page_size=16, num_pages=10, reserved=0, k=FAKE, v=FAKE,
             k_page_stride=4096, k_head_stride=2048, k_token_stride=128, v_page_stride=4096, v_head_stride=2048,
             v_token_stride=128, k_scale=None, v_scale=None)
    a.update(kw)
    return E.KvCache(**a)


def batch(**kw):
    a = dict(n_seqs=2, n_tokens=3, max_new=2, table_pages=4, table_stride=4, q_start=FAKE, kv_len=FAKE, page_table=FAKE)
    a.update(kw)
    return E.KvBatch(**a)


BAD_CACHE = [(dict(kv_fmt=2), INVALID), (dict(reserved=1), INVALID), (dict(kv_heads=0), INVALID),
             (dict(kv_heads=3), INVALID), (dict(head_dim=96), UNSUP), (dict(head_dim=256), UNSUP),
             (dict(page_size=8), UNSUP), (dict(page_size=48), UNSUP), (dict(page_size=512), UNSUP),
             (dict(page_size=0), INVALID), (dict(num_pages=0), INVALID), (dict(k=None), INVALID), (dict(v=FAKE + 8), INVALID),
             (dict(k_token_stride=130), INVALID), (dict(v_head_stride=64), INVALID), (dict(k_page_stride=0), INVALID),
             (dict(kv_fmt=E.KV_E4M3), INVALID), (dict(kv_fmt=E.KV_E4M3, k_scale=FAKE, v_scale=FAKE + 2), INVALID),
             (dict(kv_fmt=E.KV_E4M3, k_scale=FAKE, v_scale=FAKE, k_token_stride=136), INVALID)]
BAD_BATCH = [(dict(n_seqs=-1), INVALID), (dict(n_tokens=-1), INVALID), (dict(max_new=-1), INVALID),
             (dict(table_pages=-1), INVALID), (dict(table_stride=3), INVALID), (dict(q_start=None), INVALID),
             (dict(kv_len=None), INVALID), (dict(page_table=None), INVALID), (dict(q_start=FAKE + 2), INVALID),
             (dict(table_pages=1 << 27, table_stride=1 << 27), UNSUP)]


def append(c=None, b=None, **kw):
    a = dict(heads=8, Q=FAKE, qs=(1536, 128), K=FAKE, ks=(1536, 128), V=FAKE, vs=(1536, 128), cs=FAKE, n_pos=100,
             rot=128, Qout=2 * FAKE, qos=(1024, 128))
    a.update(kw)
    return E.epilora_kv_append(c or cache(), b or batch(), a["heads"], a["Q"], a["qs"], a["K"], a["ks"], a["V"],
                               a["vs"], a["cs"], a["n_pos"], a["rot"], False, a["Qout"], a["qos"], None, 0)


def paged(c=None, b=None, **kw):
    a = dict(heads=8, Q=FAKE, qs=(1024, 128), scale=0.1, O=FAKE, os=(1024, 128), lse=None, ws=FAKE,
             n=E.epilora_attention_workspace_bytes(128))
    a.update(kw)
    return E.epilora_paged_attention(c or cache(), b or batch(), a["heads"], a["Q"], a["qs"], a["scale"], a["O"],
                                     a["os"], a["lse"], a["ws"], a["n"], None, 0)


def prompt(**kw):
    a = dict(n=2, T=3, qs0=FAKE, heads=8, kv=2, dim=128, Q=FAKE, qs=(1536, 128), K=FAKE, ks=(1536, 128), V=FAKE,
             vs=(1536, 128), scale=0.1, O=FAKE, os=(1024, 128), lse=None, ws=FAKE,
             wn=E.epilora_attention_workspace_bytes(128))
    a.update(kw)
    return E.epilora_prompt_attention(a["n"], a["T"], a["qs0"], a["heads"], a["kv"], a["dim"], a["Q"], a["qs"], a["K"],
                                      a["ks"], a["V"], a["vs"], a["scale"], a["O"], a["os"], a["lse"], a["ws"],
                                      a["wn"], None, 0)


@no_gpu
@pytest.mark.parametrize("kw,want", BAD_CACHE)
def test_cache_checks(kw, want):
    assert append(cache(**kw)) == want and paged(cache(**kw)) == want


@no_gpu
@pytest.mark.parametrize("kw,want", BAD_BATCH)
def test_batch_checks(kw, want):
    assert append(b=batch(**kw)) == want and paged(b=batch(**kw)) == want


@no_gpu
@pytest.mark.parametrize("kw", [dict(heads=7), dict(heads=0), dict(Q=None), dict(Qout=None), dict(Q=None, Qout=None),
                                dict(Q=FAKE + 8), dict(K=None), dict(V=None), dict(ks=(1536, 130)), dict(qs=(64, 128)),
                                dict(vs=(1536, 64)), dict(qos=(1024, 120)), dict(cs=FAKE + 4), dict(rot=24),
                                dict(rot=144), dict(rot=0), dict(n_pos=-1), dict(Qout=FAKE)])
def test_append_checks(kw):
    assert append(**kw) == INVALID


@no_gpu
@pytest.mark.parametrize("kw,want", [
    (dict(heads=9), INVALID), (dict(Q=None), INVALID), (dict(O=None), INVALID), (dict(O=FAKE + 2), INVALID),
    (dict(qs=(1024, 100)), INVALID), (dict(os=(100, 128)), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(lse=FAKE + 2), INVALID), (dict(ws=None), WS), (dict(n=0), WS),
    (dict(ws=FAKE + 16), WS)])
def test_paged_checks(kw, want):
    assert paged(**kw) == want


@no_gpu
@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), INVALID), (dict(T=-1), INVALID), (dict(qs0=None), INVALID), (dict(kv=3), INVALID), (dict(kv=0), INVALID),
    (dict(dim=32), UNSUP), (dict(K=None), INVALID), (dict(V=FAKE + 8), INVALID), (dict(ks=(1536, 129)), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(ws=None), WS), (dict(wn=1), WS)])
def test_prompt_checks(kw, want):
    assert prompt(**kw) == want


@no_gpu
def test_no_tokens_is_a_no_op():
    assert append(b=batch(n_tokens=0)) == 0 and paged(b=batch(n_tokens=0), Q=None, O=None, ws=None) == 0
    assert prompt(T=0, Q=None, O=None, ws=None) == 0


def test_null_structs_are_refused():
    lib = E.load()
    assert lib.epilora_kv_append(None, None, 8, *[None if i not in (1, 2, 4, 5, 7, 8) else 0 for i in range(9)], None,
                                 0, 0, 0, None, 0, 0, None, None) == INVALID


def test_workspace_sizes():
    assert E.epilora_attention_workspace_bytes(128) > 0 and E.epilora_attention_workspace_bytes(64) > 0
    assert E.epilora_attention_workspace_bytes(96) == 0 and E.epilora_attention_workspace_bytes(0) == 0


def test_struct_sizes_match_the_header(tmp_path):
    import ctypes
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "sizes.c"
    src.write_text('#include "epilora.h"\n#include <stdio.h>\nint main(void) { printf("%zu %zu %zu %zu", '
                   'sizeof(epilora_kv_cache), sizeof(epilora_kv_batch), offsetof(epilora_kv_cache, k_scale), '
                   'offsetof(epilora_kv_batch, page_table)); return 0; }\n')
    exe = str(tmp_path / "sizes")
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", exe], check=True)
    got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(E.KvCache), ctypes.sizeof(E.KvBatch), E.KvCache.k_scale.offset,
                   E.KvBatch.page_table.offset]


def test_tensor_helpers_refuse():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)   # noqa: E731
    with pytest.raises(E.EpiloraError):
        A.PagedKVCache(bf(4, 2, 16, 128), bf(4, 2, 16, 64))
    with pytest.raises(E.EpiloraError):
        A.PagedKVCache(bf(4, 2, 16, 128).float(), bf(4, 2, 16, 128).float())
    with pytest.raises(E.EpiloraError):
        A.PagedKVCache(bf(4, 2, 16, 128).to(torch.uint8), bf(4, 2, 16, 128).to(torch.uint8))
    with pytest.raises(E.EpiloraError):
        A.PagedKVCache(bf(4, 2, 16, 128), bf(4, 2, 16, 128), torch.ones(2), torch.ones(2))
    with pytest.raises(E.EpiloraError):
        A.PagedKVCache(bf(4, 2, 128, 16).transpose(2, 3), bf(4, 2, 128, 16).transpose(2, 3))
    c = A.PagedKVCache(bf(4, 16, 2, 128).transpose(1, 2), bf(4, 16, 2, 128).transpose(1, 2))
    assert (c.struct.k_page_stride, c.struct.k_head_stride, c.struct.k_token_stride) == (4096, 128, 256)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)    # noqa: E731
    table = torch.zeros(1, 2, dtype=torch.int32)
    for args in ((bf(1, 8, 128), c, i32(0, 1), i32(1), table),                      # not on a GPU
                 (bf(1, 8, 64), c, i32(0, 1), i32(1), table), (bf(8, 128), c, i32(0, 1), i32(1), table),
                 (bf(1, 8, 128).float(), c, i32(0, 1), i32(1), table), (bf(1, 8, 128), c, i32(0, 1).long(), i32(1), table),
                 (bf(1, 8, 128), c, i32(0, 1), i32(1, 1), table), (bf(1, 8, 128), c, i32(0, 1), i32(1), table[0])):
        with pytest.raises((E.EpiloraError, ValueError)):
            A.paged_attention(*args)
    with pytest.raises(E.EpiloraError):
        A.prompt_attention(bf(3, 8, 128), bf(2, 2, 128), bf(3, 2, 128), i32(0, 3))
    with pytest.raises(E.EpiloraError):
        A.kv_append(bf(3, 8, 128), bf(3, 1, 128), bf(3, 1, 128), c, i32(0, 3), i32(3), table)


def test_oracle_pins():
    """Equal scores average; one visible position is copied; the rotation
    keeps norms and depends on position differences only."""
    rng = np.random.default_rng(0)
    k, v = np.zeros((5, 1, 64)), rng.standard_normal((5, 1, 64))
    q = rng.standard_normal((2, 2, 64))
    o, lse, _ = AO.attention_rows(q, k, v, [4, 0], 0.3)
    assert np.allclose(o[0], v[:, 0].mean(0)) and np.allclose(o[1], v[0, 0])
    assert np.allclose(lse[0], np.log(5)) and np.allclose(lse[1], 0)
    o, lse, _ = AO.attention_rows(q, k, v, [-1, 2], 0.3)
    assert (o[0] == 0).all() and np.isneginf(lse[0]).all()
    x, y = rng.standard_normal((2, 64)).astype(np.float32)
    for inter in (False, True):
        dots = []
        for a in (3, 10):
            t = lambda p: (np.cos(p * 0.1 ** np.arange(32)).astype(np.float32),   # noqa: E731
                           np.sin(p * 0.1 ** np.arange(32)).astype(np.float32))
            xr, yr = AO.rotate_f32(x, *t(a), inter), AO.rotate_f32(y, *t(a + 4), inter)
            assert np.isclose(np.linalg.norm(xr), np.linalg.norm(x), rtol=1e-5)
            dots.append(float(xr @ yr))
        assert np.isclose(dots[0], dots[1], rtol=1e-3, atol=1e-3)
