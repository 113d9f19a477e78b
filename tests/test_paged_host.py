"""Refusals of the paged-cache entry points, on the host (no GPU is touched)."""
import ctypes as C

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from semi_ar_draft_gb300 import build

    build.build()
    from semi_ar_draft_gb300 import binding

    return binding.lib()


A = [C.c_void_p(0x10000 * (i + 1)) for i in range(16)]  # addresses that nothing reads


def test_cache_params(L):
    from semi_ar_draft_gb300 import binding as b

    ok = dict(B=4, page_size=16, num_pages=10, max_blocks=5, max_tokens=40, extra=1)
    assert b.dspark_cache_workspace_size(b.CacheParams(**ok)) == 256
    for bad in ({"B": 0}, {"page_size": 0}, {"page_size": 24}, {"page_size": 8192}, {"num_pages": 0}, {"max_blocks": 0},
                {"B": 8193}):
        p = b.CacheParams(**{**ok, **bad})
        assert b.dspark_cache_workspace_size(p) == 0
        want = 2 if bad.get("B") == 8193 else 1
        assert L.dspark_cache_plan(C.byref(p), *A[:13], 256, None) == want
        assert L.dspark_cache_commit(C.byref(p), *A[:11], 256, None) == want
    for bad in ({"max_tokens": -1}, {"extra": -1}):
        assert L.dspark_cache_plan(C.byref(b.CacheParams(**{**ok, **bad})), *A[:13], 256, None) == 1


def test_plan_and_commit_pointers(L):
    from semi_ar_draft_gb300 import binding as b

    p = b.CacheParams(4, 16, 10, 5, 40, 1)
    names = ["cache_len", "new_len", "block_table", "n_blocks", "free_pages", "n_free", "seq_len", "offsets", "slots",
             "positions", "n_blocks_out", "n_free_out"]
    for i, name in enumerate(names):
        args = list(A[:13])
        args[i] = None
        if name not in ("new_len", "positions"):
            assert L.dspark_cache_plan(C.byref(p), *args, 256, None) == 1, name
    # an output over an input, also in part
    for i, o in ((0, 6), (3, 10), (5, 11), (1, 7)):
        args = list(A[:13])
        args[o] = C.c_void_p(args[i].value + (4 if i in (0, 3) else 0))
        assert L.dspark_cache_plan(C.byref(p), *args, 256, None) == 1, (i, o)
    # workspace: missing, misaligned, short
    assert L.dspark_cache_plan(C.byref(p), *A[:12], None, 256, None) == 6
    assert L.dspark_cache_plan(C.byref(p), *A[:12], C.c_void_p(0x1010), 256, None) == 6
    assert L.dspark_cache_plan(C.byref(p), *A[:13], 255, None) == 6
    for i in range(11):
        args = list(A[:11])
        args[i] = None
        if i not in (1, 2, 10):  # add_len, done; the workspace has its own status
            assert L.dspark_cache_commit(C.byref(p), *args, 256, None) == 1, i
    assert L.dspark_cache_commit(C.byref(p), *A[:10], None, 256, None) == 6
    for i, o in ((0, 7), (3 + 1, 8), (6, 9)):
        args = list(A[:11])
        args[o] = args[i]
        assert L.dspark_cache_commit(C.byref(p), *args, 256, None) == 1, (i, o)


def test_append_arguments(L):
    from semi_ar_draft_gb300 import binding as b

    ok = dict(T=4, Hk=2, D=128, page_size=16, num_pages=9, dtype=b.BF16, kv_dtype=b.BF16, k_token_stride=256, k_head_stride=128,
              v_token_stride=256, v_head_stride=128, kv_page_stride=4096, kv_token_stride=256, kv_head_stride=128)
    call = lambda p, *a: L.dspark_cache_append(C.byref(b.AppendParams(**p)), *(a or A[:7]), None)  # noqa: E731
    for bad, want in (({"T": -1}, 1), ({"Hk": 0}, 1), ({"D": 0}, 1), ({"D": 120}, 2), ({"D": 8192}, 2), ({"page_size": 3}, 1),
                      ({"num_pages": 0}, 1), ({"dtype": b.F32}, 1), ({"dtype": b.E4M3}, 1), ({"kv_dtype": b.F16}, 1),
                      ({"kv_dtype": 9}, 1), ({"kv_page_stride": 4097}, 1), ({"kv_token_stride": 4}, 1),
                      ({"kv_dtype": b.E4M3, "kv_head_stride": 136}, 1)):
        assert call({**ok, **bad}) == want, bad
    for i in (0, 1, 2, 3, 4):
        args = list(A[:7])
        args[i] = None
        assert call(ok, *args) == 1, i
    odd = list(A[:7])
    odd[2] = C.c_void_p(odd[2].value + 8)
    assert call(ok, *odd) == 1
    assert call({**ok, "T": 0}) == 0  # nothing to do, nothing enqueued


def test_attention_arguments(L):
    from semi_ar_draft_gb300 import binding as b

    ok = dict(T=4, B=4, Hq=8, Hk=2, D=128, page_size=16, num_pages=9, max_blocks=3, max_new=1, dtype=b.BF16, kv_dtype=b.BF16,
              causal=1, window=0, scale=0.1, softcap=0.0, q_token_stride=1024, q_head_stride=128, kv_page_stride=4096,
              kv_token_stride=256, kv_head_stride=128)
    size = b.dspark_paged_attention_workspace_size(b.AttentionParams(**ok))
    assert size > 256

    def call(p, nbytes=size, **ptr):
        names = ["q", "k", "v", "table", "seq", "offsets", "ks", "vs", "out", "lse", "ws"]
        args = [ptr.get(n, A[i]) for i, n in enumerate(names)]
        return L.dspark_paged_attention(C.byref(b.AttentionParams(**p)), *args, nbytes, None)

    nan, inf = float("nan"), float("inf")
    for bad, want in (({"T": -1}, 1), ({"B": 0}, 1), ({"Hk": 0}, 1), ({"Hq": 7}, 1), ({"Hq": 0}, 1), ({"D": 0}, 1), ({"D": 72}, 2),
                      ({"D": 272}, 2), ({"page_size": 17}, 1), ({"num_pages": 0}, 1), ({"max_blocks": 0}, 1), ({"window": -1}, 1),
                      ({"dtype": b.F32}, 1), ({"dtype": b.E4M3, "kv_dtype": b.E4M3}, 1), ({"kv_dtype": b.F16}, 1),
                      ({"scale": nan}, 1), ({"scale": inf}, 1), ({"softcap": -1.0}, 1), ({"softcap": nan}, 1),
                      ({"softcap": inf}, 1), ({"kv_page_stride": 4100}, 1), ({"kv_token_stride": 1}, 1),
                      ({"kv_head_stride": 132}, 1), ({"T": 1 << 28}, 2)):
        assert call({**ok, **bad}) == want, bad
    for name in ("q", "k", "v", "table", "seq", "out"):
        assert call(ok, **{name: None}) == 1, name
    assert call({**ok, "T": 3}, offsets=None) == 1  # one token a request: T >= B
    for name, by in (("k", 8), ("v", 4), ("out", 2), ("q", 1)):
        assert call(ok, **{name: C.c_void_p(0x90000 + by)}) == 1, name
    assert call(ok, nbytes=size - 1) == 6
    assert call(ok, ws=None) == 6
    assert call(ok, ws=C.c_void_p(0x1010)) == 6
    for bad in ({"D": 72}, {"B": 0}):
        assert b.dspark_paged_attention_workspace_size(b.AttentionParams(**{**ok, **bad})) == 0


def test_status_string(L):
    from semi_ar_draft_gb300 import binding as b

    assert "cache" in b.dspark_status_string(8)


def test_api_checks():
    """Shapes and types, before any address is taken."""
    from semi_ar_draft_gb300 import api

    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        api.cache_plan(i(4), i(3), i(4, 2), i(4), i(9), i(1), 16, 10)
    with pytest.raises(ValueError):
        api.cache_plan(i(4).long(), i(4), i(4, 2), i(4), i(9), i(1), 16, 10)
    with pytest.raises(ValueError):
        api.cache_plan(i(4), i(4), i(3, 2), i(4), i(9), i(1), 16, 10)
    with pytest.raises(ValueError):
        api.cache_commit(i(4), i(4), i(4, 2), i(4), i(9), i(1), 16, done=torch.zeros(4))
    pool = torch.zeros((5, 16, 2, 64), dtype=torch.bfloat16)
    q = torch.zeros((4, 4, 64), dtype=torch.bfloat16)
    k = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    slots = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        api.cache_append(k, k[:3], pool, pool, slots)
    with pytest.raises(ValueError):
        api.cache_append(k, k, pool, pool, slots.int())
    with pytest.raises(ValueError):
        api.cache_append(k, k, pool, pool, slots, k_scale=torch.ones(2))  # not an 8-bit cache
    with pytest.raises(ValueError):
        api.cache_append(k, k, pool, pool.transpose(0, 1), slots)
    with pytest.raises(TypeError):
        api.cache_append(k.float(), k.float(), pool, pool, slots)
    with pytest.raises(ValueError):
        api.paged_attention(q[:, :, :32], pool, pool, i(4, 3), i(4))
    with pytest.raises(ValueError):
        api.paged_attention(q, pool, pool, i(3, 3), i(4))
    with pytest.raises(ValueError):
        api.paged_attention(q, pool, pool, i(4, 3), i(4), offsets=i(4))
    with pytest.raises(ValueError):
        api.paged_attention(q, pool, pool, i(4, 3), i(4), lse=torch.zeros(4, 4, dtype=torch.float64))
    with pytest.raises(ValueError):  # host memory
        api.paged_attention(q, pool, pool, i(4, 3), i(4), ws=torch.zeros(1, dtype=torch.uint8))
