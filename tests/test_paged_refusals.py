"""Refusals of the paged cache's Python side and of the decoding rounds, on the host (no GPU is touched)."""
import ctypes as C
import os
import shutil
import subprocess
import sys

import pytest
import torch

from semi_ar_draft_gb300 import decode_round as D


@pytest.mark.parametrize("n,rounds,max_len,places", [(24, 100, 512, 512), (513, 0, 512, 1024), (24, 9, 200, 100), (9, 1, 17, 64)])
def test_rounds_that_could_outgrow_the_cache_or_the_positions_are_refused(n, rounds, max_len, places):
    """A round feeds up to gamma + 1 = 9 tokens a request; positions past the table would be read out of bounds."""
    target = D.ToyTarget(32, 16, 1, 2, 1, 16, places, device="cpu")
    draft = D.ToyDraft(8, target)
    with pytest.raises(ValueError, match="tokens"):
        D.generate(target, draft, torch.zeros((2, n), dtype=torch.int32), rounds, max_len=max_len)


def test_positions_past_the_table_are_not_read():
    """What plan reports as an error must not fault in the embedding of the positions: they stop at the table's end."""
    target = D.ToyTarget(32, 16, 1, 2, 1, 16, 8, device="cpu")
    got = target.places(torch.tensor([-1, 0, 7, 8, 1 << 30], dtype=torch.int32))
    assert torch.equal(got, target.place[torch.tensor([0, 0, 7, 7, 7])])


def test_a_misaligned_error_word_is_refused():
    from semi_ar_draft_gb300 import binding as b, build

    build.build()
    assert b.dspark_cache_workspace_size(b.CacheParams(4, 16, 10, 5, 40, 1, 0x1004)) == 256
    assert b.dspark_cache_workspace_size(b.CacheParams(4, 16, 10, 5, 40, 1, 0x1002)) == 0
    p = b.AttentionParams(4, 4, 8, 2, 128, 16, 9, 3, 1, b.BF16, b.BF16, 1, 0, 0.1, 0.0, 1024, 128, 4096, 256, 128, 0x1004)
    assert b.dspark_paged_attention_workspace_size(p) > 256
    p.error = 0x1001
    assert b.dspark_paged_attention_workspace_size(p) == 0


A = [C.c_void_p(0x10000 * (i + 1)) for i in range(16)]  # addresses that nothing reads


@pytest.fixture(scope="module")
def L():
    from semi_ar_draft_gb300 import build

    build.build()
    from semi_ar_draft_gb300 import binding

    return binding.lib()


def test_plan_and_commit_refuse_every_output_over_an_input(L):
    """Blocks read cache_len, new_len, n_blocks, n_free, the stack and the table while others write the outputs."""
    from semi_ar_draft_gb300 import binding as b

    p = b.CacheParams(4, 16, 10, 5, 40, 1)
    # cache_len, new_len, block_table, n_blocks, free_pages, n_free | seq_len, offsets, slots, positions, n_blocks, n_free
    size = [16, 16, 80, 16, 40, 4, 16, 20, 320, 160, 16, 4]
    for i in range(6):
        for o in range(6, 12):
            for at in (A[i].value, A[i].value + size[i] - 4, A[i].value - size[o] + 4):  # over it, at its end, at its beginning
                args = list(A[:13])
                args[o] = C.c_void_p(at)
                assert L.dspark_cache_plan(C.byref(p), *args, 256, None) == 1, (i, o, at)
    for a, o in ((2, 0), (2, 4), (2, 5), (2, 3), (2, 1)):  # the table is written too
        args = list(A[:13])
        args[a] = A[o]
        assert L.dspark_cache_plan(C.byref(p), *args, 256, None) == 1, (a, o)
    # cache_len, add_len, done, block_table, n_blocks, free_pages, n_free | cache_len, n_blocks, n_free
    size = [16, 16, 4, 80, 16, 40, 4, 16, 16, 4]
    for i in range(7):
        for o in range(7, 10):
            for at in (A[i].value, A[i].value + size[i] - 4, A[i].value - size[o] + 4):
                args = list(A[:11])
                args[o] = C.c_void_p(at)
                assert L.dspark_cache_commit(C.byref(p), *args, 256, None) == 1, (i, o, at)
    for i in (0, 1, 2, 3, 4, 6):  # the stack is written too
        args = list(A[:11])
        args[5] = A[i]
        assert L.dspark_cache_commit(C.byref(p), *args, 256, None) == 1, i


def test_tensors_of_two_devices_are_refused():
    """Told apart before anything else is looked at (here: host memory beside tensors without memory)."""
    from semi_ar_draft_gb300 import api

    i = lambda *s, device="cpu": torch.zeros(s, dtype=torch.int32, device=device)  # noqa: E731
    z = lambda *s, device="cpu": torch.zeros(s, dtype=torch.bfloat16, device=device)  # noqa: E731
    ws = torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="one device"):
        api.cache_plan(i(4), i(4, device="meta"), i(4, 2), i(4), i(9), i(1), 16, 10, ws=ws)
    with pytest.raises(ValueError, match="one device"):
        api.cache_commit(i(4), i(4), i(4, 2), i(4), i(9, device="meta"), i(1), 16, ws=ws)
    with pytest.raises(ValueError, match="one device"):
        api.cache_append(z(4, 2, 64), z(4, 2, 64), z(5, 16, 2, 64), z(5, 16, 2, 64), torch.zeros(4, dtype=torch.int64, device="meta"))
    with pytest.raises(ValueError, match="one device"):
        api.paged_attention(z(4, 4, 64), z(5, 16, 2, 64), z(5, 16, 2, 64, device="meta"), i(4, 3), i(4))
    with pytest.raises(ValueError, match="device tensors"):
        api.paged_attention(z(4, 4, 64), z(5, 16, 2, 64), z(5, 16, 2, 64), i(4, 3), i(4), ws=ws)


def test_a_built_package_works_where_it_is_moved(L, tmp_path):
    """The native module finds the library beside it, and both loaders map the same one file."""
    from semi_ar_draft_gb300 import binding as b

    src = os.path.dirname(os.path.abspath(b.__file__))
    dst = tmp_path / "moved" / "semi_ar_draft_gb300"
    shutil.copytree(src, dst, ignore=shutil.ignore_patterns("__pycache__", "_build", "csrc"))
    code = ("from semi_ar_draft_gb300 import binding as b; b.native(); "
            "print('MAPS', sorted({l.split()[-1] for l in open('/proc/self/maps') if 'libdspark' in l or '_native.so' in l}))")
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path / "moved", capture_output=True, text=True,
                       env={**os.environ, "PYTHONPATH": str(tmp_path / "moved")})
    assert r.returncode == 0, r.stderr[-2000:]
    want = sorted(str(dst.resolve() / f) for f in ("libdspark.so", "_native.so"))
    assert f"MAPS {want}" in r.stdout, r.stdout


def test_an_argument_without_a_truth_value_says_so():
    """The error of `causal`'s own truth value comes through, and no result beside it."""
    from semi_ar_draft_gb300 import api

    class Neither:
        def __bool__(self):
            raise ArithmeticError("neither")

    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(ArithmeticError, match="neither"):
        api.paged_attention(z(4, 4, 64), z(5, 16, 2, 64), z(5, 16, 2, 64), i(4, 3), i(4), causal=Neither(),
                            ws=torch.zeros(256, dtype=torch.uint8))


def test_commit_refuses_settled_counts_over_anything_but_the_counts(L):
    from semi_ar_draft_gb300 import binding as b

    # cache_len, add_len, done, block_table, n_blocks, free_pages, n_free | cache_len, n_blocks, n_free
    size = [16, 16, 4, 80, 16, 40, 4, 16, 16, 4]
    for i in (1, 2, 3, 5, 7, 8, 9):
        for at in (A[i].value, A[i].value + size[i] - 4, A[i].value - 36 + 4):
            p = b.CacheParams(4, 16, 10, 5, 0, 1, None, at)
            assert L.dspark_cache_commit(C.byref(p), *A[:11], 256, None) == 1, (i, at)
    p = b.CacheParams(4, 16, 10, 5, 0, 1, None, 0x200002)
    assert L.dspark_cache_commit(C.byref(p), *A[:11], 256, None) == 1
