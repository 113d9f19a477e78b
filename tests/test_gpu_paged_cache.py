"""PagedCache: rounds replayed from a graph, errors kept until they are read, memory at construction, steps of other
token counts."""
import pytest
import torch

from semi_ar_draft_gb300 import api
from semi_ar_draft_gb300.paged import PagedCache

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Round:
    """A round's inputs in tensors that stay where they are, and the round itself."""

    def __init__(self, B, T, Hq=4, Hk=1, D=64):
        self.new, self.acc, self.done = i32([0] * B), i32([0] * B), torch.zeros(B, dtype=torch.uint8, device="cuda")
        self.q, self.k, self.v = (torch.zeros((T, h, D), dtype=torch.bfloat16, device="cuda") for h in (Hq, Hk, Hk))

    def fill(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.new.random_(0, 8, generator=g)
        self.acc.copy_((torch.rand(len(self.new), generator=g, device="cuda") * (self.new + 1)).int())
        self.done.copy_(torch.rand(len(self.new), generator=g, device="cuda") < 0.2)
        for x in (self.q, self.k, self.v):
            x.normal_(generator=g)

    def run(self, cache, stream=None):
        cache.plan(self.new, extra=1, max_new=8, stream=stream)
        cache.append(0, self.k, self.v, stream=stream)
        out, _ = cache.attend(0, self.q, stream=stream)
        cache.commit(self.acc, extra=1, done=self.done, stream=stream)
        return out


@pytest.mark.parametrize("calls", [1, 2])
def test_rounds_replay_from_a_graph(calls):
    """A graph of one round (or of two), replayed: every replay goes on from where the last one stopped."""
    B, T = 6, 48
    eager, replayed = (PagedCache(B, 80, 8, 40, 1, 1, 64, T) for _ in range(2))
    inputs = [Round(B, T) for _ in range(calls)]
    inputs[0].run(PagedCache(B, 80, 8, 40, 1, 1, 64, T))  # the kernels' first launches, beside both caches
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [r.run(replayed) for r in inputs]
    for n in range(4):
        for i, r in enumerate(inputs):
            r.fill(10 * n + i)
        want = [r.run(eager) for r in inputs]
        graph.replay()
        torch.cuda.synchronize()
        for out, ref in zip(outs, want):
            assert torch.equal(out, ref), n
        assert replayed.cache_len.tolist() == eager.cache_len.tolist(), n
        assert int(replayed.n_free) == int(eager.n_free) and torch.equal(replayed.offsets, eager.offsets)
    assert eager.status() == 0 and replayed.status() == 0 and int(eager.cache_len.max()) > 8


@pytest.mark.parametrize("times", [1, 60])  # the commit's kernel in one block; in a cluster of three
def test_finished_requests_replay_from_a_graph(times):
    """A graph of a commit alone."""
    cache = PagedCache(3 * times, 12 * times, 4, 4, 1, 1, 64, 24 * times)
    done = torch.ones(3 * times, dtype=torch.uint8, device="cuda")
    new = i32([5, 1, 8] * times)
    cache.plan(new)
    cache.commit(new)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        cache.commit(done=done)
    for _ in range(3):
        graph.replay()
        assert int(cache.n_free) == 12 * times and cache.cache_len.tolist() == [0, 0, 0] * times
        assert cache.free_pages.unique().numel() == 12 * times
        cache.plan(new)
        cache.commit(new)
        assert int(cache.n_free) == (12 - 5) * times and cache.cache_len.tolist() == [5, 1, 8] * times


def test_counts_are_read_through_the_same_tensors():
    """cache_len and n_free taken once show the counts after every later call, also on a stream of its own."""
    cache = PagedCache(2, 9, 4, 4, 1, 1, 64, 16)
    lengths, free = cache.cache_len, cache.n_free
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, side, side.cuda_stream, 0):
        cache.plan(i32([3, 1]), stream=stream)
        cache.commit(i32([3, 1]), stream=stream)
        torch.cuda.synchronize()
    assert lengths.tolist() == [12, 4] and int(free) == 9 - 4 and cache.status() == 0


# ------------------------------------------------------------------ errors
def test_a_plans_error_outlives_the_commit():
    """More tokens than max_tokens: some have no slot, their keys are never written, and the commit finds nothing wrong."""
    cache = PagedCache(2, 9, 4, 4, 1, 1, 64, 8)
    cache.plan(i32([6, 6]))
    cache.commit(i32([1, 1]))
    assert cache.status() == 8
    cache.plan(i32([3, 3]))
    cache.commit(i32([1, 1]))
    assert cache.status() == 0  # reading it clears it


def test_a_full_pool_is_still_known_after_the_commit():
    cache = PagedCache(2, 3, 4, 8, 1, 1, 64, 40)
    cache.plan(i32([9, 9]))
    cache.commit(i32([1, 1]))
    assert cache.status() == 8 and cache.status() == 0


@pytest.mark.parametrize("Hq,max_new", [(4, 1), (64, 9)])  # row tiles of 16, of 128
@pytest.mark.parametrize("other_stream", [False, True])
def test_an_error_of_attention_is_seen(Hq, max_new, other_stream):
    cache = PagedCache(2, 8, 4, 4, 1, 1, 64, 16)
    cache.plan(i32([8, 3]), max_new=max_new)
    good = int(cache.block_table[0, 1])
    q = torch.randn((16, Hq, 64), device="cuda").to(torch.bfloat16)
    cache.block_table[0, 1] = 77
    side = torch.cuda.Stream() if other_stream else None
    torch.cuda.synchronize()
    cache.attend(0, q, stream=side)
    torch.cuda.synchronize()
    cache.block_table[0, 1] = good
    cache.attend(0, q)
    cache.commit(i32([8, 3]))
    assert cache.status() == 8 and cache.status() == 0


def test_the_error_word_of_the_calls():
    """The first error stays until its owner clears it; the workspace's status is each call's own."""
    error = i32([0])
    args = lambda n_free: (i32([3]), i32([4]), i32([[0, -1]]), i32([1]), i32([1, 2, 3, 0]), i32([n_free]), 4, 8)  # noqa: E731
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    status = lambda: api.b.dspark_get_device_status(ws)  # noqa: E731
    api.cache_plan(*args(3), ws=ws, error=error)
    assert status() == 0 and int(error) == 0
    api.cache_plan(*args(0), ws=ws, error=error)
    assert status() == 8 and int(error) == 8
    api.cache_plan(*args(3), ws=ws, error=error)
    assert status() == 0 and int(error) == 8
    error.fill_(4)
    api.cache_commit(i32([99]), None, i32([[0, -1]]), i32([1]), i32([1, 2, 3, 0]), i32([3]), 4, ws=ws, error=error)
    assert status() == 8 and int(error) == 4
    with pytest.raises(ValueError):
        api.cache_plan(*args(3), error=torch.zeros(1, device="cuda"))
    with pytest.raises(ValueError):
        api.cache_commit(i32([9]), None, i32([[0, -1]]), i32([1]), i32([1, 2, 3, 0]), i32([3]), 4, error=i32([0, 0]))


# ------------------------------------------------------------------ streams
def test_tensors_made_for_a_stream_given_by_its_address_stay_reserved():
    """Memory of an output that is let go while its stream still works is not handed out to the current stream."""
    cache = PagedCache(1, 64, 16, 64, 1, 1, 64, 512)
    cache.plan(i32([512]))
    q = torch.zeros((512, 8, 64), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    api.paged_attention(q, cache.k_pages[0], cache.v_pages[0], cache.block_table, cache.seq_len, cache.offsets)  # loads the kernels
    for stream in (side, side.cuda_stream):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(600_000_000)  # cycles: a third of a second of work before the call
        out, _, ws = api.paged_attention(q, cache.k_pages[0], cache.v_pages[0], cache.block_table, cache.seq_len, cache.offsets,
                                         stream=stream)
        at, n, size = out.data_ptr(), out.numel(), ws.numel()
        del out, ws
        assert not side.query()
        made = [torch.empty(n, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
        made += [torch.empty(size, dtype=torch.uint8, device="cuda")]
        assert at not in [x.data_ptr() for x in made]
        del made
    torch.cuda.synchronize()


# ------------------------------------------------------------------ memory and steps
def test_an_8_bit_cache_is_built_without_a_wider_copy():
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    cache = PagedCache(4, 4096, 64, 64, 1, 4, 128, 64, kv_dtype=E4M3)
    pools = cache.k_pages.nbytes + cache.v_pages.nbytes
    assert pools == 2 * 4096 * 64 * 4 * 128 and not cache.k_pages.view(torch.uint8).any()
    assert torch.cuda.max_memory_allocated() - before <= pools + (4 << 20)


@pytest.mark.parametrize("kv", [None, E4M3])
def test_steps_of_different_token_counts(kv):
    """Prompts and decoding steps through one cache: a step's tensors have its own number of rows."""
    B, D, Hk, Hq = 3, 64, 2, 8
    g = torch.Generator(device="cuda").manual_seed(2)
    small, full = (PagedCache(B, 60, 16, 20, 1, Hk, D, 300, kv_dtype=kv) for _ in range(2))
    for new, tokens in (([100, 9, 120], 240), ([1, 1, 1], 3), ([4, 2, 1], 10)):
        n = i32(new)
        small.plan(n, tokens=tokens)
        full.plan(n)
        assert small.slots.numel() == small.positions.numel() == tokens and full.slots.numel() == 300
        assert torch.equal(full.slots[:tokens], small.slots) and torch.equal(full.positions[:tokens], small.positions)
        q, k, v = (torch.randn((300, h, D), generator=g, device="cuda").to(torch.bfloat16) for h in (Hq, Hk, Hk))
        for c, T in ((small, tokens), (full, 300)):
            c.append(0, k[:T], v[:T])
        (out, _), (ref, _) = small.attend(0, q[:tokens]), full.attend(0, q)
        # (the same keys and values; which kernel runs may differ, so a rounding of p and of the output either way)
        assert bool(((out - ref[:tokens]).abs() <= 2.0 ** -7 * (ref[:tokens].abs() + 4)).all())
        small.commit(n)
        full.commit(n)
    assert torch.equal(small.k_pages.view(torch.uint8), full.k_pages.view(torch.uint8))
    assert small.status() == 0 and full.status() == 0
    small.plan(i32([5, 5, 5]), tokens=12)  # fewer than there are: an error, as with max_tokens
    assert small.status() == 8
    with pytest.raises(ValueError):
        small.plan(i32([1, 1, 1]), tokens=301)


def test_a_plan_replaces_the_one_that_no_commit_followed():
    """Planning a step again, larger or smaller, ends as if it had been planned once."""
    once, again = (PagedCache(2, 20, 4, 8, 1, 1, 64, 64) for _ in range(2))
    for first, new, acc in (([9, 1], [5, 7], [5, 2]), ([2, 2], [12, 1], [3, 1]), ([20, 3], [1, 9], [1, 9])):
        again.plan(i32(first))
        for c in (once, again):
            c.plan(i32(new))
        assert torch.equal(once.slots[: sum(new)], again.slots[: sum(new)]) and int(once.n_free) == int(again.n_free)
        for c in (once, again):
            c.commit(i32(acc))
        assert once.cache_len.tolist() == again.cache_len.tolist() and int(once.n_free) == int(again.n_free)
        held = [p for j in range(2) for p in again.block_table[j, : -(-int(again.cache_len[j]) // 4)].tolist()]
        assert sorted(held + again.free_pages[: int(again.n_free)].tolist()) == list(range(20))
    assert once.status() == 0 and again.status() == 0
