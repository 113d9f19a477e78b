"""Pages on their way through plan and commit where some are missing: given back early, not to be had, or not of the pool."""
import pytest
import torch

from semi_ar_draft_gb300 import api, binding

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def commit_reference(cache_len, add, table, n_blocks, free, n_free, page, extra, done, num_pages):
    """(cache_len, n_blocks, n_free, free, bad): entries that are no page do not go back, those past the pool are an error."""
    free, top, bad, length, held = list(free), n_free, False, [], []
    for j in range(len(cache_len)):
        n = 0 if done[j] else cache_len[j] + add[j] + extra
        bad |= n < 0 or n > n_blocks[j] * page
        n = min(max(n, 0), n_blocks[j] * page)
        keep = -(-n // page)
        for p in table[j][keep:n_blocks[j]]:
            if p < 0:
                continue
            if p >= num_pages or top == num_pages:
                bad = True
                continue
            free[top] = p
            top += 1
        length.append(n)
        held.append(keep)
    return length, held, top, free, bad


@pytest.mark.parametrize("B,most,window,beyond", [(1, 9, 3, 0), (3, 40, 5, 0), (64, 30, 7, 0), (65, 33, 1, 0), (200, 70, 30, 0),
                                                  (700, 20, 8, 0), (3000, 9, 2, 0), (2, 3000, 700, 0), (90, 40, 5, 4)])
def test_commit_of_requests_whose_first_pages_are_gone(B, most, window, beyond):
    """Sliding windows: a request keeps `window` pages, its first entries are -1 (or, `beyond`, past the pool)."""
    page = 16
    g = torch.Generator().manual_seed(B + most)
    n_blocks = torch.randint(0, most + 1, (B,), generator=g).tolist()
    live = [min(n, window) for n in n_blocks]
    P = sum(live) + 5
    perm = torch.randperm(P, generator=g).tolist()
    table, used = [], 0
    for n, k in zip(n_blocks, live):
        gone = [-1 - (i % 3) for i in range(n - k)]
        if beyond and len(gone) > beyond:
            gone[beyond] = P + 7
        table.append(gone + perm[used:used + k] + [-9] * (most - n))
        used += k
    free, n_free = perm[used:] + [-5] * used, P - used
    cache_len = [max(n * page - 3, 0) for n in n_blocks]
    add = [0] * B
    done = [int(x) for x in torch.rand(B, generator=g) < 0.4]
    f = i32(free)
    length, held, left, ws = api.cache_commit(i32(cache_len), i32(add), i32(table), i32(n_blocks), f, i32([n_free]), page,
                                              done=torch.tensor(done, dtype=torch.uint8, device="cuda"))
    ref = commit_reference(cache_len, add, table, n_blocks, free, n_free, page, 0, done, P)
    got = (length.tolist(), held.tolist(), left.item(), f.tolist(), binding.dspark_get_device_status(ws) == 8)
    assert got == ref
    on_stack = got[3][: got[2]]
    assert len(set(on_stack)) == len(on_stack) and min(on_stack) >= 0 and max(on_stack) < P


def test_pages_of_windowed_requests_are_given_out_once():
    """Pages before a window go back by the caller's hand, the rest by commit, and all are handed out again."""
    page, P, width = 4, 12, 8
    table = i32([[0, 1, 2, 3, 4, -1, -1, -1], [5, 6, 7, -1, -1, -1, -1, -1]])
    free, n_free, n_blocks, cache_len = i32([11, 10, 9, 8] + [-1] * 8), i32([4]), i32([5, 3]), i32([18, 11])
    # request 0 keeps a window of two pages
    free[4:7], n_free = table[0, :3], i32([7])
    table[0, :3] = -1
    cache_len, n_blocks, n_free, ws = api.cache_commit(cache_len, None, table, n_blocks, free, n_free, page,
                                                       done=torch.tensor([1, 0], dtype=torch.uint8, device="cuda"))
    assert binding.dspark_get_device_status(ws) == 0 and int(n_free) == 9
    assert sorted(free[:9].tolist()) == [0, 1, 2, 3, 4, 8, 9, 10, 11]
    seq, off, slots, pos, n_blocks, n_free, ws = api.cache_plan(cache_len, i32([32, 5]), table, n_blocks, free, n_free, page, 40)
    assert binding.dspark_get_device_status(ws) == 0 and int(n_free) == 0
    held = table[0, :8].tolist() + table[1, :4].tolist()
    assert sorted(held) == list(range(P))
    live = slots[: int(off[-1])]
    assert int(live.min()) >= 0 and live.unique().numel() == live.numel()


@pytest.mark.parametrize("B,short", [(3, 4), (70, 30), (400, 333)])
def test_blocks_without_a_page_name_none(B, short):
    """Where the stack runs out, the table does not go on naming pages that were given back: their keys are others' now."""
    page, width = 4, 9
    g = torch.Generator().manual_seed(B)
    cache_len = torch.randint(0, 13, (B,), generator=g).tolist()
    new = torch.randint(0, 20, (B,), generator=g).tolist()
    n_blocks = [-(-x // page) for x in cache_len]
    need = [-(-(x + n) // page) - h for x, n, h in zip(cache_len, new, n_blocks)]
    short = min(short, sum(need))
    assert short > 0
    held, P = sum(n_blocks), sum(n_blocks) + sum(need) - short
    perm = torch.randperm(P, generator=g).tolist()
    table, used = [], 0
    for h in n_blocks:
        table.append(perm[used:used + h] + [perm[i % P] for i in range(width - h)])  # what earlier rounds left behind
        used += h
    free = perm[used:] + [-1] * used
    t = i32(table)
    seq, off, slots, pos, blocks, left, ws = api.cache_plan(i32(cache_len), i32(new), t, i32(n_blocks), i32(free), i32([P - held]),
                                                            page, sum(new) + 3)
    assert binding.dspark_get_device_status(ws) == 8 and left.item() == 0
    stack, want = free[: P - held][::-1], [list(r) for r in table]
    for j in range(B):
        for b in range(n_blocks[j], n_blocks[j] + need[j]):
            want[j][b] = stack.pop(0) if stack else -1
    assert t.tolist() == want
    # attention over such a step says so
    q = torch.zeros((sum(new), 1, 64), dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros((P, page, 1, 64), dtype=torch.bfloat16, device="cuda")
    _, _, ws = api.paged_attention(q, pool, pool, t, seq, off)
    assert binding.dspark_get_device_status(ws) == 8


@pytest.mark.parametrize("B", [1, 64, 65, 700, 5000])
def test_commit_settles_the_counts_over_its_inputs(B):
    """The three outputs once more, over cache_len, n_blocks and n_free: one block, clusters, several requests a thread."""
    page, most = 8, 5
    g = torch.Generator().manual_seed(B)
    n_blocks = torch.randint(0, most + 1, (B,), generator=g).int()
    cache_len = (n_blocks * page - torch.randint(0, page, (B,), generator=g).int()).clamp(min=0)
    add = -(torch.rand(B, generator=g) * cache_len).int()
    P = int(n_blocks.sum()) + 9
    perm = torch.randperm(P, generator=g).int()
    table, used = torch.full((B, most), -1, dtype=torch.int32), 0
    for j, n in enumerate(n_blocks.tolist()):
        table[j, :n] = perm[used:used + n]
        used += n
    free = torch.cat([perm[used:], torch.zeros(used, dtype=torch.int32)])
    done = torch.rand(B, generator=g) < 0.2
    dev = [x.cuda() for x in (add, table, done)]
    counts = torch.cat([cache_len, n_blocks, torch.tensor([P - used], dtype=torch.int32)]).cuda()
    stacks = [free.cuda() for _ in range(2)]
    ref = api.cache_commit(counts[:B].clone(), dev[0], dev[1], counts[B:2 * B].clone(), stacks[0], counts[2 * B:].clone(), page,
                           done=dev[2])
    out = api.cache_commit(counts[:B], dev[0], dev[1], counts[B:2 * B], stacks[1], counts[2 * B:], page, done=dev[2], settled=counts)
    assert all(torch.equal(x, y) for x, y in zip(out[:3], ref)) and torch.equal(*stacks)
    assert torch.equal(counts, torch.cat(ref[:3])) and binding.dspark_get_device_status(out[3]) == 0
