"""Ended sequences whose table rows hold numbers that name no page (GPU)."""
import pytest
import torch

import sparse_attention_aware_b200 as sa

pytestmark = pytest.mark.gpu

DEVICE_FAULT = 5


def _plain(table, lens, new, stack, page, num_pages):
    """New (table, lens, stack) and the tokens' slots, one page at a time."""
    table, stack = [r[:] for r in table], stack[:]
    for b, a in enumerate(new):
        if a < 0:
            stack += [p for p in table[b][:-(-lens[b] // page)] if 0 <= p < num_pages]
    out, slots = [], []
    for b, a in enumerate(new):
        n = 0 if a < 0 else lens[b]
        for _ in range(max(a, 0)):
            if n % page == 0:
                table[b][n // page] = stack.pop()
            slots.append(table[b][n // page] * page + n % page)
            n += 1
        out.append(n)
    return table, out, stack, slots


def _run(dev, table, lens, new, stack, page, num_pages, cap, room):
    i32 = dict(dtype=torch.int32, device=dev)
    t, sl = torch.tensor(table, **i32), torch.tensor(lens, **i32)
    free = torch.full((room,), -55, **i32)
    free[:len(stack)] = torch.tensor(stack, **i32)
    pool = sa.PagePool(free, torch.tensor([len(stack)], **i32), num_pages, page)
    ws = sa.Workspace(dev)
    p = sa.plan_append(t, sl, torch.tensor(new, **i32), pool, cap, ws=ws)
    n = int(pool.free_count)
    return t.tolist(), sl.tolist(), free[:n].tolist(), p, ws.status()


# max_tokens of up to 4096, 32768 and more: a cluster of one CTA, of 8 and of 16
@pytest.mark.parametrize("cap", [64, 5000, 40000])
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_numbers_that_are_no_pages_stay_off_the_stack(cuda_dev, cap, seed):
    g = torch.Generator().manual_seed(seed)
    page, B, per = 16, 41, 40
    lens = torch.randint(0, 16 * 30, (B,), generator=g).tolist()
    new = torch.randint(0, 2, (B,), generator=g).tolist()
    for b in range(0, B, 3):
        new[b] = -1
    lens[0], lens[39] = 16 * 40, 16 * 33 + 1      # more pages than a warp has lanes
    num_pages = B * per
    perm = torch.randperm(num_pages, generator=g).tolist()
    table = [perm[b * per:(b + 1) * per] for b in range(B)]
    bad = [-1, num_pages, -2 ** 31, 2 ** 31 - 1, num_pages + 7]
    first = None
    for b in range(0, B, 6):                       # every other ended sequence
        held = -(-lens[b] // page)
        for i in torch.randperm(held, generator=g).tolist()[:1 + held // 4]:
            table[b][i] = bad[(b + i) % len(bad)]
            first = b
    if seed == 3:                                  # a row of nothing else
        table[0][:40] = [-1] * 40
    assert first is not None
    stack = [num_pages - 1 - i for i in range(5)]
    ref = _plain(table, lens, new, stack, page, num_pages)
    got = _run(cuda_dev, table, lens, new, stack, page, num_pages, cap, num_pages + 5)
    assert got[4][0] == DEVICE_FAULT and got[4][1][1] == 2 and not 0 <= got[4][1][2] < num_pages
    assert got[1] == ref[1] and got[2] == ref[2] and got[0] == ref[0]
    slots = got[3].slots.tolist()
    assert slots[:len(ref[3])] == ref[3] and set(slots[len(ref[3]):]) <= {-1}
    # later steps draw pages alone
    table, lens, stack = got[0], got[1], got[2]
    new = [17 if n < 16 * 30 else 0 for n in lens]
    if sum(new) <= cap and 2 * len(lens) <= len(stack):
        ref = _plain(table, lens, new, stack, page, num_pages)
        got = _run(cuda_dev, table, lens, new, stack, page, num_pages, cap, num_pages + 5)
        assert got[4][0] == 0 and got[0] == ref[0] and got[2] == ref[2] and got[3].slots.tolist()[:len(ref[3])] == ref[3]


@pytest.mark.parametrize("cap", [64, 5000, 40000])
@pytest.mark.parametrize("short", [0, 1])
def test_a_step_that_lacks_pages_without_them_changes_nothing(cuda_dev, cap, short):
    """An ended sequence of 4 entries, two of which are pages; a new one needs 3 or 4 with one free."""
    table = [[3, -1, 99, 5], [-9] * 4, [7, -9, -9, -9]]
    lens, new, stack = [64, 0, 16], [-1, 48 + 16 * short - 5, 0], [6]
    got = _run(cuda_dev, table, lens, new, stack, 16, 8, cap, 8)
    assert got[4][0] == DEVICE_FAULT and got[4][1][1] == 2
    if short:
        assert (got[0], got[1], got[2]) == (table, lens, stack)
        assert got[3].cu_tokens.tolist() == [0] * 4 and set(got[3].slots.tolist()) == {-1}
        assert set(got[3].positions.tolist()) == {0} and set(got[3].seq_ids.tolist()) == {-1}
    else:
        ref = _plain(table, lens, new, stack, 16, 8)
        assert (got[0], got[1], got[2]) == ref[:3] and got[3].slots.tolist()[:43] == ref[3]
