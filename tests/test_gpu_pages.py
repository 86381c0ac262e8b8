"""Page plan and K/V append against plain Python and torch indexing; every
value is moved whole, so everything is compared bit for bit."""
import random

import pytest
import torch

import prompt_ref as R
from medusa_tree_speculative_heads_b200 import api
from medusa_tree_speculative_heads_b200 import binding as B

pytestmark = pytest.mark.gpu


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _state(rng, n, page, max_len, extra, max_pages=0):
    """A pool in use: n sequences with random cached lengths, their pages and
    a few more than needed, the rest on the stack in random order."""
    prefix = [rng.randint(0, max_len) for _ in range(n)]
    owned = [-(-p // page) + (rng.randint(0, 2) if rng.random() < 0.3 else 0) for p in prefix]
    mp = max(max(owned) + -(-max_len // page) + 3, max_pages)
    num = sum(owned) + extra
    perm = list(range(num))
    rng.shuffle(perm)
    table, k = [], 0
    for o in owned:
        table.append(perm[k:k + o] + [-1] * (mp - o))
        k += o
    return prefix, owned, table, perm[k:], num


def _run(prefix, new, owned, table, stack, num, page, room, max_tokens):
    free = _ints(stack + [-7] * (num - len(stack)))
    tb = _ints(table)
    out = api.kv_page_plan(_ints(prefix), _ints(new), tb, _ints(owned), free, _ints([len(stack)]), page, max_tokens,
                           room=room)
    torch.cuda.synchronize()
    return out, tb.cpu().tolist(), free.cpu().tolist()


def _check(got, tb, free, want, stack_before, page):
    row, slots, owned, table, stack, count, _ = want
    assert got["row_start"].tolist() == row
    assert got["slot_map"].tolist() == slots
    assert got["owned"].tolist() == owned
    assert tb == table
    assert got["free_count"].item() == count
    assert free[:len(stack)] == stack
    assert all(x == -7 for x in free[max(len(stack), stack_before):])


@pytest.mark.parametrize("n,page,max_len,room,top", [
    (1, 16, 40, 0, 1), (1, 1, 5, 3, 4), (3, 16, 0, 0, 0), (7, 8, 100, 5, 33), (64, 16, 300, 5, 1),
    (65, 64, 700, 0, 200), (300, 16, 200, 2, 90), (1025, 5, 30, 1, 12), (2100, 16, 64, 5, 3)])
def test_plan_matches_the_sequential_form(n, page, max_len, room, top):
    for seed in range(3):
        rng = random.Random(1000 * n + seed)
        prefix, owned, table, stack, num = _state(rng, n, page, max_len, 4000)
        new = [rng.choice([-1, 0, 1, rng.randint(0, top), rng.randint(0, top)]) for _ in range(n)]
        max_tokens = sum(max(x, 0) for x in new) + rng.randint(1, 40)
        want = R.plan(prefix, new, owned, table, stack, room, page, max_tokens)
        got, tb, free = _run(prefix, new, owned, table, stack, num, page, room, max_tokens)
        assert not want[-1]
        assert got["status"].item() == 0
        _check(got, tb, free, want, len(stack), page)


def test_plan_refuses_what_does_not_fit_and_serves_the_rest():
    # stack of 5: sequence 0 takes 2, 1 wants 4 (refused), 2 needs none, 3 wants 1 (behind the refused one), 4 ends
    prefix, new, page = [16, 0, 10, 0, 33], [32, 64, 6, 1, -1], 16
    owned, table = [1, 0, 1, 0, 3], [[9, -1, -1, -1], [-1] * 4, [8, -1, -1, -1], [-1] * 4, [5, 6, 7, -1]]
    stack = [0, 1]
    got, tb, free = _run(prefix, new, owned, table, stack, 12, page, 0, 110)
    want = R.plan(prefix, new, owned, table, stack, 0, page, 110)
    assert want[-1] == {1, 3}
    assert got["status"].item() == B.STATUS_CACHE_OVERFLOW
    _check(got, tb, free, want, len(stack), page)
    # a table row too short for the request
    got, tb, free = _run([0, 0], [65, 3], [0, 0], [[-1] * 4, [-1] * 4], [3, 2, 1, 0], 4, page, 0, 70)
    assert got["status"].item() == B.STATUS_CACHE_OVERFLOW
    assert got["owned"].tolist() == [0, 1] and tb[1][0] == 0 and got["slot_map"].tolist()[65:68] == [0, 1, 2]
    assert got["slot_map"].tolist()[:65] == [-1] * 65


def test_plan_serves_what_takes_nothing_behind_refused_growth_past_32_bits():
    """Five sequences that would take 2^29 - 1 pages each are refused; the
    sixth needs no page and gets its slot."""
    mp = 2 ** 29
    table = torch.empty((6, mp), dtype=torch.int32, device="cuda")
    table[5, 0] = 3
    out = api.kv_page_plan(_ints([mp - 1] * 5 + [0]), _ints([0] * 5 + [1]), table, _ints([0] * 5 + [1]),
                           _ints([0, 1, 2, 4]), _ints([4]), 1, 2)
    assert out["status"].item() == B.STATUS_CACHE_OVERFLOW
    assert out["slot_map"].tolist() == [3, -1] and out["row_start"].tolist() == [0] * 6 + [1]
    assert out["owned"].tolist() == [0] * 5 + [1] and out["free_count"].item() == 4


def test_plan_reports_values_out_of_range():
    def status(prefix=(0,), new=(1,), owned=(0,), stack=(1, 0), table=((-1, -1),), max_tokens=8):
        return _run(list(prefix), list(new), list(owned), [list(r) for r in table], list(stack), 4, 16, 0, max_tokens)
    assert status(new=(-2,))[0]["status"].item() == B.STATUS_BAD_LENGTH
    # (three owned pages clamped to the table's two, whose entries are no pages)
    assert status(owned=(3,))[0]["status"].item() == B.STATUS_BAD_LENGTH | B.STATUS_BAD_PAGE
    assert status(prefix=(-1,))[0]["status"].item() == B.STATUS_BAD_PREFIX
    got, _, _ = status(new=(9,))
    assert got["status"].item() == B.STATUS_BAD_LENGTH and got["row_start"].tolist() == [0, 8]
    got, tb, _ = status(stack=(1, 77))
    assert got["status"].item() == B.STATUS_BAD_PAGE and tb[0][0] == -1 and got["slot_map"].tolist() == [-1] * 8
    # pages given back twice cannot overrun the stack
    got, _, free = status(prefix=(32, 32), new=(-1, -1), owned=(2, 2), table=((0, 1), (2, 3)), stack=(1, 0))
    assert got["status"].item() == B.STATUS_BAD_PAGE and got["free_count"].item() == 4 and free[2:] == [0, 1]


def test_plan_in_place_step_by_step():
    """PromptStep.plan updates the pool's state in place: a pool run through
    random arrivals, growth and ends never hands a page out twice."""
    rng = random.Random(4)
    n, page, num, mp = 9, 16, 60, 12
    step = api.PromptStep(B=n, Hq=4, Hkv=4, D=64, max_tokens=600, dtype=torch.bfloat16, page_size=page, max_pages=mp,
                          num_pages=num, room=3)
    table, owned = torch.full((n, mp), -1, dtype=torch.int32, device="cuda"), _ints([0] * n)
    free, count = _ints(list(range(num))), _ints([num])
    prefix = [0] * n
    for it in range(40):
        new = [rng.choice([-1, 0, 1, rng.randint(1, 40)]) if prefix[b] < 120 else -1 for b in range(n)]
        before = owned.tolist(), table.tolist(), free.tolist()[:count.item()]
        want = R.plan(prefix, new, *before[:1], before[1], before[2], 3, page, 600)
        step.plan(_ints(prefix), _ints(new), table, owned, free, count)
        torch.cuda.synchronize()
        assert owned.tolist() == want[2] and table.tolist() == want[3] and count.item() == want[5]
        assert step.slot_map.tolist() == want[1] and step.row_start.tolist() == want[0]
        for b in range(n):
            if new[b] == -1:
                prefix[b] = 0
            elif b not in want[6]:
                prefix[b] += new[b]
        held = [p for b in range(n) for p in table.tolist()[b][:owned.tolist()[b]]] + free.tolist()[:count.item()]
        assert sorted(held) == list(range(num))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,Hkv,D,page,fused", [
    (1, 1, 64, 16, False), (3, 8, 128, 16, True), (77, 3, 64, 5, True), (1030, 8, 128, 64, True),
    (513, 2, 128, 1, False), (40, 5, 64, 24, True)])
def test_append_matches_indexing(dtype, N, Hkv, D, page, fused):
    g = torch.Generator(device="cuda").manual_seed(N)
    num = -(-N // page) + 4
    rows = torch.randn((N, 6 * Hkv, D), generator=g, device="cuda").to(dtype)
    k, v = (rows[:, 4 * Hkv:5 * Hkv], rows[:, 5 * Hkv:]) if fused else (rows[:, :Hkv].contiguous(),
                                                                       rows[:, Hkv:2 * Hkv].contiguous())
    kp, vp = (torch.randn((num, Hkv, page, D), generator=g, device="cuda").to(dtype) for _ in range(2))
    slot = torch.randperm(num * page, generator=g, device="cuda")[:N]
    slot[::7] = -1
    wk, wv = kp.clone(), vp.clone()
    at = (slot >= 0).nonzero()[:, 0]
    wk[slot[at] // page, :, slot[at] % page] = k[at]
    wv[slot[at] // page, :, slot[at] % page] = v[at]
    out = api.kv_append_paged(k, v, slot, kp, vp)
    torch.cuda.synchronize()
    assert out["status"].item() == 0
    assert torch.equal(kp, wk) and torch.equal(vp, wv)
    # a slot outside the pool is skipped and reported
    bad = slot.clone()
    bad[0] = num * page
    if N > 2:
        bad[1], bad[2] = -2, 1 << 40
    keep = (bad >= 0) & (bad < num * page)
    kp2, vp2 = torch.zeros_like(kp), torch.zeros_like(vp)
    out = api.kv_append_paged(k, v, bad, kp2, vp2)
    torch.cuda.synchronize()
    assert out["status"].item() == B.STATUS_BAD_PAGE
    wk = torch.zeros_like(kp)
    at = keep.nonzero()[:, 0]
    wk[bad[at] // page, :, bad[at] % page] = k[at]
    assert torch.equal(kp2, wk)


def test_append_slots_past_32_bits():
    """A pool of more than 2^31 elements (4.5 GB): its last pages are reached."""
    num, Hkv, page, D = 2 ** 31 // (8 * 16 * 128) + 9, 8, 16, 128
    kp = torch.zeros((num, Hkv, page, D), dtype=torch.bfloat16, device="cuda")
    k = torch.randn((5, Hkv, D), device="cuda").to(torch.bfloat16)
    slot = torch.tensor([num * page - 1, 0, (num - 3) * page + 5, -1, 2 ** 31 // (8 * 128)], device="cuda")
    vp = torch.zeros_like(kp)
    out = api.kv_append_paged(k, k, slot, kp, vp)
    torch.cuda.synchronize()
    assert out["status"].item() == 0
    for t, s in enumerate(slot.tolist()):
        if s >= 0:
            assert torch.equal(kp[s // page, :, s % page], k[t]) and torch.equal(vp[s // page, :, s % page], k[t])
    assert int((kp != 0).sum()) == int((k[[0, 1, 2, 4]] != 0).sum())


def test_append_of_no_rows():
    kp = torch.zeros((2, 2, 8, 64), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    out = api.kv_append_paged(k, k, torch.zeros(0, dtype=torch.int64, device="cuda"), kp, kp.clone())
    assert out["status"].item() == 0


@pytest.mark.parametrize("room", [0, 40])
def test_plan_takes_lengths_below_minus_one_as_zero(room):
    """Reported, and otherwise planned like a sequence without new tokens: it
    keeps its pages and gets those that its prefix and the room need."""
    prefix, owned, stack = [20, 16, 5, 40, 0], [1, 1, 0, 3, 2], [0, 1, 2, 3, 9, 10, 11, 12, 13, 14]
    table = [[4] + [-1] * 5, [5] + [-1] * 5, [-1] * 6, [6, 7, 8] + [-1] * 3, [15, 16] + [-1] * 4]
    new, meant = [-2, 1, -7, -2 ** 31, -1], [0, 1, 0, 0, -1]
    want = R.plan(prefix, meant, owned, table, stack, room, 16, 5)
    got, tb, free = _run(prefix, new, owned, table, stack, 17, 16, room, 5)
    assert not want[-1]
    assert got["status"].item() == B.STATUS_BAD_LENGTH
    _check(got, tb, free, want, len(stack), 16)
    # where it does not fit, or its prefix is out of range, that is reported too
    got, tb, _ = _run([20], [-2], [0], [[-1] * 2], [0], 4, 16, room, 5)
    assert got["status"].item() == B.STATUS_BAD_LENGTH | B.STATUS_CACHE_OVERFLOW
    assert got["owned"].tolist() == [0] and tb == [[-1] * 2] and got["free_count"].item() == 1
    got, _, _ = _run([-3], [-2], [0], [[-1] * 2], [0], 4, 16, room, 5)
    assert got["status"].item() == B.STATUS_BAD_LENGTH | B.STATUS_BAD_PREFIX
