"""The prompt-side operators as they are used: together, over several steps,
beside the tree step on the same cache, captured in a graph, with many
sequences, and with their waits cut short."""
import numpy as np
import pytest
import torch

import oracle
import prompt_ref as R
from helpers import assert_float_parity
from medusa_tree_speculative_heads_b200 import api
from medusa_tree_speculative_heads_b200 import binding as B
from medusa_tree_speculative_heads_b200 import inputs as I
from medusa_tree_speculative_heads_b200.binding import Tree

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rand(shape, g, dtype=BF16):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _rows(lens):
    r = [0]
    for n in lens:
        r.append(r[-1] + n)
    return r


class _History:
    """What every sequence's cache should hold, kept on the side."""

    def __init__(self, n, layers):
        self.kv = [[[] for _ in range(n)] for _ in range(layers)]

    def add(self, layer, b, k, v):
        self.kv[layer][b].append((k.clone(), v.clone()))

    def get(self, layer, b):
        ks, vs = zip(*self.kv[layer][b])
        return torch.cat(ks), torch.cat(vs)


@pytest.mark.parametrize("dtype,page", [(BF16, 16), (BF16, 64), (torch.float32, 16)])
def test_prompts_chunks_decoding_and_a_tree_step_on_one_cache(dtype, page):
    """Three requests: prompts in chunks of different lengths, one ends and
    another takes its place, single tokens, then a tree step's attention and
    commit through the same block table; every attention against the 64-bit
    form over the whole history, the pages against what was appended."""
    g = _gen(1)
    n, layers, Hq, Hkv, D, num, mp, room = 3, 2, 8, 2, 128, 60, 20, 5
    pools = [[torch.full((num, Hkv, page, D), float("nan"), dtype=dtype, device="cuda") for _ in range(2)]
             for _ in range(layers)]
    table, owned = torch.full((n, mp), -1, dtype=torch.int32, device="cuda"), _ints([0] * n)
    free, count = _ints(list(range(num))[::-1]), _ints([num])
    step = api.PromptStep(B=n, Hq=Hq, Hkv=Hkv, D=D, max_tokens=300, dtype=dtype, page_size=page, max_pages=mp,
                          num_pages=num, room=room, want_lse=True)
    hist, prefix = _History(n, layers), [0, 0, 0]
    for it, new in enumerate([[37, 0, 150], [100, 70, 1], [1, 1, 1], [-1, 1, 65], [90, 1, 1], [1, 1, 1]]):
        if new[0] == -1:
            for layer in hist.kv:
                layer[0] = []
            prefix[0] = 0
        step.plan(_ints(prefix), _ints(new), table, owned, free, count)
        new = [max(x, 0) for x in new]
        row = _rows(new)
        assert step.row_start.tolist() == row
        for layer in range(layers):
            fused = _rand((300, Hq + 2 * Hkv, D), g, dtype)
            q, k, v = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
            step.append(k, v, *pools[layer])
            step.chunk_attention(q, *pools[layer], table, _ints(prefix))
            for b in range(n):
                at = slice(row[b], row[b + 1])
                if new[b]:
                    hist.add(layer, b, k[at], v[at])
                    ref = R.attention(q[at], *hist.get(layer, b), prefix[b])
                    R.check(step.out[at], step.lse[at], dtype, D, ref, f"step {it} layer {layer} sequence {b}")
        assert step.status.item() == 0
        prefix = [p + x for p, x in zip(prefix, new)]
    # a tree step: its commit's rows are covered by `room`
    parents = I.product_tree_parents((2, 2))
    tree, T = Tree(parents), len(parents)
    q = _rand((n, T, Hq, D), g, dtype)
    kt, vt = _rand((n, T, Hkv, D), g, dtype), _rand((n, T, Hkv, D), g, dtype)
    kp, vp = pools[0]
    got = api.tree_attention_paged(q, kt, vt, kp, vp, table, _ints(prefix), tree, want_lse=True)
    assert got["status"].item() == 0
    S = max(prefix)
    kc, vc = (torch.zeros((n, Hkv, S, D), dtype=dtype) for _ in range(2))
    for b in range(n):
        k, v = hist.get(0, b)
        kc[b, :, :prefix[b]], vc[b, :, :prefix[b]] = k.transpose(0, 1).cpu(), v.transpose(0, 1).cpu()
    ref_o, _ = oracle.tree_attention(q.cpu(), kt.cpu(), vt.cpu(), kc, vc, torch.tensor(prefix, dtype=torch.int32),
                                     parents)
    assert_float_parity(got["out"].float().cpu().reshape(-1, D), ref_o, dtype, "tree attention")
    path = _ints([[0, 1, 3], [0, 2, 5], [0, 2, 6]])
    out = api.kv_commit_paged(kp, vp, kt, vt, table, path, _ints([3, 2, 1]), _ints(prefix))
    assert out["status"].item() == 0
    for b, ln in enumerate((3, 2, 1)):
        ids = path[b, :ln].long()
        hist.add(0, b, kt[b, ids], vt[b, ids])
        prefix[b] += ln
    # and the next single tokens see what it committed
    step.plan(_ints(prefix), _ints([1, 1, 1]), table, owned, free, count)
    q1, k1, v1 = _rand((3, Hq, D), g, dtype), _rand((3, Hkv, D), g, dtype), _rand((3, Hkv, D), g, dtype)
    step.append(k1, v1, kp, vp)
    step.chunk_attention(q1, kp, vp, table, _ints(prefix))
    for b in range(n):
        hist.add(0, b, k1[b:b + 1], v1[b:b + 1])
        R.check(step.out[b:b + 1], step.lse[b:b + 1], dtype, D,
                R.attention(q1[b:b + 1], *hist.get(0, b), prefix[b]), f"after the tree step, sequence {b}")
        k, v = hist.get(0, b)
        at = torch.arange(k.shape[0], device="cuda")
        pg = table[b].long()[at // page]
        assert torch.equal(kp[pg, :, at % page], k) and torch.equal(vp[pg, :, at % page], v)
    assert step.status.item() == 0


def test_whole_prompts_equal_chunks_over_an_empty_prefix():
    g = _gen(2)
    lens, Hq, Hkv, D, page = [300, 1, 129], 8, 2, 128, 16
    row = _rows(lens)
    q, k, v = _rand((430, Hq, D), g), _rand((430, Hkv, D), g), _rand((430, Hkv, D), g)
    whole = api.prompt_attention(q, k, v, _ints(row), want_lse=True)
    num = 32
    table = torch.full((3, 19), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(num, generator=g, device="cuda").to(torch.int32)
    plan = api.kv_page_plan(_ints([0] * 3), _ints(lens), table, _ints([0] * 3), free, _ints([num]), page, 430)
    kp, vp = (torch.full((num, Hkv, page, D), float("nan"), dtype=BF16, device="cuda") for _ in range(2))
    api.kv_append_paged(k, v, plan["slot_map"], kp, vp)
    chunks = api.chunk_attention_paged(q, kp, vp, table, plan["row_start"], _ints([0] * 3), want_lse=True)
    assert chunks["status"].item() == 0 and plan["status"].item() == 0
    # the same chunks of keys in the same order: the same bits
    assert torch.equal(whole["out"], chunks["out"]) and torch.equal(whole["lse"], chunks["lse"])


def test_a_contiguous_cache_is_a_pool_of_one_page_per_sequence():
    g = _gen(3)
    n, Hq, Hkv, D, S = 3, 4, 4, 64, 512
    kc, vc = _rand((n, Hkv, S, D), g), _rand((n, Hkv, S, D), g)
    prefix, new = [500, 0, 77], [12, 300, 1]
    row = _rows(new)
    q = _rand((row[-1], Hq, D), g)
    out = api.chunk_attention_paged(q, kc, vc, _ints([[0], [1], [2]]), _ints(row), _ints(prefix), want_lse=True)
    assert out["status"].item() == 0
    for b in range(n):
        at, m = slice(row[b], row[b + 1]), prefix[b] + new[b]
        R.check(out["out"][at], out["lse"][at], BF16, D,
                R.attention(q[at], kc[b, :, :m].transpose(0, 1), vc[b, :, :m].transpose(0, 1), prefix[b]))


@pytest.mark.parametrize("max_new", [4, 64])   # few rows; the two-tile kernel
def test_captured_and_replayed_with_other_lengths(max_new):
    """plan, append and attention captured once, replayed with fewer tokens,
    other lengths and an ended sequence; rows behind the last sequence keep
    what they held."""
    g = _gen(4)
    n, Hq, Hkv, D, page, num, mp, N = 4, 8, 2, 128, 16, 100, 16, 4 * max_new
    kp, vp = (_rand((num, Hkv, page, D), g) for _ in range(2))
    state = dict(prefix=_ints([0] * n), new=_ints([0] * n),
                 table=torch.full((n, mp), -1, dtype=torch.int32, device="cuda"), owned=_ints([0] * n),
                 free=_ints(list(range(num))), count=_ints([num]))
    step = api.PromptStep(B=n, Hq=Hq, Hkv=Hkv, D=D, max_tokens=N, dtype=BF16, page_size=page, max_pages=mp,
                          num_pages=num, max_new=max_new, want_lse=True)
    q, k, v = _rand((N, Hq, D), g), _rand((N, Hkv, D), g), _rand((N, Hkv, D), g)

    def run():
        step.plan(state["prefix"], state["new"], state["table"], state["owned"], state["free"], state["count"])
        step.append(k, v, kp, vp)
        step.chunk_attention(q, kp, vp, state["table"], state["prefix"])

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        run()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    hist, prefix = _History(n, 1), [0] * n
    for it in range(6):
        new = [[max_new, 0, 1, 3], [1, max_new, 1, 1], [1, 1, -1, 1], [2, 3, max_new, 1], [1, 1, 1, -1],
               [0, 0, 0, 0]][it]
        for b in range(n):
            if new[b] == -1:
                hist.kv[0][b], prefix[b] = [], 0
        for t in (q, k, v):
            t.copy_(_rand(t.shape, g))
        state["prefix"].copy_(_ints(prefix))
        state["new"].copy_(_ints(new))
        step.out.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        assert step.status.item() == 0
        row = _rows([max(x, 0) for x in new])
        for b in range(n):
            at = slice(row[b], row[b + 1])
            if row[b + 1] > row[b]:
                hist.add(0, b, k[at], v[at])
                R.check(step.out[at], step.lse[at], BF16, D, R.attention(q[at], *hist.get(0, b), prefix[b]),
                        f"replay {it} sequence {b}")
                prefix[b] += row[b + 1] - row[b]
        assert bool((step.out[row[-1]:] == 5.0).all())


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
@pytest.mark.parametrize("top", [1, 90])
def test_many_sequences_over_a_paged_cache(dtype, top):
    """More sequences than a warp has lanes: 100 of lengths 0 to 700, some of
    them without a new token."""
    g = _gen(5)
    n, Hq, Hkv, D, page = 100, 4, 2, 64, 16
    r = np.random.default_rng(6)
    prefix = [int(x) for x in r.integers(0, 700, n)]
    new = [int(x) if i % 7 else 0 for i, x in enumerate(r.integers(1, top + 1, n))]
    need = [-(-(p + m) // page) for p, m in zip(prefix, new)]
    num = sum(need) + 1
    perm = torch.randperm(num, generator=g, device="cuda").tolist()
    table = torch.full((n, max(need)), -1, dtype=torch.int32)
    at = 0
    for b in range(n):
        table[b, :need[b]] = torch.tensor(perm[at:at + need[b]])
        at += need[b]
    kp, vp = (_rand((num, Hkv, page, D), g, dtype) for _ in range(2))
    row = _rows(new)
    q = _rand((row[-1], Hq, D), g, dtype)
    out = api.chunk_attention_paged(q, kp, vp, table.cuda(), _ints(row), _ints(prefix), max_new=top, want_lse=True)
    assert out["status"].item() == 0
    for b in list(range(0, n, 9)) + [n - 1]:
        m = prefix[b] + new[b]
        i = torch.arange(m, device="cuda")
        pg = table[b].cuda().long()[i // page]
        s = slice(row[b], row[b + 1])
        R.check(out["out"][s], out["lse"][s], dtype, D,
                R.attention(q[s], kp[pg, :, i % page], vp[pg, :, i % page], prefix[b]), f"sequence {b}")


def test_no_tokens_at_all():
    step = api.PromptStep(B=2, Hq=4, Hkv=2, D=64, max_tokens=8, dtype=BF16, page_size=16, max_pages=2, num_pages=4)
    kp = torch.zeros((4, 2, 16, 64), dtype=BF16, device="cuda")
    table, z = torch.full((2, 2), -1, dtype=torch.int32, device="cuda"), _ints([0, 0])
    step.plan(z, z, table, z.clone(), _ints([0, 1, 2, 3]), _ints([4]))
    step.out.fill_(3.0)
    q, k = torch.zeros((8, 4, 64), dtype=BF16, device="cuda"), torch.zeros((8, 2, 64), dtype=BF16, device="cuda")
    step.append(k, k, kp, kp.clone())
    step.chunk_attention(q, kp, kp, table, z)
    step.prompt_attention(q, k, k)
    step.chunk_attention(q[:0], kp, kp, table, z)
    step.prompt_attention(q[:0], k[:0], k[:0])
    torch.cuda.synchronize()
    assert step.status.item() == 0 and bool((step.out == 3.0).all())


@pytest.mark.parametrize("new,prefix", [(700, 0), (64, 3000), (1, 3000)])
def test_wait_limit_times_out_then_recovers(new, prefix):
    """With every wait giving up at once the calls return with the timeout
    reported; the next calls are right again."""
    g = _gen(7)
    Hq, Hkv, D, page = 8, 2, 128, 64
    m = prefix + new
    num = -(-m // page)
    kp, vp = (_rand((num, Hkv, page, D), g) for _ in range(2))
    q, table = _rand((new, Hq, D), g), torch.arange(num, dtype=torch.int32, device="cuda")[None]
    rows = kp.transpose(1, 2).reshape(-1, Hkv, D)[:m], vp.transpose(1, 2).reshape(-1, Hkv, D)[:m]

    def call():
        if prefix:
            return api.chunk_attention_paged(q, kp, vp, table, _ints([0, new]), _ints([prefix]), max_new=new,
                                             max_prefix=prefix, want_lse=True)
        return api.prompt_attention(q, *rows, _ints([0, new]), want_lse=True)

    B.set_wait_limit(1)
    try:
        bad = call()
        torch.cuda.synchronize()
    finally:
        B.set_wait_limit(0)
    assert bad["status"].item() & B.STATUS_TIMEOUT
    good = call()
    assert good["status"].item() == 0
    R.check(good["out"], good["lse"], BF16, D, R.attention(q, *rows, prefix))
