"""Prompt and chunk attention at calls that are allowed and unusual: offsets past
32 bits, pages that sequences share, one pool for K and V, pages of other
sizes, infinite scores, rows in front of the first sequence."""
import pytest
import torch

import prompt_ref as R
from medusa_tree_speculative_heads_b200 import api
from medusa_tree_speculative_heads_b200 import binding as B
from test_gpu_prompt import BF16, F32, INF, _gen, _ints, _paged, _rand, _rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,page,new", [(BF16, 16, 1), (BF16, 16, 40), (BF16, 24, 40), (F32, 16, 5)])
def test_pool_past_32_bits(dtype, page, new):
    """A pool of more than 2^31 elements whose last pages hold the sequence
    (K and V in one pool)."""
    g = _gen(41)
    Hq, Hkv, D, prefix = 8, 2, 128, 300
    need = -(-(prefix + new) // page)
    num = 2 ** 31 // (Hkv * page * D) + need + 3
    pool = torch.empty((num, Hkv, page, D), dtype=dtype, device="cuda")
    k = _rand((prefix + new, Hkv, D), g, dtype)
    ids = torch.arange(num - need, num, device="cuda").flip(0)
    at = torch.arange(prefix + new, device="cuda")
    pool[ids[at // page], :, at % page] = k
    q = _rand((new, Hq, D), g, dtype)
    out = api.chunk_attention_paged(q, pool, pool, ids.to(torch.int32)[None].contiguous(), _ints([0, new]),
                                    _ints([prefix]), want_lse=True)
    assert out["status"].item() == 0
    R.check(out["out"], out["lse"], dtype, D, R.attention(q, k, k, prefix))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_packed_rows_past_32_bits(dtype):
    """Row strides that put the last rows more than 2^31 elements in."""
    g = _gen(43)
    n, Hq, Hkv, D, stride = 40, 4, 2, 64, 2 ** 26
    base = torch.empty((n - 1) * stride + 4096, dtype=dtype, device="cuda")
    views = []
    for at, heads in ((0, Hq), (1024, Hkv), (2048, Hkv)):
        t = base[at:].as_strided((n, heads, D), (stride, D, 1))
        t.copy_(_rand((n, heads, D), g, dtype))
        views.append(t)
    q, k, v = views
    out = api.prompt_attention(q, k, v, _ints([0, n]), want_lse=True)
    assert out["status"].item() == 0
    R.check(out["out"], out["lse"], dtype, D, R.attention(q, k, v, 0))
    kp = torch.zeros((3, Hkv, 16, D), dtype=dtype, device="cuda")
    vp = torch.zeros_like(kp)
    slot = torch.arange(n, device="cuda") + 2
    assert api.kv_append_paged(k, v, slot, kp, vp)["status"].item() == 0
    assert torch.equal(kp[slot // 16, :, slot % 16], k) and torch.equal(vp[slot // 16, :, slot % 16], v)


@pytest.mark.parametrize("new", [[1, 1, 1], [2, 50, 3]])
def test_sequences_that_share_pages(new):
    """Three sequences over the same 128 cached tokens, each with rows of its
    own behind them."""
    g = _gen(47)
    Hq, Hkv, D, page, shared = 8, 2, 128, 16, 128
    own = [9, 40, 0]
    k, v = (_rand((shared + sum(own) + sum(new), Hkv, D), g, BF16) for _ in range(2))
    lens = [shared] + [o + n for o, n in zip(own, new)]
    kp, vp, parts = _paged(k, v, lens, page, g)
    rows = [torch.cat([parts[0, :shared // page], parts[b + 1]]) for b in range(3)]
    table = torch.stack(rows).contiguous()
    row, kr = _rows(new), _rows(lens)
    q = _rand((row[-1], Hq, D), g, BF16)
    out = api.chunk_attention_paged(q, kp, vp, table, _ints(row), _ints([shared + o for o in own]), max_new=max(new),
                                    want_lse=True)
    assert out["status"].item() == 0
    for b in range(3):
        at = slice(row[b], row[b + 1])
        kk, vv = (torch.cat([x[:shared], x[kr[b + 1]:kr[b + 2]]]) for x in (k, v))
        R.check(out["out"][at], out["lse"][at], BF16, D, R.attention(q[at], kk, vv, shared + own[b]), f"sequence {b}")


@pytest.mark.parametrize("new", [1, 33])
@pytest.mark.parametrize("page", [2, 40, 192, 256, 2048])
def test_page_sizes(page, new):
    g = _gen(page)
    Hq, Hkv, D, prefix = 4, 2, 64, [1000, 191]
    total = [p + new for p in prefix]
    k, v = (_rand((sum(total), Hkv, D), g, BF16) for _ in range(2))
    kp, vp, table = _paged(k, v, total, page, g)
    row, kr = _rows([new, new]), _rows(total)
    q = _rand((row[-1], Hq, D), g, BF16)
    out = api.chunk_attention_paged(q, kp, vp, table, _ints(row), _ints(prefix), max_new=new, want_lse=True)
    assert out["status"].item() == 0
    for b in range(2):
        at = slice(row[b], row[b + 1])
        R.check(out["out"][at], out["lse"][at], BF16, D,
                R.attention(q[at], k[kr[b]:kr[b + 1]], v[kr[b]:kr[b + 1]], prefix[b]), f"sequence {b}")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("paged", [False, True])
def test_infinite_scores(dtype, paged):
    """A key whose score is -inf weighs nothing; one whose score is +inf makes
    the rows that see it NaN (inf - inf in the formula) and no others."""
    g = _gen(53)
    Hq, Hkv, D, n, j = 8, 2, 128, 300, 140
    q, k, v = (_rand((n, h, D), g, dtype) for h in (Hq, Hkv, Hkv))
    q[:, :, 0] = q[:, :, 0].abs() + 0.5

    def run(k):
        if not paged:
            return api.prompt_attention(q, k, v, _ints([0, n]), want_lse=True)
        kp, vp, table = _paged(k, v, [n], 16, g)
        return api.chunk_attention_paged(q, kp, vp, table, _ints([0, n]), _ints([0]), want_lse=True)

    low = k.clone()
    low[j, :, 0] = -INF
    out = run(low)
    keep = [i for i in range(n) if i != j]
    R.check(out["out"][:j], out["lse"][:j], dtype, D, R.attention(q[:j], k[:j], v[:j], 0))
    R.check(out["out"][j:], out["lse"][j:], dtype, D, R.attention(q[j:], k[keep], v[keep], j - 1))
    high = k.clone()
    high[j, :, 0] = INF
    out = run(high)
    R.check(out["out"][:j], out["lse"][:j], dtype, D, R.attention(q[:j], k[:j], v[:j], 0))
    assert bool(torch.isnan(out["out"][j:]).all()) and not bool(torch.isfinite(out["lse"][j:]).any())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new", [1, 60])
def test_rows_in_front_of_the_first_sequence_are_left_alone(dtype, new):
    g = _gen(59)
    Hq, Hkv, D, page, prefix, first = 8, 2, 128, 16, 400, 5
    k, v = (_rand((prefix + new, Hkv, D), g, dtype) for _ in range(2))
    kp, vp, table = _paged(k, v, [prefix + new], page, g)
    q = _rand((first + new + 2, Hq, D), g, dtype)
    step = api.PromptStep(B=1, Hq=Hq, Hkv=Hkv, D=D, max_tokens=first + new + 2, dtype=dtype, page_size=page,
                          max_pages=table.shape[1], num_pages=kp.shape[0], max_new=new, max_prefix=prefix)
    step.out.fill_(7.0)
    step.chunk_attention(q, kp, vp, table, _ints([prefix]), row_start=_ints([first, first + new]))
    at = slice(first, first + new)
    R.check(step.out[at], None, dtype, D, R.attention(q[at], k, v, prefix))
    assert step.status.item() == 0
    assert bool((step.out[:first] == 7.0).all()) and bool((step.out[first + new:] == 7.0).all())


def test_broadcast_rows_are_refused():
    """An expanded tensor has rows 0 elements apart."""
    q, k = (torch.zeros((4, h, 64), dtype=BF16, device="cuda") for h in (4, 2))
    wide = torch.zeros((1, 2, 64), dtype=BF16, device="cuda").expand(4, 2, 64)
    with pytest.raises(B.MedusaError):
        api.prompt_attention(q, k, wide, _ints([0, 4]))
    with pytest.raises(B.MedusaError):
        api.kv_append_paged(wide, k, torch.arange(4, device="cuda"), *(torch.zeros((1, 2, 16, 64), dtype=BF16,
                                                                                  device="cuda"),) * 2)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,prefix", [([700], 0), ([2000, 3, 900], 0), ([64, 200], 3000), ([1, 1, 1], 3000)])
def test_expired_waits_end_every_call(D, lens, prefix):
    """With every wait giving up at once a call ends with the timeout reported,
    however often; its producers and consumers run at their own pace then."""
    g = _gen(61)
    Hq, Hkv, page, total = 8, 2, 16, [prefix + n for n in lens]
    k, v = (_rand((sum(total), Hkv, D), g, BF16) for _ in range(2))
    kp, vp, table = _paged(k, v, total, page, g)
    row, kr = _rows(lens), _rows(total)
    q = _rand((row[-1], Hq, D), g, BF16)

    def call():
        if prefix:
            return api.chunk_attention_paged(q, kp, vp, table, _ints(row), _ints([prefix] * len(lens)),
                                             max_new=max(lens), max_prefix=prefix)
        return api.prompt_attention(q, k, v, _ints(row))

    B.set_wait_limit(1)
    try:
        bad = [call() for _ in range(20)]
        torch.cuda.synchronize()
    finally:
        B.set_wait_limit(0)
    assert all(x["status"].item() & B.STATUS_TIMEOUT for x in bad)
    good = call()
    assert good["status"].item() == 0
    for b, n in enumerate(lens):
        at = slice(row[b], row[b + 1])
        R.check(good["out"][at], None, BF16, D, R.attention(q[at], k[kr[b]:kr[b + 1]], v[kr[b]:kr[b + 1]], prefix))


@pytest.mark.parametrize("dtype,Hq,Hkv,D,lens,prefix", [
    (F32, 8, 2, 128, [1, 1], 840),              # CUDA cores, split keys
    (BF16, 8, 2, 128, [64], 4000),              # two tiles, split keys
    (BF16, 32, 8, 128, [256] * 20, 0),          # a grid whose tiles are found first
    (BF16, 8, 2, 64, [1, 2, 1], 2500)])         # few rows
def test_replays_of_calls_of_two_launches(dtype, Hq, Hkv, D, lens, prefix):
    """Captured twice in a row over the same buffers, replayed with other values
    and with shorter sequences: bit for bit what the calls give by themselves."""
    g = _gen(67)
    page, row = 16, _rows(lens)
    total = [prefix + n for n in lens]
    k, v = (_rand((sum(total), Hkv, D), g, dtype) for _ in range(2))
    kp, vp, table = _paged(k, v, total, page, g)
    qs = [_rand((row[-1], Hq, D), g, dtype) for _ in range(2)]
    q, rs, pre = qs[0].clone(), _ints(row), _ints([prefix] * len(lens))
    step = api.PromptStep(B=len(lens), Hq=Hq, Hkv=Hkv, D=D, max_tokens=row[-1], dtype=dtype, page_size=page,
                          max_pages=table.shape[1], num_pages=kp.shape[0], max_new=max(lens), max_prefix=prefix or 1)

    def call():
        if prefix:
            step.chunk_attention(q, kp, vp, table, pre, row_start=rs)
        else:
            step.prompt_attention(q, k, v, row_start=rs)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        first = step.out.clone()
        call()
    for values, shorter in ((qs[0], 0), (qs[1], 0), (qs[1], 1)):
        q.copy_(values)
        rs.copy_(_ints([min(r, row[-1] - shorter) for r in row]))
        step.out.zero_()
        call()
        want = step.out.clone()
        step.out.zero_()
        first.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(step.out, want) and torch.equal(first, want)
        assert step.status.item() == 0
    for b, n in enumerate(lens[:2] if len(lens) > 2 else lens[:1]):
        at, keys = slice(row[b], row[b + 1]), slice(_rows(total)[b], _rows(total)[b + 1])
        ref = R.attention(q[at], k[keys], v[keys], prefix)
        if row[b + 1] <= row[-1] - 1:
            R.check(step.out[at], None, dtype, D, ref)
