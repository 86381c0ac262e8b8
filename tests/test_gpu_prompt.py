"""Prompt and chunk attention against the 64-bit plain form, at the lengths,
head layouts, page sizes and values where they can go wrong."""
import pytest
import torch

import prompt_ref as R
from medusa_tree_speculative_heads_b200 import api
from medusa_tree_speculative_heads_b200 import binding as B

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _rows(lens):
    r = [0]
    for n in lens:
        r.append(r[-1] + n)
    return r


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rand(shape, g, dtype):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _paged(k, v, lens, page, g, fill=NAN, extra=2):
    """Packed K/V [sum(lens),Hkv,D] laid into pages in random order; every
    slot that holds no token is ``fill``.  Returns pools and the table."""
    need = [-(-n // page) for n in lens]
    num, mp = sum(need) + extra, max(max(need), 1) + 1
    perm = torch.randperm(num, generator=g, device="cuda").tolist()
    _, Hkv, D = k.shape
    kp, vp = (torch.full((num, Hkv, page, D), fill, dtype=k.dtype, device="cuda") for _ in range(2))
    table = torch.full((len(lens), mp), -1, dtype=torch.int32)
    used, r0 = 0, 0
    for b, n in enumerate(lens):
        ids = perm[used:used + need[b]]
        used += need[b]
        table[b, :need[b]] = torch.tensor(ids, dtype=torch.int32)
        at = torch.arange(n, device="cuda")
        pg = torch.tensor(ids + [0], device="cuda")[at // page]
        kp[pg, :, at % page] = k[r0:r0 + n]
        vp[pg, :, at % page] = v[r0:r0 + n]
        r0 += n
    return kp, vp, table.cuda()


LAYOUTS = [  # Hq, Hkv, D
    (4, 4, 64), (8, 2, 128), (6, 2, 64), (5, 1, 128), (14, 2, 128), (32, 8, 128), (64, 1, 128), (16, 2, 64)]
LENS = [[1], [0, 5, 0, 1], [127, 128, 129], [1, 2, 300, 0, 64, 65], [513, 31]]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Hq,Hkv,D", LAYOUTS)
@pytest.mark.parametrize("lens", LENS)
def test_prompt_parity(dtype, Hq, Hkv, D, lens):
    g = _gen(sum(lens) + Hq)
    row = _rows(lens)
    N = row[-1] + 3  # rows of no sequence behind the last one
    fused = _rand((N, Hq + 2 * Hkv, D), g, dtype)
    q, k, v = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
    fused[row[-1]:] = NAN
    step = api.PromptStep(B=len(lens), Hq=Hq, Hkv=Hkv, D=D, max_tokens=N, dtype=dtype, want_lse=True)
    step.out.fill_(7.0)
    step.lse.fill_(7.0)
    step.prompt_attention(q, k, v, row_start=_ints(row))
    torch.cuda.synchronize()
    assert step.status.item() == 0
    for a, b in zip(row, row[1:]):
        R.check(step.out[a:b], step.lse[a:b], dtype, D, R.attention(q[a:b], k[a:b], v[a:b], 0), f"rows {a}..{b}")
    assert bool((step.out[row[-1]:] == 7.0).all()) and bool((step.lse[row[-1]:] == 7.0).all())


@pytest.mark.parametrize("dtype,Hq,Hkv,D,lens", [
    (BF16, 32, 8, 128, [2048]), (BF16, 4, 4, 128, [1500, 1, 700]), (BF16, 8, 2, 64, [3000, 1000]),
    (F32, 4, 2, 64, [900])])
def test_prompt_parity_long(dtype, Hq, Hkv, D, lens):
    g = _gen(3)
    row = _rows(lens)
    q, k, v = (_rand((row[-1], h, D), g, dtype) for h in (Hq, Hkv, Hkv))
    out = api.prompt_attention(q, k, v, _ints(row), max_len=max(lens), want_lse=True)
    assert out["status"].item() == 0
    for a, b in zip(row, row[1:]):
        R.check(out["out"][a:b], out["lse"][a:b], dtype, D, R.attention(q[a:b], k[a:b], v[a:b], 0))


CHUNKS = [  # page, prefix lengths, new lengths
    (16, [0], [1]), (16, [700, 0, 1, 333], [1, 1, 1, 1]), (64, [64, 999, 130], [5, 0, 70]),
    (8, [300, 47, 0], [129, 1, 17]), (128, [900, 511], [64, 2]), (32, [260, 33, 0, 5], [3, 3, 3, 3]),
    (24, [500, 73], [40, 1]), (5, [64, 9], [1, 30]), (1, [3, 129], [2, 1])]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 4, 64), (8, 2, 128), (6, 2, 128), (32, 8, 128), (14, 2, 64)])
@pytest.mark.parametrize("page,prefix,new", CHUNKS)
def test_chunk_parity(dtype, Hq, Hkv, D, page, prefix, new):
    g = _gen(sum(prefix) + page)
    total = [p + n for p, n in zip(prefix, new)]
    kr, row = _rows(total), _rows(new)
    k, v = (_rand((kr[-1], Hkv, D), g, dtype) for _ in range(2))
    kp, vp, table = _paged(k, v, total, page, g)
    N = row[-1] + 2
    q = _rand((N, Hq, D), g, dtype)
    step = api.PromptStep(B=len(new), Hq=Hq, Hkv=Hkv, D=D, max_tokens=N, dtype=dtype, page_size=page,
                          max_pages=table.shape[1], num_pages=kp.shape[0], max_new=max(new), max_prefix=max(prefix),
                          want_lse=True)
    step.out.fill_(7.0)
    step.chunk_attention(q, kp, vp, table, _ints(prefix), row_start=_ints(row))
    torch.cuda.synchronize()
    assert step.status.item() == 0
    for b, n in enumerate(new):
        at = slice(row[b], row[b + 1])
        R.check(step.out[at], step.lse[at], dtype, D,
                R.attention(q[at], k[kr[b]:kr[b + 1]], v[kr[b]:kr[b + 1]], prefix[b]), f"sequence {b}")
    assert bool((step.out[row[-1]:] == 7.0).all())


@pytest.mark.parametrize("dtype,Hq,Hkv,D,page,prefix,new", [
    (BF16, 32, 8, 128, 16, [8191], [1]),            # decoding, many splits
    (BF16, 4, 1, 64, 64, [20000, 3], [1, 1]),
    (BF16, 64, 8, 128, 16, [9000, 100], [4, 4]),    # a few tokens of each
    (BF16, 8, 2, 128, 32, [5000], [200]),
    (F32, 8, 8, 128, 16, [4000, 0], [1, 1]),
    (F32, 6, 2, 64, 64, [2500], [33])])
def test_chunk_parity_long_prefix(dtype, Hq, Hkv, D, page, prefix, new):
    g = _gen(7)
    total = [p + n for p, n in zip(prefix, new)]
    kr, row = _rows(total), _rows(new)
    k, v = (_rand((kr[-1], Hkv, D), g, dtype) for _ in range(2))
    kp, vp, table = _paged(k, v, total, page, g)
    q = _rand((row[-1], Hq, D), g, dtype)
    for bounds in (dict(max_new=max(new), max_prefix=max(prefix)), {}):
        out = api.chunk_attention_paged(q, kp, vp, table, _ints(row), _ints(prefix), want_lse=True, **bounds)
        assert out["status"].item() == 0
        for b in range(len(new)):
            at = slice(row[b], row[b + 1])
            R.check(out["out"][at], out["lse"][at], dtype, D,
                    R.attention(q[at], k[kr[b]:kr[b + 1]], v[kr[b]:kr[b + 1]], prefix[b]), f"sequence {b}")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("value,where", [(NAN, "k"), (NAN, "v"), (NAN, "kv"), (INF, "v"), (-INF, "v")])
def test_nonfinite_values_reach_only_rows_that_see_them(dtype, value, where):
    """Tokens 40 and 130 of 200 hold the value in one element of K and/or V:
    rows before them are as if it were not there."""
    Hq, Hkv, D, n = 8, 2, 128, 200
    g = _gen(11)
    q, k, v = (_rand((n, h, D), g, dtype) for h in (Hq, Hkv, Hkv))
    for t in (40, 130):
        if "k" in where:
            k[t, 1, 5] = value
        if "v" in where:
            v[t, 1, 7] = value
    ref = R.attention(q, k, v, 0)
    got = api.prompt_attention(q, k, v, _ints([0, n]), want_lse=True)
    R.check(got["out"], got["lse"], dtype, D, ref, "prompt")
    kp, vp, table = _paged(k, v, [n], 16, g)
    for first, cnt in ((0, n), (60, 140), (129, 1), (128, 2), (130, 1), (30, 20)):
        m = first + cnt
        got = api.chunk_attention_paged(q[first:m], kp, vp, table, _ints([0, cnt]), _ints([first]), max_new=cnt,
                                        max_prefix=first, want_lse=True)
        r = R.attention(q[first:m], k[:m], v[:m], first)
        R.check(got["out"], got["lse"], dtype, D, r, f"chunk {first}+{cnt}")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_extreme_scores(dtype):
    """Scores of hundreds (one key takes all the weight) and rows whose keys
    rise and fall by far more than an exponent's range."""
    Hq, Hkv, D, n = 4, 2, 64, 400
    g = _gen(13)
    q, k, v = (_rand((n, h, D), g, dtype) for h in (Hq, Hkv, Hkv))
    k *= 16
    k[200:] *= -8
    got = api.prompt_attention(q, k, v, _ints([0, n]), want_lse=True)
    out, spread, lse, mag = R.attention(q, k, v, 0)
    R.check(got["out"], got["lse"], dtype, D, (out, spread, lse, mag))
    q0 = torch.zeros_like(q)  # uniform weights
    got = api.prompt_attention(q0, k, v, _ints([0, n]), want_lse=True)
    R.check(got["out"], got["lse"], dtype, D, R.attention(q0, k, v, 0))


def test_scale_is_taken():
    g = _gen(17)
    q, k, v = (_rand((70, h, 64), g, BF16) for h in (4, 2, 2))
    got = api.prompt_attention(q, k, v, _ints([0, 70]), scale=0.25)
    want = api.prompt_attention((q.float() * 2).to(BF16), k, v, _ints([0, 70]))
    assert torch.equal(got["out"], want["out"])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_bad_page_is_reported_and_spoils_only_its_sequence(dtype):
    g = _gen(19)
    Hq, Hkv, D, page = 8, 2, 128, 16
    total, new = [300, 280], [1, 40]
    prefix = [t - n for t, n in zip(total, new)]
    k, v = (_rand((580, Hkv, D), g, dtype) for _ in range(2))
    kp, vp, table = _paged(k, v, total, page, g)
    q = _rand((41, Hq, D), g, dtype)
    good = api.chunk_attention_paged(q, kp, vp, table, _ints([0, 1, 41]), _ints(prefix))
    for b, bad in ((0, kp.shape[0]), (1, -1), (1, 1 << 30)):
        t2 = table.clone()
        t2[b, 3] = bad
        got = api.chunk_attention_paged(q, kp, vp, t2, _ints([0, 1, 41]), _ints(prefix))
        assert got["status"].item() == B.STATUS_BAD_PAGE
        other = slice(1, 41) if b == 0 else slice(0, 1)
        assert torch.equal(got["out"][other], good["out"][other])


def test_lengths_out_of_range_are_reported():
    g = _gen(23)
    q, k, v = (_rand((50, h, 64), g, BF16) for h in (4, 2, 2))
    full = api.prompt_attention(q, k, v, _ints([0, 20, 50]))
    for rows, good in (([0, 20, 51], slice(0, 20)), ([0, -1, 50], slice(0, 0)), ([20, 0, 50], slice(0, 0)),
                       ([-3, 20, 50], slice(20, 50))):
        got = api.prompt_attention(q, k, v, _ints(rows))
        assert got["status"].item() == B.STATUS_BAD_LENGTH, rows
        assert torch.equal(got["out"][good], full["out"][good])
    got = api.prompt_attention(q, k, v, _ints([0, 20, 50]), max_len=25)
    assert got["status"].item() == B.STATUS_BAD_LENGTH
    assert torch.equal(got["out"][:45], full["out"][:45]) and bool((got["out"][45:] == 0).all())
    kp, vp, table = _paged(k, v, [20, 30], 16, g, fill=0.0)
    ok = api.chunk_attention_paged(q[:6], kp, vp, table, _ints([0, 1, 6]), _ints([19, 25]))
    assert ok["status"].item() == 0
    got = api.chunk_attention_paged(q[:6], kp, vp, table, _ints([0, 1, 6]), _ints([-4, 25]))
    assert got["status"].item() == B.STATUS_BAD_PREFIX
    assert torch.equal(got["out"][1:], ok["out"][1:])
    cap = table.shape[1] * 16
    got = api.chunk_attention_paged(q[:6], kp, vp, table, _ints([0, 1, 6]), _ints([cap, 25]))
    assert got["status"].item() & B.STATUS_BAD_LENGTH  # its token is past the table
    assert torch.equal(got["out"][1:], ok["out"][1:])


def test_many_sequences():
    g = _gen(29)
    lens = [(i * 7) % 5 for i in range(700)]
    row = _rows(lens)
    q, k, v = (_rand((row[-1], h, 64), g, BF16) for h in (4, 2, 2))
    out = api.prompt_attention(q, k, v, _ints(row), max_len=4)
    assert out["status"].item() == 0
    for b in list(range(0, 700, 97)) + [699]:
        a, e = row[b], row[b + 1]
        R.check(out["out"][a:e], None, BF16, 64, R.attention(q[a:e], k[a:e], v[a:e], 0), f"sequence {b}")
    whole = torch.stack([out["out"][row[b]] for b in range(700) if lens[b]])
    first = torch.stack([v[row[b]].repeat_interleave(2, 0) for b in range(700) if lens[b]])
    assert torch.equal(whole, first)  # a first token sees itself alone


def test_results_do_not_change_from_call_to_call():
    g = _gen(31)
    lens = [900, 3, 257]
    row = _rows(lens)
    q, k, v = (_rand((row[-1], h, 128), g, BF16) for h in (8, 2, 2))
    kp, vp, table = _paged(k, v, lens, 16, g)
    runs = [(api.prompt_attention(q, k, v, _ints(row))["out"],
             api.chunk_attention_paged(q[[899, 902, 1159]], kp, vp, table, _ints([0, 1, 2, 3]), _ints([899, 2, 256]),
                                       max_new=1)["out"]) for _ in range(3)]
    for a, b in runs[1:]:
        assert torch.equal(a, runs[0][0]) and torch.equal(b, runs[0][1])


def test_two_streams_at_once():
    """Calls with separate steps on two streams do not disturb each other."""
    g = _gen(37)
    n = 600
    sets = [[_rand((n, h, 128), g, BF16) for h in (8, 2, 2)] for _ in range(2)]
    want = [api.prompt_attention(*s, _ints([0, n]))["out"] for s in sets]
    steps = [api.PromptStep(B=1, Hq=8, Hkv=2, D=128, max_tokens=n, dtype=BF16) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    rs = _ints([0, n])
    torch.cuda.synchronize()
    for _ in range(5):
        for s, st, data in zip(streams, steps, sets):
            with torch.cuda.stream(s):
                st.prompt_attention(*data, row_start=rs)
    torch.cuda.synchronize()
    for st, w in zip(steps, want):
        assert torch.equal(st.out, w) and st.status.item() == 0


def test_refusals_of_the_python_entry_points():
    q, k = torch.zeros((4, 4, 64), dtype=BF16, device="cuda"), torch.zeros((4, 2, 64), dtype=BF16, device="cuda")
    rs = _ints([0, 4])
    with pytest.raises(ValueError):
        api.prompt_attention(q, k.float(), k, rs)
    with pytest.raises(ValueError):
        api.prompt_attention(q, k[:3], k, rs)
    with pytest.raises(ValueError):
        api.prompt_attention(q, k, k, rs.long())
    with pytest.raises(ValueError):
        api.prompt_attention(q, k, k.transpose(1, 2).contiguous().transpose(1, 2), rs)
    with pytest.raises(ValueError):
        api.prompt_attention(q, k, k, rs.cpu())
    with pytest.raises(B.MedusaError):
        api.prompt_attention(torch.zeros((4, 3, 64), dtype=BF16, device="cuda"), k, k, rs)  # 3 heads over 2
    with pytest.raises(B.MedusaError):
        api.prompt_attention(*(torch.zeros((4, 2, 32), dtype=BF16, device="cuda"),) * 3, rs)
    with pytest.raises(TypeError):
        api.prompt_attention(*(torch.zeros((4, 2, 64), dtype=torch.float16, device="cuda"),) * 3, rs)
    odd = torch.zeros(4 * 132 + 4, dtype=BF16, device="cuda")[:4 * 132].view(4, 132)
    with pytest.raises(B.MedusaError):  # rows 264 bytes apart
        api.prompt_attention(q, odd.as_strided((4, 2, 64), (132, 64, 1)), k, rs)
    pool = torch.zeros((3, 2, 16, 64), dtype=BF16, device="cuda")
    with pytest.raises(ValueError):
        api.kv_append_paged(k, k, torch.zeros(3, dtype=torch.int64, device="cuda"), pool, pool)
    with pytest.raises(ValueError):
        api.kv_append_paged(k, k, torch.zeros(4, dtype=torch.int32, device="cuda"), pool, pool)
    step = api.PromptStep(B=1, Hq=4, Hkv=2, D=64, max_tokens=3, dtype=BF16, page_size=16, max_pages=2, num_pages=3)
    with pytest.raises(ValueError):
        step.prompt_attention(q, k, k, row_start=rs)  # 4 rows, room for 3
    with pytest.raises(ValueError):
        step.append(k[:3], k[:3], pool[:2], pool[:2])
