"""Attention calls of more rows than their sequences can fill (N > B * max_new:
a padded batch with a tight bound), over prefixes long enough for split keys:
the partials of the splits stay inside the workspace."""
import pytest
import torch

import prompt_ref as R
from medusa_tree_speculative_heads_b200 import api
from test_gpu_prompt import BF16, F32, _gen, _ints, _paged, _rand, _rows

pytestmark = pytest.mark.gpu

GUARD = 64 << 20  # bytes behind the workspace


def _guarded(step):
    """The step's workspace at the front of a larger filled buffer."""
    buf = torch.full((step.ws_n + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
    step.ws = buf[:step.ws_n]
    step.out.fill_(7.0)
    step.lse.fill_(7.0)
    return buf[step.ws_n:]


def _check(step, guard, row):
    torch.cuda.synchronize()
    assert step.status.item() == 0
    assert bool((guard == 0xA5).all())
    assert bool((step.out[row[-1]:] == 7.0).all()) and bool((step.lse[row[-1]:] == 7.0).all())


@pytest.mark.parametrize("dtype,N,new,prefix", [
    (BF16, 127, [64], [32768]), (BF16, 67, [60], [20000]), (BF16, 255, [64, 30], [8192, 700]),
    (BF16, 127, [64], [5]), (F32, 127, [64], [4000]), (F32, 50, [1], [4000])])
def test_chunks(dtype, N, new, prefix):
    g = _gen(71)
    Hq, Hkv, D, page = 32, 8, 128, 16
    total, row = [p + n for p, n in zip(prefix, new)], _rows(new)
    kr = _rows(total)
    k, v = (_rand((kr[-1], Hkv, D), g, dtype) for _ in range(2))
    kp, vp, table = _paged(k, v, total, page, g)
    q = _rand((N, Hq, D), g, dtype)
    step = api.PromptStep(B=len(new), Hq=Hq, Hkv=Hkv, D=D, max_tokens=N, dtype=dtype, page_size=page,
                          max_pages=table.shape[1], num_pages=kp.shape[0], max_new=max(new), max_prefix=max(prefix),
                          want_lse=True)
    guard = _guarded(step)
    step.chunk_attention(q, kp, vp, table, _ints(prefix), row_start=_ints(row))
    _check(step, guard, row)
    for b in range(len(new)):
        at, keys = slice(row[b], row[b + 1]), slice(kr[b], kr[b + 1])
        R.check(step.out[at], step.lse[at], dtype, D, R.attention(q[at], k[keys], v[keys], prefix[b]), f"sequence {b}")


def test_one_head_prompt():
    g = _gen(73)
    N, n = 6399, 6144
    q, k, v = (_rand((N, 1, 128), g, BF16) for _ in range(3))
    step = api.PromptStep(B=1, Hq=1, Hkv=1, D=128, max_tokens=N, dtype=BF16, max_new=n, want_lse=True)
    guard = _guarded(step)
    step.prompt_attention(q, k, v, row_start=_ints([0, n]))
    _check(step, guard, [0, n])
    R.check(step.out[:n], step.lse[:n], BF16, 128, R.attention(q[:n], k[:n], v[:n], 0))
