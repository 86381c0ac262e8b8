"""Host-side checks of the prompt-side calls that need no GPU: argument
errors are reported by return code before anything reaches the device."""
import ctypes

import pytest

from medusa_tree_speculative_heads_b200 import binding as B
from medusa_tree_speculative_heads_b200 import build as build_mod

FAKE, ODD, NUL = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1004), None
INV, UNS, WS = B.MEDUSA_ERR_INVALID_ARG, B.MEDUSA_ERR_UNSUPPORTED, B.MEDUSA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.lib()


def test_names_are_declared():
    names = B.declared_functions()
    for n in ("kv_page_plan", "kv_append_paged", "prompt_attention", "prompt_attention_workspace_size",
              "chunk_attention_paged", "chunk_attention_paged_workspace_size"):
        assert n in names, n


PLAN = dict(prefix_len=FAKE, new_len=FAKE, B=2, room=0, table=FAKE, max_pages=4, page=16, num=8, owned=FAKE,
            owned_out=FAKE, free=FAKE, count=FAKE, count_out=FAKE, row=FAKE, slots=FAKE, max_tokens=8, status=NUL,
            stream=NUL)


@pytest.mark.parametrize("kw,code", [
    (dict(prefix_len=NUL), INV), (dict(new_len=NUL), INV), (dict(table=NUL), INV), (dict(owned=NUL), INV),
    (dict(owned_out=NUL), INV), (dict(free=NUL), INV), (dict(count=NUL), INV), (dict(count_out=NUL), INV),
    (dict(row=NUL), INV), (dict(slots=NUL), INV), (dict(slots=ODD), INV), (dict(B=0), INV), (dict(room=-1), INV),
    (dict(max_pages=0), INV), (dict(page=0), INV), (dict(num=0), INV), (dict(max_tokens=0), INV),
    (dict(max_pages=1 << 20, page=1 << 12), INV), (dict(max_tokens=(1 << 30) + 1), INV), (dict(B=8193), UNS)])
def test_plan_refuses(lib, kw, code):
    assert lib.kv_page_plan(*{**PLAN, **kw}.values()) == code
    assert b"kv_page_plan" in lib.medusa_last_error()


APPEND = dict(k=FAKE, v=FAKE, ks=1024, vs=1024, slots=FAKE, N=3, kp=FAKE, vp=FAKE, page=16, num=8, Hkv=8, D=128, dt=1,
              status=NUL, stream=NUL)


@pytest.mark.parametrize("kw,code", [
    (dict(k=NUL), INV), (dict(v=NUL), INV), (dict(slots=NUL), INV), (dict(kp=NUL), INV), (dict(vp=NUL), INV),
    (dict(k=ODD), INV), (dict(vp=ODD), INV), (dict(ks=1023), INV), (dict(vs=1028), INV), (dict(ks=-1024), INV),
    (dict(N=-1), INV), (dict(page=0), INV), (dict(num=0), INV), (dict(Hkv=0), INV), (dict(N=1 << 28), INV),
    (dict(page=1 << 16, num=1 << 16), INV), (dict(D=96), UNS), (dict(dt=2), UNS)])
def test_append_refuses(lib, kw, code):
    assert lib.kv_append_paged(*{**APPEND, **kw}.values()) == code
    assert b"kv_append_paged" in lib.medusa_last_error()


PROMPT = dict(q=FAKE, k=FAKE, v=FAKE, qs=4096, ks=1024, vs=1024, row=FAKE, B=2, N=64, max_len=0, Hq=32, Hkv=8, D=128,
              scale=ctypes.c_float(0), dt=1, out=FAKE, lse=NUL, ws=NUL, ws_n=0, status=NUL, stream=NUL)
COMMON = [
    (dict(q=NUL), INV), (dict(row=NUL), INV), (dict(out=NUL), INV), (dict(q=ODD), INV), (dict(out=ODD), INV),
    (dict(qs=4095), INV), (dict(qs=4100), INV), (dict(B=0), INV), (dict(N=-1), INV), (dict(Hq=30), INV),
    (dict(Hkv=0), INV), (dict(D=96), UNS), (dict(dt=7), UNS), (dict(Hq=65, Hkv=1, qs=65 * 128), UNS),
    (dict(ws=FAKE, ws_n=16), WS), (dict(), WS)]


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(k=NUL), INV), (dict(v=NUL), INV), (dict(ks=1000), INV), (dict(vs=1028), INV), (dict(max_len=-1), INV)])
def test_prompt_refuses(lib, kw, code):
    assert lib.prompt_attention(*{**PROMPT, **kw}.values()) == code
    assert b"prompt_attention" in lib.medusa_last_error()


CHUNK = dict(q=FAKE, qs=4096, kp=FAKE, vp=FAKE, table=FAKE, max_pages=4, page=16, num=8, row=FAKE, prefix=FAKE, B=2,
             N=64, max_new=0, max_prefix=0, Hq=32, Hkv=8, D=128, scale=ctypes.c_float(0), dt=1, out=FAKE, lse=NUL,
             ws=NUL, ws_n=0, status=NUL, stream=NUL)


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(kp=NUL), INV), (dict(vp=ODD), INV), (dict(table=NUL), INV), (dict(prefix=NUL), INV),
    (dict(max_pages=0), INV), (dict(page=0), INV), (dict(num=0), INV), (dict(max_prefix=65), INV),
    (dict(max_new=-1), INV), (dict(num=1 << 28), INV)])
def test_chunk_refuses(lib, kw, code):
    assert lib.chunk_attention_paged(*{**CHUNK, **kw}.values()) == code
    assert b"chunk_attention_paged" in lib.medusa_last_error()


def test_workspace_queries_are_pure_and_grow_with_the_rows(lib):
    last = 0
    for n in (0, 1, 7, 64, 1000, 100000):
        a = lib.chunk_attention_paged_workspace_size(2, n, 0, 0, 512, 16, 32, 8, 128, 1)
        assert a == lib.chunk_attention_paged_workspace_size(2, n, 0, 0, 512, 16, 32, 8, 128, 1)
        assert a >= last
        last = a
        assert lib.prompt_attention_workspace_size(2, n, 0, 32, 8, 128, 1) >= 0
    assert lib.prompt_attention_workspace_size(2, 64, 0, 30, 8, 128, 1) == 0
    assert lib.chunk_attention_paged_workspace_size(2, 64, 0, 0, 0, 16, 32, 8, 128, 1) == 0
