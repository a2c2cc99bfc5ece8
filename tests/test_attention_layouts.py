"""Which layouts of a cache the attention operators accept (no GPU needed: the calls are on no
tokens, or are refused before any CUDA work is enqueued)."""
import pytest

from test_attention_abi import A, B, C, L, NULL, OK, SHAPE, attend, grad, rope, tok, write  # noqa: F401


@pytest.mark.parametrize("call", ["nvfp4_cache_write", "nvfp4_cache_read", "attend"])
def test_heads_may_lie_as_far_apart_as_a_pool_is_large(L, call):  # noqa: F811
    f = (lambda c: attend(L, T=0, Hq=c["heads"], c=c)) if call == "attend" else (lambda c: write(L, call, T=0, c=c))

    def heads_first(pages, dim=128, page=64, heads=8):
        code, scale = page * dim // 2, page * dim // 16
        return dict(pages=pages, heads=heads, dim=dim, page_size=page, code_page=code, code_row=dim // 2, code_head=pages * code,
                    scale_page=scale, scale_row=dim // 16, scale_head=pages * scale)
    for pages in (1, 131072, 140000, 10 ** 6, 2 ** 31 - 1):
        assert f(heads_first(pages)) == OK, pages
    assert f(heads_first(1000, heads=65535, dim=256, page=65536)) == OK
    # heads that overlap their own pages, or lie further apart than any memory is large
    for bad in (dict(heads_first(140000), code_head=140000 * 4096 - 16), dict(heads_first(140000), scale_head=140000 * 512 - 2),
                dict(heads_first(1000), code_head=2 ** 45 + 16), dict(heads_first(1000), scale_head=2 ** 62)):
        assert f(bad) == SHAPE, bad
    # pages behind heads that lie far apart: their stride does not reach over them
    assert f(dict(heads_first(1000), code_head=2 ** 40, code_page=2 ** 32 - 16, code_row=64)) == SHAPE


def test_tokens_and_heads_may_lie_as_far_apart_as_memory_is_large(L):  # noqa: F811
    """Refused for the missing page table or positions alone, which are looked at behind the strides."""
    for far in (2 ** 29 - 8, 2 ** 29 + 8, 2 ** 31 + 64, 2 ** 40, 2 ** 56):
        for ts, hs in ((far, 64), (64, far)):
            t = lambda p: tok(p, ts, hs)
            for p in ("q", "k", "oq", "ok"):
                assert rope(L, pos=None, **{p: t(A)}) == NULL
            for p in ("dq", "dk", "q", "k", "oq", "ok"):
                assert grad(L, pos=None, **{p: t(A)}) == NULL
            for call in ("nvfp4_cache_write", "nvfp4_cache_read"):
                assert write(L, call, k=t(A), v=t(B), T=4, b=dict(sequences=0)) == OK
            assert attend(L, q=t(A), b=dict(sequences=0)) == OK and attend(L, o=t(C), b=dict(sequences=0)) == OK
    for ts, hs in ((2 ** 57, 64), (64, 2 ** 58 + 64), (-8, 64), (64, -8)):
        t = tok(A, ts, hs)
        assert rope(L, k=t) == SHAPE and grad(L, k=t) == SHAPE and attend(L, q=t) == SHAPE and attend(L, o=t) == SHAPE
        assert write(L, k=t) == SHAPE and write(L, "nvfp4_cache_read", v=t) == SHAPE
    assert rope(L, T=1, pos=None, q=tok(A, 2 ** 62, 64)) == NULL  # not stepped over
    for stride, status in ((2 ** 31, OK), (2 ** 40, OK), (2 ** 58, SHAPE)):
        assert attend(L, T=0, b=dict(table_stride=stride)) == status
