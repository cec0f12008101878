"""Host checks of the serving calls (page tables, 4-bit cache, packed prompts): every refusal comes
before any CUDA call, so these run without a GPU on a plan that never touches one."""

import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from rag_kv_cache_gb300 import _lib
    from rag_kv_cache_gb300.build import build

    return _lib.load(build())


@pytest.fixture()
def plan():
    """Memory shaped like the head of a plan: the config alone, which is all the host checks read."""
    from rag_kv_cache_gb300 import _lib

    raw = ctypes.create_string_buffer(4096)
    cfg = _lib.CbConfig(1, 1, 0, 8, 2, 128, 1e4, 0, 15, 15)
    ctypes.memmove(raw, ctypes.byref(cfg), ctypes.sizeof(cfg))
    return raw


P = 1 << 20  # an aligned address that no refused call reads


def _refused(lib, status, word, want=1):
    assert status == want, lib.cb_last_error_string()
    assert word in lib.cb_last_error_string().decode()


def test_page_bytes(lib, plan):
    assert lib.cb_kv4_page_bytes(plan, 16) == 18 * 128
    assert lib.cb_kv4_page_bytes(plan, 1024) == 64 * 18 * 128
    for bad in (0, -16, 8, 24, 1040):
        assert lib.cb_kv4_page_bytes(plan, bad) == 0
    assert lib.cb_kv4_page_bytes(None, 16) == 0


def test_page_tables_refusals(lib, plan):
    def call(plan_=plan, ctx=P, new=P + 64, n=4, page=16, free=P, n_free=9, frm=None, table=P, width=8, cu=P, kv=P + 128,
             pos=P, slots=P, rows=5, to=P + 192):
        return lib.cb_page_tables(plan_, ctx, new, n, page, free, n_free, frm, table, width, cu, kv, pos, slots, rows, to,
                                  None)

    _refused(lib, call(plan_=None), "plan")
    for page in (0, 8, 17, 2048):
        _refused(lib, call(page=page), "page_size")
    for name in ("n", "n_free", "width", "rows"):
        _refused(lib, call(**{name: -1}), "negative")
    _refused(lib, call(n=16385), "n_seqs", 2)
    _refused(lib, call(n=16384, width=1 << 17), "too large")
    _refused(lib, call(width=1 << 28, n=1), "too large")
    for name, said in (("ctx", "ctx_lens"), ("new", "new_lens"), ("free", "free_pages"), ("table", "table"), ("cu", "cu_seqlens"),
                       ("kv", "kv_lens"), ("pos", "positions"), ("slots", "slots"), ("to", "free_to")):
        _refused(lib, call(**{name: None}), said)
    _refused(lib, call(kv=P), "kv_lens must not be")
    _refused(lib, call(kv=P + 64), "kv_lens must not be")
    _refused(lib, call(frm=P + 192), "free_to must not be")


def test_rows_refusals(lib, plan):
    for fn, order in ((lib.cb_kv4_store, "kvsn"), (lib.cb_kv4_load, "c")):
        def call(plan_=plan, k=P, v=P, slots=P, n=3, cache=P, pages=2, page=16):
            if order == "c":
                return fn(plan_, cache, pages, page, slots, n, k, v, None)
            return fn(plan_, k, v, slots, n, cache, pages, page, None)

        _refused(lib, call(plan_=None), "plan")
        _refused(lib, call(n=-1), "n < 0")
        _refused(lib, call(pages=-1), "n_pages")
        _refused(lib, call(page=20), "page_size")
        _refused(lib, call(pages=1 << 27), "2^31")
        for name in ("k", "v", "slots", "cache"):
            _refused(lib, call(**{name: None}), name)
        for name in ("k", "v", "cache"):
            _refused(lib, call(**{name: P + 8}), "16-byte")
        assert call(n=0, k=None, v=None, slots=None, cache=None) == 0  # nothing to do


def test_decode_refusals(lib, plan):
    def call(plan_=plan, q=P, cache=P, pages=2, page=16, table=P, width=4, lens=P, n=3, out=P + 4096):
        return lib.cb_kv4_decode_attention(plan_, q, cache, pages, page, table, width, lens, n, 0.0, out, None)

    _refused(lib, call(plan_=None), "plan")
    _refused(lib, call(page=12), "page_size")
    _refused(lib, call(pages=-2), "n_pages")
    for name in ("n", "width"):
        _refused(lib, call(**{name: -1}), "negative")
    _refused(lib, call(n=1 << 30), "2^31")
    _refused(lib, call(width=1 << 28), "2^31")
    _refused(lib, call(n=1 << 11, width=1 << 18), "2^34", 2)  # 2^11 requests of 2 heads and 2^22 keys
    _refused(lib, call(n=1 << 20, width=1 << 10, page=1024), "2^34", 2)
    for name, said in (("q", "q"), ("cache", "cache"), ("table", "table"), ("lens", "kv_lens"), ("out", "out")):
        _refused(lib, call(**{name: None}), said)
    for name in ("q", "cache", "out"):
        _refused(lib, call(**{name: P + 4}), "16-byte")
    _refused(lib, call(q=P + 4096, out=P + 4096), "out must not be q")
    assert call(n=0, q=None) == 0


def test_prompt_refusals(lib, plan):
    def call(plan_=plan, q=P, k=P + 4096, v=P + 4096, cu=P, n=2, rows=8, out=P + 8192):
        return lib.cb_prompt_attention(plan_, q, k, v, cu, n, rows, 0.0, out, None)

    _refused(lib, call(plan_=None), "plan")
    for name in ("n", "rows"):
        _refused(lib, call(**{name: -1}), "negative")
    _refused(lib, call(n=16385), "n_seqs", 2)
    for name, said in (("q", "q"), ("k", "k"), ("v", "v"), ("cu", "cu_seqlens"), ("out", "out")):
        _refused(lib, call(**{name: None}), said)
    for name in ("q", "k", "v", "out"):
        _refused(lib, call(**{name: P + 8192 + 2}), "16-byte")
    _refused(lib, call(out=P), "out must not be")
    _refused(lib, call(out=P + 4096), "out must not be")
    assert call(n=0, q=None) == 0 and call(rows=0, q=None) == 0


class _FakePlan:
    hq, hkv, head_dim, device, handle = 8, 2, 128, 0, None


def test_binding_checks_shapes_before_the_library(lib, plan):
    import rag_kv_cache_gb300 as cb

    p = _FakePlan()
    p.handle = plan
    assert cb.cb_kv4_page_bytes(p, 64) == 4 * 18 * 128
    with pytest.raises(cb.CacheBlendError):
        cb.cb_kv4_page_bytes(p, 20)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    cache = torch.zeros((3, 2, 18 * 128), dtype=torch.uint8)
    with pytest.raises(ValueError, match="cache must have shape"):
        cb.cb_kv4_store(p, bf(4, 2, 128), bf(4, 2, 128), i32(4), cache, 32)
    with pytest.raises(ValueError, match="cache must have 3 dim"):
        cb.cb_kv4_load(p, cache[0], 16, i32(4), bf(4, 2, 128), bf(4, 2, 128))
    with pytest.raises(ValueError, match="on a CUDA device"):
        cb.cb_kv4_load(p, cache, 16, i32(4), bf(4, 2, 128), bf(4, 2, 128))
    with pytest.raises(ValueError, match="table must have 2 dim"):
        cb.cb_kv4_decode_attention(p, bf(2, 8, 128), cache, 16, i32(4), i32(2), bf(2, 8, 128))
    with pytest.raises(ValueError, match="q must have shape"):
        cb.cb_prompt_attention(p, bf(5, 8, 64), bf(5, 2, 128), bf(5, 2, 128), i32(2), bf(5, 8, 128))
    with pytest.raises(ValueError, match="q must have 3 dim"):
        cb.cb_prompt_attention(p, bf(5, 1024), bf(5, 2, 128), bf(5, 2, 128), i32(2), bf(5, 8, 128))
    with pytest.raises(ValueError, match="first offset"):
        cb.cb_prompt_attention(p, bf(5, 8, 128), bf(5, 2, 128), bf(5, 2, 128), i32(0), bf(5, 8, 128))
    with pytest.raises(TypeError, match="q must be a torch.Tensor"):
        cb.cb_prompt_attention(p, None, bf(5, 2, 128), bf(5, 2, 128), i32(2), bf(5, 8, 128))
    with pytest.raises(ValueError, match="on a CUDA device"):
        cb.cb_page_tables(p, i32(3), i32(2), 16, i32(9), i32(3, 4), i32(4), i32(3), i32(5), i32(5), i32(1))
    with pytest.raises(ValueError, match="free_pages must have 1 dim"):
        cb.cb_page_tables(p, i32(3), i32(3), 16, i32(9, 1), i32(3, 4), i32(4), i32(3), i32(5), i32(5), i32(1))


TABLES = {"ctx_lens": 16, "new_lens": 16, "free_pages": 36, "free_from": 4, "table": 128, "cu_seqlens": 20, "kv_lens": 16,
          "positions": 20, "slots": 20, "free_to": 4}  # bytes: 4 requests, 9 free pages, 8 pages a row, 5 rows


@pytest.mark.parametrize("out", ["table", "cu_seqlens", "kv_lens", "positions", "slots", "free_to"])
@pytest.mark.parametrize("other", list(TABLES))
@pytest.mark.parametrize("where", ["first bytes", "last bytes"])
def test_page_tables_outputs_lie_apart(lib, plan, out, other, where):
    if out == other:
        return
    at = {name: P + 4096 * i for i, name in enumerate(TABLES)}
    # the output ends one element inside the other buffer, or begins on its last one
    at[out] = at[other] - TABLES[out] + 4 if where == "first bytes" else at[other] + TABLES[other] - 4
    a = [at[name] for name in TABLES]
    got = lib.cb_page_tables(plan, a[0], a[1], 4, 16, a[2], 9, a[3], a[4], 8, a[5], a[6], a[7], a[8], 5, a[9], None)
    said = lib.cb_last_error_string().decode()
    assert got == 1 and out in said and other in said and ("overlaps" in said or "must not be" in said), said


@pytest.mark.parametrize("where", ["first bytes", "last bytes"])
def test_rows_and_attention_outputs_lie_apart(lib, plan, where):
    row, kv = 8 * 128 * 2, 2 * 128 * 2  # bytes of a row of q and out, of k and v
    cache = 4 * 2 * 18 * 128  # four pages of 16 tokens, two kv heads

    def place(sizes, out, other):
        at = {name: P + (i << 16) for i, name in enumerate(sizes)}
        at[out] = at[other] - sizes[out] + 16 if where == "first bytes" else at[other] + (sizes[other] - 1) // 16 * 16
        return at

    def overlaps(got, out, other):
        said = lib.cb_last_error_string().decode()
        assert got == 1 and "overlaps" in said and out in said and other in said, said

    sizes = {"k": 3 * kv, "v": 3 * kv, "slots": 12, "cache": cache}
    for other in ("k", "v", "slots"):
        a = place(sizes, "cache", other)
        overlaps(lib.cb_kv4_store(plan, a["k"], a["v"], a["slots"], 3, a["cache"], 4, 16, None), "cache", other)
    for out, other in (("k", "v"), ("k", "cache"), ("k", "slots"), ("v", "k"), ("v", "cache"), ("v", "slots")):
        a = place(sizes, out, other)
        overlaps(lib.cb_kv4_load(plan, a["cache"], 4, 16, a["slots"], 3, a["k"], a["v"], None), out, other)
    sizes = {"q": 3 * row, "cache": cache, "table": 24, "kv_lens": 12, "out": 3 * row}
    for other in ("q", "cache", "table", "kv_lens"):
        a = place(sizes, "out", other)
        overlaps(lib.cb_kv4_decode_attention(plan, a["q"], a["cache"], 4, 16, a["table"], 2, a["kv_lens"], 3, 0.0, a["out"], None),
                 "out", other)
    sizes = {"q": 9 * row, "k": 9 * kv, "v": 9 * kv, "cu_seqlens": 12, "out": 9 * row}
    for other in ("q", "k", "v", "cu_seqlens"):
        a = place(sizes, "out", other)
        overlaps(lib.cb_prompt_attention(plan, a["q"], a["k"], a["v"], a["cu_seqlens"], 2, 9, 0.0, a["out"], None), "out", other)


def test_decode_wait_timeout_probe_refusals(lib, plan):
    from rag_kv_cache_gb300 import _lib

    def call(plan_=plan, q=P, cache=P + (1 << 16), table=P + (1 << 17), width=4, lens=P + (1 << 18), n=3, out=P + (1 << 19)):
        return lib.cb_test_kv4_decode_wait_timeout(plan_, q, cache, 2, 16, table, width, lens, n, out, None)

    _refused(lib, call(plan_=None), "plan")
    for name, said in (("q", "q"), ("cache", "cache"), ("table", "table"), ("lens", "kv_lens"), ("out", "out")):
        _refused(lib, call(**{name: None}), said)
    _refused(lib, call(out=P + 16), "overlaps")
    for heads, dim in ((16, 128), (8, 64)):  # 16 query heads per kv head, 64 dims
        cfg = _lib.CbConfig(1, 1, 0, heads, 1, dim, 1e4, 0, 15, 15)
        raw = ctypes.create_string_buffer(4096)
        ctypes.memmove(raw, ctypes.byref(cfg), ctypes.sizeof(cfg))
        _refused(lib, call(plan_=raw), "head_dim 128", 2)


def test_prompt_wait_timeout_probe_refusals(lib, plan):
    from rag_kv_cache_gb300 import _lib

    def call(plan_=plan, q=P, k=P + (1 << 16), v=P + (1 << 17), cu=P + (1 << 18), n=2, rows=8, out=P + (1 << 19)):
        return lib.cb_test_prompt_wait_timeout(plan_, q, k, v, cu, n, rows, out, None)

    _refused(lib, call(plan_=None), "plan")
    for name, said in (("q", "q"), ("k", "k"), ("v", "v"), ("cu", "cu_seqlens"), ("out", "out")):
        _refused(lib, call(**{name: None}), said)
    _refused(lib, call(out=P + 16), "overlaps")
    cfg = _lib.CbConfig(1, 1, 0, 8, 2, 64, 1e4, 0, 15, 15)
    raw = ctypes.create_string_buffer(4096)
    ctypes.memmove(raw, ctypes.byref(cfg), ctypes.sizeof(cfg))
    _refused(lib, call(plan_=raw), "head_dim 128", 2)
