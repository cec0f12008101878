"""Serving calls (page tables, 4-bit cache rows, decode over 4-bit pages, packed prompts) against the
oracle, with the sizes, masks and contents where they can go wrong, and a run of them together.

Tolerances. Page tables, slots, codes and loaded rows are exact. Attention in 64 bits over the same
rows, s = sum_j p_j |v_j|: the softmax weights (decode: times V's scale) are rounded to bf16 once,
2^-8 relative each, so at most 2^-8 s; the output's rounding adds 2^-8 |out|. Scores are fp32 sums:
of D products |q k| (prompt), or of groups of 32 products of |q| with 8 + code <= 15 and the offset
8 |q| (decode; q scaled into fp16, within 2^-35 of its head's largest), each of at most 40 roundings of
2^-23 (the matrix unit truncates); their error e changes a weight by a factor within exp(2 e). Decode sums V's codes with an offset of 136 that it takes
off record by record: two products per record, each truncated within two units in the last place of partial sums that
reach 143 times the record's weights times the row's steps, so over all records at most 4 * 2^-23 * 143 times
the mean step, and as much again for the merges: 8 * 2^-23 * 143 of the largest step. It shows only where the keys
that weigh something have code 0.
"""

import numpy as np
import pytest
import torch

from oracle import serving
from oracle.attention import causal_gqa_attention, decode_attention
from oracle.deviation import bf16_bits_to_f64
from workloads.generator import f32_to_bf16_bits
from workloads.torch_io import bf16_bits, bf16_tensor

pytestmark = pytest.mark.gpu

HEADS = [(4, 2, 64), (32, 8, 128), (16, 16, 128), (32, 16, 64), (16, 1, 64), (32, 2, 128), (8, 4, 128)]


def _plan(cb, hq, hkv, d):
    return cb.Plan(1, 1, 0, hq, hkv, d, 1e4)


def _bits(rng, *shape, scale=1.0):
    return f32_to_bf16_bits((scale * rng.standard_normal(shape)).astype(np.float32))


def _f64(t):
    return bf16_bits_to_f64(bf16_bits(t))


def _i32(x):
    return torch.as_tensor(np.ascontiguousarray(np.asarray(x, dtype=np.int32))).cuda()


def _close(got, ref, vs, e, what, least=1e-30):
    err = np.abs(got - ref)
    lim = (2.0**-8 + 2 * e) * vs + (2.0**-8) * np.abs(ref) + least
    assert np.isfinite(got).all(), f"{what}: {int((~np.isfinite(got)).sum())} values are not finite"
    assert (err <= lim).all(), f"{what}: err/limit {float((err / lim).max()):.3f}"


# ---- page tables ----------------------------------------------------------------------------


def _tables(cb, plan, ctx, new, page, free, table, rows, free_from=0):
    n = len(ctx)
    t = _i32(table)
    out = dict(cu_seqlens=_i32(np.full(n + 1, -7)), kv_lens=_i32(np.full(n, -7)), positions=_i32(np.full(rows, -7)),
               slots=_i32(np.full(rows, -7)), free_to=_i32([-7]))
    args = (plan, _i32(ctx), _i32(new), page, _i32(free), t)
    cb.cb_page_tables(*args, free_from=_i32([free_from]) if free_from else None, **out)
    return [x.cpu().numpy().astype(np.int64) for x in (t, *out.values())]


@pytest.mark.parametrize("n,most_ctx,most_new,page,pad", [
    (1, 0, 1, 16, 0), (1, 16, 1, 16, 3), (3, 40, 40, 16, 0), (64, 8448, 1, 64, 0), (65, 300, 5, 48, 129),
    (513, 100, 700, 256, 1), (700, 0, 40, 1024, 0), (4099, 200, 3, 32, 11), (16384, 50, 2, 16, 5)])
def test_page_tables(cb, n, most_ctx, most_new, page, pad):
    rng = np.random.default_rng(n + page)
    plan = _plan(cb, 4, 2, 64)
    ctx, new = rng.integers(0, most_ctx + 1, n), rng.integers(0, most_new + 1, n)
    if n > 2:
        ctx[1], new[1], new[n - 1] = 0, 0, 0  # a request that holds nothing and adds nothing
    have = -(-ctx // page)
    width = int((-(-(ctx + new) // page)).max()) + 1
    ids = rng.permutation(int(have.sum() + (new + 1).sum()) + 5)
    table = np.full((n, width), -1)
    table[np.arange(width) < have[:, None]] = ids[:have.sum()]
    free = ids[have.sum():]
    got = _tables(cb, plan, ctx, new, page, free, table, int(new.sum()) + pad, free_from=2)
    plan.check()
    want = serving.page_tables(ctx.tolist(), new.tolist(), page, free, table, int(new.sum()) + pad, 2)
    for name, g, w in zip(("table", "cu", "kv_lens", "positions", "slots", "free_to"), got, want):
        assert np.array_equal(g.reshape(-1), np.asarray(w).reshape(-1)), name
    plan.close()


@pytest.mark.parametrize("shift", [0, 1, 2])
def test_page_tables_rows_at_any_address(cb, shift):
    # rows that are no multiple of four, in buffers off a 16-byte boundary, with rows before and behind them kept
    rng = np.random.default_rng(48)
    plan = _plan(cb, 4, 2, 64)
    ctx, new = rng.integers(0, 90, 9), rng.integers(0, 60, 9)
    new[3] = 0
    rows = int(new.sum()) + 6
    free, width = rng.permutation(99), 12
    have = -(-ctx // 16)
    table = np.where(np.arange(width) < have[:, None], 100 + np.arange(9 * width).reshape(9, width), -1)
    t, pos, slots = _i32(table), _i32(np.full(rows + 8, -7)), _i32(np.full(rows + 8, -7))
    cu, kv, to = _i32([0] * 10), _i32([0] * 9), _i32([0])
    cb.cb_page_tables(plan, _i32(ctx), _i32(new), 16, _i32(free), t, cu, kv, pos[shift:shift + rows], slots[shift:shift + rows], to)
    plan.check()
    want = serving.page_tables(ctx.tolist(), new.tolist(), 16, free, table, rows)
    for got, w in ((pos, want[3]), (slots, want[4])):
        got = got.cpu().numpy()
        assert np.array_equal(got[shift:shift + rows], w)
        assert (got[:shift] == -7).all() and (got[shift + rows:] == -7).all()
    assert np.array_equal(t.cpu().numpy(), want[0])
    plan.close()


def test_page_tables_without_requests_or_rows(cb):
    plan = _plan(cb, 4, 2, 64)
    t, cu, kv, pos, slots, to = _tables(cb, plan, [], [], 16, [1, 2], np.zeros((0, 4)), 5, free_from=1)
    assert cu.tolist() == [0] and slots.tolist() == [-1] * 5 and pos.tolist() == [0] * 5 and to.tolist() == [1]
    t, cu, kv, pos, slots, to = _tables(cb, plan, [3], [0], 16, [], [[5]], 0)
    assert cu.tolist() == [0, 0] and kv.tolist() == [3] and t.tolist() == [[5]] and to.tolist() == [0]
    plan.check()
    plan.close()


@pytest.mark.parametrize("case", ["free list ends", "table too narrow", "rows too few", "negative length", "bad free page",
                                  "bad held page", "negative start"])
def test_page_tables_findings(cb, case):
    plan = _plan(cb, 4, 2, 64)
    ctx, new, free, table, rows, frm = [20, 3], [20, 30], [3, 4, 5, 6], [[8, 9, -1], [7, -1, -1]], 50, 0
    if case == "free list ends":
        free = [3, 4]
    elif case == "table too narrow":
        table = [[8, 9], [7, -1]]
    elif case == "rows too few":
        rows = 25
    elif case == "negative length":
        new = [20, -30]
    elif case == "bad free page":
        free = [3, 1 << 28, -2, 6]
    elif case == "bad held page":
        table[0][1] = -1
    else:
        frm = -5
    t, cu, kv, pos, slots, to = _tables(cb, plan, ctx, new, 16, free, table, rows, free_from=frm)
    with pytest.raises(cb.CacheBlendError) as e:
        plan.check()
    assert e.value.status == 5
    clean = [0 if x < 0 else x for x in new]
    ids = [x if 0 <= x < (1 << 26) else -1 for x in free]
    wt, wcu, wkv, wpos, wslots, wto = serving.page_tables(ctx, clean, 16, ids, table, rows, max(frm, 0))
    assert np.array_equal(cu, wcu) and np.array_equal(kv, wkv) and np.array_equal(pos, wpos) and to[0] == wto
    assert np.array_equal(slots, wslots)
    if case not in ("bad free page", "rows too few"):
        assert np.array_equal(t, wt)
    plan.check()
    plan.close()


# ---- rows of the 4-bit cache ----------------------------------------------------------------


@pytest.mark.parametrize("hkv,d", [(2, 64), (8, 128), (1, 64), (3, 128), (16, 128)])
@pytest.mark.parametrize("n,page", [(1, 16), (7, 48), (130, 64), (333, 16)])
def test_store_and_load(cb, hkv, d, n, page):
    rng = np.random.default_rng(hkv * n + d)
    plan = _plan(cb, hkv, hkv, d)
    n_pages = -(-2 * n // page) + 2
    slots = rng.permutation(n_pages * page)[:n]
    if n > 3:
        slots[2] = -1
    k, v = _bits(rng, n, hkv, d), _bits(rng, n, hkv, d, scale=20.0)
    kf, vf = bf16_bits_to_f64(k), bf16_bits_to_f64(v)
    if n > 9:  # rows that a quantiser meets seldom: zeros, a single value, tiny, huge, not finite
        for x in (k, v):
            x[0] = 0
            x[1] = 0
            x[1, :, 5] = 0xC040  # -3
            x[3, :, :] = f32_to_bf16_bits((rng.standard_normal((hkv, d)) * 1e-39).astype(np.float32))
            x[4] = f32_to_bf16_bits((rng.standard_normal((hkv, d)) * 5e37).astype(np.float32))
            x[5, 0, 33] = 0x7F80
            x[6, 0, 1] = 0x7FC1
        kf, vf = bf16_bits_to_f64(k), bf16_bits_to_f64(v)
    before = rng.integers(0, 256, (n_pages, hkv, serving.page_bytes(page, d)), dtype=np.uint8)
    cache = torch.as_tensor(before).cuda()
    assert cache.shape[2] == cb.cb_kv4_page_bytes(plan, page)
    cb.cb_kv4_store(plan, bf16_tensor(k), bf16_tensor(v), _i32(slots), cache, page)
    want = before.copy()
    serving.store(want, page, slots, kf, vf)
    got = cache.cpu().numpy()
    ok, ov = (torch.full((n, hkv, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cb.cb_kv4_load(plan, cache, page, _i32(slots), ok, ov)
    plan.check()
    if n <= 9:
        assert np.array_equal(got, want)  # every byte, also those of other tokens and the unused ones
    wk, wv = serving.load(want, page, np.maximum(slots, 0), d)
    for g, w in ((_f64(ok), wk), (_f64(ov), wv)):
        w = np.where((slots >= 0)[:, None, None], serving._to_bf16(w), 7.0)
        assert np.array_equal(np.isnan(g), np.isnan(w))
        assert np.array_equal(g[~np.isnan(w)], w[~np.isnan(w)])
    # NaN scales may differ in their payload: all other bytes are the oracle's
    differ = got != want
    assert differ.sum() <= 4 * n * hkv and (n > 9 or not differ.any())
    plan.close()


@pytest.mark.parametrize("hkv,d,page", [(2, 64, 16), (3, 128, 48), (8, 128, 256)])
def test_store_and_load_by_runs(cb, hkv, d, page):
    # calls of 4,096 rows and more: whole records at any offset of the rows, broken runs, runs that begin
    # or end inside a record, padding, rows that a quantiser meets seldom, the last record of the cache
    rng = np.random.default_rng(hkv + d + page)
    plan = _plan(cb, hkv, hkv, d)
    n_pages = -(-1500 // page) + 3
    total = n_pages * page
    pieces, at = [], 0
    for size in (16, 5, 32, 11, 64, 16, 15, 17, 1, 100, 16, 240, 30, 33, 200, 7, 129):
        start = at if len(pieces) % 3 else -(-at // 16) * 16  # some pieces begin inside a record
        pieces.append(np.arange(start, start + size))
        at = start + size
        if size == 30:
            pieces.append(np.full(3, -1))
    rest = np.arange(-(-at // 16) * 16, total - 16)
    pieces.append(rng.permutation(rest)[:150])
    pieces.append(np.arange(total - 16, total))
    pieces.insert(4, np.full(1000, -1))  # padding among the rows and behind them
    pieces.append(np.full(2100, -1))
    slots = np.concatenate(pieces)
    slots[1130], slots[1300] = slots[1131], -1
    slots[1131] = -1  # (a slot that was there is named once)
    n = len(slots)
    assert n >= 4096 and len(set(slots[slots >= 0])) == (slots >= 0).sum()
    k, v = _bits(rng, n, hkv, d), _bits(rng, n, hkv, d, scale=9.0)
    for x in (k, v):
        x[3], x[40], x[41, 0] = 0, f32_to_bf16_bits((rng.standard_normal((hkv, d)) * 1e-39).astype(np.float32)), 0x8000
        x[50] = f32_to_bf16_bits((rng.standard_normal((hkv, d)) * 5e37).astype(np.float32))
        x[60, 0, 33], x[61, 1, 1] = 0xFF80, 0x7FC1
    before = rng.integers(0, 256, (n_pages, hkv, serving.page_bytes(page, d)), dtype=np.uint8)
    cache = torch.as_tensor(before).cuda()
    cb.cb_kv4_store(plan, bf16_tensor(k), bf16_tensor(v), _i32(slots), cache, page)
    want = before.copy()
    serving.store(want, page, slots, bf16_bits_to_f64(k), bf16_bits_to_f64(v))
    assert np.array_equal(cache.cpu().numpy(), want)
    ok, ov = (torch.full((n, hkv, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cb.cb_kv4_load(plan, cache, page, _i32(slots), ok, ov)
    plan.check()
    wk, wv = serving.load(want, page, np.maximum(slots, 0), d)
    for g, w in ((_f64(ok), wk), (_f64(ov), wv)):
        w = np.where((slots >= 0)[:, None, None], serving._to_bf16(w), 7.0)
        assert np.array_equal(np.isnan(g), np.isnan(w))
        assert np.array_equal(g[~np.isnan(w)], w[~np.isnan(w)])
    # one slot past the cache in a long call
    slots[1700] = total
    cb.cb_kv4_load(plan, cache, page, _i32(slots), ok, ov)
    with pytest.raises(cb.CacheBlendError):
        plan.check()
    plan.close()


@pytest.mark.parametrize("padding", [0, 3100])
def test_store_every_quotient(cb, padding):
    """Every bf16 mantissa of a group's largest magnitude with every mantissa of its other values, ties among
    them, from subnormal steps to the largest: scales and codes are those of exact arithmetic."""
    plan, hkv, d = _plan(cb, 8, 8, 128), 8, 128
    rng = np.random.default_rng(5)
    exps = [0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 20, 60, 100, 126, 127, 128, 140, 200, 240, 252, 253, 254]
    tops = (np.array(exps)[:, None] * 128 + np.arange(128)).astype(np.int64)  # bf16 bits
    others = tops[:, :, None, None] // 128 * 128 - 128 * np.arange(5)[:, None] + np.arange(128)
    others = np.minimum(np.maximum(others, 0), tops[:, :, None, None]).reshape(len(exps), 128, 640)
    groups = np.broadcast_to(tops[:, :, None, None], (len(exps), 128, 21, 32)).copy()
    groups[..., 1:] = np.concatenate((others, others[..., :11]), -1).reshape(len(exps), 128, 21, 31)
    groups = rng.permuted(groups, axis=-1) | (rng.integers(0, 2, groups.shape) << 15)
    kv = groups.astype(np.uint16).reshape(1050, 2, hkv, d)
    cache = torch.zeros(66, hkv, cb.cb_kv4_page_bytes(plan, 16), dtype=torch.uint8, device="cuda")
    k, v = (bf16_tensor(np.concatenate((kv[:, i], np.zeros((padding, hkv, d), np.uint16)))) for i in range(2))
    slots = _i32(np.concatenate((np.arange(1050), np.full(padding, -1))))
    cb.cb_kv4_store(plan, k, v, slots, cache, 16)
    kk, vv = torch.empty_like(k), torch.empty_like(v)
    cb.cb_kv4_load(plan, cache, 16, slots, kk, vv)
    for i, got in enumerate((kk, vv)):
        want = serving._to_bf16(serving.dequantise(*serving.quantise(bf16_bits_to_f64(kv[:, i]))))
        assert np.array_equal(_f64(got)[:1050], want)
    plan.check()
    plan.close()


def test_store_skips_and_records_slots_past_the_cache(cb):
    rng = np.random.default_rng(5)
    plan = _plan(cb, 4, 2, 64)
    cache = torch.zeros((2, 2, serving.page_bytes(16, 64)), dtype=torch.uint8, device="cuda")
    k = bf16_tensor(_bits(rng, 4, 2, 64))
    cb.cb_kv4_store(plan, k, k, _i32([-1, 32, 1 << 30, -(1 << 31)]), cache, 16)
    with pytest.raises(cb.CacheBlendError) as e:
        plan.check()
    assert e.value.status == 5 and not cache.any()
    out = k.clone()
    cb.cb_kv4_load(plan, cache, 16, _i32([-1, 32, 1 << 30, -5]), out, k.clone())
    with pytest.raises(cb.CacheBlendError):
        plan.check()
    assert torch.equal(out.view(torch.int16), k.view(torch.int16))
    plan.close()


def test_rows_far_into_a_large_cache(cb):
    # byte offsets past 2^32: pages at the end of a 6 GB cache
    rng = np.random.default_rng(6)
    plan = _plan(cb, 8, 8, 128)
    page = 64
    n_pages = 6 * (1 << 30) // (8 * serving.page_bytes(page, 128))
    cache = torch.empty((n_pages, 8, serving.page_bytes(page, 128)), dtype=torch.uint8, device="cuda")
    pages = np.array([n_pages - 1, 3, n_pages - 2])
    n = 3 * page
    slots = (pages[:, None] * page + np.arange(page)).reshape(-1)
    k, v = _bits(rng, n, 8, 128), _bits(rng, n, 8, 128)
    cb.cb_kv4_store(plan, bf16_tensor(k), bf16_tensor(v), _i32(slots), cache, page)
    ok, ov = (torch.empty((n, 8, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cb.cb_kv4_load(plan, cache, page, _i32(slots), ok, ov)
    qk, qv = (serving.dequantise(*serving.quantise(bf16_bits_to_f64(x))) for x in (k, v))
    assert np.array_equal(_f64(ok), serving._to_bf16(qk)) and np.array_equal(_f64(ov), serving._to_bf16(qv))
    q = _bits(rng, 1, 8, 128)
    out = torch.empty((1, 8, 128), dtype=torch.bfloat16, device="cuda")
    cb.cb_kv4_decode_attention(plan, bf16_tensor(q), cache, page, _i32(pages[None]), _i32([n - 3]), out)
    plan.check()
    ref, vs = decode_attention(bf16_bits_to_f64(q)[0], qk[:n - 3], qv[:n - 3], return_vscale=True)
    _close(_f64(out)[0], ref, vs, 1e-3, "decode at large offsets")
    plan.close()


# ---- decode over 4-bit pages ----------------------------------------------------------------


def _cache(cb, plan, rng, lens, page, spare=2, kscale=1.0, koffset=0.5):
    """A pool with the requests' rows stored to shuffled pages, every other byte random: (cache, table,
    K, V rows as the cache holds them per request)."""
    hkv, d = plan.hkv, plan.head_dim
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + spare
    ids = rng.permutation(n_pages)
    table = np.full((len(lens), max(need + [1])), -1)
    slots, at = [], 0
    for s, n in enumerate(lens):
        table[s, :need[s]] = ids[at:at + need[s]]
        at += need[s]
        pos = np.arange(n)
        slots.append(table[s][pos // page] * page + pos % page if n else np.zeros(0, int))
    total = sum(lens)
    kf = kscale * rng.standard_normal((total, hkv, d)) + koffset * rng.standard_normal((1, hkv, d))
    k, v = f32_to_bf16_bits(kf.astype(np.float32)), _bits(rng, total, hkv, d)
    cache = torch.as_tensor(rng.integers(0, 256, (n_pages, hkv, serving.page_bytes(page, d)), dtype=np.uint8)).cuda()
    if total:
        cb.cb_kv4_store(plan, bf16_tensor(k), bf16_tensor(v), _i32(np.concatenate(slots)), cache, page)
    qk, qv = (serving.dequantise(*serving.quantise(bf16_bits_to_f64(x))) for x in (k, v))
    cut = np.cumsum([0] + list(lens))
    return cache, table, [qk[a:b] for a, b in zip(cut, cut[1:])], [qv[a:b] for a, b in zip(cut, cut[1:])]


def _score_error(q, rows_scale, d, scale):
    """Bound of the fp32 error of a decode score (docstring of this file)."""
    return scale * (d / 32) * 40 * 2.0**-23 * 32 * (15 + 8) * np.abs(q).max() * rows_scale


def _check_decode(plan, q, out, ks, vs_rows, what, scale=None):
    d = plan.head_dim
    for s in range(len(ks)):
        if len(ks[s]) == 0:
            assert not _f64(out[s]).any(), f"{what}: request {s} without keys"
            continue
        ref, vs = decode_attention(bf16_bits_to_f64(q)[s], ks[s], vs_rows[s], scale=scale, return_vscale=True)
        e = _score_error(bf16_bits_to_f64(q)[s], np.abs(ks[s]).max() / 7, d, scale or d**-0.5)
        step = np.abs(vs_rows[s]).reshape(len(vs_rows[s]), -1, d // 32, 32).max((0, 3)) / 7  # [hkv, groups]
        least = np.repeat(np.repeat(8 * 2.0**-23 * 143 * step, 32, axis=1), plan.hq // plan.hkv, axis=0) + 1e-30
        _close(_f64(out[s]), ref, vs, min(e, 0.01), f"{what}, request {s} of {len(ks[s])} keys", least)


@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("lens,page", [([1], 16), ([0], 16), ([15, 16, 17], 16), ([33, 0, 1, 100, 48], 48),
                                       ([700, 3, 0, 0, 257], 64), ([2500], 256), ([5] * 40, 16)])
def test_decode_lengths_and_heads(cb, hq, hkv, d, lens, page):
    rng = np.random.default_rng(hq + hkv + d + sum(lens))
    plan = _plan(cb, hq, hkv, d)
    cache, table, ks, vs = _cache(cb, plan, rng, lens, page)
    q = _bits(rng, len(lens), hq, d)
    out = torch.full((len(lens), hq, d), 9.0, dtype=torch.bfloat16, device="cuda")
    cb.cb_kv4_decode_attention(plan, bf16_tensor(q), cache, page, _i32(table), _i32(lens), out)
    plan.check()
    _check_decode(plan, q, out, ks, vs, "decode")
    first = out.clone()
    out.fill_(4.0)
    cb.cb_kv4_decode_attention(plan, bf16_tensor(q), cache, page, _i32(table), _i32(lens), out)
    assert torch.equal(first.view(torch.int16), out.view(torch.int16))  # the same bits from call to call
    plan.close()


@pytest.mark.parametrize("hq,hkv,d,n,page", [(32, 8, 128, 32897, 64), (16, 1, 64, 20011, 128), (4, 2, 64, 9000, 16)])
def test_decode_long_request(cb, hq, hkv, d, n, page):
    rng = np.random.default_rng(n)
    plan = _plan(cb, hq, hkv, d)
    cache, table, ks, vs = _cache(cb, plan, rng, [n], page)
    q = _bits(rng, 1, hq, d)
    out = torch.empty((1, hq, d), dtype=torch.bfloat16, device="cuda")
    cb.cb_kv4_decode_attention(plan, bf16_tensor(q), cache, page, _i32(table), _i32([n]), out)
    plan.check()
    _check_decode(plan, q, out, ks, vs, "long decode")
    cb.cb_kv4_decode_attention(plan, bf16_tensor(q), cache, page, _i32(table), _i32([4321]), out, scale=0.02)
    plan.check()
    _check_decode(plan, q, out, [ks[0][:4321]], [vs[0][:4321]], "shorter, custom scale", scale=0.02)
    plan.close()


def test_decode_batch_of_many_lengths(cb):
    rng = np.random.default_rng(12)
    plan = _plan(cb, 32, 8, 128)
    lens = [int(x) for x in rng.integers(0, 1500, 90)]
    cache, table, ks, vs = _cache(cb, plan, rng, lens, 32)
    q = _bits(rng, len(lens), 32, 128)
    out = torch.empty((len(lens), 32, 128), dtype=torch.bfloat16, device="cuda")
    cb.cb_kv4_decode_attention(plan, bf16_tensor(q), cache, 32, _i32(table), _i32(lens), out)
    plan.check()
    _check_decode(plan, q, out, ks, vs, "batch")
    plan.close()


def test_decode_scores_that_jump_late(cb):
    # keys aligned with their heads' queries far into the cache: the running max moves by large steps,
    # within a warp's run and between the partials that are merged
    rng = np.random.default_rng(13)
    hq, hkv, d, page, n = 8, 2, 128, 64, 6000
    plan = _plan(cb, hq, hkv, d)
    q = _bits(rng, 1, hq, d)
    qf = bf16_bits_to_f64(q).reshape(hkv, hq // hkv, d).mean(1)
    kf = 0.3 * rng.standard_normal((n, hkv, d))
    for at, size in ((40, 2.0), (41, 6.0), (3000, 12.0), (n - 1, 14.0)):
        kf[at] = size * qf
    k, v = f32_to_bf16_bits(kf.astype(np.float32)), _bits(rng, n, hkv, d)
    table = rng.permutation(-(-n // page))[None]
    cache = torch.zeros((table.size, hkv, serving.page_bytes(page, d)), dtype=torch.uint8, device="cuda")
    pos = np.arange(n)
    cb.cb_kv4_store(plan, bf16_tensor(k), bf16_tensor(v), _i32(table[0][pos // page] * page + pos % page), cache, page)
    qk, qv = (serving.dequantise(*serving.quantise(bf16_bits_to_f64(x))) for x in (k, v))
    out = torch.empty((1, hq, d), dtype=torch.bfloat16, device="cuda")
    cb.cb_kv4_decode_attention(plan, bf16_tensor(q), cache, page, _i32(table), _i32([n]), out)
    plan.check()
    _check_decode(plan, q, out, [qk], [qv], "late jumps")
    plan.close()


@pytest.mark.parametrize("q_power,spike", [(-100, 1), (100, 1), (0, 2**12), (-130, 2**6), (20, 2**20)])
def test_decode_queries_far_from_one(cb, q_power, spike):
    # magnitudes of q from 2^-130 to 2^120 with keys that bring the scores back to the order of one, heads of
    # one group that lie far apart, and values beside one that is much larger, where K is much smaller
    rng = np.random.default_rng(abs(q_power) + spike)
    hq, hkv, d, page, lens = 8, 2, 128, 16, [37, 200]
    plan = _plan(cb, hq, hkv, d)
    n_pages = sum(-(-n // page) for n in lens)
    table = np.full((2, 13), -1)
    table[0, :3], table[1] = [5, 2, 9], np.setdiff1d(np.arange(n_pages), [5, 2, 9])
    cache = torch.zeros(n_pages, hkv, cb.cb_kv4_page_bytes(plan, page), dtype=torch.uint8, device="cuda")
    q, k = rng.standard_normal((2, hq, d)), rng.standard_normal((sum(lens), hkv, d))
    q[:, :, 64:96] *= spike  # a group of dims: K's scale there is its own
    k[:, :, 64:96] /= spike
    q[:, :, 65:96] /= spike  # small values beside a large one: next to nothing
    q[:, 1::4] *= 2.0**-10
    q, k = (f32_to_bf16_bits((x * 2.0**p).astype(np.float32)) for x, p in ((q, q_power), (k, -max(q_power, -120))))
    v = _bits(rng, sum(lens), hkv, d)
    pos = [np.arange(n) for n in lens]
    slots = np.concatenate([table[s][p // page] * page + p % page for s, p in enumerate(pos)])
    cb.cb_kv4_store(plan, bf16_tensor(k), bf16_tensor(v), _i32(slots), cache, page)
    out = torch.empty(2, hq, d, dtype=torch.bfloat16, device="cuda")
    cb.cb_kv4_decode_attention(plan, bf16_tensor(q), cache, page, _i32(table), _i32(lens), out)
    plan.check()
    qk, qv = (serving.dequantise(*serving.quantise(bf16_bits_to_f64(x))) for x in (k, v))
    qf = bf16_bits_to_f64(q)
    for s, (a, b) in enumerate(((0, 37), (37, 237))):
        ref, vs = decode_attention(qf[s], qk[a:b], qv[a:b], return_vscale=True)
        # per (head, group of dims), as in _score_error; q itself is within 2^-35 of its head's largest
        top = np.abs(qk[a:b]).max(0).reshape(hkv, 4, 32).max(-1) / 7
        sums = np.abs(qf[s]).reshape(hkv, hq // hkv, 4, 32).max(-1)
        e = (sums * (32 * (15 + 8) * 40 * 2.0**-23) + 2.0**-35 * 32 * 7 * sums.max(-1, keepdims=True)) * top[:, None]
        _close(_f64(out[s]), ref, vs, min(d**-0.5 * e.sum(-1).max(), 0.02), f"request {s}")
    plan.close()


@pytest.mark.parametrize("scale", [1e-30, 0.02, 3.0])
def test_decode_scales_and_a_zero_query(cb, scale):
    # head 1 asks with zeros: every key weighs the same, also at a scale whose product with q's power underflows
    rng = np.random.default_rng(47)
    plan = _plan(cb, 8, 2, 64)
    lens = [21, 300]
    cache, table, ks, vs = _cache(cb, plan, rng, lens, 16)
    q = _bits(rng, 2, 8, 64)
    q[:, 1] = 0
    out = torch.empty((2, 8, 64), dtype=torch.bfloat16, device="cuda")
    cb.cb_kv4_decode_attention(plan, bf16_tensor(q), cache, 16, _i32(table), _i32(lens), out, scale=scale)
    plan.check()
    _check_decode(plan, q, out, ks, vs, f"scale {scale}", scale=scale)
    plan.close()


def test_decode_rows_that_are_not_finite_stay_with_their_request(cb):
    rng = np.random.default_rng(14)
    plan = _plan(cb, 8, 2, 64)
    lens, page = [40, 40, 21], 16
    cache, table, ks, vs = _cache(cb, plan, rng, lens, page)
    bad = _bits(rng, 2, 2, 64)
    bad[0, 0, 3], bad[1, 0, 3] = 0x7F80, 0x7FC0
    # one inside request 1, one in the unused part of request 2's last page (position 21)
    slots = [table[1, 1] * page + 2, table[2, 1] * page + 5]
    cb.cb_kv4_store(plan, bf16_tensor(bad), bf16_tensor(bad), _i32(slots), cache, page)
    q = _bits(rng, 3, 8, 64)
    out = torch.empty((3, 8, 64), dtype=torch.bfloat16, device="cuda")
    cb.cb_kv4_decode_attention(plan, bf16_tensor(q), cache, page, _i32(table), _i32(lens), out)
    plan.check()
    got = _f64(out)
    assert np.isnan(got[1, :4]).all()  # kv head 0 of request 1: its scores hold a NaN
    assert np.isfinite(got[[0, 2]]).all() and np.isfinite(got[1, 4:]).all()
    for s in (0, 2):
        ref, sc = decode_attention(bf16_bits_to_f64(q)[s], ks[s], vs[s], return_vscale=True)
        _close(got[s], ref, sc, 1e-3, f"request {s}")
    plan.close()


def test_decode_bad_pages_and_lengths_are_left_out_and_recorded(cb):
    rng = np.random.default_rng(15)
    plan = _plan(cb, 8, 2, 128)
    lens, page = [64, 40, 30], 16
    cache, table, ks, vs = _cache(cb, plan, rng, lens, page)
    q = _bits(rng, 3, 8, 128)
    out = torch.empty((3, 8, 128), dtype=torch.bfloat16, device="cuda")
    broken = table.copy()
    broken[0, 1], broken[0, 2] = cache.shape[0], -3
    cb.cb_kv4_decode_attention(plan, bf16_tensor(q), cache, page, _i32(broken), _i32(lens), out)
    with pytest.raises(cb.CacheBlendError) as e:
        plan.check()
    assert e.value.status == 5
    keep = np.r_[0:16, 48:64]
    _check_decode(plan, q, out, [ks[0][keep], ks[1], ks[2]], [vs[0][keep], vs[1], vs[2]], "bad pages")
    cb.cb_kv4_decode_attention(plan, bf16_tensor(q), cache, page, _i32(table), _i32([1000, -5, 30]), out)
    with pytest.raises(cb.CacheBlendError):
        plan.check()
    _check_decode(plan, q, out, [ks[0], [], ks[2]], [vs[0], [], vs[2]], "bad lengths")
    cb.cb_kv4_decode_attention(plan, bf16_tensor(q), cache, page, _i32(table), _i32(lens), out)
    plan.check()  # and the plan works as before
    _check_decode(plan, q, out, ks, vs, "after")
    plan.close()


# ---- packed prompts -------------------------------------------------------------------------


def _prompt(cb, plan, q, k, v, cu, scale=0.0, out=None):
    out = torch.full(q.shape, 9.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    cb.cb_prompt_attention(plan, bf16_tensor(q), bf16_tensor(k), bf16_tensor(v), _i32(cu), out, scale=scale)
    return out


def _check_prompt(q, k, v, cu, out, what, scale=None):
    qf, kf, vf = (bf16_bits_to_f64(x) for x in (q, k, v))
    ref, vs = serving.packed_attention(qf, kf, vf, cu, scale=scale)
    got = _f64(out)
    inside = np.zeros(len(q), bool)
    for a, b in zip(cu, cu[1:]):
        inside[a:b] = True
    assert (got[~inside] == 9.0).all(), f"{what}: rows of no sequence were written"
    d = q.shape[2]
    e = (scale or d**-0.5) * 40 * 2.0**-23 * d * np.abs(qf).max() * np.abs(kf).max()
    _close(got[inside], ref[inside], vs[inside], min(e, 0.01), what)


@pytest.mark.parametrize("hq,hkv,d", HEADS + [(64, 8, 128)])
@pytest.mark.parametrize("lens,pad", [([1], 0), ([1, 1, 1], 5), ([0, 5, 0], 1), ([127, 128, 129], 0), ([64, 65, 63, 1, 300], 17),
                                      ([513], 3), ([256, 0, 31, 32, 33], 0)])
def test_prompt_lengths_and_heads(cb, hq, hkv, d, lens, pad):
    rng = np.random.default_rng(hq + d + sum(lens))
    plan = _plan(cb, hq, hkv, d)
    n = sum(lens) + pad
    q, k, v = _bits(rng, n, hq, d), _bits(rng, n, hkv, d), _bits(rng, n, hkv, d)
    cu = np.cumsum([0] + lens)
    out = _prompt(cb, plan, q, k, v, cu)
    plan.check()
    _check_prompt(q, k, v, cu, out, "prompt")
    plan.close()


@pytest.mark.parametrize("lens", [[2100], [1500, 40, 700, 0, 1, 900], [31] * 70])
def test_prompt_more_items_than_sms(cb, lens):
    rng = np.random.default_rng(sum(lens))
    plan = _plan(cb, 32, 8, 128)
    n = sum(lens)
    q, k, v = _bits(rng, n, 32, 128), _bits(rng, n, 8, 128), _bits(rng, n, 8, 128)
    cu = np.cumsum([0] + lens)
    out = _prompt(cb, plan, q, k, v, cu, scale=0.05)
    plan.check()
    _check_prompt(q, k, v, cu, out, "prompt", scale=0.05)
    again = _prompt(cb, plan, q, k, v, cu, scale=0.05)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    plan.close()


def test_prompt_many_sequences(cb):
    rng = np.random.default_rng(30)
    plan = _plan(cb, 4, 2, 64)
    lens = [int(x) for x in rng.integers(0, 40, 1500)]
    n = sum(lens) + 2
    q, k, v = _bits(rng, n, 4, 64), _bits(rng, n, 2, 64), _bits(rng, n, 2, 64)
    cu = np.cumsum([0] + lens)
    out = _prompt(cb, plan, q, k, v, cu)
    plan.check()
    _check_prompt(q, k, v, cu, out, "many sequences")
    plan.close()


def test_prompt_long_sequences_in_groups_of_two(cb):
    # K and V of 20 MB at the mean length: the order of the work goes by two sequences at a time
    rng = np.random.default_rng(46)
    plan = _plan(cb, 16, 16, 128)
    lens = [2600, 0, 3300, 2450, 3900, 2450]
    cu, rows = np.cumsum([0] + lens), sum(lens)
    q, k, v = (_bits(rng, rows, 16, 128) for _ in range(3))
    out = torch.full((rows, 16, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    cb.cb_prompt_attention(plan, bf16_tensor(q), bf16_tensor(k), bf16_tensor(v), _i32(cu), out)
    plan.check()
    qf, kf, vf, got = bf16_bits_to_f64(q), bf16_bits_to_f64(k), bf16_bits_to_f64(v), _f64(out)
    for a, b in zip(cu, cu[1:]):  # every 37th row of each, and its ends
        at = np.unique(np.r_[np.arange(0, b - a, 37), b - a - 1]) if b > a else np.zeros(0, int)
        if not len(at):
            continue
        ref, vs = causal_gqa_attention(qf[a + at], at, kf[a:b], vf[a:b], return_vscale=True)
        _close(got[a + at], ref, vs, 40 * 2.0**-23 * 128**0.5 * np.abs(qf).max() * np.abs(kf).max(), f"rows from {a}")
    plan.close()


def test_prompt_first_offset_and_unaligned_output(cb):
    # the first sequence starts behind row 0; the output is 16-byte but not 32-byte aligned
    rng = np.random.default_rng(31)
    plan = _plan(cb, 8, 2, 64)
    cu = np.array([6, 106, 170])
    q, k, v = _bits(rng, 190, 8, 64), _bits(rng, 190, 2, 64), _bits(rng, 190, 2, 64)
    whole = torch.full((190 * 8 * 64 + 8,), 9.0, dtype=torch.bfloat16, device="cuda")
    out = _prompt(cb, plan, q, k, v, cu, out=whole[8:].view(190, 8, 64))
    plan.check()
    _check_prompt(q, k, v, cu, out, "unaligned")
    assert (whole[:8] == 9.0).all()
    plan.close()


def test_prompt_scores_that_jump(cb):
    # keys aligned with the queries in later key tiles: the softmax's reference has to move
    rng = np.random.default_rng(32)
    hq, hkv, d, n = 8, 2, 128, 700
    plan = _plan(cb, hq, hkv, d)
    q = _bits(rng, n, hq, d)
    base = rng.standard_normal((hkv, d))
    qf = 0.5 * rng.standard_normal((n, hq, d)) + np.repeat(base, hq // hkv, 0)
    q = f32_to_bf16_bits(qf.astype(np.float32))
    kf = 0.3 * rng.standard_normal((n, hkv, d))
    for at, size in ((3, 0.5), (130, 1.5), (300, 3.0), (301, -3.0), (511, 5.0), (640, 9.0)):
        kf[at] = size * base
    k, v = f32_to_bf16_bits(kf.astype(np.float32)), _bits(rng, n, hkv, d)
    out = _prompt(cb, plan, q, k, v, [0, n])
    plan.check()
    _check_prompt(q, k, v, [0, n], out, "jumps")
    plan.close()


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (32, 8, 128), (4, 4, 128)])
def test_prompt_values_that_are_not_finite_reach_only_rows_that_see_them(cb, hq, hkv, d):
    rng = np.random.default_rng(33)
    plan = _plan(cb, hq, hkv, d)
    lens, pad = [70, 100, 300], 30
    n = sum(lens) + pad
    cu = np.cumsum([0] + lens)
    q, k, v = _bits(rng, n, hq, d), _bits(rng, n, hkv, d), _bits(rng, n, hkv, d)
    clean_k, clean_v = k.copy(), v.copy()
    k[470:], v[470:] = 0x7FC0, 0x7F80  # behind the last sequence
    v[90, 1, 5], k[95, 1, 7] = 0x7FC0, 0x7F80  # in sequence 1, at its tokens 20 and 25
    v[170 + 250, 0, 9] = 0xFF80  # -inf in sequence 2, at its token 250
    v[170 + 20, 1, 11], v[170 + 220, 1, 11] = 0x7F80, 0xFF80  # +inf, then -inf: NaN from token 220 on
    out = _prompt(cb, plan, q, k, v, cu)
    plan.check()
    got = _f64(out)
    ref, vs = serving.packed_attention(*(bf16_bits_to_f64(x) for x in (q, clean_k, clean_v)), cu)
    g = hq // hkv
    want_nan = np.zeros(got.shape, bool)
    want_inf = np.zeros(got.shape)
    want_nan[90:170, g:2 * g, 5] = True
    want_nan[95:170, g:2 * g, :] |= bf16_bits_to_f64(q)[95:170, g:2 * g, 7:8] > 0  # a score of +inf
    want_inf[420:470, :g, 9] = -np.inf
    want_inf[190:390, g:2 * g, 11] = np.inf
    want_nan[390:470, g:2 * g, 11] = True
    # an infinite key gives a score of +inf (NaN weights) or -inf (no weight: that row stays finite)
    row_inf = np.zeros(got.shape, bool)
    row_inf[95:170, g:2 * g, :] = True
    assert np.isnan(got[want_nan]).all()
    fixed = (want_inf != 0) & ~want_nan
    assert np.array_equal(got[fixed], want_inf[fixed])
    rest = ~want_nan & ~fixed & ~row_inf
    rest[470:] = False
    assert np.isfinite(got[rest]).all()
    err = np.abs(got - ref)[rest]
    assert (err <= (2.0**-8 + 0.002) * vs[rest] + 2.0**-8 * np.abs(ref[rest])).all()
    assert (got[470:] == 9.0).all()
    plan.close()


def test_prompt_offsets_that_fall_or_leave_the_rows(cb):
    rng = np.random.default_rng(34)
    plan = _plan(cb, 8, 2, 128)
    q, k, v = _bits(rng, 100, 8, 128), _bits(rng, 100, 2, 128), _bits(rng, 100, 2, 128)
    for cu, clean in (([0, 60, 140], [0, 60, 100]), ([-4, 50, 100], [0, 50, 100]), ([0, 70, 50, 50], [0, 70]),
                      ([200, 300], [100])):
        out = _prompt(cb, plan, q, k, v, cu)
        with pytest.raises(cb.CacheBlendError) as e:
            plan.check()
        assert e.value.status == 5
        _check_prompt(q, k, v, clean, out, f"offsets {cu}")
    plan.close()


# ---- together ---------------------------------------------------------------------------------


def test_serving_a_batch_end_to_end(cb):
    """Three prompts are laid out, encoded, attended and cached in 4 bits, then two decode steps follow,
    the second and later ones as one captured graph; every step against the oracle."""
    from oracle.rope import rope_rotate

    hq, hkv, d, page, theta = 8, 2, 128, 32, 1e4
    rng = np.random.default_rng(40)
    plan = cb.Plan(1, 512, 0, hq, hkv, d, theta)
    lens, width, pool = [75, 0, 200], 9, 24
    n = len(lens)
    free = rng.permutation(pool)
    cache = torch.as_tensor(rng.integers(0, 256, (pool, hkv, serving.page_bytes(page, d)), dtype=np.uint8)).cuda()
    table = _i32(np.full((n, width), -1))
    ctx, kv, new, frm, to = _i32([0] * n), _i32([0] * n), _i32(lens), _i32([0]), _i32([0])
    host_k, host_v = [[] for _ in lens], [[] for _ in lens]

    def bufs(rows):
        return {"cu_seqlens": _i32(np.zeros(n + 1)), "positions": _i32(np.zeros(rows)), "slots": _i32(np.zeros(rows))}

    def lay_out(b):
        cb.cb_page_tables(plan, ctx, new, page, _i32_free, table, kv_lens=kv, free_to=to, free_from=frm, **b)

    _i32_free = _i32(free)
    # the prompts: 275 rows in buffers of 300
    rows = 300
    b = bufs(rows)
    q0, k0, v0 = _bits(rng, rows, hq, d), _bits(rng, rows, hkv, d), _bits(rng, rows, hkv, d)
    q, k, v = bf16_tensor(q0), bf16_tensor(k0), bf16_tensor(v0)
    lay_out(b)
    qe, ke = torch.empty_like(q), torch.empty_like(k)
    cb.cb_rope_rerotate(plan, qe, q, b["positions"])
    cb.cb_rope_rerotate(plan, ke, k, b["positions"])
    out = torch.full_like(q, 9.0)
    cb.cb_prompt_attention(plan, qe, ke, v, b["cu_seqlens"], out)
    cb.cb_kv4_store(plan, ke, v, b["slots"], cache, page)
    plan.check()
    cu = np.cumsum([0] + lens)
    assert b["cu_seqlens"].cpu().numpy().tolist() == cu.tolist() and kv.cpu().numpy().tolist() == lens
    pos = np.concatenate([np.arange(x) for x in lens])
    assert np.array_equal(b["positions"].cpu().numpy()[:275], pos)
    ref = rope_rotate(bf16_bits_to_f64(k0[:275]), pos, theta, "half")
    assert np.abs(_f64(ke)[:275] - ref).max() <= 2e-2 + 1e-2 * np.abs(ref).max()
    _check_prompt(bf16_bits(qe), bf16_bits(ke), v0, cu, out, "prompts")
    for s in range(n):
        host_k[s] = [bf16_bits(ke)[cu[s]:cu[s + 1]]]
        host_v[s] = [v0[cu[s]:cu[s + 1]]]
    # decode steps: request 1 joins with its first token, request 2 crosses a page
    b = bufs(n)
    q1, k1, v1 = (torch.zeros((n, h, d), dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv))
    qe, ke, out = torch.empty_like(q1), torch.empty_like(k1), torch.empty_like(q1)
    new.fill_(1)

    def decode_step():
        ctx.copy_(kv)
        frm.copy_(to)
        lay_out(b)
        cb.cb_rope_rerotate(plan, qe, q1, b["positions"])
        cb.cb_rope_rerotate(plan, ke, k1, b["positions"])
        cb.cb_kv4_store(plan, ke, v1, b["slots"], cache, page)
        cb.cb_kv4_decode_attention(plan, qe, cache, page, table, kv, out)

    graph = None
    for step in range(26):
        q0, k0, v0 = _bits(rng, n, hq, d), _bits(rng, n, hkv, d), _bits(rng, n, hkv, d)
        for dst, src in ((q1, q0), (k1, k0), (v1, v0)):
            dst.copy_(bf16_tensor(src))
        if step == 0:
            decode_step()
        elif graph is None:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                decode_step()
        if graph is not None:
            graph.replay()
        plan.check()
        for s in range(n):
            host_k[s].append(bf16_bits(ke)[s:s + 1])
            host_v[s].append(v0[s:s + 1])
        if step in (0, 1, 24, 25):
            ks, vs = ([serving.dequantise(*serving.quantise(bf16_bits_to_f64(np.concatenate(x)))) for x in h]
                      for h in (host_k, host_v))
            assert kv.cpu().numpy().tolist() == [len(x) for x in ks]
            _check_decode(plan, bf16_bits(qe), out, ks, vs, f"decode step {step}")
    # the first request's chunk read back for a blend
    slots = _i32(table.cpu().numpy()[0][np.arange(75) // page] * page + np.arange(75) % page)
    ko, vo = (torch.empty((75, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cb.cb_kv4_load(plan, cache, page, slots, ko, vo)
    plan.check()
    want = serving._to_bf16(serving.dequantise(*serving.quantise(bf16_bits_to_f64(host_k[0][0]))))
    assert np.array_equal(_f64(ko), want)
    plan.close()


def test_calls_on_another_stream(cb):
    rng = np.random.default_rng(41)
    plan = _plan(cb, 8, 2, 64)
    lens, page = [90, 33], 16
    cache, table, ks, vs = _cache(cb, plan, rng, lens, page)
    q = _bits(rng, 2, 8, 64)
    out = torch.empty((2, 8, 64), dtype=torch.bfloat16, device="cuda")
    dq, dt, dl = bf16_tensor(q), _i32(table), _i32(lens)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        cb.cb_kv4_decode_attention(plan, dq, cache, page, dt, dl, out)
    cb.cb_kv4_decode_attention(plan, dq, cache, page, dt, dl, out, stream=side)
    side.synchronize()
    plan.check()
    _check_decode(plan, q, out, ks, vs, "another stream")
    plan.close()


def test_two_calls_of_one_plan_at_once(cb):
    # page tables and packed prompts have no scratch: two streams, one plan, many calls in flight
    rng = np.random.default_rng(42)
    plan = _plan(cb, 8, 2, 64)
    jobs = []
    for lens in ([300, 7, 1000], [64] * 20):
        n, rows = len(lens), sum(lens)
        q, k, v = _bits(rng, rows, 8, 64), _bits(rng, rows, 2, 64), _bits(rng, rows, 2, 64)
        table = np.full((n, 70), -1)
        free = rng.permutation(200)
        t = dict(ctx=_i32([0] * n), new=_i32(lens), free=_i32(free), table=_i32(table), cu=_i32(np.zeros(n + 1)), kv=_i32([0] * n),
                 pos=_i32(np.zeros(rows)), slots=_i32(np.zeros(rows)), to=_i32([0]))
        jobs.append((lens, free, table, (q, k, v), t, [bf16_tensor(x) for x in (q, k, v)],
                     torch.empty(rows, 8, 64, dtype=torch.bfloat16, device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for lens, free, table, _, t, dev, out, s in jobs:
            cb.cb_page_tables(plan, t["ctx"], t["new"], 16, t["free"], t["table"], t["cu"], t["kv"], t["pos"], t["slots"], t["to"],
                              stream=s)
            cb.cb_prompt_attention(plan, *dev, t["cu"], out, stream=s)
    torch.cuda.synchronize()
    plan.check()
    for lens, free, table, (q, k, v), t, _, out, _ in jobs:
        want = serving.page_tables([0] * len(lens), lens, 16, free, table, sum(lens))
        for w, name in zip(want, ("table", "cu", "kv", "pos", "slots", "to")):
            assert np.array_equal(t[name].cpu().numpy().reshape(-1), np.asarray(w).reshape(-1)), name
        _check_prompt(q, k, v, np.cumsum([0] + lens), out, "two at once")
    plan.close()


def test_decodes_of_two_plans_at_once_and_shared_pages(cb):
    rng = np.random.default_rng(43)
    jobs = []
    for lens in ([5000, 40], [900] * 6):
        plan = _plan(cb, 8, 2, 128)
        cache, table, ks, vs = _cache(cb, plan, rng, lens, 16)
        # a further request that shares the first one's pages, cut inside a record
        table, lens = np.concatenate((table, table[:1])), lens + [lens[0] - 21]
        ks, vs = ks + [ks[0][:lens[-1]]], vs + [vs[0][:lens[-1]]]
        q = _bits(rng, len(lens), 8, 128)
        jobs.append((plan, cache, _i32(table), _i32(lens), q, bf16_tensor(q), ks, vs,
                     torch.empty(len(lens), 8, 128, dtype=torch.bfloat16, device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for plan, cache, table, lens, _, q, _, _, out, s in jobs:
            cb.cb_kv4_decode_attention(plan, q, cache, 16, table, lens, out, stream=s)
    torch.cuda.synchronize()
    for plan, _, _, _, q, _, ks, vs, out, _ in jobs:
        plan.check()
        _check_decode(plan, q, out, ks, vs, "two plans")
        plan.close()


def test_captured_prompts_of_other_lengths(cb):
    # one graph, captured for 2,000 rows and 8 sequences, replayed for batches that leave most of them empty
    rng = np.random.default_rng(44)
    plan = _plan(cb, 8, 2, 128)
    rows = 2000
    q, k, v = _bits(rng, rows, 8, 128), _bits(rng, rows, 2, 128), _bits(rng, rows, 2, 128)
    dev, cu = [bf16_tensor(x) for x in (q, k, v)], _i32(np.zeros(9))
    out = torch.full((rows, 8, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    cb.cb_prompt_attention(plan, *dev, cu, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cb.cb_prompt_attention(plan, *dev, cu, out)
    for lens in ([0] * 8, [1] + [0] * 7, [500, 0, 1, 64, 65, 0, 1300, 70], [0] * 7 + [2000], [3, 0, 0, 0, 0, 0, 0, 130]):
        cu.copy_(_i32(np.cumsum([0] + lens)))
        out.fill_(9.0)
        graph.replay()
        plan.check()
        _check_prompt(q, k, v, np.cumsum([0] + lens), out, f"lengths {lens}")
        assert (_f64(out)[sum(lens):] == 9.0).all()
    plan.close()


@pytest.mark.parametrize("n", [40, 4400])
def test_store_of_one_slot_named_twice(cb, n):
    # what that slot holds is open; every other slot is as it would be
    rng = np.random.default_rng(45)
    plan, page = _plan(cb, 2, 2, 64), 16
    slots = np.arange(n)
    slots[32:40], slots[17] = np.arange(8), 3
    k, v = _bits(rng, n, 2, 64), _bits(rng, n, 2, 64)
    cache = torch.zeros(n // page + 1, 2, cb.cb_kv4_page_bytes(plan, page), dtype=torch.uint8, device="cuda")
    cb.cb_kv4_store(plan, bf16_tensor(k), bf16_tensor(v), _i32(slots), cache, page)
    ok, ov = (torch.empty((n, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cb.cb_kv4_load(plan, cache, page, _i32(slots), ok, ov)
    plan.check()
    once = slots > 7
    for x, got in ((k, ok), (v, ov)):
        want = serving._to_bf16(serving.dequantise(*serving.quantise(bf16_bits_to_f64(x))))
        assert np.array_equal(_f64(got)[once], want[once])
    plan.close()


def test_binding_refuses_wrong_tensors(cb):
    plan = _plan(cb, 8, 2, 128)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = torch.zeros((3, 2, 18 * 128), dtype=torch.uint8, device="cuda")
    k, t, n = bf(4, 2, 128), i32(2, 3), i32(2)
    for args, said in (((bf(4, 3, 128), k, i32(4), cache), "k must have shape"),
                       ((k, bf(4, 128, 2).transpose(1, 2), i32(4), cache), "v must be contiguous"),
                       ((k, k, i32(5), cache), "k must have shape"), ((k, k.float(), i32(4), cache), "v must be torch.bfloat16"),
                       ((k, k, i32(4).long(), cache), "slots must be torch.int32"),
                       ((k, k.cpu(), i32(4), cache), "v must be on a CUDA device")):
        with pytest.raises(ValueError, match=said):
            cb.cb_kv4_store(plan, *args, 16)
    for q, table, out, said in ((bf(3, 8, 128), t, bf(2, 8, 128), "q must have shape"), (bf(2, 8, 128), i32(3, 3), bf(2, 8, 128), "table"),
                                (bf(2, 8, 128), t, bf(2, 8, 64), "out must have shape")):
        with pytest.raises(ValueError, match=said):
            cb.cb_kv4_decode_attention(plan, q, cache, 16, table, n, out)
    q = bf(5, 8, 128)
    for kk, vv, cu, out, said in ((bf(4, 2, 128), bf(5, 2, 128), n, q.clone(), "k must have shape"),
                                  (bf(5, 2, 128), bf(5, 2, 64), n, q.clone(), "v must have shape"),
                                  (bf(5, 2, 128), bf(5, 2, 128), n.float(), q.clone(), "cu_seqlens must be torch.int32"),
                                  (bf(5, 2, 128), bf(5, 2, 128), n, bf(5, 8, 256)[:, :, ::2], "out must be contiguous")):
        with pytest.raises(ValueError, match=said):
            cb.cb_prompt_attention(plan, q, kk, vv, cu, out)
    with pytest.raises(cb.CacheBlendError, match="out must not be"):
        cb.cb_prompt_attention(plan, q, bf(5, 2, 128), bf(5, 2, 128), n, q)
    with pytest.raises(ValueError, match="new_lens must have shape"):
        cb.cb_page_tables(plan, i32(3), n, 16, i32(9), i32(3, 4), i32(4), i32(3), i32(5), i32(5), i32(1))
    with pytest.raises(ValueError, match="cu_seqlens must have shape"):
        cb.cb_page_tables(plan, i32(3), i32(3), 16, i32(9), i32(3, 4), i32(3), i32(3), i32(5), i32(5), i32(1))
    with pytest.raises(cb.CacheBlendError, match="free_to is NULL"):
        cb.cb_page_tables(plan, i32(3), i32(3), 16, i32(9), i32(3, 4), i32(4), i32(3), i32(5), i32(5), None)
    plan.check()
    plan.close()


# ---- values that are not finite, however the batch is split --------------------------------------


@pytest.mark.parametrize("others", [[], [0] * 3 + [7000], [30, 9000, 9000, 9000], [600] * 60])
def test_decode_value_that_is_not_finite_under_a_weight_of_nothing(cb, others):
    # Keys 96 to 511 of request 0 score 180 below the others: e^-180 is 0 in 32 bits. One of their values is NaN, which
    # every split of the batch (runs of 1 to 4 records per warp, within one CTA or over several) has to show, in its group
    # alone.
    rng = np.random.default_rng(50 + len(others))
    hq, hkv, d, page = 8, 2, 128, 32
    plan = _plan(cb, hq, hkv, d)
    lens = [640] + others
    cache, table, ks, vs = _cache(cb, plan, rng, lens, page)
    base = np.sign(rng.standard_normal((hkv, d)))
    q = _bits(rng, len(lens), hq, d)
    q[0] = f32_to_bf16_bits(np.repeat(base, hq // hkv, 0).astype(np.float32))
    low = (np.arange(640) >= 96) & (np.arange(640) < 512)
    k = f32_to_bf16_bits((np.where(low, -8.0, 8.0)[:, None, None] * base + 0.1 * rng.standard_normal((640, hkv, d)))
                         .astype(np.float32))
    v = _bits(rng, 640, hkv, d)
    slots = _i32(table[0][np.arange(640) // page] * page + np.arange(640) % page)
    cb.cb_kv4_store(plan, bf16_tensor(k), bf16_tensor(v), slots, cache, page)
    bad = v[300:301].copy()
    bad[0, 0, 33] = 0x7F80  # its group of 32 dims of kv head 0 stands for NaN
    cb.cb_kv4_store(plan, bf16_tensor(k[300:301].copy()), bf16_tensor(bad), slots[300:301], cache, page)
    out = torch.empty((len(lens), hq, d), dtype=torch.bfloat16, device="cuda")
    cb.cb_kv4_decode_attention(plan, bf16_tensor(q), cache, page, _i32(table), _i32(lens), out)
    plan.check()
    got = _f64(out)
    assert np.isnan(got[0, :4, 32:64]).all()
    ks[0], vs[0] = (serving.dequantise(*serving.quantise(bf16_bits_to_f64(x))) for x in (k, v))
    got[0, :4, 32:64] = decode_attention(bf16_bits_to_f64(q)[0], ks[0], vs[0])[:4, 32:64]
    _check_decode(plan, q, bf16_tensor(f32_to_bf16_bits(got.astype(np.float32))), ks, vs, "beside it")
    plan.close()


def test_page_tables_in_one_buffer(cb):
    # every array a slice of one buffer, each right behind the one before: neighbours are no overlap
    rng = np.random.default_rng(51)
    plan, n, width, rows = _plan(cb, 4, 2, 64), 7, 5, 90
    ctx, new = rng.integers(0, 40, n), rng.integers(0, 13, n)
    have = -(-ctx // 16)
    table = np.where(np.arange(width) < have[:, None], 50 + np.arange(n * width).reshape(n, width), -1)
    free = rng.permutation(30)
    parts = [ctx, new, free, [2], table, np.full(n + 1, -7), np.full(n, -7), np.full(rows, -7), np.full(rows, -7), [-7]]
    whole = _i32(np.concatenate([np.ravel(x) for x in parts]))
    t = list(whole.split([np.size(x) for x in parts]))
    t[4] = t[4].view(n, width)
    cb.cb_page_tables(plan, t[0], t[1], 16, t[2], *t[4:], free_from=t[3])
    plan.check()
    want = serving.page_tables(ctx.tolist(), new.tolist(), 16, free, table, rows, 2)
    for got, w in zip(t[4:], want):
        assert np.array_equal(got.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1))
    assert np.array_equal(torch.cat(t[:4]).cpu().numpy(), np.concatenate([ctx, new, free, [2]]))
    # a decode step whose positions would be written over its lengths
    with pytest.raises(cb.CacheBlendError, match="positions overlaps ctx_lens"):
        cb.cb_page_tables(plan, t[0], t[1], 16, t[2], t[4], t[5], t[6], t[0][:n], t[8][:n], t[9])
    plan.close()


def test_prompt_over_neighbouring_buffers(cb):
    # q, k, v and out as neighbours in one buffer are no overlap; out half a batch into q is
    rng = np.random.default_rng(52)
    plan, n = _plan(cb, 8, 2, 64), 70
    q, k, v = _bits(rng, n, 8, 64), _bits(rng, n, 2, 64), _bits(rng, n, 2, 64)
    whole = torch.cat([bf16_tensor(x).view(-1) for x in (q, k, v)] + [torch.full((n * 512,), 9.0, dtype=torch.bfloat16, device="cuda")])
    dq, dk, dv, out = (x.view(n, -1, 64) for x in whole.split([n * 512, n * 128, n * 128, n * 512]))
    cb.cb_prompt_attention(plan, dq, dk, dv, _i32([0, 40, 70]), out)
    plan.check()
    _check_prompt(q, k, v, [0, 40, 70], out, "neighbours")
    assert torch.equal(dq.contiguous().view(torch.int16), bf16_tensor(q).view(torch.int16))
    half = whole[n * 256:n * 768].view(n, 8, 64)
    with pytest.raises(cb.CacheBlendError, match="out overlaps q"):
        cb.cb_prompt_attention(plan, dq, dk, dv, _i32([0, 40, 70]), half)
    plan.close()


def test_calls_from_many_threads(cb):
    # each thread makes every serving call on a plan and stream of its own, all at the same time
    import threading

    jobs, errors = [], []
    for i in range(6):
        rng = np.random.default_rng(60 + i)
        d, page, lens = (64, 128)[i % 2], 16, [33 + 7 * i, 0, 150]
        n, rows = len(lens), sum(lens) + 2
        plan, free = _plan(cb, 8, 2, d), rng.permutation(40)
        q, k, v = _bits(rng, rows, 8, d), _bits(rng, rows, 2, d), _bits(rng, rows, 2, d)
        q1 = _bits(rng, n, 8, d)
        t = dict(ctx=_i32([0] * n), new=_i32(lens), free=_i32(free), table=_i32(np.full((n, 12), -1)), cu=_i32([0] * (n + 1)),
                 kv=_i32([0] * n), pos=_i32([0] * rows), slots=_i32([0] * rows), to=_i32([0]),
                 cache=torch.zeros(40, 2, cb.cb_kv4_page_bytes(plan, page), dtype=torch.uint8, device="cuda"),
                 out=torch.full((rows, 8, d), 9.0, dtype=torch.bfloat16, device="cuda"),
                 out1=torch.zeros(n, 8, d, dtype=torch.bfloat16, device="cuda"), s=torch.cuda.Stream())
        jobs.append((plan, lens, page, (q, k, v, q1), [bf16_tensor(x) for x in (q, k, v, q1)], t))
    torch.cuda.synchronize()
    start = threading.Barrier(len(jobs))

    def work(plan, lens, page, _, dev, t):
        try:
            q, k, v, q1 = dev
            start.wait()
            for _ in range(10):
                cb.cb_page_tables(plan, t["ctx"], t["new"], page, t["free"], t["table"], t["cu"], t["kv"], t["pos"], t["slots"],
                                  t["to"], stream=t["s"])
                cb.cb_kv4_store(plan, k, v, t["slots"], t["cache"], page, stream=t["s"])
                cb.cb_prompt_attention(plan, q, k, v, t["cu"], t["out"], stream=t["s"])
                cb.cb_kv4_decode_attention(plan, q1, t["cache"], page, t["table"], t["kv"], t["out1"], stream=t["s"])
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for plan, lens, page, (q, k, v, q1), _, t in jobs:
        plan.check()
        cu = np.cumsum([0] + lens)
        _check_prompt(q, k, v, cu, t["out"], "threads")
        ks, vs = ([serving.dequantise(*serving.quantise(bf16_bits_to_f64(x[a:b]))) for a, b in zip(cu, cu[1:])] for x in (k, v))
        _check_decode(plan, q1, t["out1"], ks, vs, "threads")
        plan.close()


@pytest.mark.parametrize("hkv,d", [(2, 64), (8, 128), (1, 64), (3, 128)])
@pytest.mark.parametrize("n,page", [(10, 16), (130, 64), (333, 48)])
def test_store_leaves_every_other_byte(cb, hkv, d, n, page):
    # every byte of the cache after a store row by row, with groups of zeros, tiny, huge and not finite among the rows: the
    # bytes of other tokens, of padding and of unused slots stay, and a NaN scale is the same bits in each form
    rng = np.random.default_rng(70 + hkv * n + d)
    plan = _plan(cb, hkv, hkv, d)
    n_pages = -(-2 * n // page) + 2
    slots = rng.permutation(n_pages * page)[:n]
    slots[2], slots[n - 1] = -1, -5
    k, v = _bits(rng, n, hkv, d), _bits(rng, n, hkv, d, scale=20.0)
    for x in (k, v):
        x[0], x[1, :, 5] = 0, 0xC040
        x[3] = f32_to_bf16_bits((rng.standard_normal((hkv, d)) * 1e-39).astype(np.float32))
        x[4] = f32_to_bf16_bits((rng.standard_normal((hkv, d)) * 5e37).astype(np.float32))
        x[5, 0, 33], x[6, 0, 1], x[7] = 0x7F80, 0x7FC1, 0xFF80
    before = rng.integers(0, 256, (n_pages, hkv, serving.page_bytes(page, d)), dtype=np.uint8)
    cache = torch.as_tensor(before).cuda()
    cb.cb_kv4_store(plan, bf16_tensor(k), bf16_tensor(v), _i32(slots), cache, page)
    plan.check()
    want = before.copy()
    serving.store(want, page, slots, bf16_bits_to_f64(k), bf16_bits_to_f64(v))
    assert np.array_equal(cache.cpu().numpy(), want)
    plan.close()


def test_page_tables_with_too_few_rows_still_give_out_all_pages(cb):
    plan = _plan(cb, 4, 2, 64)
    ctx, new, free, table = [20, 3, 0], [20, 30, 40], [3, 4, 5, 6, 1, 2, 0, 9], [[8, 10, -1], [7, -1, -1], [-1, -1, -1]]
    t, cu, kv, pos, slots, to = _tables(cb, plan, ctx, new, 16, free, table, 25)
    with pytest.raises(cb.CacheBlendError):
        plan.check()
    want = serving.page_tables(ctx, new, 16, free, table, 25)
    for got, w in zip((t, cu, kv, pos, slots, to), want):
        assert np.array_equal(got.reshape(-1), np.asarray(w).reshape(-1))
    plan.close()


@pytest.mark.parametrize("hkv,d,page", [(1, 64, 16), (2, 64, 16), (3, 128, 48), (16, 128, 64)])
@pytest.mark.parametrize("below", [0, 1])
def test_store_and_load_on_both_sides_of_the_choice(cb, hkv, d, page, below):
    # the first call that is taken by whole records (32,768 rows times kv heads), and the last that is taken row by row
    rng = np.random.default_rng(71 + hkv + d)
    plan = _plan(cb, hkv, hkv, d)
    n = -(-32768 // hkv) - below
    n_pages = -(-600 // page) + 2
    slots = np.full(n, -1)
    at = 3 if hkv > 2 else 13  # records that begin off the warps' windows, a run that ends inside a record, single rows
    for start, size in ((0, 48), (64, 37), (112, 16), (131, 5), (160, 240)):
        slots[at:at + size] = np.arange(start, start + size)
        at += size + 3
    rest = np.arange(400, n_pages * page - 16)
    slots[at:at + 60] = rng.permutation(rest)[:60]
    slots[n - 16:] = np.arange(n_pages * page - 16, n_pages * page)  # the cache's last record in the call's last rows
    k, v = (np.zeros((n, hkv, d), np.uint16) for _ in range(2))
    used = slots >= 0
    k[used], v[used] = _bits(rng, used.sum(), hkv, d), _bits(rng, used.sum(), hkv, d, scale=9.0)
    k[20], v[21] = 0, f32_to_bf16_bits((rng.standard_normal((hkv, d)) * 1e-39).astype(np.float32))
    v[60, 0, 33], k[70, hkv - 1, 1] = 0xFF80, 0x7FC1
    before = rng.integers(0, 256, (n_pages, hkv, serving.page_bytes(page, d)), dtype=np.uint8)
    cache = torch.as_tensor(before).cuda()
    cb.cb_kv4_store(plan, bf16_tensor(k), bf16_tensor(v), _i32(slots), cache, page)
    want = before.copy()
    serving.store(want, page, slots[used], bf16_bits_to_f64(k[used]), bf16_bits_to_f64(v[used]))
    assert np.array_equal(cache.cpu().numpy(), want)
    ok, ov = (torch.full((n, hkv, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cb.cb_kv4_load(plan, cache, page, _i32(slots), ok, ov)
    plan.check()
    wk, wv = serving.load(want, page, slots[used], d)
    for g, w in ((ok, wk), (ov, wv)):
        g, w = _f64(g), serving._to_bf16(w)
        assert (g[~used] == 7.0).all()
        assert np.array_equal(np.isnan(g[used]), np.isnan(w)) and np.array_equal(g[used][~np.isnan(w)], w[~np.isnan(w)])
    plan.close()


@pytest.mark.parametrize("hq,hkv,d,most", [(4, 2, 64, 1152), (8, 2, 128, 960), (16, 1, 64, 896), (32, 2, 128, 896)])
def test_decode_on_both_sides_of_the_split(cb, hq, hkv, d, most):
    # the longest request that a CTA takes alone, one key more, and batches beside them
    rng = np.random.default_rng(72 + hq + d)
    plan, page = _plan(cb, hq, hkv, d), 32
    for lens in ([most], [most + 1], [most - 15, 0, 17, most], [1, most + 1, 400]):
        cache, table, ks, vs = _cache(cb, plan, rng, lens, page)
        q = _bits(rng, len(lens), hq, d)
        out = torch.full((len(lens), hq, d), 9.0, dtype=torch.bfloat16, device="cuda")
        cb.cb_kv4_decode_attention(plan, bf16_tensor(q), cache, page, _i32(table), _i32(lens), out)
        plan.check()
        _check_decode(plan, q, out, ks, vs, f"lengths {lens}")
    plan.close()


@pytest.mark.parametrize("power", [84, -100])
def test_values_of_any_magnitude_that_the_header_allows(cb, power):
    # A weight is at most 2^8 (decode) of its reference, a prompt's tile of weights at most 2^16 in sum: over 2^31 keys,
    # times 143 / 7 for decode's codes, 2^43.4 times the largest value, below 2^128 up to 2^84. Scores jump at 40 and 600.
    rng = np.random.default_rng(80 + abs(power))
    hq, hkv, d, page, n = 8, 2, 128, 32, 700
    plan = _plan(cb, hq, hkv, d)
    q, k = _bits(rng, n, hq, d), _bits(rng, n, hkv, d, scale=0.3)
    base = bf16_bits_to_f64(q).reshape(n, hkv, hq // hkv, d).mean((0, 2))
    q = f32_to_bf16_bits((bf16_bits_to_f64(q) + np.repeat(np.sign(base), hq // hkv, 0)).astype(np.float32))
    for at, size in ((40, 0.4), (600, 1.2)):
        k[at] = f32_to_bf16_bits((size * np.sign(base)).astype(np.float32))
    v = rng.standard_normal((n, hkv, d))
    v = f32_to_bf16_bits((np.clip(v / 4, -1, 1) * 2.0**power).astype(np.float32))
    out = _prompt(cb, plan, q, k, v, [0, n])
    plan.check()
    _check_prompt(q, k, v, [0, n], out, f"prompt, values up to 2^{power}")
    table = rng.permutation(-(-n // page))[None]
    cache = torch.zeros((table.size, hkv, serving.page_bytes(page, d)), dtype=torch.uint8, device="cuda")
    pos = np.arange(n)
    cb.cb_kv4_store(plan, bf16_tensor(k), bf16_tensor(v), _i32(table[0][pos // page] * page + pos % page), cache, page)
    ks, vs = (serving.dequantise(*serving.quantise(bf16_bits_to_f64(x))) for x in (k, v))
    out = torch.empty((1, hq, d), dtype=torch.bfloat16, device="cuda")
    cb.cb_kv4_decode_attention(plan, bf16_tensor(q[-1:].copy()), cache, page, _i32(table), _i32([n]), out)
    plan.check()
    _check_decode(plan, q[-1:], out, [ks], [vs], f"decode, values up to 2^{power}")
    plan.close()


@pytest.mark.parametrize("hq,hkv,d,page", [(4, 2, 64, 16), (16, 2, 128, 64)])
def test_chunks_cached_loaded_blended_cached_and_decoded(cb, hq, hkv, d, page):
    """What ties these calls to the blend: chunks are encoded on their own and cached in 4 bits, read back as the blend's
    k_old / v_old, blended, the fused cache stored as a request's pages, and its first token decoded over them."""
    import dataclasses

    from conftest import assert_close_attention, assert_close_bf16
    from oracle.blend import blend_layer
    from workloads import get_config
    from workloads.generator import generate_layer, hkvd_noise_sets
    from workloads.torch_io import layer_tensors

    cfg = dataclasses.replace(get_config("tiny"), n_chunks=3, chunk_len=84, n_suffix=21, hq=hq, hkv=hkv, head_dim=d)
    rng = np.random.default_rng(90 + d)
    inp = generate_layer(cfg, 1, hkvd_noise_sets(cfg))
    plan, serve = cb.Plan.from_config(cfg), cb.Plan(1, 512, 0, hq, hkv, d, cfg.rope_theta)
    n_ctx, n = cfg.n_ctx, cfg.n_tokens
    pool, lens = 64, [cfg.chunk_len] * 3
    free, cache = _i32(rng.permutation(pool)), torch.zeros((pool, hkv, serving.page_bytes(page, d)), dtype=torch.uint8, device="cuda")
    i0 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    # the chunks: laid out, attended on their own, cached
    cu, kv, pos, slots, to = i0(4), i0(3), i0(n_ctx), i0(n_ctx), i0(1)
    cb.cb_page_tables(serve, i0(3), _i32(lens), page, free, i0(3, 8) - 1, cu, kv, pos, slots, to)
    t = layer_tensors(inp)
    qc = _bits(rng, n_ctx, hq, d)
    out = torch.empty((n_ctx, hq, d), dtype=torch.bfloat16, device="cuda")
    cb.cb_prompt_attention(serve, bf16_tensor(qc), t["k_old"], t["v_old"], cu, out)
    cb.cb_kv4_store(serve, t["k_old"], t["v_old"], slots, cache, page)
    serve.check()
    _check_prompt(qc, inp.k_old, inp.v_old, np.cumsum([0] + lens), out, "chunks")
    # read back, blended
    t["k_old"], t["v_old"] = torch.empty_like(t["k_old"]), torch.empty_like(t["v_old"])
    cb.cb_kv4_load(serve, cache, page, slots, t["k_old"], t["v_old"])
    for got, x in ((t["k_old"], inp.k_old), (t["v_old"], inp.v_old)):
        assert np.array_equal(_f64(got), serving._to_bf16(serving.dequantise(*serving.quantise(bf16_bits_to_f64(x)))))
    bufs = cb.LayerBuffers(plan)
    cb.cb_blend_layer(plan, 1, cand=None, bufs=bufs, **t)
    plan.check()
    _, k, mq, selects = plan.layer_sizes(1)
    want = blend_layer(cfg, dataclasses.replace(inp, k_old=bf16_bits(t["k_old"]), v_old=bf16_bits(t["v_old"])), 1,
                       np.arange(n_ctx), k, bool(selects))
    assert np.array_equal(bufs.sel_tok[:k].cpu().numpy(), want.sel_tok)
    assert np.array_equal(_f64(bufs.v_fused), want.v_fused)
    assert_close_bf16(_f64(bufs.k_fused), want.k_fused, what="fused K")
    assert_close_attention(_f64(bufs.out[:mq]), want.out, want.out_vscale)
    # the fused cache as a request's pages, behind those of the chunks, which stay
    table, cu, kv, pos, slots2, end = i0(1, 36 if page == 16 else 8) - 1, i0(2), i0(1), i0(n), i0(n), i0(1)
    cb.cb_page_tables(serve, i0(1), _i32([n]), page, free, table, cu, kv, pos, slots2, end, free_from=to)
    cb.cb_kv4_store(serve, bufs.k_fused, bufs.v_fused, slots2, cache, page)
    # its first token
    q1, k1, v1 = _bits(rng, 1, hq, d), _bits(rng, 1, hkv, d), _bits(rng, 1, hkv, d)
    dq, dk = bf16_tensor(q1), bf16_tensor(k1)
    qe, ke, kv1 = torch.empty_like(dq), torch.empty_like(dk), i0(1)
    cu, pos, slot, last = i0(2), i0(1), i0(1), i0(1)
    cb.cb_page_tables(serve, kv, _i32([1]), page, free, table, cu, kv1, pos, slot, last, free_from=end)
    cb.cb_rope_rerotate(serve, qe, dq, pos)
    cb.cb_rope_rerotate(serve, ke, dk, pos)
    cb.cb_kv4_store(serve, ke, bf16_tensor(v1), slot, cache, page)
    out = torch.empty((1, hq, d), dtype=torch.bfloat16, device="cuda")
    cb.cb_kv4_decode_attention(serve, qe, cache, page, table, kv1, out)
    serve.check()
    assert pos.tolist() == [n] and kv1.tolist() == [n + 1]
    ks, vs = (serving.dequantise(*serving.quantise(bf16_bits_to_f64(np.concatenate((bf16_bits(a), b)))))
              for a, b in ((bufs.k_fused, bf16_bits(ke)), (bufs.v_fused, v1)))
    _check_decode(serve, bf16_bits(qe), out, [ks], [vs], "first token")
    again = [torch.empty_like(x) for x in (t["k_old"], t["v_old"])]
    cb.cb_kv4_load(serve, cache, page, slots, *again)
    for a, b in zip(again, (t["k_old"], t["v_old"])):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    plan.close()
    serve.close()


# ---- calls at the ends of what is allowed ---------------------------------------------------------


@pytest.mark.parametrize("page", [1024, 1008])
def test_largest_pages(cb, page):
    rng = np.random.default_rng(100 + page)
    plan, lens = _plan(cb, 8, 2, 64), [page, 3 * page - 5, 0, 17, page + 1]
    cache, table, ks, vs = _cache(cb, plan, rng, lens, page)
    q = _bits(rng, len(lens), 8, 64)
    out = torch.full((len(lens), 8, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    cb.cb_kv4_decode_attention(plan, bf16_tensor(q), cache, page, _i32(table), _i32(lens), out)
    slots = _i32(table[1][np.arange(lens[1]) // page] * page + np.arange(lens[1]) % page)
    k, v = (torch.empty((lens[1], 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cb.cb_kv4_load(plan, cache, page, slots, k, v)
    plan.check()
    _check_decode(plan, q, out, ks, vs, f"pages of {page}")
    assert np.array_equal(_f64(k), serving._to_bf16(ks[1])) and np.array_equal(_f64(v), serving._to_bf16(vs[1]))
    plan.close()


@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 64), (1, 1, 128), (256, 16, 128), (512, 32, 64), (32, 32, 64)])
def test_smallest_and_largest_head_layouts(cb, hq, hkv, d):
    rng = np.random.default_rng(101 + hq)
    plan, lens, page = _plan(cb, hq, hkv, d), [40, 0, 141, 3], 48
    cu, n = np.cumsum([0] + lens), sum(lens) + 2
    q, k, v = _bits(rng, n, hq, d), _bits(rng, n, hkv, d), _bits(rng, n, hkv, d)
    out = _prompt(cb, plan, q, k, v, cu)
    cache, table, ks, vs = _cache(cb, plan, rng, lens, page)
    q1 = _bits(rng, len(lens), hq, d)
    out1 = torch.full((len(lens), hq, d), 9.0, dtype=torch.bfloat16, device="cuda")
    cb.cb_kv4_decode_attention(plan, bf16_tensor(q1), cache, page, _i32(table), _i32(lens), out1)
    plan.check()
    _check_prompt(q, k, v, cu, out, "prompt")
    _check_decode(plan, q1, out1, ks, vs, "decode")
    plan.close()


def test_decode_of_thousands_of_requests(cb):
    rng = np.random.default_rng(102)
    plan, page = _plan(cb, 4, 2, 64), 16
    lens = [int(x) for x in rng.integers(0, 36, 3001)]
    cache, table, ks, vs = _cache(cb, plan, rng, lens, page)
    q = _bits(rng, len(lens), 4, 64)
    out = torch.full((len(lens), 4, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    cb.cb_kv4_decode_attention(plan, bf16_tensor(q), cache, page, _i32(table), _i32(lens), out)
    plan.check()
    _check_decode(plan, q, out, ks, vs, "many requests")
    plan.close()


def test_prompt_of_the_most_sequences(cb):
    rng = np.random.default_rng(103)
    plan = _plan(cb, 4, 2, 64)
    lens = rng.integers(0, 3, 16384)
    lens[[0, 5000, 16383]] = 0, 150, 70
    cu, n = np.cumsum(np.r_[0, lens]), int(lens.sum()) + 1
    q, k, v = _bits(rng, n, 4, 64), _bits(rng, n, 2, 64), _bits(rng, n, 2, 64)
    out = _prompt(cb, plan, q, k, v, cu)
    plan.check()
    _check_prompt(q, k, v, cu, out, "most sequences")
    plan.close()


def test_no_pages_no_width_no_requests(cb):
    plan, page = _plan(cb, 8, 2, 64), 16
    bf = lambda *s: torch.full(s, 9.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    none = torch.zeros((0, 2, serving.page_bytes(page, 64)), dtype=torch.uint8, device="cuda")
    some = torch.zeros((3, 2, serving.page_bytes(page, 64)), dtype=torch.uint8, device="cuda")
    # nothing to do
    cb.cb_kv4_store(plan, bf(0, 2, 64), bf(0, 2, 64), _i32([]), some, page)
    cb.cb_kv4_load(plan, none, page, _i32([]), bf(0, 2, 64), bf(0, 2, 64))
    cb.cb_kv4_decode_attention(plan, bf(0, 8, 64), none, page, _i32(np.zeros((0, 4))), _i32([]), bf(0, 8, 64))
    cb.cb_prompt_attention(plan, bf(0, 8, 64), bf(0, 2, 64), bf(0, 2, 64), _i32([0, 0]), bf(0, 8, 64))
    out = bf(5, 8, 64)
    cb.cb_prompt_attention(plan, bf(5, 8, 64), bf(5, 2, 64), bf(5, 2, 64), _i32([3]), out)  # no sequence
    plan.check()
    assert (out == 9.0).all()
    # requests without keys over a table without columns and a cache without pages
    out = bf(3, 8, 64)
    cb.cb_kv4_decode_attention(plan, bf(3, 8, 64), none, page, _i32(np.zeros((3, 0))), _i32([0, 0, 0]), out)
    plan.check()
    assert not out.any()
    # keys that the table has no room for, pages that the cache does not have: left out, and recorded
    for cache, table in ((some, np.zeros((3, 0))), (none, np.zeros((3, 2)))):
        out = bf(3, 8, 64)
        cb.cb_kv4_decode_attention(plan, bf(3, 8, 64), cache, page, _i32(table), _i32([0, 20, 9]), out)
        with pytest.raises(cb.CacheBlendError) as e:
            plan.check()
        assert e.value.status == 5 and not out.any()
    for n in (3, 17000):  # row by row, and by runs
        k, v = bf(n, 2, 64), bf(n, 2, 64)
        cb.cb_kv4_load(plan, none, page, _i32(np.arange(n)), k, v)
        with pytest.raises(cb.CacheBlendError):
            plan.check()
        assert (k == 9.0).all() and (v == 9.0).all()
        cb.cb_kv4_store(plan, k, v, _i32(np.arange(n)), none, page)
        with pytest.raises(cb.CacheBlendError):
            plan.check()
    plan.close()


def test_page_tables_at_the_ends_of_32_bits(cb):
    plan, top = _plan(cb, 4, 2, 64), (1 << 31) - 1
    ctx, new, free = [top, 5, top - 3, 0], [3, 20, 2, 0], [4, 8, 9]
    table = [[1, -1, -1], [2, -1, -1], [3, 6, 7], [-1, -1, -1]]
    t, cu, kv, pos, slots, to = _tables(cb, plan, ctx, new, 16, free, table, 27, free_from=1)
    with pytest.raises(cb.CacheBlendError) as e:
        plan.check()
    assert e.value.status == 5
    want = serving.page_tables(ctx, new, 16, free, table, 27, 1)
    for got, w in zip((t, cu, kv, pos, slots, to), (*want[:3], np.minimum(want[3], top), *want[4:])):
        assert np.array_equal(got.reshape(-1), np.asarray(w).reshape(-1))
    # a free list whose start lies behind its end, or is the last of 32 bits
    for frm in (7, top):
        t, cu, kv, pos, slots, to = _tables(cb, plan, [0], [20], 16, free, [[-1, -1]], 20, free_from=frm)
        with pytest.raises(cb.CacheBlendError):
            plan.check()
        assert to.tolist() == [frm] and t.tolist() == [[-1, -1]] and (slots == -1).all() and kv.tolist() == [20]
    # rows for none of the new tokens
    t, cu, kv, pos, slots, to = _tables(cb, plan, [0, 16], [20, 1], 16, free, [[-1, -1], [5, -1]], 0)
    with pytest.raises(cb.CacheBlendError):
        plan.check()
    assert t.tolist() == [[4, 8], [5, 9]] and cu.tolist() == [0, 0, 0] and kv.tolist() == [20, 17] and to.tolist() == [3]
    plan.close()


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (16, 1, 128), (4, 4, 128)])
def test_queries_that_are_not_finite_stay_with_their_row_and_head(cb, hq, hkv, d):
    rng = np.random.default_rng(104 + hq)
    plan, page = _plan(cb, hq, hkv, d), 16
    cu, n = [0, 150, 200], 200
    q, k, v = _bits(rng, n, hq, d), _bits(rng, n, hkv, d), _bits(rng, n, hkv, d)
    clean = q.copy()
    bad = np.zeros((n, hq), bool)
    for row, head, bits in ((0, 0, 0x7FC0), (77, 1, 0x7F80), (140, hq - 1, 0xFF80), (160, 2, 0x7FC1)):
        q[row, head, 5], bad[row, head] = bits, True
    got = _f64(_prompt(cb, plan, q, k, v, cu))
    plan.check()
    assert np.isnan(got[bad & (np.arange(n) % 10 == 0)[:, None]]).all()  # NaNs, and an infinity over many keys
    ref, vs = serving.packed_attention(*(bf16_bits_to_f64(x) for x in (clean, k, v)), cu)
    _close(got[~bad], ref[~bad], vs[~bad], 40 * 2.0**-23 * d**0.5 * np.abs(bf16_bits_to_f64(clean)).max() * np.abs(bf16_bits_to_f64(k)).max(), "prompt")
    lens = [50, 700, 3]
    cache, table, ks, vs4 = _cache(cb, plan, rng, lens, page)
    q1 = _bits(rng, 3, hq, d)
    clean = q1.copy()
    for s, head, bits in ((0, 0, 0x7FC0), (1, hq - 1, 0x7F80)):
        q1[s, head, 9] = bits
    out = torch.empty((3, hq, d), dtype=torch.bfloat16, device="cuda")
    cb.cb_kv4_decode_attention(plan, bf16_tensor(q1), cache, page, _i32(table), _i32(lens), out)
    plan.check()
    got = _f64(out)
    assert np.isnan(got[0, 0]).all() and np.isnan(got[1, hq - 1]).all()
    for s, head in ((0, 0), (1, hq - 1)):  # the rest is as it would be
        got[s, head] = decode_attention(bf16_bits_to_f64(clean)[s], ks[s], vs4[s])[head]
    _check_decode(plan, clean, bf16_tensor(f32_to_bf16_bits(got.astype(np.float32))), ks, vs4, "decode")
    plan.close()
