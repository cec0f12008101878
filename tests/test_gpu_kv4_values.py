"""Chunk attention and attention weights over 4-bit pages on contents whose parts differ by orders of magnitude, and on a
long context whose parts can be told apart, against the oracle in 64 bits.

Tolerances. With s = sum_j p_j |v_j| of the output's own dim, an output is within (2^-11 + 2 e + 2^-20 + t) s of the exact
value, and 2^-8 of itself by its rounding to bf16: a softmax weight is rounded to fp16 once (2^-11), scores are off by at most
e = (D + 16) 2^-23 scale max_j sum_d |q_d| max|k_d| (fp32 sums of D products, each of D + 8 roundings of 2^-23 since the
matrix unit truncates) and 2^-35 scale max|q| sum_d max|k_d| (q is held to within 2^-35 of its head's largest, which moves a score
by no more than that times the sum of the key's magnitudes: small beside the first term where q's dims are of one size, not
where some are 2^24 of the others), 2^x and its sum by 2^-20, and the sum over n keys by
t = (n / 16 + 16) 2^-22: one truncation of 2^-23 for every 16 keys, and as much for the joins. Where a weight is below 2^-14 in
the units in which the row's largest is at least 2^4, its rounding is 2^-25 of those units instead: n 2^-29 p_max of the
group's largest value. Requests of few rows round the weights times V's scales instead, in units of the largest scale of all
groups, which the row's largest weight brings to 2^6 at least: n 2^-31 p_max of the largest value of all groups. lse is within
e + 2^-20 + 2^-22 |lse| + n 2^-24.
"""

import numpy as np
import pytest
import torch
from test_gpu_kv4_batch import Batch, _f64, _i32

from oracle import serving

pytestmark = pytest.mark.gpu


class Values(Batch):
    def error(self, q, k, c):
        top = np.abs(k).max(0, initial=0.0)
        return super().error(q, k, c) + float(c * 2.0**-35 * np.abs(q).max(initial=0.0) * top.sum(-1).max(initial=0.0))


def check(b, out, lse, rows_of=None, few=False):
    """Every request's out and lse (of its rows rows_of(request) only, where that is given) within the limits above."""
    got, glse, q = _f64(out), lse.cpu().numpy().astype(np.float64), _f64(b.q)
    c = b.d**-0.5
    for s in range(len(b.lens)):
        a, m = int(b.cu[s]), b.new[s]
        if m == 0:
            continue
        k, v = b.cached(s)
        for i in range(m) if rows_of is None else rows_of(s):
            n = len(k) - m + i + 1
            kk, vv, qq = k[:n], v[:n], q[a + i:a + i + 1]
            ref, rlse, vs = serving.chunk_attention(qq, kk, vv)
            e = b.error(qq, kk, c)
            g = np.arange(b.hq) * b.hkv // b.hq
            peak = np.exp(c * np.einsum("nhd,hd->hn", kk[:, g], qq[0]).max(-1) - rlse[0])  # [hq]
            top = np.abs(vv).reshape(n, b.hkv, -1, 32).max((0, 3))[g]  # [hq, groups]
            top = np.repeat(top, 32, 1) * 2.0**-29 if not few else top.max(1, keepdims=True) * 2.0**-31
            lim = (2.0**-11 + 2 * e + 2.0**-20 + (n / 16 + 16) * 2.0**-22) * vs[0] + 2.0**-8 * np.abs(ref[0])
            lim += n * peak[:, None] * top + 1e-37
            err = np.abs(got[a + i] - ref[0])
            assert (err <= lim).all(), f"request {s}, row {i}: err/limit {np.nanmax(err / lim):.3f}"
            err, lim = np.abs(glse[a + i] - rlse[0]), e + 2.0**-20 + 2.0**-22 * np.abs(rlse[0]) + n * 2.0**-24
            assert (err <= lim).all(), f"lse of request {s}, row {i}: err/limit {np.nanmax(err / lim):.3f}"


def _segments(k, v):
    """Values that are 1 in one dim and 0 in the others, by the part of the context: an output is the weight of a part."""
    n, _, d = v.shape
    v[:] = 0
    v[np.arange(n), :, np.arange(n) * d // n] = 1


@pytest.mark.parametrize("m", [1, 3, 40, 150])
@pytest.mark.parametrize("heads", [(32, 8, 128), (16, 1, 64), (8, 4, 128), (16, 16, 128)])
def test_each_part_of_a_long_context_has_its_weight(cb, heads, m):
    # one request over all SMs, joined: a part that is lost or weighed wrongly shows in the dim that stands for it
    b = Values(cb, heads, [20011], [m], 64, qs=0.5, edit=_segments)
    out, lse = b.chunk()
    b.plan.check()
    check(b, out, lse, rows_of=lambda s: range(m) if m < 4 else (0, m // 2, m - 1))
    b.plan.close()


@pytest.mark.parametrize("heads,n", [((32, 8, 128), 33), ((16, 1, 64), 70), ((32, 16, 64), 20)])
def test_each_part_of_a_long_context_has_its_weight_with_few_rows(cb, heads, n):
    # a long request among short ones, on the kernel for few rows: its parts are merged within CTAs and over them
    lens, new = [50] * n, [1] * n
    lens[n // 2] = 20011
    at = 50 * (n // 2)
    b = Values(cb, heads, lens, new, 32, qs=0.5, edit=lambda k, v: _segments(k[at:at + 20011], v[at:at + 20011]))
    out, lse = b.chunk()
    b.plan.check()
    check(b, out, lse, few=True)
    b.plan.close()


@pytest.mark.parametrize("down", [4, 12, 16, 24])
@pytest.mark.parametrize("heads,few", [((8, 2, 128), False), ((8, 4, 64), False), ((16, 16, 128), False), ((32, 8, 128), True)])
def test_a_group_of_values_far_below_the_others(cb, heads, few, down):
    # dims 32 .. 63 are 2^-down of the others: their outputs are as close to their own magnitude
    def edit(k, v):
        v[:, :, 32:64] *= 2.0**-down

    lens, new = ([300] * 33, [1] * 33) if few else ([300, 129], [140, 1])
    b = Values(cb, heads, lens, new, 32, edit=edit)
    out, lse = b.chunk()
    b.plan.check()
    check(b, out, lse, few=few)
    b.plan.close()


@pytest.mark.parametrize("down", [4, 12, 16, 24])
@pytest.mark.parametrize("heads,few", [((8, 2, 128), False), ((8, 4, 64), False), ((32, 8, 128), True)])
def test_a_group_of_keys_far_below_the_others_with_queries_above(cb, heads, few, down):
    # dims 32 .. 63 of k are 2^-down of the others, of q 2^down: they count as much in the scores
    def edit(k, v):
        k[:, :, 32:64] *= 2.0**-down

    lens, new = ([300] * 33, [1] * 33) if few else ([300, 129], [140, 1])
    b = Values(cb, heads, lens, new, 32, edit=edit)
    b.q[:, :, 32:64] *= 2.0**down
    out, lse = b.chunk()
    b.plan.check()
    check(b, out, lse, few=few)
    w = b.weights(lse)
    b.plan.check()
    b.check_weights(w, lse)
    b.plan.close()


@pytest.mark.parametrize("how", ["up", "down", "waves", "once", "none"])
@pytest.mark.parametrize("m", [3, 140])
def test_values_hundreds_of_powers_apart_leave_the_weights_as_they_are(cb, how, m):
    # (enough requests for several rounds of 128 keys of one request to meet in a CTA)
    def edit(k, v):
        x = np.arange(len(v)) % 3000
        e = {"up": np.where(x < 1500, -100, 60), "down": np.where(x < 1500, 60, -100), "waves": np.where(x // 128 % 2, 60, -100),
             "once": np.where(x == 900, 60, -100), "none": np.where(x < 1500, -100, -30)}[how]
        v *= np.exp2(e)[:, None, None].astype(np.float32)
        if how == "none":
            v[x < 700] = 0

    b = Values(cb, (8, 2, 128), [3000] * 20, [m] + [3] * 19, 16, edit=edit)
    out, lse = b.chunk()
    b.plan.check()
    b.check_chunk(out, lse, skip=range(3 if m == 3 else 1, 20))
    b.plan.close()


@pytest.mark.parametrize("how", ["up", "down", "waves", "once"])
def test_values_hundreds_of_powers_apart_with_few_rows(cb, how):
    def edit(k, v):
        x = np.arange(len(v))
        e = {"up": np.where(x < 1500, -100, 60), "down": np.where(x < 1500, 60, -100), "waves": np.where(x // 16 % 2, 60, -100),
             "once": np.where(x == 900, 60, -100)}[how]
        v *= np.exp2(np.where(x < 3000, e, 0))[:, None, None].astype(np.float32)

    b = Values(cb, (32, 8, 128), [3000] + [90] * 32, [2] + [1] * 32, 16, edit=edit)
    out, lse = b.chunk()
    b.plan.check()
    b.check_chunk(out, lse)
    b.plan.close()


def test_rows_of_different_magnitudes(cb):
    # rows that share a tile, 2^-20 and 2^-30 of one another: the softmax of each is its own
    b = Values(cb, (8, 2, 128), [300, 90], [140, 9], 16)
    scale = torch.tensor([1.0, 2.0**-20, 2.0**-30], device="cuda")[torch.arange(b.rows, device="cuda") % 3]
    b.q.mul_(scale[:, None, None].bfloat16())
    out, lse = b.chunk()
    b.plan.check()
    b.check_chunk(out, lse)
    w = b.weights(lse)
    b.plan.check()
    b.check_weights(w, lse)
    b.plan.close()


@pytest.mark.parametrize("up", [20, 40, 100])
@pytest.mark.parametrize("what", ["keys", "values", "both"])
@pytest.mark.parametrize("heads,few,m", [((8, 2, 128), False, 140), ((16, 16, 64), False, 40), ((32, 2, 128), False, 12),
                                         ((8, 8, 128), True, 8), ((16, 8, 64), True, 4), ((32, 8, 128), True, 2)])
def test_later_keys_of_any_size_do_not_reach_a_row(cb, heads, few, m, what, up):
    # keys and values 2^up of the others from the request's last rows on: hidden from its rows before
    n, late = 300, max(m // 3, 1)
    at = n - late  # the first such key

    def edit(k, v):
        if what != "values":
            k[at:n] *= 2.0**up
        if what != "keys":
            v[at:n] *= 2.0**up

    lens, new = ([n] + [50] * 33, [m] + [1] * 33) if few else ([n, 129], [m, 5])
    b = Values(cb, heads, lens, new, 16, edit=edit)
    out, lse = b.chunk()
    b.plan.check()
    check(b, out, lse, rows_of=lambda s: range(m - late if s == 0 else b.new[s]), few=few)
    # rows that see them: an average of the values
    assert torch.isfinite(lse).all()
    assert (_f64(out)[:m] <= 1.01 * np.repeat(np.abs(b.cached(0)[1]).max(0), b.hq // b.hkv, 0)).all()
    b.plan.close()


@pytest.mark.parametrize("down", [30, 70])
@pytest.mark.parametrize("what", ["keys", "values", "both"])
def test_keys_of_many_sizes_in_a_round(cb, what, down):
    # every third key (or value) 2^-down of the others, some zero; enough requests for a CTA to take several rounds
    def edit(k, v):
        x = np.arange(len(v)) % 3000
        for t, name in ((k, "keys"), (v, "values")):
            if what in (name, "both"):
                t[x % 3 == 1] *= 2.0**-down
                t[x % 50 == 7] = 0

    b = Values(cb, (8, 2, 128), [3000] * 20, [40] + [3] * 19, 16, qs=0.5, edit=edit)
    out, lse = b.chunk()
    b.plan.check()
    b.check_chunk(out, lse, skip=range(3, 20))
    again, l2 = b.chunk()
    assert torch.equal(again, out) and torch.equal(l2, lse)
    b.plan.close()


@pytest.mark.parametrize("up", [20, 40, 100])
@pytest.mark.parametrize("heads,few,m", [((8, 2, 128), False, 140), ((16, 16, 64), False, 40), ((32, 2, 128), False, 12),
                                         ((8, 8, 128), True, 8), ((16, 8, 64), True, 4), ((32, 8, 128), True, 2)])
def test_later_keys_of_any_size_leave_the_weights_of_others(cb, heads, few, m, up):
    n, late = 300, max(m // 3, 1)
    at = n - late  # the first such key

    def edit(k, v):
        k[at:n] *= 2.0**up

    lens, new = ([n] + [50] * 33, [m] + [1] * 33) if few else ([n, 129], [m, 5])
    b = Values(cb, heads, lens, new, 16, edit=edit)
    _, lse = b.chunk()
    b.plan.check()
    lse[m - late:m] = -float("inf")  # (the rows that see them add nothing to the weights)
    w = b.weights(lse).cpu().numpy().astype(np.float64)
    b.plan.check()
    k, q = b.cached(0)[0][:at], _f64(b.q)[:m - late]
    ref = serving.attention_weights(q, lse.cpu().numpy().astype(np.float64)[:m - late], k)
    rel = 2 * b.error(q, k, b.d**-0.5) + 2.0**-20 + 2.0**-22 * 20 + (m * b.hq // b.hkv) * 2.0**-23
    assert (np.abs(w[0, :, :at] - ref) <= rel * ref + 1e-37).all()
    assert (w[0, :, at:n] == 0).all() and (w[0, :, n:] == 7).all()
    b.plan.close()


@pytest.mark.parametrize("what", [np.nan, np.inf, 1e30])
@pytest.mark.parametrize("heads,few,m", [((8, 2, 128), False, 140), ((16, 16, 64), False, 40), ((8, 8, 128), True, 8),
                                         ((32, 8, 128), True, 2)])
def test_a_row_without_lse_adds_nothing_whatever_its_query_is(cb, heads, few, m, what):
    lens, new = ([300] + [50] * 33, [m] + [1] * 33) if few else ([300, 129], [m, 5])
    b = Values(cb, heads, lens, new, 16)
    _, lse = b.chunk()
    lse[1::2] = -float("inf")
    want = b.weights(lse)
    q = b.q.clone()
    b.q[1::2] = what
    got = b.weights(lse)
    assert torch.equal(got, want)
    b.q = q
    b.check_weights(got, lse)
    b.plan.check()
    b.plan.close()


def test_as_many_requests_as_a_call_takes(cb):
    rng = np.random.default_rng(4)
    n = 16384
    new = np.ones(n, np.int64)
    new[rng.integers(n, size=9)] = [0, 2, 3, 5, 9, 40, 70, 130, 0]
    lens = new + rng.integers(0, 30, n)
    b = Values(cb, (4, 2, 64), lens, new, 16, pad=1)
    some = set(rng.integers(n, size=60)) | set(np.flatnonzero(new != 1)) | {0, n - 1}
    skip = set(range(n)) - some
    out, lse = b.chunk()
    b.plan.check()
    b.check_chunk(out, lse, skip=skip)
    w = b.weights(lse)
    b.plan.check()
    b.check_weights(w, lse, skip=skip)
    kept = torch.full((n, 2, 20), -5, dtype=torch.int32, device="cuda")
    kept_lens = torch.zeros(n, dtype=torch.int32, device="cuda")
    cb.cb_kv4_keep(b.plan, w, b.t_lens, torch.full_like(kept_lens, 20), kept, kept_lens, first=1, recent=2)
    b.plan.check()
    assert np.array_equal(kept_lens.cpu().numpy(), np.minimum(lens, 20))
    wh, kh = w.cpu().numpy(), kept.cpu().numpy()
    for s in some:
        for g in range(2):
            want = serving.keep(wh[s, g], lens[s], 20, 1, 2)
            assert np.array_equal(kh[s, g, :len(want)], want)
    b.plan.close()


@pytest.mark.parametrize("few", [False, True])
def test_pages_behind_the_first_4_gigabytes(cb, few):
    # the same requests in a small cache and at the end of one of 6 GB: the same bits
    lens, new = ([700] * 33, [1] * 33) if few else ([700, 1500], [60, 3])
    b = Values(cb, (32, 8, 128), lens, new, 256)
    out, lse = b.chunk()
    w = b.weights(lse)
    small, n = b.cache, 6 * 2**30 // b.cache[0].numel()
    b.cache = torch.zeros((n, *small.shape[1:]), dtype=torch.uint8, device="cuda")
    b.cache[n - len(small):] = small
    b.t_table = torch.where(b.t_table >= 0, b.t_table + (n - len(small)), b.t_table)
    far, l2 = b.chunk()
    w2 = b.weights(l2)
    assert torch.equal(far, out) and torch.equal(l2, lse) and torch.equal(w2, w)
    # the last rows of each request moved to the first pages, read back
    kept = (b.t_lens[:, None, None] - 20 + torch.arange(20, device="cuda").int()).expand(-1, 8, -1).contiguous()
    to = torch.arange(len(lens), dtype=torch.int32, device="cuda")[:, None].contiguous()
    cb.cb_kv4_move(b.plan, b.cache, 256, b.t_table, kept, torch.full_like(b.t_lens, 20), to)
    b.plan.check()
    k, v = (torch.zeros(20, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k2, v2 = torch.zeros_like(k), torch.zeros_like(v)
    for s in range(len(lens)):
        at = np.arange(lens[s] - 20, lens[s])
        cb.cb_kv4_load(b.plan, small, 256, _i32(b.table[s][at // 256] * 256 + at % 256), k, v)
        cb.cb_kv4_load(b.plan, b.cache, 256, _i32(s * 256 + np.arange(20)), k2, v2)
        assert torch.equal(k, k2) and torch.equal(v, v2)
    b.plan.check()
    b.plan.close()
