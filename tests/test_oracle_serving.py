"""Pins of the serving oracle: quantisation, the record's byte layout, page tables, packed prompts."""

import numpy as np
import pytest

from oracle import serving
from oracle.attention import causal_gqa_attention
from oracle.deviation import bf16_bits_to_f64
from workloads.generator import f32_to_bf16_bits


def _bf16(x):
    return bf16_bits_to_f64(f32_to_bf16_bits(np.asarray(x, dtype=np.float32)))


def test_bf16_rounding_agrees_with_the_generator():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal(4096) * 10.0 ** rng.integers(-39, 38, 4096)).astype(np.float32)
    assert np.array_equal(serving._to_bf16(x.astype(np.float64)), _bf16(x))


def test_codes_worked_by_hand():
    x = np.zeros(64)
    x[:5] = [7.0, -7.0, 3.5, 2.5, -0.5]  # scale 1: 3.5 and 2.5 are ties and go to even
    x[32:35] = [0.875, -0.125, 0.3125]  # scale 1/8: 7, -1, 2.5 -> 2
    c, s = serving.quantise(x)
    assert s.tolist() == [1.0, 0.125]
    assert c[:5].tolist() == [7, -7, 4, 2, 0] and c[32:35].tolist() == [7, -1, 2]
    assert not c[5:32].any() and not c[35:].any()


def test_groups_of_zeros_and_of_values_that_are_not_finite():
    x = np.zeros((3, 64))
    x[1, 3], x[2, 40] = np.inf, np.nan
    c, s = serving.quantise(x)
    assert not c.any() and s[0].tolist() == [0.0, 0.0]
    assert np.isnan(s[1, 0]) and s[1, 1] == 0.0 and s[2, 0] == 0.0 and np.isnan(s[2, 1])


def test_quantisation_error_is_half_a_step():
    rng = np.random.default_rng(1)
    x = _bf16(rng.standard_normal((200, 4, 128)))
    c, s = serving.quantise(x)
    err = np.abs(serving.dequantise(c, s) - x)
    # half a step, plus the largest value's own excess over 7 scales (the scale's rounding, 7 * 2^-9)
    assert (err <= np.repeat(s, 32, axis=-1) * (0.5 + 7 * 2.0**-9)).all()


@pytest.mark.parametrize("d", [64, 128])
def test_record_layout_by_bytes(d):
    # one token in slot 11 of a 16-token page, one kv head: K dim 37 and V dim 37 alone are not zero
    cache = np.zeros((1, 1, serving.page_bytes(16, d)), dtype=np.uint8)
    x = np.zeros((1, 1, d))
    x[0, 0, 37] = 7.0
    serving.store(cache, 16, [11], x, x)
    rec = cache[0, 0]
    ng = d // 32
    # K: token 11, c = (37 - 32) // 8 = 0, group 1, e = 5: bits 4 * 2 + 16 = 24 of the word
    word = int(rec[(11 * 4 * ng + 1) * 4:][:4].view("<u4")[0])
    assert word == 0x88888888 & ~(0xF << 24) | 15 << 24
    # V: half 1, r = (37 - 32) // 4 = 1, c = 3 // 2 = 1, token odd: high 16 bits, i = 1
    word = int(rec[8 * d + ((8 + 1) * 4 * ng + 1 * ng + 1) * 4:][:4].view("<u4")[0])
    assert word >> 16 == 0x8888 & ~0xF0 | 0xF0 and word & 0xFFFF == 0
    # scales of token 11: K groups, V groups
    s = rec[16 * d + 11 * 4 * ng:][:4 * ng].view("<u2")
    want = np.zeros(2 * ng, dtype=np.uint16)
    want[1] = want[ng + 1] = 0x3F80
    assert np.array_equal(s, want)
    # every nibble of the token holds code 0 (8) or 15, and nothing else was written
    assert np.count_nonzero(rec[:16 * d]) == 2 * (d // 2) and np.count_nonzero(rec[16 * d:]) == 4


@pytest.mark.parametrize("d", [64, 128])
def test_store_then_load(d):
    rng = np.random.default_rng(2)
    page, hkv, n_pages = 48, 3, 4
    cache = rng.integers(0, 256, (n_pages, hkv, serving.page_bytes(page, d)), dtype=np.uint8)
    slots = rng.permutation(n_pages * page)[:90]
    slots[7] = -1
    k, v = _bf16(rng.standard_normal((90, hkv, d))), _bf16(3 * rng.standard_normal((90, hkv, d)))
    serving.store(cache, page, slots, k, v)
    keep = slots >= 0
    gk, gv = serving.load(cache, page, slots[keep], d)
    assert np.array_equal(gk, serving.dequantise(*serving.quantise(k[keep])))
    assert np.array_equal(gv, serving.dequantise(*serving.quantise(v[keep])))


def test_page_tables_worked_by_hand():
    # pages of 16: request 0 fills its page, 1 starts, 2 grows over two pages, 3 sits out
    table = np.full((4, 4), -1)
    table[0, :1], table[2, :2], table[3, :1] = 9, (5, 6), 7
    t, cu, kv, pos, slots, to = serving.page_tables([15, 0, 20, 16], [1, 17, 13, 0], 16, [30, 31, 32, 33, 34], table, 34,
                                                    free_from=1)
    assert t.tolist() == [[9, -1, -1, -1], [31, 32, -1, -1], [5, 6, 33, -1], [7, -1, -1, -1]]
    assert cu.tolist() == [0, 1, 18, 31, 31] and kv.tolist() == [16, 17, 33, 16] and to == 4
    assert slots[0] == 9 * 16 + 15 and slots[1] == 31 * 16 and slots[17] == 32 * 16
    assert slots[18] == 6 * 16 + 4 and slots[29] == 6 * 16 + 15 and slots[30] == 33 * 16
    assert slots[31:].tolist() == [-1] * 3 and pos[18] == 20 and pos[31:].tolist() == [0] * 3


def test_page_tables_when_something_runs_out():
    t, cu, kv, pos, slots, to = serving.page_tables([0, 0], [20, 20], 16, [3, 4, 5], np.full((2, 2), -1), 30)
    assert t.tolist() == [[3, 4], [5, -1]] and to == 3
    assert cu.tolist() == [0, 20, 30] and slots[20] == 5 * 16 and slots[29] == 5 * 16 + 9
    t, cu, kv, pos, slots, to = serving.page_tables([0], [40], 16, [3, 4, 5], np.full((1, 2), -1), 40)
    assert kv.tolist() == [32] and slots[31] == 4 * 16 + 15 and (slots[32:] == -1).all() and to == 2


def test_packed_attention_is_each_sequence_alone():
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((12, 4, 8)), rng.standard_normal((12, 2, 8)), rng.standard_normal((12, 2, 8))
    out, vs = serving.packed_attention(q, k, v, [0, 5, 5, 11])
    assert np.array_equal(out[:5], causal_gqa_attention(q[:5], np.arange(5), k[:5], v[:5]))
    assert np.array_equal(out[5:11], causal_gqa_attention(q[5:11], np.arange(6), k[5:11], v[5:11]))
    assert np.isnan(out[11]).all() and np.allclose(out[5], np.repeat(v[5], 2, axis=0))
