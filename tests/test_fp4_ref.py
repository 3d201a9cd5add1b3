"""The E2M1 reference of the GPU tests, pinned on the CPU: tables, ties, ranges, layout."""
import numpy as np
import pytest

import fp4_ref as ref
from paged_kv_cache_458_b200 import gen


def test_e4m3_table_matches_the_oracle(orc):
    for c in range(256):
        want = orc.e4m3_to_f64(c)
        assert (np.isnan(want) and np.isnan(ref.E4M3[c])) or ref.E4M3[c] == want


def test_e2m1_ties_go_to_the_even_code():
    # block scale 1 (amax 6, head scale 1): the codes are those of the values themselves
    x = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, 0.0], np.float32)
    code, s = ref.quantise4(x.reshape(1, 1, 16), np.ones(1, np.float32))
    assert ref.E4M3[s].item() == 1.0
    assert code.ravel().tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 8, 10, 10, 12, 12, 14, 14, 0]


def test_zero_nan_and_infinite_blocks():
    x = np.zeros((1, 1, 64), np.float32)
    x[..., 16] = np.nan
    x[..., 32] = np.inf
    x[..., 48] = 1e-9
    code, s = ref.quantise4(x, np.full(1, 0.1, np.float32))
    assert s.ravel().tolist() == [0, 0x7F, 0x7E, 0]
    assert code[0, 0, 32] == 7 and not code[0, 0, 48:].any()


@pytest.mark.parametrize("d", [64, 128])
def test_store_and_rows_agree_and_hold_the_error_bound(d):
    rng = np.random.default_rng(5 + d)
    hkv, bs, nb, t = 3, 24, 4, 50
    scale = rng.uniform(0.08, 0.18, hkv).astype(np.float32)
    x = rng.standard_normal((t, hkv, d)).astype(np.float32)
    slots = rng.choice(nb * bs, t, replace=False)
    slots[7] = -1
    pool = ref.empty_pool4(nb, bs, hkv, d, 0xEE)
    ref.store4(pool, bs, d, slots, x, scale)
    keep = slots >= 0
    got = ref.rows4(pool, bs, d, slots[keep], scale)
    amax = np.abs(x[keep]).reshape(keep.sum(), hkv, -1, 16).max(-1).repeat(16, axis=-1)
    # half an E2M1 step at the top (1 of 6), and the scale's own half step (2^-4 relative) where it clips
    assert (np.abs(got - x[keep]) <= amax * (1 / 6 + 2.0 ** -4) * 1.001).all()
    untouched = np.setdiff1d(np.arange(nb * bs), slots)
    codes, scales = ref.pool4_views(pool, bs, d)
    assert (codes[untouched // bs, :, untouched % bs] == 0xEE).all()
    assert (scales[untouched // bs, :, untouched % bs] == 0xEE).all()


def test_rotation_keeps_norms_and_inverts():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((4, 2, 64))
    th = rng.uniform(0, 6, (4, 24))
    for inter in (False, True):
        y = ref.rotate(x, np.cos(th), np.sin(th), 48, inter, np.float64)
        z = ref.rotate(y, np.cos(th), -np.sin(th), 48, inter, np.float64)
        assert np.allclose(z, x, atol=1e-14) and np.array_equal(y[..., 48:], x[..., 48:])
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))


def test_case_poison_is_only_where_nothing_may_read():
    rng = np.random.default_rng(9)
    c = ref.quantised_case(rng, dtype=gen.BF16, hq=4, hkv=2, d=64, bs=8, ctx=[0, 5, 17])
    out = ref.decode4(c, gen.BF16)
    assert np.isfinite(out).all() and not out[0].any()
    assert (c["block_tables"][1, 1:] == 1 << 30).all()
