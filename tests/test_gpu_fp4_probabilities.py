"""How many bits the E2M1 decode's probabilities keep in the product with V (needs a B200).

Two tokens with opposite V: out = 6 (p0 - p1) / (p0 + p1), where p1 / p0 = e^-delta is close to 1.  The output is
small beside what is summed, so its own rounding does not hide the probabilities'.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import fp4_ref as ref  # noqa: E402
from gpu_util import dev, dev_i32, host_bits  # noqa: E402
from paged_kv_cache_458_b200 import gen, pa  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_458_b200 import build

    build.build()
    pa.pa_last_device_error()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [gen.F16, gen.BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("group", [1, 4, 8, 16])
@pytest.mark.parametrize("d", [64, 128])
def test_probabilities_keep_more_than_one_f16(dtype, group, d):
    n, bs = 24, 8
    rng = np.random.default_rng(d + group)
    c = ref.quantised_case(rng, dtype=dtype, hq=group, hkv=1, d=d, bs=bs, ctx=[2] * n)
    one = np.ones(1, np.float32)
    for name in ("k", "v"):
        pool = ref.empty_pool4(c["num_blocks"], bs, 1, d, 0x7F)
        codes, scales = ref.pool4_views(pool, bs, d)
        for i in range(n):
            for t in range(2):
                row = np.full(d, 2, np.uint8)  # 1.0
                if name == "k" and t == 1:
                    row[:i + 1] = 1            # 0.5: a logit lower by (i + 1) / 2 of the scale
                if name == "v":
                    row[:] = 15 if t else 7    # 6, then -6
                b = c["block_tables"][i, 0]
                codes[b, 0, t] = row[0::2] | (row[1::2] << 4)
                scales[b, 0, t] = 0x38         # 1.0
        pool[..., :bs * d // 2], pool[..., bs * d // 2:] = codes.reshape(*pool.shape[:2], -1), scales.reshape(*pool.shape[:2], -1)
        c[name + "_pool"], c[name + "_scale"] = pool, one
    c["q"] = gen.to_bits(np.ones((n, group, d), np.float32), dtype)
    c["scale"] = 2.0 ** -9
    exact = ref.decode4(c, dtype)
    shape = pa.make_shape(num_seqs=n, num_q_heads=group, num_kv_heads=1, head_dim=d, block_size=bs,
                          num_blocks=c["num_blocks"], max_blocks_per_seq=c["block_tables"].shape[1], dtype=dtype,
                          cache_format=pa.PA_CACHE_FP4_E2M1)
    out = torch.full((n, group, d), float("nan"), dtype=pa.torch_dtype(dtype), device="cuda")
    ws = torch.empty(pa.pa_decode_workspace_bytes(shape, 2), dtype=torch.uint8, device="cuda")
    pa.pa_decode_fp4(dev(c["q"], dtype), *(torch.from_numpy(c[k]).cuda() for k in ("k_pool", "v_pool", "k_scale", "v_scale")),
                     dev_i32(c["block_tables"]), dev_i32(c["context_lens"]), c["scale"], out, shape, 2, ws)
    assert pa.pa_last_device_error()[0] == pa.PA_OK
    got = gen.bits_to_f32(host_bits(out), dtype)
    # Relative to each p: 2^-22 for an exponent of up to 8 in magnitude, rounded to 2^-21 (x ln 2), 2^-22 for the
    # exponential, 2^-23 for p as two f16; the sums' roundings are smaller.  Below 2^-20 together; both p's errors reach the
    # output through 6 / (p0 + p1), numerator and denominator: 6 x 2^-19 at most.  (One f16 for p alone: 6 x 2^-13.)
    half = {gen.F16: 2.0 ** -11, gen.BF16: 2.0 ** -8}[dtype]
    assert (np.abs(exact) > 1e-3).all() and (np.abs(exact) < 0.2).all()
    assert (np.abs(got - exact) <= np.abs(exact) * half * (1 + 2.0 ** -8) + 6 * 2.0 ** -19).all(), np.abs(got - exact).max()


@pytest.mark.parametrize("dtype", [gen.F16, gen.BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("scale", [0.0, 1e-30, 0.1])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_a_query_that_is_no_number_shows_at_any_scale(dtype, scale, bad):
    """NaN times a scale of zero is NaN, and so is infinity: not the mean of V.  (An infinite query meets codes of both
    signs, so its logits are NaN or of both signs at any other scale.)"""
    rng = np.random.default_rng(1)
    c = ref.quantised_case(rng, dtype=dtype, hq=8, hkv=2, d=64, bs=16, ctx=[70, 9])
    q = np.zeros((2, 8, 64), np.float32)
    q[0, 3, 5] = bad
    shape = pa.make_shape(num_seqs=2, num_q_heads=8, num_kv_heads=2, head_dim=64, block_size=16, num_blocks=c["num_blocks"],
                          max_blocks_per_seq=c["block_tables"].shape[1], dtype=dtype, cache_format=pa.PA_CACHE_FP4_E2M1)
    out = torch.zeros((2, 8, 64), dtype=pa.torch_dtype(dtype), device="cuda")
    ws = torch.empty(pa.pa_decode_workspace_bytes(shape, 70), dtype=torch.uint8, device="cuda")
    pa.pa_decode_fp4(dev(gen.to_bits(q, dtype), dtype),
                     *(torch.from_numpy(c[k]).cuda() for k in ("k_pool", "v_pool", "k_scale", "v_scale")),
                     dev_i32(c["block_tables"]), dev_i32(c["context_lens"]), scale, out, shape, 70, ws)
    assert pa.pa_last_device_error()[0] == pa.PA_OK
    nan = np.isnan(gen.bits_to_f32(host_bits(out), dtype)).all(-1)
    want = np.zeros((2, 8), bool)
    want[0, 3] = True
    assert np.array_equal(nan, want)
