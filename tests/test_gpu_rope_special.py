"""The rotating append against the plain one on rows of extreme values (needs a B200)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from gpu_util import dev, dev_i32  # noqa: E402
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


@pytest.mark.parametrize("dtype,top", [(gen.BF16, 3e38), (gen.F16, 6e4)], ids=["bf16", "f16"])
@pytest.mark.parametrize("scale", [0.1, 2.0 ** -70, 2.0 ** 70, 1.7e-38, 3e38])
def test_e4m3_codes_of_nan_infinity_and_overflow(dtype, top, scale):
    """NaN, infinities, zeros of both signs and quotients beyond fp32, together in the 8 dims that one lane converts and
    apart: the codes are those of pa_cache_append_fp8, byte for byte.  What rotates turns by zero degrees and is finite."""
    hkv, d, bs, rotary = 2, 64, 16, 16
    specials = np.array([np.nan, np.inf, -np.inf, top, -top, 0.0, -0.0, 1.0, -1e-7, 448.0], np.float32)
    rows = []
    for i in range(len(specials)):
        for j in range(len(specials)):
            x = np.full(d, 0.25, np.float32)
            x[rotary + 3], x[rotary + 6] = specials[i], specials[j]  # in one unit of 8
            x[rotary + 9], x[rotary + 17] = specials[j], specials[i]  # each with finite neighbours
            rows.append(np.stack([x, np.roll(x, 8 * (i % 3))]))
    t = len(rows)
    v = gen.to_bits(np.stack(rows), dtype)
    k = gen.to_bits(np.stack([np.stack([r[0], r[0]]) for r in rows]), dtype)
    nb = -(-t // bs)
    shape = pa.make_shape(num_seqs=1, num_q_heads=hkv, num_kv_heads=hkv, head_dim=d, block_size=bs, num_blocks=nb,
                          max_blocks_per_seq=1, dtype=dtype, cache_format=pa.PA_CACHE_FP8_E4M3)
    slots = dev_i32(np.arange(t))
    ks, vs = (torch.full((hkv,), scale, dtype=torch.float32, device="cuda") for _ in range(2))
    want = [torch.full((nb, bs, hkv, d), 0x55, dtype=torch.uint8, device="cuda") for _ in range(2)]
    got = [w.clone() for w in want]
    pa.pa_cache_append_fp8(dev(k, dtype), dev(v, dtype), slots, t, *want, ks, vs, shape)
    cos_sin = torch.tensor([[1.0] * (rotary // 2) + [0.0] * (rotary // 2)], device="cuda")
    q = torch.zeros((t, hkv, d), dtype=pa.torch_dtype(dtype), device="cuda")
    pa.pa_rope_append(q, dev(k, dtype), dev(v, dtype), torch.zeros(t, dtype=torch.int32, device="cuda"), cos_sin,
                      pa.make_rope(rotary_dim=rotary, max_position=1), slots, t, torch.empty_like(q), *got, ks, vs, shape)
    assert pa.pa_last_device_error()[0] == pa.PA_OK
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w.cpu().numpy())
