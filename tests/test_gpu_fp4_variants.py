"""Every compiled form of the E2M1 decode against fp64 attention (needs a B200).

A form is a type, a head size, a group class (up to 4, 8, 16 heads), the tokens of one copy (8, 16 or 32, by the block
size), and at 16 heads of 64 whether a CTA's warps share a span (fewer items than the 444 CTAs of a device) or not.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import fp4_ref as ref  # noqa: E402
from gpu_util import dev, dev_i32, host_bits  # noqa: E402
from paged_kv_cache_458_b200 import gen, pa  # noqa: E402
from tolerance import assert_decode_close  # noqa: E402

pytestmark = pytest.mark.gpu
DTYPES = pytest.mark.parametrize("dtype", [gen.F16, gen.BF16], ids=["f16", "bf16"])


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_458_b200 import build

    build.build()
    pa.pa_last_device_error()
    yield
    torch.cuda.empty_cache()


def _check(c, dtype, partitions):
    exact = ref.decode4(c, dtype)
    s, hq, d = c["q"].shape
    args = [dev(c["q"], dtype)] + [torch.from_numpy(c[k]).cuda() for k in ("k_pool", "v_pool", "k_scale", "v_scale")]
    args += [dev_i32(c["block_tables"]), dev_i32(c["context_lens"]), c["scale"]]
    n = int(c["context_lens"].max())
    for p in partitions:
        shape = pa.make_shape(num_seqs=s, num_q_heads=hq, num_kv_heads=c["k_pool"].shape[1], head_dim=d,
                              block_size=c["block_size"], num_blocks=c["num_blocks"],
                              max_blocks_per_seq=c["block_tables"].shape[1], dtype=dtype, partition_tokens=p,
                              cache_format=pa.PA_CACHE_FP4_E2M1)
        ws = torch.randint(0, 256, (pa.pa_decode_workspace_bytes(shape, n),), dtype=torch.uint8, device="cuda")
        got = []
        for _ in range(2):
            out = torch.full(c["q"].shape, float("nan"), dtype=pa.torch_dtype(dtype), device="cuda")
            pa.pa_decode_fp4(*args, out, shape, n, ws)
            status, bits = pa.pa_last_device_error()
            assert status == pa.PA_OK, f"device check fired: {bits:#x}"
            got.append(host_bits(out))
        assert_decode_close(got[0], exact, dtype, f"partition {p}")
        assert np.array_equal(got[0], got[1])


@DTYPES
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [2, 8, 16])
@pytest.mark.parametrize("bs", [8, 16, 24, 32, 48, 64, 96, 256])
def test_few_items(dtype, d, group, bs):
    """Cut into parts, whole short ones between long ones, empty ones; blocks that end inside a copy's reach."""
    rng = np.random.default_rng(bs + group + d + dtype)
    c = ref.quantised_case(rng, dtype=dtype, hq=2 * group, hkv=2, d=d, bs=bs,
                           ctx=[bs, 0, 2500, 1, 64, 65, bs - 1, bs + 1, 0, 256, 257, 200, 31, 3 * bs + 7, 1100, 5])
    _check(c, dtype, (0, 320, 2048))


@DTYPES
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 4, 8, 16])
@pytest.mark.parametrize("bs", [8, 32])
@pytest.mark.parametrize("items", [443, 444])
def test_many_items(dtype, d, group, bs, items):
    rng = np.random.default_rng(bs + group + d + items)
    ctx = rng.integers(0, 140, items)
    ctx[[5, 200, 440]] = 0, 1900, 700
    c = ref.quantised_case(rng, dtype=dtype, hq=group, hkv=1, d=d, bs=bs, ctx=list(ctx))
    _check(c, dtype, (0, 640))
