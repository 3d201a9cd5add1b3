"""partition_tokens of the E2M1 decode is the least a warp takes, whatever bound the caller gives (needs a B200)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import fp4_ref as ref  # noqa: E402
from gpu_util import dev, dev_i32, host_bits  # noqa: E402
from paged_kv_cache_458_b200 import gen, pa  # noqa: E402
from tolerance import assert_decode_close  # noqa: E402

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


@pytest.mark.parametrize("group,d,partition", [(4, 128, 2048), (4, 128, 320), (8, 64, 1024), (16, 64, 256), (16, 128, 2048)])
def test_a_loose_bound_does_not_shorten_the_spans(group, d, partition):
    """The split follows from the contexts and partition_tokens: with a bound far above them, as a captured step has,
    the same spans are cut, and the bits show it."""
    rng = np.random.default_rng(group + d + partition)
    c = ref.quantised_case(rng, dtype=gen.F16, hq=2 * group, hkv=2, d=d, bs=16,
                           ctx=[64] * 5 + [3000, 0, 1, 130, 5000, 900, 64, 64, 2050])
    exact = ref.decode4(c, gen.F16)
    c["block_tables"] = np.pad(c["block_tables"], ((0, 0), (0, 8192 - c["block_tables"].shape[1])), constant_values=-1)
    s, hq, _ = c["q"].shape
    shape = pa.make_shape(num_seqs=s, num_q_heads=hq, num_kv_heads=2, head_dim=d, block_size=16, num_blocks=c["num_blocks"],
                          max_blocks_per_seq=8192, dtype=gen.F16, cache_format=pa.PA_CACHE_FP4_E2M1,
                          partition_tokens=partition)
    args = [dev(c["q"], gen.F16)] + [torch.from_numpy(c[k]).cuda() for k in ("k_pool", "v_pool", "k_scale", "v_scale")]
    args += [dev_i32(c["block_tables"]), dev_i32(c["context_lens"]), c["scale"]]
    got = []
    for bound in (5000, 8000, 131072):
        ws = torch.empty(pa.pa_decode_workspace_bytes(shape, bound), dtype=torch.uint8, device="cuda")
        out = torch.full(c["q"].shape, float("nan"), dtype=torch.float16, device="cuda")
        pa.pa_decode_fp4(*args, out, shape, bound, ws)
        assert pa.pa_last_device_error()[0] == pa.PA_OK
        got.append(host_bits(out))
        assert_decode_close(got[-1], exact, gen.F16, f"bound {bound}")
    assert np.array_equal(got[0], got[1]) and np.array_equal(got[0], got[2])
