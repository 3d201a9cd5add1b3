"""The E2M1 decode repeated: the same inputs must give the same bits, whoever arrives last (needs a B200)."""
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


def _repeat(c, dtype, times):
    """Runs a case `times` times on one workspace, a copy of other data between the runs (the cache's state differs);
    checks the first output against fp64 and all of them against it."""
    s, hq, d = c["q"].shape
    shape = pa.make_shape(num_seqs=s, num_q_heads=hq, num_kv_heads=c["k_pool"].shape[1], head_dim=d,
                          block_size=c["block_size"], num_blocks=c["num_blocks"],
                          max_blocks_per_seq=c["block_tables"].shape[1], dtype=dtype, cache_format=pa.PA_CACHE_FP4_E2M1)
    n = int(c["context_lens"].max())
    ws = torch.randint(0, 256, (pa.pa_decode_workspace_bytes(shape, n),), dtype=torch.uint8, device="cuda")
    args = [dev(c["q"], dtype)] + [torch.from_numpy(c[k]).cuda() for k in ("k_pool", "v_pool", "k_scale", "v_scale")]
    args += [dev_i32(c["block_tables"]), dev_i32(c["context_lens"]), c["scale"]]
    outs = torch.full((times, s, hq, d), float("nan"), dtype=pa.torch_dtype(dtype), device="cuda")
    noise = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    for i in range(times):
        if i % 3 == 1:
            noise[: (i % 7 + 1) << 20].add_(1)
        elif i % 3 == 2:
            noise.add_(1)
        pa.pa_decode_fp4(*args, outs[i], shape, n, ws)
    status, bits = pa.pa_last_device_error()
    assert status == pa.PA_OK, f"device check fired: {bits:#x}"
    got = host_bits(outs)
    assert_decode_close(got[0], ref.decode4(c, dtype), dtype)
    differ = [i for i in range(1, times) if not np.array_equal(got[i], got[0])]
    assert not differ, f"runs {differ} of {times} differ from the first"


@pytest.mark.parametrize("dtype", [gen.F16, gen.BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("group,d", [(1, 64), (4, 128), (8, 64), (8, 128), (16, 128)])
def test_merges_repeat(dtype, group, d):
    """Items cut into one to hundreds of parts: every level of the merges, many times."""
    rng = np.random.default_rng(group + d + dtype)
    c = ref.quantised_case(rng, dtype=dtype, hq=2 * group, hkv=2, d=d, bs=16, ctx=[130, 700, 1600, 5000, 12000])
    _repeat(c, dtype, 40)


@pytest.mark.parametrize("dtype", [gen.F16, gen.BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("ctx", [[20000], [8000, 7000, 50, 300, 0, 8192], [64, 5, 0, 2000, 63, 65, 192, 256, 257, 320, 9, 8000],
                                 [130, 250, 40, 1, 200, 100, 64, 12, 31] * 4 + [3000]],
                         ids=["one", "long", "ragged", "short"])
@pytest.mark.parametrize("bs", [8, 16, 64])
def test_teams_repeat(dtype, ctx, bs):
    """16 heads of 64 and fewer items than CTAs: a CTA's warps share a span, and which of them adds what up must not
    follow from whose copies land first."""
    rng = np.random.default_rng(len(ctx) + bs)
    c = ref.quantised_case(rng, dtype=dtype, hq=32, hkv=2, d=64, bs=bs, ctx=ctx)
    _repeat(c, dtype, 60)
