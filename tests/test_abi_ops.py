"""Host-side validation of the rotating append, the E2M1 cache calls and the gather (no GPU)."""
import ctypes

import pytest

from paged_kv_cache_458_b200 import pa

FAKE = 1 << 20  # a 16-byte-aligned non-null address; validation fails before any use
OK, INVALID, UNSUPPORTED = pa.PA_OK, pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_458_b200 import build

    build.build()
    return pa.lib()


def _shape(**kw):
    base = dict(num_seqs=4, num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16, num_blocks=64,
                max_blocks_per_seq=8, dtype=pa.PA_F16, cache_format=pa.PA_CACHE_FP4_E2M1)
    base.update(kw)
    return ctypes.byref(pa.make_shape(**base))


def _decode(lib, shape, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, bt=FAKE, cl=FAKE, scale=0.1, out=FAKE, maxlen=100, ws=FAKE,
             nbytes=1 << 30)
    a.update(kw)
    return lib.pa_decode_fp4(a["q"], a["k"], a["v"], a["ks"], a["vs"], a["bt"], a["cl"], a["scale"], a["out"], shape,
                             a["maxlen"], a["ws"], a["nbytes"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(cache_format=pa.PA_CACHE_AS_DTYPE), INVALID), (dict(cache_format=pa.PA_CACHE_FP8_E4M3), INVALID),
    (dict(cache_format=3), UNSUPPORTED), (dict(variant=pa.PA_DECODE_CUDA_CORES), UNSUPPORTED),
    (dict(variant=pa.PA_DECODE_TENSOR_CORES), UNSUPPORTED), (dict(variant=7), INVALID),
    (dict(shared_prefix=1), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED), (dict(block_size=12), UNSUPPORTED),
    (dict(num_q_heads=7), INVALID), (dict(num_q_heads=64), UNSUPPORTED), (dict(partition_tokens=24), UNSUPPORTED),
    (dict(partition_tokens=4096), UNSUPPORTED), (dict(num_blocks=1 << 27), UNSUPPORTED), (dict(num_seqs=-1), INVALID),
    (dict(num_blocks=0), INVALID), (dict(dtype=2), UNSUPPORTED), (dict(max_blocks_per_seq=6), INVALID),
    (dict(num_seqs=1 << 30), INVALID), (dict(num_seqs=1 << 28, num_kv_heads=8), UNSUPPORTED),
])
def test_decode_fp4_rejects_bad_shapes(lib, kw, want):
    assert _decode(lib, _shape(**kw)) == want


@pytest.mark.parametrize("kw", [{n: None} for n in ("q", "k", "v", "ks", "vs", "bt", "cl", "out", "ws")]
                         + [{n: FAKE + 8} for n in ("q", "k", "v", "out", "ws")]
                         + [{n: FAKE + 2} for n in ("ks", "vs", "bt", "cl")]
                         + [dict(scale=float("nan")), dict(scale=float("inf")), dict(maxlen=-1), dict(nbytes=100),
                            dict(maxlen=129)])
def test_decode_fp4_rejects_bad_arguments(lib, kw):
    assert _decode(lib, _shape(), **kw) == INVALID


def test_decode_fp4_refuses_more_than_2_to_the_30_sequences_or_tokens(lib):
    one = dict(num_q_heads=1, num_kv_heads=1, max_blocks_per_seq=(1 << 27) + 1)
    assert _decode(lib, _shape(num_seqs=(1 << 30) + 1, **one), maxlen=16) == UNSUPPORTED
    assert _decode(lib, _shape(num_seqs=1, **one), maxlen=(1 << 30) + 1) == UNSUPPORTED


def test_decode_fp4_of_no_sequences_launches_nothing(lib):
    n = pa.pa_kernel_launches()
    assert _decode(lib, _shape(num_seqs=0), q=None) == OK
    assert pa.pa_kernel_launches() == n


def test_other_calls_refuse_an_fp4_cache(lib):
    s = _shape()
    args = (FAKE, FAKE, FAKE, FAKE, FAKE, 0.1, FAKE, s)
    assert lib.pa_decode(*args, 100, FAKE, 1 << 30, None) == INVALID
    assert lib.pa_decode_noalloc(*args, 100, None) == INVALID
    assert lib.pa_decode_multi(*args, 2, 100, FAKE, 1 << 30, None) == INVALID
    assert lib.pa_decode_fp8(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0.1, FAKE, s, 100, FAKE, 1 << 30, None) == INVALID
    assert lib.pa_cache_append(FAKE, FAKE, FAKE, 3, FAKE, FAKE, s, None) == INVALID
    assert lib.pa_cache_append_fp8(FAKE, FAKE, FAKE, 3, FAKE, FAKE, FAKE, FAKE, s, None) == INVALID


def test_fp4_workspace_follows_the_work(lib):
    """Larger partitions never need more workspace, and no batch more than a full device's workers do."""
    most = 0
    for seqs, maxlen in ((1, 0), (1, 1), (1, 1000), (6, 131071), (64, 1024), (256, 4096), (4096, 4096)):
        s = pa.make_shape(num_seqs=seqs, num_q_heads=32, num_kv_heads=8, head_dim=128, block_size=16, num_blocks=64,
                          max_blocks_per_seq=8192, cache_format=pa.PA_CACHE_FP4_E2M1)
        auto = pa.pa_decode_workspace_bytes(s, maxlen)
        most = max(most, auto)
        for pt in (64, 128, 2048):
            s.partition_tokens = pt
            assert 0 < pa.pa_decode_workspace_bytes(s, maxlen) <= auto
        assert pa.pa_decode_partition_tokens(s) == 2048
    assert auto == most < 1 << 25
    assert pa.pa_decode_resolved_variant(s) == pa.PA_DECODE_TENSOR_CORES


@pytest.mark.parametrize("i", range(8))
def test_append_fp4_rejects_bad_arguments(lib, i):
    args = [FAKE, FAKE, FAKE, 3, FAKE, FAKE, FAKE, FAKE]
    for bad in ((-1,) if i == 3 else (None, FAKE + 2)):
        a = list(args)
        a[i] = bad
        assert lib.pa_cache_append_fp4(*a, _shape(), None) == INVALID
    assert lib.pa_cache_append_fp4(*args, _shape(cache_format=0), None) == INVALID
    assert lib.pa_cache_append_fp4(None, None, None, 0, None, None, None, None, _shape(), None) == OK


def _rope(lib, shape, rope_kw=None, **kw):
    rope = pa.make_rope(**dict(dict(rotary_dim=64, max_position=100), **(rope_kw or {})))
    a = dict(q=FAKE, k=FAKE, v=FAKE, pos=FAKE, cs=FAKE, slots=FAKE, n=3, qo=2 * FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE)
    a.update(kw)
    return lib.pa_rope_append(a["q"], a["k"], a["v"], a["pos"], a["cs"], kw.get("rope", ctypes.byref(rope)), a["slots"],
                              a["n"], a["qo"], a["kc"], a["vc"], a["ks"], a["vs"], shape, None)


@pytest.mark.parametrize("kw", [{n: None} for n in ("q", "k", "v", "pos", "cs", "slots", "qo", "kc", "vc", "ks", "vs", "rope")]
                         + [{n: FAKE + 8} for n in ("q", "k", "v", "cs", "qo", "kc", "vc")]
                         + [{n: FAKE + 2} for n in ("pos", "slots", "ks", "vs")] + [dict(n=-1)])
def test_rope_append_rejects_bad_arguments(lib, kw):
    assert _rope(lib, _shape(), **kw) == INVALID


@pytest.mark.parametrize("rope_kw,want", [
    (dict(rotary_dim=0), INVALID), (dict(rotary_dim=-16), INVALID), (dict(rotary_dim=144), INVALID),
    (dict(rotary_dim=24), UNSUPPORTED), (dict(max_position=0), INVALID), (dict(interleaved=2), INVALID),
    (dict(q_stride=1016), INVALID), (dict(k_stride=248), INVALID), (dict(v_stride=260), INVALID),
    (dict(q_out_stride=1030), INVALID), (dict(q_stride=-1024), INVALID),
])
def test_rope_append_rejects_bad_rotations(lib, rope_kw, want):
    assert _rope(lib, _shape(), rope_kw) == want


def test_rope_append_scales_follow_the_format(lib):
    assert _rope(lib, _shape(cache_format=pa.PA_CACHE_AS_DTYPE)) == INVALID
    assert _rope(lib, _shape(cache_format=pa.PA_CACHE_FP8_E4M3), ks=None) == INVALID
    assert _rope(lib, _shape(num_q_heads=0)) == INVALID
    # in place only with q's own stride
    assert _rope(lib, _shape(), dict(q_stride=2048), qo=FAKE) == INVALID
    assert _rope(lib, _shape(), n=0, q=None) == OK


@pytest.mark.parametrize("i", range(8))
def test_gather_rejects_bad_arguments(lib, i):
    args = [FAKE, 3, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE]
    for bad in ((-1,) if i == 1 else (None, FAKE + 2)):
        a = list(args)
        a[i] = bad
        assert lib.pa_cache_gather(*a, _shape(), None) == INVALID
    assert lib.pa_cache_gather(None, 0, None, None, None, None, None, None, _shape(), None) == OK


def test_rope_append_refuses_a_reserved_field_in_use(lib):
    rope = pa.make_rope(rotary_dim=64, max_position=100)
    rope.reserved = 1
    assert _rope(lib, _shape(), rope=ctypes.byref(rope)) == INVALID
