"""The E2M1 cache against plain fp64 references, through the C ABI (needs a B200).

Appends must leave the pools byte-identical to the reference's codes; the
decode must meet the decode tolerance against fp64 attention over the stored
values.  What that tolerance has to cover: the output's rounding; for bf16
outputs the probabilities' rounding to fp16 (2^-11 of each, an eighth of the
output's half step); logits summed in fp32.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import fp4_ref as ref  # noqa: E402
from gpu_util import dev, dev_i32, host_bits  # noqa: E402
from paged_kv_cache_458_b200 import gen, pa  # noqa: E402
from tolerance import assert_decode_close  # noqa: E402

pytestmark = pytest.mark.gpu
F32 = np.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_458_b200 import build

    build.build()
    pa.pa_last_device_error()
    yield
    torch.cuda.empty_cache()


def _gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _shape(c, dtype, **kw):
    s, hq, d = c["q"].shape
    return pa.make_shape(**dict(dict(num_seqs=s, num_q_heads=hq, num_kv_heads=c["k_pool"].shape[1], head_dim=d,
                                     block_size=c["block_size"], num_blocks=c["num_blocks"],
                                     max_blocks_per_seq=c["block_tables"].shape[1], dtype=dtype,
                                     cache_format=pa.PA_CACHE_FP4_E2M1), **kw))


def _decode(c, dtype, maxlen=None, ok=True, scale=None, **kw):
    shape = _shape(c, dtype, **kw)
    maxlen = int(np.max(c["context_lens"], initial=0)) if maxlen is None else maxlen
    nbytes = pa.pa_decode_workspace_bytes(shape, maxlen)
    ws = torch.randint(0, 256, (max(16, nbytes),), dtype=torch.uint8, device="cuda")
    out = torch.full(c["q"].shape, float("nan"), dtype=pa.torch_dtype(dtype), device="cuda")
    pa.pa_decode_fp4(dev(c["q"], dtype), _gpu(c["k_pool"]), _gpu(c["v_pool"]), _gpu(c["k_scale"]), _gpu(c["v_scale"]),
                     dev_i32(c["block_tables"]), dev_i32(c["context_lens"]), c["scale"] if scale is None else scale, out,
                     shape, maxlen, ws, nbytes)
    if ok:
        status, bits = pa.pa_last_device_error()
        assert status == pa.PA_OK, f"device check fired: {bits:#x}"
    return host_bits(out)


# ---------------------------------------------------------------------------
# append


@pytest.mark.parametrize("dtype", [gen.F16, gen.BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("hkv,d,bs,t", [(1, 64, 8, 1), (4, 128, 16, 60), (3, 64, 24, 131), (32, 128, 256, 300),
                                        (7, 128, 40, 77)])
def test_append_bit_exact(dtype, hkv, d, bs, t):
    rng = np.random.default_rng(t + d)
    nb = -(-t // bs) + 2
    k, v = (gen.normal_bits(rng, (t, hkv, d), dtype) for _ in range(2))
    f = gen.bits_to_f32(k, dtype).copy()
    f[0, :, :16] = 0.0
    f[0, :, 16:32] = -1e-7
    f[0, 0, 40] = 3e4
    f[0, 0, 50:60] = 2.0 ** -14
    k = gen.to_bits(f, dtype)
    ks, vs = (rng.uniform(0.05, 0.2, hkv).astype(F32) for _ in range(2))
    slots = rng.choice(nb * bs, t, replace=False).astype(np.int32)
    if t > 20:
        slots[[3, 17]] = -1
    k0 = rng.integers(0, 256, (nb, hkv, bs * d * 9 // 16), dtype=np.uint8)
    kc, vc = _gpu(k0), _gpu(k0)
    shape = pa.make_shape(num_seqs=1, num_q_heads=hkv, num_kv_heads=hkv, head_dim=d, block_size=bs, num_blocks=nb,
                          max_blocks_per_seq=1, dtype=dtype, cache_format=pa.PA_CACHE_FP4_E2M1)
    pa.pa_cache_append_fp4(dev(k, dtype), dev(v, dtype), dev_i32(slots), t, kc, vc, _gpu(ks), _gpu(vs), shape)
    assert pa.pa_last_device_error()[0] == pa.PA_OK
    for x, got, scale in ((k, kc, ks), (v, vc, vs)):
        want = k0.copy()
        ref.store4(want, bs, d, slots, gen.bits_to_f32(x, dtype), scale)
        assert np.array_equal(got.cpu().numpy(), want)


def test_append_every_tie_and_scale():
    """Midpoints between codes under every block scale, and block maxima between scales."""
    hkv, d, bs = 1, 64, 16
    mids = (ref.E2M1[1:] + ref.E2M1[:-1]) / 2
    base = np.concatenate([[6.0], mids, -mids, [0.0]])
    scales = ref.E4M3[1:0x7F]
    x = (scales[:, None] * base).astype(F32)                    # block scale = that scale, values at ties
    amax = np.zeros((126, 16), F32)
    amax[:125, 0] = 6 * (scales[1:] + scales[:-1]) / 2          # the scale itself at a tie
    x = np.concatenate([x, amax])
    x = np.concatenate([x, np.zeros((-len(x) % 4, 16), F32)]).reshape(-1, hkv, d)
    bits = gen.to_bits(x, gen.F16)
    t = len(x)
    nb = -(-t // bs)
    slots = np.arange(t, dtype=np.int32)
    kc = _gpu(ref.empty_pool4(nb, bs, hkv, d))
    vc = _gpu(ref.empty_pool4(nb, bs, hkv, d))
    one = np.ones(1, F32)
    shape = pa.make_shape(num_seqs=1, num_q_heads=1, num_kv_heads=1, head_dim=d, block_size=bs, num_blocks=nb,
                          max_blocks_per_seq=1, dtype=gen.F16, cache_format=pa.PA_CACHE_FP4_E2M1)
    pa.pa_cache_append_fp4(dev(bits, gen.F16), dev(bits, gen.F16), dev_i32(slots), t, kc, vc, _gpu(one), _gpu(one), shape)
    want = ref.empty_pool4(nb, bs, hkv, d)
    ref.store4(want, bs, d, slots, gen.bits_to_f32(bits, gen.F16), one)
    assert np.array_equal(kc.cpu().numpy(), want) and np.array_equal(vc.cpu().numpy(), want)


def test_append_nan_and_infinity():
    hkv, d, bs, t = 2, 64, 8, 3
    x = np.ones((t, hkv, d), F32)
    x[0, 0, 17] = np.nan
    x[1, 1, 33] = np.inf
    x[2, 0, 5] = -np.inf
    for dtype in (gen.F16, gen.BF16):
        bits = gen.to_bits(x, dtype)
        kc, vc = _gpu(ref.empty_pool4(1, bs, hkv, d)), _gpu(ref.empty_pool4(1, bs, hkv, d))
        sc = np.full(hkv, 0.25, F32)
        shape = pa.make_shape(num_seqs=1, num_q_heads=2, num_kv_heads=2, head_dim=d, block_size=bs, num_blocks=1,
                              max_blocks_per_seq=1, dtype=dtype, cache_format=pa.PA_CACHE_FP4_E2M1)
        pa.pa_cache_append_fp4(dev(bits, dtype), dev(bits, dtype), dev_i32([0, 1, 2]), t, kc, vc, _gpu(sc), _gpu(sc), shape)
        ko, vo = (torch.zeros((t, hkv, d), dtype=pa.torch_dtype(dtype), device="cuda") for _ in range(2))
        pa.pa_cache_gather(dev_i32([0, 1, 2]), t, kc, vc, _gpu(sc), _gpu(sc), ko, vo, shape)
        assert pa.pa_last_device_error()[0] == pa.PA_OK
        got = ko.float().cpu().numpy()
        nan = np.zeros(x.shape, bool)
        nan[0, 0, 16:32] = True
        assert np.array_equal(np.isnan(got), nan)
        # an infinity: block scale 448, code 6; its neighbours fall below the smallest code
        assert got[1, 1, 33] == 6 * 448 * 0.25 and got[2, 0, 5] == -6 * 448 * 0.25 and got[1, 1, 32] == 0


# ---------------------------------------------------------------------------
# attention


@pytest.mark.parametrize("dtype", [gen.F16, gen.BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("group", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_matches_fp64(dtype, group, d):
    rng = np.random.default_rng(100 * group + d + dtype)
    hkv = 3
    c = ref.quantised_case(rng, dtype=dtype, hq=hkv * group, hkv=hkv, d=d, bs=16,
                           ctx=[1, 0, 17, 300, 64, 15, 16, 129, 1000, 33])
    exact = ref.decode4(c, dtype)
    for pt in (0, 16, 48, 128, 2048):
        assert_decode_close(_decode(c, dtype, partition_tokens=pt), exact, dtype, f"partition {pt}")


@pytest.mark.parametrize("bs", [8, 16, 24, 32, 40, 48, 64, 128, 256])
def test_decode_block_sizes(bs):
    for d, group, hkv in ((128, 4, 2), (64, 1, 5)):
        rng = np.random.default_rng(bs + d)
        c = ref.quantised_case(rng, dtype=gen.BF16, hq=hkv * group, hkv=hkv, d=d, bs=bs,
                               ctx=[bs, bs - 1, bs + 1, 1, 3 * bs + 7, 777, 0, 2500])
        exact = ref.decode4(c, gen.BF16)
        for pt in (0, 16, 80, 1024):
            assert_decode_close(_decode(c, gen.BF16, partition_tokens=pt), exact, gen.BF16, f"bs {bs} partition {pt}")


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 31, 32, 33, 63, 64, 65, 127, 128, 255, 257])
def test_decode_every_tail(n):
    rng = np.random.default_rng(n)
    c = ref.quantised_case(rng, dtype=gen.F16, hq=8, hkv=2, d=128, bs=8, ctx=[n])
    assert_decode_close(_decode(c, gen.F16), ref.decode4(c, gen.F16), gen.F16, f"ctx {n}")


def test_decode_all_contexts_empty():
    rng = np.random.default_rng(1)
    c = ref.quantised_case(rng, dtype=gen.F16, hq=4, hkv=2, d=64, bs=16, ctx=[0, 0])
    assert not _decode(c, gen.F16).any()
    assert not _decode(c, gen.F16, maxlen=16).any()


def test_decode_long_context_and_many_sequences():
    rng = np.random.default_rng(2)
    c = ref.quantised_case(rng, dtype=gen.BF16, hq=16, hkv=2, d=128, bs=16, ctx=[30011, 5, 0, 9000])
    assert_decode_close(_decode(c, gen.BF16), ref.decode4(c, gen.BF16), gen.BF16, "long")
    c = ref.quantised_case(rng, dtype=gen.F16, hq=4, hkv=1, d=64, bs=16, ctx=list(rng.integers(0, 200, 300)))
    assert_decode_close(_decode(c, gen.F16), ref.decode4(c, gen.F16), gen.F16, "many")


@pytest.mark.parametrize("dtype,d,group,bs", [(gen.BF16, 128, 4, 16), (gen.F16, 64, 1, 8), (gen.F16, 128, 8, 64),
                                              (gen.BF16, 64, 16, 24)])
def test_decode_many_items_with_long_ones(dtype, d, group, bs):
    """More items than CTAs: warps work alone; a long item among short ones is merged over several levels."""
    rng = np.random.default_rng(20 + d + group)
    ctx = rng.integers(0, 150, 160)
    ctx[[3, 77]] = 9000, 2100
    ctx[[0, 50, 159]] = 0
    c = ref.quantised_case(rng, dtype=dtype, hq=3 * group, hkv=3, d=d, bs=bs, ctx=list(ctx))
    exact = ref.decode4(c, dtype)
    for pt in (0, 64, 640):
        assert_decode_close(_decode(c, dtype, partition_tokens=pt), exact, dtype, f"partition {pt}")


def test_decode_one_item_in_hundreds_of_parts():
    rng = np.random.default_rng(30)
    # one item over all warps
    c = ref.quantised_case(rng, dtype=gen.BF16, hq=2, hkv=1, d=64, bs=256, ctx=[100003])
    exact = ref.decode4(c, gen.BF16)
    for pt in (64, 0):
        assert_decode_close(_decode(c, gen.BF16, partition_tokens=pt), exact, gen.BF16, f"partition {pt}")
    # a warp per part: one long item among items of one token
    c = ref.quantised_case(rng, dtype=gen.F16, hq=4, hkv=1, d=64, bs=16, ctx=[1] * 300 + [30001] + [1] * 200)
    assert_decode_close(_decode(c, gen.F16), ref.decode4(c, gen.F16), gen.F16, "warps")


@pytest.mark.parametrize("group,dtype", [(4, gen.BF16), (8, gen.F16), (16, gen.BF16)])
def test_decode_few_ragged_items(group, dtype):
    """Few items, long and short: some cut into many parts, some whole within a warp's span."""
    rng = np.random.default_rng(40 + group)
    c = ref.quantised_case(rng, dtype=dtype, hq=4 * group, hkv=4, d=128, bs=16,
                           ctx=[64, 5, 0, 2000, 63, 65, 192, 256, 257, 320, 9, 8000, 1, 1, 1, 700])
    exact = ref.decode4(c, dtype)
    for pt in (0, 320, 2048):
        assert_decode_close(_decode(c, dtype, partition_tokens=pt), exact, dtype, f"partition {pt}")


def test_decode_uniform_tiny_probabilities():
    """One key far above the others: what is left of 131072 equal, tiny probabilities must not round away."""
    n, d, bs = 131072, 64, 256
    rng = np.random.default_rng(50)
    for dtype in (gen.BF16, gen.F16):
        one = np.ones(1, F32)
        c = ref.quantised_case(rng, dtype=dtype, hq=1, hkv=1, d=d, bs=bs, ctx=[n])
        # K: rows of +1 (row 0) and of -1; V: 0 in row 0, 6 elsewhere; block scales 1
        code_k, code_v = np.full((n, d), 10, np.uint8), np.full((n, d), 7, np.uint8)
        code_k[0], code_v[0] = 2, 0
        t = np.arange(n)
        blk, off = c["block_tables"][0][t // bs], t % bs
        for name, code in (("k", code_k), ("v", code_v)):
            pool = ref.empty_pool4(c["num_blocks"], bs, 1, d, 0x38)  # E4M3 1.0
            codes = np.zeros((c["num_blocks"], bs, d // 2), np.uint8)
            codes[blk, off] = code[:, 0::2] | (code[:, 1::2] << 4)
            pool[:, 0, :bs * d // 2] = codes.reshape(c["num_blocks"], -1)
            c[name + "_pool"], c[name + "_scale"] = pool, one
        c["q"] = gen.to_bits(np.ones((1, 1, d), F32), dtype)
        # logits 64 s and -64 s: the others' probabilities are e^(-128 s), 2^-24 times 1.4 of the first one's
        s = -np.log(1.4 * 2.0 ** -24) / 128
        c["scale"] = float(F32(s))
        exact = ref.decode4(c, dtype)
        got = gen.bits_to_f32(_decode(c, dtype), dtype)
        # the output's rounding, and 2^-10 for the probabilities' and the logits' (2^-16 absolute)
        half = {gen.F16: 2.0 ** -11, gen.BF16: 2.0 ** -8}[dtype]
        assert (np.abs(got - exact) <= np.abs(exact) * (half + 2.0 ** -10)).all(), (got.max(), exact.max())


def test_decode_bound_above_the_contexts():
    """max_context_len is only a bound: a larger one gives the same attention."""
    rng = np.random.default_rng(3)
    c = ref.quantised_case(rng, dtype=gen.BF16, hq=8, hkv=2, d=128, bs=16, ctx=[100, 260, 1])
    c["block_tables"] = np.pad(c["block_tables"], ((0, 0), (0, 400)), constant_values=-7)
    assert_decode_close(_decode(c, gen.BF16, maxlen=5000), ref.decode4(c, gen.BF16), gen.BF16, "bound")


@pytest.mark.parametrize("dtype", [gen.F16, gen.BF16], ids=["f16", "bf16"])
def test_decode_power_of_two_scaling(dtype):
    """2^k in q against 2^-k in the scale changes nothing but exponents."""
    rng = np.random.default_rng(4)
    c = ref.quantised_case(rng, dtype=dtype, hq=4, hkv=2, d=128, bs=16, ctx=[200, 33])
    want = _decode(c, dtype)
    q = gen.bits_to_f32(c["q"], dtype)
    for k in ((6, -4) if dtype == gen.F16 else (60, 14, -40)):
        c2 = dict(c, q=gen.to_bits(q * F32(2.0 ** k), dtype))
        got = _decode(c2, dtype, scale=c["scale"] * 2.0 ** -k)
        if dtype == gen.BF16 or k > 0:
            assert np.array_equal(got, want)
        else:  # fp16's small elements become subnormal: their own error counts
            assert_decode_close(got, ref.decode4(dict(c2, scale=c["scale"] * 2.0 ** -k), dtype), dtype)


def test_decode_rows_of_mixed_magnitude():
    """Heads whose queries differ by 2^100 share a tile; none disturbs another."""
    rng = np.random.default_rng(5)
    c = ref.quantised_case(rng, dtype=gen.BF16, hq=8, hkv=1, d=128, bs=16, ctx=[90, 300])
    q = gen.bits_to_f32(c["q"], gen.BF16).copy()
    q *= (2.0 ** np.array([-100, 0, -3, -60, 1, -20, 2, 0.0], F32))[None, :, None]
    q[1, 4] = 0.0
    c["q"] = gen.to_bits(q.astype(F32), gen.BF16)
    assert_decode_close(_decode(c, gen.BF16), ref.decode4(c, gen.BF16), gen.BF16)


def test_decode_sharp_and_growing_logits():
    """The running maximum moves at every token: keys grow along the context, then fall."""
    rng = np.random.default_rng(6)
    for dtype in (gen.F16, gen.BF16):
        c = ref.quantised_case(rng, dtype=dtype, hq=8, hkv=2, d=128, bs=16, ctx=[700, 400])
        bs, d = 16, 128
        for i, n in enumerate((700, 400)):
            t = np.arange(n)
            slots = c["block_tables"][i][t // bs].astype(np.int64) * bs + t % bs
            up = np.linspace(0, 1, n) if i == 0 else np.linspace(1, 0, n)
            q = gen.bits_to_f32(c["q"], dtype)[i].reshape(2, 4, d).mean(1)
            x = (q[None] * up[:, None, None] * 6 + rng.standard_normal((n, 2, d)) * 0.05).astype(F32)
            ref.store4(c["k_pool"], bs, d, slots, x, c["k_scale"])
        for pt in (0, 16, 2048):
            assert_decode_close(_decode(c, dtype, partition_tokens=pt), ref.decode4(c, dtype), dtype, f"pt {pt}")


@pytest.mark.parametrize("dtype", [gen.F16, gen.BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("group,ctx", [(4, 300), (8, 70), (16, 2000)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_decode_logits_beyond_the_resolution_of_fp32(dtype, group, ctx, sign):
    """Logits of 2^20 to 2^123, where one step of fp32 is more than any exponent that the kernel may form.

    The keys have two values, one half of the other, and the queries are 1 or -1: every product and sum is exact, the
    largest logits are equal and the others away by 2^19 at least, so the output is the mean of V over the former.
    """
    rng = np.random.default_rng(12)
    bs, d, hkv = 16, 128, 1
    c = ref.quantised_case(rng, dtype=dtype, hq=group * hkv, hkv=hkv, d=d, bs=bs, ctx=[ctx])
    t = np.arange(ctx)
    slots = c["block_tables"][0][t // bs].astype(np.int64) * bs + t % bs
    x = np.where(t % 3 == 0, 6.0, 3.0).astype(F32)[:, None, None] * np.ones((1, hkv, d), F32)
    c["k_scale"] = np.ones_like(c["k_scale"])
    ref.store4(c["k_pool"], bs, d, slots, x, c["k_scale"])
    c["q"] = gen.to_bits(np.full(c["q"].shape, sign, F32), dtype)
    c["scale"] = 1.0
    want = ref.decode4(c, dtype)
    for e in range(12, 115):  # a key's dot product is 768 or 384
        scale = float(F32(2.0 ** e * (1 + (e * 37 % 64) / 64 + 1 / 128 + 1 / 65536)))
        assert_decode_close(_decode(c, dtype, scale=scale), want, dtype, f"2^{e}")


@pytest.mark.parametrize("sign", [0.0, -1.0])
def test_decode_zero_and_negative_scale(sign):
    rng = np.random.default_rng(7)
    c = ref.quantised_case(rng, dtype=gen.F16, hq=4, hkv=2, d=64, bs=16, ctx=[50, 1])
    c["scale"] = sign * c["scale"]
    assert_decode_close(_decode(c, gen.F16), ref.decode4(c, gen.F16), gen.F16)


def test_decode_nan_in_a_read_row_stays_in_its_head():
    rng = np.random.default_rng(8)
    c = ref.quantised_case(rng, dtype=gen.BF16, hq=4, hkv=2, d=128, bs=16, ctx=[40, 40])
    exact = ref.decode4(c, gen.BF16)
    n = 16 * 64
    blk = c["block_tables"][0, 1]
    c["k_pool"][blk, 1, n + 3 * 8 + 2] = 0x7F  # token 19 of sequence 0, kv head 1
    got = gen.bits_to_f32(_decode(c, gen.BF16), gen.BF16)
    assert np.isnan(got[0, 2:]).all()
    keep = np.ones((2, 4), bool)
    keep[0, 2:] = False
    assert np.isfinite(got[keep]).all() and np.abs(got[keep] - exact[keep]).max() < 2e-2


def test_decode_reports_bad_blocks_and_lengths():
    """An entry outside the pool reads as zero rows; lengths are clamped to the bound."""
    rng = np.random.default_rng(10)
    for bs in (8, 16, 64):
        c = ref.quantised_case(rng, dtype=gen.F16, hq=4, hkv=2, d=128, bs=bs, ctx=[3 * bs, 2 * bs + 3, 40])
        bad = dict(c, block_tables=c["block_tables"].copy())
        bad["block_tables"][0, 1] = c["num_blocks"]
        bad["block_tables"][1, 0] = -1
        got = _decode(bad, gen.F16, ok=False)
        status, bits = pa.pa_last_device_error()
        assert status == pa.PA_ERR_DEVICE_CHECK and bits == pa.PA_DEVERR_BLOCK_ID
        # the same with those blocks' stored values zero
        zero = dict(c, k_pool=np.concatenate([c["k_pool"], np.zeros_like(c["k_pool"][:1])]),
                    v_pool=np.concatenate([c["v_pool"], np.zeros_like(c["v_pool"][:1])]),
                    block_tables=bad["block_tables"].copy())
        zero["block_tables"][1, 0] = c["num_blocks"]
        assert_decode_close(got, ref.decode4(zero, gen.F16), gen.F16, f"bs {bs}")
    c = ref.quantised_case(rng, dtype=gen.F16, hq=4, hkv=2, d=64, bs=16, ctx=[64, 32, 48])
    want = ref.decode4(dict(c, context_lens=np.array([32, 32, 0])), gen.F16)
    c["context_lens"] = np.array([64, 32, -5], np.int32)
    got = _decode(c, gen.F16, maxlen=32, ok=False)
    status, bits = pa.pa_last_device_error()
    assert status == pa.PA_ERR_DEVICE_CHECK and bits == pa.PA_DEVERR_CONTEXT_LEN
    assert_decode_close(got, want, gen.F16)


def test_decode_shared_blocks_and_repeated_entries():
    rng = np.random.default_rng(11)
    c = ref.quantised_case(rng, dtype=gen.BF16, hq=8, hkv=2, d=128, bs=16, ctx=[300, 310, 305, 40],
                           shared_prefix_blocks=12)
    c["block_tables"][3, :3] = c["block_tables"][3, 0]  # the same block three times
    assert_decode_close(_decode(c, gen.BF16), ref.decode4(c, gen.BF16), gen.BF16)


def test_decode_is_deterministic():
    rng = np.random.default_rng(12)
    c = ref.quantised_case(rng, dtype=gen.BF16, hq=32, hkv=8, d=128, bs=16, ctx=[1000, 3000, 17])
    first = _decode(c, gen.BF16)
    for _ in range(3):
        assert np.array_equal(_decode(c, gen.BF16), first)


def _device_args(c, dtype):
    return (dev(c["q"], dtype), _gpu(c["k_pool"]), _gpu(c["v_pool"]), _gpu(c["k_scale"]), _gpu(c["v_scale"]),
            dev_i32(c["block_tables"]), dev_i32(c["context_lens"]), c["scale"])


def test_decode_graphs_sharing_a_workspace():
    """Two captured decodes of different shapes use one workspace, replayed in turn; buffers change between."""
    rng = np.random.default_rng(13)
    cases = [ref.quantised_case(rng, dtype=gen.BF16, hq=16, hkv=2, d=128, bs=16, ctx=[900, 5, 0, 2000]),
             ref.quantised_case(rng, dtype=gen.BF16, hq=4, hkv=4, d=64, bs=8, ctx=[333, 1500])]
    shapes = [_shape(c, gen.BF16) for c in cases]
    lens = [int(c["context_lens"].max()) for c in cases]
    nbytes = max(pa.pa_decode_workspace_bytes(s, n) for s, n in zip(shapes, lens))
    ws = torch.randint(0, 256, (nbytes,), dtype=torch.uint8, device="cuda")
    outs, args, graphs = [], [], []
    for c, s, n in zip(cases, shapes, lens):
        args.append(_device_args(c, gen.BF16))
        outs.append(torch.empty(c["q"].shape, dtype=torch.bfloat16, device="cuda"))
        pa.pa_decode_fp4(*args[-1], outs[-1], s, n, ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pa.pa_decode_fp4(*args[-1], outs[-1], s, n, ws)
        graphs.append(g)
    for step in range(3):
        for c, a, out, g in zip(cases, args, outs, graphs):
            out.fill_(float("nan"))
            if step:
                c["context_lens"] = np.maximum(c["context_lens"] - 7 * step, 0)
                a[6].copy_(dev_i32(c["context_lens"]))
            g.replay()
            assert pa.pa_last_device_error()[0] == pa.PA_OK
            assert_decode_close(host_bits(out), ref.decode4(c, gen.BF16), gen.BF16, f"step {step}")
    del graphs


def test_decode_two_streams_at_once():
    rng = np.random.default_rng(14)
    cases = [ref.quantised_case(rng, dtype=gen.F16, hq=8, hkv=2, d=128, bs=16, ctx=[900, 700]) for _ in range(2)]
    state = []
    for c in cases:
        shape = _shape(c, gen.F16)
        ws = torch.empty(pa.pa_decode_workspace_bytes(shape, 900), dtype=torch.uint8, device="cuda")
        state.append((shape, ws, _device_args(c, gen.F16), torch.empty(c["q"].shape, dtype=torch.float16, device="cuda"),
                      torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for shape, ws, args, out, stream in state:
            pa.pa_decode_fp4(*args, out, shape, 900, ws, stream=stream)
    torch.cuda.synchronize()
    assert pa.pa_last_device_error()[0] == pa.PA_OK
    for c, (_, _, _, out, _) in zip(cases, state):
        assert_decode_close(host_bits(out), ref.decode4(c, gen.F16), gen.F16)


# ---------------------------------------------------------------------------
# together, as a server uses them


def test_serving_steps_over_an_fp4_cache():
    """Prompts and next tokens through the rotating append, a beam fork with copy-on-write, a swap out and in, decode
    and gather, against one host model of the whole."""
    rng = np.random.default_rng(15)
    dtype, hq, hkv, d, bs, nb, maxpos = gen.BF16, 8, 2, 128, 16, 64, 512
    ks, vs = (rng.uniform(0.08, 0.18, hkv).astype(F32) for _ in range(2))
    th = np.arange(maxpos)[:, None] * 10000.0 ** (-np.arange(0, d, 2) / d)
    cs = np.concatenate([np.cos(th), np.sin(th)], axis=1).astype(F32)
    kp, vp = ref.empty_pool4(nb, bs, hkv, d, 0x7F), ref.empty_pool4(nb, bs, hkv, d, 0x7F)
    kc, vc = _gpu(kp), _gpu(vp)
    dks, dvs, dcs = _gpu(ks), _gpu(vs), _gpu(cs)
    alloc = pa.Allocator(nb, bs, rng.permutation(nb))
    rope = pa.make_rope(rotary_dim=d, max_position=maxpos)

    def shape(s):
        return pa.make_shape(num_seqs=s, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=bs, num_blocks=nb,
                             max_blocks_per_seq=16, dtype=dtype, cache_format=pa.PA_CACHE_FP4_E2M1)

    def append(pos, slots):
        t = len(pos)
        q, k, v = (gen.normal_bits(rng, (t, h, d), dtype) for h in (hq, hkv, hkv))
        qo = torch.empty((t, hq, d), dtype=torch.bfloat16, device="cuda")
        pa.pa_rope_append(dev(q, dtype), dev(k, dtype), dev(v, dtype), dev_i32(pos), dcs, rope, dev_i32(slots), t, qo, kc,
                          vc, dks, dvs, shape(1))
        c, s = cs[pos][:, :d // 2], cs[pos][:, d // 2:]
        rot = [gen.to_bits(ref.rotate(gen.bits_to_f32(x, dtype), c, s, d, False, F32), dtype) for x in (q, k)]
        ref.store4(kp, bs, d, slots, gen.bits_to_f32(rot[1], dtype), ks)
        ref.store4(vp, bs, d, slots, gen.bits_to_f32(v, dtype), vs)
        assert np.array_equal(host_bits(qo), rot[0])
        return qo, rot[0]

    lens = {0: 37, 1: 100, 2: 16}
    for s, n in lens.items():
        alloc.add_seq(s, n)
        bt, _ = alloc.block_tables([s], 16)
        t = np.arange(n)
        append(t.astype(np.int32), (bt[0][t // bs] * bs + t % bs).astype(np.int32))
    alloc.fork(1, 3)
    lens[3] = lens[1]
    seqs = [0, 1, 2, 3]
    for step in range(4):
        slots, pairs = alloc.append_slots(seqs)
        if len(pairs):
            pa.pa_copy_blocks(dev_i32(pairs), len(pairs), kc, vc, shape(4))
            for src, dst in pairs:
                kp[dst], vp[dst] = kp[src], vp[src]
        qo, qbits = append(np.array([lens[s] for s in seqs], np.int32), slots)
        for s in seqs:
            lens[s] += 1
        bt, cl = alloc.block_tables(seqs, 16)
        if step == 1:  # sequence 0 goes to host memory and comes back
            held = bt[0][:-(-lens[0] // bs)]
            host = [torch.zeros((8, *kp.shape[1:]), dtype=torch.uint8).pin_memory() for _ in range(2)]
            out = np.stack([held, np.arange(len(held))], axis=1)
            pa.pa_swap_blocks(dev_i32(out), len(held), kc, vc, nb, *host, 8, shape(4))
            torch.cuda.synchronize()
            kc[_gpu(held.astype(np.int64))] = 0
            vc[_gpu(held.astype(np.int64))] = 0
            pa.pa_swap_blocks(dev_i32(out[:, ::-1].copy()), len(held), *host, 8, kc, vc, nb, shape(4))
        sh = shape(4)
        n = int(cl.max())
        ws = torch.empty(pa.pa_decode_workspace_bytes(sh, n), dtype=torch.uint8, device="cuda")
        got = torch.empty((4, hq, d), dtype=torch.bfloat16, device="cuda")
        pa.pa_decode_fp4(qo, kc, vc, dks, dvs, dev_i32(bt), dev_i32(cl), d ** -0.5, got, sh, n, ws)
        assert pa.pa_last_device_error()[0] == pa.PA_OK
        want = ref.decode4(dict(q=qbits, block_size=bs, context_lens=cl, block_tables=bt, k_pool=kp, v_pool=vp,
                                k_scale=ks, v_scale=vs, scale=d ** -0.5), dtype)
        assert_decode_close(host_bits(got), want, dtype, f"step {step}")
    assert np.array_equal(kc.cpu().numpy(), kp) and np.array_equal(vc.cpu().numpy(), vp)
    t = np.arange(lens[1])
    slots = (bt[1][t // bs] * bs + t % bs).astype(np.int32)
    ko, vo = (torch.empty((len(t), hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pa.pa_cache_gather(dev_i32(slots), len(t), kc, vc, dks, dvs, ko, vo, shape(4))
    assert np.array_equal(host_bits(ko), gen.to_bits(ref.rows4(kp, bs, d, slots, ks, F32), dtype))
    assert np.array_equal(host_bits(vo), gen.to_bits(ref.rows4(vp, bs, d, slots, vs, F32), dtype))
