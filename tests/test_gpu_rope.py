"""The rotating append and the gather against plain references, through the C ABI (needs a B200).

Rotation is fp32 with one rounding per product and sum, then one to the
element type: computed the same way on the host it must match bit for bit, so
that the codes of the quantised formats match too.  Against fp64 the error is
half a step of the element type plus three fp32 roundings.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import fp4_ref as ref  # noqa: E402
from gpu_util import dev, dev_i32, host_bits  # noqa: E402
from paged_kv_cache_458_b200 import gen, pa  # noqa: E402

pytestmark = pytest.mark.gpu
FORMATS = {"16": pa.PA_CACHE_AS_DTYPE, "fp8": pa.PA_CACHE_FP8_E4M3, "fp4": pa.PA_CACHE_FP4_E2M1}
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


def _ok():
    status, bits = pa.pa_last_device_error()
    assert status == pa.PA_OK, f"device check fired: {bits:#x}"


class Case:
    """Rows, slots, positions and a poisoned pool pair; `expect` fills the host copies."""

    def __init__(self, orc, seed, fmt, dtype, t, hq, hkv, d, bs, rotary, interleaved, fused=False, pad=0,
                 max_position=97, positions=None):
        self.__dict__.update(locals())
        rng = np.random.default_rng(seed)
        self.nb = -(-t // bs) + 3
        self.q = gen.normal_bits(rng, (t, hq, d), dtype)
        self.k = gen.normal_bits(rng, (t, hkv, d), dtype)
        self.v = gen.normal_bits(rng, (t, hkv, d), dtype)
        self.slots = rng.choice(self.nb * bs, t, replace=False).astype(np.int32)
        if pad:
            self.slots[rng.choice(t, pad, replace=False)] = -1 - rng.integers(0, 5, pad)
        self.pos = rng.integers(0, max_position, t).astype(np.int32) if positions is None else positions
        th = np.arange(max_position)[:, None] * 10000.0 ** (-np.arange(0, rotary, 2) / rotary)
        self.cs = np.concatenate([np.cos(th), np.sin(th)], axis=1).astype(F32)
        self.ks = rng.uniform(0.08, 0.18, hkv).astype(F32)
        self.vs = rng.uniform(0.08, 0.18, hkv).astype(F32)
        if fmt == "fp4":
            self.k0 = rng.integers(0, 256, (self.nb, hkv, bs * d * 9 // 16), dtype=np.uint8)
        elif fmt == "fp8":
            self.k0 = rng.integers(0, 256, (self.nb, bs, hkv, d), dtype=np.uint8)
        else:
            self.k0 = rng.integers(0, 1 << 16, (self.nb, bs, hkv, d), dtype=np.uint16)
        self.v0 = self.k0[::-1].copy()
        self.qo0 = rng.integers(0, 1 << 16, self.q.shape, dtype=np.uint16)

    def shape(self):
        return pa.make_shape(num_seqs=1, num_q_heads=self.hq, num_kv_heads=self.hkv, head_dim=self.d,
                             block_size=self.bs, num_blocks=self.nb, max_blocks_per_seq=1, dtype=self.dtype,
                             cache_format=FORMATS[self.fmt])

    def pool(self, a):
        return dev(a, self.dtype) if self.fmt == "16" else _gpu(a)

    def host(self, t):
        return host_bits(t) if self.fmt == "16" else t.cpu().numpy()

    def rotated(self, bits, dtype=F32):
        x = gen.bits_to_f32(bits, self.dtype)
        h = self.rotary // 2
        cs = self.cs[np.clip(self.pos, 0, self.max_position - 1)]
        return ref.rotate(x, cs[:, :h], cs[:, h:], self.rotary, self.interleaved, dtype)

    def expect(self, slots=None):
        """(q_out bits, K pool, V pool)."""
        slots = self.slots if slots is None else slots
        kr, vr = gen.to_bits(self.rotated(self.k), self.dtype), self.v
        qo, kp, vp = self.qo0.copy(), self.k0.copy(), self.v0.copy()
        keep = slots >= 0
        qo[keep] = gen.to_bits(self.rotated(self.q), self.dtype)[keep]
        if self.fmt == "fp4":
            ref.store4(kp, self.bs, self.d, slots, gen.bits_to_f32(kr, self.dtype), self.ks)
            ref.store4(vp, self.bs, self.d, slots, gen.bits_to_f32(vr, self.dtype), self.vs)
        elif self.fmt == "fp8":
            self.orc.cache_append_fp8(self.dtype, kr, vr, slots, self.ks, self.vs, kp, vp)
        else:
            self.orc.cache_append(kr, vr, slots, kp, vp)
        return qo, kp, vp

    def run(self, slots=None, stream=None):
        n, d = self.t, self.d
        slots = self.slots if slots is None else slots
        if self.fused:
            pad = 8  # rows a little wider than their parts, as a padded projection has
            both = np.concatenate([self.q.reshape(n, -1), self.k.reshape(n, -1), self.v.reshape(n, -1),
                                   np.zeros((n, pad), np.uint16)], axis=1)
            x = dev(both, self.dtype)
            w = x.shape[1]
            q, k, v = x, x[:, self.hq * d:], x[:, (self.hq + self.hkv) * d:]
            rope = pa.make_rope(rotary_dim=self.rotary, interleaved=int(self.interleaved),
                                max_position=self.max_position, q_stride=w, k_stride=w, v_stride=w)
        else:
            q, k, v = (dev(a, self.dtype) for a in (self.q, self.k, self.v))
            rope = pa.make_rope(rotary_dim=self.rotary, interleaved=int(self.interleaved),
                                max_position=self.max_position)
        qo, kc, vc = dev(self.qo0, self.dtype), self.pool(self.k0), self.pool(self.v0)
        scales = (None, None) if self.fmt == "16" else (_gpu(self.ks), _gpu(self.vs))
        args = (q, k, v, _gpu(self.pos), _gpu(self.cs), rope, dev_i32(slots), n, qo, kc, vc, *scales, self.shape())
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        pa.pa_rope_append(*args, stream=stream)
        if stream is not None:
            stream.synchronize()
        return qo, kc, vc

    def check(self, slots=None, got=None, ok=True):
        qo, kc, vc = self.run(slots) if got is None else got
        if ok:
            _ok()
        eq, ek, ev = self.expect(slots)
        assert np.array_equal(host_bits(qo), eq)
        assert np.array_equal(self.host(vc), ev)
        assert np.array_equal(self.host(kc), ek)


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("dtype", [gen.F16, gen.BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d,rotary,interleaved,fused", [
    (4, 4, 64, 64, False, False), (8, 1, 128, 128, False, True), (6, 3, 128, 64, True, False),
    (5, 5, 64, 16, True, True), (16, 1, 64, 48, False, False), (14, 7, 128, 48, False, True),
    (64, 8, 128, 128, True, True), (40, 40, 128, 96, False, False), (1, 1, 64, 32, False, False),
    (1, 1, 128, 112, True, False)])
def test_rope_append_bit_exact(orc, fmt, dtype, hq, hkv, d, rotary, interleaved, fused):
    for t, bs, pad in ((1, 8, 0), (37, 16, 5), (70, 24, 0)):
        Case(orc, 11 * t + d, fmt, dtype, t, hq, hkv, d, bs, rotary, interleaved, fused, pad).check()


@pytest.mark.parametrize("dtype", [gen.F16, gen.BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_append_against_fp64(orc, dtype, interleaved):
    c = Case(orc, 5, "16", dtype, 64, 8, 2, 128, 16, 128, interleaved)
    qo, kc, _ = c.run()
    _ok()
    half = {gen.F16: 2.0 ** -11, gen.BF16: 2.0 ** -8}[dtype]
    slots = c.slots.astype(np.int64)
    for bits, got in ((c.q, host_bits(qo)), (c.k, host_bits(kc).reshape(-1, 2, 128)[slots])):
        exact = c.rotated(bits, np.float64)
        # |a c| + |b s| <= |a| + |b|: each product and the sum add at most 2^-24 of that
        room = np.abs(gen.bits_to_f32(bits, dtype)).astype(np.float64).max(-1, keepdims=True) * 2
        tiny = 2.0 ** -25  # half the spacing of fp16 subnormals
        err = np.abs(gen.bits_to_f32(got, dtype) - exact)
        assert (err <= half * np.abs(exact) * (1 + 2.0 ** -10) + 3 * 2.0 ** -24 * room + tiny).all()


def test_rope_append_many_tokens(orc):
    Case(orc, 8, "fp4", gen.BF16, 3001, 8, 2, 128, 16, 128, False, True, 100).check()


@pytest.mark.parametrize("fmt", list(FORMATS))
def test_rope_append_in_place(orc, fmt):
    c = Case(orc, 21, fmt, gen.BF16, 19, 8, 2, 128, 16, 64, False, False, 3)
    c.qo0 = c.q.copy()  # rows of padding tokens stay as they were
    q = dev(c.q, c.dtype)
    kc, vc = c.pool(c.k0), c.pool(c.v0)
    scales = (None, None) if fmt == "16" else (_gpu(c.ks), _gpu(c.vs))
    pa.pa_rope_append(q, dev(c.k, c.dtype), dev(c.v, c.dtype), _gpu(c.pos), _gpu(c.cs),
                      pa.make_rope(rotary_dim=64, max_position=c.max_position), dev_i32(c.slots), c.t, q, kc, vc,
                      *scales, c.shape())
    c.check(got=(q, kc, vc))


def test_rope_append_q_out_stride(orc):
    c = Case(orc, 22, "16", gen.F16, 9, 4, 2, 64, 16, 64, False)
    wide = dev(np.full((9, 4 * 64 + 24), 0x3333, np.uint16), c.dtype)
    kc, vc = c.pool(c.k0), c.pool(c.v0)
    pa.pa_rope_append(dev(c.q, 0), dev(c.k, 0), dev(c.v, 0), _gpu(c.pos), _gpu(c.cs),
                      pa.make_rope(rotary_dim=64, max_position=c.max_position, q_out_stride=4 * 64 + 24),
                      dev_i32(c.slots), 9, wide, kc, vc, None, None, c.shape())
    _ok()
    got = host_bits(wide)
    assert (got[:, 256:] == 0x3333).all()
    assert np.array_equal(got[:, :256].reshape(9, 4, 64), c.expect()[0])


@pytest.mark.parametrize("fmt", list(FORMATS))
def test_rope_append_reports_bad_slots_and_positions(orc, fmt):
    c = Case(orc, 31, fmt, gen.F16, 12, 4, 2, 64, 8, 32, False)
    slots = c.slots.copy()
    slots[3], slots[4] = c.nb * c.bs, 2 ** 31 - 1
    c.pos = c.pos.copy()
    c.pos[5], c.pos[6], c.pos[7] = -1, c.max_position, 2 ** 31 - 1
    got = c.run(slots)
    status, bits = pa.pa_last_device_error()
    assert status == pa.PA_ERR_DEVICE_CHECK and bits == pa.PA_DEVERR_SLOT | pa.PA_DEVERR_POSITION
    skipped = slots.copy()
    skipped[3:8] = -1
    c.check(skipped, got)


def test_rope_append_far_positions(orc):
    pos = np.array([0, 1, 65535, 131071, 131070], np.int32)
    Case(orc, 41, "fp8", gen.BF16, 5, 8, 8, 128, 16, 128, False, max_position=131072, positions=pos).check()


def test_rope_append_special_values(orc):
    for fmt in FORMATS:
        c = Case(orc, 51, fmt, gen.F16, 6, 4, 2, 64, 16, 32, False)
        f = gen.bits_to_f32(c.k, gen.F16).copy()
        f[0] = 0.0
        f[1, :, ::3] = 6.0e-8  # subnormal
        f[2, :, 5] = 60000.0
        c.k = gen.to_bits(f, gen.F16)
        c.v = c.k[::-1].copy()
        c.check()


@pytest.mark.parametrize("fmt", ["fp4", "16"])
def test_rope_append_on_another_stream_and_captured(orc, fmt):
    c = Case(orc, 61, fmt, gen.BF16, 33, 8, 2, 128, 16, 128, False, True)
    c.check(got=c.run(stream=torch.cuda.Stream()))
    q, k, v = (dev(a, c.dtype) for a in (c.q, c.k, c.v))
    qo, kc, vc = dev(c.qo0, c.dtype), c.pool(c.k0), c.pool(c.v0)
    pos, cs, slots = _gpu(c.pos), _gpu(c.cs), dev_i32(c.slots)
    scales = (None, None) if fmt == "16" else (_gpu(c.ks), _gpu(c.vs))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.pa_rope_append(q, k, v, pos, cs, pa.make_rope(rotary_dim=128, max_position=c.max_position), slots, c.t, qo,
                          kc, vc, *scales, c.shape())
    for seed in (62, 63):  # new rows, positions and slots in the same buffers
        n = Case(orc, seed, fmt, gen.BF16, 33, 8, 2, 128, 16, 128, False, False, 4)
        n.ks, n.vs = c.ks, c.vs
        for buf, a in ((q, n.q), (k, n.k), (v, n.v), (qo, n.qo0)):
            buf.copy_(dev(a, c.dtype).view_as(buf))
        kc.copy_(n.pool(n.k0)), vc.copy_(n.pool(n.v0))
        pos.copy_(_gpu(n.pos)), slots.copy_(dev_i32(n.slots))
        g.replay()
        n.check(got=(qo, kc, vc))
    del g


# ---------------------------------------------------------------------------
# gather


def _gather_case(seed, fmt, dtype, nb, bs, hkv, d):
    rng = np.random.default_rng(seed)
    ks, vs = (rng.uniform(0.05, 2.0, hkv).astype(F32) for _ in range(2))
    if fmt == "16":
        pools = [gen.normal_bits(rng, (nb, bs, hkv, d), dtype) for _ in range(2)]
    elif fmt == "fp8":
        pools = [rng.integers(0, 256, (nb, bs, hkv, d), dtype=np.uint8) for _ in range(2)]
    else:
        pools = [rng.integers(0, 256, (nb, hkv, bs * d * 9 // 16), dtype=np.uint8) for _ in range(2)]
    return rng, ks, vs, pools


def _rows(fmt, pool, bs, d, slots, scale, dtype):
    if fmt == "16":
        return pool.reshape(-1, *pool.shape[2:])[slots]
    if fmt == "fp8":
        v = ref.E4M3[pool.reshape(-1, *pool.shape[2:])[slots]].astype(F32) * scale[:, None]
    else:
        v = ref.rows4(pool, bs, d, slots, scale, F32)
    return gen.to_bits(v.astype(F32), dtype)


def _same(got, want, dtype):
    """Equal bits, any NaN for a NaN."""
    nan = np.isnan(gen.bits_to_f32(want, dtype))
    assert np.array_equal(np.isnan(gen.bits_to_f32(got, dtype)), nan)
    assert np.array_equal(got[~nan], want[~nan])


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("dtype", [gen.F16, gen.BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("hkv,d,bs,t", [(1, 64, 8, 1), (3, 128, 24, 50), (8, 128, 16, 333), (40, 64, 256, 600),
                                        (5, 64, 32, 77)])
def test_gather_bit_exact(fmt, dtype, hkv, d, bs, t):
    nb = -(-t // bs) + 1
    rng, ks, vs, (kp, vp) = _gather_case(t + d, fmt, dtype, nb, bs, hkv, d)
    slots = rng.integers(0, nb * bs, t).astype(np.int32)  # repeats allowed
    slots[t // 2:t // 2 + t // 5] = -3
    shape = pa.make_shape(num_seqs=1, num_q_heads=hkv, num_kv_heads=hkv, head_dim=d, block_size=bs, num_blocks=nb,
                          max_blocks_per_seq=1, dtype=dtype, cache_format=FORMATS[fmt])
    ko0 = rng.integers(0, 1 << 14, (t, hkv, d)).astype(np.uint16)
    ko, vo = dev(ko0, dtype), dev(ko0, dtype)
    pools = [dev(p, dtype) if fmt == "16" else _gpu(p) for p in (kp, vp)]
    scales = (None, None) if fmt == "16" else (_gpu(ks), _gpu(vs))
    pa.pa_cache_gather(dev_i32(slots), t, *pools, *scales, ko, vo, shape)
    _ok()
    keep = slots >= 0
    for got, pool, scale in ((ko, kp, ks), (vo, vp, vs)):
        got = host_bits(got)
        assert np.array_equal(got[~keep], ko0[~keep])
        _same(got[keep], _rows(fmt, pool, bs, d, slots[keep], scale, dtype), dtype)


@pytest.mark.parametrize("fmt", list(FORMATS))
def test_gather_reports_bad_slots_as_zero_rows(fmt):
    nb, bs, hkv, d = 3, 8, 2, 64
    _, ks, vs, (kp, vp) = _gather_case(3, fmt, gen.F16, nb, bs, hkv, d)
    slots = np.array([0, nb * bs, 2 ** 31 - 1, 5], np.int32)
    shape = pa.make_shape(num_seqs=1, num_q_heads=hkv, num_kv_heads=hkv, head_dim=d, block_size=bs, num_blocks=nb,
                          max_blocks_per_seq=1, dtype=gen.F16, cache_format=FORMATS[fmt])
    ko, vo = (dev(np.full((4, hkv, d), 0x3C00, np.uint16), gen.F16) for _ in range(2))
    pools = [dev(p, gen.F16) if fmt == "16" else _gpu(p) for p in (kp, vp)]
    pa.pa_cache_gather(dev_i32(slots), 4, *pools, _gpu(ks), _gpu(vs), ko, vo, shape)
    status, bits = pa.pa_last_device_error()
    assert status == pa.PA_ERR_DEVICE_CHECK and bits == pa.PA_DEVERR_SLOT
    for got, pool, scale in ((ko, kp, ks), (vo, vp, vs)):
        got = host_bits(got)
        assert not got[1:3].any()
        _same(got[[0, 3]], _rows(fmt, pool, bs, d, slots[[0, 3]], scale, gen.F16), gen.F16)
