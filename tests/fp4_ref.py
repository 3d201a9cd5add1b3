"""Plain references for the E2M1 cache, the rotating append and the gather (numpy).

What the library stores is defined by single roundings in fp32, so the stored codes
are computed here with numpy's fp32 operations and must match byte for byte;
attention and rotation are computed in fp64.
"""
import numpy as np

from paged_kv_cache_458_b200 import gen

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
F32 = np.float32


def _e4m3_table():
    v = np.empty(256)
    for c in range(256):
        e, m, sign = (c >> 3) & 15, c & 7, -1.0 if c & 128 else 1.0
        v[c] = sign * (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    v[0x7F] = v[0xFF] = np.nan
    return v


E4M3 = _e4m3_table()


def _nearest(x, grid):
    """Index into the ascending grid of the value nearest to x >= 0 (ties to the even index, saturating)."""
    x = np.asarray(x, dtype=np.float64)
    hi = np.minimum(np.searchsorted(grid, x), len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    with np.errstate(invalid="ignore"):
        dl, dh = x - grid[lo], grid[hi] - x
    take_lo = (dl < dh) | ((dl == dh) & (lo % 2 == 0))
    return np.where(take_lo, lo, hi).astype(np.uint8)


def quantise4(x, scale):
    """x fp32 [..., Hkv, D], scale fp32 [Hkv]: codes 0..15 [..., D], E4M3 block scale codes [..., D / 16]."""
    x = np.asarray(x, dtype=F32)
    b = x.reshape(*x.shape[:-1], -1, 16)
    h = np.asarray(scale, dtype=F32).reshape(-1, 1)
    nan = np.isnan(b).any(-1)
    with np.errstate(all="ignore"):
        amax = np.nanmax(np.abs(np.where(np.isnan(b), F32(0), b)), axis=-1)
        s = _nearest(np.minimum((amax / F32(6) / h).astype(F32), F32(448)), E4M3[:0x7F])
        f = E4M3[s].astype(F32)
        r = np.where(f > 0, F32(1) / (f * h), F32(0)).astype(F32)
        y = (b * r[..., None]).astype(F32)
        code = _nearest(np.minimum(np.nan_to_num(np.abs(y), nan=6.0, posinf=6.0), 6.0), E2M1)
    code = code | (np.signbit(b).astype(np.uint8) << 3)
    return code.reshape(x.shape), np.where(nan, 0x7F, s).astype(np.uint8)


def values4(code, s, scale, dtype=np.float64):
    """The stored values; dtype float32 rounds the product with the head scale once (the rest is exact)."""
    v = np.where(code & 8, -1.0, 1.0) * E2M1[code & 7] * np.repeat(E4M3[s], 16, axis=-1)
    return v.astype(dtype) * np.asarray(scale, dtype=F32).reshape(-1, 1).astype(dtype)


def empty_pool4(nb, bs, hkv, d, fill=0):
    return np.full((nb, hkv, bs * d * 9 // 16), fill, dtype=np.uint8)


def pool4_views(pool, bs, d):
    """(codes [NB, Hkv, bs, D / 2], scales [NB, Hkv, bs, D / 16]) of a pool."""
    nb, hkv, _ = pool.shape
    n = bs * d // 2
    return pool[..., :n].reshape(nb, hkv, bs, d // 2), pool[..., n:].reshape(nb, hkv, bs, d // 16)


def store4(pool, bs, d, slots, x, scale):
    """Rows x fp32 [T, Hkv, D] into their slots (negative: skipped)."""
    code, s = quantise4(x, scale)
    codes, n = pool.reshape(pool.shape[0], pool.shape[1], -1), bs * d // 2
    for t, slot in enumerate(np.asarray(slots).tolist()):
        if slot < 0:
            continue
        blk, off = divmod(slot, bs)
        packed = code[t, :, 0::2] | (code[t, :, 1::2] << 4)
        codes[blk, :, off * d // 2:(off + 1) * d // 2] = packed
        codes[blk, :, n + off * d // 16:n + (off + 1) * d // 16] = s[t]


def rows4(pool, bs, d, slots, scale, dtype=np.float64):
    """Stored values [T, Hkv, D] of slots >= 0."""
    c, s = pool4_views(pool, bs, d)
    slots = np.asarray(slots, dtype=np.int64)
    c, s = c[slots // bs, :, slots % bs], s[slots // bs, :, slots % bs]
    code = np.stack([c & 15, c >> 4], axis=-1).reshape(*c.shape[:-1], d)
    return values4(code, s, scale, dtype)


def attention(q, rows_k, rows_v, scale):
    """One sequence: q [Hq, D], rows [ctx, Hkv, D] fp64 -> [Hq, D]; an empty context gives zeros."""
    hq, d = q.shape
    ctx, hkv, _ = rows_k.shape
    if ctx == 0:
        return np.zeros((hq, d))
    g = hq // hkv
    out = np.empty((hq, d))
    for h in range(hq):
        x = rows_k[:, h // g] @ q[h] * scale
        p = np.exp(x - x.max())
        out[h] = p @ rows_v[:, h // g] / p.sum()
    return out


def decode4(c, dtype):
    """fp64 attention of a case made by quantised_case."""
    q = gen.bits_to_f32(c["q"], dtype).astype(np.float64)
    bs, d = c["block_size"], q.shape[-1]
    out = np.zeros(q.shape)
    for i, n in enumerate(np.asarray(c["context_lens"]).tolist()):
        t = np.arange(n)
        slots = c["block_tables"][i][t // bs].astype(np.int64) * bs + t % bs if n else t
        out[i] = attention(q[i], rows4(c["k_pool"], bs, d, slots, c["k_scale"]),
                           rows4(c["v_pool"], bs, d, slots, c["v_scale"]), c["scale"])
    return out


def quantised_case(rng, *, dtype, hq, hkv, d, bs, ctx, **kw):
    """A paged case with both pools quantised from N(0, 1) rows.

    What no sequence may read is poisoned: slots beyond the contexts hold NaN
    block scales, table entries beyond them name no block.
    """
    c = gen.random_decode_case(rng, num_seqs=len(ctx), num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                               block_size=bs, dtype=dtype, context_lens=ctx, poison=False, **kw)
    nb = c["num_blocks"]
    valid = gen.valid_slot_mask(c["block_tables"], c["context_lens"], nb, bs).reshape(nb, bs)
    out = dict(c, block_size=bs)
    for name in ("k", "v"):
        scale = rng.uniform(0.08, 0.18, hkv).astype(F32)
        x = gen.bits_to_f32(c[name + "_cache"], dtype)
        code, s = quantise4(x, scale)
        s = np.where(valid[:, :, None, None], s, 0x7F).astype(np.uint8)
        pool = empty_pool4(nb, bs, hkv, d)
        codes, scales = pool4_views(pool, bs, d)
        n = bs * d // 2
        pool[..., :n] = (code[..., 0::2] | (code[..., 1::2] << 4)).transpose(0, 2, 1, 3).reshape(nb, hkv, n)
        pool[..., n:] = s.transpose(0, 2, 1, 3).reshape(nb, hkv, -1)
        out[name + "_pool"], out[name + "_scale"] = pool, scale
    bt = out["block_tables"].copy()
    for i, n in enumerate(np.asarray(ctx).tolist()):
        bt[i, -(-n // bs):] = 1 << 30
    out["block_tables"] = bt
    return out


def rotate(x, cos, sin, rotary, interleaved, dtype):
    """x [T, H, D]; cos, sin [T, rotary / 2]; every product and sum rounded to `dtype`."""
    x = x.astype(dtype)
    c, s = cos.astype(dtype)[:, None, :], sin.astype(dtype)[:, None, :]
    y = x.copy()
    i = np.arange(0, rotary, 2) if interleaved else np.arange(rotary // 2)
    j = i + (1 if interleaved else rotary // 2)
    a, b = x[..., i], x[..., j]
    y[..., i] = a * c - b * s
    y[..., j] = b * c + a * s
    return y
