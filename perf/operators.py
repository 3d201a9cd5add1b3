"""Measured cases of the cache operators: the rotating append, the 4-bit cache and the gather.

Four kinds of pass, named by ``case["kind"]``:

* ``rope``: q and k rotated at their positions, q written out, k and v
  appended into a paged cache (16-bit, E4M3 or E2M1);
* ``append4``: k and v appended into an E2M1 cache without rotation;
* ``gather``: rows of a paged cache read back as 16-bit rows;
* ``decode4``: single-token attention over an E2M1 cache.

An append into a quantised cache is followed by a gather of the same slots:
the pass returns the values that the cache then stands for.  ``own`` selects
the library's calls; otherwise the same results come from plain torch
operations in 32 bits.

An E2M1 pool is uint8 [num_blocks][num_kv_heads][block_size * D * 9 / 16]:
per (block, head) the codes [block_size][D / 2] (even dim in the low nibble),
then the E4M3 block scales [block_size][D / 16].  value = code * block scale *
head scale.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
FORMATS = {"16": 0, "fp8": 1, "fp4": 4}     # pa_cache_format values
MAX_POSITION = 8192                          # rows of the rotation table
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # the tiny workload's next tokens: the smallest call, all latency
        dict(name="rope next token x4, 16-bit", kind="rope", tokens=4, hq=4, hkv=4, d=64, bs=16, dtype="f16",
             fmt="16", rotary=64, interleaved=False, fused=False, runs=False, padded=0),
        # one decode step of a 256-sequence batch, 64/8 heads, into the 4-bit cache; 5 padding rows as a captured step has
        dict(name="rope next token x256, 4-bit", kind="rope", tokens=256, hq=64, hkv=8, d=128, bs=16, dtype="bf16",
             fmt="fp4", rotary=128, interleaved=False, fused=True, runs=False, padded=5),
        # a chunk of prompts, 32/8 heads, sliced out of a fused projection
        dict(name="rope prompts 8191, 16-bit", kind="rope", tokens=8191, hq=32, hkv=8, d=128, bs=16, dtype="bf16",
             fmt="16", rotary=128, interleaved=False, fused=True, runs=True, padded=0),
        # long prompts of a 32/32-head model that rotates half of each head in interleaved pairs, E4M3 cache, blocks of 256
        dict(name="rope prompts 16384, 8-bit", kind="rope", tokens=16384, hq=32, hkv=32, d=128, bs=256, dtype="f16",
             fmt="fp8", rotary=64, interleaved=True, fused=False, runs=True, padded=0),
        # one decode step of a 64-sequence batch, 32/32 heads, rotation done elsewhere
        dict(name="append4 next token x64", kind="append4", tokens=64, hq=32, hkv=32, d=128, bs=16, dtype="f16",
             fmt="fp4", runs=False, padded=0),
        # prompts of a 32/8-head model into the 4-bit cache
        dict(name="append4 prompts 20011", kind="append4", tokens=20011, hq=32, hkv=8, d=128, bs=16, dtype="bf16",
             fmt="fp4", runs=True, padded=11),
        # one sequence's prompt read back out of an E4M3 cache
        dict(name="gather one sequence, 8-bit", kind="gather", tokens=333, hq=32, hkv=32, d=128, bs=16, dtype="f16",
             fmt="fp8", runs=True, padded=0),
        # the prompts of a batch read back out of the 4-bit cache, for a dense attention over the continuation
        dict(name="gather prompts 65536, 4-bit", kind="gather", tokens=65536, hq=32, hkv=8, d=128, bs=16, dtype="bf16",
             fmt="fp4", runs=True, padded=0),
        # one sequence alone: latency
        dict(name="decode4 one sequence", kind="decode4", seqs=1, hq=32, hkv=8, d=128, bs=16, dtype="bf16",
             lo=1000, hi=1000, empty=0),
        # a 64-sequence batch of short contexts, one query head per kv head
        dict(name="decode4 64 x 32/32", kind="decode4", seqs=64, hq=32, hkv=32, d=128, bs=16, dtype="f16",
             lo=64, hi=1024, empty=0),
        # a 128-sequence batch, 32/8 heads
        dict(name="decode4 128 x 32/8", kind="decode4", seqs=128, hq=32, hkv=8, d=128, bs=16, dtype="bf16",
             lo=1024, hi=4096, empty=0),
        # few long contexts, 64/8 heads: work split along the context
        dict(name="decode4 6 long x 64/8", kind="decode4", seqs=6, hq=64, hkv=8, d=128, bs=16, dtype="bf16",
             lo=8191, hi=131071, empty=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "rope", "append4", "gather", "decode4", "decode4", "decode4"])
    d = rng.choice([64, 128, 128])
    bs = rng.choice([8, 16, 16, 24, 32, 64, 256])
    group = rng.choice([1, 2, 4, 8, 16])
    hkv = rng.choice([1, 2, 3, 4, 5, 8, 8, 16]) if group > 1 else rng.choice([1, 4, 7, 12, 32])
    while group * hkv > 64:
        hkv = max(1, hkv // 2)
    case = dict(kind=kind, hq=group * hkv, hkv=hkv, d=d, bs=bs, dtype=rng.choice(["f16", "bf16"]))
    if kind == "decode4":
        hi = _log_int(rng, 1, 65536)
        lo = _log_int(rng, 1, hi)
        # at most 2^28 cached elements in each pool
        most = max(1, (1 << 28) // (hi * hkv * d))
        seqs = _log_int(rng, 1, min(256, most))
        case.update(seqs=seqs, lo=lo, hi=hi, empty=rng.choice([0, 0, 1]) if seqs > 1 else 0)
        return case
    # at most 2^25 elements of a token's q, k and v rows together
    most = max(2, (1 << 25) // ((case["hq"] + 2 * hkv) * d))
    tokens = _log_int(rng, 1, min(most, 50000))
    case.update(tokens=tokens, runs=rng.choice([False, True]), padded=rng.choice([0, tokens // 5]))
    case["fmt"] = "fp4" if kind == "append4" else rng.choice(["16", "fp8", "fp4", "fp4"])
    if kind == "rope":
        case.update(rotary=rng.choice([d, d, d // 2, 16, 48, 32]), interleaved=rng.choice([False, True]),
                    fused=rng.choice([False, True]))
    if kind == "gather":
        case["padded"] = 0
    return case


# ---------------------------------------------------------------------------
# inputs


def _scales(g, hkv):
    """Head scales near 1 / 8, as calibration on rows of unit variance gives them."""
    return (torch.rand(hkv, generator=g, device="cuda") * 0.1 + 0.08).float()


def _e2m1_index(y):
    """0..7: the E2M1 magnitude nearest to y >= 0 (ties to the even code)."""
    return ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))


def _quantise4(x, scale):
    """x fp32 [..., Hkv, D], scale [Hkv]: signed codes (0..15) [..., D] and E4M3 block scales [..., D / 16]."""
    b = x.unflatten(-1, (-1, 16))
    h = scale.view(-1, 1)
    s = (b.abs().amax(-1) / 6.0 / h).clamp(max=448.0).to(torch.float8_e4m3fn)
    f = s.float()
    r = torch.where(f > 0, 1.0 / (f * h), torch.zeros_like(f))
    y = b * r.unsqueeze(-1)
    code = _e2m1_index(y.abs()) + (b.signbit().to(torch.uint8) << 3)
    return code.flatten(-2), s


def _fill_pool4(pool, scale, g, bs, hkv, d):
    """Random unit-variance rows in an E2M1 pool [NB][Hkv][bs * D * 9 / 16]."""
    nb, codes = pool.shape[0], bs * d // 2
    step = max(1, (1 << 25) // (bs * hkv * d))
    for i in range(0, nb, step):
        n = min(step, nb - i)
        x = torch.randn((n, bs, hkv, d), generator=g, device="cuda")
        c, s = _quantise4(x, scale)
        c, s = c.transpose(1, 2), s.transpose(1, 2)
        pool[i:i + n, :, :codes] = (c[..., 0::2] | (c[..., 1::2] << 4)).reshape(n, hkv, codes)
        pool[i:i + n, :, codes:] = s.contiguous().view(torch.uint8).reshape(n, hkv, -1)


def _lens(case, g=None):
    """Context lengths: evenly spread over [lo, hi] (the first `empty` of them 0), in an order the seed gives."""
    n, e = case["seqs"], case["empty"]
    m = n - e
    lens = [0] * e + [case["hi"] - (case["hi"] - case["lo"]) * i // max(1, m - 1) for i in range(m)]
    if g is not None:
        order = torch.randperm(n, generator=g, device="cuda").tolist()
        lens = [lens[i] for i in order]
    return lens


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, d, bs, hq, hkv = DTYPES[case["dtype"]], case["d"], case["bs"], case["hq"], case["hkv"]
    st = dict(case=case)
    st["ks"], st["vs"] = _scales(g, hkv), _scales(g, hkv)

    if case["kind"] == "decode4":
        lens = _lens(case, g)
        need = [-(-n // bs) for n in lens]
        nb = sum(need) + max(1, sum(need) // 4)
        order = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
        mbs = max(need)
        tables = torch.full((len(lens), mbs), -1, dtype=torch.int32, device="cuda")
        at = 0
        for i, n in enumerate(need):
            tables[i, :n] = order[at:at + n]
            at += n
        st["tables"], st["lens"] = tables, torch.tensor(lens, dtype=torch.int32, device="cuda")
        st["maxlen"], st["scale"] = max(lens), 1.0 / math.sqrt(d)
        st["nb"] = nb
        st["kc"] = torch.empty((nb, hkv, bs * d * 9 // 16), dtype=torch.uint8, device="cuda")
        st["vc"] = torch.empty_like(st["kc"])
        _fill_pool4(st["kc"], st["ks"], g, bs, hkv, d)
        _fill_pool4(st["vc"], st["vs"], g, bs, hkv, d)
        st["q"] = torch.randn((len(lens), hq, d), generator=g, device="cuda").to(dt)
        st["out"] = torch.zeros_like(st["q"])
        return st

    # token rows: slots of whole runs of blocks (prompts), or scattered (one token per sequence)
    n = case["tokens"]
    nb = -(-n // bs) + max(2, n // bs // 4)
    if case["runs"]:
        order = torch.randperm(nb, generator=g, device="cuda")
        t = torch.arange(n, device="cuda")
        slots = order[t // bs] * bs + t % bs
    else:
        slots = torch.randperm(nb * bs, generator=g, device="cuda")[:n]
    if case["padded"]:
        slots[n - case["padded"]:] = -1
    st["slots"], st["nb"] = slots.to(torch.int32), nb
    fmt = case["fmt"]
    if fmt == "fp4":
        st["kc"] = torch.zeros((nb, hkv, bs * d * 9 // 16), dtype=torch.uint8, device="cuda")
        st["vc"] = torch.zeros_like(st["kc"])
    elif fmt == "fp8":
        st["kc"] = torch.zeros((nb, bs, hkv, d), dtype=torch.uint8, device="cuda")
        st["vc"] = torch.zeros_like(st["kc"])
    else:
        st["kc"] = torch.zeros((nb, bs, hkv, d), dtype=dt, device="cuda")
        st["vc"] = torch.zeros_like(st["kc"])
    if case["kind"] == "gather":
        if fmt == "fp4":
            _fill_pool4(st["kc"], st["ks"], g, bs, hkv, d)
            _fill_pool4(st["vc"], st["vs"], g, bs, hkv, d)
        elif fmt == "fp8":
            for c, s in ((st["kc"], st["ks"]), (st["vc"], st["vs"])):
                x = torch.randn(c.shape, generator=g, device="cuda") / s.view(-1, 1)
                c.copy_(x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8))
        else:
            st["kc"].normal_(generator=g)
            st["vc"].normal_(generator=g)
    else:
        if case.get("fused"):
            x = torch.randn((n, (hq + 2 * hkv) * d), generator=g, device="cuda").to(dt)
            q, k, v = x.split([hq * d, hkv * d, hkv * d], dim=1)
            st["q"], st["k"], st["v"] = (y.unflatten(1, (-1, d)) for y in (q, k, v))
        else:
            if case["kind"] == "rope":
                st["q"] = torch.randn((n, hq, d), generator=g, device="cuda").to(dt)
            st["k"] = torch.randn((n, hkv, d), generator=g, device="cuda").to(dt)
            st["v"] = torch.randn((n, hkv, d), generator=g, device="cuda").to(dt)
    if case["kind"] == "rope":
        r = case["rotary"]
        if case["runs"]:
            first = int(torch.randint(0, MAX_POSITION, (1,), generator=g, device="cuda"))
            st["positions"] = ((torch.arange(n, device="cuda") + first) % MAX_POSITION).to(torch.int32)
        else:
            st["positions"] = torch.randint(0, MAX_POSITION, (n,), generator=g, device="cuda", dtype=torch.int32)
        inv = 10000.0 ** (-torch.arange(0, r, 2, device="cuda", dtype=torch.float64) / r)
        ang = torch.arange(MAX_POSITION, device="cuda", dtype=torch.float64)[:, None] * inv
        st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], dim=1).float()
        st["q_out"] = torch.zeros((n, hq, d), dtype=dt, device="cuda")
    if fmt != "16" or case["kind"] == "gather":
        st["k_out"] = torch.zeros((n, hkv, d), dtype=dt, device="cuda")
        st["v_out"] = torch.zeros_like(st["k_out"])
    return st


# ---------------------------------------------------------------------------
# plain forms


def _unpack4(rows, codes, scale, d):
    """Pool rows [..., bytes of one (block, head)] with `codes` code bytes: fp32 values [..., bs, D]; scale broadcasts over [..., bs, D]."""
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=rows.device)
    c = rows[..., :codes]
    c = torch.stack([c & 15, c >> 4], dim=-1).flatten(-2).unflatten(-1, (-1, d))
    s = rows[..., codes:].contiguous().view(torch.float8_e4m3fn).float().unflatten(-1, (-1, d // 16))
    return lut[c.int()] * s.repeat_interleave(16, dim=-1) * scale


def _stored(x, scale, fmt):
    """The value that the cache holds for x fp32 [..., Hkv, D]."""
    if fmt == "fp8":
        return (x / scale.view(-1, 1)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float() * scale.view(-1, 1)
    if fmt == "fp4":
        code, s = _quantise4(x, scale)
        lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=x.device)
        return lut[code.int()] * s.float().repeat_interleave(16, dim=-1) * scale.view(-1, 1)
    return x


def _rotate(x, cos, sin, rotary, interleaved):
    """x fp32 [T, H, D]; cos, sin [T, 1, rotary / 2]."""
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rotary:2], x[..., 1:rotary:2]
        y[..., 0:rotary:2] = a * cos - b * sin
        y[..., 1:rotary:2] = b * cos + a * sin
    else:
        h = rotary // 2
        a, b = x[..., :h], x[..., h:rotary]
        y[..., :h] = a * cos - b * sin
        y[..., h:rotary] = b * cos + a * sin
    return y


def _plain_append(st, k, v):
    """k, v fp32 rows, rounded to the element type: into the pool, or the values a quantised pool stands for."""
    case, dt = st["case"], DTYPES[st["case"]["dtype"]]
    k, v = k.to(dt), v.to(dt)
    keep = st["slots"] >= 0
    if case["fmt"] == "16":
        at = st["slots"][keep].long()
        st["kc"].flatten(0, 1)[at] = k[keep]
        st["vc"].flatten(0, 1)[at] = v[keep]
        return st["kc"], st["vc"]
    keep = keep[:, None, None]
    return (torch.where(keep, _stored(k.float(), st["ks"], case["fmt"]).to(dt), st["k_out"]),
            torch.where(keep, _stored(v.float(), st["vs"], case["fmt"]).to(dt), st["v_out"]))


def _plain_rope(st):
    case, dt = st["case"], DTYPES[st["case"]["dtype"]]
    cs = st["cos_sin"][st["positions"].long()].unsqueeze(1)
    cos, sin = cs.chunk(2, dim=-1)
    q = _rotate(st["q"].float(), cos, sin, case["rotary"], case["interleaved"]).to(dt)
    k = _rotate(st["k"].float(), cos, sin, case["rotary"], case["interleaved"])
    q = torch.where((st["slots"] >= 0)[:, None, None], q, st["q_out"])
    return (q,) + _plain_append(st, k, st["v"].float())


def _plain_gather(st):
    case, dt = st["case"], DTYPES[st["case"]["dtype"]]
    bs, d, at = case["bs"], case["d"], st["slots"].long()

    def rows(pool, scale):
        if case["fmt"] == "fp4":
            codes = bs * d // 2
            c = pool[..., :codes].unflatten(-1, (bs, d // 2))[at // bs, :, at % bs]
            s = pool[..., codes:].unflatten(-1, (bs, d // 16))[at // bs, :, at % bs]
            x = _unpack4(torch.cat([c, s], dim=-1), d // 2, scale.view(-1, 1, 1), d).squeeze(-2)
        else:
            x = pool.flatten(0, 1)[at]
            if case["fmt"] == "fp8":
                x = x.view(torch.float8_e4m3fn).float() * scale.view(-1, 1)
        return x.to(dt)

    return rows(st["kc"], st["ks"]), rows(st["vc"], st["vs"])


def _plain_decode4(st):
    case = st["case"]
    d, bs, hq, hkv = case["d"], case["bs"], case["hq"], case["hkv"]
    n, m = st["tables"].shape
    blocks = st["tables"].clamp(min=0).long()
    valid = torch.arange(m * bs, device="cuda") < st["lens"][:, None]                     # [S, L]
    k = _unpack4(st["kc"][blocks], bs * d // 2, st["ks"].view(-1, 1, 1), d)               # [S, M, Hkv, bs, D]
    k = k.transpose(1, 2).reshape(n, hkv, m * bs, d)
    x = st["q"].float().view(n, hkv, hq // hkv, d) @ k.transpose(-1, -2) * st["scale"]
    del k
    x = x.masked_fill(~valid[:, None, None, :], -math.inf)
    p = (x - x.amax(-1, keepdim=True).clamp(min=-1e30)).exp()
    v = _unpack4(st["vc"][blocks], bs * d // 2, st["vs"].view(-1, 1, 1), d)
    v = v.transpose(1, 2).reshape(n, hkv, m * bs, d)
    v = v.masked_fill(~valid[:, None, :, None], 0.0)
    o = p @ v / p.sum(-1, keepdim=True)
    o = torch.where(st["lens"].view(-1, 1, 1, 1) > 0, o, torch.zeros_like(o))
    return o.reshape(n, hq, d).to(DTYPES[case["dtype"]])


# ---------------------------------------------------------------------------
# the library's calls


def _handle(st, pa):
    """The shape record (and for the attention its workspace, for the rotation its parameters) that a program keeps."""
    if "shape" not in st:
        c = st["case"]
        st["shape"] = pa.make_shape(
            num_seqs=c.get("seqs", 1), num_q_heads=c["hq"], num_kv_heads=c["hkv"], head_dim=c["d"],
            block_size=c["bs"], num_blocks=st["nb"],
            max_blocks_per_seq=st["tables"].shape[1] if "tables" in st else 1,
            dtype=pa.PA_F16 if c["dtype"] == "f16" else pa.PA_BF16, cache_format=FORMATS[c.get("fmt", "fp4")])
        if c["kind"] == "decode4":
            st["ws"] = torch.empty(pa.pa_decode_workspace_bytes(st["shape"], st["maxlen"]), dtype=torch.uint8, device="cuda")
        if c["kind"] == "rope":
            st["rope"] = pa.make_rope(rotary_dim=c["rotary"], interleaved=int(c["interleaved"]), max_position=MAX_POSITION,
                                      q_stride=st["q"].stride(0), k_stride=st["k"].stride(0), v_stride=st["v"].stride(0))
    return st["shape"]


def run(state):
    st, kind = state, state["case"]["kind"]
    if not own:
        if kind == "rope":
            return _plain_rope(st)
        if kind == "append4":
            return _plain_append(st, st["k"].float(), st["v"].float())
        if kind == "gather":
            return _plain_gather(st)
        return _plain_decode4(st)
    from paged_kv_cache_458_b200 import pa
    shape = _handle(st, pa)
    if kind == "decode4":
        pa.pa_decode_fp4(st["q"], st["kc"], st["vc"], st["ks"], st["vs"], st["tables"], st["lens"], st["scale"],
                         st["out"], shape, st["maxlen"], st["ws"])
        return st["out"]
    n, quantised = st["case"]["tokens"], st["case"]["fmt"] != "16"
    scales = (st["ks"], st["vs"]) if quantised else (None, None)
    if kind == "rope":
        pa.pa_rope_append(st["q"], st["k"], st["v"], st["positions"], st["cos_sin"], st["rope"], st["slots"], n,
                          st["q_out"], st["kc"], st["vc"], *scales, shape)
    elif kind == "append4":
        pa.pa_cache_append_fp4(st["k"], st["v"], st["slots"], n, st["kc"], st["vc"], *scales, shape)
    if quantised or kind == "gather":
        pa.pa_cache_gather(st["slots"], n, st["kc"], st["vc"], *scales, st["k_out"], st["v_out"], shape)
        kv = st["k_out"], st["v_out"]
    else:
        kv = st["kc"], st["vc"]
    return (st["q_out"],) + kv if kind == "rope" else kv


def work(case):
    d, hq, hkv, bs = case["d"], case["hq"], case["hkv"], case["bs"]
    if case["kind"] == "decode4":
        lens = _lens(case)
        cached = sum(lens) * hkv * d
        return {"bytes": 2 * cached * 9 / 16 + 4 * len(lens) * hq * d + 4 * sum(-(-n // bs) for n in lens) + 4 * len(lens),
                "flops": 4.0 * sum(lens) * hq * d}
    n = case["tokens"] - case["padded"]
    kv = 2 * n * hkv * d                                        # elements of K and V together
    held = {"16": 2, "fp8": 1, "fp4": 9 / 16}[case["fmt"]]
    if case["kind"] == "gather":
        return {"bytes": kv * (held + 2) + 4 * n, "flops": 2.0 * kv}
    # an append reads its rows and writes the cache; a quantised one is then read back
    total = kv * (2 + held) + 4 * n + (kv * (held + 2) + 4 * n if case["fmt"] != "16" else 0)
    flops = 4.0 * kv
    if case["kind"] == "rope":
        total += 4 * n * hq * d + 4 * n + 4 * min(n, MAX_POSITION) * case["rotary"]
        flops += 3.0 * n * (hq + hkv) * case["rotary"]
    return {"bytes": total, "flops": flops}


# ---------------------------------------------------------------------------
# 64 bits


def _grid(bits_exponent, bits_mantissa, bias, top):
    """Every non-negative value of a small float type, ascending."""
    vals = set()
    for e in range(1 << bits_exponent):
        for m in range(1 << bits_mantissa):
            f = m / (1 << bits_mantissa)
            vals.add((f if e == 0 else 1.0 + f) * 2.0 ** ((e if e else 1) - bias))
    return torch.tensor(sorted(v for v in vals if v <= top), dtype=torch.float64, device="cuda")


def _nearest(y, grid):
    """The entry of `grid` nearest to y >= 0, ties to the even index (the even code)."""
    hi = torch.searchsorted(grid, y).clamp(max=grid.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    dl, dh = y - grid[lo], grid[hi] - y
    return grid[torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)]


def _exact_stored(x, scale, fmt):
    h = scale.double().view(-1, 1)
    if fmt == "fp8":
        return torch.sign(x) * _nearest((x / h).abs(), _grid(4, 3, 7, 448.0)) * h
    b = x.unflatten(-1, (-1, 16))
    s = _nearest(b.abs().amax(-1) / (6.0 * h), _grid(4, 3, 7, 448.0)).unsqueeze(-1) * h.unsqueeze(-1)
    y = torch.where(s > 0, b.abs() / s.clamp(min=1e-300), torch.zeros_like(b))
    return (torch.sign(b) * _nearest(y, _grid(2, 1, 1, 6.0)) * s).flatten(-2)


def _exact_rows4(pool, block, head, offset, case, scale):
    """fp64 rows [n, D] of slots (block, offset) of one head."""
    bs, d = case["bs"], case["d"]
    raw = pool[:, head]
    byte = torch.arange(d, device="cuda") // 2
    c = raw[block[:, None], offset[:, None] * (d // 2) + byte].long()
    c = (c >> (4 * (torch.arange(d, device="cuda") % 2))) & 15
    s = raw[block[:, None], bs * d // 2 + offset[:, None] * (d // 16) + torch.arange(d, device="cuda") // 16]
    grid = _grid(2, 1, 1, 6.0)
    return grid[c & 7] * (1 - 2 * (c >> 3)).double() * s.view(torch.float8_e4m3fn).double() * scale[head].double()


def exact(case, seed):
    st = prepare(case, seed)
    d, bs, hq, hkv = case["d"], case["bs"], case["hq"], case["hkv"]
    if case["kind"] == "decode4":
        out = torch.zeros((case["seqs"], hq, d), dtype=torch.float64, device="cuda")
        for i, n in enumerate(st["lens"].tolist()):
            t = torch.arange(n, device="cuda")
            block = st["tables"][i].long()[t // bs]
            for h in range(hkv if n else 0):
                heads = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
                k = _exact_rows4(st["kc"], block, h, t % bs, case, st["ks"])
                w = torch.softmax(st["q"][i, heads].double() @ k.T * st["scale"], dim=-1)
                out[i, heads] = w @ _exact_rows4(st["vc"], block, h, t % bs, case, st["vs"])
        return out
    slots = st["slots"].long()
    keep = (slots >= 0)[:, None, None]
    if case["kind"] == "gather":
        got = []
        for pool, scale in ((st["kc"], st["ks"]), (st["vc"], st["vs"])):
            if case["fmt"] == "fp4":
                got.append(torch.stack([_exact_rows4(pool, slots // bs, h, slots % bs, case, scale) for h in range(hkv)], dim=1))
            elif case["fmt"] == "fp8":
                got.append(pool.flatten(0, 1)[slots].view(torch.float8_e4m3fn).double() * scale.double().view(-1, 1))
            else:
                got.append(pool.flatten(0, 1)[slots].double())
        return tuple(got)
    k, v, got = st["k"].double(), st["v"].double(), ()
    if case["kind"] == "rope":
        r = case["rotary"]
        first = torch.arange(0, r, 2, device="cuda") if case["interleaved"] else torch.arange(r // 2, device="cuda")
        second = first + (1 if case["interleaved"] else r // 2)
        cs = st["cos_sin"][st["positions"].long()].double()
        turn = torch.complex(cs[:, :r // 2], cs[:, r // 2:]).unsqueeze(1)

        def rotated(x):
            z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
            y = x.clone()
            y[..., first], y[..., second] = z.real, z.imag
            return y

        got = (torch.where(keep, rotated(st["q"].double()), 0.0),)
        k = rotated(k)
    if case["fmt"] == "16":
        for pool, x in ((st["kc"], k), (st["vc"], v)):
            full = pool.double()
            full.flatten(0, 1)[slots[slots >= 0]] = x[slots >= 0]
            got += (full,)
        return got
    # a quantised cache holds the codes of the rows as the element type has them
    k, v = k.to(DTYPES[case["dtype"]]).double(), v.to(DTYPES[case["dtype"]]).double()
    return got + tuple(torch.where(keep, _exact_stored(x, s, case["fmt"]), 0.0) for x, s in ((k, st["ks"]), (v, st["vs"])))
