"""Inputs and a plain 64-bit attention for the tests of int8 pools, with the error each output element may have."""
import torch

import paged_kv_cache_409_b200 as pkv


def make_pools(lens, B, Hkv, D, seed, k_size=1.0, v_size=1.0, v_spread=0, NB_extra=3, device="cuda"):
    """Pools whose live rows are quantised normal rows (V rows scaled by 2^[-v_spread, v_spread]); every other slot
    holds random codes and the scale NaN, unused table entries are -1.  Returns (key pool, value pool, tables)."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // B) for n in lens]
    NB = sum(need) + NB_extra
    perm = torch.randperm(NB, generator=g)
    tables = torch.full((len(lens), max(max(need), 1) + 1), -1, dtype=torch.int32)
    slots, at = [], 0
    for i, (n, k) in enumerate(zip(lens, need)):
        ids = perm[at: at + k]
        at += k
        tables[i, :k] = ids.to(torch.int32)
        pos = torch.arange(n)
        slots.append(ids[pos // B] * B + pos % B)
    slots = torch.cat(slots) if slots else torch.zeros(0, dtype=torch.int64)
    pools = []
    for size in (k_size, v_size):
        pool = torch.randint(0, 256, (NB, B, Hkv, D + 4), generator=g, dtype=torch.uint8)
        pkv.int8_pool_views(pool)[1].fill_(float("nan"))
        x = torch.randn(len(slots), Hkv, D, generator=g) * size
        if v_spread and len(pools) == 1:
            x = x * torch.exp2(torch.randint(-v_spread, v_spread + 1, (len(slots), Hkv, 1), generator=g).float())
        codes, scales = pkv.int8_pool_views(pool)
        s = x.abs().amax(-1) / 127
        codes[slots // B, slots % B] = (128 + torch.round(x / s[..., None])).to(torch.uint8)
        scales[slots // B, :, slots % B] = s
        pools.append(pool.to(device))
    return pools[0], pools[1], tables.to(device)


def rows_of(pool, table, n):
    """The first n rows of a sequence, [n, Hkv, D], and their scales [n, Hkv], in 64 bits."""
    B = pool.shape[1]
    codes, scales = pkv.int8_pool_views(pool)
    pos = torch.arange(n, device=pool.device)
    ids = table.long()[pos // B]
    s = scales[ids, :, pos % B].double()
    return (codes[ids, pos % B].double() - 128) * s[..., None], s


def reference(q, kp, vp, table, n, scale, dtype, first=None):
    """Attention of the rows q [r, Hq, D] over the first n cached rows (row i over first[i] + 1 of them when `first`
    is given: a chunk), in 64 bits, and the error bound of each element of a result rounded to `dtype`.

    Decode: the query's 16-bit integer row is off by at most 0.52 steps of max |q| / 32639 an element (half a step,
    and fp32's product), a score by that times the key's sum of magnitudes.  Chunks: keys and values are widened to
    f16, off by half a step, 2^-11 (2^-25 below 2^-14), and the scale's second part, under 2^-20.
    Scores, exponentials and sums in fp32, and the hardware's base-2 functions: 2e-5 of a weight at the sizes used
    here (scores below 64 in log2 units: 4 roundings of 2^-24 each, 2^-22 for the functions).  A weight goes into
    the product as f16: half a step, 2^-11, of it, or 2^-25 of the base for the small ones; the base is at most the
    largest product of weight and V scale (decode; then times codes up to 127) or weight (chunks)."""
    K, _ = rows_of(kp, table, n)
    V, vs = rows_of(vp, table, n)
    G = q.shape[1] // K.shape[1]
    K, V, vs = (t.repeat_interleave(G, 1) for t in (K, V, vs))
    q = q.double()
    t = torch.einsum("rhd,nhd->rhn", q, K) * scale
    if first is not None:
        hidden = torch.arange(n, device=q.device)[None, None, :] > first[:, None, None]
        t = t.masked_fill(hidden, -float("inf"))
    p = torch.softmax(t, -1)
    ref = torch.einsum("rhn,nhd->rhd", p, V)
    size = torch.einsum("rhn,nhd->rhd", p, V.abs())
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    if first is None:
        ds = abs(scale) * 0.52 * q.abs().amax(-1) / 32639 * K.abs().sum(-1).amax(0)
        weight, top = 2.0 ** -11, (p * vs.T[None]).amax(-1) * 127
    else:
        ds = abs(scale) * ((2.0 ** -11 + 2.0 ** -20) * torch.einsum("rhd,nhd->rhn", q.abs(), K.abs()).amax(-1)
                           + 2.0 ** -25 * q.abs().sum(-1))
        weight, top = 2.0 ** -10 + 2.0 ** -20, p.amax(-1) * V.abs().amax()
        tiny += 2.0 ** -25
    bound = torch.finfo(dtype).eps / 2 * ref.abs() * (1 + 2.0 ** -10) + (weight + 2e-5 + 2 * ds)[..., None] * size \
        + (n * 2.0 ** -25 * top)[..., None] + tiny
    return ref, bound


def check(out, ref, bound, what=""):
    assert bool(torch.isfinite(out.double()).all()), f"{what}: non-finite"
    over = (out.double() - ref).abs() - bound
    assert over.numel() == 0 or float(over.max()) <= 0, f"{what}: over by {float(over.max())}"
