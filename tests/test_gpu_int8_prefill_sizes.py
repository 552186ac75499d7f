"""Chunked prefill over int8 pools whose rows are very small, very large or of mixed sizes, against plain 64-bit attention over
the same codes and scales, with one, two and many visible keys."""
import pytest
import torch

import paged_kv_cache_409_b200 as pkv
from int8_helpers import check, make_pools, rows_of

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def reference(q, kp, vp, table, n, first, scale, dtype):
    """Attention in 64 bits of the rows q [r, Hq, D] over cached rows 0 .. first[i], and the error each element may have.

    Fp16 queries take keys and values exactly, and are off by less than what follows for bf16 ones, whose keys and values go
    into the products as f16 numbers in units of their own: the unit puts the largest K row of a tile of 128
    keys at 2^14 or above, the largest V row so far at 2^12 or above (an element is then below 2^15).  An element c S, |c| <= 1,
    is formed from S in two f16 parts: the split is off by 2^-22 of S, the second part's product by half a step (2^-22 of c S),
    the sum by half a step, 2^-11: 2^-11 + 2^-20 of the element, and 2^-25 for each of the three where f16 is subnormal, 3 *
    2^-25 / 2^12 < 2^-35 of the largest row.  A bf16 query row is scaled likewise, exactly, but for elements below 2^-28 of its
    largest (2^-39 of that).  A weight goes into the product as f16: 2^-11 of it, or 2^-25 of the base, which is at most the
    largest weight.  Scores, exponentials and sums in fp32: 2e-5 of a weight at these sizes (scores below 64 in log2 units).
    The result is rounded to its type: half a step, or 2^-25 (fp16)."""
    K, _ = rows_of(kp, table, n)
    V, _ = rows_of(vp, table, n)
    G = q.shape[1] // K.shape[1]
    K, V = (t.repeat_interleave(G, 1) for t in (K, V))
    q = q.double()
    t = torch.einsum("rhd,nhd->rhn", q, K) * scale
    t = t.masked_fill(torch.arange(n, device=q.device)[None, None, :] > first[:, None, None], -float("inf"))
    p = torch.softmax(t, -1)
    ref = torch.einsum("rhn,nhd->rhd", p, V)
    size = torch.einsum("rhn,nhd->rhd", p, V.abs())
    k_top, v_top = (x.abs().amax((0, 2)) for x in (K, V))  # [Hq]
    one = 2.0 ** -11 + 2.0 ** -20
    ds = abs(scale) * (one * torch.einsum("rhd,nhd->rhn", q.abs(), K.abs()).amax(-1)
                       + 2.0 ** -35 * k_top * q.abs().sum(-1) + 2.0 ** -39 * q.abs().amax(-1) * K.abs().sum(-1).amax(0))
    bound = torch.finfo(dtype).eps / 2 * ref.abs() * (1 + 2.0 ** -10) + (2.0 ** -11 + one + 2e-5 + 2 * ds)[..., None] * size \
        + ((2.0 ** -35 + n * 2.0 ** -25 * p.amax(-1)) * v_top)[..., None] + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    return ref, bound


def prefill(q, kp, vp, bt, ns, lens, scale):
    out = torch.full_like(q, 7.0)
    qsl = torch.tensor([0] + ns, device="cuda").cumsum(0).to(torch.int32)
    pkv.paged_attention_prefill_chunk_int8(out, q, kp, vp, bt, torch.tensor(lens, dtype=torch.int32, device="cuda"), qsl,
                                           max(ns), scale)
    assert pkv.get_device_error() == 0
    return out


def compare(q, kp, vp, bt, ns, lens, scale, what):
    out = prefill(q, kp, vp, bt, ns, lens, scale)
    at = 0
    for i, (n, L) in enumerate(zip(ns, lens)):
        ref, bound = reference(q[at: at + n], kp, vp, bt[i], L, torch.arange(L - n, L, device="cuda"), scale, q.dtype)
        check(out[at: at + n], ref, bound, f"{what} chunk {i}")
        at += n


# (visible keys of a chunk's rows): one, two, nine, and several tiles; one long sequence of few items is shared by a cluster
CHUNKS = [([1, 2, 9, 140], [1, 2, 9, 333]), ([3], [1500])]


@pytest.mark.parametrize("chunks", CHUNKS, ids=["whole", "shared"])
@pytest.mark.parametrize("D,G", [(128, 4), (64, 1)])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("v_size", [400.0, 1e-2, 1e-3, 1e-4, 1e-5, 3e-6, 1e-8, 1e-15])
def test_small_value_rows(v_size, dt, D, G, chunks):
    ns, lens = chunks
    kp, vp, bt = make_pools(lens, 16, 2, D, seed=D, v_size=v_size)
    q = torch.randn(sum(ns), 2 * G, D, device="cuda").to(DT[dt])
    compare(q, kp, vp, bt, ns, lens, D ** -0.5, f"V rows of {v_size}")


@pytest.mark.parametrize("chunks", CHUNKS, ids=["whole", "shared"])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("k_size", [100.0, 1e-3, 1e-5, 1e-7, 1e-12])
def test_small_key_rows(k_size, dt, chunks):
    """Keys of any size under a score scale that undoes it."""
    ns, lens = chunks
    kp, vp, bt = make_pools(lens, 32, 2, 128, seed=7, k_size=k_size)
    q = torch.randn(sum(ns), 4, 128, device="cuda").to(DT[dt])
    compare(q, kp, vp, bt, ns, lens, 0.09 / k_size, f"K rows of {k_size}")


@pytest.mark.parametrize("chunks", CHUNKS, ids=["whole", "shared"])
@pytest.mark.parametrize("D,G", [(128, 2), (64, 8)])
def test_bf16_queries_of_any_size(D, G, chunks):
    """Every query row has a size of its own, and its scores are near zero or moderate; a zero row attends evenly."""
    ns, lens = chunks
    kp, vp, bt = make_pools(lens, 8, 2, D, seed=11)
    q = torch.randn(sum(ns), 2 * G, D, device="cuda")
    q *= torch.exp2(-30.0 * torch.rand(sum(ns), 2 * G, 1, device="cuda"))
    q[-1, 0] = 0
    for size, scale in ((1e30, 1e-31), (1e6, 1e-7), (1.0, 0.1), (1e-10, 1e9), (1e-30, 1e29)):
        compare((q * size).bfloat16(), kp, vp, bt, ns, lens, scale, f"queries of {size}")


def tiles_of_sizes(exponents, Hkv, D, which):
    """Pools of one sequence whose rows of tile i (128 keys) have sizes around 2^exponents[i]; None: zero rows."""
    n = 128 * len(exponents)
    pools = list(make_pools([n], 32, Hkv, D, seed=13))
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(n, Hkv, D, device="cuda", generator=g)
    for i, e in enumerate(exponents):
        x[128 * i: 128 * (i + 1)] *= 0.0 if e is None else 2.0 ** e
    y = torch.randn(n, Hkv, D, device="cuda", generator=g)
    pos = torch.arange(n, device="cuda")
    slots = pools[2][0].long()[pos // 32] * 32 + pos % 32
    k, v = (x, y) if which == "K" else (y, x)
    pkv.reshape_and_cache_int8(k, v, pools[0], pools[1], slots)
    return pools, n


@pytest.mark.parametrize("Hkv,ns_last", [(2, 5), (2, 200), (160, 130)], ids=["cluster", "two tiles", "whole"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("exponents", [(0, 1, 2, 3, 4, 5, 6), (-40, -30, -20, -10, 0, 4), (6, 0, -6, -12), (None, None, -14, 2),
                                       (0, None, 5, None, 8), (None, None, None)], ids=str)
def test_value_rows_that_grow_and_shrink_from_tile_to_tile(exponents, D, Hkv, ns_last):
    (kp, vp, bt), n = tiles_of_sizes(exponents, Hkv, D, "V")
    q = torch.randn(ns_last, Hkv, D, device="cuda").bfloat16()
    compare(q.half(), kp, vp, bt, [ns_last], [n], D ** -0.5, f"tiles of {exponents}, fp16")
    compare(q, kp, vp, bt, [ns_last], [n], D ** -0.5, f"tiles of {exponents}")


@pytest.mark.parametrize("Hkv,ns_last", [(2, 5), (2, 200), (160, 130)], ids=["cluster", "two tiles", "whole"])
@pytest.mark.parametrize("exponents", [(-3, 0, 3, -6, 2), (-40, -20, 0, None), (None, None)], ids=str)
def test_key_rows_that_grow_and_shrink_from_tile_to_tile(exponents, Hkv, ns_last):
    (kp, vp, bt), n = tiles_of_sizes(exponents, Hkv, 128, "K")
    q = torch.randn(ns_last, Hkv, 128, device="cuda").bfloat16()
    compare(q.half(), kp, vp, bt, [ns_last], [n], 0.04, f"tiles of {exponents}, fp16")
    compare(q, kp, vp, bt, [ns_last], [n], 0.04, f"tiles of {exponents}")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_rows_of_one_tile_of_mixed_sizes(dt):
    """V rows over 2^-12 .. 2^12 in one tile, and a visible row alone among larger ones that the causal mask hides."""
    ns, lens = [60, 131], [60, 400]
    kp, vp, bt = make_pools(lens, 16, 2, 128, seed=17, v_spread=12)
    slot = (bt[0, 0].long() * 16).view(1)
    row = torch.randn(1, 2, 128, device="cuda")
    pkv.reshape_and_cache_int8(row, row * 2.0 ** -14, kp, vp, slot)
    q = torch.randn(sum(ns), 4, 128, device="cuda").to(DT[dt])
    out = prefill(q, kp, vp, bt, ns, lens, 0.09)
    compare(q, kp, vp, bt, ns, lens, 0.09, "mixed rows")
    v, _ = rows_of(vp, bt[0], 1)  # the first row sees only key 0: its result is that V row, whatever comes behind it
    seen = v[0].repeat_interleave(2, 0)
    half = torch.finfo(DT[dt]).eps / 2
    assert bool(((out[0].double() - seen).abs() <= seen.abs() * (half + 2.0 ** -10) + 2.0 ** -24 + 2.0 ** -35 * 2.0 ** 15).all())


def test_every_finite_fp16_row_is_taken():
    """Rows up to fp16's largest value, 65504, in K and in V; the decode over the same pool agrees."""
    ns, lens = [40, 1], [40, 77]
    for D in (64, 128):
        kp, vp, bt = make_pools(lens, 16, 2, D, seed=19)
        for pos, where in ((3, (0,)), (20, (1,)), (39, (0, 1))):
            k, v = (torch.randn(1, 2, D, device="cuda") for _ in range(2))
            for i, x in enumerate((k, v)):
                if i in where:
                    x *= 30000 / x.abs().amax()
                    x[..., pos], x[..., pos + 1] = 65504.0, -65504.0
            pkv.reshape_and_cache_int8(k.half(), v.half(), kp, vp, (bt[0, pos // 16].long() * 16 + pos % 16).view(1))
        q = torch.randn(41, 2, D, device="cuda").half()
        compare(q, kp, vp, bt, ns, lens, 1e-4, "rows of 65504")


def test_bad_chunk_offsets_leave_the_other_chunks_alone():
    """Offsets that run backwards, with no row in two chunks: the chunk of negative length is flagged and writes nothing, the
    others' rows are what they are without it, and rows of no chunk stay as they were."""
    kp, vp, bt = make_pools([60, 30, 90], 16, 2, 64, seed=23)
    q = torch.randn(70, 4, 64, device="cuda").half()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731

    def run(offsets, lens):
        out = torch.full_like(q, 7.0)
        pkv.paged_attention_prefill_chunk_int8(out, q, kp, vp, bt[: len(lens)], i32(*lens), i32(*offsets), 40, 0.1)
        return out, pkv.get_device_error()

    for offsets, lens, rows, bad in (([0, 20, 10, 10], [60, 30, 90], [(0, 0, 20)], 1), ([20, 10, 40, 50], [60, 30, 90],
                                                                                     [(1, 10, 40), (2, 40, 50)], 0)):
        out, err = run(offsets, lens)
        assert err == pkv._binding.DEVERR_LENGTH
        written = torch.zeros(70, dtype=torch.bool, device="cuda")
        for chunk, lo, hi in rows:
            written[lo:hi] = True
            ref, bound = reference(q[lo:hi], kp, vp, bt[chunk], lens[chunk],
                                   torch.arange(lens[chunk] - (hi - lo), lens[chunk], device="cuda"), 0.1, q.dtype)
            check(out[lo:hi], ref, bound, f"offsets {offsets} chunk {chunk}")
        assert bool((out[~written] == 7.0).all())


def test_wide_tables():
    """Tables far wider than the contexts: the same rows."""
    ns, lens = [70, 3, 1], [300, 60, 1]
    kp, vp, bt = make_pools(lens, 16, 2, 128, seed=29)
    q = torch.randn(sum(ns), 8, 128, device="cuda").bfloat16()
    wide = torch.full((3, 8192), -1, dtype=torch.int32, device="cuda")
    wide[:, : bt.shape[1]] = bt
    compare(q, kp, vp, wide, ns, lens, 0.09, "table for 131072 tokens")


@pytest.mark.parametrize("Hkv", [1, 8, 30])
@pytest.mark.parametrize("cols", [129, 1000, 8192])
def test_wide_tables_with_items_of_every_length(cols, Hkv):
    """Clusters chosen for a table's width, with items from one key tile on; the same bits twice, and a
    NaN query row shows in its own row alone."""
    ns, lens = [1, 130, 3, 200, 64], [1, 130, 700, 1500, 2060]
    kp, vp, bt = make_pools(lens, 16, Hkv, 64, seed=31)
    wide = torch.full((5, max(cols, bt.shape[1])), -1, dtype=torch.int32, device="cuda")
    wide[:, : bt.shape[1]] = bt
    q = torch.randn(sum(ns), 2 * Hkv, 64, device="cuda").half()
    compare(q, kp, vp, wide, ns, lens, 0.125, f"tables of {cols}")
    out = prefill(q, kp, vp, wide, ns, lens, 0.125)
    assert torch.equal(out, prefill(q, kp, vp, wide, ns, lens, 0.125))
    q[140, 0, 5] = float("nan")
    nan = prefill(q, kp, vp, wide, ns, lens, 0.125)
    assert bool(torch.isnan(nan[140, 0]).all())
    nan[140, 0] = out[140, 0]
    assert torch.equal(nan, out)


@pytest.mark.parametrize("D,G,B", [(128, 4, 32), (64, 2, 8), (128, 1, 16)])
@pytest.mark.parametrize("ns,lens", [([9], [60]), ([140, 5], [400, 1500]), ([1, 2, 3], [1, 2, 3])])
def test_fp16_queries_round_weights_and_results_alone(ns, lens, D, G, B):
    """Large keys: a score off by 2^-11 of its terms would move the weights by more than the bound.  What is left with fp16
    queries: a weight times its V row's scale to f16 (2^-11, or 2^-25 of the largest such product), the result's half step
    (2^-11, or 2^-25), and fp32 scores: their sums, 2^-21 of the sum of the terms' magnitudes, the factor, the logarithm of
    V's scale and the exponent, 4 roundings of 2^-24 of at most 2^9, and 2e-5 for the base-2 functions."""
    kp, vp, bt = make_pools(lens, B, 2, D, seed=37, k_size=30.0)
    q = torch.randn(sum(ns), 2 * G, D, device="cuda").half()
    scale = D ** -0.5
    out = prefill(q, kp, vp, bt, ns, lens, scale)
    at = 0
    for i, (n, L) in enumerate(zip(ns, lens)):
        K, _ = rows_of(kp, bt[i], L)
        V, vs = rows_of(vp, bt[i], L)
        K, V, vs = (t.repeat_interleave(G, 1) for t in (K, V, vs))
        qd = q[at: at + n].double()
        t = torch.einsum("rhd,nhd->rhn", qd, K) * scale
        t = t.masked_fill(torch.arange(L, device="cuda")[None, None, :] > torch.arange(L - n, L, device="cuda")[:, None, None],
                          -float("inf"))
        p = torch.softmax(t, -1)
        ref, size = torch.einsum("rhn,nhd->rhd", p, V), torch.einsum("rhn,nhd->rhd", p, V.abs())
        terms = scale * torch.einsum("rhd,nhd->rhn", qd.abs(), K.abs()).amax(-1)
        ds = 2.0 ** -21 * terms + 4 * 2.0 ** -24 * 2.0 ** 9
        bound = 2.0 ** -11 * ref.abs() * (1 + 2.0 ** -10) + (2.0 ** -11 + 2e-5 + 2 * ds)[..., None] * size \
            + (L * 2.0 ** -25 * 127 * (p * vs.T[None]).amax(-1))[..., None] + 2.0 ** -25
        check(out[at: at + n], ref, bound, f"chunk {i}")
        at += n


def test_fp16_queries_take_rows_of_any_finite_size():
    """Rows beyond fp16's largest value, in K and in V, under fp16 queries: the scores' scale undoes K's size, and a V row of
    1e6 weighs little enough (or shows as an infinity, as the decode's result does)."""
    ns, lens = [20], [90]
    kp, vp, bt = make_pools(lens, 16, 2, 128, seed=41, k_size=1e7)
    q = torch.randn(20, 4, 128, device="cuda").half()
    compare(q, kp, vp, bt, ns, lens, 9e-9, "K rows of 1e7")
    kp, vp, bt = make_pools(lens, 16, 2, 128, seed=43, v_size=1e6)
    out = prefill(q, kp, vp, bt, ns, lens, 0.09)
    dec = torch.empty_like(q[:1])
    pkv.paged_attention_decode_int8(dec, q[-1:], kp, vp, bt, torch.tensor([90], dtype=torch.int32, device="cuda"), 0.09, 90)
    assert bool(torch.isinf(out).any()) and not bool(torch.isnan(out).any())
    far = dec.abs() > 60000
    assert torch.equal(torch.isinf(out[-1]) | far[0], far[0])
    assert bool(((out[-1] - dec[0]).abs()[~far[0]] <= 2.0 ** -6 * 65504).all())
