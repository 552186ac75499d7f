"""Chunked prefill over int8 pools against plain 64-bit attention over the same codes and scales, and a serving run
of the row calls together: table, rotation and append, prefill, decode steps."""
import pytest
import torch

import paged_kv_cache_409_b200 as pkv
from int8_helpers import check, make_pools, reference

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def starts(ns):
    return torch.tensor([0] + list(ns), device="cuda").cumsum(0).to(torch.int32)


def run(q, kp, vp, bt, ns, lens, scale, max_n=None, out=None, **kw):
    out = torch.full_like(q, 7.0) if out is None else out
    return pkv.paged_attention_prefill_chunk_int8(out, q, kp, vp, bt, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                                  starts(ns), max_n or max(ns), scale, **kw)


def verify(out, q, kp, vp, bt, ns, lens, scale, what="", only=None):
    at = 0
    for i, (n, L) in enumerate(zip(ns, lens)):
        if n and (only is None or i in only):
            first = torch.arange(L - n, L, device="cuda")
            ref, bound = reference(q[at: at + n], kp, vp, bt[i], L, scale, q.dtype, first=first)
            check(out[at: at + n], ref, bound, f"{what} chunk {i}")
        at += n


CASES = [
    # dt, D, B, Hq, Hkv, cached before, new
    ("bf16", 128, 32, 32, 8, [0, 300], [512, 77]),
    ("f16", 128, 16, 8, 8, [5, 0, 129], [1, 130, 128]),
    ("bf16", 64, 8, 16, 2, [1000, 0], [33, 257]),
    ("f16", 64, 16, 4, 2, [17], [300]),
    ("bf16", 128, 16, 16, 2, [255, 64], [200, 16]),
    ("f16", 128, 8, 4, 1, [0, 127, 1, 0], [1, 1, 0, 2]),
    ("bf16", 128, 32, 2, 2, [640], [384]),
    ("f16", 64, 32, 8, 1, [4000, 3], [6, 5]),
]


@pytest.mark.parametrize("case", CASES, ids=[f"case{i}" for i in range(len(CASES))])
def test_prefill(case):
    dt, D, B, Hq, Hkv, c0, ns = case
    lens = [a + b for a, b in zip(c0, ns)]
    kp, vp, bt = make_pools(lens, B, Hkv, D, seed=D + B)
    q = torch.randn(sum(ns) + 3, Hq, D, device="cuda").to(DT[dt])  # three rows behind the last chunk
    out = run(q, kp, vp, bt, ns, lens, D ** -0.5)
    assert pkv.get_device_error() == 0
    verify(out, q, kp, vp, bt, ns, lens, D ** -0.5)
    assert bool((out[sum(ns):] == 7.0).all())


@pytest.mark.parametrize("case", [
    # chunks of few rows over long contexts: clusters of 2, 4 and 8 CTAs share the key tiles
    ("bf16", 128, 32, 8, 2, [5000], [3]),            # 2 items: 8 parts of 5 tiles
    ("f16", 64, 8, 8, 8, [900, 900, 20], [4, 1, 6]),  # 24 items
    ("bf16", 128, 16, 32, 8, [3000, 11], [70, 1]),   # parts without a visible key for the short chunk
    ("f16", 128, 16, 16, 8, [2000] * 5, [2, 3, 4, 5, 6]),
    ("bf16", 64, 16, 4, 1, [0], [1]),
    ("f16", 128, 8, 8, 1, [1920], [128]),            # the query tiles end on different key tiles
    ("bf16", 128, 32, 8, 2, [4096, 0], [1, 700]),
], ids=lambda c: f"{c[0]}D{c[1]}n{c[6][0]}")
def test_prefill_few_items(case):
    dt, D, B, Hq, Hkv, c0, ns = case
    lens = [a + b for a, b in zip(c0, ns)]
    kp, vp, bt = make_pools(lens, B, Hkv, D, seed=D + B + Hq)
    q = torch.randn(sum(ns) + 1, Hq, D, device="cuda").to(DT[dt])
    out = run(q, kp, vp, bt, ns, lens, D ** -0.5)
    assert pkv.get_device_error() == 0
    verify(out, q, kp, vp, bt, ns, lens, D ** -0.5)
    assert bool((out[sum(ns):] == 7.0).all())
    # the same rows with a NaN query row and a NaN key row, seen by the last row alone
    q[0, 0, 0] = float("nan")
    nan = torch.full((1, Hkv, D), float("nan"), device="cuda")
    last = lens[0] - 1
    pkv.reshape_and_cache_int8(nan, torch.ones_like(nan), kp, vp, (bt[0, last // B].long() * B + last % B).view(1))
    bad = run(q, kp, vp, bt, ns, lens, D ** -0.5)
    want = torch.zeros(sum(ns), Hq, dtype=torch.bool, device="cuda")
    want[0, 0] = True
    want[ns[0] - 1] = True
    assert torch.equal(torch.isnan(bad[: sum(ns)]).all(-1), want) and torch.equal(torch.isnan(bad[: sum(ns)]).any(-1), want)
    assert torch.equal(bad[: sum(ns)][~want], out[: sum(ns)][~want])


@pytest.mark.parametrize("G,D", [(1, 64), (2, 128)])
@pytest.mark.parametrize("Hkv", [12, 16, 24, 30, 40, 60])
def test_prefill_clusters_of_every_size(Hkv, G, D):
    """Head counts that give clusters of 8, 6, 5, 4, 3 and 2 CTAs: shares of the key tiles and of the merged rows that
    do not divide evenly."""
    lens, ns = [2531], [101]
    kp, vp, bt = make_pools(lens, 16, Hkv, D, seed=Hkv)
    q = torch.randn(sum(ns), Hkv * G, D, device="cuda").half()
    out = run(q, kp, vp, bt, ns, lens, D ** -0.5)
    assert pkv.get_device_error() == 0
    verify(out, q, kp, vp, bt, ns, lens, D ** -0.5, f"{Hkv} heads")
    assert torch.equal(out, run(q, kp, vp, bt, ns, lens, D ** -0.5))


def test_prefill_few_items_bad_tables_and_wait_limit():
    ns, lens = [5, 2], [3000, 2500]
    kp, vp, bt = make_pools(lens, 16, 2, 128, seed=9)
    q = torch.randn(7, 4, 128, device="cuda").half()
    ref = run(q, kp, vp, bt, ns, lens, 0.1)
    # ids of the first and last tiles of the cluster's CTAs, which read a tile ahead
    for col, bad in ((0, -7), (16, kp.shape[0]), (24, 2**31 - 1), (100, -7), (161, 2**31 - 1), (187, kp.shape[0] + 5)):
        t = bt.clone()
        t[0, col] = bad
        out = run(q, kp, vp, t, ns, lens, 0.1)
        assert pkv.get_device_error() == pkv._binding.DEVERR_BLOCK_ID
        assert torch.equal(out[5:], ref[5:])
    pkv.set_wait_limit_ns(0)
    try:
        out = run(q, kp, vp, bt, ns, lens, 0.1)
        torch.cuda.synchronize()
        assert pkv.get_device_error() & pkv._binding.DEVERR_TIMEOUT
    finally:
        pkv.set_wait_limit_ns(pkv.DEFAULT_WAIT_LIMIT_NS)
    assert torch.equal(run(q, kp, vp, bt, ns, lens, 0.1), ref) and pkv.get_device_error() == 0


def test_prefill_many_chunks():
    """More chunks than the longest-first order takes (64), of different lengths, a bound above the longest."""
    ns = [(5 * i) % 7 for i in range(70)]
    lens = [n + (37 * i) % 300 for i, n in enumerate(ns)]
    kp, vp, bt = make_pools(lens, 16, 2, 64, seed=1)
    q = torch.randn(sum(ns), 4, 64, device="cuda").half()
    out = run(q, kp, vp, bt, ns, lens, 0.125, max_n=200)
    assert pkv.get_device_error() == 0
    verify(out, q, kp, vp, bt, ns, lens, 0.125)


@pytest.mark.parametrize("kw", [dict(v_size=1e-3), dict(v_size=200.0), dict(k_size=6.0), dict(v_spread=5)], ids=str)
def test_prefill_row_scales(kw):
    ns, lens = [140, 9], [333, 9]
    kp, vp, bt = make_pools(lens, 8, 2, 128, seed=2, **kw)
    q = torch.randn(149, 8, 128, device="cuda").bfloat16()
    for scale in (0.088, -0.05, 0.0):
        verify(run(q, kp, vp, bt, ns, lens, scale), q, kp, vp, bt, ns, lens, scale, str(kw))


def test_prefill_nan_rows_show_where_they_are_seen():
    """A K or V row of scale NaN, or beyond f16, reaches the rows at or behind its position and no other; a NaN query
    row reaches itself."""
    ns, lens = [150, 40], [190, 90]
    kp, vp, bt = make_pools(lens, 16, 2, 64, seed=3)
    q = torch.randn(190, 4, 64, device="cuda").bfloat16()
    ref = run(q, kp, vp, bt, ns, lens, 0.1)
    good = torch.ones(1, 2, 64, device="cuda")
    slot = (bt[0, 5].long() * 16 + 4).view(1)  # position 84: row 44 of chunk 0
    for bad in (torch.full_like(good, float("nan")), torch.full_like(good, 1e6)):
        for which in (0, 1):
            k2, v2 = kp.clone(), vp.clone()
            pkv.reshape_and_cache_int8(bad if which == 0 else good, bad if which == 1 else good, k2, v2, slot)
            out = run(q, k2, v2, bt, ns, lens, 0.1)
            assert bool(torch.isnan(out[44:150]).all())
            assert torch.equal(out[:44], ref[:44]) and torch.equal(out[150:], ref[150:])
    q[160, 1, 3] = float("nan")
    out = run(q, kp, vp, bt, ns, lens, 0.1)
    nan = torch.zeros(190, 4, dtype=torch.bool, device="cuda")
    nan[160, 1] = True
    assert torch.equal(torch.isnan(out).all(-1), nan) and torch.equal(torch.isnan(out).any(-1), nan)
    assert torch.equal(out[~nan], ref[~nan])


def test_prefill_bad_tables_are_flagged():
    ns, lens = [64, 30, 50], [200, 30, 180]
    kp, vp, bt = make_pools(lens, 16, 2, 128, seed=4)
    q = torch.randn(144, 4, 128, device="cuda").half()
    ref = run(q, kp, vp, bt, ns, lens, 0.1)
    assert pkv.get_device_error() == 0
    for col, bad in ((0, -1), (7, kp.shape[0]), (12, 1 << 30)):
        t = bt.clone()
        t[0, col] = bad
        out = run(q, kp, vp, t, ns, lens, 0.1)
        assert pkv.get_device_error() == pkv._binding.DEVERR_BLOCK_ID
        assert torch.equal(out[64:], ref[64:])
    for wrong in ([200, 20, 180], [200, 30, bt.shape[1] * 16 + 1]):  # shorter than its chunk; beyond the table
        out = run(q, kp, vp, bt, ns, wrong, 0.1)
        assert pkv.get_device_error() == pkv._binding.DEVERR_LENGTH
        assert torch.equal(out[:64], ref[:64])


def test_prefill_bad_chunk_offsets_are_flagged():
    """Offsets that leave the packed query, run backwards or start below it: the chunk is skipped, the others stay."""
    ns, lens = [20, 30, 10], [60, 30, 90]
    kp, vp, bt = make_pools(lens, 16, 2, 64, seed=11)
    q = torch.randn(60, 4, 64, device="cuda").half()
    ref = run(q, kp, vp, bt, ns, lens, 0.1)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for offsets, kept in (([0, 20, 50, 61], slice(0, 50)), ([-1, 20, 50, 60], slice(20, 60)), ([0, 20, 10, 20], slice(0, 20))):
        out = torch.full_like(q, 7.0)
        pkv.paged_attention_prefill_chunk_int8(out, q, kp, vp, bt, sl, torch.tensor(offsets, dtype=torch.int32, device="cuda"),
                                               32, 0.1)
        assert pkv.get_device_error() == pkv._binding.DEVERR_LENGTH
        if offsets != [0, 20, 10, 20]:
            assert torch.equal(out[kept], ref[kept])
            rest = torch.ones(60, dtype=torch.bool, device="cuda")
            rest[kept] = False
            assert bool((out[rest] == 7.0).all())


def test_prefill_row_of_one_equals_decode_closely_and_repeats():
    """Chunks of one row are decode; the same call twice gives the same bits, on two streams at once too."""
    lens = [513, 100, 1]
    kp, vp, bt = make_pools(lens, 32, 2, 128, seed=5)
    q = torch.randn(3, 16, 128, device="cuda").half()
    a = run(q, kp, vp, bt, [1, 1, 1], lens, 0.09)
    verify(a, q, kp, vp, bt, [1, 1, 1], lens, 0.09)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        for st in streams:
            with torch.cuda.stream(st):
                outs.append(run(q, kp, vp, bt, [1, 1, 1], lens, 0.09))
    torch.cuda.synchronize()
    assert all(torch.equal(o, a) for o in outs)


def test_prefill_wait_limit():
    ns, lens = [256] * 4, [4096] * 4
    kp, vp, bt = make_pools(lens, 16, 2, 128, seed=6)
    q = torch.randn(1024, 8, 128, device="cuda").bfloat16()
    pkv.set_wait_limit_ns(0)
    try:
        run(q, kp, vp, bt, ns, lens, 0.1)
        torch.cuda.synchronize()
        assert pkv.get_device_error() & pkv._binding.DEVERR_TIMEOUT
    finally:
        pkv.set_wait_limit_ns(pkv.DEFAULT_WAIT_LIMIT_NS)
    out = run(q, kp, vp, bt, ns, lens, 0.1)
    assert pkv.get_device_error() == 0
    verify(out, q, kp, vp, bt, ns, lens, 0.1, only=[0, 3])


def test_serving_run():
    """Two sequences through one layer: rotary table, chunked prompts (rotation and append, then prefill), and decode
    steps in a captured graph, against 64-bit attention over the rows as they were rotated and quantised."""
    B, Hq, Hkv, D, R = 16, 8, 2, 128, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    table = torch.empty(2048, R, device="cuda")
    pkv.rope_table(table, base=10000.0, scaling="by_parts", factor=4.0, original_max_position=512, beta=8.0)
    NB = 64
    perm = torch.randperm(NB, device="cuda", generator=g).to(torch.int32)
    bt = perm.view(2, 32).contiguous()
    kp, vp = (torch.zeros(NB, B, Hkv, D + 4, dtype=torch.uint8, device="cuda") for _ in range(2))
    kw = dict(q_norm_weight=torch.ones(D, device="cuda").half(), k_norm_weight=torch.ones(D, device="cuda").half())
    lens = [0, 0]

    def project(n):
        x = torch.randn(n, (Hq + 2 * Hkv) * D, device="cuda", generator=g).half()
        return (x[:, : Hq * D].view(n, Hq, D), x[:, Hq * D: (Hq + Hkv) * D].view(n, Hkv, D),
                x[:, (Hq + Hkv) * D:].view(n, Hkv, D))

    for ns in ([130, 7], [60, 200]):
        seq = torch.repeat_interleave(torch.arange(2, device="cuda"), torch.tensor(ns, device="cuda"))
        pos = torch.cat([torch.arange(c, c + n, device="cuda") for c, n in zip(lens, ns)])
        slots = bt[seq, pos // B].long() * B + pos % B
        q, k, v = project(sum(ns))
        qr = torch.empty(sum(ns), Hq, D, dtype=torch.half, device="cuda")
        pkv.rope_and_cache_int8(qr, q, k, v, table, pos, kp, vp, slots, **kw)
        lens = [c + n for c, n in zip(lens, ns)]
        out = run(qr, kp, vp, bt, ns, lens, D ** -0.5)
        verify(out, qr, kp, vp, bt, ns, lens, D ** -0.5)
    q, k, v = (t.contiguous() for t in project(2))
    qr, out = torch.empty_like(q), torch.empty_like(q)
    pos = torch.tensor(lens, device="cuda")
    slots, cl = torch.empty_like(pos), torch.empty(2, dtype=torch.int32, device="cuda")

    def step():
        slots.copy_(bt.gather(1, (pos // B)[:, None])[:, 0].long() * B + pos % B)
        cl.copy_(pos + 1)
        pkv.rope_and_cache_int8(qr, q, k, v, table, pos, kp, vp, slots, **kw)
        pkv.paged_attention_decode_int8(out, qr, kp, vp, bt, cl, D ** -0.5, 512, partition_size=0)
        pos.add_(1)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(20):
        for t, new in zip((q, k, v), project(2)):
            t.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        for i, n in enumerate(pos.tolist()):
            ref, bound = reference(qr[i: i + 1], kp, vp, bt[i], n, D ** -0.5, torch.half)
            check(out[i: i + 1], ref, bound, f"step at {n}")
    assert pkv.get_device_error() == 0


def test_pools_beyond_four_gib():
    """Blocks whose bytes lie past 2^32: append, rotation, read, decode and prefill."""
    NB, B, Hkv, D = 262_000, 16, 8, 128  # 4.4 GB a pool
    kp, vp = (torch.empty(NB, B, Hkv, D + 4, dtype=torch.uint8, device="cuda") for _ in range(2))
    L, n = 200, 40
    ids = torch.arange(NB - 14, NB - 1, device="cuda").flip(0)
    bt = ids.to(torch.int32).view(1, -1).contiguous()
    pos = torch.arange(L, device="cuda")
    slots = ids[pos // B] * B + pos % B
    k, v = (torch.randn(L, Hkv, D, device="cuda").half() for _ in range(2))
    pkv.reshape_and_cache_int8(k[:150], v[:150], kp, vp, slots[:150])
    q = torch.randn(n, 16, D, device="cuda").half()
    out = torch.empty(50, 16, D, dtype=torch.half, device="cuda")
    pkv.rope_and_cache_int8(out, torch.cat([q, q[:10]]), k[150:], v[150:], None, None, kp, vp, slots[150:])
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    pkv.read_cache_int8(ko, vo, kp, vp, slots)
    for x, y in ((k, ko), (v, vo)):
        assert bool(((x.float() - y.float()).abs() <= x.float().abs().amax(-1, keepdim=True) * (0.51 / 127 + 2.0 ** -10)).all())
    verify(run(q, kp, vp, bt, [n], [L], 0.09), q, kp, vp, bt, [n], [L], 0.09)
    dec = torch.empty_like(q[:1])
    cl = torch.tensor([L], dtype=torch.int32, device="cuda")
    pkv.paged_attention_decode_int8(dec, q[:1], kp, vp, bt, cl, 0.09, L, partition_size=64)
    check(dec, *reference(q[:1], kp, vp, bt[0], L, 0.09, torch.half))
    assert pkv.get_device_error() == 0


def test_checked_mode_refuses_bad_tables():
    """PKV_CHECK=1: the host reads the tables first and launches nothing when one is out of range."""
    import os
    import subprocess
    import sys

    code = """
import torch, paged_kv_cache_409_b200 as pkv
from int8_helpers import make_pools
kp, vp, bt = make_pools([40, 20], 8, 2, 64, seed=1)
q = torch.zeros(2, 4, 64, device='cuda').half()
i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device='cuda')
i64 = lambda *x: torch.tensor(x, device='cuda')
k = torch.zeros(2, 2, 64, device='cuda').half()
table = torch.zeros(50, 32, device='cuda')
bad = bt.clone()
bad[1, 0] = kp.shape[0]
good = [lambda: pkv.paged_attention_decode_int8(q, q, kp, vp, bt, i32(40, 20), 0.1, 40),
        lambda: pkv.paged_attention_prefill_chunk_int8(q, q, kp, vp, bt, i32(40, 20), i32(0, 1, 2), 1, 0.1),
        lambda: pkv.reshape_and_cache_int8(k, k, kp, vp, i64(3, -1)), lambda: pkv.read_cache_int8(k, k, kp, vp, i64(3, -1)),
        lambda: pkv.rope_and_cache_int8(q, q, k, k, table, i64(0, 49), kp, vp, i64(3, 4))]
wrong = [lambda: pkv.paged_attention_decode_int8(q, q, kp, vp, bad, i32(40, 20), 0.1, 40),
         lambda: pkv.paged_attention_decode_int8(q, q, kp, vp, bt, i32(41, 20), 0.1, 40),
         lambda: pkv.paged_attention_prefill_chunk_int8(q, q, kp, vp, bad, i32(40, 20), i32(0, 1, 2), 1, 0.1),
         lambda: pkv.paged_attention_prefill_chunk_int8(q, q, kp, vp, bt, i32(40, 20), i32(0, 1, 3), 2, 0.1),
         lambda: pkv.reshape_and_cache_int8(k, k, kp, vp, i64(3, kp.shape[0] * 8)),
         lambda: pkv.read_cache_int8(k, k, kp, vp, i64(3, kp.shape[0] * 8)),
         lambda: pkv.rope_and_cache_int8(q, q, k, k, table, i64(0, 50), kp, vp, i64(3, 4)),
         lambda: pkv.rope_and_cache_int8(q, q, k, k, table, i64(0, 1), kp, vp, i64(3, kp.shape[0] * 8))]
for f in good:
    f()
for n, f in enumerate(wrong):
    try:
        f()
        raise SystemExit(f'call {n} was not refused')
    except pkv.PagedKVError as e:
        assert e.status == -3, (n, e.status)
assert pkv.get_device_error() == 0
print('refused')
"""
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PKV_CHECK="1", PYTHONPATH=os.pathsep.join([here, os.path.dirname(here)]))
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=200)
    assert r.returncode == 0 and "refused" in r.stdout, r.stdout + r.stderr
