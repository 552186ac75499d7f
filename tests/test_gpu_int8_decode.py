"""Decode attention over int8 pools against plain 64-bit attention over the same codes and scales."""
import pytest
import torch

import paged_kv_cache_409_b200 as pkv
from int8_helpers import check, make_pools, reference

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def ragged(B):
    # empty, one token, block edges, a ragged tail, several partitions
    return [1, 0, B - 1, B, B + 1, 3 * B + 5, 37, 300]


def run(q, kp, vp, bt, lens, scale, part, out=None, **kw):
    out = torch.full_like(q, 7.0) if out is None else out
    cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    need = pkv.decode_workspace_size(q.shape[0], q.shape[1], q.shape[2], max(lens), part) if part else 0
    ws = torch.full((need + 16,), 255, dtype=torch.uint8, device="cuda")  # NaN
    return pkv.paged_attention_decode_int8(out, q, kp, vp, bt, cl, scale, max(lens), partition_size=part, workspace=ws, **kw)


def verify(out, q, kp, vp, bt, lens, scale, what=""):
    for i, n in enumerate(lens):
        if n == 0:
            assert bool((out[i] == 0).all()), f"{what}: empty context"
            continue
        ref, bound = reference(q[i: i + 1], kp, vp, bt[i], n, scale, q.dtype)
        check(out[i: i + 1], ref, bound, f"{what} sequence {i}, {n} tokens")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B", [8, 16, 32])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_decode(dt, G, B, D):
    lens = ragged(B)
    kp, vp, bt = make_pools(lens, B, 2, D, seed=B + G + D)
    q = torch.randn(len(lens), 2 * G, D, device="cuda").to(DT[dt])
    for part in (0, B, 3 * B, 4 * B):  # partitions of one and three blocks end inside a unit of grouped blocks
        out = run(q, kp, vp, bt, lens, D ** -0.5, part)
        assert pkv.get_device_error() == 0
        verify(out, q, kp, vp, bt, lens, D ** -0.5, f"partition {part}")


def test_one_long_sequence_is_split_by_itself():
    """The recommended partition of a batch with one long context: parts, and the result of the whole."""
    lens = [40] * 99 + [3001]
    kp, vp, bt = make_pools(lens, 16, 8, 64, seed=77)
    q = torch.randn(100, 16, 64, device="cuda").half()
    part = pkv.decode_partition_size(100, 16, 8, 64, 16, 3001, pkv.INT8, sum(lens))
    assert 0 < part < 3001 and part % 16 == 0
    cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = pkv.paged_attention_decode_int8(torch.full_like(q, 7.0), q, kp, vp, bt, cl, 0.125, 3001, total_context_tokens=sum(lens))
    assert pkv.get_device_error() == 0
    for i in (0, 98, 99):
        ref, bound = reference(q[i: i + 1], kp, vp, bt[i], lens[i], 0.125, q.dtype)
        check(out[i: i + 1], ref, bound, f"sequence {i}")


@pytest.mark.parametrize("case", [dict(v_size=1e-4), dict(v_size=1e-15), dict(v_size=3e5), dict(k_size=1e-6), dict(k_size=8.0),
                                  dict(v_spread=12), dict(v_spread=30)], ids=str)
@pytest.mark.parametrize("G", [1, 8])
def test_decode_row_scales(case, G):
    """Rows of very small, very large and very different scales (bf16 outputs have the range)."""
    lens = [200, 77, 1]
    kp, vp, bt = make_pools(lens, 16, 2, 128, seed=G, **case)
    q = torch.randn(3, 2 * G, 128, device="cuda").bfloat16()
    for part in (0, 64):
        out = run(q, kp, vp, bt, lens, 128 ** -0.5, part)
        assert pkv.get_device_error() == 0
        verify(out, q, kp, vp, bt, lens, 128 ** -0.5, str(case))


@pytest.mark.parametrize("scale", [-0.1, 0.0, 1.0])
def test_decode_score_scales(scale):
    lens = [90, 33]
    kp, vp, bt = make_pools(lens, 8, 1, 64, seed=2, k_size=0.7)
    q = torch.randn(2, 4, 64, device="cuda").half()
    verify(run(q, kp, vp, bt, lens, scale, 0), q, kp, vp, bt, lens, scale, f"scale {scale}")


def test_decode_zero_query_and_outlier_query():
    lens = [64, 100]
    kp, vp, bt = make_pools(lens, 16, 2, 128, seed=3)
    q = torch.randn(2, 4, 128, device="cuda").bfloat16()
    q[0, 1] = 0
    q[1, 2, 5] = 60.0
    verify(run(q, kp, vp, bt, lens, 0.08, 0), q, kp, vp, bt, lens, 0.08)


def test_decode_zero_rows_and_zeroed_pool():
    """Zero rows (codes 128), and a pool of zero bytes (scale 0): values 0, and they take their share of the sum."""
    lens = [40]
    kp, vp, bt = make_pools(lens, 8, 1, 64, seed=4)
    z = torch.zeros(1, 1, 64, device="cuda").half()
    slot = (bt[0, 1].long() * 8 + 3).view(1)
    pkv.reshape_and_cache_int8(z, z, kp, vp, slot)
    q = torch.randn(1, 2, 64, device="cuda").half()
    verify(run(q, kp, vp, bt, lens, 0.1, 0), q, kp, vp, bt, lens, 0.1)
    kz, vz = torch.zeros_like(kp), torch.zeros_like(vp)
    assert bool((run(q, kz, vz, bt, lens, 0.1, 0) == 0).all())  # at most 128 * 2^-80, which f16 rounds to zero
    for t in (kp, vp):  # one slot inside the context never written: zero bytes
        c, s = pkv.int8_pool_views(t)
        c[bt[0, 2].long(), 1] = 0
        s[bt[0, 2].long(), :, 1] = 0
    verify(run(q, kp, vp, bt, lens, 0.1, 0), q, kp, vp, bt, lens, 0.1)


@pytest.mark.parametrize("part", [0, 32])
def test_decode_nan_shows(part):
    """A NaN or infinity in a query row, a row of scale NaN inside the context: NaN there, and nowhere else."""
    lens = [70, 70, 70, 1]
    kp, vp, bt = make_pools(lens, 16, 2, 64, seed=5)
    q = torch.randn(4, 4, 64, device="cuda").half()
    q[0, 1, 3] = float("nan")
    q[1, 2, 0] = float("inf")
    bad = torch.full((2, 2, 64), float("nan"), device="cuda").half()
    rows = torch.ones_like(bad)
    slots = torch.stack([bt[2, 1].long() * 16 + 2, bt[3, 0].long() * 16])
    pkv.reshape_and_cache_int8(rows, bad, kp, vp, slots)  # V's rows only
    out = run(q, kp, vp, bt, lens, 0.1, part)
    want = torch.zeros(4, 4, dtype=torch.bool, device="cuda")
    want[0, 1] = want[1, 2] = True
    want[2] = want[3] = True
    assert torch.equal(torch.isnan(out).all(-1), want) and torch.equal(torch.isnan(out).any(-1), want)
    pkv.reshape_and_cache_int8(bad, rows, kp, vp, slots)  # K's rows only
    assert torch.equal(torch.isnan(run(q, kp, vp, bt, lens, 0.1, part)).all(-1), want)


def test_decode_bad_tables_are_flagged():
    lens = [100, 200, 90]
    for B in (8, 16):
        kp, vp, bt = make_pools(lens, B, 2, 128, seed=6)
        q = torch.randn(3, 4, 128, device="cuda").half()
        ref = run(q, kp, vp, bt, lens, 0.09, 0)
        assert pkv.get_device_error() == 0
        for col in (0, 1, 3):
            for bad in (kp.shape[0] + 77, -5):
                t = bt.clone()
                t[1, col] = bad
                out = run(q, kp, vp, t, lens, 0.09, 0)
                assert pkv.get_device_error() == pkv._binding.DEVERR_BLOCK_ID
                assert torch.equal(out[0], ref[0]) and torch.equal(out[2], ref[2])
    cl = torch.tensor([100, bt.shape[1] * 16 + 1, -3], dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    pkv.paged_attention_decode_int8(out, q, kp, vp, bt, cl, 0.09, 300, partition_size=0)
    assert pkv.get_device_error() & pkv._binding.DEVERR_LENGTH
    assert torch.equal(out[0], ref[0]) and bool((out[2] == 0).all())


def test_decode_long_and_automatic_partitions():
    """A long context beside short ones, with the recommended partition; and one query repeated in two rows."""
    lens = [20011, 3, 640, 20011]
    kp, vp, bt = make_pools(lens, 32, 2, 128, seed=7)
    bt[3] = bt[0]  # the same blocks twice
    q = torch.randn(4, 8, 128, device="cuda").bfloat16()
    q[3] = q[0]
    out = torch.empty_like(q)
    cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    pkv.paged_attention_decode_int8(out, q, kp, vp, bt, cl, 0.088, max(lens), total_context_tokens=sum(lens))
    assert pkv.get_device_error() == 0
    verify(out, q, kp, vp, bt, lens, 0.088)
    assert torch.equal(out[0], out[3])


@pytest.mark.parametrize("S,Hkv", [(40, 16), (256, 4), (257, 4), (129, 8)])
def test_decode_batches_taken_by_length(S, Hkv):
    """More CTAs than run at once: every sequence is taken once, whatever the lengths (all alike, one class, empty
    and bad ones among them)."""
    g = torch.Generator().manual_seed(S)
    for kind in range(3):
        lens = [torch.randint(0, 200, (S,), generator=g), torch.full((S,), 33),
                torch.where(torch.rand(S, generator=g) < 0.9, 5, 190)][kind].tolist()
        kp, vp, bt = make_pools(lens, 16, Hkv, 64, seed=kind)
        q = torch.randn(S, Hkv, 64, device="cuda").half()
        for part in (0, 48):
            out = run(q, kp, vp, bt, lens, 0.125, part)
            assert pkv.get_device_error() == 0
            verify(out, q, kp, vp, bt, lens, 0.125, f"kind {kind} partition {part}")
        cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        cl[3], cl[7] = -4, 1 << 30  # flagged: an empty row, and a length cut to the table
        bad = torch.full_like(q, 7.0)
        pkv.paged_attention_decode_int8(bad, q, kp, vp, bt, cl, 0.125, max(lens), partition_size=0)
        assert pkv.get_device_error() & pkv._binding.DEVERR_LENGTH
        keep = [i for i in range(S) if i not in (3, 7)]
        assert torch.equal(bad[keep], run(q, kp, vp, bt, lens, 0.125, 0)[keep]) and bool((bad[3] == 0).all())


def test_step_equals_append_then_decode():
    for B, D, G in ((16, 128, 4), (8, 64, 1)):
        lens = [1, B, 3 * B + 1, 150]
        kp, vp, bt = make_pools(lens, B, 2, D, seed=8)
        new = [torch.randn(4, 2, D, device="cuda").half() for _ in range(2)]
        q = torch.randn(4, 2 * G, D, device="cuda").half()
        cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        last = cl.long() - 1
        slots = bt.gather(1, (last // B)[:, None])[:, 0].long() * B + last % B
        k2, v2 = kp.clone(), vp.clone()
        pkv.reshape_and_cache_int8(*new, k2, v2, slots)
        ref = run(q, k2, v2, bt, lens, 0.1, 2 * B)
        out = torch.empty_like(q)
        pkv.paged_attention_decode_step_int8(*new, slots, out, q, kp, vp, bt, cl, 0.1, max(lens), partition_size=2 * B)
        assert pkv.get_device_error() == 0
        assert torch.equal(out, ref) and torch.equal(kp, k2) and torch.equal(vp, v2)
        verify(out, q, kp, vp, bt, lens, 0.1)
        # no new token: the decode alone
        out.zero_()
        pkv.paged_attention_decode_step_int8(new[0][:0], new[1][:0], slots[:0], out, q, kp, vp, bt, cl, 0.1, max(lens),
                                             partition_size=2 * B)
        assert torch.equal(out, ref)


def test_graph_two_streams_and_shared_inputs():
    """A captured step replayed on new contents, and two decodes at once on streams of their own."""
    lens = [130, 64, 33]
    kp, vp, bt = make_pools(lens, 16, 2, 128, seed=9)
    q = torch.randn(3, 8, 128, device="cuda").bfloat16()
    cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = torch.empty(pkv.decode_workspace_size(3, 8, 128, 130, 32), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    call = lambda o, w: pkv.paged_attention_decode_int8(o, q, kp, vp, bt, cl, 0.1, 130, partition_size=32, workspace=w)  # noqa: E731
    call(out, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out, ws)
    for seed in (10, 11):
        k2, v2, b2 = make_pools(lens, 16, 2, 128, seed=seed)
        kp.copy_(k2)
        vp.copy_(v2)
        bt.copy_(b2)
        q.copy_(torch.randn_like(q))
        graph.replay()
        torch.cuda.synchronize()
        verify(out, q, kp, vp, bt, lens, 0.1, "replayed")
    ref = out.clone()
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    torch.cuda.synchronize()
    for _ in range(5):
        for st in streams:
            with torch.cuda.stream(st):
                outs.append(call(torch.empty_like(q), torch.empty_like(ws)))
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
    # a stream given by hand, its workspace made by the call
    st, outs = torch.cuda.Stream(), []
    for _ in range(10):
        outs.append(pkv.paged_attention_decode_int8(torch.empty_like(q), q, kp, vp, bt, cl, 0.1, 130, partition_size=32,
                                                    stream=st))
        torch.full_like(ws, 255)  # memory that the call has let go of, if it came from this stream's pool
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
    assert pkv.get_device_error() == 0


def test_decode_wait_limit():
    """With the wait limit at zero the kernel gives up, flags it and leaves; restored, it is right again."""
    lens = [1024] * 24
    kp, vp, bt = make_pools(lens, 16, 8, 128, seed=12)
    q = torch.randn(24, 8, 128, device="cuda").half()
    pkv.set_wait_limit_ns(0)
    try:
        torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")  # the pools leave L2, so that waits block
        run(q, kp, vp, bt, lens, 0.1, 0)
        torch.cuda.synchronize()
        assert pkv.get_device_error() & pkv._binding.DEVERR_TIMEOUT
    finally:
        pkv.set_wait_limit_ns(pkv.DEFAULT_WAIT_LIMIT_NS)
    out = run(q, kp, vp, bt, lens, 0.1, 0)
    assert pkv.get_device_error() == 0
    verify(out, q, kp, vp, bt, lens, 0.1)
