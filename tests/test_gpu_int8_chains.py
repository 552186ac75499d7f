"""Calls whose kernels are dependent launches, one behind the other without a synchronisation: each sees what those before it
wrote, also behind a merge that has no row to merge."""
import pytest
import torch

import paged_kv_cache_409_b200 as pkv
from int8_helpers import make_pools

pytestmark = pytest.mark.gpu


def chained(attend, T, H, D, rounds=20):
    """`attend(q, out)` then the append of its result and its read back, over and over; the reads with and without a
    synchronisation behind every call."""
    g = torch.Generator(device="cuda").manual_seed(2)
    qs = [torch.randn(T, H, D, device="cuda", generator=g).half() for _ in range(rounds)]
    pool = [torch.zeros(-(-T // 16) + 1, 16, H, D + 4, dtype=torch.uint8, device="cuda") for _ in range(2)]
    slots = torch.randperm(T, device="cuda", generator=g)
    results = []
    for sync in (True, False):
        out, reads = torch.empty_like(qs[0]), [torch.empty(2, T, H, D, device="cuda") for _ in range(rounds)]
        torch.cuda.synchronize()
        for q, r in zip(qs, reads):
            for call in (lambda: attend(q, out), lambda: pkv.reshape_and_cache_int8(out, out, *pool, slots),
                         lambda: pkv.read_cache_int8(r[0], r[1], *pool, slots)):
                call()
                if sync:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        results.append(reads)
    assert pkv.get_device_error() == 0
    for a, b in zip(*results):
        assert torch.equal(a, b) and bool(a.abs().sum() > 0)


@pytest.mark.parametrize("kind", ["f16", "int8"])
@pytest.mark.parametrize("lens", [[16] * 300, [16, 1, 700, 15] * 20], ids=["one part each", "some in parts"])
def test_append_behind_a_decode_and_its_merge(kind, lens):
    S, Hq, Hkv, D, B = len(lens), 8, 2, 64, 16
    kp, vp, bt = make_pools(lens, B, Hkv, D, seed=1)
    bt = torch.cat([bt, bt.new_full((S, 60), -1)], 1).contiguous()
    cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if kind == "f16":
        kp, vp = (torch.randn(kp.shape[0], B, Hkv, D, device="cuda").half() for _ in range(2))
    call = pkv.paged_attention_decode if kind == "f16" else pkv.paged_attention_decode_int8
    ws = torch.empty(pkv.decode_workspace_size(S, Hq, D, 1000, 16), dtype=torch.uint8, device="cuda")
    chained(lambda q, out: call(out, q, kp, vp, bt, cl, 0.1, 1000, partition_size=16, workspace=ws), S, Hq, D)


def test_append_behind_a_multi_token_call_and_its_merge():
    R, n, Hq, Hkv, D, B = 40, 3, 8, 2, 64, 16
    lens = torch.full((R,), 30, dtype=torch.int32, device="cuda")
    NB = R * 2
    kp, vp = (torch.randn(NB, B, Hkv, D, device="cuda").half() for _ in range(2))
    bt = torch.full((R, 64), -1, dtype=torch.int32, device="cuda")
    bt[:, :2] = torch.randperm(NB, device="cuda").view(R, 2).to(torch.int32)
    qsl = torch.arange(0, R * n + 1, n, dtype=torch.int32, device="cuda")
    chained(lambda q, out: pkv.paged_attention_decode_multi(out, q, kp, vp, bt, lens, qsl, n, 1000, 0.1, partition_size=64), R * n,
            Hq, D)


def test_a_step_that_checked_mode_refuses_has_changed_nothing():
    """PKV_CHECK=1: a step with a bad table, or a bad length, writes no row of its new tokens."""
    import os
    import subprocess
    import sys

    code = """
import torch, paged_kv_cache_409_b200 as pkv
i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device='cuda')
B, H, D = 16, 2, 128
bt = i32(0, 1, 2, 3).view(2, 2)
bad = i32(0, 1, 2, 4).view(2, 2)
slots = torch.tensor([3, 35], device='cuda')
q = torch.randn(2, 4, D, device='cuda').half()
k = torch.randn(2, H, D, device='cuda').half()
pools = {'f16': lambda: torch.zeros(4, B, H, D, dtype=torch.half, device='cuda'),
         'fp8': lambda: torch.zeros(4, B, H, D, dtype=torch.uint8, device='cuda'),
         'int8': lambda: torch.zeros(4, B, H, D + 4, dtype=torch.uint8, device='cuda')}
for kind, make in pools.items():
    kp, vp = make(), make()
    call = {'f16': pkv.paged_attention_decode_step, 'fp8': pkv.paged_attention_decode_step_fp8,
            'int8': pkv.paged_attention_decode_step_int8}[kind]
    scales = (0.1, 0.1) if kind == 'fp8' else ()
    for tables, lens in ((bad, i32(20, 20)), (bt, i32(20, 33)), (bt, i32(-1, 20))):
        try:
            call(k, k, slots, torch.empty_like(q), q, kp, vp, tables, lens, 0.1, *scales, 32)
            raise SystemExit(kind + ' was not refused')
        except pkv.PagedKVError as e:
            assert e.status == -3, e
        torch.cuda.synchronize()
        assert not kp.any() and not vp.any(), kind
    call(k, k, slots, torch.empty_like(q), q, kp, vp, bt, i32(20, 20), 0.1, *scales, 32)
    torch.cuda.synchronize()
    assert kp.any() and vp.any()
print('refused')
"""
    env = dict(os.environ, PKV_CHECK="1", PYTHONPATH=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=200)
    assert r.returncode == 0 and "refused" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
def test_a_captured_step_replays_on_new_inputs(dt):
    """Rotation and append, prefill of the chunks, a decode step and the rows read back, captured in one graph (the chunks of few
    items take clusters), replayed on other inputs: the bits of the same calls one by one."""
    B, Hq, H, D = 16, 8, 2, 128
    ns, lens = [40, 3], [700, 130]
    g = torch.Generator(device="cuda").manual_seed(5)
    kp, vp, bt = make_pools([n + 1 for n in lens], B, H, D, seed=3)
    start = [kp.clone(), vp.clone()]
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    sl, qsl, cl = i32(*lens), i32(0, 40, 43), i32(*[n + 1 for n in lens])
    pos = torch.cat([torch.arange(L - n, L, device="cuda") for n, L in zip(ns, lens)])
    seq = torch.repeat_interleave(torch.arange(2, device="cuda"), torch.tensor(ns, device="cuda"))
    slots = bt[seq, pos // B].long() * B + pos % B
    last = torch.tensor(lens, device="cuda")
    new_slots = bt[torch.arange(2, device="cuda"), last // B].long() * B + last % B
    table = torch.empty(1024, 64, device="cuda")
    pkv.rope_table(table)
    q, k, v = (torch.zeros(43, h, D, dtype=dt, device="cuda") for h in (Hq, H, H))
    q1, k1, v1 = (torch.zeros(2, h, D, dtype=dt, device="cuda") for h in (Hq, H, H))
    qr, out, out1 = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q1)
    rows = [torch.empty(43, H, D, device="cuda") for _ in range(2)]

    def step():
        pkv.rope_and_cache_int8(qr, q, k, v, table, pos, kp, vp, slots)
        pkv.paged_attention_prefill_chunk_int8(out, qr, kp, vp, bt, sl, qsl, 40, 0.09)
        pkv.paged_attention_decode_step_int8(k1, v1, new_slots, out1, q1, kp, vp, bt, cl, 0.09, max(lens) + 1,
                                             total_context_tokens=sum(lens) + 2)
        pkv.read_cache_int8(*rows, kp, vp, slots)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in (q, k, v, q1, k1, v1):
            t.copy_(torch.randn(t.shape, device="cuda", generator=g))
        results = []
        for call in (step, graph.replay):
            kp.copy_(start[0])
            vp.copy_(start[1])
            for t in (qr, out, out1, *rows):
                t.fill_(7.0)
            call()
            torch.cuda.synchronize()
            results.append([t.clone() for t in (qr, out, out1, *rows, kp, vp)])
        for a, b in zip(*results):
            assert torch.equal(a, b)
        assert bool(torch.isfinite(results[0][1]).all()) and bool(torch.isfinite(results[0][2]).all())
    assert pkv.get_device_error() == 0
