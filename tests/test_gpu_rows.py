"""Rotary tables, norm + rotation + append, and 8-bit rows on the GPU against plain 64-bit torch.

Tolerances.  A result rounded once to a type is off by at most half a step, ``finfo.eps / 2`` of its value.
fp32 work before that: a row's sum of squares goes through at most 8 products and 7 + 5 sums in a tree (each
2^-24 of a sum of positives), so the norm's factor carries at most (13 / 2 + 4) 2^-24; two products and a
rotation (two products, a sum) follow: under 16 * 2^-24 of |a| + |b|, a and b the pair the element comes from."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_409_b200 as pkv

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
F32 = 2.0 ** -24


def frequencies(R, base, scaling="none", factor=1.0, alpha=1.0, beta=32.0, original=1):
    """theta_i, in Python floats from the definitions."""
    if scaling == "ntk":
        base = base * factor ** (R / (R - 2))
    out = []
    for i in range(R // 2):
        th = base ** (-2.0 * i / R)
        if scaling == "linear":
            th /= factor
        if scaling == "by_parts":
            g = min(1.0, max(0.0, (original * th / (2 * math.pi) - alpha) / (beta - alpha)))
            th = (1 - g) * th / factor + g * th
        out.append(th)
    return torch.tensor(out, dtype=torch.float64)


@pytest.mark.parametrize("R,n,first,kw", [
    (8, 1, 0, {}), (64, 257, 0, {}), (128, 1000, 1 << 20, {}), (96, 33, 4095, dict(scaling="linear", factor=4.0)),
    (128, 511, 7, dict(scaling="ntk", factor=8.0)), (16, 5, 0, dict(scaling="ntk", factor=2.0)),
    (128, 300, 130000, dict(scaling="by_parts", factor=8.0, alpha=1.0, beta=4.0, original_max_position=8192)),
    (256, 17, 12345, dict(scaling="by_parts", factor=32.0, original_max_position=4096, attention_factor=1.3466)),
])
def test_table(R, n, first, kw):
    buf = torch.full((n + 1, R), 7.0, device="cuda")  # a row behind the last stays as it was
    pkv.rope_table(buf[:n], base=500000.0, first_position=first, **kw)
    th = frequencies(R, 500000.0, kw.get("scaling", "none"), kw.get("factor", 1.0), kw.get("alpha", 1.0),
                     kw.get("beta", 32.0), kw.get("original_max_position", 1))
    a = torch.arange(first, first + n, dtype=torch.float64)[:, None] * th[None, :]
    ref = torch.cat([a.cos(), a.sin()], 1) * kw.get("attention_factor", 1.0)
    err = (buf[:n].cpu().double() - ref).abs()
    # half a step of fp32, and angles off by a few 2^-53 of a position's at most 2^20 radians (a and the kernel's)
    assert bool((err <= F32 * ref.abs() + 2e-9).all()), float((err - F32 * ref.abs()).max())
    assert bool((buf[n] == 7.0).all())


def reference(x, w, eps, table, pos, interleaved):
    """Normed and rotated rows in 64 bits, and |a| + |b| of each element's pair."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    size = x.abs()
    if table is None:
        return x, size
    R = table.shape[1]
    row = table.double()[pos][:, None, :]
    c, s = row[..., : R // 2], row[..., R // 2:]
    out = x.clone()
    ia = torch.arange(0, R, 2) if interleaved else torch.arange(R // 2)
    ib = ia + 1 if interleaved else ia + R // 2
    a, b = x[..., ia], x[..., ib]
    out[..., ia] = a * c - b * s
    out[..., ib] = a * s + b * c
    size[..., ia] = size[..., ib] = a.abs() + b.abs()
    return out, size


def check_quantised(x, codes, scales, what=""):
    """Scales are max |x| * (1 / 127) in fp32, codes 128 + the quotient 127 x / max |x| rounded to fp32 and then to an
    integer, ties to even: both bit for bit."""
    x = x.numpy().astype(np.float32)
    top = np.abs(x).max(-1)
    assert np.array_equal(scales, np.maximum(top * np.float32(1 / 127), np.float32(2.0 ** -80))), what
    with np.errstate(divide="ignore"):
        inv = np.minimum(127 / top.astype(np.float64), 2.0 ** 80)
    quotient = (x.astype(np.float64) * inv[..., None]).astype(np.float32)
    assert np.array_equal(codes, 128 + np.rint(quotient)), what


CASES = [
    # T, Hq, Hkv, D, R, interleaved, norm, B
    (1, 4, 1, 64, 64, False, True, 16),
    (3, 8, 8, 128, 128, False, False, 8),
    (37, 32, 8, 128, 128, False, True, 16),
    (65, 5, 1, 96, 48, True, True, 8),
    (20, 7, 2, 128, 32, False, True, 32),
    (33, 2, 2, 256, 256, True, False, 16),
    (9, 3, 3, 80, 16, False, True, 4),
    (17, 6, 2, 112, 0, False, True, 16),
    (130, 64, 8, 64, 8, True, False, 16),
    (21, 4, 2, 72, 24, True, True, 8),
    (5, 3, 1, 248, 40, False, True, 16),
]


def build(case, dtype, seed=0):
    T, Hq, Hkv, D, R, interleaved, norm, B = case
    g = torch.Generator().manual_seed(seed + T * 7 + D)
    qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g).to(dtype)
    NB = -(-T // B) + 3
    slots = torch.randperm(NB * B, generator=g)[:T]
    if T > 4:
        slots[::5] = -1
    pos = torch.randint(0, 4000, (T,), generator=g)
    table = None
    if R:
        a = torch.arange(4000, dtype=torch.float64)[:, None] * frequencies(R, 10000.0)[None, :]
        table = torch.cat([a.cos(), a.sin()], 1).float()
    qw = (1 + 0.2 * torch.randn(D, generator=g)).to(dtype) if norm else None
    kw = (1 + 0.2 * torch.randn(D, generator=g)).to(dtype) if norm else None
    return qkv, NB, slots, pos, table, qw, kw


def parts(qkv, case):
    T, Hq, Hkv, D = case[:4]
    return (qkv[:, : Hq * D].view(T, Hq, D), qkv[:, Hq * D: (Hq + Hkv) * D].view(T, Hkv, D),
            qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D))


def on_gpu(t):
    return None if t is None else t.cuda()


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=[f"T{c[0]}D{c[3]}R{c[4]}" for c in CASES])
def test_rotate_and_cache(case, dt):
    T, Hq, Hkv, D, R, interleaved, norm, B = case
    dtype = DT[dt]
    qkv, NB, slots, pos, table, qw, kw = build(case, dtype)
    q, k, v = parts(qkv, case)
    kc, vc = torch.randn(NB, B, Hkv, D).to(dtype), torch.randn(NB, B, Hkv, D).to(dtype)
    dq, dk, dv = parts(qkv.cuda(), case)  # strided slices of one tensor
    out, kd, vd = torch.empty(T, Hq, D, dtype=dtype, device="cuda"), kc.cuda(), vc.cuda()
    pkv.rope_and_cache(out, dq, dk, dv, on_gpu(table), pos.cuda(), kd, vd, slots.cuda(), interleaved=interleaved,
                       q_norm_weight=on_gpu(qw), k_norm_weight=on_gpu(kw), eps=1e-5)
    assert pkv.get_device_error() == 0
    step = torch.finfo(dtype).eps / 2

    def near(got, ref, size):
        err = (got.cpu().double() - ref).abs()
        bound = step * ref.abs() + 17 * F32 * size + (2.0 ** -25 if dtype == torch.float16 else 0.0)  # f16 subnormals
        assert bool((err <= bound).all()), float((err - bound).max())

    ref, size = reference(q, qw, 1e-5, table, pos, interleaved)
    near(out, ref, size)
    live = slots >= 0
    ref, size = reference(k, kw, 1e-5, table, pos, interleaved)
    got = kd.view(-1, Hkv, D).cpu()
    near(got[slots[live]], ref[live], size[live])
    assert torch.equal(vd.view(-1, Hkv, D).cpu()[slots[live]], v[live])
    dead = torch.ones(NB * B, dtype=torch.bool)
    dead[slots[live]] = False
    assert torch.equal(got[dead], kc.view(-1, Hkv, D)[dead])
    assert torch.equal(vd.view(-1, Hkv, D).cpu()[dead], vc.view(-1, Hkv, D)[dead])


def test_rotate_in_place_and_on_another_stream():
    case = (37, 32, 8, 128, 128, False, True, 16)
    qkv, NB, slots, pos, table, qw, kw = build(case, torch.bfloat16)
    q, k, v = (t.contiguous().cuda() for t in parts(qkv, case))
    pools = [torch.zeros(NB, 16, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    args = (table.cuda(), pos.cuda())
    kw2 = dict(q_norm_weight=qw.cuda(), k_norm_weight=kw.cuda())
    out = torch.empty_like(q)
    pkv.rope_and_cache(out, q, k, v, *args, pools[0], pools[1], slots.cuda(), **kw2)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    sl = slots.cuda()
    torch.cuda.synchronize()
    pkv.rope_and_cache(q, q, k, v, *args, pools[2], pools[3], sl, stream=st, **kw2)
    st.synchronize()
    assert torch.equal(q, out) and torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", [c for c in CASES if c[3] % 16 == 0], ids=lambda c: f"T{c[0]}D{c[3]}R{c[4]}")
def test_rotate_into_int8_pools(case, dt):
    T, Hq, Hkv, D, R, interleaved, norm, B = case
    dtype = DT[dt]
    qkv, NB, slots, pos, table, qw, kw = build(case, dtype)
    q, k, v = parts(qkv, case)
    before = torch.randint(0, 256, (NB, B, Hkv, D + 4), dtype=torch.uint8)
    dq, dk, dv = parts(qkv.cuda(), case)
    out, kd, vd = torch.empty(T, Hq, D, dtype=dtype, device="cuda"), before.cuda(), before.cuda()
    same = torch.empty_like(out)
    pools = [torch.zeros(NB, B, Hkv, D, dtype=dtype, device="cuda") for _ in range(2)]
    more = dict(interleaved=interleaved, q_norm_weight=on_gpu(qw), k_norm_weight=on_gpu(kw), eps=1e-5)
    pkv.rope_and_cache_int8(out, dq, dk, dv, on_gpu(table), pos.cuda(), kd, vd, slots.cuda(), **more)
    pkv.rope_and_cache(same, dq, dk, dv, on_gpu(table), pos.cuda(), *pools, slots.cuda(), **more)
    assert pkv.get_device_error() == 0
    assert torch.equal(out, same)
    live = slots >= 0
    at, off = slots[live] // B, slots[live] % B
    kcodes, kscales = pkv.int8_pool_views(kd.cpu())
    vcodes, vscales = pkv.int8_pool_views(vd.cpu())
    check_quantised(v[live].float(), vcodes[at, off].numpy(), vscales[at, :, off].numpy())
    ref, size = reference(k, kw, 1e-5, table, pos, interleaved)
    ref, size = ref[live], size[live]
    # the row in fp32 is within 17 * 2^-24 of its pairs' sizes; a scale within that and two roundings; a code within
    # half a step of a quotient known within 2^-24, and the read value's scale off by two roundings
    slack = 17 * F32 * size.amax(-1)
    s_ref = ref.abs().amax(-1) / 127
    s_got = kscales[at, :, off].double()
    assert bool(((s_got - s_ref).abs() <= slack / 127 + 2 * F32 * s_ref).all())
    value = (kcodes[at, off].double() - 128) * s_got[..., None]
    assert bool(((value - ref).abs() <= s_got[..., None] * (0.5 + 127 * 4 * F32) + slack[..., None]).all())
    # the rest of both pools is as it was
    for got in (kd, vd):
        codes, scales = pkv.int8_pool_views(got.cpu().clone())
        c0, s0 = pkv.int8_pool_views(before.clone())
        for c, s_ in ((codes, scales), (c0, s0)):
            c[at, off] = 0
            s_.view(torch.int32)[at, :, off] = 0
        assert torch.equal(codes, c0) and torch.equal(scales.view(torch.int32), s0.view(torch.int32))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_rotate_into_e4m3_pools_equals_rotating_first(dt):
    """fp32 rows rounded once into E4M3 are what the quantising append makes of the fp32 rotated rows."""
    case = (37, 8, 4, 128, 64, False, True, 16)
    T, Hq, Hkv, D, R, interleaved, norm, B = case
    qkv, NB, slots, pos, table, qw, kw = build(case, DT[dt])
    wide = [t.float().cuda() for t in parts(qkv, case)]
    narrow = parts(qkv.cuda(), case)
    a, b = ([torch.zeros(NB, B, Hkv, D, dtype=torch.uint8, device="cuda") for _ in range(2)] for _ in range(2))
    pools = [torch.zeros(NB, B, Hkv, D, device="cuda") for _ in range(2)]
    out = torch.empty(T, Hq, D, dtype=DT[dt], device="cuda")
    pkv.rope_and_cache_fp8(out, *narrow, table.cuda(), pos.cuda(), *a, slots.cuda(), 0.031, 0.017, q_norm_weight=qw.cuda(),
                           k_norm_weight=kw.cuda())
    pkv.rope_and_cache(torch.empty(T, Hq, D, device="cuda"), *wide, table.cuda(), pos.cuda(), *pools, slots.cuda(),
                       q_norm_weight=qw.float().cuda(), k_norm_weight=kw.float().cuda())
    live = slots[slots >= 0].cuda()
    rows = [p.view(-1, Hkv, D)[live].contiguous() for p in pools]
    pkv.reshape_and_cache_fp8(*rows, *b, live, 0.031, 0.017)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_rotate_flags_bad_positions_and_slots():
    case = (6, 4, 2, 64, 64, False, False, 8)
    qkv, NB, _, pos, table, _, _ = build(case, torch.float16)
    dq, dk, dv = parts(qkv.cuda(), case)
    slots = torch.arange(6)
    pos[1], pos[4], slots[2] = 4000, -1, NB * 8
    out = torch.full((6, 4, 64), 3.0, dtype=torch.float16, device="cuda")
    kd, vd = (torch.full((NB, 8, 2, 64), 2.0, dtype=torch.float16, device="cuda") for _ in range(2))
    pkv.rope_and_cache(out, dq, dk, dv, table.cuda(), pos.cuda(), kd, vd, slots.cuda())
    assert pkv.get_device_error() == pkv._binding.DEVERR_POSITION | pkv._binding.DEVERR_SLOT
    for t in range(6):
        skipped = t in (1, 4)
        assert bool((out[t] == 3.0).all()) == skipped
        assert bool((kd.view(-1, 2, 64)[t] == 2.0).all()) == (skipped or t == 2)
    assert bool((kd.view(-1, 2, 64)[6:] == 2.0).all())


@pytest.mark.parametrize("src", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,Hkv,D,B", [(1, 1, 64, 8), (120, 4, 64, 16), (77, 8, 128, 32), (33, 2, 256, 8), (50, 5, 112, 16),
                                       (9, 1, 16, 4)])
def test_int8_append_and_read(src, T, Hkv, D, B):
    dtype = DT[src]
    g = torch.Generator().manual_seed(T + D)
    NB = -(-T // B) + 4
    k = torch.randn(T, Hkv, D, generator=g).to(dtype)
    v = (torch.randn(T, Hkv, D, generator=g) * torch.exp2(torch.randint(-12, 12, (T, Hkv, 1), generator=g).float())).to(dtype)
    k[0, 0] = 0.0                      # a zero row
    v[-1, -1] = 0.0
    v[-1, -1, 3] = 127.0               # codes at exact ties: s = 1
    v[-1, -1, 4], v[-1, -1, 5], v[-1, -1, 6] = 2.5, -3.5, 0.5
    if T > 40:  # scales that are powers of two, and every tie: quotients of n + 1/2
        k[4:36] = ((torch.arange(32 * Hkv * D) % 254).float() / 2 - 63.25).view(32, Hkv, D).to(dtype)
        k[4:36, :, 0] = 127.0
        v[4:36] = (k[4:36].float() * 127 / 64).to(dtype)
        v[4:36, :, 0] = 127.0 * 127 / 64
    if T > 4:
        k[1, 0, 1] = float("nan")
        v[2, 0, 0] = float("inf")
        if dtype != torch.float16:
            k[3, 0] = k[3, 0] * 1e-30  # below the smallest scale
    slots = torch.randperm(NB * B, generator=g)[:T]
    if T > 4:
        slots[5::5] = -1
    pools = [torch.randint(0, 256, (NB, B, Hkv, D + 4), generator=g, dtype=torch.uint8) for _ in range(2)]
    kd, vd = pools[0].cuda(), pools[1].cuda()
    pkv.reshape_and_cache_int8(k.cuda(), v.cuda(), kd, vd, slots.cuda())
    assert pkv.get_device_error() == 0
    live = slots >= 0
    at, off = slots[live] // B, slots[live] % B
    for x, got, old in ((k, kd.cpu(), pools[0]), (v, vd.cpu(), pools[1])):
        codes, scales = pkv.int8_pool_views(got)
        rows = x[live].float()
        fine = torch.isfinite(rows).all(-1).numpy()
        check_quantised(rows[torch.from_numpy(fine)], codes[at, off].numpy()[fine], scales[at, :, off].numpy()[fine])
        assert np.isnan(scales[at, :, off].numpy()[~fine]).all()
        a, b = got.clone(), old.clone()
        for p in (a, b):
            c, s_ = pkv.int8_pool_views(p)
            c[at, off] = 0
            s_.view(torch.int32)[at, :, off] = 0
        assert torch.equal(a, b)
    # read back: once per type, a slot listed twice, skipped slots left as they were
    again = torch.cat([slots, slots[:1], torch.tensor([-1])])
    for dst in DT.values():
        ko, vo = (torch.full((T + 2, Hkv, D), 9.0, dtype=dst, device="cuda") for _ in range(2))
        pkv.read_cache_int8(ko, vo, kd, vd, again.cuda())
        assert pkv.get_device_error() == 0
        for o, got in ((ko.cpu(), kd.cpu()), (vo.cpu(), vd.cpu())):
            codes, scales = pkv.int8_pool_views(got)
            ok = again >= 0
            a, f = again[ok] // B, again[ok] % B
            ref = ((codes[a, f].float() - 128) * scales[a, :, f][..., None]).to(dst)
            assert torch.equal(torch.nan_to_num(o[ok].float(), 5.0), torch.nan_to_num(ref.float(), 5.0))
            assert bool((o[~ok] == 9.0).all())


@pytest.mark.parametrize("T,Hkv,D,B", [(4001, 20, 128, 16), (4099, 40, 64, 32), (3001, 11, 256, 8)])
def test_int8_append_of_many_rows(T, Hkv, D, B):
    """Batches and head counts at which a thread of the append takes two heads: the last ones are missing here."""
    g = torch.Generator().manual_seed(D)
    k, v = torch.randn(T, Hkv, D, generator=g).half(), torch.randn(T, Hkv, D, generator=g).half()
    NB = -(-T // B)
    slots = torch.randperm(NB * B, generator=g)[:T]
    pools = [torch.full((NB, B, Hkv, D + 4), 77, dtype=torch.uint8, device="cuda") for _ in range(2)]
    pkv.reshape_and_cache_int8(k.cuda(), v.cuda(), *pools, slots.cuda())
    assert pkv.get_device_error() == 0
    rest = torch.ones(NB * B, dtype=torch.bool)
    rest[slots] = False
    for x, got in ((k, pools[0].cpu()), (v, pools[1].cpu())):
        codes, scales = pkv.int8_pool_views(got)
        check_quantised(x.float(), codes[slots // B, slots % B].numpy(), scales[slots // B, :, slots % B].numpy())
        assert bool((codes.reshape(-1, Hkv, D)[rest] == 77).all())
    ko, vo = torch.empty(T, Hkv, D, device="cuda"), torch.empty(T, Hkv, D, device="cuda")
    pkv.read_cache_int8(ko, vo, *pools, slots.cuda())
    for o, got in ((ko, pools[0].cpu()), (vo, pools[1].cpu())):
        codes, scales = pkv.int8_pool_views(got)
        at, off = slots // B, slots % B
        assert torch.equal(o.cpu(), (codes[at, off].float() - 128) * scales[at, :, off][..., None])


def test_int8_blocks_move_whole():
    """copy_blocks and swap_blocks move an int8 pool's codes and scales together."""
    NB, B, Hkv, D = 6, 16, 2, 64
    pools = [torch.randint(0, 256, (NB, B, Hkv, D + 4), dtype=torch.uint8, device="cuda") for _ in range(2)]
    before = [p.clone() for p in pools]
    pkv.copy_blocks([pools[0]], [pools[1]], torch.tensor([[1, 4]], device="cuda"))
    host = [torch.zeros(3, B, Hkv, D + 4, dtype=torch.uint8).pin_memory() for _ in range(2)]
    pkv.swap_blocks(*pools, *host, torch.tensor([[4, 2]], device="cuda"))
    torch.cuda.synchronize()
    for p, old, h in zip(pools, before, host):
        assert torch.equal(p[4], old[1]) and torch.equal(p[1], old[1]) and torch.equal(h[2], old[1].cpu())
