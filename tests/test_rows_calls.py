"""The row calls without a GPU: arguments in their places, refusals before any launch, a scale of frequencies."""
import ctypes

import pytest
import torch

import paged_kv_cache_409_b200 as pkv
from paged_kv_cache_409_b200 import _binding
from test_binding_marshalling import f32, mock  # noqa: F401

EINVAL, EUNSUPPORTED = -1, -2


def test_rope_arguments(mock):  # noqa: F811
    T, Hq, Hkv, D, B, NB, R = 5, 8, 2, 64, 16, 7, 32
    qkv = torch.zeros(T, (Hq + 2 * Hkv) * D, dtype=torch.bfloat16)
    q, k, v = (qkv[:, : Hq * D].view(T, Hq, D), qkv[:, Hq * D: (Hq + Hkv) * D].view(T, Hkv, D),
               qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D))
    out = torch.zeros(T, Hq, D, dtype=torch.bfloat16)
    table, pos, slots = torch.zeros(99, R), torch.zeros(T, dtype=torch.int64), torch.zeros(T, dtype=torch.int64)
    w = torch.zeros(D, dtype=torch.bfloat16)
    kc, vc = torch.zeros(NB, B, Hkv, D, dtype=torch.bfloat16), torch.zeros(NB, B, Hkv, D, dtype=torch.bfloat16)
    pkv.rope_and_cache(out, q, k, v, table, pos, kc, vc, slots, interleaved=True, q_norm_weight=w, eps=0.25, stream=3)
    name, a = mock.last()
    want = {"query_out": out.data_ptr(), "query": q.data_ptr(), "key": k.data_ptr(), "value": v.data_ptr(),
            "query_stride": 768, "key_stride": 768, "value_stride": 768, "q_norm_weight": w.data_ptr(),
            "k_norm_weight": 0, "eps": 0.25, "cos_sin": table.data_ptr(), "max_position": 99, "rotary_dim": R,
            "interleaved": 1, "positions": pos.data_ptr(), "key_cache": kc.data_ptr(), "value_cache": vc.data_ptr(),
            "slot_mapping": slots.data_ptr(), "num_tokens": T, "num_q_heads": Hq, "num_kv_heads": Hkv, "head_dim": D,
            "block_size": B, "num_blocks": NB, "dtype": 2, "stream": 3}
    assert name == "pkv_rope_and_cache" and a == want
    p8 = [torch.zeros(NB, B, Hkv, D, dtype=torch.uint8) for _ in range(2)]
    pkv.rope_and_cache_fp8(out, q, k, v, None, None, *p8, slots, 0.1, 0.2, k_norm_weight=w, stream=3)
    name, a = mock.last()
    assert name == "pkv_rope_and_cache_fp8"
    assert a == {**want, "q_norm_weight": 0, "k_norm_weight": w.data_ptr(), "eps": f32(1e-6), "cos_sin": 0,
                 "max_position": 0, "rotary_dim": 0, "interleaved": 0, "positions": 0, "key_cache": p8[0].data_ptr(),
                 "value_cache": p8[1].data_ptr(), "k_scale": f32(0.1), "v_scale": f32(0.2)}
    pi = [torch.zeros(NB, B, Hkv, D + 4, dtype=torch.uint8) for _ in range(2)]
    pkv.rope_and_cache_int8(out[:1], q[:1], k[:1], v[:1], table, pos[:1], *pi, slots[:1], stream=3)
    name, a = mock.last()
    assert name == "pkv_rope_and_cache_int8"
    assert (a["query_stride"], a["key_stride"], a["num_tokens"], a["head_dim"], a["num_blocks"]) == (512, 128, 1, D, NB)
    pkv.reshape_and_cache_int8(k.contiguous(), v.contiguous(), *pi, slots, stream=3)
    name, a = mock.last()
    assert name == "pkv_reshape_and_cache_int8"
    assert (a["key_cache"], a["value_cache"], a["num_tokens"], a["num_kv_heads"], a["head_dim"], a["block_size"],
            a["num_blocks"], a["src_dtype"]) == (pi[0].data_ptr(), pi[1].data_ptr(), T, Hkv, D, B, NB, 2)
    ko, vo = torch.zeros(T, Hkv, D), torch.zeros(T, Hkv, D)
    pkv.read_cache_int8(ko, vo, *pi, slots, stream=3)
    name, a = mock.last()
    assert name == "pkv_read_cache_int8" and a["dst_dtype"] == 0 and a["key_out"] == ko.data_ptr()
    pkv.rope_table(table, first_position=12, stream=3)
    name, a = mock.last()
    assert name == "pkv_rope_table" and (a["cos_sin"], a["first_position"], a["num_positions"]) == (table.data_ptr(), 12, 99)
    assert pkv.int8_block_bytes(16, 2, 64) == 0  # the stand-in's answer
    assert mock.last() == ("pkv_int8_block_bytes", {"block_size": 16, "num_kv_heads": 2, "head_dim": 64})


def test_binding_refuses_what_does_not_fit_together(mock):  # noqa: F811
    T, Hq, Hkv, D = 3, 4, 2, 64
    q, k = torch.zeros(T, Hq, D), torch.zeros(T, Hkv, D)
    pool, table = torch.zeros(4, 8, Hkv, D), torch.zeros(9, 32)
    i = torch.zeros(T, dtype=torch.int64)

    def call(**kw):
        a = dict(query_out=q, query=q, key=k, value=k, cos_sin=table, positions=i, key_cache=pool, value_cache=pool,
                 slot_mapping=i)
        a.update(kw)
        pkv.rope_and_cache(**a)

    call()
    for bad in (dict(key=k[:2]), dict(value=torch.zeros(T, Hkv, 32)), dict(query_out=q.half()), dict(key=k.half()),
                dict(cos_sin=table.double()), dict(positions=i.int()), dict(positions=None), dict(slot_mapping=i[:2]),
                dict(q_norm_weight=torch.zeros(32)), dict(k_norm_weight=torch.zeros(D).half()),
                dict(key_cache=pool.half()), dict(value_cache=pool[:2]), dict(key=torch.zeros(T, D, Hkv).transpose(1, 2))):
        with pytest.raises(ValueError):
            call(**bad)
    u8 = torch.zeros(4, 8, Hkv, D + 4, dtype=torch.uint8)
    with pytest.raises(ValueError):
        pkv.reshape_and_cache_int8(k, k, u8, u8[:2], i)
    with pytest.raises(ValueError):
        pkv.reshape_and_cache_int8(k, k, u8.int(), u8, i)
    with pytest.raises(ValueError):
        pkv.reshape_and_cache_int8(k, k[:2], u8, u8, i)
    with pytest.raises(ValueError):
        pkv.read_cache_int8(k, k.half(), u8, u8, i)
    with pytest.raises(ValueError):
        pkv.rope_table(table, scaling="other")
    with pytest.raises(ValueError):
        pkv.rope_table(table.double())


def test_host_refusals():
    """Statuses of the C calls for arguments they refuse; every pointer is made up and never read."""
    from paged_kv_cache_409_b200 import build
    build.build()
    lib = pkv.load_library()
    P = 1 << 20

    def rope(fn, *tail, **kw):
        a = dict(query_out=P, query=2 * P, key=3 * P, value=4 * P, qs=512, ks=128, vs=128, qw=0, kw=0, eps=1e-6, cos=5 * P,
                 maxp=100, R=64, il=0, pos=6 * P, kc=7 * P, vc=8 * P, slots=9 * P, T=0, Hq=8, Hkv=2, D=64, B=16, NB=4, dt=1)
        a.update(kw)
        return fn(*a.values(), *tail, None)

    same, fp8, i8 = lib.pkv_rope_and_cache, lib.pkv_rope_and_cache_fp8, lib.pkv_rope_and_cache_int8
    assert rope(same) == 0 and rope(i8) == 0 and rope(fp8, 1.0, 1.0) == 0  # no token: nothing to do
    for kw in (dict(dt=3), dict(dt=9), dict(D=60, R=0), dict(D=264), dict(R=20)):
        assert rope(same, **kw) == EUNSUPPORTED, kw
    for kw in (dict(T=-1), dict(Hq=0), dict(Hkv=0), dict(B=0), dict(NB=0), dict(R=72), dict(R=-8), dict(maxp=-1),
               dict(eps=-1.0), dict(eps=float("nan"))):
        assert rope(same, **kw) == EINVAL, kw
    for kw in (dict(query=0), dict(query_out=0), dict(key=0), dict(value=0), dict(kc=0), dict(vc=0), dict(slots=0),
               dict(cos=0), dict(pos=0), dict(qs=504), dict(ks=120), dict(vs=0), dict(qs=516), dict(key=3 * P + 8),
               dict(kc=7 * P + 4), dict(qw=P + 2), dict(pos=6 * P + 4), dict(query_out=2 * P, qs=1024)):
        assert rope(same, **{**dict(T=3), **kw}) == EINVAL, kw
    assert rope(fp8, 0.0, 1.0) == EINVAL and rope(fp8, 1.0, float("nan")) == EINVAL
    assert rope(fp8, 1.0, 1.0, D=72, R=0) == EUNSUPPORTED
    assert rope(i8, D=72, R=0) == EUNSUPPORTED and rope(i8, B=1, Hkv=2) == EUNSUPPORTED

    for fn in (lib.pkv_reshape_and_cache_int8, lib.pkv_read_cache_int8):
        assert fn(P, P, P, P, P, 0, 2, 64, 16, 4, 1, None) == 0
        assert fn(P, P, P, P, P, 3, 2, 64, 16, 4, 3, None) == EUNSUPPORTED
        assert fn(P, P, P, P, P, 3, 2, 72, 16, 4, 1, None) == EUNSUPPORTED
        assert fn(P, P, P, P, P, 3, 2, 272, 16, 4, 1, None) == EUNSUPPORTED
        assert fn(P, P, P, P, P, 3, 1, 64, 2, 4, 1, None) == EUNSUPPORTED
        assert fn(P, P, P, P, P, -3, 2, 64, 16, 4, 1, None) == EINVAL
        assert fn(P, 0, P, P, P, 3, 2, 64, 16, 4, 1, None) == EINVAL
        assert fn(P, P, P + 8, P, P, 3, 2, 64, 16, 4, 1, None) == EINVAL
        assert fn(P, P, P, P, P + 4, 3, 2, 64, 16, 4, 1, None) == EINVAL
    assert lib.pkv_int8_block_bytes(16, 8, 128) == 16 * 8 * 132 and lib.pkv_int8_block_bytes(0, 8, 128) == EINVAL

    def table(first=0, n=0, ptr=P, **kw):
        a = dict(base=1e4, factor=2.0, alpha=1.0, beta=4.0, attention_factor=1.0, original_max_position=100,
                 rotary_dim=64, scaling=0)
        a.update(kw)
        return lib.pkv_rope_table(ptr, first, n, ctypes.byref(_binding.RopeSpec(*a.values())), None)

    assert table() == 0
    for kw in (dict(scaling=4), dict(scaling=-1), dict(rotary_dim=60), dict(rotary_dim=264), dict(rotary_dim=8, scaling=2)):
        assert table(**kw) == EUNSUPPORTED, kw
    for kw in (dict(first=-1), dict(n=-1), dict(first=1 << 40, n=1), dict(base=0.0), dict(rotary_dim=0),
               dict(attention_factor=float("inf")), dict(scaling=1, factor=0.0), dict(scaling=3, alpha=4.0),
               dict(scaling=3, original_max_position=0), dict(n=3, ptr=0), dict(n=3, ptr=P + 4)):
        assert table(**kw) == EINVAL, kw
    assert lib.pkv_rope_table(P, 0, 0, None, None) == EINVAL


def test_decode_int8_arguments(mock):  # noqa: F811
    S, Hq, Hkv, D, B, NB, MB = 4, 16, 4, 64, 32, 19, 3
    q = torch.zeros(S, Hq, D, dtype=torch.bfloat16)
    out = torch.zeros_like(q)
    kc, vc = (torch.zeros(NB, B, Hkv, D + 4, dtype=torch.uint8) for _ in range(2))
    bt, cl = torch.zeros(S, MB, dtype=torch.int32), torch.zeros(S, dtype=torch.int32)
    pkv.paged_attention_decode_int8(out, q, kc, vc, bt, cl, 0.1, 90, partition_size=0, stream=2)
    name, a = mock.last()
    want = {"out": out.data_ptr(), "query": q.data_ptr(), "key_cache": kc.data_ptr(), "value_cache": vc.data_ptr(),
            "block_tables": bt.data_ptr(), "context_lens": cl.data_ptr(), "scale": f32(0.1), "num_seqs": S,
            "num_q_heads": Hq, "num_kv_heads": Hkv, "head_dim": D, "block_size": B, "max_blocks_per_seq": MB,
            "num_blocks": NB, "max_context_len": 90, "partition_size": 0, "dtype": 2, "workspace": 0,
            "workspace_bytes": 0, "stream": 2}
    assert name == "pkv_paged_attention_decode_int8" and a == want
    kn, vn, sm = torch.zeros(3, Hkv, D).bfloat16(), torch.zeros(3, Hkv, D).bfloat16(), torch.zeros(3, dtype=torch.int64)
    pkv.paged_attention_decode_step_int8(kn, vn, sm, out, q, kc, vc, bt, cl, 0.1, 90, partition_size=0, stream=2)
    name, a = mock.last()
    assert name == "pkv_paged_attention_decode_step_int8"
    assert a == {**want, "new_keys": kn.data_ptr(), "new_values": vn.data_ptr(), "slot_mapping": sm.data_ptr(),
                 "num_new_tokens": 3}
    for bad in (dict(query=q[:, :, :32]), dict(out=out.half()), dict(block_tables=bt.long()), dict(context_lens=cl[:2]),
                dict(block_tables=bt[:2]), dict(key_cache=kc[:3]), dict(key_cache=kc.half())):
        kw = dict(out=out, query=q, key_cache=kc, value_cache=vc, block_tables=bt, context_lens=cl)
        with pytest.raises(ValueError):
            pkv.paged_attention_decode_int8(**{**kw, **bad}, scale=0.1, max_context_len=90)


def test_decode_int8_refusals():
    from paged_kv_cache_409_b200 import build
    build.build()
    lib = pkv.load_library()
    P = 1 << 20

    def dec(fn=lib.pkv_paged_attention_decode_int8, head=(), **kw):
        a = dict(out=P, q=P, kc=P, vc=P, bt=P, cl=P, scale=0.1, S=0, Hq=4, Hkv=2, D=64, B=16, MB=4, NB=8, mx=64, part=0,
                 dt=1, ws=0, wb=0)
        a.update(kw)
        return fn(*head, *a.values(), None)

    assert dec() == 0
    for kw in (dict(dt=0), dict(dt=3), dict(dt=4), dict(D=96), dict(D=256), dict(B=64), dict(Hq=6), dict(Hq=32),
               dict(S=1, MB=5000, mx=16 * 4097)):
        assert dec(**kw) == EUNSUPPORTED, kw
    for kw in (dict(S=-1), dict(Hq=5), dict(NB=0), dict(MB=0), dict(scale=float("nan")), dict(part=8), dict(mx=-1),
               dict(S=1, q=0), dict(S=1, kc=P + 8), dict(S=1, cl=P + 2)):
        assert dec(**kw) == EINVAL, kw
    assert dec(S=1, part=16) == -5 and dec(S=1, part=16, ws=P, wb=100) == -5
    step = lib.pkv_paged_attention_decode_step_int8
    assert dec(step, (P, P, P, 0)) == 0
    assert dec(step, (P, 0, P, 3)) == EINVAL and dec(step, (P, P, P, -1)) == EINVAL
    assert dec(step, (P, P, P, 0), dt=0) == EUNSUPPORTED
    assert pkv.decode_partition_size(64, 32, 32, 128, 16, 2048, pkv.INT8) == 0
    # a context is split once it outlasts its share of four CTAs per SM (592 with no device visible) 2.5 times, into
    # parts of 1.5 shares or sqrt(pairs * max / 2) tokens, whichever is more
    share = 8 * 100000 // 592
    assert pkv.decode_partition_size(128, 32, 8, 128, 16, 5 * share // 2, pkv.INT8, 100000) == 0
    assert pkv.decode_partition_size(128, 32, 8, 128, 16, 4096, pkv.INT8, 100000) == -(-(share + share // 2) // 16) * 16
    assert pkv.decode_partition_size(64, 64, 8, 128, 16, 4096, pkv.INT8, 63 * 512 + 4096) == 1024
    assert lib.pkv_paged_attention_decode(P, P, P, P, P, P, 0.1, 1, 4, 2, 64, 16, 4, 8, 64, 0, 4, None, 0, None) == -2


def test_prefill_int8_arguments_and_refusals(mock):  # noqa: F811
    R, Tq, Hq, Hkv, D, B, NB, MB = 2, 9, 8, 2, 128, 16, 23, 6
    q = torch.zeros(Tq, Hq, D, dtype=torch.float16)
    out = torch.zeros_like(q)
    kc, vc = (torch.zeros(NB, B, Hkv, D + 4, dtype=torch.uint8) for _ in range(2))
    bt, sl = torch.zeros(R, MB, dtype=torch.int32), torch.zeros(R, dtype=torch.int32)
    qsl = torch.zeros(R + 1, dtype=torch.int32)
    pkv.paged_attention_prefill_chunk_int8(out, q, kc, vc, bt, sl, qsl, 5, 0.7, stream=4)
    name, a = mock.last()
    assert name == "pkv_paged_attention_prefill_chunk_int8"
    assert a == {"out": out.data_ptr(), "query": q.data_ptr(), "key_cache": kc.data_ptr(), "value_cache": vc.data_ptr(),
                 "block_tables": bt.data_ptr(), "seq_lens": sl.data_ptr(), "query_start_loc": qsl.data_ptr(),
                 "num_chunks": R, "total_q_tokens": Tq, "max_q_len": 5, "scale": f32(0.7), "num_q_heads": Hq,
                 "num_kv_heads": Hkv, "head_dim": D, "block_size": B, "max_blocks_per_seq": MB, "num_blocks": NB,
                 "dtype": 1, "stream": 4}
    for bad in (dict(query=q[:, :, :64]), dict(out=out.bfloat16()), dict(query_start_loc=qsl[:2]),
                dict(block_tables=bt[:1]), dict(seq_lens=sl.long()), dict(value_cache=vc[:2])):
        kw = dict(out=out, query=q, key_cache=kc, value_cache=vc, block_tables=bt, seq_lens=sl, query_start_loc=qsl)
        with pytest.raises(ValueError):
            pkv.paged_attention_prefill_chunk_int8(**{**kw, **bad}, max_q_len=5, scale=0.7)


def test_prefill_int8_refusals():
    from paged_kv_cache_409_b200 import build
    build.build()
    fn = pkv.load_library().pkv_paged_attention_prefill_chunk_int8
    P = 1 << 20

    def pre(**kw):
        a = dict(out=P, q=P, kc=P, vc=P, bt=P, sl=P, qsl=P, R=0, Tq=4, mq=4, scale=0.1, Hq=4, Hkv=2, D=64, B=16, MB=4, NB=8,
                 dt=1)
        a.update(kw)
        return fn(*a.values(), None)

    assert pre() == 0 and pre(R=1, Tq=0) == 0 and pre(R=1, mq=0) == 0
    for kw in (dict(dt=0), dict(dt=3), dict(dt=4), dict(D=96), dict(B=64), dict(Hq=6), dict(Hq=32)):
        assert pre(**kw) == EUNSUPPORTED, kw
    for kw in (dict(R=-1), dict(Tq=-1), dict(mq=-1), dict(Hq=5), dict(NB=0), dict(MB=0), dict(scale=float("inf")),
               dict(R=1, q=0), dict(R=1, vc=P + 8), dict(R=1, qsl=P + 2)):
        assert pre(**kw) == EINVAL, kw
