"""The operators between a layer's projections and its attention output over a quantised paged cache: their plain forms, the calls
of the framework that compute them, and the cases at which they are measured.

``op`` names the operator of a case:

  table    cos / sin rows of (scaled) rotary positions
  rotate   RMS norm of every query and key head, rotary positions, and the append of K and V, in one pass; the pools hold the
           inputs' type or 8-bit rows ("pool": "same" | "int8")
  append   quantising K and V into 8-bit pools, and reading the rows back
  decode   attention of one query token per sequence over 8-bit pools
  prefill  causal attention of chunks of new tokens over 8-bit pools

An 8-bit pool is a uint8 tensor [blocks, block_size, kv_heads, head_dim + 4]; a block's bytes are the codes [block_size, kv_heads,
head_dim] and then the fp32 scales [kv_heads, block_size].  A row (token, KV head) with scale s and codes u stands for s * (u - 128),
s = max |x| / 127.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a short context's table, as a small model builds it once
        dict(name="table 4096x64", op="table", positions=4096, rotary=64, base=10000.0, scaling="none", factor=1.0, alpha=1.0,
             beta=4.0, original=4096, attention=1.0),
        # a long context, extended by parts: high frequencies kept, low ones interpolated
        dict(name="table 131072x128 by parts", op="table", positions=131072, rotary=128, base=500000.0, scaling="by_parts",
             factor=8.0, alpha=1.0, beta=4.0, original=8192, attention=1.0),
        # one decode step: a token per sequence, grouped heads, 16-bit pools (launch-bound)
        dict(name="rotate 64 tokens bf16", op="rotate", tokens=64, hq=32, hkv=8, dim=128, rotary=128, interleaved=False, norm=True,
             block=16, dtype="bf16", pool="same", far=32768),
        # the chunks of a large prefill step, written as 8-bit rows
        dict(name="rotate 8192 tokens bf16 int8", op="rotate", tokens=8192, hq=32, hkv=8, dim=128, rotary=128, interleaved=False,
             norm=True, block=32, dtype="bf16", pool="int8", far=131072),
        # interleaved pairs over half of a small head, no norm, an odd token count
        dict(name="rotate 2049 tokens f16 part", op="rotate", tokens=2049, hq=32, hkv=32, dim=64, rotary=32, interleaved=True,
             norm=False, block=16, dtype="f16", pool="same", far=4096),
        # one token per sequence of a batch of 256 into 8-bit pools
        dict(name="append 256 tokens bf16", op="append", tokens=256, hkv=8, dim=128, block=16, dtype="bf16"),
        # a long prompt's rows, 32 KV heads
        dict(name="append 8191 tokens f16", op="append", tokens=8191, hkv=32, dim=128, block=16, dtype="f16"),
        # the smallest batch: latency counts
        dict(name="decode 4 short f16", op="decode", seqs=4, lo=1, hi=100, lens="uniform", lens_seed=1, hq=4, hkv=4, dim=64, block=16,
             dtype="f16"),
        # 64 sequences over [128, 2048], one query head per KV head
        dict(name="decode 64 f16", op="decode", seqs=64, lo=128, hi=2048, lens="uniform", lens_seed=2, hq=32, hkv=32, dim=128,
             block=16, dtype="f16"),
        # 256 sequences with long-tailed lengths, 8 query heads per KV head
        dict(name="decode 256 grouped bf16", op="decode", seqs=256, lo=16, hi=4096, lens="lognormal", lens_seed=3, hq=64, hkv=8,
             dim=128, block=16, dtype="bf16"),
        # a continuous-batching step's four prompt chunks over what is cached already
        dict(name="prefill 4x512 bf16", op="prefill", chunks=4, nlo=512, nhi=512, plo=0, phi=8192, lens_seed=4, hq=32, hkv=8, dim=128,
             block=32, dtype="bf16"),
        # ragged verification-sized chunks, small heads, small blocks
        dict(name="prefill 7 ragged f16", op="prefill", chunks=7, nlo=1, nhi=130, plo=0, phi=1000, lens_seed=5, hq=16, hkv=8, dim=64,
             block=8, dtype="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["table", "rotate", "append", "decode", "prefill"])
    if op == "table":
        scaling = rng.choice(["none", "linear", "ntk", "by_parts"])
        rotary = rng.choice([16, 32, 64, 96, 128])
        return dict(op=op, positions=_log(rng, 100, 131072), rotary=rotary, base=rng.choice([10000.0, 500000.0, 1000000.0]),
                    scaling=scaling, factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 32.0]),
                    alpha=1.0, beta=rng.choice([4.0, 32.0]), original=rng.choice([2048, 4096, 8192]),
                    attention=rng.choice([1.0, 1.2079]))
    if op == "rotate":
        dim = rng.choice([64, 96, 128, 128])
        hkv = rng.choice([1, 2, 4, 8])
        return dict(op=op, tokens=_log(rng, 1, 8192), hq=hkv * rng.choice([1, 2, 4, 5, 8] if hkv < 8 else [1, 2, 4]), hkv=hkv, dim=dim,
                    rotary=rng.choice([16, 32, dim // 2, dim]), interleaved=rng.random() < 0.4, norm=rng.random() < 0.6,
                    block=rng.choice([8, 16, 32]), dtype=rng.choice(["f16", "bf16"]), pool=rng.choice(["same", "int8"]),
                    far=rng.choice([4096, 32768, 131072]))
    if op == "append":
        return dict(op=op, tokens=_log(rng, 1, 8191), hkv=rng.choice([1, 2, 5, 8, 32]), dim=rng.choice([64, 96, 128]),
                    block=rng.choice([8, 16, 32]), dtype=rng.choice(["f16", "bf16"]))
    dtype, dim, block = rng.choice(["f16", "bf16"]), rng.choice([64, 128, 128]), rng.choice([8, 16, 32])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 8])
    if op == "decode":
        hi = _log(rng, 40, 32768)
        seqs = max(1, min(256, _log(rng, 1, max(2, int(500000 / hi)))))
        return dict(op=op, seqs=seqs, lo=1, hi=hi, lens=rng.choice(["uniform", "lognormal"]), lens_seed=rng.randrange(1 << 20), hq=hq,
                    hkv=hkv, dim=dim, block=block, dtype=dtype)
    nhi = _log(rng, 1, 512)
    return dict(op=op, chunks=rng.randint(1, 4), nlo=rng.randint(1, nhi), nhi=nhi, plo=0, phi=_log(rng, 8, 8192),
                lens_seed=rng.randrange(1 << 20), hq=min(hq, 32), hkv=min(hkv, 8), dim=dim, block=block, dtype=dtype)


def _lengths(case):
    """Lengths of a decode batch, or (chunk lengths, cached tokens before them); of the case alone."""
    rng = random.Random(case["lens_seed"])
    if case["op"] == "decode":
        if case["lens"] == "uniform":
            return [rng.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]
        mid = math.sqrt(case["lo"] * case["hi"]) * 4
        return [min(case["hi"], max(case["lo"], int(round(math.exp(rng.gauss(math.log(mid), 1.0)))))) for _ in range(case["seqs"])]
    n = [rng.randint(case["nlo"], case["nhi"]) for _ in range(case["chunks"])]
    return n, [rng.randint(case["plo"], case["phi"]) for _ in range(case["chunks"])]


def work(case):
    op = case["op"]
    if op == "table":
        n = case["positions"] * case["rotary"]
        return {"bytes": 4 * n, "flops": 10 * n}
    eb = 4 if case["dtype"] == "f32" else 2
    D = case["dim"]
    if op == "rotate":
        T, hq, hkv = case["tokens"], case["hq"], case["hkv"]
        row = D + 4 if case["pool"] == "int8" else D * eb
        b = T * (2 * hq * D * eb + 2 * hkv * (D * eb + row) + 4 * case["rotary"] + 16)
        if case["pool"] == "int8":
            b += T * 2 * hkv * (row + D * eb)  # the rows read back
        return {"bytes": b, "flops": T * (hq + hkv) * D * 8}
    if op == "append":
        T, hkv = case["tokens"], case["hkv"]
        return {"bytes": T * (2 * hkv * 2 * (D * eb + D + 4) + 8), "flops": T * hkv * D * 8}
    if op == "decode":
        total = sum(_lengths(case))
        return {"bytes": total * 2 * case["hkv"] * (D + 4) + 2 * case["seqs"] * case["hq"] * D * eb, "flops": 4 * total * case["hq"] * D}
    n, prior = _lengths(case)
    pairs = sum(a * p + a * (a + 1) // 2 for a, p in zip(n, prior))
    return {"bytes": sum(a + p for a, p in zip(n, prior)) * 2 * case["hkv"] * (D + 4) + 2 * sum(n) * case["hq"] * D * eb,
            "flops": 4 * pairs * case["hq"] * D}


# ------------------------------------------------------------------ inputs
def _views(pool):
    """Codes [NB, B, H, D] and scales [NB, H, B] of an 8-bit pool, as views of it."""
    NB, B, H, W = pool.shape
    flat = pool.view(NB, B * H * W)
    n = B * H * (W - 4)
    return flat[:, :n].view(NB, B, H, W - 4), flat.view(torch.float32)[:, n // 4:].view(NB, H, B)


def _rows(g, n, hkv, dim, loud):
    """Cached rows: unit normal, with a few loud channels in K as projections have."""
    x = torch.randn(n, hkv, dim, generator=g, device=DEV)
    if loud:
        x[..., :: max(1, dim // 4)] *= 4.0
    return x


def _filled_pool(g, NB, B, hkv, dim, loud):
    x = _rows(g, NB * B, hkv, dim, loud)
    s = x.abs().amax(-1) / 127.0
    u = torch.round(x / s[..., None]) + 128.0
    pool = torch.empty(NB, B, hkv, dim + 4, dtype=torch.uint8, device=DEV)
    codes, scales = _views(pool)
    codes.copy_(u.view(NB, B, hkv, dim).to(torch.uint8))
    scales.copy_(s.view(NB, B, hkv).permute(0, 2, 1))
    return pool


def _tables(lens, B, g):
    """Block tables over one permutation of the pool; unused entries are -1."""
    need = [-(-n // B) for n in lens]
    NB = sum(need) + max(1, sum(need) // 10)
    perm = torch.randperm(NB, generator=g, device=DEV).to(torch.int32)
    start = torch.tensor([0] + need[:-1], device=DEV).cumsum(0)
    col = torch.arange(max(max(need), 1), device=DEV)
    live = col[None, :] < torch.tensor(need, device=DEV)[:, None]
    at = (start[:, None] + col[None, :]).clamp(max=NB - 1)
    return NB, torch.where(live, perm[at], torch.full_like(perm[at], -1)).contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op == "table":
        # the caller's own buffer; the seed moves the window of positions
        s["first"] = int(torch.randint(0, 4096, (1,), generator=g, device=DEV))
        s["out"] = torch.empty(case["positions"], case["rotary"], device=DEV)
        return s
    dt, D = TYPES[case["dtype"]], case["dim"]
    if op in ("rotate", "append"):
        T, hkv, B = case["tokens"], case["hkv"], case["block"]
        NB = -(-T // B) + 2
        s["slots"] = torch.randperm(NB * B, generator=g, device=DEV)[:T].contiguous()
    if op == "rotate":
        hq, R = case["hq"], case["rotary"]
        qkv = torch.randn(T, (hq + 2 * hkv) * D, generator=g, device=DEV).to(dt)  # the projection's output, taken apart below
        s["q"] = qkv[:, : hq * D].view(T, hq, D)
        s["k"] = qkv[:, hq * D: (hq + hkv) * D].view(T, hkv, D)
        s["v"] = qkv[:, (hq + hkv) * D:].view(T, hkv, D)
        s["positions"] = torch.randint(0, case["far"], (T,), generator=g, device=DEV)
        i = torch.arange(0, R, 2, device=DEV, dtype=torch.float64)
        angle = torch.arange(case["far"], device=DEV, dtype=torch.float64)[:, None] * 10000.0 ** (-i / R)[None, :]
        s["table"] = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        s["qw"] = s["kw"] = None
        if case["norm"]:
            s["qw"] = (1 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(dt)
            s["kw"] = (1 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(dt)
        s["q_out"] = torch.empty(T, hq, D, dtype=dt, device=DEV)
        if case["pool"] == "same":
            s["kc"] = torch.randn(NB, B, hkv, D, generator=g, device=DEV).to(dt)
            s["vc"] = torch.randn(NB, B, hkv, D, generator=g, device=DEV).to(dt)
    if op == "append":
        s["k"] = _rows(g, T, hkv, D, True).to(dt)
        s["v"] = _rows(g, T, hkv, D, False).to(dt)
    if op == "append" or (op == "rotate" and case["pool"] == "int8"):
        s["kc"] = _filled_pool(g, NB, B, hkv, D, True)
        s["vc"] = _filled_pool(g, NB, B, hkv, D, False)
        s["k_read"] = torch.empty(T, hkv, D, dtype=dt, device=DEV)
        s["v_read"] = torch.empty(T, hkv, D, dtype=dt, device=DEV)
    if op in ("rotate", "append"):
        return s
    # attention
    B = case["block"]
    if op == "decode":
        lens = _lengths(case)
        rows = case["seqs"]
        s["total"] = sum(lens)
    else:
        n, prior = _lengths(case)
        lens = [a + p for a, p in zip(n, prior)]
        rows = sum(n)
        s["max_n"] = max(n)
        s["start"] = torch.tensor([0] + n, device=DEV).cumsum(0).to(torch.int32)
    s["max_len"] = max(lens)
    s["lens_t"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    NB, s["bt"] = _tables(lens, B, g)
    s["q"] = torch.randn(rows, case["hq"], D, generator=g, device=DEV).to(dt)
    s["out"] = torch.empty_like(s["q"])
    s["kc"] = _filled_pool(g, NB, B, case["hkv"], D, True)
    s["vc"] = _filled_pool(g, NB, B, case["hkv"], D, False)
    s["scale"] = D ** -0.5
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import paged_kv_cache_409_b200 as pkv
    op = s["op"]
    if op == "table":
        return pkv.rope_table(s["out"], base=s["base"], first_position=s["first"], scaling=s["scaling"], factor=s["factor"],
                              alpha=s["alpha"], beta=s["beta"], original_max_position=s["original"],
                              attention_factor=s["attention"])
    if op == "rotate":
        call = pkv.rope_and_cache if s["pool"] == "same" else pkv.rope_and_cache_int8
        call(s["q_out"], s["q"], s["k"], s["v"], s["table"], s["positions"], s["kc"], s["vc"], s["slots"],
             interleaved=s["interleaved"], q_norm_weight=s["qw"], k_norm_weight=s["kw"], eps=EPS)
        if s["pool"] == "same":
            return {"q": s["q_out"], "k": s["kc"], "v": s["vc"]}
        pkv.read_cache_int8(s["k_read"], s["v_read"], s["kc"], s["vc"], s["slots"])
        return {"q": s["q_out"], "k": s["k_read"], "v": s["v_read"]}
    if op == "append":
        pkv.reshape_and_cache_int8(s["k"], s["v"], s["kc"], s["vc"], s["slots"])
        pkv.read_cache_int8(s["k_read"], s["v_read"], s["kc"], s["vc"], s["slots"])
        return {"k": s["k_read"], "v": s["v_read"]}
    if op == "decode":
        return pkv.paged_attention_decode_int8(s["out"], s["q"], s["kc"], s["vc"], s["bt"], s["lens_t"], s["scale"], s["max_len"],
                                               total_context_tokens=s["total"])
    return pkv.paged_attention_prefill_chunk_int8(s["out"], s["q"], s["kc"], s["vc"], s["bt"], s["lens_t"], s["start"], s["max_n"],
                                                  s["scale"])


def _frequencies(s, device):
    """The rotary frequencies of a case, in 64 bits."""
    R = s["rotary"]
    i = torch.arange(0, R, 2, device=device, dtype=torch.float64)
    base = s["base"] * s["factor"] ** (R / (R - 2)) if s["scaling"] == "ntk" else s["base"]
    theta = base ** (-i / R)
    if s["scaling"] == "linear":
        theta = theta / s["factor"]
    if s["scaling"] == "by_parts":
        turns = s["original"] * theta / (2 * math.pi)
        keep = ((turns - s["alpha"]) / (s["beta"] - s["alpha"])).clamp(0, 1)
        theta = (1 - keep) * theta / s["factor"] + keep * theta
    return theta


def _norm_rotate(x, w, cos, sin, interleaved):
    """RMS norm over the last dimension (w given) and the rotation of its first dims; fp32 in, fp32 out."""
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    half = cos.shape[-1]
    r, rest = x[..., : 2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = r[..., :half], r[..., half:]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, rest], -1)


def _put_rows(pool, slots, x):
    """Quantise rows x [T, H, D] (fp32) into the pool's slots."""
    B = pool.shape[1]
    codes, scales = _views(pool)
    s = x.abs().amax(-1) / 127.0
    u = torch.round(x / s[..., None]) + 128.0
    codes[slots // B, slots % B] = u.to(torch.uint8)
    scales[slots // B, :, slots % B] = s


def _get_rows(pool, slots):
    B = pool.shape[1]
    codes, scales = _views(pool)
    return (codes[slots // B, slots % B].float() - 128.0) * scales[slots // B, :, slots % B][..., None]


def _gathered(pool, bt):
    """The sequences' rows as values [S, H, L, D], L the table's reach."""
    B, H, D = pool.shape[1], pool.shape[2], pool.shape[3] - 4
    codes, scales = _views(pool)
    at = bt.clamp(min=0).long()
    x = (codes[at].float() - 128.0) * scales[at].transpose(-1, -2)[..., None]  # [S, MB, B, H, D]
    return x.flatten(1, 2).transpose(1, 2)


def _softmax_v(scores, v):
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - m)
    return (p @ v) / p.sum(-1, keepdim=True)


def _plain(s):
    op = s["op"]
    if op == "table":
        p = torch.arange(s["first"], s["first"] + s["positions"], device=DEV, dtype=torch.float64)
        angle = p[:, None] * _frequencies(s, DEV)[None, :]
        s["out"].copy_(torch.cat([angle.cos(), angle.sin()], 1) * s["attention"])
        return s["out"]
    if op == "rotate":
        row = s["table"][s["positions"]]
        half = row.shape[1] // 2
        cos, sin = row[:, None, :half], row[:, None, half:]
        q = _norm_rotate(s["q"].float(), s["qw"], cos, sin, s["interleaved"])
        k = _norm_rotate(s["k"].float(), s["kw"], cos, sin, s["interleaved"])
        s["q_out"].copy_(q)
        if s["pool"] == "same":
            B = s["block"]
            s["kc"][s["slots"] // B, s["slots"] % B] = k.to(s["kc"].dtype)
            s["vc"][s["slots"] // B, s["slots"] % B] = s["v"]
            return {"q": s["q_out"], "k": s["kc"], "v": s["vc"]}
        _put_rows(s["kc"], s["slots"], k)
        _put_rows(s["vc"], s["slots"], s["v"].float())
        s["k_read"].copy_(_get_rows(s["kc"], s["slots"]))
        s["v_read"].copy_(_get_rows(s["vc"], s["slots"]))
        return {"q": s["q_out"], "k": s["k_read"], "v": s["v_read"]}
    if op == "append":
        _put_rows(s["kc"], s["slots"], s["k"].float())
        _put_rows(s["vc"], s["slots"], s["v"].float())
        s["k_read"].copy_(_get_rows(s["kc"], s["slots"]))
        s["v_read"].copy_(_get_rows(s["vc"], s["slots"]))
        return {"k": s["k_read"], "v": s["v_read"]}
    K, V = _gathered(s["kc"], s["bt"]), _gathered(s["vc"], s["bt"])  # [S, Hkv, L, D]
    S, H, L, D = K.shape
    G = s["hq"] // H
    j = torch.arange(L, device=DEV)
    if op == "decode":
        q = s["q"].float().view(S, H, G, D)
        scores = (q @ K.transpose(-1, -2)) * s["scale"]
        scores = scores.masked_fill(j >= s["lens_t"][:, None, None, None], -math.inf)
        s["out"].copy_(_softmax_v(scores, V).view(S, s["hq"], D))
        return s["out"]
    # prefill: the chunks padded to the longest, [R, Hkv, G * n, D]
    start, n = s["start"][:-1].long(), s["max_n"]
    count = (s["start"][1:] - s["start"][:-1]).long()
    i = torch.arange(n, device=DEV)
    at = (start[:, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[at].view(S, n, H, G, D).permute(0, 2, 3, 1, 4).reshape(S, H, G * n, D)
    scores = ((q @ K.transpose(-1, -2)) * s["scale"]).view(S, H, G, n, L)
    last = (s["lens_t"].long() - count)[:, None] + i  # the position of each row
    scores = scores.masked_fill(j > last[:, None, None, :, None], -math.inf).view(S, H, G * n, L)
    o = _softmax_v(scores, V).view(S, H, G, n, D).permute(0, 3, 1, 2, 4).reshape(S * n, H * G, D)
    chunk = torch.repeat_interleave(torch.arange(S, device=DEV), count, output_size=s["q"].shape[0])
    s["out"].copy_(o[chunk * n + torch.arange(s["q"].shape[0], device=DEV) - start[chunk]])
    return s["out"]


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """The same results from the definitions, in 64 bits, sequence by sequence."""
    s = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "table":
        R, f = case["rotary"], case["factor"]
        cols = []
        for k in range(R // 2):
            base = case["base"]
            if case["scaling"] == "ntk":
                base *= f ** (R / (R - 2))
            th = math.exp(-2 * k / R * math.log(base))
            if case["scaling"] == "linear":
                th /= f
            elif case["scaling"] == "by_parts":
                r = case["original"] / (2 * math.pi / th)
                keep = min(1.0, max(0.0, (r - case["alpha"]) / (case["beta"] - case["alpha"])))
                th = th / f * (1 - keep) + th * keep
            cols.append(th)
        p = torch.arange(case["positions"], dtype=f64, device=DEV) + s["first"]
        a = torch.outer(p, torch.tensor(cols, dtype=f64, device=DEV))
        return torch.cat([torch.cos(a), torch.sin(a)], 1) * case["attention"]

    def quantised(x):
        s_ = x.abs().max(-1, keepdim=True).values / 127
        return torch.round(x / s_) * s_

    def turned(x, w):
        x = x.to(f64)
        if w is not None:
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.to(f64)
        h = case["rotary"] // 2
        row = s["table"].to(f64)[s["positions"]]
        z = torch.complex(row[:, :h], row[:, h:])[:, None, :]
        r = x[..., : 2 * h]
        if case["interleaved"]:
            r = torch.view_as_real(torch.view_as_complex(r.reshape(*r.shape[:-1], h, 2).contiguous()) * z).flatten(-2)
        else:
            c = torch.complex(r[..., :h].contiguous(), r[..., h:].contiguous()) * z
            r = torch.cat([c.real, c.imag], -1)
        return torch.cat([r, x[..., 2 * h:]], -1)

    if op == "rotate":
        q, k, v = turned(s["q"], s["qw"]), turned(s["k"], s["kw"]), s["v"].to(f64)
        if case["pool"] == "int8":
            return {"q": q, "k": quantised(k), "v": quantised(v)}
        kc, vc = s["kc"].to(f64), s["vc"].to(f64)
        kc.view(-1, *k.shape[1:])[s["slots"]] = k
        vc.view(-1, *v.shape[1:])[s["slots"]] = v
        return {"q": q, "k": kc, "v": vc}
    if op == "append":
        return {"k": quantised(s["k"].to(f64)), "v": quantised(s["v"].to(f64))}

    B, D, H = case["block"], case["dim"], case["hkv"]
    G = case["hq"] // H
    n_codes = B * H * D

    def rows(pool, ids, length):
        raw = pool.view(pool.shape[0], -1)[ids]
        u = raw[:, :n_codes].reshape(-1, H, D).to(f64) - 128
        sc = raw[:, n_codes:].contiguous().view(torch.float32).view(-1, H, B).permute(0, 2, 1).reshape(-1, H).to(f64)
        return (u * sc[..., None])[:length]

    out = torch.empty(s["q"].shape, dtype=f64, device=DEV)
    lens = s["lens_t"].tolist()
    starts = s["start"].tolist() if op == "prefill" else None
    for i, length in enumerate(lens):
        ids = s["bt"][i, : -(-length // B)].long()
        K, V = rows(s["kc"], ids, length), rows(s["vc"], ids, length)
        lo, hi = (i, i + 1) if op == "decode" else (starts[i], starts[i + 1])
        q = s["q"][lo:hi].to(f64).view(hi - lo, H, G, D)
        t = torch.einsum("nhgd,lhd->nhgl", q, K) * s["scale"]
        if op == "prefill":
            pos = torch.arange(length - (hi - lo), length, device=DEV)
            t = t.masked_fill(torch.arange(length, device=DEV)[None, None, None, :] > pos[:, None, None, None], -math.inf)
        out[lo:hi] = torch.einsum("nhgl,lhd->nhgd", torch.softmax(t, -1), V).reshape(hi - lo, H * G, D)
    return out
