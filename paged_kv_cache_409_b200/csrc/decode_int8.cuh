// decode_int8.cuh -- paged decode attention over int8 pools (rows of one-byte
// codes with an fp32 scale each, row_kernels.cuh), head dim 64 or 128, query
// and output in fp16 or bf16, 1, 2, 4 or 8 query heads per KV head.
//
// With K row j = ks_j (u_j - 128) and V row j = vs_j (v_j - 128):
//
//   * Scores.  The query row is written once as a 16-bit integer row,
//     q = qs (256 hi + lo), qs = max |q| / 32639, hi and lo signed bytes, and
//     q . (u - 128) = 256 (hi . u) + lo . u - 128 (256 sum hi + sum lo) is an
//     integer below 2^31: two u8 x s8 MMAs (m16n8k32, s32 accumulators that
//     start at -128 sum hi and -128 sum lo) give it exactly, from the bytes as
//     they lie in shared memory -- K is never widened.  hi and lo are two
//     columns of one MMA's eight for up to four heads.  The only rounding is
//     the query's, half a step of 2^-15 of its row's largest element: below
//     the step that bf16 or fp16 gave that element.
//   * Weights.  V's scale goes into the exponent: with s_j the score in log2
//     units, w_j = exp2(s_j + log2 vs_j - M), M a running base of that sum, is
//     the weight of the integer row v_j - 128, and w_j / vs_j = exp2(s_j - M)
//     its share of the softmax sum.  So the largest w is near 1 whatever the
//     rows' scales are, P goes into the MMA as one f16 term without scaling,
//     and a score still costs one FMA, one exponential and one FMA.
//   * O.  O^T += (v - 128)^T . P^T on mma.sync m16n8k16 in f16: a byte permute
//     puts 0x64 over a code (the f16 1024 + v), a subtraction of 1152 leaves
//     v - 128, exact.
//
// Every row past the context has weight 0 and codes that are finite f16
// values, so V needs no masking; a bad block (flagged) reads as zeros.  A row
// whose scale is NaN makes the result NaN.  Partitions, per-warp TMA pipelines
// and the CTA merge are those of decode.cuh; a block's scales (one KV head's)
// come through tensor maps of their own, with the codes' coordinates and on the
// same barrier.
//
// Bound by memory.  64 sequences of [128, 2048] tokens x 32 heads of 128, fp16:
// 92-94 us in graph replays over three sets of inputs, 6.4 TB/s (0.98 of a copy);
// 93-99 us as a call on new inputs.  256 sequences x 8 KV heads, 8 query heads
// each: 118-128 us, 5.7-6.2 TB/s; there the eight columns of an MMA are all in
// use, and what is left is the ranking and the last wave.  Four warps of two
// stages and units of 16 tokens: 8 warps, 2 warps, 3 stages and units of 32 are
// all slower on the latter (172, 148, 145, 140 us when this version took 130).
#pragma once

#include "decode.cuh"
#include "row_kernels.cuh"

namespace pkv {

__device__ __forceinline__ float lg2_approx(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// max that keeps NaN
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// C (s32) += A (u8, 16 x 32, row) . B (s8, 32 x 8, col)
__device__ __forceinline__ void mma_16832_u8s8(int (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The tensor maps of both pools: K codes, V codes, K scales, V scales, all of
// four dimensions with the coordinates (0, KV head, 0, block).
struct Int8Maps {
    CUtensorMap m[4];
};

__device__ __forceinline__ uint32_t hsub2_1152(uint32_t x) {
    uint32_t y;
    asm("add.f16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(0xE480E480u));
    return y;
}

// Byte offset of 16-byte chunk `ch` of row `tok` in a TMA-swizzled tile of
// D-byte rows (128-byte swizzle, or 64-byte for 64-byte rows).
template <int D>
__device__ __forceinline__ int int8_chunk(int tok, int ch) {
    if constexpr (D == 128) return tok * 128 + ((ch ^ (tok & 7)) << 4);
    else return tok * 64 + ((ch ^ ((tok >> 1) & 3)) << 4);
}

// U consecutive blocks of a sequence form one unit of B * U tokens (a multiple
// of 16): one stage, one softmax step.
template <int D, int B, int G, int NST, int NW, int U>
struct DecodeInt8Cfg {
    static constexpr int BU = B * U;
    static constexpr int TILE = BU * D;      // one unit-head of K (or V) codes
    static constexpr int STAGE = 2 * TILE;
    static constexpr int STAGES_BYTES = NW * NST * STAGE;
    static constexpr int SC_OFF = STAGES_BYTES;  // [warp][stage][K, V][U] boxes of B scales
    static constexpr int SC_BOX = 32;            // floats from box to box: a tensor copy's target is 128-byte aligned
    static constexpr int SC_STAGE = 2 * U * SC_BOX;
    static constexpr uint32_t TX = STAGE + 2 * BU * 4;  // bytes of a stage
    static constexpr int RED_BYTES = NW * G * (D + 2) * 4;  // the merge reuses the stage buffers
    static constexpr int SC_END = SC_OFF + NW * NST * SC_STAGE * 4;
    static constexpr int BT_OFF = SC_END > RED_BYTES ? SC_END : RED_BYTES;
    static_assert(B <= 32 && BU % 16 == 0 && TILE % 1024 == 0 && BT_OFF % 16 == 0, "unit shape");
    static_assert(RED_BYTES <= SC_END, "merge scratch");
    static_assert(U <= 8, "a lane per copy");
    static size_t smem_bytes(int pb) { return 1024 + BT_OFF + static_cast<size_t>(pb) * 4 + 16 + NW * NST * 8; }
};

// The sequence that comes r-th when the batch is ordered by length, longest
// first: lengths fall into 32 classes (len >> shift, shift chosen for the call's
// bound), sequences of one class keep their order.  Every CTA finds its own: a
// histogram and a scan give the class, ballots the place in it.  No CTA then
// starts a long sequence last.  Up to 256 sequences, two lengths a thread; larger
// batches go in the listed order and by the other pools' split rule, which costs
// most just behind the limit and nothing further on (lognormal lengths up to
// 4096, 64 heads over 8: 256 sequences 120 us, 6.0 TB/s; 257 135, 5.3; 300 154,
// 5.5; 512 252, 5.9; 1024 510, 5.9).
constexpr int kMaxRankedSeqs = 256;

template <int kThreads>
__device__ __forceinline__ int sequence_by_length(const int32_t* lens, int n, int shift, int r) {
    constexpr int kPer = kMaxRankedSeqs / kThreads, kWarps = kThreads / 32;
    __shared__ int hist[32];
    __shared__ int hits[kPer * kWarps];
    __shared__ int found;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int cls[kPer];  // of sequences tid, tid + kThreads, ...
#pragma unroll
    for (int m = 0; m < kPer; ++m) {
        const int i = tid + m * kThreads;
        cls[m] = i < n ? min(max(lens[i], 0) >> shift, 31) : -1;
    }
    if (tid < 32) hist[tid] = 0;
    __syncthreads();
#pragma unroll
    for (int m = 0; m < kPer; ++m)
        if (cls[m] >= 0) atomicAdd(&hist[cls[m]], 1);
    __syncthreads();
    const int count = hist[31 - lane];
    int upto = count;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += v;
    }
    const int at = __ffs(__ballot_sync(0xffffffffu, upto > r)) - 1;  // r < n: some lane's count reaches it
    int k = r - (__shfl_sync(0xffffffffu, upto, at) - __shfl_sync(0xffffffffu, count, at));  // place in the class
    unsigned mine[kPer];
#pragma unroll
    for (int m = 0; m < kPer; ++m) {
        mine[m] = __ballot_sync(0xffffffffu, cls[m] == 31 - at);
        if (lane == 0) hits[m * kWarps + warp] = __popc(mine[m]);
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < kPer; ++m) {
        int before = 0;
#pragma unroll
        for (int j = 0; j < kPer * kWarps; ++j) before += j < m * kWarps + warp ? hits[j] : 0;
        if ((mine[m] >> lane & 1) && before + __popc(mine[m] & ((1u << lane) - 1)) == k) found = tid + m * kThreads;
    }
    __syncthreads();
    return found;
}

// CTAs per SM that the registers are told to allow: four (106-124 registers) where
// that is faster than what the compiler takes by itself (96-98 at head dim 128,
// 64-95 at 64).  us, by itself | four, of 128 sequences over [512, 4096], blocks of
// 16, 16 KV heads for 1 and 2 query heads each, 8 for 4 and 8:
//   head dim 128: 184.0 | 185.7, 190.1 | 193.6, 102.3 | 99.1, 111.9 | 107.4
//   head dim 64:  109.8 | 109.9, 109.0 | 107.3, 51.6 | 51.1, 51.9 | 53.8
constexpr int int8_min_ctas(int D, int G) { return (D == 128 ? G >= 4 : G < 8) ? 4 : 0; }

template <typename T, int D, int B, int G, int NST, int NW, int U>
__global__ void __launch_bounds__(NW * 32, int8_min_ctas(D, G)) paged_decode_int8_kernel(const DecodeParams p,
                                                                    const __grid_constant__ Int8Maps tm) {
    using C = DecodeInt8Cfg<D, B, G, NST, NW, U>;
    constexpr int kThreads = NW * 32;
    constexpr int BU = C::BU;
    constexpr int MT = BU / 16;          // 16-token tiles per unit
    constexpr int KP = D / 32;           // 32-dim steps of the scores
    constexpr int KS = D / 16;           // 16-dim chunks of the output
    constexpr int NH = G == 8 ? 2 : 1;   // heads per lane
    constexpr int NQ = G == 8 ? 2 : 1;   // MMAs per step: hi and lo apart, or as columns of one
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align_1024(smem_raw);
    if (p.wait_first) griddep_wait();

    const int per_seq = p.num_partitions * p.num_kv_heads;
    const int turn = blockIdx.x / per_seq;
    const int rem = blockIdx.x - turn * per_seq;
    const int part = rem / p.num_kv_heads;
    const int g = rem - part * p.num_kv_heads;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int s = p.length_shift < 0 ? turn : sequence_by_length<kThreads>(p.context_lens, p.num_seqs, p.length_shift, turn);

    const int ctx_raw = p.context_lens[s];
    const int nblk = decode_seq_blocks(ctx_raw, B, p.max_blocks_per_seq, p.num_partitions * p.partition_blocks,
                                       threadIdx.x == 0 && part == 0 && g == 0);
    const int ctx = min(max(ctx_raw, 0), nblk * B);
    const int nparts = nblk > 0 ? (nblk + p.partition_blocks - 1) / p.partition_blocks : 1;
    if (part >= nparts) return;
    const int b0 = part * p.partition_blocks;
    const int nb = max(0, min(nblk - b0, p.partition_blocks));
    const bool direct = nparts == 1;
    const int end = min(ctx - b0 * B, nb * B);  // keys of the partition; a unit may reach past it

    int* bt_s = reinterpret_cast<int*>(smem + C::BT_OFF);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + ((C::BT_OFF + p.partition_blocks * 4 + 15) & ~15));
    const int32_t* bt_row = p.block_tables + static_cast<int64_t>(s) * p.max_blocks_per_seq + b0;
    for (int i = threadIdx.x; i < nb; i += kThreads) {
        int id = bt_row[i];
        if (id < 0 || id >= p.num_blocks) {
            flag_error(PKV_DEVERR_BLOCK_ID);
            id = static_cast<int>(p.num_blocks);  // read as zeros
        }
        bt_s[i] = id;
    }
    if (lane == 0) {
#pragma unroll
        for (int st = 0; st < NST; ++st) mbar_init(&bars[warp * NST + st], 1);
        fence_mbar_init();
    }
    __syncthreads();

    const int nu = (nb + U - 1) / U;  // units of the partition
    const int nw = nu > warp ? (nu - warp + NW - 1) / NW : 0;
    uint8_t* wstage = smem + warp * NST * C::STAGE;
    float* wscale = reinterpret_cast<float*>(smem + C::SC_OFF) + warp * NST * C::SC_STAGE;
    uint64_t* wbar = bars + warp * NST;
    const uint64_t policy = l2_policy_evict_first();

    // A unit's copies, one per lane: lane 4 i + j takes block i's part j (K codes,
    // V codes, K scales, V scales).
    const CUtensorMap* my_map = &tm.m[lane & 3];
    const int my_block = lane >> 2;
    uint8_t* my_dst = (lane & 2) ? reinterpret_cast<uint8_t*>(wscale) + ((lane & 1) * U + my_block) * C::SC_BOX * 4
                                 : wstage + (lane & 1) * C::TILE + my_block * B * D;
    constexpr int kStageStep[2] = {C::STAGE, C::SC_STAGE * 4};
    const int my_step = (lane & 2) ? kStageStep[1] : kStageStep[0];
    auto issue = [&](int k) {  // whole warp
        const int st = k % NST;
        if (lane == 0) mbar_arrive_expect_tx(&wbar[st], C::TX);
        __syncwarp();
        if (lane < 4 * U) {
            const int bi = (warp + k * NW) * U + my_block;
            const int id = U > 1 && bi >= nb ? static_cast<int>(p.num_blocks) : bt_s[bi];  // beyond the pool: zero fill
            tma_load_4d_hint(my_dst + st * my_step, my_map, 0, g, 0, id, &wbar[st], policy);
        }
    };
    // The pools may still be in the writes of a grid this one depends on (the
    // append of a decode step): their loads start after it completes.
    griddep_wait();
    for (int k = 0; k < NST && k < nw; ++k) issue(k);

    // ---- the query as integers, while the first stages are in flight.  B
    // fragment column n = lane / 4 holds dims 32 kp + 4 (lane % 4) + {0..3} and
    // the same + 16; columns are (hi, lo) of head n / 2, or heads 0-7 twice.
    uint32_t qf[NQ][KP][2];
    int c_init[NQ][2];
    float qsl[NH];
    {
        const int col = lane >> 2;
        const int hq = G == 8 ? col : col >> 1;
        const T* qrow = reinterpret_cast<const T*>(p.query) +
                        (static_cast<int64_t>(s) * p.num_q_heads + static_cast<int64_t>(g) * G + hq) * D;
        float qv[KP][2][4];
        uint32_t top = 0;
#pragma unroll
        for (int kp = 0; kp < KP; ++kp) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int i = 0; i < 4; ++i) qv[kp][e][i] = 0.f;
                if (hq < G) load4(qrow + 32 * kp + 16 * e + 4 * (lane & 3), qv[kp][e]);
                top = max(top, absmax4(qv[kp][e]));
            }
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // an infinity or NaN in the row: a NaN scale, and a NaN result
        const float amax = top >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : __uint_as_float(top);
        const float inv = 32639.f / amax;
        int sum_hi = 0, sum_lo = 0;
#pragma unroll
        for (int kp = 0; kp < KP; ++kp) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                // Adding 1.5 * 2^23 + 128 rounds q to an integer and leaves
                // q + 128 in the sum's low 16 bits: the upper byte is hi, the
                // lower one lo + 128.  (A zero row has inv = inf: whatever
                // integers come out, its scale is 0.)
                uint32_t u[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) u[i] = __float_as_uint(fmaf(qv[kp][e][i], inv, 12583040.f));
                const uint32_t p01 = __byte_perm(u[0], u[1], 0x5140), p23 = __byte_perm(u[2], u[3], 0x5140);
                const uint32_t lo = __byte_perm(p01, p23, 0x5410) ^ 0x80808080u, hi = __byte_perm(p01, p23, 0x7632);
                sum_hi = __dp4a(static_cast<int>(hi), 0x01010101, sum_hi);
                sum_lo = __dp4a(static_cast<int>(lo), 0x01010101, sum_lo);
                if constexpr (G == 8) qf[0][kp][e] = hi, qf[NQ - 1][kp][e] = lo;
                else qf[0][kp][e] = (col & 1) ? lo : hi;
            }
        }
#pragma unroll
        for (int off = 1; off < 4; off <<= 1) {
            sum_hi += __shfl_xor_sync(0xffffffffu, sum_hi, off);
            sum_lo += __shfl_xor_sync(0xffffffffu, sum_lo, off);
        }
        // to the accumulator's layout: columns 2 (lane % 4) and the next
        const int c0 = 8 * (lane & 3), c1 = c0 + 4;
        const float qs = amax * (1.f / 32639.f) * p.scale_log2;
        if constexpr (G == 8) {
            c_init[0][0] = -128 * __shfl_sync(0xffffffffu, sum_hi, c0);
            c_init[0][1] = -128 * __shfl_sync(0xffffffffu, sum_hi, c1);
            c_init[NQ - 1][0] = -128 * __shfl_sync(0xffffffffu, sum_lo, c0);
            c_init[NQ - 1][1] = -128 * __shfl_sync(0xffffffffu, sum_lo, c1);
            qsl[0] = __shfl_sync(0xffffffffu, qs, c0);
            qsl[NH - 1] = __shfl_sync(0xffffffffu, qs, c1);
        } else {
            c_init[0][0] = -128 * __shfl_sync(0xffffffffu, sum_hi, c0);
            c_init[0][1] = -128 * __shfl_sync(0xffffffffu, sum_lo, c0);
            qsl[0] = __shfl_sync(0xffffffffu, qs, c0);
        }
    }

    float m[NH], l[NH];  // exponent base; this lane's share of the sum
#pragma unroll
    for (int h = 0; h < NH; ++h) m[h] = -INFINITY, l[h] = 0.f;
    // O^T: [chunk t][c0: (dim 16t + 2(lane/4), head A), c1: (same dim, head B), c2: (dim + 1, A), c3: (dim + 1, B)],
    // heads (A, B) = columns 2(lane%4) and the next; with up to four heads the odd columns are unused
    float o[KS][4];
#pragma unroll
    for (int t = 0; t < KS; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;

    const int lr = lane & 7, lm = lane >> 3;

    int k = 0;
    for (; k < nw; ++k) {
        const int st = k % NST;
        const bool ok = mbar_wait_main(&wbar[st], (k / NST) & 1);
        if (!__all_sync(0xffffffffu, ok)) break;
        {
            const int valid = end - (warp + k * NW) * BU;  // keys of the unit inside the partition, or more
            const uint8_t* Ks = wstage + st * C::STAGE;
            const uint8_t* Vs = Ks + C::TILE;
            const float* sk = wscale + st * C::SC_STAGE + (lane >> 2);
            float t[MT][2][NH], iv[MT][2];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                int acc[NQ][4];
#pragma unroll
                for (int q = 0; q < NQ; ++q)
                    acc[q][0] = acc[q][2] = c_init[q][0], acc[q][1] = acc[q][3] = c_init[q][1];
#pragma unroll
                for (int kp = 0; kp < KP; ++kp) {
                    uint32_t a[4];  // tokens g | g + 8, bytes 0-15 | 16-31 of the 32-dim step
                    ldsm_x4(a, Ks + int8_chunk<D>(16 * mt + lr + 8 * (lm & 1), 2 * kp + (lm >> 1)));
#pragma unroll
                    for (int q = 0; q < NQ; ++q) mma_16832_u8s8(acc[q], a, qf[q][kp][0], qf[q][kp][1]);
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int row = 16 * mt + 8 * r;  // + lane / 4
                    const float ks = sk[row / B * C::SC_BOX + row % B];
                    const float vs = max_nan(sk[(U + row / B) * C::SC_BOX + row % B], kInt8MinScale);
                    const float lv = lg2_approx(vs);
                    iv[mt][r] = rcp_approx(vs);
#pragma unroll
                    for (int h = 0; h < NH; ++h) {
                        const int dot = G == 8 ? 256 * acc[0][2 * r + h] + acc[NQ - 1][2 * r + h]
                                               : 256 * acc[0][2 * r] + acc[0][2 * r + 1];
                        t[mt][r][h] = fmaf(static_cast<float>(dot), ks * qsl[h], lv);
                    }
                }
            }
            if (valid < BU) {  // the partition ends in this unit: no weight, whatever the slots hold
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        if (16 * mt + 8 * r + (lane >> 2) >= valid) {
                            iv[mt][r] = 0.f;
#pragma unroll
                            for (int h = 0; h < NH; ++h) t[mt][r][h] = -INFINITY;
                        }
            }
            // ---- the base moves, and O and the sum are rescaled, only when a
            // unit exceeds it by more than 2^8: weights stay below 256
            bool grow = false;
            float bm[NH];
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                bm[h] = -INFINITY;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) bm[h] = fmaxf(bm[h], fmaxf(t[mt][0][h], t[mt][1][h]));
                grow = grow || bm[h] > m[h] + 8.f;
            }
            if (__any_sync(0xffffffffu, grow)) {
                float al[2] = {1.f, 1.f};
#pragma unroll
                for (int h = 0; h < NH; ++h) {
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1)
                        bm[h] = fmaxf(bm[h], __shfl_xor_sync(0xffffffffu, bm[h], off));
                    if (bm[h] > m[h] + 8.f) {
                        al[h] = ex2_approx(m[h] - bm[h]);  // 0 when m was -inf
                        m[h] = bm[h];
                        l[h] *= al[h];
                    }
                }
#pragma unroll
                for (int c = 0; c < KS; ++c) {
                    o[c][0] *= al[0];
                    o[c][2] *= al[0];
                    if constexpr (NH == 2) o[c][1] *= al[1], o[c][3] *= al[1];
                }
            }
            float w[MT][2][2];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    w[mt][r][1] = 0.f;
#pragma unroll
                    for (int h = 0; h < NH; ++h) {
                        w[mt][r][h] = ex2_approx(t[mt][r][h] - (m[h] == -INFINITY ? 0.f : m[h]));
                        l[h] = fmaf(w[mt][r][h], iv[mt][r], l[h]);
                    }
                }
            // ---- O^T += (V - 128)^T . P^T
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const uint32_t bh0 = movmatrix_trans(pack_half2(w[mt][0][0], w[mt][0][1]));
                const uint32_t bh1 = movmatrix_trans(pack_half2(w[mt][1][0], w[mt][1][1]));
#pragma unroll
                for (int jp = 0; jp < KP; ++jp) {
                    // bytes (tok 2c, dim 2g) (tok 2c, dim 2g+1) (tok 2c+1, dim 2g) (tok 2c+1, dim 2g+1) of
                    // r[0]: chunk 2jp; r[1]: tokens + 8; r[2], r[3]: chunk 2jp + 1
                    uint32_t r[4];
                    ldsm_x4_trans(r, Vs + int8_chunk<D>(16 * mt + lr + 8 * (lm & 1), 2 * jp + (lm >> 1)));
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t a[4] = {hsub2_1152(__byte_perm(r[2 * h], 0x64646464u, 0x4240)),
                                               hsub2_1152(__byte_perm(r[2 * h], 0x64646464u, 0x4341)),
                                               hsub2_1152(__byte_perm(r[2 * h + 1], 0x64646464u, 0x4240)),
                                               hsub2_1152(__byte_perm(r[2 * h + 1], 0x64646464u, 0x4341))};
                        mma_16816<false>(o[2 * jp + h], a, bh0, bh1);
                    }
                }
            }
        }
        __syncwarp();
        if (k + NST < nw) {
            fence_proxy_async();
            issue(k + NST);
        }
    }
    if (k < nw && lane == 0) {
        // a wait gave up: wait (bounded) for this warp's copies still in flight, stage k's included
        for (int kk = k; kk < min(nw, k + NST); ++kk) mbar_wait(&wbar[kk % NST], (kk / NST) & 1);
    }
#pragma unroll
    for (int h = 0; h < NH; ++h) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], off);
        if (k < nw) m[h] = -INFINITY, l[h] = 0.f;
        if (isnan(l[h]) && m[h] == -INFINITY) m[h] = 0.f;  // only NaN scores: the merge must not take it for empty
    }

    // ---- hand this warp's state to the CTA merge
    __syncthreads();
    float* red_m = reinterpret_cast<float*>(smem);
    float* red_l = red_m + NW * G;
    float* red_o = red_l + NW * G;
#pragma unroll
    for (int h = 0; h < NH; ++h) {
        const int head = NH * (lane & 3) + h;
        if (head < G) {
            if (lane < 4) red_m[warp * G + head] = m[h], red_l[warp * G + head] = l[h];
#pragma unroll
            for (int c = 0; c < KS; ++c) {
                const int d = 16 * c + 2 * (lane >> 2);
                red_o[(warp * G + head) * D + d] = o[c][h];
                red_o[(warp * G + head) * D + d + 1] = o[c][2 + h];
            }
        }
    }
    __syncthreads();
    decode_finish<T, D, G, NW>(p, red_m, s, g, part, direct);
}

}  // namespace pkv
