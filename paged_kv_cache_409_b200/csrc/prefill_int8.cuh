// prefill_int8.cuh -- causal chunked-prefill attention over int8 pools on the
// tcgen05 tensor cores: the pipeline of prefill.cuh (two query tiles of 128
// rows per CTA, S and P in tensor memory, one softmax thread per row) with the
// K and V tiles widened in shared memory by warps of their own, so that the
// cache is read once, as it lies, and no scratch is needed.
//
// fp16 queries: exact codes.  Tile rows arrive as codes (16 KB at head_dim 128)
// with one fp32 scale each.  A converter thread turns four codes into two f16 pairs:
// a byte permute puts 0x64 over each code (1024 + u), a subtraction of 1152 leaves
// u - 128 exactly.  The scales go into the softmax, as in decode_int8.cuh: K's
// multiplies its column of S, the logarithm of V's is added to the exponent, and
// the sum takes each weight over V's scale.  So P is near 1 for the largest
// product whatever the rows' sizes are, and only P and the result are rounded: an
// fp16 result is off by 2.6-2.9e-4 of its norm against 64 bits, where an fp32 form
// rounded once is off by 2.1e-4 and elements rounded to f16 (below) come to
// 4.7-7.0e-4.  Three 16-byte reads and two packed FMAs more for four scores: four
// chunks of 512 rows (below) 206 us against 168, seven ragged ones 22.9 against 22.1.
//
// bf16 queries: elements rounded to f16, whose error (2^-11 of an element) is well
// below the result's own rounding (2^-8).  A byte permute puts 0x48 over a code (8 +
// u / 128), a subtraction of 9 leaves c = (u - 128) / 128 exactly, and the element is
// c * hi + c * lo with S, 128 times the scale in the units below, split in two f16
// parts (2^-22 of it), so that what is rounded is the product.
// Units.  f16 keeps those 11 bits over 30 binades only, and rows may be of any
// size: rows of 1e-4 taken as they are came out 4 % off (the split itself fell
// on the subnormal grid), rows of 3e-6 as zeros.  So the loader, which has a
// tile's 128 scales in a warp's registers, gives every K tile a power of two of
// its own that puts the largest S at 2^14 or above (never 2^15), and V a running
// one, 2^12 or above for the largest row so far, which only grows: the scores
// are multiplied back with the scale they take anyway, and O is rescaled, as for
// a new maximum, in the few tiles where V's unit grows.  An f16 subnormal is then
// below 2^-35 of the largest such row.  Query rows are narrowed in units of their
// own likewise.  All of it costs the softmax one 16-byte read and two
// multiplications a tile.
//
// Rows past the sequence and those of bad blocks have finite tile elements (bf16:
// zeros), since 0 * NaN must not reach O.  For the same reason a row of scale NaN
// (bf16: or beyond f16's largest value / 127) shows in its scores alone, K and V
// rows both: those that the causal mask hides stay out of it.
//
// Roles (512 threads; the registers of the second half go to the softmax):
//   warps 0-7   softmax, four per query tile, as in prefill.cuh; with bf16
//               queries they first turn the two Q tiles into f16 in place
//   warp 8      loader: Q tiles, then the codes and scales of K_j and V_j into
//               one staging buffer each, refilled when it has been widened
//   warp 9      MMA issue
//   warp 10     fp16: what the softmax takes of the scales, a tile ahead (K's factors
//               and V's logarithms in two stages, V's inverses, read last, in one)
//   warps 12-15 converters: staging -> f16 K (two stages) and V (two stages)
// Every wait is bounded, as in prefill.cuh.
//
// Few items.  An item is (pair of query tiles, chunk, KV head); where the launch
// has few of them, each goes to a cluster of CTAs that share out its key tiles.
// Their partial O, row maxima and sums meet in shared memory: every CTA merges
// a share of the rows from all of the cluster's (distributed shared memory), so
// that no scratch is needed for this either.
//
// Bound by the chain of a query tile's steps (S, softmax, P.V: 2.25 us per 128
// keys for two tiles, of which the tensor cores work 1.5): four chunks of 512
// rows over up to 8446 keys, 32 query heads on 8 KV heads of 128, bf16, 167 us, 701
// TFLOP/s (0.43 of the bf16 rate), set by the items of 66 key tiles.  In the
// chain it is the softmax threads' issue slots and latency that count, not the
// exponential unit: a polynomial for an eighth, a quarter, half of the
// exponentials took 170, 180, 194 us, P handed over in two halves 190, scores
// read again from tensor memory in loops of 32 to 128 columns 179-195.
#pragma once

#include "decode_int8.cuh"
#include "prefill.cuh"

namespace pkv {

struct PrefillInt8Params {
    PrefillParams base;
    const uint8_t* k_scales;  // scales of block 0
    const uint8_t* v_scales;
    int64_t block_bytes;
    int total_q_tokens;
};

constexpr int kPrefillInt8Threads = 512;
#ifndef PKV_PREFILL_WIDEN_UNROLL
#define PKV_PREFILL_WIDEN_UNROLL 1  // 2, 4, 8: slower, the loops compete for the instruction caches
#endif
#ifndef PKV_PREFILL_CONV_REGS
#define PKV_PREFILL_CONV_REGS 64  // registers of the second half's threads; the softmax gets 256 minus this
#endif
constexpr int kPrefillInt8ScaleWarp = 10;  // fp16 queries
constexpr int kPrefillInt8ConvWarp = 12;   // first of four
constexpr int kPrefillInt8ConvThreads = 128;

template <int D, int G>
struct PrefillInt8Cfg {
    static constexpr int BM = 128, TT = BM / G, BN = 128;
    static constexpr int NP = D / 64;               // 128-byte panels per f16 row
    static constexpr int Q_BYTES = NP * BM * 128;   // one query tile
    static constexpr int KT_BYTES = NP * BN * 128;  // one f16 K (or V) tile
    static constexpr int C_BYTES = BN * D;          // the codes of a tile
    static constexpr int Q_OFF = 0;
    static constexpr int K_OFF = Q_OFF + 2 * Q_BYTES;    // [2] stages
    static constexpr int V_OFF = K_OFF + 2 * KT_BYTES;   // [2] stages
    static constexpr int KC_OFF = V_OFF + 2 * KT_BYTES;  // staging of K, then of V
    static constexpr int VC_OFF = KC_OFF + C_BYTES;
    // scales.  bf16: K [BN], V [2][BN] (tile j in j & 1), and the units of tile j
    // [4] in j & 3; fp16: K's factors [2][BN], log2 of V's [2][BN], V's inverses [BN]
    static constexpr int SC_OFF = VC_OFF + C_BYTES;
    static constexpr int UNIT_OFF = SC_OFF + 3 * BN * 4;
    static constexpr int IV_OFF = SC_OFF + 4 * BN * 4;
    static constexpr int BAR_OFF = SC_OFF + 5 * BN * 4;
    static constexpr int NBAR = 33;
    static constexpr int SMEM = BAR_OFF + NBAR * 8;
    static constexpr uint32_t TMEM_COLS = 512, S_COL0 = 0, O_COL0 = 256;
    static_assert(SMEM <= 227 * 1024, "shared memory");
    // the cluster's merge: O [256][D] in fp32 (16-byte chunks swizzled by row), then (max, sum) per row
    static constexpr int ML_OFF = 256 * D * 4;
    static constexpr int W_OFF = ML_OFF + 256 * 8;  // the merge's weights, [128][8]
    static_assert(W_OFF + 128 * 32 <= KC_OFF, "merge scratch");
};

// ---- thread-block clusters
__device__ __forceinline__ int cluster_size() {
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
    return static_cast<int>(n);
}
__device__ __forceinline__ int cluster_rank() {
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(n));
    return static_cast<int>(n);
}
// Every thread of every CTA of the cluster, its writes before it visible after it.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// This CTA's shared address `a` in the CTA of the given rank.
__device__ __forceinline__ uint32_t cluster_map(uint32_t a, int rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    return r;
}
__device__ __forceinline__ float4 cluster_ld4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ float2 cluster_ld2(uint32_t a) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a));
    return v;
}

template <int kRegs>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs)); }
template <int kRegs>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs)); }

__device__ __forceinline__ uint32_t hmul2_u(uint32_t a, uint32_t b) {
    uint32_t y;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
}
__device__ __forceinline__ uint32_t hfma2_u(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t y;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(a), "r"(b), "r"(c));
    return y;
}

__device__ __forceinline__ uint32_t hsub2_9(uint32_t x) {
    uint32_t y;
    asm("add.f16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(0xC880C880u));
    return y;
}

// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// The binade of a positive finite float's bits, no less than -100 (zeros, and
// what would take a unit's inverse out of fp32).
__device__ __forceinline__ int binade(uint32_t bits) { return max(static_cast<int>(bits >> 23) - 127, -100); }

// Four codes (one 32-bit word), as (u - 128) / 128, times a number split in two f16 parts.
__device__ __forceinline__ uint2 widen_codes4(uint32_t u, uint32_t s_hi, uint32_t s_lo) {
    const uint32_t a = hsub2_9(__byte_perm(u, 0x48484848u, 0x4140));
    const uint32_t b = hsub2_9(__byte_perm(u, 0x48484848u, 0x4342));
    return make_uint2(hfma2_u(a, s_hi, hmul2_u(a, s_lo)), hfma2_u(b, s_hi, hmul2_u(b, s_lo)));
}

// Four codes as u - 128.
__device__ __forceinline__ uint2 exact_codes4(uint32_t u) {
    return make_uint2(hsub2_1152(__byte_perm(u, 0x64646464u, 0x4140)), hsub2_1152(__byte_perm(u, 0x64646464u, 0x4342)));
}

// T: the query's and output's type; the MMAs run in f16.
template <typename T, int D, int G>
__global__ void __launch_bounds__(kPrefillInt8Threads, 1)
    paged_prefill_int8_kernel(const PrefillInt8Params prm, const __grid_constant__ CUtensorMap tm_q,
                              const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
    using C = PrefillInt8Cfg<D, G>;
    const PrefillParams& p = prm.base;
    const int B = p.block_size;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
    constexpr bool kNarrowQ = Elem<T>::kCuType == CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    constexpr bool kExact = !kNarrowQ;  // the tiles hold the codes, the softmax takes the scales
    uint64_t* q_full = bars + 0;
    uint64_t* q_ready = bars + 1;   // Q tiles in f16 (256 arrivals; bf16 queries)
    uint64_t* c_full = bars + 2;    // [2] codes of K and both scales | codes of V landed
    uint64_t* c_free = bars + 4;    // [2] widened (128 arrivals)
    uint64_t* k_full = bars + 6;    // [2] f16 K tile written (128 arrivals)
    uint64_t* k_free = bars + 8;    // [2] the S MMAs that read the stage are done
    uint64_t* v_full = bars + 10;   // [2]
    uint64_t* v_free = bars + 12;   // [2]
    uint64_t* s_full = bars + 14;   // [2] per tile: S_x(j) done
    uint64_t* p_full = bars + 16;   // [2] per tile: P_x(j) written (128 arrivals)
    uint64_t* o_full = bars + 18;   // [2] per tile: the tile's last P.V done
    uint64_t* mma_done = bars + 20;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 21);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 22);
    uint64_t* u_full = bars + 23;   // [4] units of tile j written, in j & 3 (bf16)
    uint64_t* f_full = bars + 23;   // [2] K's factors and V's logarithms of tile j written, in j & 1 (fp16)
    uint64_t* f_free = bars + 25;   // [2][2] per query tile: read (4 arrivals)
    uint64_t* i_full = bars + 29;   // V's inverses of tile j written (fp16)
    uint64_t* i_free = bars + 30;   // [2] per query tile: read (4 arrivals)

    griddep_wait();  // launched as a dependent of whatever comes before it
    const int parts = cluster_size(), rank = cluster_rank();
    const int cluster = static_cast<int>(blockIdx.x) / parts;
    const int g = cluster % p.num_kv_heads;
    const int item = cluster / p.num_kv_heads;
    int r, pair;
    if (p.num_chunks <= kLptChunks) {
        if (!prefill_item(p.seq_lens, p.query_start_loc, p.num_chunks, C::TT, p.tile_pairs, item, r, pair)) return;
    } else {
        pair = p.tile_pairs - 1 - item / p.num_chunks;
        r = item % p.num_chunks;
    }
    const int tid = threadIdx.x;
    const int warp = tid >> 5;

    const int q0 = p.query_start_loc[r];
    const int n = p.query_start_loc[r + 1] - q0;
    const int L = p.seq_lens[r];
    const int c0 = L - n;
    const bool bad = n < 0 || c0 < 0 || q0 < 0 || q0 + static_cast<int64_t>(n) > prm.total_q_tokens ||
                     L > p.max_blocks_per_seq * B;
    if (bad || n > 2 * p.tile_pairs * C::TT) {  // the latter is cut to the call's bound
        if (tid == 0 && pair == 0 && g == 0 && rank == 0) flag_error(PKV_DEVERR_LENGTH);
        if (bad) return;
    }
    const int qt0 = 2 * pair;
    if (qt0 * C::TT >= n) return;
    const bool has_b = (qt0 + 1) * C::TT < n;
    const int nkt_a = (c0 + min((qt0 + 1) * C::TT, n) - 1) / C::BN + 1;
    const int nkt_b = has_b ? (c0 + min((qt0 + 2) * C::TT, n) - 1) / C::BN + 1 : 0;
    // this CTA's share of the key tiles, [tb, tb + nkt), and how many of it each query tile needs
    const int all = max(nkt_a, nkt_b);
    const int tb = rank * all / parts;
    const int nkt = (rank + 1) * all / parts - tb;
    const int nka = min(max(nkt_a - tb, 0), nkt), nkb = min(max(nkt_b - tb, 0), nkt);
    const int nblk = (L + B - 1) / B;
    const int32_t* bt_row = p.block_tables + static_cast<int64_t>(r) * p.max_blocks_per_seq;

    if (warp == 0) {
        tmem_alloc(tmem_slot, C::TMEM_COLS);
        tmem_relinquish();
    }
    if (tid == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_ready, 256);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&c_full[i], 1);
            mbar_init(&c_free[i], kPrefillInt8ConvThreads);
            mbar_init(&k_full[i], kPrefillInt8ConvThreads);
            mbar_init(&v_full[i], kPrefillInt8ConvThreads);
            mbar_init(&k_free[i], 1);
            mbar_init(&v_free[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 128);
            mbar_init(&o_full[i], 1);
        }
        if constexpr (kExact) {
            for (int i = 0; i < 2; ++i) {
                mbar_init(&f_full[i], 1);
                mbar_init(&f_free[i], 4);
                mbar_init(&f_free[2 + i], 4);
                mbar_init(&i_free[i], 4);
            }
            mbar_init(i_full, 1);
        } else {
            for (int i = 0; i < 4; ++i) mbar_init(&u_full[i], 1);
        }
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // 512 threads launch with 128 registers each; half of them hand 64 of
    // theirs to the softmax threads, which hold a row of 128 scores:
    // 256 * 192 + 256 * 64 = 512 * 128.
    if (warp >= 8) {
        regs_dec<PKV_PREFILL_CONV_REGS>();
        // For the warps that follow the block table.  Block ids of this CTA's key
        // tile j, one per lane; read one tile ahead.
        const int lane = tid & 31;
        const int per_tile = C::BN / B;  // blocks per key tile (4..16)
        auto fetch_ids = [&](int j) -> int {
            const int lb = (tb + j) * per_tile + lane;
            return (lane < per_tile && lb < nblk) ? bt_row[lb] : -1;
        };
        // Ids checked when they arrive; -1: nothing to load (the tiles behind
        // this CTA's last are another's to check and flag).
        auto checked_ids = [&](int j, int id, bool flag) -> int {
            if (lane >= per_tile || j >= nkt || (tb + j) * per_tile + lane >= nblk) return -1;
            if (id >= 0 && id < p.num_blocks) return id;
            if (flag) flag_error(PKV_DEVERR_BLOCK_ID);
            return -1;
        };
        // The tile's scales, four K and four V rows per lane, into registers a
        // tile ahead of their use (copies of 32 to 128 bytes each would cost as
        // many bulk copies as the codes); rows of blocks that are not loaded
        // get 0: zeros.
        auto fetch_scales = [&](int id, float4& ks, float4& vs) {
            const int own = __shfl_sync(0xffffffffu, id, 4 * lane / B);
            ks = vs = make_float4(0.f, 0.f, 0.f, 0.f);
            if (own >= 0) {
                const int64_t off = own * prm.block_bytes + (g * B + (4 * lane) % B) * 4;
                ks = *reinterpret_cast<const float4*>(prm.k_scales + off);
                vs = *reinterpret_cast<const float4*>(prm.v_scales + off);
            }
        };
        if (warp == kPrefillLoadWarp) {
            // ============================================================ loader (whole warp, lane 0 issues)
            const bool leader = lane == 0;
            float* scales = reinterpret_cast<float*>(smem + C::SC_OFF);
            // The largest scale a row may have: fp16's largest value / 127, and what
            // the rounding of a scale adds.
            constexpr float kMaxScale = 65504.f / 127.f * (1.f + 0x1p-20f);
            int v_unit = -103;  // below every binade: the first tile sets it
            // The fetched scales of tile j in its units, on their way to the
            // converters (rows past the sequence 0; rows that do not fit: K NaN, V
            // 0), and the units for the softmax: (K's, V's, V's last over V's, -).
            auto scale_units = [&](int j, float4& ks4, float4& vs4) -> float4 {
                float ks[4] = {ks4.x, ks4.y, ks4.z, ks4.w}, vs[4] = {vs4.x, vs4.y, vs4.z, vs4.w};
                const int live = L - ((tb + j) * C::BN + 4 * lane);
                uint32_t k_top = 0, v_top = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (i >= live) {
                        ks[i] = vs[i] = 0.f;
                    } else if (!(fabsf(ks[i]) <= kMaxScale && fabsf(vs[i]) <= kMaxScale)) {
                        ks[i] = __uint_as_float(0x7fc00000u), vs[i] = 0.f;
                    } else {
                        k_top = max(k_top, abs_bits(ks[i])), v_top = max(v_top, abs_bits(vs[i]));
                    }
                }
                const int k_unit = binade(__reduce_max_sync(0xffffffffu, k_top));
                const int v_new = binade(__reduce_max_sync(0xffffffffu, v_top));
                float grown = 1.f;
                if (v_new > v_unit + 2) {  // S would pass 2^15
                    grown = pow2(v_unit - v_new);
                    v_unit = v_new;
                }
                const float km = pow2(14 - k_unit), vm = pow2(12 - v_unit);
                ks4 = make_float4(ks[0] * km, ks[1] * km, ks[2] * km, ks[3] * km);
                vs4 = make_float4(vs[0] * vm, vs[1] * vm, vs[2] * vm, vs[3] * vm);
                return make_float4(pow2(k_unit - 7), pow2(v_unit - 5), grown, 0.f);
            };
            // The codes of a tile, K (0) or V (1): lane i copies block i.
            auto load_codes = [&](int which, const CUtensorMap* map, int id) {
                if (leader) mbar_arrive_expect_tx(&c_full[which], C::C_BYTES);
                __syncwarp();
                if (lane < per_tile) {
                    fence_proxy_async();  // the converters' reads before the next copies
                    tma_load_4d(smem + (which ? C::VC_OFF : C::KC_OFF) + lane * B * D, map, 0, g, 0,
                                id >= 0 ? id : static_cast<int>(p.num_blocks), &c_full[which]);  // out of range: zero fill
                }
                __syncwarp();
            };
            if (leader && nkt > 0) {
                mbar_arrive_expect_tx(q_full, (has_b ? 2 : 1) * C::Q_BYTES);
                for (int x = 0; x < (has_b ? 2 : 1); ++x) {
#pragma unroll
                    for (int pn = 0; pn < C::NP; ++pn)
                        tma_load_3d(smem + C::Q_OFF + x * C::Q_BYTES + pn * C::BM * 128, &tm_q, pn * 64, g * G,
                                    q0 + (qt0 + x) * C::TT, q_full);
                }
            }
            int ids = checked_ids(0, fetch_ids(0), true);
            int ids_next = fetch_ids(1);
            float4 ks, vs, units;
            if constexpr (!kExact) fetch_scales(ids, ks, vs);
            int loaded_k = 0, loaded_v = 0;
            for (int j = 0; j < nkt; ++j) {
                const int ids_later = fetch_ids(j + 2);
                if constexpr (!kExact) units = scale_units(j, ks, vs);
                if (j > 0 && !__all_sync(0xffffffffu, mbar_wait_or_abort_idle(&c_free[0], (j - 1) & 1, abort_flag))) break;
                if constexpr (!kExact) {
                    *reinterpret_cast<float4*>(scales + 4 * lane) = ks;
                    *reinterpret_cast<float4*>(scales + (1 + (j & 1)) * C::BN + 4 * lane) = vs;
                    // Read by the softmax threads of tile j, which are done with it before
                    // S(j + 1) runs, whose K stage tile j + 3 is widened into: j + 4 may
                    // overwrite it.
                    if (leader) {
                        *reinterpret_cast<float4*>(smem + C::UNIT_OFF + (j & 3) * 16) = units;
                        mbar_arrive(&u_full[j & 3]);
                    }
                    __syncwarp();
                }
                load_codes(0, &tm_k, ids);
                loaded_k = j + 1;
                if (j > 0 && !__all_sync(0xffffffffu, mbar_wait_or_abort_idle(&c_free[1], (j - 1) & 1, abort_flag))) break;
                load_codes(1, &tm_v, ids);
                loaded_v = j + 1;
                ids = checked_ids(j + 1, ids_next, true);
                if constexpr (!kExact) fetch_scales(ids, ks, vs);
                ids_next = ids_later;
            }
            if (leader) {
                // wait (bounded) for this warp's last copies before the CTA may exit
                if (nkt > 0) mbar_wait(q_full, 0);
                if (loaded_k > 0) mbar_wait(&c_full[0], (loaded_k - 1) & 1);
                if (loaded_v > 0) mbar_wait(&c_full[1], (loaded_v - 1) & 1);
            }
        } else if (warp == kPrefillMmaWarp) {
            // ============================================================ MMA issue (lane 0)
            if ((tid & 31) == 0) {
                constexpr uint32_t IDESC_S = umma_idesc_f16(128, C::BN, false, false, false);
                constexpr uint32_t IDESC_O = umma_idesc_f16(128, D, false, false, true);
                uint64_t qdesc[2], kdesc[2], vdesc[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    qdesc[i] = smem_desc_sw128(smem_u32(smem + C::Q_OFF + i * C::Q_BYTES), 16, 1024);
                    kdesc[i] = smem_desc_sw128(smem_u32(smem + C::K_OFF + i * C::KT_BYTES), 16, 1024);
                    vdesc[i] = smem_desc_sw128(smem_u32(smem + C::V_OFF + i * C::KT_BYTES), C::BN * 128, 1024);
                }
                auto issue_s = [&](int x, int t) {  // S_x(t) = Q_x . K_t^T
                    const uint64_t qd = x ? qdesc[1] : qdesc[0], kd = (t & 1) ? kdesc[1] : kdesc[0];
                    const uint32_t s_col = C::S_COL0 + 128 * x;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        constexpr int kQ = C::BM * 128 / 16, kK = C::BN * 128 / 16;  // panel strides / 16
                        umma_f16_ss(tmem + s_col, qd + (kk / 4) * kQ + (kk % 4) * 2, kd + (kk / 4) * kK + (kk % 4) * 2,
                                    IDESC_S, kk > 0);
                    }
                    umma_commit(&s_full[x]);
                };
                auto issue_pv = [&](int x, int t, bool last) {  // O_x += P_x(t) . V_t, P from tensor memory
                    const uint64_t vd = (t & 1) ? vdesc[1] : vdesc[0];
                    const uint32_t p_col = C::S_COL0 + 128 * x, o_col = C::O_COL0 + D * x;
#pragma unroll
                    for (int kk = 0; kk < C::BN / 16; ++kk)
                        umma_f16_ts(tmem + o_col, tmem + p_col + kk * 8, vd + kk * (16 * 128 / 16), IDESC_O,
                                    t > 0 || kk > 0);
                    if (last) umma_commit(&o_full[x]);
                };
                bool ok = nkt > 0 && mbar_wait_or_abort(kNarrowQ ? q_ready : q_full, 0, abort_flag) &&
                          mbar_wait_or_abort(&k_full[0], 0, abort_flag);
                if (ok) {
                    tc_fence_after();
                    if (nka > 0) issue_s(0, 0);
                    if (nkb > 0) issue_s(1, 0);
                    umma_commit(&k_free[0]);
                }
                for (int t = 0; ok && t < nkt; ++t) {
                    const bool next = t + 1 < nkt;
                    bool k_next = false;
                    ok = mbar_wait_or_abort(&v_full[t & 1], (t >> 1) & 1, abort_flag);
#pragma unroll 1  // one copy of the MMA code for both tiles
                    for (int x = 0; ok && x < 2; ++x) {
                        const int nk = x == 0 ? nka : nkb;
                        if (t >= nk) continue;
                        ok = mbar_wait_or_abort(&p_full[x], t & 1, abort_flag);
                        if (!ok) break;
                        tc_fence_after();
                        issue_pv(x, t, t + 1 == nk);
                        if (t + 1 < nk) {
                            if (!k_next) {
                                ok = k_next = mbar_wait_or_abort(&k_full[(t + 1) & 1], ((t + 1) >> 1) & 1, abort_flag);
                                if (!ok) break;
                                tc_fence_after();
                            }
                            issue_s(x, t + 1);
                        }
                    }
                    if (ok) {
                        umma_commit(&v_free[t & 1]);
                        if (next) umma_commit(&k_free[(t + 1) & 1]);
                    }
                }
                umma_commit(mma_done);  // every MMA done before tensor memory is released
                mbar_wait(mma_done, 0);
            }
        } else if (kExact && warp == kPrefillInt8ScaleWarp) {
            // ============================================================ scales (fp16): what the softmax takes of them
            float* factors = reinterpret_cast<float*>(smem + C::SC_OFF) + 4 * lane;
            int ids_next = fetch_ids(1);
            float4 ks, vs;
            fetch_scales(checked_ids(0, fetch_ids(0), false), ks, vs);
            for (int j = 0; j < nkt; ++j) {
                const int ids_later = fetch_ids(j + 2), st = j & 1;
                float k[4] = {ks.x, ks.y, ks.z, ks.w}, v[4] = {vs.x, vs.y, vs.z, vs.w}, lg[4];
                const int live = L - ((tb + j) * C::BN + 4 * lane);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    k[i] *= p.scale_log2;
                    if (i >= live) k[i] = 0.f, v[i] = 1.f;
                    // a row that is not finite shows in the scores alone
                    if (!(abs_bits(k[i]) < 0x7f800000u && abs_bits(v[i]) < 0x7f800000u)) k[i] = __uint_as_float(0x7fc00000u), v[i] = 1.f;
                    v[i] = fmaxf(v[i], kInt8MinScale);
                    lg[i] = log2f(v[i]);
                }
                bool ok = true;
                for (int x = 0; x < 2; ++x)
                    if (j >= 2 && j - 2 < (x == 0 ? nka : nkb))
                        ok = ok && mbar_wait_or_abort_idle(&f_free[2 * x + st], ((j - 2) >> 1) & 1, abort_flag);
                if (!__all_sync(0xffffffffu, ok)) break;
                *reinterpret_cast<float4*>(factors + st * C::BN) = make_float4(k[0], k[1], k[2], k[3]);
                *reinterpret_cast<float4*>(factors + (2 + st) * C::BN) = make_float4(lg[0], lg[1], lg[2], lg[3]);
                __syncwarp();
                if (lane == 0) mbar_arrive(&f_full[st]);
                for (int x = 0; x < 2; ++x)
                    if (j >= 1 && j - 1 < (x == 0 ? nka : nkb))
                        ok = ok && mbar_wait_or_abort_idle(&i_free[x], (j - 1) & 1, abort_flag);
                if (!__all_sync(0xffffffffu, ok)) break;
                *reinterpret_cast<float4*>(smem + C::IV_OFF + 16 * lane) = make_float4(1.f / v[0], 1.f / v[1], 1.f / v[2], 1.f / v[3]);
                __syncwarp();
                if (lane == 0) mbar_arrive(i_full);
                fetch_scales(checked_ids(j + 1, ids_next, false), ks, vs);
                ids_next = ids_later;
            }
        } else if (warp >= kPrefillInt8ConvWarp) {
            // ============================================================ converters
            const int ct = tid - kPrefillInt8ConvWarp * 32;
            const float* scales = reinterpret_cast<const float*>(smem + C::SC_OFF);
            // Widen the staged codes of key tile j into an f16 tile, a row per
            // thread.  Row r of the code tile is swizzled over D bytes, the f16
            // tile is D / 64 panels of 128-byte rows, swizzled over 128 bytes:
            // eight neighbouring lanes touch eight different 16-byte columns
            // of either.
            const int row = ct, sw = row & 7;
            auto widen = [&](int which, int j, uint8_t* dst) {
                const uint8_t* src = smem + (which ? C::VC_OFF : C::KC_OFF);
                const float s = kExact ? 0.f : scales[(which ? 1 + (j & 1) : 0) * C::BN + row];
                const __half hi = __float2half_rn(s);
                const __half2 hi2 = __half2half2(hi), lo2 = __half2half2(__float2half_rn(s - __half2float(hi)));
                const uint32_t sh = *reinterpret_cast<const uint32_t*>(&hi2);
                const uint32_t sl = *reinterpret_cast<const uint32_t*>(&lo2);
                uint8_t* out = dst + row * 128;
                constexpr int kUnroll = PKV_PREFILL_WIDEN_UNROLL;
#pragma unroll kUnroll
                for (int ch = 0; ch < D / 16; ++ch) {
                    const uint4 u = *reinterpret_cast<const uint4*>(src + int8_chunk<D>(row, ch));
                    auto widen4 = [&](uint32_t w) { return kExact ? exact_codes4(w) : widen_codes4(w, sh, sl); };
                    const uint2 a = widen4(u.x), b = widen4(u.y), c = widen4(u.z), d = widen4(u.w);
                    uint8_t* panel = out + (ch / 4) * C::BN * 128;
                    const int v0 = 2 * (ch % 4);
                    *reinterpret_cast<uint4*>(panel + ((v0 ^ sw) << 4)) = make_uint4(a.x, a.y, b.x, b.y);
                    *reinterpret_cast<uint4*>(panel + (((v0 + 1) ^ sw) << 4)) = make_uint4(c.x, c.y, d.x, d.y);
                }
                fence_proxy_async();  // the f16 tile -> the tensor cores' (async) proxy
            };
            for (int j = 0; j < nkt; ++j) {
                const int st = j & 1;
                if (!__all_sync(0xffffffffu, mbar_wait_or_abort_idle(&c_full[0], j & 1, abort_flag))) break;
                if (j >= 2 && !__all_sync(0xffffffffu, mbar_wait_or_abort_idle(&k_free[st], ((j - 2) >> 1) & 1, abort_flag)))
                    break;
                widen(0, j, smem + C::K_OFF + st * C::KT_BYTES);
                mbar_arrive(&c_free[0]);
                mbar_arrive(&k_full[st]);
                if (!__all_sync(0xffffffffu, mbar_wait_or_abort_idle(&c_full[1], j & 1, abort_flag))) break;
                if (j >= 2 && !__all_sync(0xffffffffu, mbar_wait_or_abort_idle(&v_free[st], ((j - 2) >> 1) & 1, abort_flag)))
                    break;
                widen(1, j, smem + C::V_OFF + st * C::KT_BYTES);
                mbar_arrive(&c_free[1]);
                mbar_arrive(&v_full[st]);
            }
        }
        if (parts > 1) {  // the other roles' share of the merge's barriers
            __syncwarp();
            __syncthreads();
            cluster_sync();
            cluster_sync();
        }
    } else {
        regs_inc<256 - PKV_PREFILL_CONV_REGS>();
        // ================================================================ softmax: one thread per row
        const int x = warp >> 2;
        const int row = (warp & 3) * 32 + (tid & 31);
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const int tok = (qt0 + x) * C::TT + row / G;
        const int qpos = c0 + tok;
        const int nk = x == 0 ? nka : nkb;
        const uint32_t ts = tmem + lane_base + C::S_COL0 + 128 * x;
        const uint32_t to = tmem + lane_base + C::O_COL0 + D * x;
        float q_unit = 1.f, v_unit = 1.f;  // of this thread's query row; of O
        constexpr float kRescaleLog2 = 8.f;
        float m_used = -INFINITY, lsum = 0.f;
        bool ok = true;
        if constexpr (kNarrowQ) {  // this warpgroup's Q tile to f16, in place
            ok = nkt > 0 && __all_sync(0xffffffffu, mbar_wait_or_abort(q_full, 0, abort_flag));
            if (ok) {
                if (x == 0 || has_b) {
                    // A row per thread: its largest element, then every element in
                    // the row's unit (16-byte columns in the order of the swizzle:
                    // eight lanes touch eight different ones).
                    uint8_t* q = smem + C::Q_OFF + x * C::Q_BYTES + row * 128;
                    uint32_t top2 = 0;
#pragma unroll 4
                    for (int c = 0; c < D / 8; ++c) {
                        const uint4 v = *reinterpret_cast<const uint4*>(q + (c >> 3) * C::BM * 128 + (((c ^ row) & 7) << 4));
                        top2 = __vmaxu2(__vmaxu2(top2, __vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu)),
                                        __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
                    }
                    const uint32_t top = max(top2 & 0xffffu, top2 >> 16) << 16;
                    float mul = 1.f;
                    if (top < 0x7f800000u) {  // else NaN or an infinity, which shows in the result
                        q_unit = pow2(binade(top) - 14);
                        mul = pow2(14 - binade(top));
                    }
#pragma unroll 4
                    for (int c = 0; c < D / 8; ++c) {
                        uint4* at = reinterpret_cast<uint4*>(q + (c >> 3) * C::BM * 128 + (((c ^ row) & 7) << 4));
                        const uint4 v = *at;
                        auto narrow = [&](uint32_t u) {
                            const float2 f = Elem<__nv_bfloat16>::pair(u);
                            return pack_half2(f.x * mul, f.y * mul);
                        };
                        *at = make_uint4(narrow(v.x), narrow(v.y), narrow(v.z), narrow(v.w));
                    }
                    fence_proxy_async();
                }
                mbar_arrive(q_ready);
            }
        }
        for (int j = 0; ok && j < nk; ++j) {
            if (!__all_sync(0xffffffffu, mbar_wait_or_abort(kExact ? &f_full[j & 1] : &u_full[j & 3],
                                                            (j >> (kExact ? 1 : 2)) & 1, abort_flag) &&
                                             mbar_wait_or_abort(&s_full[x], j & 1, abort_flag))) {
                ok = false;
                break;
            }
            tc_fence_after();
            float sl2 = 1.f, grown = 1.f;
            if constexpr (!kExact) {
                const float4 units = *reinterpret_cast<const float4*>(smem + C::UNIT_OFF + (j & 3) * 16);
                sl2 = p.scale_log2 * (q_unit * units.x);
                v_unit = units.y;
                grown = units.z;
            }
            float sv[C::BN];
            {
                uint32_t u[C::BN];
#pragma unroll
                for (int c = 0; c < C::BN / 32; ++c)
                    tmem_ld32_nowait(ts + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&u[c * 32]));
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < C::BN; ++i) sv[i] = __uint_as_float(u[i]);
            }
            const int k0 = (tb + j) * C::BN;
            const bool all_vis = k0 + C::BN - 1 <= qpos;
            if constexpr (kExact) {  // the scores by their keys' factors, plus the logarithms of V's scales
                const float4* kf = reinterpret_cast<const float4*>(smem + C::SC_OFF + (j & 1) * C::BN * 4);
#pragma unroll
                for (int i = 0; i < C::BN; i += 4) {
                    const float4 a = kf[i / 4], b = kf[C::BN / 2 + i / 4];
                    const float2 t0 = __ffma2_rn(make_float2(sv[i], sv[i + 1]), make_float2(a.x, a.y), make_float2(b.x, b.y));
                    const float2 t1 = __ffma2_rn(make_float2(sv[i + 2], sv[i + 3]), make_float2(a.z, a.w), make_float2(b.z, b.w));
                    sv[i] = t0.x, sv[i + 1] = t0.y, sv[i + 2] = t1.x, sv[i + 3] = t1.y;
                }
                __syncwarp();
                if ((tid & 31) == 0) mbar_arrive(&f_free[2 * x + (j & 1)]);
            }
            float mrow;
            if (all_vis) {
                float r0 = sv[0], r1 = sv[1], r2 = sv[2], r3 = sv[3];
                if (sl2 >= 0.f) {
#pragma unroll
                    for (int i = 4; i < C::BN - 4; i += 8)
                        r0 = fmax3(r0, sv[i], sv[i + 4]), r1 = fmax3(r1, sv[i + 1], sv[i + 5]),
                        r2 = fmax3(r2, sv[i + 2], sv[i + 6]), r3 = fmax3(r3, sv[i + 3], sv[i + 7]);
                    r0 = fmax3(r0, sv[C::BN - 4], sv[C::BN - 3]), r1 = fmax3(r1, sv[C::BN - 2], sv[C::BN - 1]);
                    mrow = fmaxf(fmaxf(r0, r1), fmaxf(r2, r3)) * sl2;
                } else {
#pragma unroll
                    for (int i = 4; i < C::BN - 4; i += 8)
                        r0 = fmin3(r0, sv[i], sv[i + 4]), r1 = fmin3(r1, sv[i + 1], sv[i + 5]),
                        r2 = fmin3(r2, sv[i + 2], sv[i + 6]), r3 = fmin3(r3, sv[i + 3], sv[i + 7]);
                    r0 = fmin3(r0, sv[C::BN - 4], sv[C::BN - 3]), r1 = fmin3(r1, sv[C::BN - 2], sv[C::BN - 1]);
                    mrow = fminf(fminf(r0, r1), fminf(r2, r3)) * sl2;
                }
            } else {
                float r0 = -INFINITY, r1 = -INFINITY;
#pragma unroll
                for (int i = 0; i < C::BN; i += 2) {
                    sv[i] = k0 + i <= qpos ? sv[i] * sl2 : -INFINITY;
                    sv[i + 1] = k0 + i + 1 <= qpos ? sv[i + 1] * sl2 : -INFINITY;
                    r0 = fmaxf(r0, sv[i]);
                    r1 = fmaxf(r1, sv[i + 1]);
                }
                mrow = fmaxf(r0, r1);
            }
            const bool rescale = mrow > m_used + kRescaleLog2 || (m_used == -INFINITY && mrow != -INFINITY);
            float alpha = 1.f;
            if (rescale) {
                alpha = ex2_approx(m_used - mrow);  // 0 when m_used is -inf
                m_used = mrow;
            }
            const float mexp = m_used == -INFINITY ? 0.f : m_used;
            const float smul = all_vis ? sl2 : 1.f;
            float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            const float2 smul2 = make_float2(smul, smul), nm2 = make_float2(-mexp, -mexp);
            if constexpr (kExact) ok = __all_sync(0xffffffffu, mbar_wait_or_abort(i_full, j & 1, abort_flag));
#pragma unroll
            for (int c = 0; c < C::BN / 32; ++c) {
                uint32_t pw[16];
                if constexpr (kExact) {
                    const float4* iv = reinterpret_cast<const float4*>(smem + C::IV_OFF + c * 128);
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const float4 r = iv[i / 4];
                        const float2 u0 = __fadd2_rn(make_float2(sv[c * 32 + i], sv[c * 32 + i + 1]), nm2);
                        const float2 u1 = __fadd2_rn(make_float2(sv[c * 32 + i + 2], sv[c * 32 + i + 3]), nm2);
                        const float p0 = ex2_approx(u0.x), p1 = ex2_approx(u0.y), p2 = ex2_approx(u1.x), p3 = ex2_approx(u1.y);
                        acc[0] = __ffma2_rn(make_float2(p0, p1), make_float2(r.x, r.y), acc[0]);
                        acc[1] = __ffma2_rn(make_float2(p2, p3), make_float2(r.z, r.w), acc[1]);
                        pw[i / 2] = pack_half2(p0, p1), pw[i / 2 + 1] = pack_half2(p2, p3);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float2 arg = __ffma2_rn(make_float2(sv[c * 32 + i], sv[c * 32 + i + 1]), smul2, nm2);
                        const float p0 = ex2_approx(arg.x), p1 = ex2_approx(arg.y);
                        acc[(i / 2) & 1] = __fadd2_rn(acc[(i / 2) & 1], make_float2(p0, p1));
                        pw[i / 2] = pack_half2(p0, p1);
                    }
                }
                tmem_st16_nowait(ts + c * 16, pw);
            }
            lsum = lsum * alpha + ((acc[0].x + acc[0].y) + (acc[1].x + acc[1].y));
            if constexpr (kExact) {
                __syncwarp();
                if ((tid & 31) == 0) mbar_arrive(&i_free[x]);
            }
            alpha *= grown;
            if (j >= 1 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    float v[32];
                    tmem_ld32(to + c * 32, v);
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] *= alpha;
                    tmem_st32(to + c * 32, v);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&p_full[x]);
        }
        const bool have = ok && nk > 0 && __all_sync(0xffffffffu, mbar_wait_or_abort(&o_full[x], 0, abort_flag));
        tc_fence_after();
        T* out = reinterpret_cast<T*>(p.out);
        if (parts == 1) {
            if (have) {
                const bool live = tok < n && !*abort_flag;
                const float inv = v_unit / lsum;
                T* dst = out + (static_cast<int64_t>(q0 + tok) * p.num_q_heads + static_cast<int64_t>(g) * G + row % G) * D;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    float v[32];
                    tmem_ld32(to + c * 32, v);
                    if (live) {
#pragma unroll
                        for (int d = 0; d < 32; d += 8) {
                            uint4 w;
                            w.x = Elem<T>::pack(v[d] * inv, v[d + 1] * inv);
                            w.y = Elem<T>::pack(v[d + 2] * inv, v[d + 3] * inv);
                            w.z = Elem<T>::pack(v[d + 4] * inv, v[d + 5] * inv);
                            w.w = Elem<T>::pack(v[d + 6] * inv, v[d + 7] * inv);
                            *reinterpret_cast<uint4*>(dst + c * 32 + d) = w;
                        }
                    }
                }
            }
        } else {
            // ---- the cluster's merge.  Every role of this CTA is done with the
            // tiles, whose memory takes the partial results: O by rows, and (base,
            // sum) per row; no key seen: (-inf, 0); given up: a negative sum.
            __syncthreads();
            const int r256 = x * 128 + row;
            if (have) {
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    float v[32];
                    tmem_ld32(to + c * 32, v);
#pragma unroll
                    for (int d = 0; d < 8; ++d)
                        *reinterpret_cast<float4*>(smem + r256 * D * 4 + (((c * 8 + d) ^ (row & 7)) << 4)) =
                            make_float4(v[4 * d] * v_unit, v[4 * d + 1] * v_unit, v[4 * d + 2] * v_unit, v[4 * d + 3] * v_unit);
                }
            }
            *reinterpret_cast<float2*>(smem + C::ML_OFF + r256 * 8) =
                *abort_flag ? make_float2(0.f, -1.f) : have ? make_float2(m_used, lsum) : make_float2(-INFINITY, 0.f);
            cluster_sync();
            // This CTA's rows, rank * 256 / parts and on: a thread per row turns the
            // parts' bases and sums into their weights, then D / 4 lanes of four
            // elements to a row add the parts up.
            float* weights = reinterpret_cast<float*>(smem + C::W_OFF);  // [row][8]
            const uint32_t base = smem_u32(smem);
            const int rr0 = rank * 256 / parts, rows = (rank + 1) * 256 / parts - rr0;
            if (tid < rows) {
                float m[8], l[8], mx = -INFINITY, least = 0.f, sum = 0.f;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    m[k] = -INFINITY, l[k] = 0.f;
                    if (k < parts) {
                        const float2 ml = cluster_ld2(cluster_map(base + C::ML_OFF + (rr0 + tid) * 8, k));
                        m[k] = ml.x, l[k] = ml.y;
                    }
                    mx = fmaxf(mx, m[k]);
                    least = fminf(least, l[k]);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    // a base of -inf: nothing seen, or (sum NaN) nothing but NaN
                    m[k] = m[k] == -INFINITY ? (l[k] == 0.f ? 0.f : 1.f) : ex2_approx(m[k] - mx);
                    sum = fmaf(l[k], m[k], sum);
                }
                const float inv = 1.f / sum;
#pragma unroll
                for (int k = 0; k < 8; ++k) weights[tid * 8 + k] = least < 0.f ? -1.f : m[k] * inv;
            }
            asm volatile("bar.sync 1, 256;" ::: "memory");  // the softmax warps
            constexpr int LPR = D / 4, kPass = 256 / LPR, kRows = 4;
            const int lane_d = tid % LPR;
            // kRows rows of a thread at once, so that their loads from another
            // CTA's memory (hundreds of cycles each) are in flight together
            for (int i0 = tid / LPR; i0 < rows; i0 += kPass * kRows) {
                float4 o[kRows];
                float first[kRows];
                bool live[kRows], any = false;
#pragma unroll
                for (int e = 0; e < kRows; ++e) {
                    const int rr = rr0 + i0 + e * kPass;
                    live[e] = i0 + e * kPass < rows && (qt0 + rr / 128) * C::TT + (rr % 128) / G < n;
                    any = any || live[e];
                    o[e] = make_float4(0.f, 0.f, 0.f, 0.f), first[e] = 0.f;
                }
                if (!any) continue;
#pragma unroll 2
                for (int k = 0; k < parts; ++k) {
                    const uint32_t peer = cluster_map(base, k);
                    float4 v[kRows];
#pragma unroll
                    for (int e = 0; e < kRows; ++e) {
                        const int rr = rr0 + i0 + e * kPass;
                        if (live[e]) v[e] = cluster_ld4(peer + rr * D * 4 + ((lane_d ^ (rr & 7)) << 4));
                    }
#pragma unroll
                    for (int e = 0; e < kRows; ++e) {
                        const float w = live[e] ? weights[(i0 + e * kPass) * 8 + k] : 0.f;
                        first[e] = fminf(first[e], w);
                        if (w != 0.f) {  // else that part's O may be unwritten
                            o[e].x = fmaf(v[e].x, w, o[e].x), o[e].y = fmaf(v[e].y, w, o[e].y);
                            o[e].z = fmaf(v[e].z, w, o[e].z), o[e].w = fmaf(v[e].w, w, o[e].w);
                        }
                    }
                }
#pragma unroll
                for (int e = 0; e < kRows; ++e) {
                    const int rr = rr0 + i0 + e * kPass;
                    const int rtok = (qt0 + rr / 128) * C::TT + (rr % 128) / G;
                    if (live[e] && !(first[e] < 0.f)) {
                        T* dst = out + (static_cast<int64_t>(q0 + rtok) * p.num_q_heads + static_cast<int64_t>(g) * G + rr % G) * D + 4 * lane_d;
                        *reinterpret_cast<uint2*>(dst) = make_uint2(Elem<T>::pack(o[e].x, o[e].y), Elem<T>::pack(o[e].z, o[e].w));
                    }
                }
            }
            cluster_sync();  // no CTA leaves while another reads its shared memory
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

}  // namespace pkv
