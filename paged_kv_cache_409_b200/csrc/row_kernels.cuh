// row_kernels.cuh -- rows of K (and Q) on their way into the paged cache:
//   rope_table_kernel      cos / sin rows of rotary positions,
//   rope_rows_kernel       norm of every query and key head, rotation, append
//                          (kPlain: the append alone, into pools of 8-bit rows),
//   read_int8_kernel       the stored rows as values again.
//
// Pools of 8-bit rows ("int8 pools").  A row is one token's head_dim elements
// of one KV head.  Row x is stored as codes u = 128 + rint(127 x / max |x|), one
// byte each, and its own fp32 scale s = max |x| / 127; it stands for s (u - 128).
// A block's bytes are the codes [block_size, num_kv_heads, head_dim] followed
// by the scales [num_kv_heads, block_size], so a block stays one contiguous
// unit that copy_blocks and swap_blocks move whole, its codes have the layout
// of the other pools, and the scales a decode CTA needs from a block (one KV
// head's) are one contiguous run.
#pragma once

#include "index_kernels.cuh"

namespace pkv {

// Pool kinds a row can be written to.
enum { kPoolSame = 0, kPoolE4M3 = 1, kPoolInt8 = 2 };

// Rows whose largest element is below 127 * 2^-80 get this scale: the readers
// divide by scales and take their logarithm, and 2^80 times a weight stays
// far inside fp32.  (A zero row's codes are all 128.)
constexpr float kInt8MinScale = 8.271806125530277e-25f;  // 2^-80
constexpr float kInt8MaxInverse = 1.2089258196146292e24f;  // 2^80

__host__ __device__ __forceinline__ int64_t int8_block_bytes(int block_size, int num_kv_heads, int head_dim) {
    return static_cast<int64_t>(block_size) * num_kv_heads * (head_dim + 4);
}

// The scale of a row from the bits of its largest magnitude (compared as
// integers, NaN ranks above infinity, which ranks above every finite value).
// A row that holds a NaN or an infinity has no scale: it gets NaN, and
// everything read from it is NaN.
__device__ __forceinline__ float int8_scale(uint32_t absmax_bits) {
    if (absmax_bits >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
    return fmaxf(__uint_as_float(absmax_bits) * (1.f / 127.f), kInt8MinScale);
}

// 127 / max |x| as a sum of two fp32 numbers (the rounded quotient, and what
// its remainder adds): one division per row, and element times inverse is as
// exact as a division per element.  With the first part alone, codes of
// quotients that lie on a tie went astray (rows of fp16 whose largest element
// is a multiple of 127 steps), and the error of rows read back grew by half.
struct Int8Inverse {
    float hi, lo;
};
__device__ __forceinline__ Int8Inverse int8_inverse(uint32_t absmax_bits) {
    const float a = __uint_as_float(absmax_bits), hi = 127.f / a;
    if (!(hi < kInt8MaxInverse)) return {kInt8MaxInverse, 0.f};
    return {hi, fmaf(-a, hi, 127.f) * (hi * (1.f / 127.f))};
}

// Codes of four elements: the quotient rounded to fp32, then to the nearest
// integer, ties to even, by adding 1.5 * 2^23 + 128, which leaves the code in
// the sum's low byte.
__device__ __forceinline__ uint32_t int8_codes4(const float (&x)[4], const Int8Inverse& inv) {
    const float2 hi = make_float2(inv.hi, inv.hi), lo = make_float2(inv.lo, inv.lo);
    const float2 magic = make_float2(12583040.f, 12583040.f);
    const float2 x01 = make_float2(x[0], x[1]), x23 = make_float2(x[2], x[3]);
    const float2 q01 = __fadd2_rn(__ffma2_rn(x01, hi, __fmul2_rn(x01, lo)), magic);
    const float2 q23 = __fadd2_rn(__ffma2_rn(x23, hi, __fmul2_rn(x23, lo)), magic);
    return __byte_perm(__byte_perm(__float_as_uint(q01.x), __float_as_uint(q01.y), 0x0040),
                       __byte_perm(__float_as_uint(q23.x), __float_as_uint(q23.y), 0x0040), 0x5410);
}

// Four codes as the integers u - 128, in fp32: a byte over 2^23 is the float
// 2^23 + u.
__device__ __forceinline__ void int8_values4(uint32_t u, float (&f)[4]) {
    constexpr float kMagic = 8388736.f;  // 2^23 + 128
    f[0] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440)) - kMagic;
    f[1] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7441)) - kMagic;
    f[2] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7442)) - kMagic;
    f[3] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7443)) - kMagic;
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

__device__ __forceinline__ uint32_t absmax4(const float (&x)[4]) {
    return max(max(abs_bits(x[0]), abs_bits(x[1])), max(abs_bits(x[2]), abs_bits(x[3])));
}

// E consecutive elements (4 or 8) as loaded, and as fp32.
template <typename T, int E>
struct Vec {
    static constexpr int kWords = E * static_cast<int>(sizeof(T)) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (kWords == 2) {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            w[0] = v.x, w[1] = v.y;
        } else {
#pragma unroll
            for (int i = 0; i < kWords; i += 4) {
                const uint4 v = *reinterpret_cast<const uint4*>(p + i * 4 / static_cast<int>(sizeof(T)));
                w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
            }
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0u;
    }
    __device__ __forceinline__ void unpack(float (&f)[E]) const {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < E; ++i) f[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                const float2 v = Elem<T>::pair(w[i]);
                f[2 * i] = v.x, f[2 * i + 1] = v.y;
            }
        }
    }
    __device__ __forceinline__ void pack(const float (&f)[E]) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < E; ++i) w[i] = __float_as_uint(f[i]);
        } else {
#pragma unroll
            for (int i = 0; i < E / 2; ++i) w[i] = Elem<T>::pack(f[2 * i], f[2 * i + 1]);
        }
    }
    __device__ __forceinline__ void store(T* p) const {
        if constexpr (kWords == 2) {
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        } else {
#pragma unroll
            for (int i = 0; i < kWords; i += 4)
                *reinterpret_cast<uint4*>(p + i * 4 / static_cast<int>(sizeof(T))) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
        }
    }
};

template <typename T, int E>
__device__ __forceinline__ void load_f(const T* p, float (&f)[E]) {
    Vec<T, E> v;
    v.load(p);
    v.unpack(f);
}

template <typename T>
__device__ __forceinline__ void load4(const T* p, float (&f)[4]) {
    load_f<T, 4>(p, f);
}

template <int E>
__device__ __forceinline__ uint32_t absmax_bits(const float (&x)[E]) {
    uint32_t m = abs_bits(x[0]);
#pragma unroll
    for (int i = 1; i < E; ++i) m = max(m, abs_bits(x[i]));
    return m;
}

// Block and token of a slot; slots past 2^32 take the 64-bit division.
__device__ __forceinline__ void split_slot(int64_t slot, int block_size, int64_t& blk, int& tok) {
    if (slot >> 32) {
        blk = slot / block_size;
        tok = static_cast<int>(slot - blk * block_size);
    } else {
        const uint32_t b = static_cast<uint32_t>(slot) / static_cast<uint32_t>(block_size);
        blk = b;
        tok = static_cast<int>(static_cast<uint32_t>(slot) - b * block_size);
    }
}

// ---------------------------------------------------------------- rotary table
// out[p][i] = af * cos((first + p) * theta_i), out[p][R/2 + i] the sine.  The
// angle is formed in 64 bits: at position 2^20 a 32-bit angle is off by 0.06.
// A thread takes one frequency and kRopeTableRows consecutive positions: two
// 64-bit sine / cosine pairs (the first angle and one step), then a complex
// product per row, each of which adds a few 2^-53.  Bound by the writes:
// 131072 rows of 128 take 11.4 us, 5.9 TB/s (a sine and cosine per element:
// 75 us, the 64-bit units).
struct RopeTableParams {
    float* out;
    int64_t first;
    int64_t count;
    int half;                  // R / 2
    double attention_factor;
    double turns[128];         // theta_i / pi, in half turns per position
};

constexpr int kRopeTableRows = 16;

__global__ void __launch_bounds__(128) rope_table_kernel(const __grid_constant__ RopeTableParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t runs = (p.count + kRopeTableRows - 1) / kRopeTableRows;
    for (int64_t e = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; e < runs * p.half;
         e += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t run = e / p.half;
        const int i = static_cast<int>(e - run * p.half);
        const int64_t row = run * kRopeTableRows;
        double s, c, ds, dc;
        sincospi(static_cast<double>(p.first + row) * p.turns[i], &s, &c);
        sincospi(p.turns[i], &ds, &dc);
        s *= p.attention_factor;
        c *= p.attention_factor;
        float* out = p.out + row * 2 * p.half + i;
        const int n = static_cast<int>(min(static_cast<int64_t>(kRopeTableRows), p.count - row));
        for (int k = 0; k < n; ++k) {
            out[0] = static_cast<float>(c);
            out[p.half] = static_cast<float>(s);
            out += 2 * p.half;
            const double c1 = c * dc - s * ds;
            s = s * dc + c * ds;
            c = c1;
        }
    }
}

// ---------------------------------------------------------------- norm, rotation, append
#ifndef PKV_ROPE_MIN_CTAS
#define PKV_ROPE_MIN_CTAS 7  // resident CTAs per SM the registers must allow
#endif

struct RopeRowsParams {
    void* query_out;
    const void *query, *key, *value;
    int64_t q_stride, k_stride, v_stride;  // elements between tokens
    const void *q_weight, *k_weight;       // [D] or null (no norm)
    float eps, inv_dim;                    // 1 / D
    const float* cos_sin;                  // [max_position, R]
    int64_t max_position;
    int rotary_dim;
    const int64_t* positions;
    void *key_cache, *value_cache;
    const int64_t* slot_mapping;
    int64_t num_tokens, num_slots;
    int num_q_heads, num_kv_heads, head_dim, block_size;
    float k_scale, v_scale;                // E4M3 pools
    int q_blocks;                          // blockIdx.y below it: query heads, from it on: K and V heads
    int q_shift, kv_shift;                 // log2 of the heads side by side in a CTA
};

// Norm and rotation of a lane's elements of one row; every lane of the warp
// calls it.  Lanes past the rotated part have c = 1, s = 0.  The sums and
// products go two at a time (packed fp32 arithmetic).
template <int E, int LPR, bool kNorm, bool kInterleaved>
__device__ __forceinline__ void norm_rotate(float (&x)[E], float (&y)[E], bool norm, const float (&wa)[E],
                                            const float (&wb)[E], const RopeRowsParams& p, const float (&c)[E],
                                            const float (&s)[E]) {
    if (kNorm && norm) {
        float2 acc = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < E; i += 2) {
            const float2 a = make_float2(x[i], x[i + 1]), b = make_float2(y[i], y[i + 1]);
            acc = __ffma2_rn(a, a, __ffma2_rn(b, b, acc));
        }
        float ss = acc.x + acc.y;
#pragma unroll
        for (int off = 1; off < LPR; off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
        const float f = rsqrtf(fmaf(ss, p.inv_dim, p.eps));
        const float2 ff = make_float2(f, f);
#pragma unroll
        for (int i = 0; i < E; i += 2) {
            const float2 a = __fmul2_rn(__fmul2_rn(make_float2(x[i], x[i + 1]), ff), make_float2(wa[i], wa[i + 1]));
            const float2 b = __fmul2_rn(__fmul2_rn(make_float2(y[i], y[i + 1]), ff), make_float2(wb[i], wb[i + 1]));
            x[i] = a.x, x[i + 1] = a.y, y[i] = b.x, y[i + 1] = b.y;
        }
    }
    if constexpr (kInterleaved) {
#pragma unroll
        for (int i = 0; i < E; i += 2) {
            const float x0 = x[i], x1 = x[i + 1], y0 = y[i], y1 = y[i + 1];
            x[i] = x0 * c[i / 2] - x1 * s[i / 2];
            x[i + 1] = x0 * s[i / 2] + x1 * c[i / 2];
            y[i] = y0 * c[E / 2 + i / 2] - y1 * s[E / 2 + i / 2];
            y[i + 1] = y0 * s[E / 2 + i / 2] + y1 * c[E / 2 + i / 2];
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; i += 2) {
            const float2 a = make_float2(x[i], x[i + 1]), b = make_float2(y[i], y[i + 1]);
            const float2 cc = make_float2(c[i], c[i + 1]), sn = make_float2(s[i], s[i + 1]);
            const float2 u = __ffma2_rn(b, make_float2(-s[i], -s[i + 1]), __fmul2_rn(a, cc));
            const float2 v = __ffma2_rn(a, sn, __fmul2_rn(b, cc));
            x[i] = u.x, x[i + 1] = u.y, y[i] = v.x, y[i + 1] = v.y;
        }
    }
}

template <int E>
__device__ __forceinline__ void store_codes(uint8_t* p, const float (&x)[E], const Int8Inverse& inv) {
    uint32_t w[E / 4];
#pragma unroll
    for (int i = 0; i < E; i += 4) {
        const float q[4] = {x[i], x[i + 1], x[i + 2], x[i + 3]};
        w[i / 4] = int8_codes4(q, inv);
    }
    if constexpr (E == 4) *reinterpret_cast<uint32_t*>(p) = w[0];
    else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

template <int E>
__device__ __forceinline__ void store_e4m3(uint8_t* p, const float (&x)[E], float scale) {
#pragma unroll
    for (int i = 0; i < E; i += 4) {
        uint32_t lo = e4m3x2_from_f32(quotient_round_to_odd(x[i + 1], scale), quotient_round_to_odd(x[i], scale));
        uint32_t hi = e4m3x2_from_f32(quotient_round_to_odd(x[i + 3], scale), quotient_round_to_odd(x[i + 2], scale));
        *reinterpret_cast<uint32_t*>(p + i) = lo | (hi << 16);
    }
}

// Every row is read once and written once: the bound is memory, and to stay
// near it the kernel has to spend few instructions on an element.  A lane
// holds 2 E elements of a row: E from `a` and E from `b`.  In the half layout
// the rotated pairs are (i, i + R/2), so the two are partners (a = E l, b =
// R/2 + E l); pairs of the interleaved layout, and elements past the rotated
// part, are neighbours (a = 2 E l, b = a + E).  Either way no lane needs
// another's elements to rotate.  LPR lanes (a power of two, at least D / 2E)
// share a row; the sums of the norm and the largest magnitude go over them by
// shuffles.  E = 8 where head_dim and rotary_dim are multiples of 16, else 4.
// A thread stays with one token: U query heads, or U / 2 heads of both K and
// V, so that position, slot, table row and weights are looked up once, what a
// row is is known per CTA, and U rows are in flight before the first is used.
// kPlain: K and V as they are (the append).
// Measured: 8192 tokens of 32 + 8 + 8 heads of 128 in bf16, norm and rotation
// into int8 pools, 40 us = 4.6 TB/s, 61 % of the issue slots, 28 warps per SM
// (72 registers; 6 or 8 CTAs per SM are slower); the append of 8191 tokens of
// 32 heads of 128 in fp16 31 us = 6.5 TB/s.  A thread that goes on to further tokens, weights
// kept and their rows fetched ahead, gains 5-7 % there and loses more than that
// on small batches.
template <typename T, int kPool, int E, int LPR, int U, bool kPlain, bool kNorm, bool kInterleaved>
__global__ void __launch_bounds__(128, PKV_ROPE_MIN_CTAS) rope_rows_kernel(const RopeRowsParams p) {
    griddep_wait();  // before the first read: see launch_after
    griddep_launch_dependents();
    constexpr int kPer = 128 / LPR;
    const int sub = threadIdx.x % LPR, rs = threadIdx.x / LPR;
    const bool kv = kPlain || blockIdx.y >= p.q_blocks;
    const int shift = kv ? p.kv_shift : p.q_shift;
    const int side = 1 << shift;  // heads side by side
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * (kPer >> shift);
    if (t0 >= p.num_tokens) return;
    const int64_t t = min(t0 + (rs >> shift), p.num_tokens - 1);
    const bool live_t = t0 + (rs >> shift) < p.num_tokens;
    const int D = p.head_dim, half = p.rotary_dim / 2;
    const bool on = 2 * E * sub < D;
    const bool rot = !kPlain && 2 * E * sub < p.rotary_dim;
    const int a = rot && !kInterleaved ? E * sub : 2 * E * sub;
    const int b = rot && !kInterleaved ? half + E * sub : 2 * E * sub + E;
    const int64_t pos = !kPlain && p.positions ? p.positions[t] : 0;
    const bool bad_pos = !kPlain && p.positions && (pos < 0 || pos >= p.max_position);
    const bool first = live_t && sub == 0 && (rs & (side - 1)) == 0;
    float c[E], s[E], wa[E], wb[E];
#pragma unroll
    for (int i = 0; i < E; ++i) c[i] = wa[i] = wb[i] = 1.f, s[i] = 0.f;
    Vec<T, E> ra[U], rb[U];
    const int h0 = rs & (side - 1);
    if (!kv) {
        const int hq = h0 + blockIdx.y * (side * U);
        const T* src = static_cast<const T*>(p.query) + t * p.q_stride + hq * D;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            ra[u].zero(), rb[u].zero();
            if (on && hq + u * side < p.num_q_heads) ra[u].load(src + u * side * D + a), rb[u].load(src + u * side * D + b);
        }
        if (bad_pos && first && blockIdx.y == 0) flag_error(PKV_DEVERR_POSITION);
        const bool ok = on && live_t && !bad_pos;
        if (ok && rot) {
            load_f(p.cos_sin + pos * p.rotary_dim + E * sub, c);
            load_f(p.cos_sin + pos * p.rotary_dim + half + E * sub, s);
        }
        if (kNorm && p.q_weight && on) {
            load_f(static_cast<const T*>(p.q_weight) + a, wa);
            load_f(static_cast<const T*>(p.q_weight) + b, wb);
        }
        T* dst = static_cast<T*>(p.query_out) + (t * p.num_q_heads + hq) * D;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float x[E], y[E];
            ra[u].unpack(x), rb[u].unpack(y);
            norm_rotate<E, LPR, kNorm, kInterleaved>(x, y, p.q_weight, wa, wb, p, c, s);
            if (ok && hq + u * side < p.num_q_heads) {
                ra[u].pack(x), rb[u].pack(y);
                ra[u].store(dst + u * side * D + a), rb[u].store(dst + u * side * D + b);
            }
        }
    } else {
        const int hk = h0 + (blockIdx.y - p.q_blocks) * (side * (U / 2));
        const T* ks = static_cast<const T*>(p.key) + t * p.k_stride + hk * D;
        const T* vs = static_cast<const T*>(p.value) + t * p.v_stride + hk * D;
        const int64_t slot = p.slot_mapping[t];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            ra[u].zero(), rb[u].zero();
            const T* src = (u & 1 ? vs : ks) + (u / 2) * side * D;
            if (on && hk + (u / 2) * side < p.num_kv_heads) ra[u].load(src + a), rb[u].load(src + b);
        }
        if (slot >= p.num_slots && !bad_pos && first && blockIdx.y == p.q_blocks) flag_error(PKV_DEVERR_SLOT);
        const bool ok = on && live_t && !bad_pos && slot >= 0 && slot < p.num_slots;
        if (ok && rot) {
            load_f(p.cos_sin + pos * p.rotary_dim + E * sub, c);
            load_f(p.cos_sin + pos * p.rotary_dim + half + E * sub, s);
        }
        if (kNorm && p.k_weight && on) {
            load_f(static_cast<const T*>(p.k_weight) + a, wa);
            load_f(static_cast<const T*>(p.k_weight) + b, wb);
        }
        // where head hk's row goes in either pool: bytes from the pool's start
        int64_t at, scale_at = 0;
        constexpr int kBytes = kPool == kPoolSame ? static_cast<int>(sizeof(T)) : 1;
        if constexpr (kPool == kPoolInt8) {
            int64_t blk = 0;
            int tok = 0;
            if (ok) split_slot(slot, p.block_size, blk, tok);
            const int64_t base = blk * int8_block_bytes(p.block_size, p.num_kv_heads, D);
            at = base + (tok * p.num_kv_heads + hk) * D;
            scale_at = base + p.block_size * p.num_kv_heads * D + (hk * p.block_size + tok) * 4;
        } else {
            at = (slot * p.num_kv_heads + hk) * D * kBytes;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool is_v = u & 1;
            uint8_t* pool = static_cast<uint8_t*>(is_v ? p.value_cache : p.key_cache);
            uint8_t* dst = pool + at + (u / 2) * side * D * kBytes;
            const bool live = ok && hk + (u / 2) * side < p.num_kv_heads;
            float x[E], y[E];
            ra[u].unpack(x), rb[u].unpack(y);
            if (!kPlain && !is_v) norm_rotate<E, LPR, kNorm, kInterleaved>(x, y, p.k_weight, wa, wb, p, c, s);
            if constexpr (kPool == kPoolInt8) {
                uint32_t top = max(absmax_bits(x), absmax_bits(y));
#pragma unroll
                for (int off = 1; off < LPR; off <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
                const Int8Inverse inv = int8_inverse(top);
                if (live) {
                    store_codes(dst + a, x, inv);
                    store_codes(dst + b, y, inv);
                    if (sub == 0) *reinterpret_cast<float*>(pool + scale_at + (u / 2) * side * p.block_size * 4) = int8_scale(top);
                }
            } else if constexpr (kPool == kPoolE4M3) {
                if (live) store_e4m3(dst + a, x, is_v ? p.v_scale : p.k_scale), store_e4m3(dst + b, y, is_v ? p.v_scale : p.k_scale);
            } else if (live) {
                if (!is_v) ra[u].pack(x), rb[u].pack(y);
                ra[u].store(reinterpret_cast<T*>(dst) + a), rb[u].store(reinterpret_cast<T*>(dst) + b);
            }
        }
    }
}

// ---------------------------------------------------------------- 8-bit rows read back
struct ReadRowsParams {
    void *key_out, *value_out;  // [num_tokens, num_kv_heads, head_dim]
    const uint8_t *key_cache, *value_cache;
    const int64_t* slot_mapping;
    int64_t num_tokens, num_slots;
    int num_kv_heads, head_dim, block_size;
    int shift;  // log2 of the heads side by side in a CTA
};

// Rows of the listed slots as values (scale * (code - 128), rounded once to
// TD); the rows of skipped slots are left as they were.  The map is that of
// rope_rows_kernel with sixteen elements per lane: a thread reads U / 2 heads
// of K and V of one token.  Bound by memory: 203 MB (8191 tokens, 32 heads of
// 128 to fp16) in 39 us, 5.2 TB/s.
template <typename TD, int LPR, int U>
__global__ void __launch_bounds__(128) read_int8_kernel(const ReadRowsParams p) {
    griddep_wait();
    griddep_launch_dependents();
    constexpr int kPer = 128 / LPR;
    const int sub = threadIdx.x % LPR, rs = threadIdx.x / LPR;
    const int side = 1 << p.shift;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (kPer >> p.shift) + (rs >> p.shift);
    const int D = p.head_dim;
    if (t >= p.num_tokens || 16 * sub >= D) return;
    const int h0 = (rs & (side - 1)) + blockIdx.y * (side * (U / 2));
    const int64_t slot = p.slot_mapping[t];
    if (slot < 0) return;
    if (slot >= p.num_slots) {
        if (h0 == 0 && sub == 0) flag_error(PKV_DEVERR_SLOT);
        return;
    }
    int64_t blk;
    int tok;
    split_slot(slot, p.block_size, blk, tok);
    const int64_t base = blk * int8_block_bytes(p.block_size, p.num_kv_heads, D);
    const int scales = p.block_size * p.num_kv_heads * D + 4 * tok;
    uint4 code[U];
    float sc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = h0 + (u / 2) * side;
        if (h >= p.num_kv_heads) continue;
        const uint8_t* pool = (u & 1 ? p.value_cache : p.key_cache) + base;
        code[u] = *reinterpret_cast<const uint4*>(pool + (tok * p.num_kv_heads + h) * D + 16 * sub);
        sc[u] = *reinterpret_cast<const float*>(pool + scales + 4 * h * p.block_size);
    }
    const int64_t row = t * p.num_kv_heads * D + 16 * sub;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = h0 + (u / 2) * side;
        if (h >= p.num_kv_heads) continue;
        TD* dst = static_cast<TD*>(u & 1 ? p.value_out : p.key_out) + row + h * D;
        float v[16];
        const uint32_t w[4] = {code[u].x, code[u].y, code[u].z, code[u].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float x[4];
            int8_values4(w[q], x);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[4 * q + i] = x[i] * sc[u];
        }
        if constexpr (sizeof(TD) == 4) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                reinterpret_cast<float4*>(dst)[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        } else {
#pragma unroll
            for (int q = 0; q < 2; ++q)
                reinterpret_cast<uint4*>(dst)[q] =
                    make_uint4(Elem<TD>::pack(v[8 * q], v[8 * q + 1]), Elem<TD>::pack(v[8 * q + 2], v[8 * q + 3]),
                               Elem<TD>::pack(v[8 * q + 4], v[8 * q + 5]), Elem<TD>::pack(v[8 * q + 6], v[8 * q + 7]));
        }
    }
}

}  // namespace pkv
