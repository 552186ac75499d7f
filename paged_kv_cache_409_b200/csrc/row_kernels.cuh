// row_kernels.cuh -- rows of K (and Q) on their way into the paged cache:
//   rope_table_kernel      cos / sin rows of rotary positions,
//   rope_rows_kernel       norm of every query and key head, rotation, append,
//   append_int8_kernel     quantising append into pools of 8-bit rows,
//   read_int8_kernel       the stored rows as values again.
//
// Pools of 8-bit rows ("int8 pools").  A row is one token's head_dim elements
// of one KV head.  Row x is stored as codes u = 128 + rint(x / s), one byte
// each, and its own fp32 scale s = max |x| / 127; it stands for s * (u - 128).
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

__host__ __device__ __forceinline__ int64_t int8_block_bytes(int block_size, int num_kv_heads, int head_dim) {
    return static_cast<int64_t>(block_size) * num_kv_heads * (head_dim + 4);
}

// The scale of a row from the bits of its largest magnitude (compared as
// integers, NaN ranks above infinity, which ranks above every finite value).
// A row that holds a NaN or an infinity has no scale: it gets NaN, and
// everything read from it is NaN.
__device__ __forceinline__ float int8_scale(uint32_t absmax_bits) {
    if (absmax_bits >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
    return fmaxf(__uint_as_float(absmax_bits) / 127.f, kInt8MinScale);
}

// u = 128 + rint(x / s): the quotient rounded to fp32, then to the nearest
// integer, ties to even; clamped so that a NaN scale still gives a code.
__device__ __forceinline__ uint32_t int8_code(float x, float s) {
    return static_cast<uint32_t>(min(127, max(-127, __float2int_rn(x / s))) + 128);
}

__device__ __forceinline__ uint32_t int8_codes4(const float (&x)[4], float s) {
    return int8_code(x[0], s) | (int8_code(x[1], s) << 8) | (int8_code(x[2], s) << 16) | (int8_code(x[3], s) << 24);
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

__device__ __forceinline__ uint32_t absmax4(const float (&x)[4]) {
    return max(max(abs_bits(x[0]), abs_bits(x[1])), max(abs_bits(x[2]), abs_bits(x[3])));
}

template <typename T>
__device__ __forceinline__ void load4(const T* p, float (&f)[4]) {
    if constexpr (sizeof(T) == 4) {
        const float4 v = *reinterpret_cast<const float4*>(p);
        f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        const float2 a = Elem<T>::pair(v.x), b = Elem<T>::pair(v.y);
        f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
    }
}

template <typename T>
__device__ __forceinline__ void store4(T* p, const float (&f)[4]) {
    if constexpr (sizeof(T) == 4)
        *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    else
        *reinterpret_cast<uint2*>(p) = make_uint2(Elem<T>::pack(f[0], f[1]), Elem<T>::pack(f[2], f[3]));
}

// ---------------------------------------------------------------- rotary table
// out[p][i] = af * cos((first + p) * theta_i), out[p][R/2 + i] the sine.  The
// angle is formed in 64 bits: at position 2^20 a 32-bit angle is off by 0.06.
struct RopeTableParams {
    float* out;
    int64_t first;
    int64_t count;
    int half;                  // R / 2
    double attention_factor;
    double turns[128];         // theta_i / pi, in half turns per position
};

__global__ void __launch_bounds__(256) rope_table_kernel(const __grid_constant__ RopeTableParams p) {
    for (int64_t e = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; e < p.count * p.half;
         e += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t row = e / p.half;
        const int i = static_cast<int>(e - row * p.half);
        double s, c;
        sincospi(static_cast<double>(p.first + row) * p.turns[i], &s, &c);
        p.out[row * 2 * p.half + i] = static_cast<float>(c * p.attention_factor);
        p.out[row * 2 * p.half + p.half + i] = static_cast<float>(s * p.attention_factor);
    }
}

// ---------------------------------------------------------------- norm, rotation, append
struct RopeRowsParams {
    void* query_out;
    const void *query, *key, *value;
    int64_t q_stride, k_stride, v_stride;  // elements between tokens
    const void *q_weight, *k_weight;       // [D] or null (no norm)
    float eps;
    const float* cos_sin;                  // [max_position, R]
    int64_t max_position;
    int rotary_dim;
    int interleaved;
    const int64_t* positions;
    void *key_cache, *value_cache;
    const int64_t* slot_mapping;
    int64_t num_tokens, num_slots;
    int num_q_heads, num_kv_heads, head_dim, block_size;
    float k_scale, v_scale;                // E4M3 pools
};

// A lane holds eight elements of a row: four from `a` and four from `b`.  In
// the half layout the rotated pairs are (i, i + R/2), so a lane's two quads
// are partners (a = 4 l, b = R/2 + 4 l); pairs of the interleaved layout, and
// elements past the rotated part, are eight neighbours (a = 8 l, b = 8 l + 4).
// Either way no lane needs another's elements to rotate.  LPR lanes (a power
// of two, at least D / 8) share a row; the sums of the norm and the largest
// magnitude go over them by shuffles.
template <typename T, int kPool, int LPR>
__global__ void __launch_bounds__(128) rope_rows_kernel(const RopeRowsParams p) {
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, sub = lane % LPR;
    const int rows = p.num_q_heads + 2 * p.num_kv_heads;
    const int D = p.head_dim, half = p.rotary_dim / 2;
    const bool on = 8 * sub < D;
    const bool rot = 8 * sub < p.rotary_dim;
    const int a = rot && !p.interleaved ? 4 * sub : 8 * sub;
    const int b = rot && !p.interleaved ? half + 4 * sub : 8 * sub + 4;
    const int64_t t = blockIdx.x;
    const int64_t pos = p.positions ? p.positions[t] : 0;
    const int64_t slot = p.slot_mapping[t];
    if (p.positions && (pos < 0 || pos >= p.max_position)) {
        if (threadIdx.x == 0 && blockIdx.y == 0) flag_error(PKV_DEVERR_POSITION);
        return;
    }
    const bool store = slot >= 0 && slot < p.num_slots;
    if (slot >= p.num_slots && threadIdx.x == 0 && blockIdx.y == 0) flag_error(PKV_DEVERR_SLOT);
    float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
    if (on && rot) {
        load4(p.cos_sin + pos * p.rotary_dim + 4 * sub, c);
        load4(p.cos_sin + pos * p.rotary_dim + half + 4 * sub, s);
    }
    const int per = 128 / LPR;
    for (int r0 = blockIdx.y * per; r0 < rows; r0 += gridDim.y * per) {
        const int r = r0 + threadIdx.x / LPR;
        const bool live = on && r < rows;
        const int kind = r < p.num_q_heads ? 0 : r < p.num_q_heads + p.num_kv_heads ? 1 : 2;
        const int h = kind == 0 ? r : kind == 1 ? r - p.num_q_heads : r - p.num_q_heads - p.num_kv_heads;
        const T* src = kind == 0 ? static_cast<const T*>(p.query) + t * p.q_stride
                       : kind == 1 ? static_cast<const T*>(p.key) + t * p.k_stride
                                   : static_cast<const T*>(p.value) + t * p.v_stride;
        src += static_cast<int64_t>(h) * D;
        float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
        if (live) {
            load4(src + a, x);
            load4(src + b, y);
        }
        const T* w = static_cast<const T*>(kind == 0 ? p.q_weight : kind == 1 ? p.k_weight : nullptr);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) ss += x[i] * x[i] + y[i] * y[i];
#pragma unroll
        for (int off = 1; off < LPR; off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
        if (w && live) {
            const float f = 1.f / sqrtf(ss / D + p.eps);
            float wa[4], wb[4];
            load4(w + a, wa);
            load4(w + b, wb);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = x[i] * f * wa[i], y[i] = y[i] * f * wb[i];
        }
        if (kind < 2 && rot) {
            if (p.interleaved) {
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    const float x0 = x[i], x1 = x[i + 1], y0 = y[i], y1 = y[i + 1];
                    x[i] = x0 * c[i / 2] - x1 * s[i / 2];
                    x[i + 1] = x0 * s[i / 2] + x1 * c[i / 2];
                    y[i] = y0 * c[2 + i / 2] - y1 * s[2 + i / 2];
                    y[i + 1] = y0 * s[2 + i / 2] + y1 * c[2 + i / 2];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x0 = x[i], y0 = y[i];
                    x[i] = x0 * c[i] - y0 * s[i];
                    y[i] = x0 * s[i] + y0 * c[i];
                }
            }
        }
        uint32_t top = 0;
        if constexpr (kPool == kPoolInt8) {
            top = max(absmax4(x), absmax4(y));
#pragma unroll
            for (int off = 1; off < LPR; off <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
        }
        if (!live) continue;
        if (kind == 0) {
            T* dst = static_cast<T*>(p.query_out) + (t * p.num_q_heads + h) * D;
            store4(dst + a, x);
            store4(dst + b, y);
        } else if (store) {
            void* pool = kind == 1 ? p.key_cache : p.value_cache;
            if constexpr (kPool == kPoolInt8) {
                const int64_t blk = slot / p.block_size;
                const int tok = static_cast<int>(slot - blk * p.block_size);
                uint8_t* base = static_cast<uint8_t*>(pool) + blk * int8_block_bytes(p.block_size, p.num_kv_heads, D);
                uint8_t* dst = base + (static_cast<int64_t>(tok) * p.num_kv_heads + h) * D;
                const float sc = int8_scale(top);
                *reinterpret_cast<uint32_t*>(dst + a) = int8_codes4(x, sc);
                *reinterpret_cast<uint32_t*>(dst + b) = int8_codes4(y, sc);
                if (sub == 0)
                    reinterpret_cast<float*>(base + static_cast<int64_t>(p.block_size) * p.num_kv_heads * D)[h * p.block_size + tok] = sc;
            } else if constexpr (kPool == kPoolE4M3) {
                uint8_t* dst = static_cast<uint8_t*>(pool) + (slot * p.num_kv_heads + h) * D;
                const float f[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
                const uint2 q = quantise8(f, kind == 1 ? p.k_scale : p.v_scale);
                *reinterpret_cast<uint32_t*>(dst + a) = q.x;
                *reinterpret_cast<uint32_t*>(dst + b) = q.y;
            } else {
                T* dst = static_cast<T*>(pool) + (slot * p.num_kv_heads + h) * D;
                store4(dst + a, x);
                store4(dst + b, y);
            }
        }
    }
}

// ---------------------------------------------------------------- 8-bit rows: append and read
// LPR lanes per row of eight elements each, as above; blockIdx.x strides over
// (token, K or V, head) rows.
template <typename TS, int LPR>
__global__ void __launch_bounds__(128) append_int8_kernel(const TS* __restrict__ key, const TS* __restrict__ value,
                                                          uint8_t* __restrict__ key_cache,
                                                          uint8_t* __restrict__ value_cache,
                                                          const int64_t* __restrict__ slot_mapping, int64_t num_tokens,
                                                          int num_kv_heads, int head_dim, int block_size,
                                                          int64_t num_slots) {
    griddep_launch_dependents();
    const int sub = (threadIdx.x & 31) % LPR;
    const int64_t rows = num_tokens * 2 * num_kv_heads;
    const int64_t bytes = int8_block_bytes(block_size, num_kv_heads, head_dim);
    const int per = 128 / LPR;
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * per; r0 < rows; r0 += static_cast<int64_t>(gridDim.x) * per) {
        const int64_t r = r0 + threadIdx.x / LPR;
        const int64_t t = r / (2 * num_kv_heads);
        const int hh = static_cast<int>(r - t * 2 * num_kv_heads);
        const bool is_v = hh >= num_kv_heads;
        const int h = is_v ? hh - num_kv_heads : hh;
        const int64_t slot = r < rows ? slot_mapping[t] : -1;
        if (slot >= num_slots && sub == 0 && hh == 0) flag_error(PKV_DEVERR_SLOT);
        const bool live = slot >= 0 && slot < num_slots && 8 * sub < head_dim;
        float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (live) load8((is_v ? value : key) + (t * num_kv_heads + h) * head_dim + 8 * sub, f);
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, abs_bits(f[i]));
#pragma unroll
        for (int off = 1; off < LPR; off <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
        if (!live) continue;
        const int64_t blk = slot / block_size;
        const int tok = static_cast<int>(slot - blk * block_size);
        uint8_t* base = (is_v ? value_cache : key_cache) + blk * bytes;
        const float sc = int8_scale(top);
        const float lo[4] = {f[0], f[1], f[2], f[3]}, hi[4] = {f[4], f[5], f[6], f[7]};
        *reinterpret_cast<uint2*>(base + (static_cast<int64_t>(tok) * num_kv_heads + h) * head_dim + 8 * sub) =
            make_uint2(int8_codes4(lo, sc), int8_codes4(hi, sc));
        if (sub == 0)
            reinterpret_cast<float*>(base + static_cast<int64_t>(block_size) * num_kv_heads * head_dim)[h * block_size + tok] = sc;
    }
}

// Rows of the listed slots as values (scale * (code - 128), rounded once to
// TD); the rows of skipped slots are left as they were.
template <typename TD>
__global__ void __launch_bounds__(128) read_int8_kernel(TD* __restrict__ key_out, TD* __restrict__ value_out,
                                                        const uint8_t* __restrict__ key_cache,
                                                        const uint8_t* __restrict__ value_cache,
                                                        const int64_t* __restrict__ slot_mapping, int64_t num_tokens,
                                                        int num_kv_heads, int head_dim, int block_size,
                                                        int64_t num_slots) {
    const int64_t bytes = int8_block_bytes(block_size, num_kv_heads, head_dim);
    const int groups = head_dim / 8;  // eight elements per thread
    const int64_t n = num_tokens * 2 * num_kv_heads * groups;
    for (int64_t e = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; e < n;
         e += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t r = e / groups;
        const int d = static_cast<int>(e - r * groups) * 8;
        const int64_t t = r / (2 * num_kv_heads);
        const int hh = static_cast<int>(r - t * 2 * num_kv_heads);
        const bool is_v = hh >= num_kv_heads;
        const int h = is_v ? hh - num_kv_heads : hh;
        const int64_t slot = slot_mapping[t];
        if (slot < 0) continue;
        if (slot >= num_slots) {
            if (hh == 0 && d == 0) flag_error(PKV_DEVERR_SLOT);
            continue;
        }
        const int64_t blk = slot / block_size;
        const int tok = static_cast<int>(slot - blk * block_size);
        const uint8_t* base = (is_v ? value_cache : key_cache) + blk * bytes;
        const uint2 u = *reinterpret_cast<const uint2*>(base + (static_cast<int64_t>(tok) * num_kv_heads + h) * head_dim + d);
        const float sc = reinterpret_cast<const float*>(base + static_cast<int64_t>(block_size) * num_kv_heads * head_dim)[h * block_size + tok];
        float lo[4], hi[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = sc * static_cast<float>(static_cast<int>((u.x >> (8 * i)) & 255u) - 128);
            hi[i] = sc * static_cast<float>(static_cast<int>((u.y >> (8 * i)) & 255u) - 128);
        }
        TD* dst = (is_v ? value_out : key_out) + (t * num_kv_heads + h) * head_dim + d;
        store4(dst, lo);
        store4(dst + 4, hi);
    }
}

}  // namespace pkv
