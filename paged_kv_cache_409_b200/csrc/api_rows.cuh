// api_rows.cuh -- host side of the row calls (row_kernels.cuh): rotary tables,
// norm + rotation + append, and the append and read of 8-bit rows.  Included
// at the end of pagedkv.cu (one translation unit, one error word).

namespace {

// Lanes per row of head_dim elements, eight elements each.
int row_lanes(int head_dim) { return head_dim <= 64 ? 8 : head_dim <= 128 ? 16 : 32; }

// A row call's grid counts tokens in x and blocks of heads in y.
constexpr int kMaxRowHeads = 1 << 15;

// The shape rules of int8 pools: 16-byte rows of codes and 16-byte blocks.
bool int8_shape(int num_kv_heads, int head_dim, int block_size) {
    return head_dim % 16 == 0 && head_dim <= 256 && (int64_t)block_size * num_kv_heads % 4 == 0 &&
           (int64_t)block_size * num_kv_heads <= INT32_MAX / (head_dim + 4);
}

// Slots of a pool are counted in 64 bits.
bool countable_slots(int64_t num_blocks, int block_size) { return num_blocks <= INT64_MAX / block_size; }

int check_slots(const int64_t* slot_mapping, int64_t num_tokens, int64_t num_slots, cudaStream_t s) {
    if (!checked_mode()) return PKV_OK;
    std::vector<int64_t> sm;
    int rc = fetch(sm, slot_mapping, (size_t)num_tokens, s);
    if (rc) return rc;
    for (int64_t v : sm)
        if (v >= num_slots) return PKV_ERANGE;
    return PKV_OK;
}

// Argument checks of the append into and the read from int8 pools (x, y: the
// rows outside the pools).
int rows_int8_check(const void* x, const void* y, const void* key_cache, const void* value_cache,
                    const int64_t* slot_mapping, int64_t num_tokens, int num_kv_heads, int head_dim, int block_size,
                    int64_t num_blocks, int dtype) {
    if (!query_type(dtype)) return PKV_EUNSUPPORTED;
    if (num_tokens < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks <= 0 ||
        !countable_slots(num_blocks, block_size))
        return PKV_EINVAL;
    if (!int8_shape(num_kv_heads, head_dim, block_size)) return PKV_EUNSUPPORTED;
    if (num_tokens == 0) return PKV_OK;
    if (num_tokens > INT32_MAX || num_kv_heads > kMaxRowHeads) return PKV_EUNSUPPORTED;
    if (!x || !y || !key_cache || !value_cache || !slot_mapping) return PKV_EINVAL;
    if (!aligned16(x) || !aligned16(y) || !aligned16(key_cache) || !aligned16(value_cache) ||
        (reinterpret_cast<uintptr_t>(slot_mapping) & 7))
        return PKV_EINVAL;
    return PKV_OK;
}

// A row kernel, launched as a programmatic dependent of whatever comes before
// it in the stream: its CTAs are set up while that kernel drains, and the first
// thing they do is wait for its completion (griddepcontrol.wait).  Only then do
// they let a dependent of their own (a step's decode) start, so that one never
// runs beside anything but this kernel.  The wait covers that one kernel; what lies
// before it is done because every kernel here that is a dependent launch itself
// waits in each of its grids, whatever the data.
template <typename P>
int launch_after(void (*kern)(P), dim3 grid, cudaStream_t s, const std::remove_const_t<P>& p) {
    return launch_kernel(kern, grid, dim3(128), 0, Launch{s, true}, p);
}

int log2_ceil(int64_t n) {
    int k = 0;
    while ((int64_t(1) << k) < n) ++k;
    return k;
}

#ifndef PKV_ROPE_UNROLL
#define PKV_ROPE_UNROLL 2  // rows per thread of norm + rotation + append
#endif

template <typename T, int kPool, int E, int LPR, int U, bool kPlain, bool kNorm, bool kInterleaved>
int launch_rows(pkv::RopeRowsParams p, cudaStream_t s) {
    constexpr int kPer = 128 / LPR;
    const int most = log2_ceil(kPer);
    p.q_shift = std::min(most, log2_ceil(std::max(p.num_q_heads, 1)));
    p.kv_shift = std::min(most, log2_ceil(p.num_kv_heads));
    p.q_blocks = kPlain ? 0 : (int)ceil_div(p.num_q_heads, (int64_t)U << p.q_shift);
    const int64_t kv_blocks = ceil_div(p.num_kv_heads, (int64_t)(U / 2) << p.kv_shift);
    const int64_t groups = ceil_div(p.num_tokens, kPer >> (kPlain ? p.kv_shift : std::max(p.q_shift, p.kv_shift)));
    const dim3 grid((unsigned)groups, (unsigned)(p.q_blocks + kv_blocks));
    return launch_after(pkv::rope_rows_kernel<T, kPool, E, LPR, U, kPlain, kNorm, kInterleaved>, grid, s, p);
}

template <typename T, int kPool, bool kNorm, bool kInterleaved>
int launch_rope_as(const pkv::RopeRowsParams& p, cudaStream_t s) {
    constexpr int U = PKV_ROPE_UNROLL;
    // eight-element vectors need rows, and the rotated halves of the half
    // layout, in multiples of sixteen; the rest goes by four (one variant)
    if (p.head_dim % 16 || p.rotary_dim % 16)
        return launch_rows<T, kPool, 4, 32, U, false, kNorm, kInterleaved>(p, s);
    if (p.head_dim <= 64) return launch_rows<T, kPool, 8, 4, U, false, kNorm, kInterleaved>(p, s);
    if (p.head_dim <= 128) return launch_rows<T, kPool, 8, 8, U, false, kNorm, kInterleaved>(p, s);
    return launch_rows<T, kPool, 8, 16, U, false, kNorm, kInterleaved>(p, s);
}

template <typename T, int U>
int launch_append_as(const pkv::RopeRowsParams& p, cudaStream_t s) {
    constexpr int kPool = pkv::kPoolInt8;
    if (p.head_dim <= 64) return launch_rows<T, kPool, 8, 4, U, true, false, false>(p, s);
    if (p.head_dim <= 128) return launch_rows<T, kPool, 8, 8, U, true, false, false>(p, s);
    return launch_rows<T, kPool, 8, 16, U, true, false, false>(p, s);
}

// Rows per thread of the append: K and V of one head, or of two, which keeps
// more bytes in flight.  Two pay with 16-bit rows, more heads than stand side
// by side in a CTA (else the second is empty: 8 heads of 128, 16384 tokens: 18
// against 22 us) and sixteen CTAs per SM (32 heads of 128: 1024 tokens 6.1
// against 7.0 us, 2048 the same, 16384 65 against 60; fp32, 8191 tokens: 52
// against 56).
template <typename T>
int launch_append_int8(const pkv::RopeRowsParams& p, cudaStream_t s) {
    const int side = 256 / row_lanes(p.head_dim);
    const int64_t rows = 2 * p.num_tokens * p.num_kv_heads;
    if (sizeof(T) == 2 && p.num_kv_heads > side && rows >= (int64_t)side * 4 * 16 * sm_count())
        return launch_append_as<T, 4>(p, s);
    return launch_append_as<T, 2>(p, s);
}

template <typename T, int kPool>
int launch_rope(const pkv::RopeRowsParams& p, bool interleaved, cudaStream_t s) {
    if (p.q_weight || p.k_weight)
        return interleaved ? launch_rope_as<T, kPool, true, true>(p, s) : launch_rope_as<T, kPool, true, false>(p, s);
    return interleaved ? launch_rope_as<T, kPool, false, true>(p, s) : launch_rope_as<T, kPool, false, false>(p, s);
}

template <typename TD, int LPR>
int launch_read_as(pkv::ReadRowsParams p, cudaStream_t s) {
    constexpr int U = 2, kPer = 128 / LPR;  // four: 5 % faster with 8 heads, 2-25 % slower with 32
    p.shift = std::min(log2_ceil(kPer), log2_ceil(p.num_kv_heads));
    const dim3 grid((unsigned)ceil_div(p.num_tokens, kPer >> p.shift),
                    (unsigned)ceil_div(p.num_kv_heads, (int64_t)(U / 2) << p.shift));
    return launch_after(pkv::read_int8_kernel<TD, LPR, U>, grid, s, p);
}

template <typename TD>
int launch_read(const pkv::ReadRowsParams& p, cudaStream_t s) {
    const int lanes = row_lanes(p.head_dim) / 2;
    if (lanes == 4) return launch_read_as<TD, 4>(p, s);
    if (lanes == 8) return launch_read_as<TD, 8>(p, s);
    return launch_read_as<TD, 16>(p, s);
}

// CTAs that share an item's key tiles: a cluster of 1 to 8.  Measured on B200: a
// key tile takes a CTA about 2.4 us, its start and end 9 us alone and 13 us
// with the cluster's merge, and an SM holds one CTA.  So a launch of few items
// is cut (8 items of 16385 keys, head_dim 128: 293 us in one part, 51 in eight),
// one that fills the SMs is not (256 items of up to 66 tiles: 167 us in one
// part, 202 in two).  fit[k]: clusters of k CTAs that run at once; a GPC's SMs
// limit it (15 of eight, 22 of six: 16 items of 16128 keys take 108 us in
// eight parts, whose last cluster runs alone, and 68 in six).  The lengths are
// not known here: max_tiles is the table's reach, so tables far wider than the
// contexts cut items that are better whole (19 chunks of 64 rows over 1024 keys,
// 8 KV heads: 60 us with tables of 1056 tokens, 103 with 8192 or more).  Letting
// CTAs that a short item does not need leave at once does not help (97 us): their
// SMs go to no other cluster until theirs is done.
int prefill_parts(int64_t items, int64_t max_tiles, const int (&fit)[9]) {
    auto cost = [&](int parts) {
        const double waves = (double)items / fit[parts];
        return (waves > 4 ? waves : std::ceil(waves)) * ((parts == 1 ? 9.0 : 13.0) + 2.4 * ceil_div(max_tiles, parts));
    };
    int best = 1;
    double best_us = 0.9 * cost(1);  // the model's margin
    for (int parts = 2; parts <= 8; ++parts)
        if (fit[parts] > 0 && cost(parts) < best_us) best = parts, best_us = cost(parts);
    return best;
}

template <typename T, int D, int G>
int launch_prefill_int8(const pkv::PrefillInt8Params& prm, const CUtensorMap& tq, const CUtensorMap& tk,
                        const CUtensorMap& tv, int items, int live_items, int64_t max_tiles, cudaStream_t s) {
    using C = pkv::PrefillInt8Cfg<D, G>;
    auto kern = pkv::paged_prefill_int8_kernel<T, D, G>;
    int dev = 0;
    PKV_CUDA(cudaGetDevice(&dev));
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(pkv::kPrefillInt8Threads);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    static std::atomic<bool> configured[64];
    static std::mutex filling;
    static int fit[64][9];  // clusters of k CTAs that a device runs at once; written once, under the lock
    if (!configured[dev & 63]) {
        std::lock_guard<std::mutex> lock(filling);
        if (!configured[dev & 63]) {
            // the softmax threads' share (192) comes out of what the block is
            // launched with: 512 threads x 128 registers, no fewer
            cudaFuncAttributes a;
            PKV_CUDA(cudaFuncGetAttributes(&a, kern));
            if (a.numRegs < 128) return PKV_EUNSUPPORTED;
            PKV_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM));
            cfg.numAttrs = 1;
            for (int k = 1; k <= 8; ++k) {
                cfg.gridDim = dim3((unsigned)k);
                attr[0].val.clusterDim.x = k;
                PKV_CUDA(cudaOccupancyMaxActiveClusters(&fit[dev & 63][k], kern, &cfg));
            }
            configured[dev & 63] = true;
        }
    }
    const int parts = prefill_parts(live_items, max_tiles, fit[dev & 63]);
    cfg.gridDim = dim3((unsigned)(items * parts));
    attr[0].val.clusterDim.x = parts;
    cfg.numAttrs = 2;
    PKV_CUDA(cudaLaunchKernelEx(&cfg, kern, prm, tq, tk, tv));
    PKV_CUDA(cudaGetLastError());
    return PKV_OK;
}

template <typename T, int D>
int prefill_int8_by_group(int group, const pkv::PrefillInt8Params& prm, const CUtensorMap& tq, const CUtensorMap& tk,
                          const CUtensorMap& tv, int items, int live_items, int64_t max_tiles, cudaStream_t s) {
    switch (group) {
        case 1: return launch_prefill_int8<T, D, 1>(prm, tq, tk, tv, items, live_items, max_tiles, s);
        case 2: return launch_prefill_int8<T, D, 2>(prm, tq, tk, tv, items, live_items, max_tiles, s);
        case 4: return launch_prefill_int8<T, D, 4>(prm, tq, tk, tv, items, live_items, max_tiles, s);
        case 8: return launch_prefill_int8<T, D, 8>(prm, tq, tk, tv, items, live_items, max_tiles, s);
        default: return PKV_EUNSUPPORTED;
    }
}

template <int kPool>
int rope_impl(void* query_out, const void* query, const void* key, const void* value, int64_t query_stride,
              int64_t key_stride, int64_t value_stride, const void* q_norm_weight, const void* k_norm_weight, float eps,
              const float* cos_sin, int64_t max_position, int rotary_dim, int interleaved, const int64_t* positions,
              void* key_cache, void* value_cache, const int64_t* slot_mapping, int64_t num_tokens, int num_q_heads,
              int num_kv_heads, int head_dim, int block_size, int64_t num_blocks, int dtype, float k_scale,
              float v_scale, pkv_stream_t stream) {
    if (!query_type(dtype)) return PKV_EUNSUPPORTED;
    if (num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
        num_blocks <= 0 || !countable_slots(num_blocks, block_size) || rotary_dim < 0 || rotary_dim > head_dim || max_position < 0 || !(eps >= 0.f) ||
        !std::isfinite(eps))
        return PKV_EINVAL;
    if (kPool == pkv::kPoolE4M3 &&
        !(std::isfinite(k_scale) && k_scale > 0.f && std::isfinite(v_scale) && v_scale > 0.f))
        return PKV_EINVAL;
    if (head_dim % 8 || head_dim > 256 || rotary_dim % 8) return PKV_EUNSUPPORTED;
    if (kPool == pkv::kPoolE4M3 && head_dim % 16) return PKV_EUNSUPPORTED;
    if (kPool == pkv::kPoolInt8 && !int8_shape(num_kv_heads, head_dim, block_size)) return PKV_EUNSUPPORTED;
    if (num_tokens == 0) return PKV_OK;
    if (num_tokens > INT32_MAX || num_q_heads > kMaxRowHeads || num_kv_heads > kMaxRowHeads) return PKV_EUNSUPPORTED;
    if (!query_out || !query || !key || !value || !key_cache || !value_cache || !slot_mapping) return PKV_EINVAL;
    if (rotary_dim > 0 && (!cos_sin || !positions)) return PKV_EINVAL;
    const int eb = elem_bytes(dtype);
    const int64_t qrow = (int64_t)num_q_heads * head_dim, krow = (int64_t)num_kv_heads * head_dim;
    if (query_stride < qrow || key_stride < krow || value_stride < krow) return PKV_EINVAL;
    if (query_out == query && query_stride != qrow) return PKV_EINVAL;
    const void* ptrs[9] = {query_out, query, key, value, key_cache, value_cache, q_norm_weight, k_norm_weight, cos_sin};
    for (const void* q : ptrs)
        if (!aligned16(q)) return PKV_EINVAL;
    if (query_stride * eb % 16 || key_stride * eb % 16 || value_stride * eb % 16 ||
        (reinterpret_cast<uintptr_t>(positions) & 7) || (reinterpret_cast<uintptr_t>(slot_mapping) & 7))
        return PKV_EINVAL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t num_slots = num_blocks * block_size;
    if (checked_mode()) {
        int rc = check_slots(slot_mapping, num_tokens, num_slots, s);
        if (rc) return rc;
        if (rotary_dim > 0) {
            std::vector<int64_t> ps;
            rc = fetch(ps, positions, (size_t)num_tokens, s);
            if (rc) return rc;
            for (int64_t v : ps)
                if (v < 0 || v >= max_position) return PKV_ERANGE;
        }
    }
    pkv::RopeRowsParams p;
    p.query_out = query_out;
    p.query = query, p.key = key, p.value = value;
    p.q_stride = query_stride, p.k_stride = key_stride, p.v_stride = value_stride;
    p.q_weight = q_norm_weight, p.k_weight = k_norm_weight;
    p.eps = eps;
    p.inv_dim = 1.f / head_dim;
    p.cos_sin = cos_sin;
    p.max_position = max_position;
    p.rotary_dim = rotary_dim;
    p.positions = rotary_dim > 0 ? positions : nullptr;
    p.key_cache = key_cache, p.value_cache = value_cache;
    p.slot_mapping = slot_mapping;
    p.num_tokens = num_tokens, p.num_slots = num_slots;
    p.num_q_heads = num_q_heads, p.num_kv_heads = num_kv_heads, p.head_dim = head_dim, p.block_size = block_size;
    p.k_scale = k_scale, p.v_scale = v_scale;
    switch (dtype) {
        case PKV_F32: return launch_rope<float, kPool>(p, interleaved != 0, s);
        case PKV_F16: return launch_rope<__half, kPool>(p, interleaved != 0, s);
        default: return launch_rope<__nv_bfloat16, kPool>(p, interleaved != 0, s);
    }
}

}  // namespace

extern "C" {

int pkv_rope_table(float* cos_sin, int64_t first_position, int64_t num_positions, const pkv_rope_spec* spec,
                   pkv_stream_t stream) {
    if (!spec) return PKV_EINVAL;
    const int R = spec->rotary_dim;
    if (spec->scaling < PKV_ROPE_NONE || spec->scaling > PKV_ROPE_BY_PARTS) return PKV_EUNSUPPORTED;
    if (R <= 0 || first_position < 0 || num_positions < 0 || !(spec->base > 0) || !std::isfinite(spec->base) ||
        !std::isfinite(spec->attention_factor))
        return PKV_EINVAL;
    constexpr int64_t kFar = int64_t(1) << 40;
    if (first_position > kFar || num_positions > kFar - first_position) return PKV_EINVAL;
    if (spec->scaling != PKV_ROPE_NONE && !(spec->factor > 0 && std::isfinite(spec->factor))) return PKV_EINVAL;
    if (spec->scaling == PKV_ROPE_BY_PARTS &&
        !(spec->original_max_position > 0 && std::isfinite(spec->alpha) && std::isfinite(spec->beta) &&
          spec->alpha < spec->beta))
        return PKV_EINVAL;
    if (R % 8 || R > 256 || (spec->scaling == PKV_ROPE_NTK && R < 16)) return PKV_EUNSUPPORTED;
    if (num_positions == 0) return PKV_OK;
    if (!cos_sin || !aligned16(cos_sin)) return PKV_EINVAL;
    const double pi = 3.14159265358979323846;
    pkv::RopeTableParams p;
    p.out = cos_sin;
    p.first = first_position;
    p.count = num_positions;
    p.half = R / 2;
    p.attention_factor = spec->attention_factor;
    const double base =
        spec->scaling == PKV_ROPE_NTK ? spec->base * std::pow(spec->factor, (double)R / (R - 2)) : spec->base;
    for (int i = 0; i < R / 2; ++i) {
        double theta = std::pow(base, -2.0 * i / R);
        if (spec->scaling == PKV_ROPE_LINEAR) theta /= spec->factor;
        if (spec->scaling == PKV_ROPE_BY_PARTS) {
            const double turns = spec->original_max_position * theta / (2 * pi);
            const double g = std::min(1.0, std::max(0.0, (turns - spec->alpha) / (spec->beta - spec->alpha)));
            theta = (1 - g) * theta / spec->factor + g * theta;
        }
        p.turns[i] = theta / pi;
    }
    const int64_t threads = ceil_div(num_positions, pkv::kRopeTableRows) * p.half;
    const unsigned grid = (unsigned)std::min<int64_t>(ceil_div(threads, 128), 1 << 20);
    return launch_after(pkv::rope_table_kernel, dim3(grid), static_cast<cudaStream_t>(stream), p);
}

int pkv_rope_and_cache(void* query_out, const void* query, const void* key, const void* value, int64_t query_stride,
                       int64_t key_stride, int64_t value_stride, const void* q_norm_weight, const void* k_norm_weight,
                       float eps, const float* cos_sin, int64_t max_position, int rotary_dim, int interleaved,
                       const int64_t* positions, void* key_cache, void* value_cache, const int64_t* slot_mapping,
                       int64_t num_tokens, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                       int64_t num_blocks, int dtype, pkv_stream_t stream) {
    return rope_impl<pkv::kPoolSame>(query_out, query, key, value, query_stride, key_stride, value_stride,
                                     q_norm_weight, k_norm_weight, eps, cos_sin, max_position, rotary_dim, interleaved,
                                     positions, key_cache, value_cache, slot_mapping, num_tokens, num_q_heads,
                                     num_kv_heads, head_dim, block_size, num_blocks, dtype, 1.f, 1.f, stream);
}

int pkv_rope_and_cache_fp8(void* query_out, const void* query, const void* key, const void* value,
                           int64_t query_stride, int64_t key_stride, int64_t value_stride, const void* q_norm_weight,
                           const void* k_norm_weight, float eps, const float* cos_sin, int64_t max_position,
                           int rotary_dim, int interleaved, const int64_t* positions, void* key_cache,
                           void* value_cache, const int64_t* slot_mapping, int64_t num_tokens, int num_q_heads,
                           int num_kv_heads, int head_dim, int block_size, int64_t num_blocks, int dtype,
                           float k_scale, float v_scale, pkv_stream_t stream) {
    return rope_impl<pkv::kPoolE4M3>(query_out, query, key, value, query_stride, key_stride, value_stride,
                                     q_norm_weight, k_norm_weight, eps, cos_sin, max_position, rotary_dim, interleaved,
                                     positions, key_cache, value_cache, slot_mapping, num_tokens, num_q_heads,
                                     num_kv_heads, head_dim, block_size, num_blocks, dtype, k_scale, v_scale, stream);
}

int pkv_rope_and_cache_int8(void* query_out, const void* query, const void* key, const void* value,
                            int64_t query_stride, int64_t key_stride, int64_t value_stride, const void* q_norm_weight,
                            const void* k_norm_weight, float eps, const float* cos_sin, int64_t max_position,
                            int rotary_dim, int interleaved, const int64_t* positions, void* key_cache,
                            void* value_cache, const int64_t* slot_mapping, int64_t num_tokens, int num_q_heads,
                            int num_kv_heads, int head_dim, int block_size, int64_t num_blocks, int dtype,
                            pkv_stream_t stream) {
    return rope_impl<pkv::kPoolInt8>(query_out, query, key, value, query_stride, key_stride, value_stride,
                                     q_norm_weight, k_norm_weight, eps, cos_sin, max_position, rotary_dim, interleaved,
                                     positions, key_cache, value_cache, slot_mapping, num_tokens, num_q_heads,
                                     num_kv_heads, head_dim, block_size, num_blocks, dtype, 1.f, 1.f, stream);
}

int64_t pkv_int8_block_bytes(int block_size, int num_kv_heads, int head_dim) {
    if (block_size <= 0 || num_kv_heads <= 0 || head_dim <= 0) return PKV_EINVAL;
    if ((int64_t)block_size * num_kv_heads > INT64_MAX / ((int64_t)head_dim + 4)) return PKV_EINVAL;
    return (int64_t)block_size * num_kv_heads * ((int64_t)head_dim + 4);
}

int pkv_reshape_and_cache_int8(const void* key, const void* value, void* key_cache, void* value_cache,
                               const int64_t* slot_mapping, int64_t num_tokens, int num_kv_heads, int head_dim,
                               int block_size, int64_t num_blocks, int src_dtype, pkv_stream_t stream) {
    int rc = rows_int8_check(key, value, key_cache, value_cache, slot_mapping, num_tokens, num_kv_heads, head_dim,
                             block_size, num_blocks, src_dtype);
    if (rc || num_tokens == 0) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t num_slots = num_blocks * block_size;
    rc = check_slots(slot_mapping, num_tokens, num_slots, s);
    if (rc) return rc;
    pkv::RopeRowsParams p = {};
    p.key = key, p.value = value;
    p.k_stride = p.v_stride = (int64_t)num_kv_heads * head_dim;
    p.key_cache = key_cache, p.value_cache = value_cache;
    p.slot_mapping = slot_mapping;
    p.num_tokens = num_tokens, p.num_slots = num_slots;
    p.num_kv_heads = num_kv_heads, p.head_dim = head_dim, p.block_size = block_size;
    switch (src_dtype) {
        case PKV_F32: return launch_append_int8<float>(p, s);
        case PKV_F16: return launch_append_int8<__half>(p, s);
        default: return launch_append_int8<__nv_bfloat16>(p, s);
    }
}

int pkv_read_cache_int8(void* key_out, void* value_out, const void* key_cache, const void* value_cache,
                        const int64_t* slot_mapping, int64_t num_tokens, int num_kv_heads, int head_dim,
                        int block_size, int64_t num_blocks, int dst_dtype, pkv_stream_t stream) {
    int rc = rows_int8_check(key_out, value_out, key_cache, value_cache, slot_mapping, num_tokens, num_kv_heads,
                             head_dim, block_size, num_blocks, dst_dtype);
    if (rc || num_tokens == 0) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t num_slots = num_blocks * block_size;
    rc = check_slots(slot_mapping, num_tokens, num_slots, s);
    if (rc) return rc;
    const pkv::ReadRowsParams p = {key_out, value_out, static_cast<const uint8_t*>(key_cache),
                                   static_cast<const uint8_t*>(value_cache), slot_mapping, num_tokens, num_slots,
                                   num_kv_heads, head_dim, block_size, 0};
    switch (dst_dtype) {
        case PKV_F32: return launch_read<float>(p, s);
        case PKV_F16: return launch_read<__half>(p, s);
        default: return launch_read<__nv_bfloat16>(p, s);
    }
}

int pkv_paged_attention_decode_int8(void* out, const void* query, const void* key_cache, const void* value_cache,
                                    const int32_t* block_tables, const int32_t* context_lens, float scale,
                                    int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                    int max_blocks_per_seq, int64_t num_blocks, int max_context_len,
                                    int partition_size, int dtype, void* workspace, size_t workspace_bytes,
                                    pkv_stream_t stream) {
    return decode_impl(out, query, key_cache, value_cache, block_tables, context_lens, scale, num_seqs, num_q_heads,
                       num_kv_heads, head_dim, block_size, max_blocks_per_seq, num_blocks, max_context_len,
                       partition_size, dtype, PKV_INT8, 1.f, 1.f, workspace, workspace_bytes, stream);
}

int pkv_paged_attention_decode_step_int8(const void* new_keys, const void* new_values, const int64_t* slot_mapping,
                                         int64_t num_new_tokens, void* out, const void* query, void* key_cache,
                                         void* value_cache, const int32_t* block_tables, const int32_t* context_lens,
                                         float scale, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                         int block_size, int max_blocks_per_seq, int64_t num_blocks,
                                         int max_context_len, int partition_size, int dtype, void* workspace,
                                         size_t workspace_bytes, pkv_stream_t stream) {
    // Every check of both calls before the first launch, so that a refused
    // step has changed nothing.
    int rc = decode_check(out, query, key_cache, value_cache, block_tables, context_lens, scale, num_seqs,
                          num_q_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq, num_blocks,
                          max_context_len, partition_size, dtype, PKV_INT8);
    if (rc) return rc;
    rc = decode_workspace_check(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_context_len,
                                partition_size, workspace, workspace_bytes);
    if (rc) return rc;
    rc = rows_int8_check(new_keys, new_values, key_cache, value_cache, slot_mapping, num_new_tokens, num_kv_heads,
                         head_dim, block_size, num_blocks, dtype);
    if (rc) return rc;
    rc = check_step_tables(block_tables, context_lens, num_seqs, max_blocks_per_seq, block_size, num_blocks,
                           max_context_len, stream);
    if (rc) return rc;
    rc = pkv_reshape_and_cache_int8(new_keys, new_values, key_cache, value_cache, slot_mapping, num_new_tokens,
                                    num_kv_heads, head_dim, block_size, num_blocks, dtype, stream);
    if (rc) return rc;
    return decode_impl(out, query, key_cache, value_cache, block_tables, context_lens, scale, num_seqs, num_q_heads,
                       num_kv_heads, head_dim, block_size, max_blocks_per_seq, num_blocks, max_context_len,
                       partition_size, dtype, PKV_INT8, 1.f, 1.f, workspace, workspace_bytes, stream,
                       /*pdl=*/num_new_tokens > 0);
}

int pkv_paged_attention_prefill_chunk_int8(void* out, const void* query, const void* key_cache,
                                           const void* value_cache, const int32_t* block_tables,
                                           const int32_t* seq_lens, const int32_t* query_start_loc, int num_chunks,
                                           int64_t total_q_tokens, int max_q_len, float scale, int num_q_heads,
                                           int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq,
                                           int64_t num_blocks, int dtype, pkv_stream_t stream) {
    if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_EUNSUPPORTED;
    if (num_chunks < 0 || total_q_tokens < 0 || max_q_len < 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
        max_blocks_per_seq <= 0 || num_blocks <= 0 || !std::isfinite(scale))
        return PKV_EINVAL;
    if (num_q_heads % num_kv_heads) return PKV_EINVAL;
    const int group = num_q_heads / num_kv_heads;
    if (!supported_group(group) || (head_dim != 64 && head_dim != 128) ||
        (block_size != 8 && block_size != 16 && block_size != 32))
        return PKV_EUNSUPPORTED;
    if (num_blocks >= (int64_t)INT32_MAX || (int64_t)max_blocks_per_seq * block_size > INT32_MAX ||
        total_q_tokens > INT32_MAX)
        return PKV_EINVAL;
    if (num_chunks == 0 || total_q_tokens == 0 || max_q_len == 0) return PKV_OK;
    if (!out || !query || !key_cache || !value_cache || !block_tables || !seq_lens || !query_start_loc)
        return PKV_EINVAL;
    if (!aligned16(out) || !aligned16(query) || !aligned16(key_cache) || !aligned16(value_cache) ||
        (reinterpret_cast<uintptr_t>(block_tables) & 3) || (reinterpret_cast<uintptr_t>(seq_lens) & 3) ||
        (reinterpret_cast<uintptr_t>(query_start_loc) & 3))
        return PKV_EINVAL;
    const int tile_tokens = 128 / group;
    const int64_t tile_pairs = ceil_div(ceil_div(max_q_len, tile_tokens), 2);
    const int64_t items = (int64_t)num_chunks * tile_pairs * num_kv_heads;
    if (items > INT32_MAX / 8) return PKV_EUNSUPPORTED;
    // items that exist, about: a chunk's last pair of tiles is half full on average
    const int64_t pairs = std::min(num_chunks * tile_pairs,
                                   std::max<int64_t>(num_chunks, (num_chunks + 1) / 2 + total_q_tokens / (2 * tile_tokens)));
    const int live_items = (int)(pairs * num_kv_heads);
    const int64_t max_tiles = ceil_div((int64_t)max_blocks_per_seq * block_size, 128);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (checked_mode()) {
        std::vector<int32_t> qsl, lens;
        int rc = fetch(qsl, query_start_loc, (size_t)num_chunks + 1, s);
        if (rc) return rc;
        rc = fetch(lens, seq_lens, (size_t)num_chunks, s);
        if (rc) return rc;
        if (qsl[0] < 0 || qsl[num_chunks] > total_q_tokens) return PKV_ERANGE;
        for (int r = 0; r < num_chunks; ++r) {
            const int n = qsl[r + 1] - qsl[r];
            if (n < 0 || n > max_q_len || lens[r] < n) return PKV_ERANGE;
        }
        rc = check_tables(block_tables, seq_lens, num_chunks, max_blocks_per_seq, block_size, num_blocks,
                          (int64_t)max_blocks_per_seq * block_size, s);
        if (rc) return rc;
    }
    CUtensorMap tq, tk, tv;
    int rc = make_query_map(&tq, query, dtype, total_q_tokens, num_q_heads, head_dim, group);
    if (rc) return rc;
    rc = make_int8_map(&tk, key_cache, num_blocks, block_size, num_kv_heads, head_dim);
    if (rc) return rc;
    rc = make_int8_map(&tv, value_cache, num_blocks, block_size, num_kv_heads, head_dim);
    if (rc) return rc;
    pkv::PrefillInt8Params prm;
    prm.base.out = out;
    prm.base.block_tables = block_tables;
    prm.base.seq_lens = seq_lens;
    prm.base.query_start_loc = query_start_loc;
    prm.base.scale_log2 = scale * 1.4426950408889634f;
    prm.base.out_scale = 1.f;
    prm.base.num_chunks = num_chunks;
    prm.base.num_q_heads = num_q_heads;
    prm.base.num_kv_heads = num_kv_heads;
    prm.base.max_blocks_per_seq = max_blocks_per_seq;
    prm.base.block_size = block_size;
    prm.base.num_blocks = num_blocks;
    prm.base.tile_pairs = (int)tile_pairs;
    const int64_t codes = (int64_t)block_size * num_kv_heads * head_dim;
    prm.k_scales = static_cast<const uint8_t*>(key_cache) + codes;
    prm.v_scales = static_cast<const uint8_t*>(value_cache) + codes;
    prm.block_bytes = pkv::int8_block_bytes(block_size, num_kv_heads, head_dim);
    prm.total_q_tokens = (int)total_q_tokens;
    const bool bf16 = dtype == PKV_BF16;
    if (head_dim == 64)
        return bf16 ? prefill_int8_by_group<__nv_bfloat16, 64>(group, prm, tq, tk, tv, (int)items, live_items, max_tiles, s)
                    : prefill_int8_by_group<__half, 64>(group, prm, tq, tk, tv, (int)items, live_items, max_tiles, s);
    return bf16 ? prefill_int8_by_group<__nv_bfloat16, 128>(group, prm, tq, tk, tv, (int)items, live_items, max_tiles, s)
                : prefill_int8_by_group<__half, 128>(group, prm, tq, tk, tv, (int)items, live_items, max_tiles, s);
}

}  // extern "C"
