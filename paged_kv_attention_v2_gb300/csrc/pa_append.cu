// pa_append.cu -- pa_append_kv: the key and value rows of a step's tokens into
// the paged cache, through the slot map; fp8 caches quantised on the way.
//
// Bound by memory: every row is read once and written once.  One CTA takes
// kTokens successive rows of one key or value head.  Three of the four cases
// (NHD, and keys of the split layout) move whole 16-byte chunks of a token's
// head: thread -> (token, chunk), lanes spread so that a warp reads and writes
// whole 32-byte sectors.  Values of the split layout, [head dim][16 tokens], are
// transposed through shared memory: runs of successive slots are cut at the
// boundaries of 16-byte units of the page row, and a (unit, head dim) item is one
// 16-byte store when its unit is full, single elements where the run ends
// inside it.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>

#include "pa_cache.h"
#include "pa_host.cuh"
#include "pa_ptx.cuh"

namespace {

constexpr int kBS = PA_BLOCK_SIZE;
constexpr int kTokens = 32;   // rows per CTA
constexpr int kThreads = 256;

struct AppendParams {
    const void* key;
    const void* value;
    void* key_cache;
    void* value_cache;
    const int32_t* slots;
    int64_t key_stride, key_head_stride, value_stride, value_head_stride;
    int num_tokens, num_key_heads, key_head_size, num_value_heads, value_head_size, num_blocks;
    float k_scale, v_scale;
    int32_t* dev_error;
};

// Cache element kinds: the input's own bits, or fp8
enum { kSame = 0, kE4M3 = 1, kE5M2 = 2 };

template <int KV>
__device__ __forceinline__ uint32_t to_fp8x2(float a, float b) {
    // round to nearest even, beyond the largest finite value: that value
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, KV == kE4M3 ? __NV_E4M3 : __NV_E5M2);
}

// 16 bytes of the cache from the input row at src (16-byte aligned): the same
// bytes, or 16 elements quantised.
template <typename T, int KV>
__device__ __forceinline__ uint4 load_chunk(const T* src, float scale) {
    const uint4* s = reinterpret_cast<const uint4*>(src);
    if constexpr (KV == kSame) {
        return __ldg(s);
    } else {
        constexpr bool BF = std::is_same<T, __nv_bfloat16>::value;
        const uint4 a = __ldg(s), b = __ldg(s + 1);
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 lo = pa::unpack2<BF>(w[2 * i]), hi = pa::unpack2<BF>(w[2 * i + 1]);
            o[i] = to_fp8x2<KV>(__fdiv_rn(lo.x, scale), __fdiv_rn(lo.y, scale)) |
                   to_fp8x2<KV>(__fdiv_rn(hi.x, scale), __fdiv_rn(hi.y, scale)) << 16;
        }
        return make_uint4(o[0], o[1], o[2], o[3]);
    }
}

template <typename T, int KV, int LAYOUT>
__global__ void __launch_bounds__(kThreads) pa_append_kernel(const AppendParams p) {
    constexpr int E = KV == kSame ? (int)sizeof(T) : 1;  // bytes of a cache element
    constexpr int X = 16 / E;                            // elements of a 16-byte chunk
    extern __shared__ __align__(16) uint8_t tile[];      // split values: [token][head size + pad] elements
    __shared__ int slot_of[kTokens];
    __shared__ int unit_first[kTokens], unit_count[kTokens], units;

    const bool is_key = (int)blockIdx.y < p.num_key_heads;
    const int head = is_key ? blockIdx.y : (int)blockIdx.y - p.num_key_heads;
    const int heads = is_key ? p.num_key_heads : p.num_value_heads;
    const int size = is_key ? p.key_head_size : p.value_head_size;
    const float scale = is_key ? p.k_scale : p.v_scale;
    const int64_t stride = is_key ? p.key_stride : p.value_stride;
    const T* src = static_cast<const T*>(is_key ? p.key : p.value) +
                   head * (is_key ? p.key_head_stride : p.value_head_stride);
    uint8_t* cache = static_cast<uint8_t*>(is_key ? p.key_cache : p.value_cache);
    const int64_t page_bytes = (int64_t)kBS * size * E;
    const int t0 = blockIdx.x * kTokens, n = min(kTokens, p.num_tokens - t0);
    const int chunks = size / X;  // 16-byte chunks of a token's head
    const int tid = threadIdx.x;

    pa::pdl_launch_dependents();
    pa::pdl_wait_primary();

    if (tid < kTokens) {
        int s = tid < n ? __ldg(p.slots + t0 + tid) : -1;
        if (s >= p.num_blocks * kBS) {
            if (blockIdx.y == 0 && p.dev_error) atomicOr(p.dev_error, PA_DEVERR_SLOT);
            s = -1;
        }
        slot_of[tid] = s < 0 ? -1 : s;
    }
    __syncthreads();

    const bool transposed = LAYOUT == PA_LAYOUT_SPLIT && !is_key;
    if (!transposed) {
        // chunk (token, c): NHD a row of chunks per token, split [chunk][token].
        // 8 tokens x 4 chunks per warp
        for (int i = tid; i < kTokens * chunks; i += kThreads) {
            const int quad = i >> 5, lane = i & 31;
            const int t = (quad % (kTokens / 8)) * 8 + (lane & 7), c = quad / (kTokens / 8) * 4 + (lane >> 3);
            const int s = slot_of[t];
            if (s < 0) continue;
            const uint4 v = load_chunk<T, KV>(src + (t0 + t) * stride + c * X, scale);
            uint8_t* page = cache + ((int64_t)(s / kBS) * heads + head) * page_bytes;
            const int off = s % kBS;
            uint8_t* dst = LAYOUT == PA_LAYOUT_SPLIT ? page + (c * kBS + off) * 16 : page + (off * chunks + c) * 16;
            *reinterpret_cast<uint4*>(dst) = v;
        }
        return;
    }

    // split values: rows to shared memory in the cache's type (row pitch padded
    // by one chunk, so that a column's reads do not fall in one bank)
    const int pitch = size * E + 16;
    for (int i = tid; i < kTokens * chunks; i += kThreads) {
        const int t = i / chunks, c = i % chunks;
        if (slot_of[t] < 0) continue;
        *reinterpret_cast<uint4*>(tile + t * pitch + c * 16) =
            load_chunk<T, KV>(src + (t0 + t) * stride + c * X, scale);
    }
    // units: maximal runs of successive slots inside one 16-byte unit of a page row
    if (tid < 32) {
        const int s = slot_of[tid], before = tid > 0 ? slot_of[tid - 1] : -2;
        const bool begins = s >= 0 && (s % X == 0 || before != s - 1);
        const unsigned b = __ballot_sync(0xffffffffu, begins), skipped = __ballot_sync(0xffffffffu, s < 0);
        if (begins) {
            const int k = __popc(b & ((1u << tid) - 1));
            const unsigned stop = (b | skipped) & ~((2u << tid) - 1);  // first token that is not this unit's
            unit_first[k] = tid;
            unit_count[k] = (stop ? __ffs(stop) - 1 : 32) - tid;
        }
        if (tid == 0) units = __popc(b);
    }
    __syncthreads();
    for (int i = tid; i < units * size; i += kThreads) {
        const int u = i / size, d = i % size;
        const int t = unit_first[u], m = unit_count[u], s = slot_of[t];
        uint8_t* dst = cache + ((int64_t)(s / kBS) * heads + head) * page_bytes + (int64_t)(d * kBS + s % kBS) * E;
        const uint8_t* col = tile + t * pitch + d * E;
        if (m == X) {
            uint32_t w[4];
            if constexpr (E == 4) {
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] = *reinterpret_cast<const uint32_t*>(col + k * pitch);
            } else if constexpr (E == 2) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    w[k] = *reinterpret_cast<const uint16_t*>(col + 2 * k * pitch) |
                           (uint32_t) * reinterpret_cast<const uint16_t*>(col + (2 * k + 1) * pitch) << 16;
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    w[k] = col[4 * k * pitch] | (uint32_t)col[(4 * k + 1) * pitch] << 8 |
                           (uint32_t)col[(4 * k + 2) * pitch] << 16 | (uint32_t)col[(4 * k + 3) * pitch] << 24;
            }
            *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            for (int k = 0; k < m; ++k) {
                if constexpr (E == 4)
                    *reinterpret_cast<uint32_t*>(dst + 4 * k) = *reinterpret_cast<const uint32_t*>(col + k * pitch);
                else if constexpr (E == 2)
                    *reinterpret_cast<uint16_t*>(dst + 2 * k) = *reinterpret_cast<const uint16_t*>(col + k * pitch);
                else
                    dst[k] = col[k * pitch];
            }
        }
    }
}

bool size_ok(int d) { return d == 64 || d == 128 || d == 256; }

template <typename T, int KV>
bool launch(const AppendParams& p, int layout, void* stream) {
    const dim3 grid((unsigned)((p.num_tokens + kTokens - 1) / kTokens), (unsigned)(p.num_key_heads + p.num_value_heads));
    const int e = KV == kSame ? (int)sizeof(T) : 1;
    if (layout == PA_LAYOUT_NHD)
        return pa::launch_pdl(pa_append_kernel<T, KV, PA_LAYOUT_NHD>, grid, kThreads, 0, stream, p);
    return pa::launch_pdl(pa_append_kernel<T, KV, PA_LAYOUT_SPLIT>, grid, kThreads,
                          (size_t)kTokens * (p.value_head_size * e + 16), stream, p);
}

}  // namespace

extern "C" pa_status pa_append_kv(const pa_append_args* a, void* stream) {
    if (!a) return PA_ERR_INVALID_ARG;
    if (a->num_tokens < 0 || a->num_key_heads <= 0 || a->num_value_heads <= 0 || a->num_blocks <= 0)
        return PA_ERR_INVALID_ARG;
    if (a->dtype != PA_DTYPE_F32 && a->dtype != PA_DTYPE_F16 && a->dtype != PA_DTYPE_BF16) return PA_ERR_INVALID_ARG;
    if (a->layout != PA_LAYOUT_SPLIT && a->layout != PA_LAYOUT_NHD) return PA_ERR_INVALID_ARG;
    if (a->kv_dtype != PA_KV_SAME && a->kv_dtype != PA_KV_FP8_E4M3 && a->kv_dtype != PA_KV_FP8_E5M2)
        return PA_ERR_INVALID_ARG;
    if (!std::isfinite(a->k_scale) || !std::isfinite(a->v_scale)) return PA_ERR_INVALID_ARG;
    if (a->kv_dtype != PA_KV_SAME && a->dtype == PA_DTYPE_F32) return PA_ERR_UNSUPPORTED;
    if (a->block_size != PA_BLOCK_SIZE || a->num_blocks >= 1 << 27) return PA_ERR_UNSUPPORTED;
    if (!size_ok(a->key_head_size) || !size_ok(a->value_head_size)) return PA_ERR_UNSUPPORTED;
    if ((int64_t)a->num_key_heads + a->num_value_heads > 65535) return PA_ERR_UNSUPPORTED;
    if (a->num_tokens == 0) return PA_OK;
    if (!a->key || !a->value || !a->key_cache || !a->value_cache || !a->slots) return PA_ERR_INVALID_ARG;
    const int e = a->dtype == PA_DTYPE_F32 ? 4 : 2;
    const int64_t strides[] = {a->key_stride, a->key_head_stride, a->value_stride, a->value_head_stride};
    for (int64_t s : strides)
        if (s % (16 / e) != 0) return PA_ERR_INVALID_ARG;
    if (!pa::aligned(a->key, 16) || !pa::aligned(a->value, 16) || !pa::aligned(a->key_cache, 16) ||
        !pa::aligned(a->value_cache, 16) || !pa::aligned(a->slots, 4) || !pa::aligned(a->dev_error, 4))
        return PA_ERR_INVALID_ARG;

    AppendParams p = {};
    p.key = a->key;
    p.value = a->value;
    p.key_cache = a->key_cache;
    p.value_cache = a->value_cache;
    p.slots = a->slots;
    p.key_stride = a->key_stride;
    p.key_head_stride = a->key_head_stride;
    p.value_stride = a->value_stride;
    p.value_head_stride = a->value_head_stride;
    p.num_tokens = a->num_tokens;
    p.num_key_heads = a->num_key_heads;
    p.key_head_size = a->key_head_size;
    p.num_value_heads = a->num_value_heads;
    p.value_head_size = a->value_head_size;
    p.num_blocks = a->num_blocks;
    p.k_scale = a->k_scale > 0.f ? a->k_scale : 1.f;
    p.v_scale = a->v_scale > 0.f ? a->v_scale : 1.f;
    p.dev_error = a->dev_error;

    bool ok;
    const int kv = a->kv_dtype;
    if (a->dtype == PA_DTYPE_F32)
        ok = launch<float, kSame>(p, a->layout, stream);
    else if (a->dtype == PA_DTYPE_F16)
        ok = kv == PA_KV_SAME       ? launch<__half, kSame>(p, a->layout, stream)
             : kv == PA_KV_FP8_E4M3 ? launch<__half, kE4M3>(p, a->layout, stream)
                                    : launch<__half, kE5M2>(p, a->layout, stream);
    else
        ok = kv == PA_KV_SAME       ? launch<__nv_bfloat16, kSame>(p, a->layout, stream)
             : kv == PA_KV_FP8_E4M3 ? launch<__nv_bfloat16, kE4M3>(p, a->layout, stream)
                                    : launch<__nv_bfloat16, kE5M2>(p, a->layout, stream);
    return ok ? PA_OK : PA_ERR_LAUNCH;
}
