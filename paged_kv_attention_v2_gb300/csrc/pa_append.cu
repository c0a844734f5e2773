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

// One head of a CTA's rows: `src` its row t0, `cache` its page of block 0 (pages
// of one head `block_bytes` apart), SIZE its head size.
template <typename T, int KV, int LAYOUT, int SIZE, bool KEY>
__device__ __forceinline__ void append_head(const AppendParams& p, const T* src, int64_t stride, uint8_t* cache,
                                            int64_t block_bytes, float scale, int t0, int n, uint8_t* tile) {
    constexpr int E = KV == kSame ? (int)sizeof(T) : 1;  // bytes of a cache element
    constexpr int X = 16 / E;                            // elements of a 16-byte chunk
    constexpr int CH = SIZE / X;                         // chunks of a token's head
    constexpr bool SPLIT = LAYOUT == PA_LAYOUT_SPLIT;
    constexpr int ITEMS = kTokens * CH, PER = (ITEMS + kThreads - 1) / kThreads;
    __shared__ int64_t base_of[kTokens];  // byte offset of token t's first element in the cache, < 0: no slot
    const int tid = threadIdx.x;

    // The rows do not wait for the slots: both are loaded at once.  Chunk (token,
    // c) of a thread's item k: 8 tokens x 4 chunks per warp where the cache is
    // [chunk][token] (split keys: whole sectors are read and written), rows of
    // chunks elsewhere.
    int slot = -1;
    if (tid < n) slot = __ldg(p.slots + t0 + tid);  // n <= kTokens
    auto place = [&](int k, int& t, int& c) {
        const int i = k * kThreads + tid;
        if constexpr (SPLIT && KEY) {
            t = (i >> 5) % (kTokens / 8) * 8 + (i & 7);
            c = (i >> 5) / (kTokens / 8) * 4 + (i >> 3 & 3);
        } else {
            t = i / CH;
            c = i % CH;
        }
        return ITEMS % kThreads == 0 || i < ITEMS;
    };
    uint4 v[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        int t, c;
        if (place(k, t, c) && t < n) v[k] = load_chunk<T, KV>(src + t * stride + c * X, scale);
    }
    if (tid < kTokens) {
        if (slot >= p.num_blocks * kBS) {
            if (blockIdx.y == 0 && p.dev_error) atomicOr(p.dev_error, PA_DEVERR_SLOT);
            slot = -1;
        }
        constexpr int STEP = SPLIT ? (KEY ? 16 : E) : SIZE * E;  // bytes from a token to the next
        base_of[tid] = slot < 0 ? -1 : (int64_t)(slot >> 4) * block_bytes + (slot & 15) * STEP;
    }
    if constexpr (!SPLIT || KEY) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            int t, c;
            if (!place(k, t, c)) break;
            const int64_t at = base_of[t];
            if (at >= 0) *reinterpret_cast<uint4*>(cache + at + c * (SPLIT ? 256 : 16)) = v[k];
        }
    } else {
        // values [head dim][16 tokens]: transposed through shared memory, rows in
        // the cache's type with a pitch of one chunk more than a row
        constexpr int PITCH = SIZE * E + 16;
        __shared__ int unit_first[kTokens], unit_count[kTokens], unit_total;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            int t, c;
            if (place(k, t, c) && t < n) *reinterpret_cast<uint4*>(tile + t * PITCH + c * 16) = v[k];
        }
        // units: maximal runs of successive slots inside one 16-byte unit of a page row
        if (tid < kTokens) {
            const int before = __shfl_up_sync(0xffffffffu, slot, 1);
            const bool begins = slot >= 0 && (tid == 0 || slot % X == 0 || before != slot - 1);
            const unsigned b = __ballot_sync(0xffffffffu, begins), skipped = __ballot_sync(0xffffffffu, slot < 0);
            if (begins) {
                const int k = __popc(b & ((1u << tid) - 1));
                const unsigned stop = (b | skipped) & ~((2u << tid) - 1);  // first token that is not this unit's
                unit_first[k] = tid;
                unit_count[k] = (stop ? __ffs(stop) - 1 : 32) - tid;
            }
            if (tid == 0) unit_total = __popc(b);
        }
        __syncthreads();
        // item -> (unit, head dim): the E units that make up a page row (16 tokens)
        // of a full page lie side by side, so a warp writes whole sectors
        const int units = unit_total;
        for (int i = tid; i < (units + E - 1) / E * (E * SIZE); i += kThreads) {
            const int u = i / (E * SIZE) * E + i % E, d = i / E % SIZE;
            if (u >= units) continue;
            const int t = unit_first[u], m = unit_count[u];
            uint8_t* dst = cache + base_of[t] + d * (kBS * E);
            const uint8_t* col = tile + t * PITCH + d * E;
            if (m == X) {
                uint32_t w[4];
                if constexpr (E == 4) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) w[k] = *reinterpret_cast<const uint32_t*>(col + k * PITCH);
                } else if constexpr (E == 2) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        w[k] = *reinterpret_cast<const uint16_t*>(col + 2 * k * PITCH) |
                               (uint32_t) * reinterpret_cast<const uint16_t*>(col + (2 * k + 1) * PITCH) << 16;
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        w[k] = col[4 * k * PITCH] | (uint32_t)col[(4 * k + 1) * PITCH] << 8 |
                               (uint32_t)col[(4 * k + 2) * PITCH] << 16 | (uint32_t)col[(4 * k + 3) * PITCH] << 24;
                }
                *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
                for (int k = 0; k < m; ++k) {
                    if constexpr (E == 4)
                        *reinterpret_cast<uint32_t*>(dst + 4 * k) = *reinterpret_cast<const uint32_t*>(col + k * PITCH);
                    else if constexpr (E == 2)
                        *reinterpret_cast<uint16_t*>(dst + 2 * k) = *reinterpret_cast<const uint16_t*>(col + k * PITCH);
                    else
                        dst[k] = col[k * PITCH];
                }
            }
        }
    }
}

template <typename T, int KV, int LAYOUT>
__global__ void __launch_bounds__(kThreads) pa_append_kernel(const AppendParams p) {
    constexpr int E = KV == kSame ? (int)sizeof(T) : 1;
    extern __shared__ __align__(16) uint8_t tile[];
    const bool key = (int)blockIdx.y < p.num_key_heads;
    const int head = key ? blockIdx.y : (int)blockIdx.y - p.num_key_heads;
    const int heads = key ? p.num_key_heads : p.num_value_heads, size = key ? p.key_head_size : p.value_head_size;
    const int t0 = blockIdx.x * kTokens, n = min(kTokens, p.num_tokens - t0);
    const int64_t stride = key ? p.key_stride : p.value_stride;
    const T* src = static_cast<const T*>(key ? p.key : p.value) + t0 * stride +
                   head * (key ? p.key_head_stride : p.value_head_stride);
    const int64_t page = (int64_t)kBS * size * E;
    uint8_t* cache = static_cast<uint8_t*>(key ? p.key_cache : p.value_cache) + head * page;

    pa::pdl_launch_dependents();
    pa::pdl_wait_primary();

    if (key) {
        if (size == 64)
            append_head<T, KV, LAYOUT, 64, true>(p, src, stride, cache, heads * page, p.k_scale, t0, n, tile);
        else if (size == 128)
            append_head<T, KV, LAYOUT, 128, true>(p, src, stride, cache, heads * page, p.k_scale, t0, n, tile);
        else
            append_head<T, KV, LAYOUT, 256, true>(p, src, stride, cache, heads * page, p.k_scale, t0, n, tile);
    } else {
        if (size == 64)
            append_head<T, KV, LAYOUT, 64, false>(p, src, stride, cache, heads * page, p.v_scale, t0, n, tile);
        else if (size == 128)
            append_head<T, KV, LAYOUT, 128, false>(p, src, stride, cache, heads * page, p.v_scale, t0, n, tile);
        else
            append_head<T, KV, LAYOUT, 256, false>(p, src, stride, cache, heads * page, p.v_scale, t0, n, tile);
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
