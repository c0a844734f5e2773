// pa_append.cu -- pa_append_kv: the key and value rows of a step's tokens into
// the paged cache, through the slot map; fp8 caches quantised on the way.
//
// Bound by memory: every row is read once and written once.  One CTA takes some
// successive rows of one key or value head.  NHD caches, and keys of the split
// layout, move whole 16-byte chunks of a token's head, thread by thread, with no
// exchange between threads.
// Values of the split layout, [head dim][16 tokens], are transposed in shared
// memory: whole pages by ldmatrix and 8-byte (fp8: 4-byte) stores that make up one
// contiguous run per warp; other runs of successive slots are cut at the
// boundaries of 16-byte units of the page row, and a (unit, head dim) item is one
// 16-byte store when its unit is full, aligned pieces where the run ends inside
// it.  The rows of a CTA (64: six pages in seven of a prompt that begins inside
// one are whole; with 32 one in two, 32768 tokens bf16 74 us) do not wait for
// their slots.  Few rows are spread over more CTAs of eight rows each: the
// scattered single-element stores of 32 tokens took 4 us on four CTAs, 2.1 now.
// Measured, 32768 tokens, both at 6.8 TB/s (floor): split keys bf16 48.8 us (40.7), e4m3
// 43.4 (30.6); split values bf16 44.1 (40.7) when they begin with a page, 50.4 when inside
// one, e4m3 54.8 (30.6); keys and values NHD, bf16 40.5 (39.5), e4m3 36.2 (29.6).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <type_traits>

#include "pa_cache.h"
#include "pa_host.cuh"
#include "pa_ptx.cuh"

namespace {

constexpr int kBS = PA_BLOCK_SIZE;
constexpr int kThreads = 256;
constexpr int kRows = 64, kFewRows = 8;  // rows per CTA

// How a cache is scaled: its values are fp8(x / scale), the quotient rounded in fp32.
// y = x (1 / scale) is at most two steps off it, and y + (x - y scale) (1 / scale), the
// residual exact in a fused multiply-add, is the quotient to 2^-22 of a step before it
// is rounded (Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990).  With rows of at most 11 bits that can differ from
// the rounded quotient at an fp8 tie (at most 5 bits) only where the scale's mantissa
// is all ones: x - tie scale is a multiple of 2^-27, and near half a step of the tie
// times the scale for no other.  There, where the residual may leave fp32's range
// (scales outside 2^-80 .. 2^80) and beyond `top`, where y may be infinite, the chunk
// is divided.  32768 tokens e4m3, keys split / values split / NHD: y alone 40.1 / 53.2 /
// 33.8 us, so 43.4 / 54.8 / 36.2, every element divided 95.7 / 99.8 / 75.6.
struct Scale {
    float inv, scale;
    float top;  // largest |y| taken so; -1: divide everything
};

struct AppendParams {
    const void* key;
    const void* value;
    void* key_cache;
    void* value_cache;
    const int32_t* slots;
    int64_t key_stride, key_head_stride, value_stride, value_head_stride;
    int num_tokens, num_key_heads, key_head_size, num_value_heads, value_head_size, num_blocks;
    Scale k, v;
    int32_t* dev_error;
};

// Cache element kinds: the input's own bits, or fp8
enum { kSame = 0, kE4M3 = 1, kE5M2 = 2 };

template <int KV>
__device__ __forceinline__ uint32_t to_fp8x2(float a, float b) {
    // round to nearest even, beyond the largest finite value: that value
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, KV == kE4M3 ? __NV_E4M3 : __NV_E5M2);
}

// 16 elements divided and quantised.  Not inlined: its registers are no chunk's in flight.
template <typename T, int KV>
__device__ __noinline__ uint4 divided_chunk(const T* src, float scale) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] = __fdiv_rn((float)src[4 * i + k], scale);
        o[i] = to_fp8x2<KV>(y[0], y[1]) | to_fp8x2<KV>(y[2], y[3]) << 16;
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// 16 bytes of the cache from the input row at src (16-byte aligned): the same
// bytes, or 16 elements quantised.  (Plain loads, of the slots too: the previous
// kernel may write rows and slots while this one is resident, waiting for it, which
// the read-only path must not be used for.)
template <typename T, int KV>
__device__ __forceinline__ uint4 load_chunk(const T* src, const Scale& q) {
    const uint4* s = reinterpret_cast<const uint4*>(src);
    if constexpr (KV == kSame) {
        return *s;
    } else {
        constexpr bool BF = std::is_same<T, __nv_bfloat16>::value;
        const uint4 a = s[0], b = s[1];
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        bool divide = false;
        auto quotient = [&](float x) {
            const float y = x * q.inv;
            divide |= !(fabsf(y) <= q.top);
            return fmaf(-fmaf(y, q.scale, -x), q.inv, y);  // (so a -0 stays one)
        };
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 lo = pa::unpack2<BF>(w[2 * i]), hi = pa::unpack2<BF>(w[2 * i + 1]);
            o[i] = to_fp8x2<KV>(quotient(lo.x), quotient(lo.y)) | to_fp8x2<KV>(quotient(hi.x), quotient(hi.y)) << 16;
        }
        if (divide) return divided_chunk<T, KV>(src, q.scale);
        return make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// The slot of row t (-1: none), out of `n` rows at t0.
__device__ __forceinline__ int slot_of(const AppendParams& p, int t0, int t, int n) {
    if (t >= n) return -1;
    const int s = p.slots[t0 + t];
    if (s >= p.num_blocks * kBS) {
        if (blockIdx.y == 0 && p.dev_error) atomicOr(p.dev_error, PA_DEVERR_SLOT);
        return -1;
    }
    return s;
}

// Rows [t0, t0 + n) of one head, moved chunk by chunk: `src` its row t0, `cache` its
// page of block 0 (pages of one head `block_bytes` apart), SIZE its head size.
template <typename T, int KV, bool SPLIT, int SIZE, int ROWS>
__device__ __forceinline__ void move_rows(const AppendParams& p, const T* src, int64_t stride, uint8_t* cache,
                                          int64_t block_bytes, const Scale& q, int t0, int n) {
    constexpr int E = KV == kSame ? (int)sizeof(T) : 1;  // bytes of a cache element
    constexpr int X = 16 / E, CH = SIZE / X;             // elements of a chunk, chunks of a token's head
    constexpr int ITEMS = ROWS * CH, PER = (ITEMS + kThreads - 1) / kThreads;
    const int tid = threadIdx.x;
    // chunk (token, c) of a thread's item k: rows of chunks (NHD), or 8 tokens x 4
    // chunks per warp where the cache is [chunk][token] (split keys), so that
    // whole sectors are read and written
    constexpr int AHEAD = PER < 4 ? PER : 4;  // chunks in flight
#pragma unroll 1
    for (int k0 = 0; k0 < PER; k0 += AHEAD) {
        uint4 v[AHEAD];
        int64_t at[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int i = (k0 + k) * kThreads + tid;
            const int t = SPLIT ? (i >> 5) % (ROWS / 8) * 8 + (i & 7) : i / CH;
            const int c = SPLIT ? (i >> 5) / (ROWS / 8) * 4 + (i >> 3 & 3) : i % CH;
            at[k] = -1;
            if (i < ITEMS && t < n) {
                v[k] = load_chunk<T, KV>(src + t * stride + c * X, q);
                const int s = slot_of(p, t0, t, n);
                if (s >= 0)
                    at[k] = (int64_t)(s >> 4) * block_bytes +
                            (SPLIT ? (c * kBS + (s & 15)) * 16 : (s & 15) * (SIZE * E) + c * 16);
            }
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (at[k] >= 0) *reinterpret_cast<uint4*>(cache + at[k]) = v[k];
    }
}

// Values of the split layout: one head's rows of a block, transposed.
template <typename T, int KV, int SIZE, int ROWS>
__device__ __forceinline__ void transpose_rows(const AppendParams& p, const T* src, int64_t stride, uint8_t* cache,
                                               int64_t block_bytes, const Scale& q, uint8_t* tile) {
    constexpr int E = KV == kSame ? (int)sizeof(T) : 1;
    constexpr int X = 16 / E, CH = SIZE / X;
    constexpr bool PAGES = ROWS >= kBS && E < 4;  // whole pages by ldmatrix
    constexpr int PITCH = SIZE * E + 16;          // tile rows, one chunk more than a row
    constexpr int PER = (ROWS * CH + kThreads - 1) / kThreads;
    static_assert(ROWS <= 64, "one bit per row");
    __shared__ int64_t base_of[ROWS];  // byte offset of row t's first element in the cache, < 0: no slot
    __shared__ int unit_first[ROWS], unit_count[ROWS], unit_total, page_first[ROWS / kBS + 1], page_total;
    const int tid = threadIdx.x, lane = tid & 31;
    const int t0 = blockIdx.x * ROWS, n = min(ROWS, p.num_tokens - t0);
    constexpr int AHEAD = PER < 4 ? PER : 4;  // chunks in flight
    uint4 v[AHEAD];
    auto load = [&](int k0) {
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int i = (k0 + k) * kThreads + tid, t = i / CH, c = i % CH;
            if (t < n) v[k] = load_chunk<T, KV>(src + (t0 + t) * stride + c * X, q);
        }
    };
    load(0);
    // Units: maximal runs of successive slots inside one 16-byte unit of a page
    // row; with PAGES what whole pages among the rows leave over.  Warp 0, a bit
    // per row, two rows per lane.
    if (tid < 32) {
        constexpr int H = (ROWS + 31) / 32;
        int slot[H];
        bool joins[H];  // its slot follows on the row before's
        uint64_t breaks = 0, skipped = 0, starts = 0, whole = 0, taken = 0;
        int last = -2;  // slot of the row before this half
#pragma unroll
        for (int h = 0; h < H; ++h) {
            slot[h] = slot_of(p, t0, h * 32 + lane, n);
            int before = __shfl_up_sync(0xffffffffu, slot[h], 1);
            if (lane == 0) before = last;
            last = __shfl_sync(0xffffffffu, slot[h], 31);
            joins[h] = slot[h] >= 0 && before == slot[h] - 1;
            breaks |= (uint64_t)__ballot_sync(0xffffffffu, !joins[h]) << (32 * h);
            skipped |= (uint64_t)__ballot_sync(0xffffffffu, slot[h] < 0) << (32 * h);
        }
        if constexpr (PAGES) {
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const int t = h * 32 + lane;
                const bool w = slot[h] >= 0 && slot[h] % kBS == 0 && t + kBS <= ROWS &&
                               !(breaks & ((uint64_t)0xfffe << t));  // the fifteen rows behind it follow on
                whole |= (uint64_t)__ballot_sync(0xffffffffu, w) << (32 * h);
            }
            for (uint64_t w = whole; w; w &= w - 1) taken |= (uint64_t)0xffff << (__ffsll(w) - 1);
        }
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const bool begins = slot[h] >= 0 && !(taken >> (h * 32 + lane) & 1) && (!joins[h] || slot[h] % X == 0);
            starts |= (uint64_t)__ballot_sync(0xffffffffu, begins) << (32 * h);
        }
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const int t = h * 32 + lane;
            const uint64_t below = ((uint64_t)1 << t) - 1, above = ~below << 1;
            if (starts >> t & 1) {
                const uint64_t stop = (starts | skipped | taken) & above;  // first row that is not this unit's
                unit_first[__popcll(starts & below)] = t;
                unit_count[__popcll(starts & below)] = (stop ? __ffsll(stop) - 1 : 32 * H) - t;
            }
            if (whole >> t & 1) page_first[__popcll(whole & below)] = t;
            if (t < ROWS) base_of[t] = slot[h] < 0 ? -1 : (int64_t)(slot[h] >> 4) * block_bytes + (slot[h] & 15) * E;
        }
        if (lane == 0) {
            unit_total = __popcll(starts);
            page_total = __popcll(whole);
        }
    }
#pragma unroll 1
    for (int k0 = 0; k0 < PER; k0 += AHEAD) {
        if (k0 > 0) load(k0);
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int i = (k0 + k) * kThreads + tid, t = i / CH, c = i % CH;
            if (t < n) *reinterpret_cast<uint4*>(tile + t * PITCH + c * 16) = v[k];
        }
    }
    __syncthreads();
    if constexpr (PAGES) {
        // 32 / E head dims at a time: ldmatrix transposes 8 x 8 blocks of 16 bits;
        // with the tokens of its two blocks in the order 0 1 4 5 .. | 2 3 6 7 .. lane
        // (r, c) gets four successive tokens 4c .. 4c + 3 of head dim r (fp8: of dims
        // 2r and 2r + 1, sorted out by bytes).
        constexpr int DIMS = 32 / E;
        const int j = lane >> 3, i = lane & 7;
        const int tok = (i >> 1) * 4 + (i & 1) + (j & 1) * 2;
        for (int w = tid >> 5; w < page_total * (SIZE / DIMS); w += kThreads / 32) {
            const int t = page_first[w / (SIZE / DIMS)], d0 = w % (SIZE / DIMS) * DIMS;
            uint32_t a[4];
            pa::ldsm_x4_trans(pa::smem_u32(tile + (t + tok) * PITCH + d0 * E + (j >> 1) * 16), a[0], a[1], a[2], a[3]);
            const int r = lane >> 2, c = lane & 3;
            uint8_t* dst = cache + base_of[t] + (int64_t)d0 * (kBS * E);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t lo = a[2 * k], hi = a[2 * k + 1];
                if constexpr (E == 2) {
                    *reinterpret_cast<uint2*>(dst + (k * 8 + r) * 32 + c * 8) = make_uint2(lo, hi);
                } else {  // bytes: (token 4c: dims 2r, 2r + 1), (4c + 1: ...) | (4c + 2), (4c + 3)
                    uint8_t* row = dst + (k * 16 + 2 * r) * 16 + c * 4;
                    *reinterpret_cast<uint32_t*>(row) = __byte_perm(lo, hi, 0x6420);
                    *reinterpret_cast<uint32_t*>(row + 16) = __byte_perm(lo, hi, 0x7531);
                }
            }
        }
    }
    // item -> (unit, head dim): the E units that make up a page row (16 tokens) of
    // a full page lie side by side, so a warp writes whole sectors
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
            // 16-bit caches: pieces of 8, 4 or 2 bytes, as large as alignment and the run
            // allow (in an fp8 cache the same cost more than it saved)
            const int o0 = (int)(base_of[t] & 15);
            for (int k = 0; k < m;) {
                const int at = o0 + k * E, left = (m - k) * E;
                const uint8_t* c = col + k * PITCH;
                if constexpr (E == 4) {
                    *reinterpret_cast<uint32_t*>(dst + 4 * k) = *reinterpret_cast<const uint32_t*>(c);
                    ++k;
                } else if constexpr (E == 2) {
                    auto pair = [&](int q) {
                        return *reinterpret_cast<const uint16_t*>(c + q * PITCH) |
                               (uint32_t) * reinterpret_cast<const uint16_t*>(c + (q + 1) * PITCH) << 16;
                    };
                    if (at % 8 == 0 && left >= 8) {
                        *reinterpret_cast<uint2*>(dst + 2 * k) = make_uint2(pair(0), pair(2));
                        k += 4;
                    } else if (at % 4 == 0 && left >= 4) {
                        *reinterpret_cast<uint32_t*>(dst + 2 * k) = pair(0);
                        k += 2;
                    } else {
                        *reinterpret_cast<uint16_t*>(dst + 2 * k) = *reinterpret_cast<const uint16_t*>(c);
                        ++k;
                    }
                } else {
                    dst[k++] = *c;
                }
            }
        }
    }
}

template <typename T, int KV, int LAYOUT, int ROWS>
__global__ void __launch_bounds__(kThreads, 5) pa_append_kernel(const AppendParams p) {
    constexpr int E = KV == kSame ? (int)sizeof(T) : 1;
    constexpr bool SPLIT = LAYOUT == PA_LAYOUT_SPLIT;
    extern __shared__ __align__(16) uint8_t tile[];
    const bool key = (int)blockIdx.y < p.num_key_heads;
    const int head = key ? blockIdx.y : (int)blockIdx.y - p.num_key_heads;
    const int heads = key ? p.num_key_heads : p.num_value_heads, size = key ? p.key_head_size : p.value_head_size;
    const int64_t stride = key ? p.key_stride : p.value_stride;
    const T* src = static_cast<const T*>(key ? p.key : p.value) + head * (key ? p.key_head_stride : p.value_head_stride);
    const int64_t page = (int64_t)kBS * size * E;
    uint8_t* cache = static_cast<uint8_t*>(key ? p.key_cache : p.value_cache) + head * page;
    const Scale q = key ? p.k : p.v;

    pa::pdl_launch_dependents();
    pa::pdl_wait_primary();

    auto with_size = [&](auto size_c) {
        constexpr int SIZE = decltype(size_c)::value;
        if (SPLIT && !key) {
            transpose_rows<T, KV, SIZE, ROWS>(p, src, stride, cache, heads * page, q, tile);
        } else {
            const int t0 = blockIdx.x * ROWS;
            move_rows<T, KV, SPLIT, SIZE, ROWS>(p, src + t0 * stride, stride, cache, heads * page, q, t0,
                                                min(ROWS, p.num_tokens - t0));
        }
    };
    if (size == 64)
        with_size(std::integral_constant<int, 64>());
    else if (size == 128)
        with_size(std::integral_constant<int, 128>());
    else
        with_size(std::integral_constant<int, 256>());
}

Scale scale_of(float scale) {
    Scale q;
    q.scale = scale > 0.f ? scale : 1.f;
    q.inv = 1.f / q.scale;
    int e;
    const bool ones = std::frexp(q.scale, &e) == 1.f - 0x1p-24f;
    q.top = ones || q.scale < 0x1p-80f || q.scale > 0x1p80f ? -1.f : 65536.f;  // above both types' largest value
    return q;
}

bool size_ok(int d) { return d == 64 || d == 128 || d == 256; }

template <typename T, int KV, int ROWS>
bool launch_rows(const AppendParams& p, int layout, void* stream) {
    const dim3 grid((unsigned)((p.num_tokens + ROWS - 1) / ROWS), (unsigned)(p.num_key_heads + p.num_value_heads));
    const int e = KV == kSame ? (int)sizeof(T) : 1;
    if (layout == PA_LAYOUT_NHD)
        return pa::launch_pdl(pa_append_kernel<T, KV, PA_LAYOUT_NHD, ROWS>, grid, kThreads, 0, stream, p);
    const size_t tile = (size_t)ROWS * (p.value_head_size * e + 16);
    if constexpr (ROWS >= kBS && sizeof(T) == 4) {  // 66 KB for fp32 heads of 256
        static std::atomic<int> ready[pa::kHostDevices];
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return false;
        if (dev >= pa::kHostDevices || !ready[dev].load()) {
            if (cudaFuncSetAttribute(pa_append_kernel<T, KV, PA_LAYOUT_SPLIT, ROWS>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, ROWS * (256 * 4 + 16)) != cudaSuccess)
                return false;
            if (dev < pa::kHostDevices) ready[dev].store(1);
        }
    }
    return pa::launch_pdl(pa_append_kernel<T, KV, PA_LAYOUT_SPLIT, ROWS>, grid, kThreads, tile, stream, p);
}

template <typename T, int KV>
bool launch(const AppendParams& p, int layout, void* stream) {
    // Blocks of eight rows while blocks of 64 would leave SMs without one (runs of
    // 700 tokens, bf16 split, 8 + 8 heads: 300 rows 3.7 us; 1000 rows 4.5 us in
    // blocks of 64 and 6.8 in blocks of eight).
    int dev = 0, sms = 0;
    if (!pa::device_and_sms(&dev, &sms)) return false;
    const int64_t blocks = (int64_t)((p.num_tokens + kRows - 1) / kRows) * (p.num_key_heads + p.num_value_heads);
    return blocks < sms ? launch_rows<T, KV, kFewRows>(p, layout, stream) : launch_rows<T, KV, kRows>(p, layout, stream);
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
    if (a->num_tokens > 1 << 30) return PA_ERR_UNSUPPORTED;  // rows rounded up to blocks in 32 bits
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
    p.k = scale_of(a->k_scale);
    p.v = scale_of(a->v_scale);
    if (!std::isfinite(p.k.inv) || !std::isfinite(p.v.inv)) return PA_ERR_INVALID_ARG;
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
