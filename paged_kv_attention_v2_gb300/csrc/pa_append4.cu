// pa_append4.cu -- pa_append_kv into 4-bit caches: every 16 successive elements x of a
// head become 16 e2m1 codes and one e4m3 scale s,
//     s = e4m3(max|x| / (6 g)),  code = e2m1(x / (g s)),     g = k_scale or v_scale,
// each quotient rounded once (half to even, saturated).
//
// A thread takes one block of 16: 32 bytes in, 8 bytes of codes and one of scale out, so
// nothing is exchanged but the scales of a row, which go out as one store.  Eight (head
// size 64: four) lanes make up a row, and the rows of successive slots lie side by side
// in the page.  Two blocks to a thread, CTAs of 128 threads: 32768 tokens of 8 + 8 heads of
// 128, bf16, 30.8 us (172 MB: 25.4 at the copy rate; one block 35, four 35, 256 threads
// 32).  The bytes alone take 26.5: the rest is the quantiser's issue slots.
//
// Rounding.  The decision between two codes is whether |x| passes t s g, with t half-way
// between the two: x has at most 11 significant bits, t s at most 7 and g 24, so the
// product has up to 31 and fp32 quotients can land on the wrong side.  Three facts settle
// it without 64 bits.  |x| >= T holds for the real T if and only if it holds for T
// rounded up to fp32, and |x| > T if and only if for T rounded down, as x is an fp32
// number itself: the comparisons of exact_codes and exact_scale are exact.  A quotient
// that is a few steps of fp32 off is on the wrong side only where T lies within a few steps
// of a number of x's own 11 (bf16: 8) bits: with the seven t's these are four significands
// (those of s g, 3 s g, 5 s g and 7 s g), looked at once for 16 elements, and in one
// block of 250 (bf16: 2000) the exact comparisons are needed.  And scales g of at most 12
// significant bits (the usual 1 or a power of two among them), whose T do lie on such
// numbers, meet none nearer than 2^-19 but them: there the quotient by one residual step
// (Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990) is right wherever it matters.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>
#include <type_traits>

#include "pa_cache.h"
#include "pa_host.cuh"
#include "pa_ptx.cuh"

namespace {

constexpr int kBS = PA_BLOCK_SIZE;
constexpr int kThreads = 128;

struct Scale4 {
    float g, inv;  // the tensor's scale and its reciprocal
    int brief;     // g has at most 12 significant bits
};

struct Append4Params {
    const void* key;
    const void* value;
    uint8_t* key_cache;
    uint8_t* value_cache;
    const int32_t* slots;
    int64_t key_stride, key_head_stride, value_stride, value_head_stride;
    int num_tokens, num_key_heads, key_head_size, num_value_heads, value_head_size, num_blocks;
    Scale4 k, v;
    int32_t* dev_error;
};

// Eight numbers rounded to e2m1 codes, the first in the lowest bits.
__device__ __forceinline__ uint32_t e2m1x8(const float (&x)[8]) {
    uint32_t d;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(d)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return d;
}

// The values of the e4m3 codes c and c + 1.
__device__ __forceinline__ float2 e4m3_pair(uint32_t c) {
    uint32_t h;
    asm("{\n\t.reg .b16 l;\n\tcvt.u16.u32 l, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(h) : "r"(c | (c + 1) << 8));
    return pa::unpack2<false>(h);
}

// e4m3(amax / (6 g)) as a code from one that is at most one off.  Not inlined: few blocks come here.
__device__ __noinline__ uint32_t exact_scale(uint32_t c, float amax, float g) {
    // 6 (half-way above c) g and 6 (half-way below c) g: 7 significant bits times g
    const float2 above = e4m3_pair(c);
    const float up = 3.f * (above.x + above.y);
    const bool odd = c & 1;
    if (c < 0x7e && (odd ? amax >= __fmul_ru(up, g) : amax > __fmul_rd(up, g))) return c + 1;
    if (c > 0) {
        const float2 below = e4m3_pair(c - 1);
        const float down = 3.f * (below.x + below.y);
        if (!(odd ? amax > __fmul_rd(down, g) : amax >= __fmul_ru(down, g))) --c;
    }
    return c;
}

// The same for a finite or infinite amax >= 0.
__device__ __forceinline__ uint32_t scale_code(float amax, const Scale4& q) {
    const float estimate = amax * q.inv * (1.f / 6);  // a few steps of fp32 off
    const uint32_t c = __nv_cvt_float_to_fp8(estimate, __NV_SATFINITE, __NV_E4M3), u = __float_as_uint(estimate);
    // within 16 steps of half-way between two normal numbers, or among the subnormal ones
    if (((u - 0x80000u + 16u) & 0xfffffu) <= 32u || estimate < 0x1p-6f) return exact_scale(c, amax, q.g);
    return c;
}

// Code of one element by exact comparisons (its sign aside).
__device__ __forceinline__ uint32_t exact_code(float x, const float (&t)[7]) {
    const float a = fabsf(x);
    // ties go to the even code: up past 0.75, 1.75 and 3.5, down at the others
    return (a > t[0]) + (a >= t[1]) + (a > t[2]) + (a >= t[3]) + (a > t[4]) + (a >= t[5]) + (a > t[6]);
}

// Not inlined: few blocks come here, and its registers are none of the others'.
template <bool BF16>
__device__ __noinline__ uint2 exact_codes(const uint4 a, const uint4 b, float s, float g) {
    const float t[7] = {__fmul_rd(0.25f * s, g), __fmul_ru(0.75f * s, g), __fmul_rd(1.25f * s, g), __fmul_ru(1.75f * s, g),
                        __fmul_rd(2.5f * s, g),  __fmul_ru(3.5f * s, g),  __fmul_rd(5.f * s, g)};
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t o[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 x = pa::unpack2<BF16>(w[i]);
        const uint32_t lo = exact_code(x.x, t) | (w[i] >> 12 & 8), hi = exact_code(x.y, t) | (w[i] >> 28 & 8);
        o[i >> 2] |= (lo | hi << 4) << (8 * (i & 3));
    }
    return make_uint2(o[0], o[1]);
}

template <bool BF16>
__device__ __forceinline__ uint32_t max_magnitude(uint32_t a, uint32_t b) {  // of pairs; a NaN stays one
    uint32_t d;
    if constexpr (BF16)
        asm("{\n\t.reg .b32 x, y;\n\tabs.bf16x2 x, %1;\n\tabs.bf16x2 y, %2;\n\tmax.NaN.bf16x2 %0, x, y;\n\t}" : "=r"(d) : "r"(a), "r"(b));
    else
        asm("{\n\t.reg .b32 x, y;\n\tabs.f16x2 x, %1;\n\tabs.f16x2 y, %2;\n\tmax.NaN.f16x2 %0, x, y;\n\t}" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Codes of a block and the code of its scale.
template <bool BF16>
__device__ __forceinline__ uint2 quantise(const uint4 a, const uint4 b, const Scale4& q, uint32_t& scale) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t m = max_magnitude<BF16>(w[0], w[1]);
#pragma unroll
    for (int i = 2; i < 8; ++i) m = max_magnitude<BF16>(m, w[i]);
    const float2 top = pa::unpack2<BF16>(m);
    const float amax = fmaxf(top.x, top.y);
    if (top.x != top.x || top.y != top.y) {  // a NaN: so is the whole block
        scale = 0x7f;
        return make_uint2(0, 0);
    }
    scale = scale_code(amax, q);
    if (scale == 0) return make_uint2(0, 0);
    const float s = e4m3_pair(scale - 1).y;
    const float p = s * q.g, inv = __frcp_rn(p);
    bool exact = !(p >= 0x1p-100f && p <= 0x1p100f);
    float y[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 x = pa::unpack2<BF16>(w[i]);
        y[2 * i] = x.x;
        y[2 * i + 1] = x.y;
    }
    if (q.brief) {
        exact |= !(amax * inv <= 0x1p60f);  // (an infinite quotient: its residual is NaN)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float v = y[i] * inv;
            y[i] = fmaf(-fmaf(v, p, -y[i]), inv, v);
        }
    } else {
        // whether a border lies within 8 steps of a number of x's precision
        constexpr uint32_t kLow = BF16 ? 0xffffu : 0x1fffu;
#pragma unroll
        for (int t = 1; t < 8; t += 2) exact |= ((__float_as_uint(t * p) + 8u) & kLow) <= 16u;
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] *= inv;
    }
    if (exact) return exact_codes<BF16>(a, b, s, q.g);
    const float lo[8] = {y[0], y[1], y[2], y[3], y[4], y[5], y[6], y[7]};
    const float hi[8] = {y[8], y[9], y[10], y[11], y[12], y[13], y[14], y[15]};
    return make_uint2(e2m1x8(lo), e2m1x8(hi));
}

// Rows [blockIdx.x * rows, ...) of one head, ITEMS blocks of 16 a thread.
template <typename T, int SIZE, int ITEMS>
__device__ __forceinline__ void store_rows(const Append4Params& p, const T* src, int64_t stride, uint8_t* cache,
                                           int64_t block_bytes, const Scale4& q) {
    constexpr int NB = SIZE / 16, ROWS = kThreads / NB;  // blocks of a row, rows at once
    const int b = threadIdx.x % NB, t0 = blockIdx.x * (ROWS * ITEMS) + threadIdx.x / NB;
    uint4 x[ITEMS][2];
    int slot[ITEMS];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int t = t0 + i * ROWS;
        slot[i] = -1;
        x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
        if (t < p.num_tokens) {
            const uint4* from = reinterpret_cast<const uint4*>(src + t * stride + b * 16);
            x[i][0] = from[0];
            x[i][1] = from[1];
            slot[i] = p.slots[t];
            if (slot[i] >= p.num_blocks * kBS) {
                if (blockIdx.y == 0 && p.dev_error) atomicOr(p.dev_error, PA_DEVERR_SLOT);
                slot[i] = -1;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        uint32_t s;
        const uint2 codes = quantise<std::is_same<T, __nv_bfloat16>::value>(x[i][0], x[i][1], q, s);
        // the scales of four neighbouring blocks in the first one's lane
        s |= __shfl_down_sync(0xffffffffu, s, 1) << 8;
        s |= __shfl_down_sync(0xffffffffu, s, 2) << 16;
        if (slot[i] < 0) continue;
        uint8_t* page = cache + (int64_t)(slot[i] >> 4) * block_bytes;
        const int o = slot[i] & 15;
        *reinterpret_cast<uint2*>(page + o * (SIZE / 2) + b * 8) = codes;
        if (b % 4 == 0) *reinterpret_cast<uint32_t*>(page + kBS * (SIZE / 2) + o * NB + b) = s;
    }
}

template <typename T, int ITEMS>
__global__ void __launch_bounds__(kThreads) pa_append4_kernel(const Append4Params p) {
    const bool key = (int)blockIdx.y < p.num_key_heads;
    const int head = key ? blockIdx.y : (int)blockIdx.y - p.num_key_heads;
    const int heads = key ? p.num_key_heads : p.num_value_heads, size = key ? p.key_head_size : p.value_head_size;
    const int64_t stride = key ? p.key_stride : p.value_stride;
    const T* src = static_cast<const T*>(key ? p.key : p.value) + head * (key ? p.key_head_stride : p.value_head_stride);
    const int64_t page = 9 * (int64_t)size;
    uint8_t* cache = (key ? p.key_cache : p.value_cache) + head * page;
    const Scale4 q = key ? p.k : p.v;
    pa::pdl_launch_dependents();
    pa::pdl_wait_primary();
    if (size == 64)
        store_rows<T, 64, ITEMS>(p, src, stride, cache, heads * page, q);
    else
        store_rows<T, 128, ITEMS>(p, src, stride, cache, heads * page, q);
}

Scale4 scale4_of(float scale) {
    Scale4 q;
    q.g = scale > 0.f ? scale : 1.f;
    q.inv = 1.f / q.g;
    int e;
    const float m = std::frexp(q.g, &e) * 4096.f;  // 12 bits in front of the point
    q.brief = m == std::floor(m);
    return q;
}

template <typename T>
bool launch(const Append4Params& p, int sms, void* stream) {
    const int heads = p.num_key_heads + p.num_value_heads;
    const int rows = kThreads / ((p.key_head_size < p.value_head_size ? p.value_head_size : p.key_head_size) / 16);
    auto grid = [&](int items) { return dim3((unsigned)((p.num_tokens + rows * items - 1) / (rows * items)), (unsigned)heads); };
    const dim3 one = grid(1);
    if ((int64_t)one.x * one.y < 8 * sms)
        return pa::launch_pdl(pa_append4_kernel<T, 1>, one, kThreads, 0, stream, p);
    return pa::launch_pdl(pa_append4_kernel<T, 2>, grid(2), kThreads, 0, stream, p);
}

}  // namespace

namespace pa {

bool append4(const pa_append_args* a, void* stream) {
    int dev = 0, sms = 0;
    if (!device_and_sms(&dev, &sms)) return false;
    Append4Params p = {};
    p.key = a->key;
    p.value = a->value;
    p.key_cache = static_cast<uint8_t*>(a->key_cache);
    p.value_cache = static_cast<uint8_t*>(a->value_cache);
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
    p.k = scale4_of(a->k_scale);
    p.v = scale4_of(a->v_scale);
    p.dev_error = a->dev_error;
    return a->dtype == PA_DTYPE_F16 ? launch<__half>(p, sms, stream) : launch<__nv_bfloat16>(p, sms, stream);
}

}  // namespace pa
