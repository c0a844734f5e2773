// pa_weights.cuh -- device code of pa_add_weights: the attention weights of a decode
// call, token by token, from its statistics.
//
//     w(row, h, t) = exp(z - M) / sum_p e_p exp(m_p - M),   M = max_p m_p,
// with the logits z computed again from the keys (the weights of all rows in memory would
// be four bytes for every row and token, and the decode would have to write them before
// their sum is known), summed over the rows of a sequence and the heads of a kv head.
//
// Every key is read once and nothing is shared between warps, so the pages go straight
// from memory to the registers of the tensor-core operand: tokens on M, rows on N, and
// the head dims in whatever order 16-byte loads bring them, the query's fragments in the
// same one.  Lane (r, cq) holds the 16-byte pieces cq, cq + 4, ... of the keys of tokens r
// and r + 8, in either layout.  A warp takes pages warp, warp + kWeightWarps, ... of the CTA's tile
// and loads one page while it works on the one before.  (Two or three pages ahead cost
// registers, so warps, and a wait for one page's loads is one for the later ones too: 32 x 4096
// fp16 38 us; a ring of asynchronous copies in shared memory 41 to 46.)  Four lanes then
// share a token's sum; no atomics, so results do not depend on the run.
// Measured: 32 x 4096 fp16, groups of seven, 24.6 us (139 MB: 20.4 at the copy rate; bound by
// memory), 4 x 100000 over 4-bit keys 31.5 (18.9; issued in 0.62 of the cycles, 216 instructions of
// a warp per page).  Tiles are cut for max_seq_len: with a window few of them have work (4 x 100000
// fp16, window of 4096: 23 us, its bytes 2.5), and of a ragged batch the longest sequence's have most.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "pa_cache.h"
#include "pa_fp4.cuh"
#include "pa_host.cuh"
#include "pa_ptx.cuh"

namespace pa {

constexpr int kWeightWarps = 8;

struct WeightParams {
    float* scores;
    const void* query;
    const void* key_cache;
    const int32_t* block_tables;
    const int32_t* seq_lens;
    const int32_t* query_start;
    const float* exp_sums;
    const float* max_logits;
    const float* alibi;
    bool relative_max;  // the maxima leave slope x (length - 1) out
    int32_t* dev_error;
    int num_seqs, num_heads, num_kv_heads, group, num_blocks, max_blocks_per_seq, max_seq_len, max_parts;
    int max_q_len, num_q_rows, window_left, tile_pages, tiles;  // tiles of the longest sequence
    uint32_t block_bytes;        // from a block of the cache to the next
    int token_step, piece_step;  // bytes between the tokens, and between the 16-byte pieces of one, in a page
    float scale, softcap, inv_softcap, decay;
};

// Cache element kinds
enum { kWSame = 0, kWE4M3 = 1, kWE5M2 = 2, kWE2M1 = 3 };

__device__ __forceinline__ void weights_report(const WeightParams& p, int bits) {
    if (p.dev_error) atomicOr(p.dev_error, bits);
}

// Keys of one page in registers, and their products with the query rows.
template <typename T, int HEAD, int KV, int NT>
struct PageKeys {
    static constexpr bool kF32 = std::is_same<T, float>::value, kBF = std::is_same<T, __nv_bfloat16>::value;
    static constexpr bool kFp4 = KV == kWE2M1;
    static constexpr int kBits = kFp4 ? 4 : (KV != kWSame ? 8 : 8 * (int)sizeof(T));
    static constexpr int kPageBytes = kFp4 ? 9 * HEAD : 16 * HEAD * kBits / 8;
    static constexpr int kWords = HEAD * kBits / 8 / 16;         // 32-bit words of a token's key in a lane
    static constexpr int kPieces = kFp4 ? 1 : kWords / 4;        // in pieces of 16 bytes (4-bit: one of 8 or 16)
    static constexpr int kValues = 32 / kBits;                   // elements of a word
    // the query's fragments: as many words of 16 bits x 2 as the key's elements need, or fp32
    static constexpr int kQWords = kF32 ? kWords : kWords * kValues / 2;

    uint32_t k[2][kWords];
    uint32_t s[2];  // 4-bit: the scales of a lane's one or two blocks

    // Bytes from a page's start to this lane's first piece of token r, and (4-bit) to its scales of that token.
    static __device__ __forceinline__ int offset(const WeightParams& p, int r, int cq) {
        return kFp4 ? r * (HEAD / 2) + cq * (HEAD / 8) : r * p.token_step + cq * p.piece_step;
    }
    static __device__ __forceinline__ int scale_offset(int r, int cq) {
        return 8 * HEAD + r * (HEAD / 16) + cq * (HEAD / 64);
    }

    // this lane's pieces of tokens r and r + 8, from its own pointers
    __device__ __forceinline__ void load(const uint8_t* at, const uint8_t* scales, const WeightParams& p) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if constexpr (kFp4) {
                const uint8_t* a = at + 8 * h * (HEAD / 2);
                const uint8_t* b = scales + 8 * h * (HEAD / 16);
                if constexpr (HEAD == 128) {
                    const uint4 v = *reinterpret_cast<const uint4*>(a);
                    k[h][0] = v.x;
                    k[h][1] = v.y;
                    k[h][2] = v.z;
                    k[h][3] = v.w;
                    s[h] = *reinterpret_cast<const uint16_t*>(b);
                } else {
                    const uint2 v = *reinterpret_cast<const uint2*>(a);
                    k[h][0] = v.x;
                    k[h][1] = v.y;
                    s[h] = *b;
                }
            } else {
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    const uint4 v = __ldcs(reinterpret_cast<const uint4*>(at + 8 * h * p.token_step + 4 * i * p.piece_step));
                    k[h][4 * i] = v.x;
                    k[h][4 * i + 1] = v.y;
                    k[h][4 * i + 2] = v.z;
                    k[h][4 * i + 3] = v.w;
                }
            }
        }
    }

    // Fragments of one query row in the order of the keys' elements (row: null for none).
    static __device__ __forceinline__ void load_query(const T* row, uint32_t (&q)[kQWords], int cq, uint32_t& top) {
        if (!row) {
#pragma unroll
            for (int i = 0; i < kQWords; ++i) q[i] = 0;
            return;
        }
        constexpr int kRun = kFp4 ? HEAD / 4 : 128 / kBits;  // successive elements of a piece
        constexpr int kRunWords = kF32 ? kRun : kRun / 2;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const T* from = row + (cq + 4 * i) * kRun;
#pragma unroll
            for (int w = 0; w < kRunWords; w += 4) {
                const uint4 v = *reinterpret_cast<const uint4*>(from + (kF32 ? w : 2 * w));
                q[i * kRunWords + w] = v.x;
                q[i * kRunWords + w + 1] = v.y;
                q[i * kRunWords + w + 2] = v.z;
                q[i * kRunWords + w + 3] = v.w;
            }
        }
        if constexpr (kBF && KV != kWSame) {  // fp16 products
#pragma unroll
            for (int i = 0; i < kQWords; ++i) {
                top = __vmaxu2(top, q[i] & 0x7fff7fffu);
                q[i] = bf16x2_to_f16(q[i]);
            }
        }
    }

    static __device__ __forceinline__ void fp8x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
        if constexpr (KV == kWE4M3)
            asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
                : "=r"(lo), "=r"(hi) : "r"(w));
        else
            asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e5m2x2 %0, l;\n\tcvt.rn.f16x2.e5m2x2 %1, h;\n\t}"
                : "=r"(lo), "=r"(hi) : "r"(w));
    }

    // z[nt]: products of tokens r (elements 0, 1) and r + 8 (2, 3) with rows 2cq and 2cq + 1 of n-tile nt
    __device__ __forceinline__ void products(const uint32_t (&q)[NT][kQWords], float (&z)[NT][4]) const {
        float b[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) z[nt][e] = b[nt][e] = 0.f;
        if constexpr (kF32) {
            // each product in three tf32 terms, summed outside the tensor core (see consumer_tf32)
#pragma unroll
            for (int w = 0; w < kWords; w += 2) {
                uint32_t h[4], l[4];
                split_tf32(k[0][w], h[0], l[0]);
                split_tf32(k[1][w], h[1], l[1]);
                split_tf32(k[0][w + 1], h[2], l[2]);
                split_tf32(k[1][w + 1], h[3], l[3]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    uint32_t qh0, ql0, qh1, ql1;
                    split_tf32(q[nt][w], qh0, ql0);
                    split_tf32(q[nt][w + 1], qh1, ql1);
                    float c[4] = {0.f, 0.f, 0.f, 0.f};
                    mma_1688_tf32(c, l[0], l[1], l[2], l[3], qh0, qh1);
                    mma_1688_tf32(c, h[0], h[1], h[2], h[3], ql0, ql1);
                    mma_1688_tf32(c, h[0], h[1], h[2], h[3], qh0, qh1);
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[nt][e] += c[e];
                }
            }
        } else if constexpr (KV == kWSame) {
#pragma unroll
            for (int w = 0; w < kWords; w += 2)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma_16816<kBF>(w & 2 ? b[nt] : z[nt], k[0][w], k[1][w], k[0][w + 1], k[1][w + 1], q[nt][w], q[nt][w + 1]);
        } else if constexpr (kFp4) {
            uint32_t f[2][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t c = e4m3x2_to_f16(s[h]);
                f[h][0] = __byte_perm(c, c, 0x1010);
                f[h][1] = HEAD == 128 ? __byte_perm(c, c, 0x3232) : f[h][0];
            }
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
                uint32_t x[4], y[4];
                e2m1x8_to_f16(k[0][w], x);
                e2m1x8_to_f16(k[1][w], y);
                const int g = HEAD == 128 ? w >> 1 : 0;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint32_t a0 = hmul2(x[2 * u], f[0][g]), a1 = hmul2(y[2 * u], f[1][g]);
                    const uint32_t a2 = hmul2(x[2 * u + 1], f[0][g]), a3 = hmul2(y[2 * u + 1], f[1][g]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_16816<false>(u ? b[nt] : z[nt], a0, a1, a2, a3, q[nt][4 * w + 2 * u], q[nt][4 * w + 2 * u + 1]);
                }
            }
        } else {
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
                uint32_t a0, a1, a2, a3;
                fp8x4(k[0][w], a0, a2);
                fp8x4(k[1][w], a1, a3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma_16816<false>(w & 1 ? b[nt] : z[nt], a0, a1, a2, a3, q[nt][2 * w], q[nt][2 * w + 1]);
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) z[nt][e] += b[nt][e];
    }
};

template <typename T, int HEAD, int KV, int NT>
__global__ void __launch_bounds__(kWeightWarps * 32) pa_weights_kernel(const WeightParams p) {
    using Page = PageKeys<T, HEAD, KV, NT>;
    constexpr int BS = PA_BLOCK_SIZE;
    constexpr float kLog2 = 1.4426950408889634f;
    __shared__ float level[NT * 8];  // log of each row's sum (of its logits relative to the last token's position)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, cq = lane & 3;
    const int unit = blockIdx.x / p.num_kv_heads, kvh = blockIdx.x - unit * p.num_kv_heads;
    const int seq = unit / p.tiles, tile = unit - seq * p.tiles;
    pdl_launch_dependents();
    pdl_wait_primary();
    const int32_t* table = p.block_tables + (int64_t)seq * p.max_blocks_per_seq;
    // the ids of this warp's pages (the i-th is first + kWeightWarps i), a lane each, with the lengths: which of them
    // there are is seen below
    const int first = tile * p.tile_pages + warp, mine = first + kWeightWarps * lane;
    int ids = mine < p.max_blocks_per_seq ? table[mine] : -1;
    int len = p.seq_lens[seq];
    if (len < 0 || len > p.max_seq_len) {
        if (threadIdx.x == 0 && tile == 0 && kvh == 0) weights_report(p, PA_DEVERR_SEQ_LEN);
        len = len < 0 ? 0 : p.max_seq_len;
    }
    int q0 = seq, qn = 1;
    if (p.query_start) {
        q0 = p.query_start[seq];
        const int n = p.query_start[seq + 1] - q0;
        qn = min(max(n, 0), p.max_q_len);
        if (q0 < 0 || q0 > p.num_q_rows) q0 = qn = 0;
        qn = min(qn, p.num_q_rows - q0);
        if (qn != n && threadIdx.x == 0 && tile == 0 && kvh == 0) weights_report(p, PA_DEVERR_SEQ_LEN);
    }
    const int pages = (len + BS - 1) / BS, page0 = tile * p.tile_pages, page1 = min(page0 + p.tile_pages, pages);
    const int G = p.group, GE = qn * G;
    // keys that some row sees: [seen0, len)
    const int seen0 = p.window_left >= 0 ? max(0, len - qn - p.window_left) : 0;
    // pages before that keep their scores where nothing fades
    const int from = p.decay == 1.f ? seen0 / BS : 0;
    if (max(page0, from) >= page1) return;

    // this lane's places in block 0; a block further, block_bytes further
    const uint8_t* lane_keys = static_cast<const uint8_t*>(p.key_cache) + kvh * Page::kPageBytes + Page::offset(p, r, cq);
    const uint8_t* lane_scales = static_cast<const uint8_t*>(p.key_cache) + kvh * Page::kPageBytes + Page::scale_offset(r, cq);
    float* lane_score = p.scores + kvh * BS + r + 8 * (cq & 1);
    auto score_of = [&](int blk) { return lane_score + (uint64_t)(uint32_t)blk * (uint32_t)(p.num_kv_heads * BS); };
    const int mine_n = (page1 - first + kWeightWarps - 1) / kWeightWarps;  // (up to 32; none: at most 0)
    const int i0 = max(0, (from - first + kWeightWarps - 1) / kWeightWarps);
    if (lane >= i0 && lane < mine_n && (unsigned)ids >= (unsigned)p.num_blocks) weights_report(p, PA_DEVERR_BLOCK_ID);
    if (lane >= mine_n || (unsigned)ids >= (unsigned)p.num_blocks) ids = -1;
    auto id = [&](int i) { return i < mine_n ? __shfl_sync(0xffffffffu, ids, i) : -1; };  // (out of range: -1)
    const int seen = GE > 0 ? seen0 : 0x7fffffff;
    // A page's keys and this lane's old score: lanes with cq 0 and 1 own tokens r and r + 8.  Of a page that is not
    // there, or that no row sees, 4-bit keys are block 0's, read and not used (loads in a branch, and each page's id
    // read and looked at in its turn: 34.0 us against 32.0, 4 x 100000); where a page is more bytes a branch is
    // cheaper (the same in fp16 with a window of 4096, all scores fading: 37 us, against 57 at the time).
    auto load = [&](int page, int blk, Page& k, float& old) {
        const bool need = blk >= 0 && (page + 1) * BS > seen;
        const uint64_t off = need ? (uint64_t)(uint32_t)blk * p.block_bytes : 0;
        if (Page::kFp4 || need) k.load(lane_keys + off, lane_scales + off, p);
        old = *score_of(max(blk, 0));
    };
    Page cur, next;
    float old_cur = 0.f, old_next = 0.f;
    int blk = id(i0), blk_next = -1;
    load(first + kWeightWarps * i0, blk, cur, old_cur);

    uint32_t q[NT][Page::kQWords], top = 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int v = nt * 8 + r;
        const T* row = v < GE ? static_cast<const T*>(p.query) +
                                    ((int64_t)(q0 + v / G) * p.num_heads + kvh * G + v % G) * HEAD
                              : nullptr;
        Page::load_query(row, q[nt], cq, top);
    }
    if (Page::kBF && KV != kWSame && ((top & 0xffffu) - 0x4780u < 0x3801u || (top >> 16) - 0x4780u < 0x3801u))
        weights_report(p, PA_DEVERR_QUERY_RANGE);

    // Each row's level from the statistics of its partitions
    const int parts = min((len + PA_PARTITION_SIZE - 1) / PA_PARTITION_SIZE, p.max_parts);
    for (int v = warp; v < NT * 8; v += kWeightWarps) {
        float M = -INFINITY, S = 0.f;
        if (v < GE) {
            const int64_t row = ((int64_t)(q0 + v / G) * p.num_heads + kvh * G + v % G) * p.max_parts;
            for (int i = lane; i < parts; i += 32) {
                const float m = p.max_logits[row + i], e = p.exp_sums[row + i];
                const float top_m = fmaxf(M, m);
                if (top_m != -INFINITY) S = S * exp2f((M - top_m) * kLog2) + e * exp2f((m - top_m) * kLog2);
                M = top_m;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float m = __shfl_xor_sync(0xffffffffu, M, o), s = __shfl_xor_sync(0xffffffffu, S, o);
            const float top_m = fmaxf(M, m);
            if (top_m != -INFINITY) S = S * exp2f((M - top_m) * kLog2) + s * exp2f((m - top_m) * kLog2);
            M = top_m;
        }
        if (lane == 0) {
            // maxima at absolute positions hold slope x position: taken off in one rounding, as the logits below leave it out
            if (p.alibi && !p.relative_max && v < GE) M = fmaf(-p.alibi[kvh * G + v % G], (float)(len - 1), M);
            level[v] = M == -INFINITY ? INFINITY : M + logf(S);  // a row that sees no key: weights zero
        }
    }
    __syncthreads();
    float lev[NT][2], slope[NT][2];
    bool there[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int v = nt * 8 + 2 * cq + e;
            there[nt][e] = v < GE;
            lev[nt][e] = v < GE ? level[v] * kLog2 : INFINITY;
            slope[nt][e] = p.alibi && v < GE ? p.alibi[kvh * G + v % G] : 0.f;
        }
    // tokens [all0, all1) are seen by every row
    const int all0 = p.window_left >= 0 ? max(0, len - 1 - p.window_left) : 0, all1 = len - qn + 1;

    const bool special = p.softcap > 0.f || p.alibi;
    const float to_log2 = special ? kLog2 : p.scale * kLog2;  // (scale and exponent in one step)

    // pages [in0, in1): every token is seen by every row and is older than this call's, so nothing is masked
    const int in0 = max((all0 + BS - 1) / BS, (seen0 + BS - 1) / BS), in1 = GE > 0 ? min(all1, len - qn) / BS : 0;
    auto work = [&](int page, int blk, const Page& keys, float old) {
        if (blk < 0) return;
        const int tok = page * BS;
        const bool edge = page < in0 || page >= in1;
        float w = 0.f;
        if (!edge || (tok + BS > seen0 && GE > 0)) {
            float z[NT][4], sum[2] = {0.f, 0.f};
            keys.products(q, z);
            if (special) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        z[nt][e] *= p.scale;
                        if (p.softcap > 0.f) z[nt][e] = p.softcap * tanhf(z[nt][e] * p.inv_softcap);
                        if (p.alibi) z[nt][e] = fmaf(slope[nt][e & 1], (float)(tok + r + 8 * (e >> 1) - (len - 1)), z[nt][e]);
                    }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    // (4-bit keys are finite or NaN for every row: rows that are not there need only their level)
                    z[nt][e] = Page::kFp4 || there[nt][e & 1] ? exp2_ftz(fmaf(z[nt][e], to_log2, -lev[nt][e & 1])) : 0.f;
            if (edge) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int t = tok + r + 8 * (e >> 1), pos = len - qn + (nt * 8 + 2 * cq + (e & 1)) / G;
                        if (t > pos || (p.window_left >= 0 && t < pos - p.window_left)) z[nt][e] = 0.f;
                    }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                sum[0] += z[nt][0] + z[nt][1];
                sum[1] += z[nt][2] + z[nt][3];
            }
            // lane cq 0 gets the first one's sum over the four lanes, cq 1 the second one's
            const float give = cq & 1 ? sum[0] : sum[1], keep = cq & 1 ? sum[1] : sum[0];
            w = keep + __shfl_xor_sync(0xffffffffu, give, 1);
            w += __shfl_xor_sync(0xffffffffu, w, 2);
        }
        const int t = tok + r + 8 * cq;
        if (cq < 2 && (!edge || t < len)) {
            // this call's tokens have no score yet
            *score_of(blk) = p.decay == 0.f || (edge && t >= len - qn) ? w : fmaf(p.decay, old, w);
        }
    };
    for (int i = i0; i < mine_n; ++i) {
        const int page = first + kWeightWarps * i;
        blk_next = id(i + 1);
        load(page + kWeightWarps, blk_next, next, old_next);
        work(page, blk, cur, old_cur);
        cur = next;
        old_cur = old_next;
        blk = blk_next;
    }
}

// Tiles: as many as fit on the GPU at once, or whole rounds of that where they would have more than kTilePages
// pages (a tile's first page comes some three dependent loads after its CTA starts, and its
// rows' statistics are read again, so few long ones), each a whole number of rounds of a CTA's warps.
constexpr int kTilePages = 32 * kWeightWarps;  // (their ids a lane each; 4 x 100000 e2m1: 128 pages 38.6 us, 256 35.0 at the time)

template <typename T, int HEAD, int KV, int NT>
bool launch_weights_rows(WeightParams& p, int sms, void* stream) {
    auto kern = pa_weights_kernel<T, HEAD, KV, NT>;
    static std::atomic<int> resident[kHostDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    int occ = dev < kHostDevices ? resident[dev].load() : 0;
    if (occ <= 0) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kern, kWeightWarps * 32, 0) != cudaSuccess || occ < 1) return false;
        if (dev < kHostDevices) resident[dev].store(occ);
    }
    const int64_t pages = (p.max_seq_len + PA_BLOCK_SIZE - 1) / PA_BLOCK_SIZE, units = (int64_t)p.num_seqs * p.num_kv_heads;
    const int64_t fit = (int64_t)sms * occ, least = (pages + kTilePages - 1) / kTilePages;  // tiles of a sequence's head
    int64_t per = (units * least + fit - 1) / fit * fit / units;
    if (per < least) per = least;
    int64_t tile = (pages + per - 1) / per;
    tile = (tile + kWeightWarps - 1) / kWeightWarps * kWeightWarps;
    p.tile_pages = (int)tile;
    p.tiles = (int)((pages + tile - 1) / tile);
    const int64_t grid = units * p.tiles;
    if (grid > 0x7fffffffLL) return false;
    return launch_pdl(kern, dim3((unsigned)grid), kWeightWarps * 32, 0, stream, p);
}

template <typename T, int HEAD, int KV>
bool launch_weights_head(WeightParams& p, int sms, void* stream) {
    return p.max_q_len * p.group <= 8 ? launch_weights_rows<T, HEAD, KV, 1>(p, sms, stream)
                                      : launch_weights_rows<T, HEAD, KV, 2>(p, sms, stream);
}

template <typename T, int KV>
bool launch_weights(WeightParams& p, int head_size, int sms, void* stream) {
    return head_size == 128 ? launch_weights_head<T, 128, KV>(p, sms, stream) : launch_weights_head<T, 64, KV>(p, sms, stream);
}

// One translation unit per query type; kv: kWSame .. kWE2M1
bool launch_weights_f32(WeightParams& p, int head_size, int sms, void* stream);
bool launch_weights_f16(WeightParams& p, int head_size, int kv, int sms, void* stream);
bool launch_weights_bf16(WeightParams& p, int head_size, int kv, int sms, void* stream);

}  // namespace pa
