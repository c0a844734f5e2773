// pa_compact.cu -- pa_compact_kv: the tokens that stay move to the front of their sequence's
// pages, in place.
//
// Bound by memory: every token that moves is read once and written once.  As kept[i] >= i and
// ascending, the place of token i of the result holds nothing that token i or a later one
// still needs but itself, so a chain of chunks is safe in place when the loads of a chunk
// come before its stores: a CTA loads a chunk into registers, waits at a barrier and stores it, with
// the next chunk's loads already on their way.  (Tokens to a chunk: 256, of NHD rows of 128 bytes
// 128, of longer ones 64.)  No CTA waits for another; the pieces of a head do not depend on
// each other: 256 bytes of a token's row (NHD), four of the 16-byte pieces of split keys, or 16 head
// dims of split values each make a chain of their own.  One sequence has few chains (8 heads of
// 128, bf16 NHD: 16, and 8 of the scores), each a round trip to memory per chunk, and is bound by
// that: 16384 to 2048 tokens 23.5 us (bytes: 2.5), 100000 to 8192 140 (10).
// Which way lanes run follows the layout: along a token's row, or along the tokens where a page holds
// [piece][token]; there successive tokens that stay are neighbours in the page, and a load takes
// few sectors.  Measured: 32 x 16384 to 2048, 8 heads of 128, bf16 NHD 94 us (542 MB: 80 at the
// copy rate); 32 x 4096 to 4032, 4 heads, fp16 split 101 (77; with the values token by token, two
// bytes to a load, 107).
#include <cuda_runtime.h>

#include <type_traits>

#include "pa_cache.h"
#include "pa_host.cuh"
#include "pa_ptx.cuh"

namespace {

constexpr int kBS = PA_BLOCK_SIZE;
constexpr int kThreads = 256;
constexpr unsigned kSingle = 1u << 16;  // above the bytes that __byte_perm reads
constexpr int kAhead = 4;         // chunks whose places are in shared memory (see move_chain)

// One array of the cache, in atoms: a token's are token * token_step into its page, a fixed step of the layout apart.
struct Array {
    uint8_t* base;
    int64_t block_bytes;  // from a block to the next
    int head_bytes;       // from a head's page to the next
    int heads;            // heads to a kv head
    int token_step;
    int chain_bytes;      // from a chain's first atom to the next one's
    int chains;           // per head
    int kind;             // kRow4 ..
};

enum { kRow2 = 0, kRow4, kRow8, kRow16, kPiece, kWide, kHalf, kByte, kWord8, kWord4 };

struct CompactParams {
    Array arrays[5];  // keys, values, 4-bit scales of both, scores
    int first[6];     // chains of a kv head before each array's
    const int32_t* block_tables;
    const int32_t* kept;
    const int32_t* new_seq_lens;
    int32_t* dev_error;
    int num_seqs, num_kv_heads, max_budget, num_blocks, max_blocks_per_seq;
};

struct Places {
    alignas(16) int64_t src[kAhead][kThreads];  // byte offsets of the tokens' first atoms; src < 0: stays
    alignas(16) int64_t dst[kAhead][kThreads];
};

// Moves a chain: LANES * NA atoms of type V of every token, from the first one of `page` (block 0's) on.  LANES
// neighbouring threads have successive atoms of a token, each of them NA of those, LANES apart, of each of NT
// tokens of a chunk.  STEP: bytes between successive atoms.
// With an element type S, an atom is two tokens' elements side by side (split values of 16 and 8 bits): a thread loads
// the one or two atoms that hold the pair it stores, and stores them at once.  An atom read that way may hold a
// neighbour that went or belongs to another pair of this chunk; a chunk's loads still come before its stores, and a
// chunk begins at an even token, so none is read that an earlier chunk's store may be writing.
template <typename V, int NA, int LANES, int NT, int STEP, typename S = void>
__device__ __forceinline__ void move_chain(const CompactParams& p, const Array& arr, uint8_t* page, int unit, int n, Places& at) {
    constexpr bool kPairs = !std::is_void<S>::value;
    constexpr int kChunk = kThreads / LANES * NT * (kPairs ? 2 : 1);  // tokens at once
    static_assert(kChunk <= kThreads, "a thread to plan each token");
    static_assert(!kPairs || kChunk % 32 == 0, "whole warps plan pairs");
    const int tid = threadIdx.x, seq = unit / p.num_kv_heads;
    const int32_t* table = p.block_tables + (int64_t)seq * p.max_blocks_per_seq;
    const int32_t* kept = p.kept + (int64_t)unit * p.max_budget;
    // Places of a chunk: each token's kept position is read one chunk before its pages' ids are looked up, so that
    // no chunk waits for both.  Written while the stores of the chunk three before may still be reading theirs, so
    // there are four.
    struct Token {
        int k, before;  // its position and the one kept before it
    };
    auto fetch = [&](int j) {
        const int i = j * kChunk + tid;
        Token t = {0, -1};
        if ((kChunk == kThreads || tid < kChunk) && i < n) {
            t.k = kept[i];
            if (i > 0) t.before = kept[i - 1];
        }
        return t;
    };
    auto plan = [&](int j, const Token& t) {
        if (kChunk < kThreads && tid >= kChunk) return;
        const int i = j * kChunk + tid;
        int64_t src = -1, dst = 0;
        if (i < n) {
            if (t.k < i || t.k <= t.before || t.k >= p.max_blocks_per_seq * kBS) {
                if (p.dev_error) atomicOr(p.dev_error, PA_DEVERR_SLOT);
            } else if (kPairs || t.k > i) {
                const int from = table[t.k / kBS], to = table[i / kBS];
                if ((unsigned)from >= (unsigned)p.num_blocks || (unsigned)to >= (unsigned)p.num_blocks) {
                    if (t.k > i && p.dev_error) atomicOr(p.dev_error, PA_DEVERR_BLOCK_ID);
                } else {
                    src = from * arr.block_bytes + t.k % kBS * arr.token_step;
                    dst = to * arr.block_bytes + i % kBS * arr.token_step;
                }
            }
        }
        if constexpr (kPairs) {
            // The even token's thread has the pair: its atoms (the second -1 where one holds both), the place and
            // the bytes of the result; kSingle where the other token of the pair is not moved.
            constexpr int E = (int)sizeof(V) / 2;
            const int64_t src1 = __shfl_down_sync(~0u, src, 1), dst1 = __shfl_down_sync(~0u, dst, 1);
            if (tid % 2 != 0) return;
            int64_t a = -1, b = -1, to = dst;
            unsigned bytes = 0;
            if (src >= 0 && src1 >= 0) {
                if (src != dst || src1 != dst1) {
                    a = src & -(int64_t)sizeof(V);
                    b = src1 & -(int64_t)sizeof(V);
                    unsigned lo = src & E, hi = src1 & E;
                    if (b == a) b = -1;
                    else hi += 4;
                    bytes = E == 2 ? (lo | (lo + 1) << 4 | hi << 8 | (hi + 1) << 12) : (lo | hi << 4);
                }
            } else if (src >= 0 || src1 >= 0) {
                const int64_t from = src >= 0 ? src : src1;
                to = src >= 0 ? dst : dst1;
                if (from != to) {
                    a = from & -(int64_t)sizeof(V);
                    const unsigned lo = from & E;
                    bytes = kSingle | lo | (lo + 1) << 4;
                }
            }
            *reinterpret_cast<longlong2*>(&at.src[j % kAhead][tid]) = make_longlong2(a, b);
            *reinterpret_cast<longlong2*>(&at.dst[j % kAhead][tid]) = make_longlong2(to, (int64_t)bytes);
            return;
        }
        at.src[j % kAhead][tid] = src;
        at.dst[j % kAhead][tid] = dst;
    };
    const int lane_token = tid / LANES, lane_atom = tid % LANES * STEP;
    constexpr int kRegs = kPairs ? 2 * NA : NA;
    V cur[NT][kRegs], next[NT][kRegs];
    auto load = [&](int j, V(&x)[NT][kRegs]) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if constexpr (kPairs) {
                const longlong2 s = *reinterpret_cast<const longlong2*>(&at.src[j % kAhead][2 * (lane_token + t * (kThreads / LANES))]);
                const uint8_t *a = page + s.x + lane_atom, *b = page + s.y + lane_atom;
                if (s.x >= 0) {
#pragma unroll
                    for (int k = 0; k < NA; ++k) x[t][k] = *reinterpret_cast<const V*>(a + k * LANES * STEP);
                }
                if (s.y >= 0) {
#pragma unroll
                    for (int k = 0; k < NA; ++k) x[t][NA + k] = *reinterpret_cast<const V*>(b + k * LANES * STEP);
                }
                continue;
            }
            const int64_t s = at.src[j % kAhead][lane_token + t * (kThreads / LANES)];
            const uint8_t* from = page + s + lane_atom;
            if (s >= 0) {
#pragma unroll
                for (int k = 0; k < NA; ++k) x[t][k] = *reinterpret_cast<const V*>(from + k * LANES * STEP);
            }
        }
    };
    auto store = [&](int j, const V(&x)[NT][kRegs]) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if constexpr (kPairs) {
                const int i = 2 * (lane_token + t * (kThreads / LANES));
                const longlong2 d = *reinterpret_cast<const longlong2*>(&at.dst[j % kAhead][i]);
                uint8_t* to = page + d.x + lane_atom;
                const unsigned bytes = (unsigned)d.y;
                if (at.src[j % kAhead][i] >= 0) {
#pragma unroll
                    for (int k = 0; k < NA; ++k) {
                        const unsigned v = __byte_perm(x[t][k], x[t][NA + k], bytes);
                        if (bytes & kSingle) *reinterpret_cast<S*>(to + k * LANES * STEP) = (S)v;
                        else *reinterpret_cast<V*>(to + k * LANES * STEP) = (V)v;
                    }
                }
                continue;
            }
            const int i = lane_token + t * (kThreads / LANES);
            uint8_t* to = page + at.dst[j % kAhead][i] + lane_atom;
            if (at.src[j % kAhead][i] >= 0) {
#pragma unroll
                for (int k = 0; k < NA; ++k) *reinterpret_cast<V*>(to + k * LANES * STEP) = x[t][k];
            }
        }
    };
    const int chunks = (n + kChunk - 1) / kChunk;
    const Token first = fetch(0), second = fetch(1);
    Token token = fetch(2);
    plan(0, first);
    plan(1, second);
    __syncthreads();
    load(0, cur);
    for (int j = 0; j < chunks; ++j) {
        const Token after = fetch(j + 3);
        load(j + 1, next);
        plan(j + 2, token);
        token = after;
        __syncthreads();  // every load of chunk j is done, and chunk j + 2's places are there
        store(j, cur);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < kRegs; ++k) cur[t][k] = next[t][k];
    }
}

__global__ void __launch_bounds__(kThreads) pa_compact_kernel(const CompactParams p) {
    __shared__ Places at;
    const int chains = p.first[5];
    const int unit = blockIdx.x / chains, chain = blockIdx.x - unit * chains;
    const int seq = unit / p.num_kv_heads, kvh = unit - seq * p.num_kv_heads;
    int which = 0;
    while (chain >= p.first[which + 1]) ++which;
    const Array& arr = p.arrays[which];
    const int c = chain - p.first[which], head = kvh * arr.heads + c / arr.chains, part = c % arr.chains;
    uint8_t* page = arr.base + (int64_t)head * arr.head_bytes;
    pa::pdl_launch_dependents();
    pa::pdl_wait_primary();
    int n = p.new_seq_lens[seq];
    if (n < 0 || n > p.max_budget) {
        if (threadIdx.x == 0 && p.dev_error) atomicOr(p.dev_error, PA_DEVERR_SEQ_LEN);
        n = n < 0 ? 0 : p.max_budget;
    }
    if (n == 0) return;
    switch (arr.kind) {
    case kRow2: move_chain<uint4, 1, 2, 2, 16>(p, arr, page, unit, n, at); break;
    case kRow4: move_chain<uint4, 1, 4, 4, 16>(p, arr, page + part * arr.chain_bytes, unit, n, at); break;
    case kRow8: move_chain<uint4, 1, 8, 4, 16>(p, arr, page + part * arr.chain_bytes, unit, n, at); break;
    case kRow16: move_chain<uint4, 1, 16, 4, 16>(p, arr, page + part * arr.chain_bytes, unit, n, at); break;
    case kPiece: move_chain<uint4, 4, 1, 1, 256>(p, arr, page + part * arr.chain_bytes, unit, n, at); break;
    case kWide: move_chain<uint32_t, 8, 2, 2, 64>(p, arr, page + part * arr.chain_bytes, unit, n, at); break;
    case kHalf: move_chain<uint32_t, 4, 4, 2, 32, uint16_t>(p, arr, page + part * arr.chain_bytes, unit, n, at); break;
    case kByte: move_chain<uint16_t, 4, 4, 2, 16, uint8_t>(p, arr, page + part * arr.chain_bytes, unit, n, at); break;
    case kWord8: move_chain<uint2, 1, 1, 1, 8>(p, arr, page, unit, n, at); break;
    default: move_chain<uint32_t, 1, 1, 1, 4>(p, arr, page, unit, n, at); break;
    }
}

bool size_ok(int d, bool fp4) { return d == 64 || d == 128 || (d == 256 && !fp4); }

}  // namespace

extern "C" pa_status pa_compact_kv(const pa_compact_args* a, void* stream) {
    if (!a) return PA_ERR_INVALID_ARG;
    if (a->num_seqs < 0 || a->num_kv_heads <= 0 || a->max_budget < 0 || a->num_key_heads <= 0 || a->num_value_heads <= 0 ||
        a->num_blocks <= 0 || a->max_blocks_per_seq < 0)
        return PA_ERR_INVALID_ARG;
    if (a->dtype != PA_DTYPE_F32 && a->dtype != PA_DTYPE_F16 && a->dtype != PA_DTYPE_BF16) return PA_ERR_INVALID_ARG;
    if (a->layout != PA_LAYOUT_SPLIT && a->layout != PA_LAYOUT_NHD) return PA_ERR_INVALID_ARG;
    const int kv = a->kv_dtype;
    if (kv != PA_KV_SAME && kv != PA_KV_FP8_E4M3 && kv != PA_KV_FP8_E5M2 && kv != PA_KV_FP4_E2M1) return PA_ERR_INVALID_ARG;
    if (a->num_key_heads % a->num_kv_heads != 0 || a->num_value_heads % a->num_kv_heads != 0) return PA_ERR_INVALID_ARG;
    const bool fp4 = kv == PA_KV_FP4_E2M1;
    if (kv != PA_KV_SAME && a->dtype == PA_DTYPE_F32) return PA_ERR_UNSUPPORTED;
    if (fp4 && a->layout != PA_LAYOUT_NHD) return PA_ERR_UNSUPPORTED;
    if (a->block_size != PA_BLOCK_SIZE || a->num_blocks >= 1 << 27 || a->max_blocks_per_seq >= 1 << 27 || a->max_budget > 1 << 30)
        return PA_ERR_UNSUPPORTED;
    if (!size_ok(a->key_head_size, fp4) || !size_ok(a->value_head_size, fp4)) return PA_ERR_UNSUPPORTED;
    if (a->num_key_heads > 65535 || a->num_value_heads > 65535) return PA_ERR_UNSUPPORTED;
    if (a->max_budget > (int64_t)a->max_blocks_per_seq * PA_BLOCK_SIZE) return PA_ERR_INVALID_ARG;
    if (a->num_seqs == 0 || a->max_budget == 0) return PA_OK;
    if (!a->key_cache || !a->value_cache || !a->block_tables || !a->kept || !a->new_seq_lens) return PA_ERR_INVALID_ARG;
    if (!pa::aligned(a->key_cache, 16) || !pa::aligned(a->value_cache, 16) || !pa::aligned(a->scores, 4) ||
        !pa::aligned(a->block_tables, 4) || !pa::aligned(a->kept, 4) || !pa::aligned(a->new_seq_lens, 4) ||
        !pa::aligned(a->dev_error, 4))
        return PA_ERR_INVALID_ARG;

    CompactParams p = {};
    const int kSlice = 256;  // bytes of a row to a chain (64: 102 us where 256 have 98, 32 x 16384 to 2048 bf16, which fill the GPU)
    const int e = kv != PA_KV_SAME ? 1 : (a->dtype == PA_DTYPE_F32 ? 4 : 2);
    for (int v = 0; v < 2; ++v) {
        Array& arr = p.arrays[v];
        const int heads = v ? a->num_value_heads : a->num_key_heads, d = v ? a->value_head_size : a->key_head_size;
        arr.base = static_cast<uint8_t*>(v ? a->value_cache : a->key_cache);
        arr.heads = heads / a->num_kv_heads;
        arr.head_bytes = fp4 ? 9 * d : kBS * d * e;
        arr.block_bytes = (int64_t)heads * arr.head_bytes;
        if (a->layout == PA_LAYOUT_NHD) {
            const int row = fp4 ? d / 2 : d * e;
            arr.token_step = row;
            const int wide = row < kSlice ? row : kSlice;
            arr.chains = row / wide;
            arr.chain_bytes = wide;
            arr.kind = wide == 32 ? kRow2 : (wide == 64 ? kRow4 : (wide == 128 ? kRow8 : kRow16));
        } else if (!v) {
            arr.token_step = 16;
            arr.chain_bytes = 4 * 16 * kBS;
            arr.chains = d * e / 64;
            arr.kind = kPiece;
        } else {
            arr.token_step = e;
            arr.chain_bytes = 16 * e * kBS;
            arr.chains = d / 16;
            arr.kind = e == 4 ? kWide : (e == 2 ? kHalf : kByte);
        }
        if (fp4) {  // the scales behind the codes
            Array& s = p.arrays[2 + v];
            s = arr;
            s.base += 8 * d;
            s.token_step = d / 16;
            s.chains = 1;
            s.kind = d == 128 ? kWord8 : kWord4;
        }
    }
    if (a->scores) {
        Array& s = p.arrays[4];
        s.base = reinterpret_cast<uint8_t*>(a->scores);
        s.heads = 1;
        s.head_bytes = kBS * 4;
        s.block_bytes = (int64_t)a->num_kv_heads * s.head_bytes;
        s.token_step = 4;
        s.chains = 1;
        s.kind = kWord4;
    }
    for (int i = 0; i < 5; ++i) p.first[i + 1] = p.first[i] + p.arrays[i].heads * p.arrays[i].chains;
    p.block_tables = a->block_tables;
    p.kept = a->kept;
    p.new_seq_lens = a->new_seq_lens;
    p.dev_error = a->dev_error;
    p.num_seqs = a->num_seqs;
    p.num_kv_heads = a->num_kv_heads;
    p.max_budget = a->max_budget;
    p.num_blocks = a->num_blocks;
    p.max_blocks_per_seq = a->max_blocks_per_seq;
    const int64_t grid = (int64_t)a->num_seqs * a->num_kv_heads * p.first[5];
    if (grid > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
    return pa::launch_pdl(pa_compact_kernel, dim3((unsigned)grid), kThreads, 0, stream, p) ? PA_OK : PA_ERR_LAUNCH;
}
