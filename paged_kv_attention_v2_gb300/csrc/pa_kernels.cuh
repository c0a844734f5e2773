// pa_kernels.cuh -- device code of the paged decode attention path (sm_103a).
//
// Partition kernel (Phase 1 of "paged_attention_v2_pytorch.py -- BI-V100
// PagedAttention V2 implementation", and the whole v1 pass):
//   persistent CTAs walk (sequence, kv head, 512-token partition) tiles; in v1
//   mode a tile is a whole (sequence, kv head).  Warp NC is the producer: it
//   walks seq_lens with a warp scan to find its tiles, reads each tile's block
//   table slice with one coalesced warp load, and streams every K/V page of
//   the tile into a STAGES-deep shared-memory ring with bulk (TMA) copies,
//   one mbarrier per stage.  Warps 0..NC-1 consume pages round-robin: the
//   whole GQA query group of the kv head is packed into the N dimension of
//   m16n8k16 tensor-core MMAs (tokens on M for Q.K^T, head dims on M for P.V),
//   so each page is read from HBM once for all heads of the group; the softmax
//   state stays online in registers.  At the end of a tile the consumer warps
//   merge their partial (max, sum, acc) through shared memory and write the
//   partition statistics (v2) or the output row (v1).
// Reduce kernel (Phase 2): per (sequence, head), M = max_p m_p,
//   w_p = exp(m_p - M) * e_p, out = sum_p w_p tmp_p / sum_p w_p.
#pragma once

#include <stdint.h>

#include <type_traits>

#include "pa_decode.h"
#include "pa_ptx.cuh"

namespace pa {

constexpr int kPart = PA_PARTITION_SIZE;  // tokens per partition
constexpr int kBS = PA_BLOCK_SIZE;        // tokens per page
constexpr int kSplit = PA_LAYOUT_SPLIT;
constexpr int kNHD = PA_LAYOUT_NHD;
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s: far beyond any legal wait (default)
constexpr float kLog2e = 1.4426950408889634f;

// Cache element kinds (template parameter KV of the partition kernel).
constexpr int kKvSame = 0;      // same 16-bit / 32-bit type as the query
constexpr int kKvE4M3 = 1;      // fp8 E4M3
constexpr int kKvE5M2 = 2;      // fp8 E5M2

// Shape of the partition kernel.  Ring stages per cache type, one 16-token
// page of K and V each.  One n-tile of 16-bit or fp32 pages: five consumer
// warps, with 10 stages (16-bit) or 5 stages of 16 KB (fp32), two CTAs of
// ~110 KB per SM; two n-tiles: four warps, 10 stages for 16-bit pages (two
// page streams of two warps, one n-tile each) or 8 stages of 16 KB for fp32
// (one CTA per SM); fp8 pages: four warps and 12 stages, so that three CTAs
// share an SM.  The stages are a multiple of the page streams.
constexpr int kStages16 = 10;      // 16-bit caches, one n-tile
constexpr int kStages16x2 = 10;    // 16-bit caches, two n-tiles (paired page streams)
constexpr int kStagesFp8 = 12;     // fp8 caches (three CTAs per SM fit)
constexpr int kStagesF32 = 5;      // fp32 caches, one n-tile (two CTAs per SM)
constexpr int kStagesF32x2 = 8;    // fp32 caches, two n-tiles (one CTA per SM)
constexpr int kStagesFp8x2Diff = 15; // fp8 caches, two n-tiles of a differential call (five warps)
constexpr int kConsumerWarps = 4;  // consumer warps per CTA
constexpr int kConsumerWarps5 = 5; // consumer warps per CTA, 16-bit or fp32 caches with one n-tile
constexpr int kPrefetchPages = 16; // pages of the first tile prefetched into L2 before the grid wait
// Value heads of 256 (differential attention with keys of 128): stages twice as
// large, one CTA per SM.  16-bit caches: five warps and ten stages (one n-tile),
// six warps in three page streams and nine stages (two), which leave the warps
// all the registers they want (eight warps are capped at 168 and spill: 64 ragged
// sequences, keys of 128 bf16, 171 -> 150 us; 4 x 50000, groups of seven, 150 -> 143).
constexpr int kStages16Wide = 10, kConsumerWarps16Wide = 5;
constexpr int kStages16Widex2 = 9, kConsumerWarps16Widex2 = 6;
// fp8 caches, 8 KB stages (one n-tile on eight warps, which spill: 32 x 4096 e4m3 92 us, on six 89)
constexpr int kStagesFp8Wide = 18, kConsumerWarpsFp8Wide = 6;
constexpr int kStagesFp8Widex2 = 16, kConsumerWarpsFp8Widex2 = 8;
constexpr int kStagesF32Wide = 5, kConsumerWarpsF32Wide = 5;   // fp32 caches: 32 KB stages
constexpr int kStagesF32Widex2 = 3, kConsumerWarpsF32Widex2 = 6;
constexpr int kStagesF32x2Diff = 8, kConsumerWarpsF32x2Diff = 8;  // fp32, value heads of 128, two n-tiles
constexpr int kReduceWarpMaxParts = 64;  // warp-per-row reduce up to this many partitions per row

constexpr int kDiffReduceFewParts = 4;  // differential rows: one warp per row up to this many partitions
constexpr int kReduceWarpsPerCta = 8;  // warp-per-row reduce: rows per CTA

struct Params {
    const void* query;
    const void* key_cache;
    const void* value_cache;
    const int32_t* block_tables;
    const int32_t* seq_lens;
    const float* alibi;
    void* out;
    float* exp_sums;
    float* max_logits;
    float* tmp_out;
    int32_t* dev_error;
    int num_seqs, num_heads, num_kv_heads, group;
    int num_blocks, max_blocks_per_seq, max_seq_len, max_parts;
    float scale, softcap, inv_softcap;  // scale includes k_scale for fp8 caches
    float v_scale;                       // fp8 caches: applied to the partition outputs
    int v1;
    int32_t* counters;  // [num_seqs][num_kv_heads] finished partitions (fused v2 only)
    int window_left;    // < 0: no window; else keys t >= pos - window_left (pos: the query's position)
    const int32_t* query_start;  // [num_seqs + 1] query rows per sequence, or NULL (one row each)
    int max_q_len;               // upper bound of query tokens per sequence (1 without query_start)
    int num_q_rows;              // rows of query / out / workspace
    int fused;          // v2 with the log-sum-exp merge done by the last CTA of each (seq, kv head)
    uint64_t wait_limit_ns;  // limit of every barrier wait (0: kWaitLimitNs)
    int withhold_page;       // test hook: CTA 0 withholds its first page copy (a wait runs out)
    int kv_evict_first;      // KV page copies marked evict_first (partition outputs small against L2)
    int32_t* tile_ctr;       // [2] dynamic schedule: tiles claimed, CTAs done (NULL: static schedule)
    int metadata_ready;      // block tables / lengths / query_start final: read before the grid wait
    uint32_t zero;           // 0 (mbar_arrive_after)
    // differential attention (the DIFF kernels): num_heads and group count
    // differential heads; statistics and tmp_out have two rows per head, one per map
    int part_len;            // tokens per partition (kPart in the other kernels)
    const float* lambdas;    // lambda of (row, head) at row * lambda_stride + head
    int64_t lambda_stride;
    const float* norm_weight;  // [value head size], or NULL (ones)
    float norm_eps, out_scale;
    int norm;                // RMS norm of each head's output
};

struct TileDesc {
    int seq, kvh, part, tok_begin, tok_end, len, flags, q0, qn, pad[3];
};
constexpr int kTileStop = 1;

__device__ __forceinline__ void report(const Params& p, int bits) {
    if (p.dev_error) atomicOr(p.dev_error, bits);
}

__device__ __forceinline__ int clamp_len(const Params& p, int raw) {
    return raw < 0 ? 0 : (raw > p.max_seq_len ? p.max_seq_len : raw);
}

// Tokens per partition: fixed, or for a differential call as the host chose.
template <bool DIFF>
__device__ __forceinline__ int part_len(const Params& p) {
    if constexpr (DIFF) return p.part_len;
    return kPart;
}

// cap * tanh(v / cap).  With QUICK (the differential kernels of 16-bit queries,
// whose consumers are short of issue slots with both maps' logits: e4m3 with four
// tokens 93 -> 88 us) as tanh(x) = 1 - 2 / (exp(2x) + 1) with the hardware's
// exponential and reciprocal; infinities included.  That is a few steps of 1 off,
// so the logit by some 2^-22 cap, whatever its size: 1.5e-5 at kQuickCap, well below
// what 16-bit keys and queries round to, but 0.1 at a cap of 1e6.  Above kQuickCap
// logits under a quarter of the cap take tanh's series instead (x^11 of it is below
// 2^-26 of x), larger ones are 2^-20 of themselves off.  (Same call, each way: no
// series 67.0 us, so 69.5, the series at any cap 72.6, and tanhf above kQuickCap 69.9
// but 2 to 5 % on calls without a cap, whose code it makes longer.)  An fp32 output
// would show the quick form (1.6e-6 against 5e-7).
constexpr float kQuickCap = 64.f;
template <bool QUICK>
__device__ __forceinline__ float soft_cap(const Params& p, float v) {
    const float x = v * p.inv_softcap;
    if constexpr (QUICK) {
        float z = p.softcap - __fdividef(2.f * p.softcap, exp2f(x * (2.f * kLog2e)) + 1.f);
        if (p.softcap > kQuickCap) {
            const float x2 = x * x;
            const float y = fmaf(x2, fmaf(x2, fmaf(x2, fmaf(x2, 62.f / 2835, -17.f / 315), 2.f / 15), -1.f / 3), 1.f);
            if (fabsf(x) < 0.25f) z = p.softcap * (x * y);
        }
        return z;
    }
    return p.softcap * tanhf(x);
}

// First key inside the sliding window of a query at position pos (0 without one).
__device__ __forceinline__ int window_lo_at(const Params& p, int pos) {
    if (p.window_left < 0) return 0;
    const int lo = pos - p.window_left;
    return lo > 0 ? lo : 0;
}

// First key any query token of a sequence sees: the window of its first query
// token, at position len - qn.
__device__ __forceinline__ int window_lo(const Params& p, int len, int qn = 1) {
    return window_lo_at(p, len - qn);
}

// Query rows of sequence s: first row and count, clamped to max_q_len tokens
// and to the rows that exist.
__device__ __forceinline__ void query_rows(const Params& p, int s, int& q0, int& qn) {
    if (!p.query_start) {
        q0 = s;
        qn = 1;
        return;
    }
    q0 = p.query_start[s];
    qn = p.query_start[s + 1] - q0;
    if (qn < 0 || qn > p.max_q_len || q0 < 0 || q0 > p.num_q_rows - min(max(qn, 0), p.max_q_len)) {
        report(p, PA_DEVERR_SEQ_LEN);
        qn = qn < 0 ? 0 : min(qn, p.max_q_len);
        if (q0 < 0 || q0 > p.num_q_rows) {
            q0 = 0;
            qn = 0;
        } else if (q0 + qn > p.num_q_rows) {
            qn = p.num_q_rows - q0;
        }
    }
}

// Pages covering tokens [tb, te): from page tb/16 to page ceil(te/16) - 1.
__device__ __forceinline__ int tile_pages(int tb, int te) {
    return te > tb ? (te + kBS - 1) / kBS - tb / kBS : 0;
}

// ------------------------------------------------------------------ config

template <typename T, int HEAD, int NT, int LAYOUT, int STAGES, int NC, int KV = kKvSame,
          bool MQ = false, bool DIFF = false>
struct Cfg {
    static constexpr bool kMQ = MQ;  // several query tokens per sequence (query_start given)
    // Differential attention: HEAD is the value head size 2d.  A pair of adjacent
    // key heads of d is one page of HEAD, [q1 | q2] one query row of HEAD, so
    // pages and queries move as they do for HEAD.  MMA column v (of NT * 8) is
    // map v / kRows of query row v % kRows: one n-tile holds both maps of up to
    // four rows, its B fragments zero where a column meets the other map's
    // keys; with two n-tiles each is one map of up to eight rows, and a warp of a
    // pair reads only its map's half of the key page.
    static constexpr bool kDiff = DIFF;
    static constexpr int kRows = DIFF ? NT * 4 : NT * 8;  // query rows (heads x query tokens)
    static constexpr int row_of(int v) { return DIFF ? v % kRows : v; }
    static constexpr bool kF32 = std::is_same<T, float>::value;
    static constexpr bool kBF16 = std::is_same<T, __nv_bfloat16>::value;
    static constexpr int kElem = sizeof(T);                // query / output element
    static constexpr int kKvElem = KV == kKvSame ? (int)sizeof(T) : 1;
    static constexpr int kPageBytes = kBS * HEAD * kKvElem;  // one page of K (or of V)
    // One page of K and one of V per ring stage.  (Two pages per fp8 NHD stage
    // halve its barrier rounds, max reductions and rescales, but their 8 KB
    // stages leave room for two CTAs per SM, against three with one-page
    // stages: measured, long100k_fp8 NHD 83.1 -> 75.9 µs and gqa4k_fp8 NHD
    // 34.2 -> 32.7 µs for the one-page stages.)
    static constexpr int kStageBytes = 2 * kPageBytes;  // K page, then V page
    static constexpr int kMaxG = NT * 8;                   // MMA columns: rows (heads x query tokens) handled
    // 16-bit caches with two n-tiles, and differential kernels with two but fp8
    // ones of value heads of 128: warps in pairs of page streams, one n-tile each;
    // every page is consumed by two warps.  (fp8: the pair would convert every
    // value twice; one warp with both n-tiles, five warps and fifteen stages: 32 x
    // 4096 e4m3 with four tokens 65 -> 57 us, both with one term of P.)
    static constexpr bool kPairs = NT == 2 && (DIFF ? (KV == kKvSame || HEAD > 128) : (KV == kKvSame && !kF32));
    static constexpr int kMergeRows = kPairs ? 8 : kMaxG;  // merge-buffer rows per warp
    static constexpr int kPageWarps = kPairs ? 2 : 1;      // warps that release each page
    // Differential fp32: K and V of a stage have barriers of their own.  A warp
    // holds its stage through a page's whole work, and there are no more stages
    // than warps: the key half is refilled while P.V runs, the value half during
    // the next page's Q.K^T (32 x 4096, groups of four, with the products still in
    // tf32: 102 -> 86 us).
    static constexpr bool kHalves = DIFF && kF32;
    static constexpr int kQBytes = kRows * HEAD * kElem;
    static constexpr int kTD = 2;                          // tile descriptor ring depth
    static constexpr int kMergeStride = HEAD + 4;          // floats; +4 breaks bank conflicts
    static constexpr int kThreads = (NC + 1) * 32;
    // NHD pages arrive through tensor maps with the 128-byte swizzle (3-D for
    // 16-bit and fp32, 2-D for fp8)
    static constexpr bool kTensorMap = LAYOUT == kNHD;
    static_assert(KV == kKvSame || !kF32, "fp8 caches: 16-bit query");

    static constexpr int oRing = 0;
    static constexpr int oQ = oRing + STAGES * kStageBytes;
    static constexpr int oMerge = oQ + kTD * kQBytes;
    static constexpr int oML = oMerge + NC * kMergeRows * kMergeStride * 4;
    static constexpr int oDesc = oML + NC * kMergeRows * 8;
    static constexpr int oBar = (oDesc + kTD * (int)sizeof(TileDesc) + 7) & ~7;
    static constexpr int oAbort = oBar + ((kHalves ? 4 : 2) * STAGES + 2 * kTD + 1) * 8;
    static constexpr int kSmemBytes = oAbort + 16 + 1024;  // + slack for 1024-B alignment

    static_assert(kPageBytes % 1024 == 0 || !kTensorMap, "swizzled pages need 1024-B alignment");
    // Within a tile, page j goes to page stream j % (NC / kPageWarps) (one
    // warp, or two with paired streams, each releasing it) and to ring stage
    // (base + j) % STAGES.  With STAGES a multiple of the streams every page of
    // a stage inside one tile belongs to the same stream, so no warp ever waits
    // on a stage's full barrier more than one phase ahead (a parity wait
    // cannot tell phase n from phase n + 2): the stage is refilled only once
    // both warps of a pair released it.  Across tiles the tile-end barrier of
    // the consumer warps gives the same guarantee.
    static_assert(STAGES % (NC / kPageWarps) == 0, "ring stages must be a multiple of the page streams");
    static_assert(STAGES <= 32, "one producer lane per stage");
    static_assert(kQBytes % 16 == 0, "bulk copy size");
};

struct Smem {
    uint32_t ring;       // shared address of stage 0
    uint32_t q;          // shared address of Q slot 0
    float* merge;
    float2* ml;
    TileDesc* desc;
    uint32_t full, empty, td_full, td_empty;  // shared addresses of barrier arrays
    uint32_t full_v, empty_v;  // of the value halves (Cfg::kHalves)
    uint32_t merge_bar;  // consumer warps: partial states written / epilogue reads done
    volatile int* abort;     // [0] give-up flag, [1] never set (drain waits), [2] last-arriver flag
    uint64_t wait_ns;        // limit of every barrier wait
};

// Ring stage and phase parity of the page NC pages further on (a consumer
// warp's next page of the tile): no division per page.
template <int STAGES, int NC>
__device__ __forceinline__ void advance_stage(uint32_t& st, uint32_t& ph) {
    static_assert(NC <= STAGES, "a warp's next page is at most one lap ahead");
    st += NC;
    if (st >= STAGES) {
        st -= STAGES;
        ph ^= 1u;
    }
}

// Bounded wait by every lane of a warp; the result is the same in all lanes.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort,
                                          uint64_t limit_ns) {
    const bool ok = mbar_wait(bar, parity, abort, limit_ns);
    return __all_sync(0xffffffffu, ok);
}

// Barrier among the NC consumer warps on an mbarrier of count NC (bounded,
// unlike bar.sync, so a warp that gave up cannot strand the others).
__device__ __forceinline__ bool consumer_sync(const Smem& sm, uint32_t& phase, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(sm.merge_bar);
    const bool ok = warp_wait(sm.merge_bar, phase & 1, sm.abort, sm.wait_ns);
    ++phase;
    return ok;
}

// ------------------------------------------------------------------ producer

// The (sequence, partition) of tile unit u when every sequence of the batch
// has max_parts partitions and there is no window (v1: one unit per
// sequence).  The producer's walk of seq_lens finds the real one; this guess
// lets the first tile's loads start before that walk.
__device__ __forceinline__ void guess_unit(const Params& p, int u, int& seq, int& part) {
    if (p.v1) {
        seq = u;
        part = 0;
    } else {
        seq = u / p.max_parts;
        part = u - seq * p.max_parts;
    }
}

// Run before the wait for the previous grid in the stream (programmatic
// dependent launch), while that grid finishes: prefetch into L2 the first
// pages of K and V of this CTA's first tile (guessed as above) and its query
// rows.  The inputs may still be written by the previous grid, so everything
// read here only steers the prefetch: lengths and block ids are read through
// L2 only (no L1 line is left behind for the reads after the wait), lengths
// are clamped and block ids outside the pool are skipped.
template <class C, int HEAD>
__device__ void prefetch_first_tile(const Params& p, int lane) {
    if (p.window_left >= 0 || p.withhold_page) return;
    const int Hkv = p.num_kv_heads;
    const int u = (int)blockIdx.x / Hkv, kvh = (int)blockIdx.x - u * Hkv;
    int seq, part;
    guess_unit(p, u, seq, part);
    if (seq >= p.num_seqs) return;
    const int len = clamp_len(p, __ldcg(p.seq_lens + seq));
    const int plen = part_len<C::kDiff>(p);
    const int tb = part * plen;
    const int te = p.v1 ? len : min(len, tb + plen);
    const int npg = min(kPrefetchPages, tile_pages(tb, te));
    if (lane < npg) {
        const int blk = __ldcg(p.block_tables + (int64_t)seq * p.max_blocks_per_seq + tb / kBS + lane);
        if ((unsigned)blk < (unsigned)p.num_blocks) {
            const int64_t off = ((int64_t)blk * Hkv + kvh) * C::kPageBytes;
            bulk_prefetch_l2(static_cast<const char*>(p.key_cache) + off, C::kPageBytes);
            bulk_prefetch_l2(static_cast<const char*>(p.value_cache) + off, C::kPageBytes);
        }
    }
    if (!C::kMQ && lane == 31)
        bulk_prefetch_l2(static_cast<const char*>(p.query) +
                             ((int64_t)seq * p.num_heads + (int64_t)kvh * p.group) * HEAD * C::kElem,
                         (uint32_t)(p.group * HEAD * C::kElem));
}

struct ProducerTile {
    int seq, kvh, part, tb, te, len, npages, q0, qn;
    bool valid;
};

template <class C, int HEAD, int STAGES>
__device__ void producer(const Params& p, const Smem& sm, const CUtensorMap* tmk,
                         const CUtensorMap* tmv, int lane) {
    const int S = p.num_seqs, Hkv = p.num_kv_heads;
    const int plen = part_len<C::kDiff>(p);
    const char* kbase = static_cast<const char*>(p.key_cache);
    const char* vbase = static_cast<const char*>(p.value_cache);
    const char* qbase = static_cast<const char*>(p.query);
    const uint32_t qbytes = (uint32_t)(p.group * HEAD * C::kElem);
    // KV pages are read once: first to leave L2, ahead of the partition outputs
    // (measured: a gain while those fit in L2, a loss once they overflow it)
    const uint64_t kvpol = p.kv_evict_first ? l2_policy_evict_first() : l2_policy_evict_normal();

    // Walk of seq_lens in chunks of 32 sequences: lane i holds sequence cb+i.
    int cb = 0, cu = 0;  // first sequence of the chunk, tile units before the chunk
    int c_len = 0, c_units = 0, c_p0 = 0, c_q0 = 0, c_qn = 0, c_incl = 0, c_total = 0;
    auto load_chunk = [&](int base) {
        const int s = base + lane;
        c_len = 0;
        c_units = 0;
        c_p0 = 0;
        c_q0 = 0;
        c_qn = 0;
        if (s < S) {
            const int raw = p.seq_lens[s];
            c_len = clamp_len(p, raw);
            if (c_len != raw) report(p, PA_DEVERR_SEQ_LEN);
            query_rows(p, s, c_q0, c_qn);  // a token at a negative position sees no key
            // v1: one tile per sequence; v2: one per partition that has keys in
            // the window (fused v2 keeps one empty tile for an empty sequence so
            // that its output row is written)
            c_p0 = window_lo(p, c_len, c_qn) / plen;
            c_units = p.v1 ? 1 : (c_len + plen - 1) / plen - c_p0;
            if (p.fused && c_units == 0) c_units = 1;
        }
        c_incl = c_units;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, c_incl, o);
            if (lane >= o) c_incl += v;
        }
        c_total = __shfl_sync(0xffffffffu, c_incl, 31);
    };
    // Ramp: in a batch whose sequences all have max_parts partitions the first
    // tile of this CTA is known before seq_lens is read; load its block ids now,
    // in parallel with the walk, and keep them only if the walk confirms the tile.
    int spec_seq = -1, spec_tb = 0, spec_ids = 0;
    if (!p.v1 && p.window_left < 0) {
        int spec_part;
        guess_unit(p, (int)blockIdx.x / Hkv, spec_seq, spec_part);
        spec_tb = spec_part * plen;
        const int idx = spec_tb / kBS + lane;
        if (spec_seq < S && idx < p.max_blocks_per_seq)
            spec_ids = p.block_tables[(int64_t)spec_seq * p.max_blocks_per_seq + idx];
    }
    load_chunk(0);
    // Final metadata: lengths and block ids are read before the wait for the
    // previous grid, which must be done before the grid-wide tile counter
    // (dynamic schedule: here), the copies and the workspace are touched.
    if (p.metadata_ready && p.tile_ctr) pdl_wait_primary();

    // Tiles of this CTA (kv head fastest): blockIdx.x, then blockIdx.x +
    // gridDim.x, ... (static schedule) or, with tile counters, whatever tile
    // index the grid-wide counter hands out next (dynamic schedule: a CTA
    // that streams faster takes more tiles).  A claim is made one tile ahead
    // by lane 0, so its round trip overlaps a whole tile; the claimed indices
    // of a CTA increase, as the walk of seq_lens below needs.
    int tile = blockIdx.x;
    const bool dyn = p.tile_ctr != nullptr;
    int claimed = 0;  // lane 0: the tile after `tile` (dynamic schedule)
    auto claim = [&]() {
        if (lane == 0) claimed = (int)gridDim.x + atomicAdd(p.tile_ctr, 1);
    };
    if (dyn) claim();
    auto next_tile = [&]() {
        ProducerTile t;
        t.valid = false;
        t.seq = t.part = t.tb = t.te = t.len = t.npages = t.q0 = t.qn = 0;
        const int u = tile / Hkv;
        t.kvh = tile - u * Hkv;
        if (dyn) {
            tile = __shfl_sync(0xffffffffu, claimed, 0);
            claim();
        } else {
            tile += gridDim.x;
        }
        while (cb < S && u >= cu + c_total) {
            cu += c_total;
            cb += 32;
            load_chunk(cb);
        }
        if (cb >= S) return t;
        const int rel = u - cu;
        const unsigned hit = __ballot_sync(0xffffffffu, c_incl > rel);
        const int j = __ffs(hit) - 1;
        t.seq = cb + j;
        const int excl = __shfl_sync(0xffffffffu, c_incl - c_units, j);
        t.len = __shfl_sync(0xffffffffu, c_len, j);
        t.q0 = __shfl_sync(0xffffffffu, c_q0, j);
        t.qn = __shfl_sync(0xffffffffu, c_qn, j);
        const int lo = window_lo(p, t.len, t.qn);
        t.part = __shfl_sync(0xffffffffu, c_p0, j) + rel - excl;
        t.tb = p.v1 ? lo : max(t.part * plen, lo);
        t.te = p.v1 ? t.len : min(t.len, t.part * plen + plen);
        t.npages = tile_pages(t.tb, t.te);
        t.valid = true;
        return t;
    };
    // Block ids of pages [pc, pc + 32) of tile t, one per lane.  The load is
    // only issued here; its range check (check_ids) comes where the ids are
    // used, so that no copy waits on the load.
    auto load_ids = [&](const ProducerTile& t, int pc) {
        return (t.valid && pc + lane < t.npages)
                   ? p.block_tables[(int64_t)t.seq * p.max_blocks_per_seq + t.tb / kBS + pc + lane]
                   : 0;
    };
    auto check_ids = [&](int blk) {
        if ((unsigned)blk >= (unsigned)p.num_blocks) {
            report(p, PA_DEVERR_BLOCK_ID);
            blk = 0;
        }
        return blk;
    };

    uint32_t g = 0;  // pages issued by this CTA
    int k = 0;       // tiles issued by this CTA
    bool ok = true;
    ProducerTile cur = next_tile();
    int ids = check_ids((cur.valid && cur.seq == spec_seq && cur.tb == spec_tb) ? (lane < cur.npages ? spec_ids : 0)
                                                                                  : load_ids(cur, 0));
    if (p.metadata_ready && !p.tile_ctr) pdl_wait_primary();  // static schedule: first tile found
    while (ok && cur.valid) {
        // The next tile is walked to, and its first block ids loaded, only once
        // the first batch of this tile's copies is out (the walk may load
        // lengths): nothing delays the first copies of a tile.
        ProducerTile nxt;
        nxt.valid = false;
        bool have_nxt = false;

        const int slot = k % C::kTD;
        if (lane == 0) {
            ok = mbar_wait(sm.td_empty + slot * 8, ((k / C::kTD) & 1) ^ 1, sm.abort, sm.wait_ns);
            if (ok) {
                TileDesc& d = sm.desc[slot];
                d.seq = cur.seq;
                d.kvh = cur.kvh;
                d.part = cur.part;
                d.tok_begin = cur.tb;
                d.tok_end = cur.te;
                d.len = cur.len;
                d.q0 = cur.q0;
                d.qn = cur.qn;
                d.flags = 0;
                // the group's rows of every query token of the sequence: slot row
                // i * group + g holds query token i, head kvh * group + g
                mbar_arrive_expect_tx(sm.td_full + slot * 8, qbytes * (uint32_t)cur.qn);
                for (int qi = 0; qi < cur.qn; ++qi)
                    bulk_g2s(sm.q + slot * C::kQBytes + (uint32_t)qi * qbytes,
                             qbase + ((int64_t)(cur.q0 + qi) * p.num_heads + (int64_t)cur.kvh * p.group) *
                                         HEAD * C::kElem,
                             qbytes, sm.td_full + slot * 8);
            }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);

        for (int pc = 0; pc < cur.npages && ok; pc += 32) {
            const int n = min(32, cur.npages - pc);
            int ids_next = 0;  // block ids of the next 32 pages (this tile or the next one)
            // Issue in batches of up to STAGES pages, one stage per lane: the
            // stages of a batch are distinct, so each lane waits for exactly the
            // previous use of its own stage.
            for (int b0 = 0; b0 < n && ok; b0 += STAGES) {
                const int nb = min(STAGES, n - b0);
                const int blk = __shfl_sync(0xffffffffu, ids, (b0 + lane) & 31);
                bool lok = true;
                if (lane < nb) {
                    const uint32_t gg = g + (uint32_t)lane;
                    const uint32_t st = gg % STAGES, ph = (gg / STAGES) & 1;
                    lok = mbar_wait(sm.empty + st * 8, ph ^ 1, sm.abort, sm.wait_ns);
                    // test hook: CTA 0 never issues its first stage, so the consumer
                    // waiting for it runs out of time (bounded, no fault)
                    const bool withhold = p.withhold_page && blockIdx.x == 0 && gg == 0;
                    if (lok && !withhold) {
                        const uint32_t fb = sm.full + st * 8;
                        const uint32_t dk = sm.ring + st * C::kStageBytes, dv = dk + C::kPageBytes;
                        mbar_arrive_expect_tx(fb, C::kHalves ? C::kPageBytes : 2 * C::kPageBytes);
                        const int64_t page = (int64_t)blk * Hkv + cur.kvh;
                        if constexpr (C::kTensorMap && C::kKvElem == 1) {
                            // fp8 NHD: one box of 16 token rows x HEAD bytes per page
                            const int y = (int)(page * kBS);
                            if constexpr (C::kDiff)
                                tensor4d_g2s_hint(dk, tmk, 0, 0, 0, (int)(2 * page), fb, kvpol);
                            else
                                tensor2d_g2s_hint(dk, tmk, 0, y, fb, kvpol);
                            if constexpr (HEAD > 128)  // two boxes of 128 bytes a row
                                tensor3d_g2s_hint(dv, tmv, 0, y, 0, fb, kvpol);
                            else
                                tensor2d_g2s_hint(dv, tmv, 0, y, fb, kvpol);
                        } else if constexpr (C::kTensorMap) {
                            // 16-bit / fp32 NHD: the whole page in one box of the
                            // 3-D view (128-byte chunk of a row, row, chunk index),
                            // staged as HEAD * elem / 128 blocks of 16 rows x 128 bytes
                            // (a pair of key heads: the same blocks, map by map)
                            const int y = (int)(page * kBS);
                            if constexpr (C::kDiff)
                                tensor4d_g2s_hint(dk, tmk, 0, 0, 0, (int)(2 * page), fb, kvpol);
                            else
                                tensor3d_g2s_hint(dk, tmk, 0, y, 0, fb, kvpol);
                            if constexpr (!C::kHalves) tensor3d_g2s_hint(dv, tmv, 0, y, 0, fb, kvpol);
                        } else {
                            bulk_g2s_hint(dk, kbase + page * C::kPageBytes, C::kPageBytes, fb, kvpol);
                            if constexpr (!C::kHalves)
                                bulk_g2s_hint(dv, vbase + page * C::kPageBytes, C::kPageBytes, fb, kvpol);
                        }
                    }
                }
                ok = __all_sync(0xffffffffu, lok);
                if constexpr (C::kHalves) {
                    if (ok && lane < nb) {
                        const uint32_t gg = g + (uint32_t)lane;
                        const uint32_t st = gg % STAGES, ph = (gg / STAGES) & 1;
                        lok = mbar_wait(sm.empty_v + st * 8, ph ^ 1, sm.abort, sm.wait_ns);
                        if (lok) {
                            const uint32_t fb = sm.full_v + st * 8;
                            const uint32_t dv = sm.ring + st * C::kStageBytes + C::kPageBytes;
                            const int64_t page = (int64_t)blk * Hkv + cur.kvh;
                            mbar_arrive_expect_tx(fb, C::kPageBytes);
                            if constexpr (C::kTensorMap)
                                tensor3d_g2s_hint(dv, tmv, 0, (int)(page * kBS), 0, fb, kvpol);
                            else
                                bulk_g2s_hint(dv, vbase + page * C::kPageBytes, C::kPageBytes, fb, kvpol);
                        }
                    }
                    ok = __all_sync(0xffffffffu, lok);
                }
                g += (uint32_t)nb;
                if (b0 == 0) {  // first batch out: load the next ids while the rest streams
                    if (pc + 32 < cur.npages) {
                        ids_next = load_ids(cur, pc + 32);
                    } else {
                        if (!have_nxt) {
                            nxt = next_tile();
                            have_nxt = true;
                        }
                        ids_next = load_ids(nxt, 0);
                    }
                }
            }
            ids = check_ids(ids_next);
        }
        if (!have_nxt) {
            nxt = next_tile();
            if (cur.npages == 0) ids = check_ids(load_ids(nxt, 0));
        }
        ++k;
        cur = nxt;
    }

    if (lane == 0) {
        if (ok) {
            const int slot = k % C::kTD;
            ok = mbar_wait(sm.td_empty + slot * 8, ((k / C::kTD) & 1) ^ 1, sm.abort, sm.wait_ns);
            if (ok) {
                sm.desc[slot].flags = kTileStop;
                mbar_arrive(sm.td_full + slot * 8);
            }
        }
        if (!ok) {
            report(p, PA_DEVERR_TIMEOUT);
            *sm.abort = 1;
        }
        // No bulk copy may still be writing shared memory when the CTA exits:
        // wait (bounded) for the last phase issued on every stage.
        for (uint32_t st = 0; st < STAGES && st < g; ++st) {
            const uint32_t last = g - 1 - ((g - 1 - st) % STAGES);
            mbar_wait(sm.full + st * 8, (last / STAGES) & 1, sm.abort + 1, sm.wait_ns);
            if constexpr (C::kHalves) mbar_wait(sm.full_v + st * 8, (last / STAGES) & 1, sm.abort + 1, sm.wait_ns);
        }
        // Dynamic schedule: the last CTA to be done with claiming (its arrival
        // releases its claims) sets both counters back to zero for the next call.
        if (dyn && atom_add_acq_rel_gpu(p.tile_ctr + 1, 1) == (int)gridDim.x - 1) {
            p.tile_ctr[0] = 0;
            p.tile_ctr[1] = 0;
        }
    }
}

// ------------------------------------------------------------------ epilogue

// Columns of an output row that a lane of a warp holds: VEC = HEAD / 32, in
// groups of at most four successive ones.
template <int HEAD>
__device__ __forceinline__ int lane_col(int lane, int v) {
    constexpr int VEC = HEAD / 32;
    return VEC <= 4 ? lane * VEC + v : (v >> 2) * 128 + lane * 4 + (v & 3);
}

// Write row `o` of an output of type T, VEC columns per lane (lane_col).
template <typename T, int HEAD>
__device__ __forceinline__ void store_row(T* row, const float (&o)[HEAD / 32], int lane) {
    constexpr int VEC = HEAD / 32;
    constexpr bool BF = std::is_same<T, __nv_bfloat16>::value;
#pragma unroll
    for (int v = 0; v < VEC; v += (VEC < 4 ? VEC : 4)) {
        T* dst = row + lane_col<HEAD>(lane, v);
        if constexpr (std::is_same<T, float>::value) {
            if constexpr (VEC >= 4)
                *reinterpret_cast<float4*>(dst) = make_float4(o[v], o[v + 1], o[v + 2], o[v + 3]);
            else
                *reinterpret_cast<float2*>(dst) = make_float2(o[v], o[v + 1]);
        } else if constexpr (VEC >= 4) {
            uint2 w;
            w.x = pack2<BF>(o[v], o[v + 1]);
            w.y = pack2<BF>(o[v + 2], o[v + 3]);
            *reinterpret_cast<uint2*>(dst) = w;
        } else {
            *reinterpret_cast<uint32_t*>(dst) = pack2<BF>(o[v], o[v + 1]);
        }
    }
}

// The output row of a differential head from its two maps' outputs, by one warp:
//     o = o1 - lambda o2,  y = out_scale * weight * o / sqrt(mean(o^2) + eps)
// (without the norm y = out_scale * o).  All in fp32; one rounding at the store.
template <typename T, int HEAD>
__device__ __forceinline__ void diff_row(const Params& p, int64_t row, int h, float (&o1)[HEAD / 32],
                                         const float (&o2)[HEAD / 32], int lane) {
    constexpr int VEC = HEAD / 32;
    const float lambda = p.lambdas[row * p.lambda_stride + h];
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        o1[v] = fmaf(-lambda, o2[v], o1[v]);
        ss = fmaf(o1[v], o1[v], ss);
    }
    float sc = p.out_scale;
    if (p.norm) {
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, x);
        sc *= rsqrtf(ss * (1.f / HEAD) + p.norm_eps);
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        o1[v] *= sc;
        if (p.norm && p.norm_weight) o1[v] *= p.norm_weight[lane_col<HEAD>(lane, v)];
    }
    store_row<T, HEAD>(static_cast<T*>(p.out) + (row * p.num_heads + h) * HEAD, o1, lane);
}

// v1 output of a differential tile: one query row per consumer warp at a time,
// both maps merged over the warps that hold them.
template <class C, typename T, int HEAD, int NC>
__device__ void diff_tile_output(const Params& p, const TileDesc& d, const Smem& sm, int warp, int lane) {
    constexpr int VEC = HEAD / 32;
    constexpr int WR = NC / C::kPageWarps;
    const int G = p.group, n = (C::kMQ ? d.qn : 1) * G;
    for (int r = warp; r < n; r += NC) {
        float o[2][VEC];
#pragma unroll
        for (int map = 0; map < 2; ++map) {
            const int w0 = C::kPairs ? map * WR : 0, hl = C::kPairs ? r : map * C::kRows + r;
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int w = 0; w < WR; ++w) M = fmaxf(M, sm.ml[(w0 + w) * C::kMergeRows + hl].x);
#pragma unroll
            for (int v = 0; v < VEC; ++v) o[map][v] = 0.f;
#pragma unroll
            for (int w = 0; w < WR; ++w) {
                const float2 e = sm.ml[(w0 + w) * C::kMergeRows + hl];
                const float c = e.x == -INFINITY ? 0.f : exp2f((e.x - M) * kLog2e);
                L = fmaf(c, e.y, L);
                const float* a = sm.merge + ((w0 + w) * C::kMergeRows + hl) * C::kMergeStride;
#pragma unroll
                for (int v = 0; v < VEC; ++v) o[map][v] = fmaf(c, a[lane_col<HEAD>(lane, v)], o[map][v]);
            }
            const float inv = L > 0.f ? p.v_scale / L : 0.f;
#pragma unroll
            for (int v = 0; v < VEC; ++v) o[map][v] *= inv;
        }
        const int qi = C::kMQ ? r / G : 0;
        diff_row<T, HEAD>(p, (int64_t)d.q0 + qi, d.kvh * G + (r - qi * G), o[0], o[1], lane);
    }
}

// Merge the NC consumer warps' partial states of one tile and write either the
// partition statistics (v2) or the final output row (v1).  Each thread owns up
// to ITEMS (row, 4-column) items; all their shared-memory loads are issued
// before any arithmetic, so the merge costs one dependency chain, not ITEMS.
template <class C, typename T, int HEAD, int NC>
__device__ void tile_epilogue(const Params& p, const TileDesc& d, const Smem& sm, int tid) {
    constexpr int D4 = HEAD / 4;
    constexpr int ITEMS = (C::kMaxG * D4 + NC * 32 - 1) / (NC * 32);
    const int G = p.group;
    // row v of the merge buffers: query token v / G, head kvh * G + v % G
    // (differential: that of v % kRows, map v / kRows, both maps side by side)
    const int qn = C::kMQ ? d.qn : 1;
    const int GE = qn * G;
    const int n = (C::kDiff ? 2 * GE : GE) * D4;
    if constexpr (C::kDiff) {
        if (p.v1) {
            diff_tile_output<C, T, HEAD, NC>(p, d, sm, tid >> 5, tid & 31);
            return;
        }
    }
    auto column = [&](int idx) {  // item -> merge row
        const int v = idx / D4;
        if constexpr (C::kDiff) return v < GE ? v : C::kRows + v - GE;
        return v;
    };
    // warps holding a partial state of row h: all of them, or with paired page
    // streams the WR warps of the row's n-tile (its rows at h % 8 of their buffers)
    constexpr int WR = NC / C::kPageWarps;
    float2 e[ITEMS][WR];
    float4 a[ITEMS][WR];
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
        const int idx = tid + it * NC * 32;
        const int h = column(idx), d4 = idx % D4;
        const int w0 = C::kPairs ? (h >> 3) * WR : 0, hl = C::kPairs ? (h & 7) : h;
#pragma unroll
        for (int w = 0; w < WR; ++w) {
            if (idx < n) {
                e[it][w] = sm.ml[(w0 + w) * C::kMergeRows + hl];
                a[it][w] = *reinterpret_cast<const float4*>(
                    sm.merge + ((w0 + w) * C::kMergeRows + hl) * C::kMergeStride + 4 * d4);
            } else {
                e[it][w] = make_float2(-INFINITY, 0.f);
                a[it][w] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
    }
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
        const int idx = tid + it * NC * 32;
        if (idx >= n) break;
        const int col = column(idx), h = C::row_of(col), d4 = idx % D4;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < WR; ++w) M = fmaxf(M, e[it][w].x);
        float L = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < WR; ++w) {
            const float c = (e[it][w].x == -INFINITY) ? 0.f : exp2f((e[it][w].x - M) * kLog2e);
            L += c * e[it][w].y;
            o.x += c * a[it][w].x;
            o.y += c * a[it][w].y;
            o.z += c * a[it][w].z;
            o.w += c * a[it][w].w;
        }
        const float inv = L > 0.f ? p.v_scale / L : 0.f;
        o.x *= inv;
        o.y *= inv;
        o.z *= inv;
        o.w *= inv;
        const int qi = C::kMQ ? h / G : 0;
        const int head = d.kvh * G + (h - qi * G);
        int64_t sh = (int64_t)(d.q0 + qi) * p.num_heads + head;
        if constexpr (C::kDiff) sh = 2 * sh + col / C::kRows;  // statistics row of the map
        if (!C::kDiff && p.v1) {
            T* dst = static_cast<T*>(p.out) + sh * HEAD + 4 * d4;
            if constexpr (C::kF32) {
                *reinterpret_cast<float4*>(dst) = o;
            } else {
                uint2 v;
                v.x = pack2<C::kBF16>(o.x, o.y);
                v.y = pack2<C::kBF16>(o.z, o.w);
                *reinterpret_cast<uint2*>(dst) = v;
            }
        } else {
            const int64_t ps = sh * p.max_parts + d.part;
            // kept in L2 for the reduce that follows (the read demotes it)
            st_global_v4_hint(p.tmp_out + ps * HEAD + 4 * d4, o, l2_policy_evict_last());
            if (d4 == 0) {
                float m = M;
                // logits are kept relative to the tile's last token; move the
                // partition max into the sequence frame (last token of the
                // sequence) -- the reduce kernel finishes the shift to absolute
                // positions after merging.
                if (p.alibi) m += p.alibi[head] * (float)(d.tok_end - d.len);
                p.max_logits[ps] = m;
                p.exp_sums[ps] = L;
            }
        }
    }
}

template <typename T, int HEAD, bool L2ONLY>
__device__ __forceinline__ void merge_row_warp(const Params& p, int64_t row, int h, int len, int qn, int qi,
                                               int lane);
template <typename T, int HEAD, bool L2ONLY>
__device__ __forceinline__ void diff_merge_row(const Params& p, int64_t row, int h, int len, int qn, int qi, int lane);

// The rows of one (sequence, kv head), one per consumer warp at a time.  Not
// inlined: its loads then never share a register allocation with the page
// loop (three fp8 CTAs per SM need the kernel within 128 registers).
template <typename T, int HEAD, int NC, bool MQ, bool DIFF>
__device__ __noinline__ void merge_group(const Params& p, int seq_kvh_base, int q0, int qn, int len, int warp,
                                         int lane) {
    const int G = p.group;
    for (int r = warp; r < qn * G; r += NC) {
        const int qi = MQ ? r / G : 0;
        if constexpr (DIFF) {
            diff_merge_row<T, HEAD, true>(p, (int64_t)q0 + qi, seq_kvh_base + (r - qi * G), len, qn, qi, lane);
        } else {
            merge_row_warp<T, HEAD, true>(p, (int64_t)q0 + qi, seq_kvh_base + (r - qi * G), len, qn, qi, lane);
        }
    }
}

// End of a tile for the consumer warps: epilogue (merge of the warps' partial
// states, partition statistics or output row), then in fused v2 mode the
// arrival count of the (sequence, kv head) and, for its last partition, the
// Phase 2 merge: one (query row, head) per consumer warp at a time, the same
// row merge as the reduce kernel, with L2-only loads.  Returns false if a
// bounded wait gave up.
template <class C, typename T, int HEAD, int NC>
__device__ bool tile_finish(const Params& p, const TileDesc& d, const Smem& sm, int warp, int lane,
                            uint32_t& mphase) {
    const int tid = warp * 32 + lane;
    tile_epilogue<C, T, HEAD, NC>(p, d, sm, tid);
    if (!consumer_sync(sm, mphase, lane)) return false;  // epilogue done, merge buffers free
    if (!p.fused || p.v1) return true;
    if (tid == 0) {
        const int plen = part_len<C::kDiff>(p);
        const int P = (d.len + plen - 1) / plen - window_lo(p, d.len, d.qn) / plen;
        int* counter = p.counters + (int64_t)d.seq * p.num_kv_heads + d.kvh;
        // releases this CTA's partition results (every warp's, seen through the
        // barrier above) before the count; acquires the others' with it
        const int last = atom_add_acq_rel_gpu(counter, 1) == (P > 0 ? P : 1) - 1;
        if (last) *counter = 0;  // every tile has arrived: zero again for the next call
        sm.abort[2] = last ? 1 : 0;
    }
    if (!consumer_sync(sm, mphase, lane)) return false;
    if (sm.abort[2])
        merge_group<T, HEAD, NC, C::kMQ, C::kDiff>(p, d.kvh * p.group, d.q0, C::kMQ ? d.qn : 1, d.len, warp, lane);
    return true;
}

// ------------------------------------------------------------ online softmax

// Logits may exceed the running reference max by this much (natural-log units,
// 8 ln 2) before the reference moves: p = exp(z - m) then stays below 2^8,
// well inside the range of the fp16 / bf16 P operand.
constexpr float kLazyMax = 5.545177444479562f;

// One page of the online softmax (running max and sum, rescaled as new
// logits arrive) with which a tile streams one partition of Phase 1
// ("paged_attention_v2_pytorch.py -- BI-V100 PagedAttention V2", per-partition
// attention): rows are the page's tokens, columns this lane's heads.  z holds
// the logits (-inf where masked) and becomes p = exp(z - m).  The reference m
// of each head is the same in every lane of the warp; it moves only when some
// logit exceeds it by more than kLazyMax, and then to the running max of the
// whole warp (three shuffle rounds), with l and acc rescaled.  Otherwise a
// page costs no shuffle and no rescale.  mx keeps this lane's running max, for
// the exact statistics at the end of the tile (settle_max).
template <int NT, int KT, bool MQ>
__device__ __forceinline__ void softmax_page(float (&z)[NT][4], float (&m)[NT][2], float (&mx)[NT][2],
                                             float (&l)[NT][2], float (&acc)[KT][NT][4], bool edge) {
    bool need = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const float a = fmaxf(z[nt][0], z[nt][2]), b = fmaxf(z[nt][1], z[nt][3]);
        mx[nt][0] = fmaxf(mx[nt][0], a);
        mx[nt][1] = fmaxf(mx[nt][1], b);
        need |= (a - m[nt][0] > kLazyMax) || (b - m[nt][1] > kLazyMax);  // -inf - -inf: false
    }
    if (__any_sync(0xffffffffu, need)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float mn0 = mx[nt][0], mn1 = mx[nt][1];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                mn0 = fmaxf(mn0, __shfl_xor_sync(0xffffffffu, mn0, o));
                mn1 = fmaxf(mn1, __shfl_xor_sync(0xffffffffu, mn1, o));
            }
            // several query tokens: a row with no key in its range so far keeps
            // max -inf (masked pages only); take 0 as reference so no -inf - -inf
            // appears.  One token: every page holds a key of every row.
            const float mr0 = (MQ && mn0 == -INFINITY) ? 0.f : mn0;
            const float mr1 = (MQ && mn1 == -INFINITY) ? 0.f : mn1;
            const float al0 = exp2f((m[nt][0] - mr0) * kLog2e);
            const float al1 = exp2f((m[nt][1] - mr1) * kLog2e);
            m[nt][0] = mn0;
            m[nt][1] = mn1;
            l[nt][0] *= al0;
            l[nt][1] *= al1;
#pragma unroll
            for (int mt = 0; mt < KT; ++mt) {
                acc[mt][nt][0] *= al0;
                acc[mt][nt][1] *= al1;
                acc[mt][nt][2] *= al0;
                acc[mt][nt][3] *= al1;
            }
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const float mr0 = (MQ && edge && m[nt][0] == -INFINITY) ? 0.f : m[nt][0];
        const float mr1 = (MQ && edge && m[nt][1] == -INFINITY) ? 0.f : m[nt][1];
        z[nt][0] = exp2f((z[nt][0] - mr0) * kLog2e);
        z[nt][1] = exp2f((z[nt][1] - mr1) * kLog2e);
        z[nt][2] = exp2f((z[nt][2] - mr0) * kLog2e);
        z[nt][3] = exp2f((z[nt][3] - mr1) * kLog2e);
        l[nt][0] += z[nt][0] + z[nt][2];
        l[nt][1] += z[nt][1] + z[nt][3];
    }
}

// End of a warp's pages of a tile: move the reference of each head to the
// warp's exact running max (what the partition statistics hold), rescaling l
// and acc once.
template <int NT, int KT>
__device__ __forceinline__ void settle_max(float (&m)[NT][2], float (&mx)[NT][2], float (&l)[NT][2],
                                           float (&acc)[KT][NT][4]) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        float mn0 = mx[nt][0], mn1 = mx[nt][1];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            mn0 = fmaxf(mn0, __shfl_xor_sync(0xffffffffu, mn0, o));
            mn1 = fmaxf(mn1, __shfl_xor_sync(0xffffffffu, mn1, o));
        }
        // equal (also both -inf: no key seen): nothing to move
        const float al0 = mn0 == m[nt][0] ? 1.f : exp2f((m[nt][0] - mn0) * kLog2e);
        const float al1 = mn1 == m[nt][1] ? 1.f : exp2f((m[nt][1] - mn1) * kLog2e);
        m[nt][0] = mn0;
        m[nt][1] = mn1;
        l[nt][0] *= al0;
        l[nt][1] *= al1;
#pragma unroll
        for (int mt = 0; mt < KT; ++mt) {
            acc[mt][nt][0] *= al0;
            acc[mt][nt][1] *= al1;
            acc[mt][nt][2] *= al0;
            acc[mt][nt][3] *= al1;
        }
    }
}

// ------------------------------------------------------------------ consumers

// What lane 0 hands the query slot back with: its last word, or where one n-tile
// holds both maps, which lanes 0-15 and 16-31 read one after the other, a
// combination of both halves' last ones.
template <class C, int KQ>
__device__ __forceinline__ uint32_t last_query_word(const uint32_t (&q)[KQ][2]) {
    if constexpr (C::kDiff && C::kMaxG == 8)
        return q[KQ / 2 - 1][1] | __shfl_xor_sync(0xffffffffu, q[KQ - 1][1], 16);
    else
        return q[KQ - 1][1];
}

// Byte offset of this lane's ldmatrix row address inside a K page for k-step kk
// (A operand of Q.K^T: rows = 16 tokens, columns = head dims 16kk..16kk+15).
template <int LAYOUT>
__device__ __forceinline__ uint32_t k_frag_off(int lane, int kk) {
    const int j = lane >> 3, r = lane & 7;
    const int tok = r + ((j & 1) << 3);
    const int c = 2 * kk + (j >> 1);  // 8-element chunk of the head dim
    if constexpr (LAYOUT == kSplit) {
        return (uint32_t)((c * kBS + tok) * 16);  // [d/8][token][8]
    } else {
        // NHD page staged as [d/64][token][64] with the 128-byte swizzle
        return (uint32_t)((c >> 3) * 2048 + tok * 128 + (((c & 7) ^ (tok & 7)) << 4));
    }
}

// Byte offset of this lane's ldmatrix row address inside a V page for m-tile mt
// (A operand of P.V: rows = head dims 16mt..16mt+15, columns = 16 tokens).
template <int LAYOUT>
__device__ __forceinline__ uint32_t v_frag_off(int lane, int mt) {
    const int j = lane >> 3, r = lane & 7;
    if constexpr (LAYOUT == kSplit) {
        const int d = mt * 16 + r + ((j & 1) << 3);  // [d][token]: row d holds 16 tokens
        return (uint32_t)(d * 32 + (j >> 1) * 16);
    } else {
        const int tok = r + ((j >> 1) << 3);  // stored as token rows: loaded transposed
        const int c = 2 * mt + (j & 1);
        return (uint32_t)((c >> 3) * 2048 + tok * 128 + (((c & 7) ^ (tok & 7)) << 4));
    }
}

// Zero the V entries of tokens [t0, t1) in a staged page.  Split: [d][16 tokens].  NHD:
// swizzled blocks of 16 token rows of up to 128 bytes (the swizzle permutes 16-byte
// chunks within a row, so a row stays one token's).
template <class C, int LAYOUT, int HEAD>
__device__ __forceinline__ void zero_v(uint32_t vpage, int t0, int t1, int lane) {
    constexpr int E = C::kKvElem;
    if constexpr (LAYOUT == kSplit) {
        for (int d = lane; d < HEAD; d += 32)
            for (int t = t0; t < t1; ++t) {
                const uint32_t a = vpage + (uint32_t)((d * kBS + t) * E);
                if constexpr (E == 4)
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(0u) : "memory");
                else if constexpr (E == 2)
                    asm volatile("st.shared.u16 [%0], %1;" ::"r"(a), "h"((unsigned short)0) : "memory");
                else
                    asm volatile("st.shared.u8 [%0], %1;" ::"r"(a), "h"((unsigned short)0) : "memory");
            }
    } else {
        constexpr int ROW = HEAD * E < 128 ? HEAD * E : 128;  // bytes of a row of a block
        constexpr int CH = ROW / 16, BLOCKS = HEAD * E / ROW;
        const int n = (t1 - t0) * CH;
        for (int i = lane; i < n * BLOCKS; i += 32) {
            const int b = i / n, c = i - b * n;
            const uint32_t a = vpage + (uint32_t)(b * kBS * ROW + t0 * ROW + c * 16);
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(a), "r"(0u) : "memory");
        }
    }
}

// Zero the V entries of a page's tokens that no row of the tile sees, before the window
// and behind the end (where a slot may hold anything): their weight is zero, but the
// P.V product of zero and an infinity or a NaN is none.
template <class C, int LAYOUT, int HEAD>
__device__ __forceinline__ void zero_unseen(uint32_t vpage, int tok0, const TileDesc& d, int lane) {
    const int first = max(d.tok_begin - tok0, 0), valid = min(kBS, d.tok_end - tok0);
    if (first > 0 || valid < kBS) {
        zero_v<C, LAYOUT, HEAD>(vpage, 0, first, lane);
        zero_v<C, LAYOUT, HEAD>(vpage, valid, kBS, lane);
        fence_proxy_async_smem();
        __syncwarp();
    }
}

template <class C, typename T, int HEAD, int NT, int LAYOUT, int STAGES, int NC>
__device__ void consumer_mma(const Params& p, const Smem& sm, int warp, int lane) {
    constexpr bool BF = C::kBF16;
    // P in two 16-bit terms: bf16 keeps 8 significant bits of it, two terms 17.  A
    // differential output is a difference, normalised, and what one map's weights lose
    // grows as the maps cancel: fp16 takes two as well, 22 bits of a weight of a 2^-10th
    // or more of the reference and an absolute 2^-25 below (fp16's subnormal step).
    // Maps that cancel to a fiftieth, against the output's own rounding: fp16 2.06e-4
    // (2.06e-4), bf16 1.66e-3 (1.65e-3); a third bf16 term changes neither that nor
    // 4 x 100000, where what is left is the fp32 sums'.
    constexpr bool kTwoP = BF || C::kDiff;
    constexpr int KT = HEAD / 16;  // k-steps of Q.K^T, m-tiles of P.V
    // Two n-tiles: the warps work in pairs of page streams, one n-tile each
    // (rows nt0 * 8 .. nt0 * 8 + 7) on the pages j = pfirst (mod PSTRIDE), so
    // every page is read by two warps, each with one n-tile's registers.
    constexpr bool kPairs = C::kPairs;
    constexpr int NTW = kPairs ? 1 : NT;          // n-tiles per warp
    constexpr int PSTRIDE = kPairs ? NC / 2 : NC; // warps per page stream
    const int nt0 = kPairs ? warp / PSTRIDE : 0;
    // k-steps of Q.K^T: a warp of a differential pair takes its own map's half
    constexpr int KQ = C::kDiff && kPairs ? KT / 2 : KT;
    const uint32_t khalf = C::kDiff && kPairs ? (uint32_t)nt0 * (C::kPageBytes / 2) : 0u;
    const int pfirst = kPairs ? warp % PSTRIDE : warp;
    const int G = p.group;
    const int r = lane >> 2, cq = lane & 3;
    const bool has_alibi = p.alibi != nullptr;
    const bool has_cap = p.softcap > 0.f;
    uint32_t gbase = 0;
    uint32_t mphase = 0;
    for (int k = 0;; ++k) {
        const int slot = k % C::kTD;
        if (!warp_wait(sm.td_full + slot * 8, (k / C::kTD) & 1, sm.abort, sm.wait_ns)) {
            report(p, PA_DEVERR_TIMEOUT);
            *sm.abort = 1;
            return;
        }
        const TileDesc d = sm.desc[slot];
        if (d.flags & kTileStop) return;
        const int qn = C::kMQ ? d.qn : 1;
        const int GE = qn * G;  // rows of N: query token v / G, head kvh * G + v % G

        // Q as B fragments: B[k = head dim][n = row], rows >= GE are zero.
        uint32_t qb[NTW][KQ][2];
        const uint32_t qs = sm.q + slot * C::kQBytes;
#pragma unroll
        for (int nt = 0; nt < NTW; ++nt) {
            const int v = (nt0 + nt) * 8 + r, h = C::row_of(v);
#pragma unroll
            for (int kk = 0; kk < KQ; ++kk) {
                uint32_t b0 = 0, b1 = 0;
                // (one n-tile of both maps: zero against the other map's keys)
                if (h < GE && (!C::kDiff || kPairs || kk / (KT / 2) == v / C::kRows)) {
                    const int k0 = C::kDiff && kPairs ? nt0 * (HEAD / 2) + kk * 16 : kk * 16;
                    const uint32_t a = qs + (uint32_t)((h * HEAD + k0 + 2 * cq) * 2);
                    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(b0) : "r"(a));
                    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(b1) : "r"(a + 16));
                }
                qb[nt][kk][0] = b0;
                qb[nt][kk][1] = b1;
            }
        }
        const uint32_t qlast = last_query_word<C, KQ>(qb[NTW - 1]);
        __syncwarp();
        // Q and descriptor are in registers (lane 0 takes part in the last read)
        if (lane == 0) mbar_arrive_after(sm.td_empty + slot * 8, qlast, p.zero);

        float sl[NTW][2];
#pragma unroll
        for (int nt = 0; nt < NTW; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int h = C::row_of((nt0 + nt) * 8 + 2 * cq + e);
                sl[nt][e] = (has_alibi && h < GE) ? p.alibi[d.kvh * G + h % G] : 0.f;
            }
        // key range of each of this lane's rows: its query token's position and
        // window, within the tile (padded rows get the tile's range)
        int klo[NTW][2], khi[NTW][2];
#pragma unroll
        for (int nt = 0; nt < NTW; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int v = C::row_of((nt0 + nt) * 8 + 2 * cq + e);
                int lo = d.tok_begin, hi = d.tok_end - 1;
                if (C::kMQ && v < GE) {
                    const int pos = d.len - qn + v / G;
                    hi = min(hi, pos);
                    lo = max(lo, window_lo_at(p, pos));
                }
                klo[nt][e] = lo;
                khi[nt][e] = hi;
            }
        // keys inside every row's range: a page within [lo_all, hi_all] needs no mask
        // (one query token: the tile's own range)
        const int hi_all = C::kMQ ? min(d.tok_end - 1, d.len - qn) : d.tok_end - 1;
        const int lo_all = C::kMQ ? max(d.tok_begin, window_lo_at(p, d.len - 1)) : d.tok_begin;
        const int origin = d.tok_end - 1;  // ALiBi positions are taken relative to this token

        float m[NTW][2], l[NTW][2], mx[NTW][2];  // reference max, sum, this lane's running max
        float acc[KT][NTW][4];
#pragma unroll
        for (int nt = 0; nt < NTW; ++nt) {
            m[nt][0] = m[nt][1] = mx[nt][0] = mx[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int mt = 0; mt < KT; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[mt][nt][e] = 0.f;
        }

        const int npages = tile_pages(d.tok_begin, d.tok_end);
        const int page0 = d.tok_begin / kBS * kBS;  // first token of the tile's first page
        // stage and phase of page j: advanced per page with one n-tile per warp,
        // computed per page with two (whose registers are all taken)
        uint32_t st = (gbase + (uint32_t)pfirst) % STAGES, ph = ((gbase + (uint32_t)pfirst) / STAGES) & 1;
        for (int j = pfirst; j < npages; j += PSTRIDE, advance_stage<STAGES, PSTRIDE>(st, ph)) {
            if constexpr (NTW > 1) {
                st = (gbase + (uint32_t)j) % STAGES;
                ph = ((gbase + (uint32_t)j) / STAGES) & 1;
            }
            if (!warp_wait(sm.full + st * 8, ph, sm.abort, sm.wait_ns)) {
                report(p, PA_DEVERR_TIMEOUT);
                *sm.abort = 1;
                return;
            }
            const uint32_t kp = sm.ring + st * C::kStageBytes;
            const uint32_t vp = kp + C::kPageBytes;
            const int tok0 = page0 + j * kBS;
            const bool edge = tok0 < lo_all || tok0 + kBS - 1 > hi_all;  // some key masked
            zero_unseen<C, LAYOUT, HEAD>(vp, tok0, d, lane);

            // S^T[token][head] = K . Q^T
            // two accumulator chains (even / odd k-steps) for MMA latency hiding
            float s[NTW][4], s2[NTW][4];
#pragma unroll
            for (int nt = 0; nt < NTW; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[nt][e] = s2[nt][e] = 0.f;
#pragma unroll
            for (int kk = 0; kk < KQ; ++kk) {
                uint32_t a0, a1, a2, a3;
                ldsm_x4(kp + khalf + k_frag_off<LAYOUT>(lane, kk), a0, a1, a2, a3);
#pragma unroll
                for (int nt = 0; nt < NTW; ++nt) {
                    if (kk & 1)
                        mma_16816<BF>(s2[nt], a0, a1, a2, a3, qb[nt][kk][0], qb[nt][kk][1]);
                    else
                        mma_16816<BF>(s[nt], a0, a1, a2, a3, qb[nt][kk][0], qb[nt][kk][1]);
                }
            }
#pragma unroll
            for (int nt = 0; nt < NTW; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[nt][e] += s2[nt][e];

            // One n-tile: the page's V fragments go to registers here and the
            // stage back to the producer, before the softmax and P.V, so the
            // stage is refilled while they run (two n-tiles have no registers
            // to spare and load V in the P.V loop).
            constexpr bool kEarlyV = NTW == 1;
            uint32_t vf[kEarlyV ? KT : 1][4];
            if constexpr (kEarlyV) {
#pragma unroll
                for (int mt = 0; mt < KT; ++mt) {
                    if constexpr (LAYOUT == kSplit)
                        ldsm_x4(vp + v_frag_off<LAYOUT>(lane, mt), vf[mt][0], vf[mt][1], vf[mt][2], vf[mt][3]);
                    else
                        ldsm_x4_trans(vp + v_frag_off<LAYOUT>(lane, mt), vf[mt][0], vf[mt][1], vf[mt][2],
                                      vf[mt][3]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive_after(sm.empty + st * 8, vf[KT - 1][3], p.zero);
            }

            // logits, online softmax, P as B fragments of P.V
            const int tlo = tok0 + r;  // this thread's tokens: tlo (e=0,1), tlo+8 (e=2,3)
            uint32_t pb[NTW][2], pbl[NTW][2];
            float z[NTW][4];
#pragma unroll
            for (int nt = 0; nt < NTW; ++nt) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float v = s[nt][e] * p.scale;
                    if (has_cap) v = soft_cap<C::kDiff>(p, v);
                    if (has_alibi) v += sl[nt][e & 1] * (float)(tlo + ((e >> 1) << 3) - origin);
                    z[nt][e] = v;
                }
                if (edge) {
                    const int t0 = tok0 + r, t1 = t0 + 8;
                    if (t0 < klo[nt][0] || t0 > khi[nt][0]) z[nt][0] = -INFINITY;
                    if (t0 < klo[nt][1] || t0 > khi[nt][1]) z[nt][1] = -INFINITY;
                    if (t1 < klo[nt][0] || t1 > khi[nt][0]) z[nt][2] = -INFINITY;
                    if (t1 < klo[nt][1] || t1 > khi[nt][1]) z[nt][3] = -INFINITY;
                }
            }
            softmax_page<NTW, KT, C::kMQ>(z, m, mx, l, acc, edge);
#pragma unroll
            for (int nt = 0; nt < NTW; ++nt) {
                const float p0 = z[nt][0], p1 = z[nt][1], p2 = z[nt][2], p3 = z[nt][3];
                const uint32_t x0 = pack2<BF>(p0, p1);  // token r,   heads 2cq, 2cq+1
                const uint32_t x1 = pack2<BF>(p2, p3);  // token r+8
                pb[nt][0] = movmatrix_trans(x0);         // -> B[k = token 2cq..][n = head r]
                pb[nt][1] = movmatrix_trans(x1);
                if constexpr (kTwoP) {
                    // the rounding residue of P as a second term
                    const float2 h0 = unpack2<BF>(x0), h1 = unpack2<BF>(x1);
                    pbl[nt][0] = movmatrix_trans(pack2<BF>(p0 - h0.x, p1 - h0.y));
                    pbl[nt][1] = movmatrix_trans(pack2<BF>(p2 - h1.x, p3 - h1.y));
                }
            }

            // acc^T[head dim][head] += V^T . P^T
            uint32_t vlast = 0;  // the page's last read
#pragma unroll
            for (int mt = 0; mt < KT; ++mt) {
                uint32_t a0, a1, a2, a3;
                if constexpr (kEarlyV) {
                    a0 = vf[mt][0];
                    a1 = vf[mt][1];
                    a2 = vf[mt][2];
                    a3 = vf[mt][3];
                } else if constexpr (LAYOUT == kSplit) {
                    ldsm_x4(vp + v_frag_off<LAYOUT>(lane, mt), a0, a1, a2, a3);
                } else {
                    ldsm_x4_trans(vp + v_frag_off<LAYOUT>(lane, mt), a0, a1, a2, a3);
                }
                vlast = a3;
#pragma unroll
                for (int nt = 0; nt < NTW; ++nt) {
                    mma_16816<BF>(acc[mt][nt], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
                    if constexpr (kTwoP) mma_16816<BF>(acc[mt][nt], a0, a1, a2, a3, pbl[nt][0], pbl[nt][1]);
                }
            }
            if constexpr (!kEarlyV) {
                __syncwarp();
                if (lane == 0) mbar_arrive_after(sm.empty + st * 8, vlast, p.zero);
            }
        }

        // this warp's partial state -> shared memory
        settle_max<NTW, KT>(m, mx, l, acc);
#pragma unroll
        for (int nt = 0; nt < NTW; ++nt) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                l[nt][0] += __shfl_xor_sync(0xffffffffu, l[nt][0], o);
                l[nt][1] += __shfl_xor_sync(0xffffffffu, l[nt][1], o);
            }
        }
        float* mw = sm.merge + warp * C::kMergeRows * C::kMergeStride;
#pragma unroll
        for (int nt = 0; nt < NTW; ++nt) {
            const int h0 = nt * 8 + 2 * cq;
#pragma unroll
            for (int mt = 0; mt < KT; ++mt) {
                const int d0 = mt * 16 + r;
                mw[h0 * C::kMergeStride + d0] = acc[mt][nt][0];
                mw[(h0 + 1) * C::kMergeStride + d0] = acc[mt][nt][1];
                mw[h0 * C::kMergeStride + d0 + 8] = acc[mt][nt][2];
                mw[(h0 + 1) * C::kMergeStride + d0 + 8] = acc[mt][nt][3];
            }
            if (r == 0) {
                sm.ml[warp * C::kMergeRows + h0] = make_float2(m[nt][0], l[nt][0]);
                sm.ml[warp * C::kMergeRows + h0 + 1] = make_float2(m[nt][1], l[nt][1]);
            }
        }
        if (!consumer_sync(sm, mphase, lane)) {  // all partial states written
            report(p, PA_DEVERR_TIMEOUT);
            *sm.abort = 1;
            return;
        }
        if (!tile_finish<C, T, HEAD, NC>(p, d, sm, warp, lane, mphase)) {  // merge buffers free again
            report(p, PA_DEVERR_TIMEOUT);
            *sm.abort = 1;
            return;
        }
        gbase += (uint32_t)npages;
    }
}

// Four fp8 cache elements (one 32-bit word, lowest address in the low byte) as
// two f16x2 pairs: lo = elements 0, 1 and hi = elements 2, 3 (exact).
template <int KV>
__device__ __forceinline__ void fp8x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (KV == kKvE4M3)
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    else
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "cvt.rn.f16x2.e5m2x2 %0, l;\n\tcvt.rn.f16x2.e5m2x2 %1, h;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
}

// Byte offset of 16-byte chunk c of token row t in an fp8 NHD page as the
// tensor copy leaves it: rows of HEAD bytes, chunks swizzled (128-byte swizzle:
// chunk ^ (t mod 8); 64-byte swizzle: chunk ^ ((t / 2) mod 4)), so the eight
// rows a warp reads at once fall in distinct banks.
// Value rows of 256 bytes are two such blocks of 128-byte rows, one after the other.
template <int HEAD>
__device__ __forceinline__ uint32_t nhd8_off(int t, int c) {
    if constexpr (HEAD > 128) return (uint32_t)((c >> 3) * 2048) + nhd8_off<128>(t, c & 7);
    const int sw = HEAD == 128 ? (t & 7) : ((t >> 1) & 3);
    return (uint32_t)(t * HEAD + ((c ^ sw) << 4));
}

// ldmatrix.x4 row address of this lane in an fp8 key page for k-steps kk and
// kk + 1.  Matrix j = lane / 8 holds the 16-byte rows of the eight tokens of
// S^T rows 0-7 (j even) or 8-15 (j odd) in k-step kk + j / 2, so register j of
// lane (r, cq) is the word (token of row r or r + 8, head dims 16k + 4cq..+3).
// A differential page (DIFF) is two pages of HEAD / 2, map by map.
template <int LAYOUT, int HEAD, bool DIFF>
__device__ __forceinline__ uint32_t k8_frag_off(int lane, int kk) {
    const int j = lane >> 3, i = lane & 7;
    const int c = kk + (j >> 1);
    if constexpr (LAYOUT == kNHD && DIFF) {
        constexpr int CM = HEAD / 32;  // chunks of one map's row
        return (uint32_t)(c / CM * (kBS * HEAD / 2)) + nhd8_off<HEAD / 2>(i + ((j & 1) << 3), c % CM);
    } else if constexpr (LAYOUT == kNHD) {
        return nhd8_off<HEAD>(i + ((j & 1) << 3), c);  // natural token order
    } else {
        const int tok = ((i >> 1) << 2) + (i & 1) + ((j & 1) << 1);  // tau(i), tau(i) + 2
        return (uint32_t)((c * kBS + tok) * 16);
    }
}

// ldmatrix.x4 row address of this lane in an fp8 value page for m-tiles mt and
// mt + 1: split [d][16 tokens] rows are head dims 16(mt + j/2) + i (+ 8 for odd
// j); NHD rows are tokens i (+ 8 for odd j), chunk mt + j/2.
template <int LAYOUT, int HEAD>
__device__ __forceinline__ uint32_t v8_frag_off(int lane, int mt) {
    const int j = lane >> 3, i = lane & 7;
    const int m = mt + (j >> 1);
    if constexpr (LAYOUT == kNHD) {
        return nhd8_off<HEAD>(i + ((j & 1) << 3), m);
    } else {
        return (uint32_t)((m * 16 + i + ((j & 1) << 3)) * kBS);
    }
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

// Consumer for fp8 caches (split layout).  The tensor-core inputs are fp16 for
// both query types: fp8 -> fp16 is exact; a bf16 query is converted once per
// tile (values beyond the fp16 range are clamped and PA_DEVERR_QUERY_RANGE is
// set); P is packed to fp16 (11 significant bits; two terms in a differential call).
// Every lane fetches four fp8 values with one 32-bit shared load.  For that
// the reduction index of each MMA is permuted identically on both operands:
//   Q.K^T  k-index 2cq+j <-> head dim 4cq+j, 2cq+8+j <-> 4cq+2+j  (per 16-dim step)
//   P.V    k-index 2cq+j <-> token    4cq+j, 2cq+8+j <-> 4cq+2+j  (per page)
// so row rr of S^T (the M index of Q.K^T) holds token tau(rr) of the page:
//   tau(r) = 4*(r/2) + (r&1) and tau(r+8) = tau(r) + 2 for r < 8.
template <class C, typename T, int HEAD, int NT, int LAYOUT, int STAGES, int NC, int KV>
__device__ void consumer_mma_fp8(const Params& p, const Smem& sm, int warp, int lane) {
    constexpr bool QBF = C::kBF16;
    // differential: P in two fp16 terms, whatever the output (see consumer_mma).  With
    // one, maps that nearly cancel pass a bf16 output's own rounding (1.65e-3 of the
    // norm): lambda 0.95 5.4e-3, lambda 1 1.4e-2; with two 1.66e-3.  The second term
    // costs 32 x 4096 e4m3 with four tokens 57.3 -> 62.9 us, 4 x 100000 e4m3, groups of
    // seven, 76.4 -> 83.5, and up to four rows nothing (28.5).
    constexpr bool kTwoP = C::kDiff;
    constexpr int KT = HEAD / 16;
    // differential, two n-tiles: warps in pairs, one map each (see consumer_mma)
    constexpr bool kPairs = C::kPairs;
    constexpr int NTW = kPairs ? 1 : NT;
    constexpr int PSTRIDE = kPairs ? NC / 2 : NC;
    constexpr int KQ = kPairs ? KT / 2 : KT;
    const int nt0 = kPairs ? warp / PSTRIDE : 0;
    const int pfirst = kPairs ? warp % PSTRIDE : warp;
    const uint32_t khalf = kPairs ? (uint32_t)nt0 * (C::kPageBytes / 2) : 0u;
    const int G = p.group;
    const int r = lane >> 2, cq = lane & 3;
    // page token of S^T rows r and r + 8: permuted for the split layout (see
    // above), natural for NHD, where the transposition of V is done by movmatrix
    const int tau = ((r >> 1) << 2) + (r & 1);
    const int tlo = LAYOUT == kNHD ? r : tau;
    const int thi = LAYOUT == kNHD ? r + 8 : tau + 2;
    const bool has_alibi = p.alibi != nullptr;
    const bool has_cap = p.softcap > 0.f;
    uint32_t gbase = 0;
    uint32_t mphase = 0;
    for (int k = 0;; ++k) {
        const int slot = k % C::kTD;
        if (!warp_wait(sm.td_full + slot * 8, (k / C::kTD) & 1, sm.abort, sm.wait_ns)) {
            report(p, PA_DEVERR_TIMEOUT);
            *sm.abort = 1;
            return;
        }
        const TileDesc d = sm.desc[slot];
        if (d.flags & kTileStop) return;
        const int qn = C::kMQ ? d.qn : 1;
        const int GE = qn * G;  // rows of N: query token v / G, head kvh * G + v % G

        // Q as fp16 B fragments in the permuted head-dim order.
        uint32_t qb[NTW][KQ][2];
        bool q_clamped = false;
        const uint32_t qs = sm.q + slot * C::kQBytes;
#pragma unroll
        for (int nt = 0; nt < NTW; ++nt) {
            const int v = (nt0 + nt) * 8 + r, h = C::row_of(v);
#pragma unroll
            for (int kk = 0; kk < KQ; ++kk) {
                uint32_t w0 = 0, w1 = 0;
                if (h < GE && (!C::kDiff || kPairs || kk / (KT / 2) == v / C::kRows)) {
                    const int k0 = kPairs ? nt0 * (HEAD / 2) + kk * 16 : kk * 16;
                    const uint32_t a = qs + (uint32_t)((h * HEAD + k0 + 4 * cq) * 2);
                    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w0), "=r"(w1) : "r"(a));
                    if constexpr (QBF) {
                        float2 f0 = unpack2<true>(w0), f1 = unpack2<true>(w1);
                        const float lim = 65504.f;
                        q_clamped |= fabsf(f0.x) > lim || fabsf(f0.y) > lim || fabsf(f1.x) > lim ||
                                     fabsf(f1.y) > lim;
                        w0 = pack2<false>(fminf(fmaxf(f0.x, -lim), lim), fminf(fmaxf(f0.y, -lim), lim));
                        w1 = pack2<false>(fminf(fmaxf(f1.x, -lim), lim), fminf(fmaxf(f1.y, -lim), lim));
                    }
                }
                qb[nt][kk][0] = w0;  // head dims 16kk + 4cq, +1  (k-index 2cq, 2cq+1)
                qb[nt][kk][1] = w1;  // head dims 16kk + 4cq+2, +3 (k-index 2cq+8, 2cq+9)
            }
        }
        if (q_clamped) report(p, PA_DEVERR_QUERY_RANGE);
        const uint32_t qlast = last_query_word<C, KQ>(qb[NTW - 1]);
        __syncwarp();
        if (lane == 0) mbar_arrive_after(sm.td_empty + slot * 8, qlast, p.zero);

        float sl[NTW][2];
#pragma unroll
        for (int nt = 0; nt < NTW; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int h = C::row_of((nt0 + nt) * 8 + 2 * cq + e);
                sl[nt][e] = (has_alibi && h < GE) ? p.alibi[d.kvh * G + h % G] : 0.f;
            }
        // key range of each of this lane's rows: its query token's position and
        // window, within the tile (padded rows get the tile's range)
        int klo[NTW][2], khi[NTW][2];
#pragma unroll
        for (int nt = 0; nt < NTW; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int v = C::row_of((nt0 + nt) * 8 + 2 * cq + e);
                int lo = d.tok_begin, hi = d.tok_end - 1;
                if (C::kMQ && v < GE) {
                    const int pos = d.len - qn + v / G;
                    hi = min(hi, pos);
                    lo = max(lo, window_lo_at(p, pos));
                }
                klo[nt][e] = lo;
                khi[nt][e] = hi;
            }
        // keys inside every row's range: a page within [lo_all, hi_all] needs no mask
        // (one query token: the tile's own range)
        const int hi_all = C::kMQ ? min(d.tok_end - 1, d.len - qn) : d.tok_end - 1;
        const int lo_all = C::kMQ ? max(d.tok_begin, window_lo_at(p, d.len - 1)) : d.tok_begin;
        const int origin = d.tok_end - 1;

        float m[NTW][2], l[NTW][2], mx[NTW][2];  // reference max, sum, this lane's running max
        float acc[KT][NTW][4];
#pragma unroll
        for (int nt = 0; nt < NTW; ++nt) {
            m[nt][0] = m[nt][1] = mx[nt][0] = mx[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int mt = 0; mt < KT; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[mt][nt][e] = 0.f;
        }

        const int npages = tile_pages(d.tok_begin, d.tok_end);
        const int page0 = d.tok_begin / kBS * kBS;
        // stage and phase of page j: advanced per page with one n-tile, computed
        // per page with two (whose registers are all taken)
        uint32_t st = (gbase + (uint32_t)pfirst) % STAGES, ph = ((gbase + (uint32_t)pfirst) / STAGES) & 1;
        for (int j = pfirst; j < npages; j += PSTRIDE, advance_stage<STAGES, PSTRIDE>(st, ph)) {
            if constexpr (NTW > 1) {
                st = (gbase + (uint32_t)j) % STAGES;
                ph = ((gbase + (uint32_t)j) / STAGES) & 1;
            }
            if (!warp_wait(sm.full + st * 8, ph, sm.abort, sm.wait_ns)) {
                report(p, PA_DEVERR_TIMEOUT);
                *sm.abort = 1;
                return;
            }
            const uint32_t kp = sm.ring + st * C::kStageBytes;
            const uint32_t vp = kp + C::kPageBytes;
            const int tok0 = page0 + j * kBS;
            const bool edge = tok0 < lo_all || tok0 + kBS - 1 > hi_all;  // some key masked
            zero_unseen<C, LAYOUT, HEAD>(vp, tok0, d, lane);

            // S^T[row][head]: key page [d/16][token][16 bytes] (split) or [token][d]
            // with swizzled 16-byte chunks (NHD)
            float s[NTW][4], s2[NTW][4];
#pragma unroll
            for (int nt = 0; nt < NTW; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[nt][e] = s2[nt][e] = 0.f;
            // one ldmatrix.x4 fetches the four 32-bit words (tokens tlo / thi,
            // k-steps kk / kk + 1) that four separate loads would
#pragma unroll
            for (int kk = 0; kk < KQ; kk += 2) {
                uint32_t w[4];
                ldsm_x4(kp + khalf + k8_frag_off<LAYOUT, HEAD, C::kDiff>(lane, kk), w[0], w[1], w[2], w[3]);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint32_t a0, a1, a2, a3;
                    fp8x4_to_f16<KV>(w[2 * u], a0, a2);
                    fp8x4_to_f16<KV>(w[2 * u + 1], a1, a3);
#pragma unroll
                    for (int nt = 0; nt < NTW; ++nt) {
                        // (differential, two n-tiles: each meets its own map's keys only)
                        if (C::kDiff && NTW == 2 && (kk + u) / (KT / 2) != nt) continue;
                        if (u)
                            mma_16816<false>(s2[nt], a0, a1, a2, a3, qb[nt][kk + u][0], qb[nt][kk + u][1]);
                        else
                            mma_16816<false>(s[nt], a0, a1, a2, a3, qb[nt][kk + u][0], qb[nt][kk + u][1]);
                    }
                }
            }

            // One n-tile: the page's V words go to registers here and the stage
            // back to the producer, before the softmax, the conversion and P.V.
            constexpr bool kEarlyV = NTW == 1;
            uint32_t vw[kEarlyV ? KT / 2 : 1][4];
            if constexpr (kEarlyV) {
#pragma unroll
                for (int mt = 0; mt < KT; mt += 2)
                    ldsm_x4(vp + v8_frag_off<LAYOUT, HEAD>(lane, mt), vw[mt / 2][0], vw[mt / 2][1],
                            vw[mt / 2][2], vw[mt / 2][3]);
                __syncwarp();
                if (lane == 0) mbar_arrive_after(sm.empty + st * 8, vw[KT / 2 - 1][3], p.zero);
            }

            uint32_t pb[NTW][2], pbl[NTW][2];
            float z[NTW][4];
#pragma unroll
            for (int nt = 0; nt < NTW; ++nt) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float v = (s[nt][e] + s2[nt][e]) * p.scale;
                    if (has_cap) v = soft_cap<C::kDiff>(p, v);
                    if (has_alibi) v += sl[nt][e & 1] * (float)(tok0 + ((e >> 1) ? thi : tlo) - origin);
                    z[nt][e] = v;
                }
                if (edge) {
                    const int t0 = tok0 + tlo, t1 = tok0 + thi;
                    if (t0 < klo[nt][0] || t0 > khi[nt][0]) z[nt][0] = -INFINITY;
                    if (t0 < klo[nt][1] || t0 > khi[nt][1]) z[nt][1] = -INFINITY;
                    if (t1 < klo[nt][0] || t1 > khi[nt][0]) z[nt][2] = -INFINITY;
                    if (t1 < klo[nt][1] || t1 > khi[nt][1]) z[nt][3] = -INFINITY;
                }
            }
            softmax_page<NTW, KT, C::kMQ>(z, m, mx, l, acc, edge);
#pragma unroll
            for (int nt = 0; nt < NTW; ++nt) {
                const uint32_t x0 = pack2<false>(z[nt][0], z[nt][1]), x1 = pack2<false>(z[nt][2], z[nt][3]);
                pb[nt][0] = movmatrix_trans(x0);  // k-index 2cq.. = tokens tlo
                pb[nt][1] = movmatrix_trans(x1);
                if constexpr (kTwoP) {
                    const float2 h0 = unpack2<false>(x0), h1 = unpack2<false>(x1);
                    pbl[nt][0] = movmatrix_trans(pack2<false>(z[nt][0] - h0.x, z[nt][1] - h0.y));
                    pbl[nt][1] = movmatrix_trans(pack2<false>(z[nt][2] - h1.x, z[nt][3] - h1.y));
                }
            }

            // acc^T[head dim][head] += V^T . P^T.  Split value page [d][16
            // tokens]: one 32-bit load is four permuted tokens of a head dim.  NHD
            // page [token][d]: one load is four head dims of a token; movmatrix
            // turns each 8 x 8 block (tokens x head dims 16mt + 4cq + {0,1} or
            // {2,3}) into the A fragment, whose rows are then head dims 16mt +
            // tau(r) (rows r) and 16mt + tau(r) + 2 (rows r + 8).
            uint32_t vlast = 0;  // the page's last read
#pragma unroll
            for (int mt = 0; mt < KT; mt += 2) {
                // words of rows r and r + 8 (head dims, or tokens for NHD) of
                // m-tiles mt and mt + 1 in one ldmatrix.x4
                uint32_t w[4];
                if constexpr (kEarlyV) {
                    w[0] = vw[mt / 2][0];
                    w[1] = vw[mt / 2][1];
                    w[2] = vw[mt / 2][2];
                    w[3] = vw[mt / 2][3];
                } else {
                    ldsm_x4(vp + v8_frag_off<LAYOUT, HEAD>(lane, mt), w[0], w[1], w[2], w[3]);
                }
                vlast = w[3];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint32_t a0, a1, a2, a3;
                    if constexpr (LAYOUT == kNHD) {
                        uint32_t lo0, hi0, lo1, hi1;
                        fp8x4_to_f16<KV>(w[2 * u], lo0, hi0);
                        fp8x4_to_f16<KV>(w[2 * u + 1], lo1, hi1);
                        a0 = movmatrix_trans(lo0);
                        a1 = movmatrix_trans(hi0);
                        a2 = movmatrix_trans(lo1);
                        a3 = movmatrix_trans(hi1);
                    } else {
                        fp8x4_to_f16<KV>(w[2 * u], a0, a2);
                        fp8x4_to_f16<KV>(w[2 * u + 1], a1, a3);
                    }
#pragma unroll
                    for (int nt = 0; nt < NTW; ++nt) {
                        mma_16816<false>(acc[mt + u][nt], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
                        if constexpr (kTwoP) mma_16816<false>(acc[mt + u][nt], a0, a1, a2, a3, pbl[nt][0], pbl[nt][1]);
                    }
                }
            }
            if constexpr (!kEarlyV) {
                __syncwarp();
                if (lane == 0) mbar_arrive_after(sm.empty + st * 8, vlast, p.zero);
            }
        }

        settle_max<NTW, KT>(m, mx, l, acc);
#pragma unroll
        for (int nt = 0; nt < NTW; ++nt) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                l[nt][0] += __shfl_xor_sync(0xffffffffu, l[nt][0], o);
                l[nt][1] += __shfl_xor_sync(0xffffffffu, l[nt][1], o);
            }
        }
        float* mw = sm.merge + warp * C::kMergeRows * C::kMergeStride;
#pragma unroll
        for (int nt = 0; nt < NTW; ++nt) {
            const int h0 = nt * 8 + 2 * cq;
#pragma unroll
            for (int mt = 0; mt < KT; ++mt) {
                // head dims of accumulator rows r and r + 8 (see the P.V step)
                const int d0 = mt * 16 + (LAYOUT == kNHD ? tau : r);
                const int d1 = d0 + (LAYOUT == kNHD ? 2 : 8);
                mw[h0 * C::kMergeStride + d0] = acc[mt][nt][0];
                mw[(h0 + 1) * C::kMergeStride + d0] = acc[mt][nt][1];
                mw[h0 * C::kMergeStride + d1] = acc[mt][nt][2];
                mw[(h0 + 1) * C::kMergeStride + d1] = acc[mt][nt][3];
            }
            if (r == 0) {
                sm.ml[warp * C::kMergeRows + h0] = make_float2(m[nt][0], l[nt][0]);
                sm.ml[warp * C::kMergeRows + h0 + 1] = make_float2(m[nt][1], l[nt][1]);
            }
        }
        if (!consumer_sync(sm, mphase, lane)) {
            report(p, PA_DEVERR_TIMEOUT);
            *sm.abort = 1;
            return;
        }
        if (!tile_finish<C, T, HEAD, NC>(p, d, sm, warp, lane, mphase)) {
            report(p, PA_DEVERR_TIMEOUT);
            *sm.abort = 1;
            return;
        }
        gbase += (uint32_t)npages;
    }
}

// fp32 inputs: tensor cores with each fp32 operand carried as two tf32 terms
// (hi + lo) and three MMAs per product (hi.hi + hi.lo + lo.hi), which keeps
// each product to ~2^-20 relative, well inside the fp32 result's error budget.
// Tokens on M, query rows on N for Q.K^T (NT n-tiles of 8 rows); head dims on
// M, rows on N for P.V, as in the 16-bit consumer.  P moves from the S^T
// fragment to the B fragment with shuffles (there is no 32-bit movmatrix).
// One n-tile keeps Q split in registers for the whole tile; two keep the raw
// fp32 words (64 registers at head size 128 instead of 128) and split them at
// each use.
//
// Shared-memory reads.  Split pages: K [d/4][16 tokens][4] gives each k-step's
// A fragment as one ldmatrix.x4; V [d][16 tokens] likewise (its 64-byte rows
// cost 4-way bank conflicts whatever the order).  NHD pages (HEAD / 32 blocks
// of 16 token rows x 128 bytes, 16-byte chunks swizzled by token % 8): K by
// ldmatrix.x4 as well; V^T needs a transpose that ldmatrix does not do for
// 32-bit elements, so its fragments are single-word loads, with the k-step's
// tokens taken in the order 0, 2, 4, 6 | 1, 3, 5, 7 (k-index t -> token 2t, t + 4
// -> 2t + 1), which puts the 32 words of each load in 32 distinct banks; the
// P^T fragment follows the same order.
template <class C, int HEAD, int NT, int LAYOUT, int STAGES, int NC>
__device__ void consumer_tf32(const Params& p, const Smem& sm, int warp, int lane) {
    constexpr int KT = HEAD / 8;   // k-steps of Q.K^T (8 head dims each)
    constexpr int MT = HEAD / 16;  // m-tiles of P.V (16 head dims each)
    static_assert(!C::kDiff && !C::kPairs, "differential heads: consumer_fma");
    constexpr bool QSPLIT = NT == 1;  // Q held split for the whole tile
    const int G = p.group;
    const int r = lane >> 2, cq = lane & 3;
    const bool has_alibi = p.alibi != nullptr;
    const bool has_cap = p.softcap > 0.f;
    uint32_t gbase = 0;
    uint32_t mphase = 0;
    for (int k = 0;; ++k) {
        const int slot = k % C::kTD;
        if (!warp_wait(sm.td_full + slot * 8, (k / C::kTD) & 1, sm.abort, sm.wait_ns)) {
            report(p, PA_DEVERR_TIMEOUT);
            *sm.abort = 1;
            return;
        }
        const TileDesc d = sm.desc[slot];
        if (d.flags & kTileStop) return;
        const int qn = C::kMQ ? d.qn : 1;
        const int GE = qn * G;  // rows of N: query token v / G, head kvh * G + v % G

        // Q as B fragments (k = head dim 8kk + cq / + 4, n = row nt * 8 + r):
        // hi and lo terms (one n-tile) or the raw words (two)
        uint32_t qa[NT][KT][2];
        uint32_t qlo[QSPLIT ? KT : 1][2];
        {
            const float* q = reinterpret_cast<const float*>(
                __cvta_shared_to_generic(sm.q + slot * C::kQBytes));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int kk = 0; kk < KT; ++kk)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int v = nt * 8 + r;
                        const uint32_t x = v < GE ? __float_as_uint(q[v * HEAD + kk * 8 + cq + 4 * e]) : 0u;
                        if constexpr (QSPLIT)
                            split_tf32(x, qa[nt][kk][e], qlo[kk][e]);
                        else
                            qa[nt][kk][e] = x;
                    }
        }
        const uint32_t qlast = last_query_word<C, KT>(qa[NT - 1]);
        __syncwarp();
        // Q and descriptor are in registers (lane 0 takes part in the last read)
        if (lane == 0) mbar_arrive_after(sm.td_empty + slot * 8, qlast, p.zero);

        float sl[NT][2];
        int klo[NT][2], khi[NT][2];  // key range of this lane's rows within the tile
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int v = nt * 8 + 2 * cq + e;
                sl[nt][e] = (has_alibi && v < GE) ? p.alibi[d.kvh * G + v % G] : 0.f;
                int lo = d.tok_begin, hi = d.tok_end - 1;
                if (C::kMQ && v < GE) {
                    const int pos = d.len - qn + v / G;
                    hi = min(hi, pos);
                    lo = max(lo, window_lo_at(p, pos));
                }
                klo[nt][e] = lo;
                khi[nt][e] = hi;
            }
        const int hi_all = C::kMQ ? min(d.tok_end - 1, d.len - qn) : d.tok_end - 1;
        const int lo_all = C::kMQ ? max(d.tok_begin, window_lo_at(p, d.len - 1)) : d.tok_begin;
        const int origin = d.tok_end - 1;

        float m[NT][2], l[NT][2], mx[NT][2];  // reference max, sum, this lane's running max
        float acc[MT][NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = mx[nt][0] = mx[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[mt][nt][e] = 0.f;
        }

        const int npages = tile_pages(d.tok_begin, d.tok_end);
        const int page0 = d.tok_begin / kBS * kBS;
        // ldmatrix row of this lane: matrix j = lane / 8, row i = lane % 8
        const int lj = lane >> 3, li = lane & 7;
        // P^T k-index cq holds token cq (split) or 2cq (NHD), cq + 4 token cq + 4 or 2cq + 1
        const int tk0 = LAYOUT == kSplit ? cq : 2 * cq, tk1 = LAYOUT == kSplit ? cq + 4 : 2 * cq + 1;
        const int src0 = 4 * tk0 + (r >> 1), src1 = 4 * tk1 + (r >> 1);
        // stage and phase of page j: advanced per page with one n-tile, computed
        // per page with two (whose registers are all taken)
        uint32_t st = (gbase + (uint32_t)warp) % STAGES, ph = ((gbase + (uint32_t)warp) / STAGES) & 1;
        for (int j = warp; j < npages; j += NC, advance_stage<STAGES, NC>(st, ph)) {
            if constexpr (NT > 1) {
                st = (gbase + (uint32_t)j) % STAGES;
                ph = ((gbase + (uint32_t)j) / STAGES) & 1;
            }
            if (!warp_wait(sm.full + st * 8, ph, sm.abort, sm.wait_ns)) {
                report(p, PA_DEVERR_TIMEOUT);
                *sm.abort = 1;
                return;
            }
            const uint32_t kp = sm.ring + st * C::kStageBytes;
            const uint32_t vp = kp + C::kPageBytes;
            const int tok0 = page0 + j * kBS;
            const bool edge = tok0 < lo_all || tok0 + kBS - 1 > hi_all;
            zero_unseen<C, LAYOUT, HEAD>(vp, tok0, d, lane);

            // S^T[token][row] = K . Q^T; the four 8 x 4 blocks (tokens 0-7 /
            // 8-15, head dims 8kk..+3 / +4..+7) of a k-step are its A fragment,
            // one ldmatrix.x4 (this lane's row: block lj, row li).  Each
            // k-step's three products go to a fresh accumulator that is then
            // added with a rounded fp32 add, so that the tensor core's own
            // accumulation (which need not round to nearest) never carries a
            // sum across the k-steps of a page or, for P.V below, the pages of
            // a tile: without it a 24-head, group-12 fp32 case missed the 1e-5
            // tolerance even with the rounded split.
            float s[NT][4], s2[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[nt][e] = s2[nt][e] = 0.f;
#pragma unroll
            for (int kk = 0; kk < KT; ++kk) {
                uint32_t a[4], ah[4], al[4];
                const int cg = 2 * kk + (lj >> 1);  // 16-byte chunk of the head dims
                const uint32_t ka =
                    LAYOUT == kSplit
                        ? kp + (uint32_t)((cg * kBS + li + ((lj & 1) << 3)) * 16)
                        : kp + (uint32_t)((cg >> 3) * 2048 + (li + ((lj & 1) << 3)) * 128 +
                                          (((cg & 7) ^ li) << 4));
                ldsm_x4(ka, a[0], a[1], a[2], a[3]);
#pragma unroll
                for (int e = 0; e < 4; ++e) split_tf32(a[e], ah[e], al[e]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    uint32_t bh[2], bl[2];
                    if constexpr (QSPLIT) {
                        bh[0] = qa[nt][kk][0];
                        bh[1] = qa[nt][kk][1];
                        bl[0] = qlo[kk][0];
                        bl[1] = qlo[kk][1];
                    } else {
                        split_tf32(qa[nt][kk][0], bh[0], bl[0]);
                        split_tf32(qa[nt][kk][1], bh[1], bl[1]);
                    }
                    float t[4] = {0.f, 0.f, 0.f, 0.f};
                    mma_1688_tf32(t, al[0], al[1], al[2], al[3], bh[0], bh[1]);
                    mma_1688_tf32(t, ah[0], ah[1], ah[2], ah[3], bl[0], bl[1]);
                    mma_1688_tf32(t, ah[0], ah[1], ah[2], ah[3], bh[0], bh[1]);
                    float (&sa)[4] = (kk & 1) ? s2[nt] : s[nt];
#pragma unroll
                    for (int e = 0; e < 4; ++e) sa[e] = __fadd_rn(sa[e], t[e]);
                }
            }

            // logits, online softmax, P^T as B fragments (hi and lo) per n-tile
            uint32_t pbh[NT][2][2], pbl[NT][2][2];
            float z[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float v = (s[nt][e] + s2[nt][e]) * p.scale;
                    if (has_cap) v = soft_cap<false>(p, v);
                    if (has_alibi) v += sl[nt][e & 1] * (float)(tok0 + r + ((e >> 1) << 3) - origin);
                    z[nt][e] = v;
                }
                if (edge) {
                    const int t0 = tok0 + r, t1 = t0 + 8;
                    if (t0 < klo[nt][0] || t0 > khi[nt][0]) z[nt][0] = -INFINITY;
                    if (t0 < klo[nt][1] || t0 > khi[nt][1]) z[nt][1] = -INFINITY;
                    if (t1 < klo[nt][0] || t1 > khi[nt][0]) z[nt][2] = -INFINITY;
                    if (t1 < klo[nt][1] || t1 > khi[nt][1]) z[nt][3] = -INFINITY;
                }
            }
            softmax_page<NT, MT, C::kMQ>(z, m, mx, l, acc, edge);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                // z[nt]: p of (token r, row 2cq), (token r, row 2cq + 1),
                // (token r + 8, row 2cq), (token r + 8, row 2cq + 1)
                const float* pv = z[nt];
                // B fragments of P^T for k-steps ks = 0, 1 (tokens 8ks..8ks+7):
                // b0 = P[row r][token 8ks + tk0], b1 = P[row r][token 8ks + tk1],
                // held by lanes (token % 8, row / 2), element by row parity and ks
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    const float e0 = __shfl_sync(0xffffffffu, pv[2 * ks], src0);
                    const float o0 = __shfl_sync(0xffffffffu, pv[2 * ks + 1], src0);
                    const float e1 = __shfl_sync(0xffffffffu, pv[2 * ks], src1);
                    const float o1 = __shfl_sync(0xffffffffu, pv[2 * ks + 1], src1);
                    split_tf32(__float_as_uint((r & 1) ? o0 : e0), pbh[nt][ks][0], pbl[nt][ks][0]);
                    split_tf32(__float_as_uint((r & 1) ? o1 : e1), pbh[nt][ks][1], pbl[nt][ks][1]);
                }
            }

            // acc^T[head dim][row] += V^T . P^T; A fragment of (m-tile mt,
            // k-step ks): head dims 16mt + r / + 8 by k-indices cq / cq + 4
            uint32_t vlast = 0;  // the page's last read
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    uint32_t a[4], ah[4], al[4];
                    if constexpr (LAYOUT == kSplit) {
                        // [d][16 tokens]: the four 8 x 4 blocks (head dims
                        // 16mt..+7 / +8..+15, tokens 8ks..+3 / +4..+7), one ldmatrix.x4
                        ldsm_x4(vp + (uint32_t)(((mt * 16 + li + ((lj & 1) << 3)) * kBS + 8 * ks +
                                                 4 * (lj >> 1)) * 4),
                                a[0], a[1], a[2], a[3]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int dim = mt * 16 + r + ((e & 1) << 3);
                            const int tok = 8 * ks + ((e >> 1) ? tk1 : tk0);
                            const uint32_t va = vp + (uint32_t)((dim >> 5) * 2048 + tok * 128 +
                                                                ((((dim >> 2) & 7) ^ (tok & 7)) << 4) +
                                                                (dim & 3) * 4);
                            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(a[e]) : "r"(va));
                        }
                    }
                    vlast = a[3];
#pragma unroll
                    for (int e = 0; e < 4; ++e) split_tf32(a[e], ah[e], al[e]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float t[4] = {0.f, 0.f, 0.f, 0.f};
                        mma_1688_tf32(t, al[0], al[1], al[2], al[3], pbh[nt][ks][0], pbh[nt][ks][1]);
                        mma_1688_tf32(t, ah[0], ah[1], ah[2], ah[3], pbl[nt][ks][0], pbl[nt][ks][1]);
                        mma_1688_tf32(t, ah[0], ah[1], ah[2], ah[3], pbh[nt][ks][0], pbh[nt][ks][1]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[mt][nt][e] = __fadd_rn(acc[mt][nt][e], t[e]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_after(sm.empty + st * 8, vlast, p.zero);
        }

        float* mw = sm.merge + warp * C::kMergeRows * C::kMergeStride;
        settle_max<NT, MT>(m, mx, l, acc);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                l[nt][0] += __shfl_xor_sync(0xffffffffu, l[nt][0], o);
                l[nt][1] += __shfl_xor_sync(0xffffffffu, l[nt][1], o);
            }
            const int h0 = nt * 8 + 2 * cq;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const int d0 = mt * 16 + r;
                mw[h0 * C::kMergeStride + d0] = acc[mt][nt][0];
                mw[(h0 + 1) * C::kMergeStride + d0] = acc[mt][nt][1];
                mw[h0 * C::kMergeStride + d0 + 8] = acc[mt][nt][2];
                mw[(h0 + 1) * C::kMergeStride + d0 + 8] = acc[mt][nt][3];
            }
            if (r == 0) {
                sm.ml[warp * C::kMergeRows + h0] = make_float2(m[nt][0], l[nt][0]);
                sm.ml[warp * C::kMergeRows + h0 + 1] = make_float2(m[nt][1], l[nt][1]);
            }
        }
        if (!consumer_sync(sm, mphase, lane)) {
            report(p, PA_DEVERR_TIMEOUT);
            *sm.abort = 1;
            return;
        }
        if (!tile_finish<C, float, HEAD, NC>(p, d, sm, warp, lane, mphase)) {
            report(p, PA_DEVERR_TIMEOUT);
            *sm.abort = 1;
            return;
        }
        gbase += (uint32_t)npages;
    }
}

// fp32 differential heads, on the fp32 units.  A tile has at most eight columns
// per warp, so a page is 16 x (HEAD / 2) x 8 + 16 x HEAD x 8 multiply-adds: 768
// instructions of a warp at value heads of 128.  (As three tf32 products each it
// is 96 m16n8k8 MMAs of some fifty cycles.  GPU time with those and so: 32 x 4096,
// groups of four, 87 and 81.4 us, of eight 116 and 119; heads of 256 247 and 162,
// of eight, 16 sequences, 135 and 131; two short sequences, call after call, 17.4 and
// 15.1 (14.4 in a graph).  And
// every product is rounded once.)  What bounds it is what shared memory returns
// to registers, 128 bytes a cycle: per page of a warp 128 + 192 cycles, so packed
// fp32 pairs, which need P or V twice, cost more than they save (86.7).  Column
// v = 4 hb + i of a lane's half hb is map hb of row i (one n-tile), or row v of
// the warp's map (a pair of warps).
//
// Q.K^T: lane (tg, dq, hb) sums four tokens by its half's four columns over a
// quarter dq of the map's head dims, one 16-byte chunk in four; its j-th token is
// tg + 4 (j ^ dq), so that eight successive lanes read eight distinct chunks of
// 128 bytes in both layouts, and two exchanges (dq bit 0, then bit 1) leave each
// lane the sum of token tg + 4 dq.  Q stays in shared memory for the whole tile.
//
// P.V: a lane owns HEAD / 32 head dims of all eight columns; P goes through the
// warp's part of the merge buffer, which is free until the end of the tile.  NHD
// pages: four successive dims per 16-byte read, token by token.  Split pages
// ([d][16 tokens], 64-byte rows): every 32nd dim, and a lane begins with token
// quad (lane / 2) % 4, so that eight lanes read 128 distinct bytes.  A page's sum
// is added to the tile's once.
template <class C, int HEAD, int LAYOUT, int STAGES, int NC>
__device__ void consumer_fma(const Params& p, const Smem& sm, int warp, int lane) {
    constexpr int IT = HEAD / 32;  // 16-byte key chunks of a lane
    constexpr int DV = HEAD / 32;  // head dims of a lane in P.V
    // Loops of value heads of 256 unrolled half as far: the whole page's work in one
    // piece misses the instruction cache (split, groups of four, 176 us; 167 so;
    // heads of 128 the other way round, 81.4 and 82.1)
    constexpr int kUC = HEAD > 128 ? 2 : 4, kUT = HEAD > 128 ? 8 : 16, kUN = HEAD > 128 ? 2 : 4;
    constexpr bool kPairs = C::kPairs;
    constexpr int PSTRIDE = kPairs ? NC / 2 : NC;
    const int pfirst = kPairs ? warp % PSTRIDE : warp;
    const int tg = lane & 3, dq = (lane >> 2) & 3, hb = lane >> 4;
    const int map = kPairs ? warp / PSTRIDE : hb, row0 = kPairs ? hb * 4 : 0;
    const int tt = tg + 4 * dq;  // this lane's token of a page, after the exchanges
    const int G = p.group;
    const bool has_alibi = p.alibi != nullptr;
    const bool has_cap = p.softcap > 0.f;
    // byte offsets in the key page of the lane's first chunk, token j
    uint32_t koff[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int t = tg + 4 * (j ^ dq), cg = map * (HEAD / 8) + dq;
        koff[j] = LAYOUT == kSplit ? (uint32_t)((cg * kBS + t) * 16)
                                   : (uint32_t)((cg >> 3) * 2048 + t * 128 + ((dq ^ (t & 7)) << 4));
    }
    float* mw = sm.merge + warp * C::kMergeRows * C::kMergeStride;
    const uint32_t ps = smem_u32(mw);  // P of the page at hand
    uint32_t gbase = 0;
    uint32_t mphase = 0;
    for (int k = 0;; ++k) {
        const int slot = k % C::kTD;
        if (!warp_wait(sm.td_full + slot * 8, (k / C::kTD) & 1, sm.abort, sm.wait_ns)) {
            report(p, PA_DEVERR_TIMEOUT);
            *sm.abort = 1;
            return;
        }
        const TileDesc d = sm.desc[slot];
        if (d.flags & kTileStop) return;
        const int qn = C::kMQ ? d.qn : 1;
        const int GE = qn * G;  // query rows: token v / G, head kvh * G + v % G
        const uint32_t qs = sm.q + slot * C::kQBytes + (uint32_t)((row0 * HEAD + map * (HEAD / 2) + dq * 4) * 4);

        float sl[4];
        int klo[4], khi[4];  // key range of this lane's columns within the tile
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int v = row0 + i;
            sl[i] = (has_alibi && v < GE) ? p.alibi[d.kvh * G + v % G] : 0.f;
            int lo = d.tok_begin, hi = d.tok_end - 1;
            if (C::kMQ && v < GE) {
                const int pos = d.len - qn + v / G;
                hi = min(hi, pos);
                lo = max(lo, window_lo_at(p, pos));
            }
            klo[i] = lo;
            khi[i] = hi;
        }
        const int hi_all = C::kMQ ? min(d.tok_end - 1, d.len - qn) : d.tok_end - 1;
        const int lo_all = C::kMQ ? max(d.tok_begin, window_lo_at(p, d.len - 1)) : d.tok_begin;
        const int origin = d.tok_end - 1;

        float m[4], l[4], mx[4];  // reference max, this lane's sum and running max
        float acc[DV][8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m[i] = mx[i] = -INFINITY;
            l[i] = 0.f;
        }
#pragma unroll
        for (int x = 0; x < DV; ++x)
#pragma unroll
            for (int v = 0; v < 8; ++v) acc[x][v] = 0.f;
        // moves the references to the warp's running max, with l and acc
        auto move_max = [&]() {
            float al[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float mn = mx[i];
#pragma unroll
                for (int o = 1; o < 16; o <<= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
                // equal: also a column without a key so far (-inf)
                al[i] = mn == m[i] ? 1.f : exp2f((m[i] - mn) * kLog2e);
                m[i] = mn;
                l[i] *= al[i];
            }
#pragma unroll
            for (int v = 0; v < 8; ++v) {
                const float a = __shfl_sync(0xffffffffu, al[v & 3], (v >> 2) << 4);
#pragma unroll
                for (int x = 0; x < DV; ++x) acc[x][v] *= a;
            }
        };

        const int npages = tile_pages(d.tok_begin, d.tok_end);
        const int page0 = d.tok_begin / kBS * kBS;
        uint32_t qlast = 0;  // the last word read of the query rows
        uint32_t st = (gbase + (uint32_t)pfirst) % STAGES, ph = ((gbase + (uint32_t)pfirst) / STAGES) & 1;
        for (int j = pfirst; j < npages; j += PSTRIDE, advance_stage<STAGES, PSTRIDE>(st, ph)) {
            if (!warp_wait(sm.full + st * 8, ph, sm.abort, sm.wait_ns)) {
                report(p, PA_DEVERR_TIMEOUT);
                *sm.abort = 1;
                return;
            }
            const uint32_t kp = sm.ring + st * C::kStageBytes;
            const uint32_t vp = kp + C::kPageBytes;
            const int tok0 = page0 + j * kBS;
            const bool edge = tok0 < lo_all || tok0 + kBS - 1 > hi_all;

            float s[4][4];  // [token j][column i]
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[t][i] = 0.f;
            uint32_t klast = 0;
#pragma unroll kUC
            for (int c = 0; c < IT; ++c) {
                float4 q[4], x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) q[i] = lds_v4(qs + (uint32_t)(i * HEAD * 4 + c * 64));
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    x[t] = lds_v4(kp + (LAYOUT == kSplit ? koff[t] + c * (4 * kBS * 16)
                                                         : (koff[t] ^ ((c & 1) << 6)) + (c >> 1) * 2048));
                qlast = __float_as_uint(q[3].w);
                klast = __float_as_uint(x[3].w);
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        s[t][i] = fmaf(q[i].x, x[t].x, s[t][i]);
                        s[t][i] = fmaf(q[i].y, x[t].y, s[t][i]);
                        s[t][i] = fmaf(q[i].z, x[t].z, s[t][i]);
                        s[t][i] = fmaf(q[i].w, x[t].w, s[t][i]);
                    }
            }
            __syncwarp();  // the key half goes back
            if (lane == 0) mbar_arrive_after(sm.empty + st * 8, klast, p.zero);

            // the quarters' sums: lane dq keeps the even j, whose tokens are the
            // odd j's of lane dq ^ 1; then j = 0 against lane dq ^ 2
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[0][i] += __shfl_xor_sync(0xffffffffu, s[1][i], 4);
                s[2][i] += __shfl_xor_sync(0xffffffffu, s[3][i], 4);
                s[0][i] += __shfl_xor_sync(0xffffffffu, s[2][i], 8);
            }

            // logits and online softmax (see softmax_page)
            float z[4];
            bool need = false;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float v = s[0][i] * p.scale;
                if (has_cap) v = soft_cap<false>(p, v);
                if (has_alibi) v += sl[i] * (float)(tok0 + tt - origin);
                if (row0 + i >= GE || (edge && (tok0 + tt < klo[i] || tok0 + tt > khi[i]))) v = -INFINITY;
                z[i] = v;
                mx[i] = fmaxf(mx[i], v);
                need |= v - m[i] > kLazyMax;
            }
            if (__any_sync(0xffffffffu, need)) move_max();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // a column without a key so far: 0 as reference, so that no -inf - -inf appears
                z[i] = exp2f((z[i] - (m[i] == -INFINITY ? 0.f : m[i])) * kLog2e);
                l[i] += z[i];
            }
            if constexpr (LAYOUT == kSplit) {  // [column][token], the halves 16 banks apart
#pragma unroll
                for (int i = 0; i < 4; ++i) sts_f32(ps + (uint32_t)((hb * 80 + i * 16 + tt) * 4), z[i]);
            } else {  // [token][column]
                sts_v4(ps + (uint32_t)((tt * 8 + hb * 4) * 4), make_float4(z[0], z[1], z[2], z[3]));
            }
            __syncwarp();

            if (!warp_wait(sm.full_v + st * 8, ph, sm.abort, sm.wait_ns)) {
                report(p, PA_DEVERR_TIMEOUT);
                *sm.abort = 1;
                return;
            }
            zero_unseen<C, LAYOUT, HEAD>(vp, tok0, d, lane);

            uint32_t vlast = 0;  // the page's last read
            float o[DV][8];      // the page's sum
#pragma unroll
            for (int x = 0; x < DV; ++x)
#pragma unroll
                for (int v = 0; v < 8; ++v) o[x][v] = 0.f;
            if constexpr (LAYOUT == kSplit) {
#pragma unroll kUN
                for (int n = 0; n < 4; ++n) {
                    const int quad = (n + (lane >> 1)) & 3;
                    float4 x[DV];
#pragma unroll
                    for (int i = 0; i < DV; ++i) x[i] = lds_v4(vp + (uint32_t)((lane + 32 * i) * 64 + quad * 16));
                    vlast = __float_as_uint(x[DV - 1].w);
#pragma unroll
                    for (int v = 0; v < 8; ++v) {
                        const float4 w = lds_v4(ps + (uint32_t)(((v >> 2) * 80 + (v & 3) * 16 + quad * 4) * 4));
#pragma unroll
                        for (int i = 0; i < DV; ++i) {
                            o[i][v] = fmaf(w.x, x[i].x, o[i][v]);
                            o[i][v] = fmaf(w.y, x[i].y, o[i][v]);
                            o[i][v] = fmaf(w.z, x[i].z, o[i][v]);
                            o[i][v] = fmaf(w.w, x[i].w, o[i][v]);
                        }
                    }
                }
            } else {
#pragma unroll kUT
                for (int t = 0; t < kBS; ++t) {
                    const float4 a = lds_v4(ps + (uint32_t)(t * 32)), b = lds_v4(ps + (uint32_t)(t * 32 + 16));
                    const float w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                    for (int i = 0; i < DV; i += 4) {
                        const float4 x = lds_v4(vp + (uint32_t)((i + (lane >> 3)) * 2048 + t * 128 +
                                                                (((lane ^ t) & 7) << 4)));
                        vlast = __float_as_uint(x.w);
#pragma unroll
                        for (int v = 0; v < 8; ++v) {
                            o[i][v] = fmaf(w[v], x.x, o[i][v]);
                            o[i + 1][v] = fmaf(w[v], x.y, o[i + 1][v]);
                            o[i + 2][v] = fmaf(w[v], x.z, o[i + 2][v]);
                            o[i + 3][v] = fmaf(w[v], x.w, o[i + 3][v]);
                        }
                    }
                }
            }
#pragma unroll
            for (int x = 0; x < DV; ++x)
#pragma unroll
                for (int v = 0; v < 8; ++v) acc[x][v] += o[x][v];
            __syncwarp();  // also: P has been read
            if (lane == 0) mbar_arrive_after(sm.empty_v + st * 8, vlast, p.zero);
        }
        __syncwarp();
        // descriptor and query rows have been read
        if (lane == 0) mbar_arrive_after(sm.td_empty + slot * 8, qlast, p.zero);

        move_max();  // the exact statistics
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
            if ((lane & 15) == 0) sm.ml[warp * C::kMergeRows + hb * 4 + i] = make_float2(m[i], l[i]);
        }
#pragma unroll
        for (int v = 0; v < 8; ++v) {
            if constexpr (LAYOUT == kSplit) {
#pragma unroll
                for (int i = 0; i < DV; ++i) mw[v * C::kMergeStride + lane + 32 * i] = acc[i][v];
            } else {
#pragma unroll
                for (int i = 0; i < DV; i += 4)
                    *reinterpret_cast<float4*>(mw + v * C::kMergeStride + (i * 32 + lane * 4)) =
                        make_float4(acc[i][v], acc[i + 1][v], acc[i + 2][v], acc[i + 3][v]);
            }
        }
        if (!consumer_sync(sm, mphase, lane)) {
            report(p, PA_DEVERR_TIMEOUT);
            *sm.abort = 1;
            return;
        }
        if (!tile_finish<C, float, HEAD, NC>(p, d, sm, warp, lane, mphase)) {
            report(p, PA_DEVERR_TIMEOUT);
            *sm.abort = 1;
            return;
        }
        gbase += (uint32_t)npages;
    }
}

// ------------------------------------------------------------------ kernels

// Two n-tiles hold 16 rows of accumulators (~200 registers uncapped), and the
// fp32 tensor-core consumer holds Q as two tf32 terms (~213): cap them so that
// two CTAs share an SM, as they do for one n-tile of 16-bit inputs.  fp32 with
// two n-tiles fills an SM's shared memory with one CTA (16 KB stages): no cap.
// fp8 with one n-tile: capped for three CTAs per SM (128 registers: fifteen
// warps put four on some SM sub-partition, whose register file is 16 K).
// Value heads of 256 hold one CTA per SM.
template <typename T, int HEAD, int NT, int LAYOUT, int STAGES, int NC, int KV, bool MQ, bool DIFF>
__global__ void __launch_bounds__((NC + 1) * 32,
                                  (HEAD > 128 || (std::is_same<T, float>::value && NT > 1))
                                      ? 1
                                      : ((NT > 1 || std::is_same<T, float>::value) ? 2 : (KV != kKvSame ? 3 : 1)))
    pa_partition_kernel(const Params p, const __grid_constant__ CUtensorMap tmk,
                        const __grid_constant__ CUtensorMap tmv) {
    using C = Cfg<T, HEAD, NT, LAYOUT, STAGES, NC, KV, MQ, DIFF>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gen = smem_raw + (base - raw);

    Smem sm;
    sm.ring = base + C::oRing;
    sm.q = base + C::oQ;
    sm.merge = reinterpret_cast<float*>(gen + C::oMerge);
    sm.ml = reinterpret_cast<float2*>(gen + C::oML);
    sm.desc = reinterpret_cast<TileDesc*>(gen + C::oDesc);
    sm.full = base + C::oBar;
    sm.empty = sm.full + STAGES * 8;
    sm.td_full = sm.empty + STAGES * 8;
    sm.td_empty = sm.td_full + C::kTD * 8;
    sm.merge_bar = sm.td_empty + C::kTD * 8;
    sm.full_v = sm.merge_bar + 8;
    sm.empty_v = sm.full_v + STAGES * 8;
    sm.abort = reinterpret_cast<volatile int*>(gen + C::oAbort);
    sm.wait_ns = p.wait_limit_ns ? p.wait_limit_ns : kWaitLimitNs;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == NC) prefetch_first_tile<C, HEAD>(p, lane);
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(sm.full + s * 8, 1);
            mbar_init(sm.empty + s * 8, C::kPageWarps);
            if constexpr (C::kHalves) {
                mbar_init(sm.full_v + s * 8, 1);
                mbar_init(sm.empty_v + s * 8, C::kPageWarps);
            }
        }
        for (int s = 0; s < C::kTD; ++s) {
            mbar_init(sm.td_full + s * 8, 1);
            mbar_init(sm.td_empty + s * 8, NC);
        }
        mbar_init(sm.merge_bar, NC);
        sm.abort[0] = 0;
        sm.abort[1] = 0;
        sm.abort[2] = 0;
        fence_mbar_init();
    }
    if constexpr (C::kTensorMap) {
        if (threadIdx.x == NC * 32) {
            prefetch_tensormap(&tmk);
            prefetch_tensormap(&tmv);
        }
    }
    __syncthreads();
    pdl_launch_dependents();  // the reduce kernel may be scheduled; it waits for our completion
    // Earlier work in the stream (inputs, workspace readers) must be done.
    // With final metadata only the producer waits, once it has its first tile
    // (producer); every other warp reaches global memory only after that
    // through the producer's barriers.
    if (!p.metadata_ready) pdl_wait_primary();

    if (warp == NC) {
        producer<C, HEAD, STAGES>(p, sm, &tmk, &tmv, lane);
    } else if constexpr (C::kF32 && DIFF) {
        consumer_fma<C, HEAD, LAYOUT, STAGES, NC>(p, sm, warp, lane);
    } else if constexpr (C::kF32) {
        consumer_tf32<C, HEAD, NT, LAYOUT, STAGES, NC>(p, sm, warp, lane);
    } else {
        if constexpr (KV == kKvSame)
            consumer_mma<C, T, HEAD, NT, LAYOUT, STAGES, NC>(p, sm, warp, lane);
        else
            consumer_mma_fp8<C, T, HEAD, NT, LAYOUT, STAGES, NC, KV>(p, sm, warp, lane);
    }
}

// Phase 2: one CTA of 32*WARPS threads per (sequence, head), one pass.  Each
// lane owns four head dims (a float4 column) of one partition row and keeps U
// partition rows in flight; it carries its own running max, so no separate
// pass over max_logits is needed.  The rows are then combined with the usual
// max rescale in shared memory.
template <typename T, int HEAD, int WARPS, int U, bool MQ>
__global__ void __launch_bounds__(WARPS * 32) pa_reduce_kernel(const Params p) {
    constexpr int D4 = HEAD / 4;          // float4 columns of a partition row
    constexpr int RPW = 32 / D4;          // partition rows per warp (1 or 2)
    constexpr int RSTEP = WARPS * RPW;    // partition rows per CTA round (U rounds in flight)
    constexpr int NT = WARPS * 32;
    __shared__ float4 part[RSTEP][D4];
    __shared__ float rowm[RSTEP], roww[RSTEP];

    // one CTA per (sequence, query token, head); query tokens beyond the
    // sequence's count return at once
    const int bid = blockIdx.x;
    const int sq = bid / p.num_heads, h = bid - sq * p.num_heads;
    const int s = MQ ? sq / p.max_q_len : sq, qi = MQ ? sq - s * p.max_q_len : 0;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_launch_dependents();  // the next launch may start its prologue; it waits for us
    pdl_wait_primary();

    int q0 = s, qn = 1;
    if constexpr (MQ) {
        query_rows(p, s, q0, qn);
        if (qi >= qn) return;
    }
    const int len = clamp_len(p, p.seq_lens[s]);
    const int hi = len - qn + qi;                      // the query token's position
    const int P = hi >= 0 ? (hi + kPart) / kPart : 0;  // partitions holding its keys
    const int p0 = window_lo_at(p, hi) / kPart;     // partitions before p0: outside the window
    const int64_t row = (int64_t)q0 + qi;
    const int64_t sb = (row * p.num_heads + h) * p.max_parts;
    float* ml = p.max_logits + sb;
    float* es = p.exp_sums + sb;
    const float* tmp = p.tmp_out + sb * HEAD;
    const uint64_t pol = l2_policy_evict_first();  // partition outputs: last use
    T* o = static_cast<T*>(p.out) + (row * p.num_heads + h) * HEAD;

    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (P > 0) {
        const int prow = warp * RPW + lane / D4, d4 = lane % D4;
        float M = -INFINITY, W = 0.f;
        for (int qb = p0 + prow; qb < P; qb += RSTEP * U) {
            float mq[U], eq[U];
            float4 t[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int q = qb + u * RSTEP;
                if (q < P) {
                    mq[u] = ml[q];
                    eq[u] = es[q];
                    t[u] = ld_global_v4_hint(tmp + (int64_t)q * HEAD + 4 * d4, pol);
                } else {
                    mq[u] = -INFINITY;
                    eq[u] = 0.f;
                    t[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (mq[u] == -INFINITY) continue;
                if (mq[u] > M) {
                    const float sc = (M == -INFINITY) ? 0.f : expf(M - mq[u]);
                    a.x *= sc;
                    a.y *= sc;
                    a.z *= sc;
                    a.w *= sc;
                    W *= sc;
                    M = mq[u];
                }
                const float c = expf(mq[u] - M) * eq[u];
                a.x += c * t[u].x;
                a.y += c * t[u].y;
                a.z += c * t[u].z;
                a.w += c * t[u].w;
                W += c;
            }
        }
        part[prow][d4] = a;
        if (d4 == 0) {
            rowm[prow] = M;
            roww[prow] = W;
        }
        __syncthreads();
        if (tid < D4) {
            float Mg = -INFINITY;
#pragma unroll
            for (int i = 0; i < RSTEP; ++i) Mg = fmaxf(Mg, rowm[i]);
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
            float Wg = 0.f;
#pragma unroll
            for (int i = 0; i < RSTEP; ++i) {
                if (rowm[i] == -INFINITY) continue;
                const float c = expf(rowm[i] - Mg);
                const float4 v = part[i][tid];
                sum.x += c * v.x;
                sum.y += c * v.y;
                sum.z += c * v.z;
                sum.w += c * v.w;
                Wg += c * roww[i];
            }
            const float inv = 1.f / Wg;
            a = make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv);
        }
        // statistics: sequence frame -> absolute ALiBi positions (every read of
        // max_logits above happened before the barrier)
        if (p.alibi) {
            const float shift = p.alibi[h] * (float)(len - 1);
            for (int q = p0 + tid; q < P; q += NT) ml[q] += shift;
        }
    }
    if (tid < D4) {
        T* dst = o + 4 * tid;
        if constexpr (std::is_same<T, float>::value) {
            *reinterpret_cast<float4*>(dst) = a;
        } else {
            constexpr bool BF = std::is_same<T, __nv_bfloat16>::value;
            uint2 v;
            v.x = pack2<BF>(a.x, a.y);
            v.y = pack2<BF>(a.z, a.w);
            *reinterpret_cast<uint2*>(dst) = v;
        }
    }
    for (int q = P + tid; q < p.max_parts; q += NT) {
        ml[q] = -INFINITY;
        es[q] = 0.f;
    }
    for (int q = tid; q < p0 && q < P; q += NT) {
        ml[q] = -INFINITY;
        es[q] = 0.f;
    }
}

// Phase 2 of one (query row, head) by one warp: M = max_p m_p, w_p = exp(m_p
// - M) e_p / sum, out = sum_p w_p tmp_p.  Lane i holds the statistics of
// partitions p0 + i, p0 + i + 32, ... and HEAD/32 columns of every partition
// output; the first eight partition outputs are loaded together with the
// statistics, so a row of up to eight partitions costs one round trip.  Then
// the row's statistics move to absolute ALiBi positions and its unused
// partitions are padded (every read of them is above, in this warp).
// L2ONLY: every load through L2 only (the merge inside the partition kernel
// reads what other CTAs of the same grid wrote); otherwise the partition
// outputs are read with an evict_first hint (their last use).
// merge_stats_row does this for one row `srow` of the statistics, leaving the
// merged output row in acc (columns lane_col).
template <int HEAD, bool L2ONLY, bool DIFF>
__device__ __forceinline__ void merge_stats_row(const Params& p, int64_t srow, int h, int len, int qn, int qi,
                                                int lane, float (&acc)[HEAD / 32]) {
    constexpr int VEC = HEAD / 32;  // columns per lane: 8 (HEAD 256), 4 (HEAD 128) or 2 (HEAD 64)
    constexpr int PRE = 8;          // partition outputs loaded before the weights are known
    const int hi = len - qn + qi;                      // the query token's position
    const int plen = part_len<DIFF>(p);
    const int P = hi >= 0 ? (hi + plen) / plen : 0;  // partitions holding its keys
    const int p0 = window_lo_at(p, hi) / plen;     // partitions before p0: outside the window
    const int64_t sb = srow * p.max_parts;
    float* ml = p.max_logits + sb;
    float* es = p.exp_sums + sb;
    const float* tmp = p.tmp_out + sb * HEAD + lane_col<HEAD>(lane, 0);

    // partition outputs p0 .. p0 + 7 and this lane's first statistics, all in flight
    const uint64_t pol = l2_policy_evict_first();  // partition outputs: last use
    auto load_out = [&](int q, float (&t)[VEC]) {
        if constexpr (VEC >= 4) {
#pragma unroll
            for (int c = 0; c < VEC; c += 4) {
                const float* at = tmp + (int64_t)q * HEAD + c * 32;
                const float4 v = L2ONLY ? __ldcg(reinterpret_cast<const float4*>(at)) : ld_global_v4_hint(at, pol);
                t[c] = v.x; t[c + 1] = v.y; t[c + 2] = v.z; t[c + 3] = v.w;
            }
        } else {
            const float2 v = L2ONLY ? __ldcg(reinterpret_cast<const float2*>(tmp + (int64_t)q * HEAD))
                                    : ld_global_v2_hint(tmp + (int64_t)q * HEAD, pol);
            t[0] = v.x; t[1] = v.y;
        }
    };
    auto ld_stat = [&](const float* a) { return L2ONLY ? __ldcg(a) : *a; };
    float pre[PRE][VEC];
#pragma unroll
    for (int k = 0; k < PRE; ++k) {
        if (p0 + k < P) {
            load_out(p0 + k, pre[k]);
        } else {
#pragma unroll
            for (int v = 0; v < VEC; ++v) pre[k][v] = 0.f;
        }
    }
    const int q1 = p0 + lane;
    const float m1 = q1 < P ? ld_stat(ml + q1) : -INFINITY;
    const float e1 = q1 < P ? ld_stat(es + q1) : 0.f;

    // global max and weight sum over the row's partitions (lanes, then the warp)
    float M = m1, W = m1 == -INFINITY ? 0.f : e1;
    for (int q = q1 + 32; q < P; q += 32) {
        const float m = ld_stat(ml + q), e = ld_stat(es + q);
        if (m == -INFINITY) continue;
        if (m > M) {
            W = (M == -INFINITY) ? 0.f : W * expf(M - m);
            M = m;
        }
        W += expf(m - M) * e;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float Mo = __shfl_xor_sync(0xffffffffu, M, o), Wo = __shfl_xor_sync(0xffffffffu, W, o);
        const float Mn = fmaxf(M, Mo);
        W = (M == -INFINITY ? 0.f : W * expf(M - Mn)) + (Mo == -INFINITY ? 0.f : Wo * expf(Mo - Mn));
        M = Mn;
    }
    const float invW = W > 0.f ? 1.f / W : 0.f;

    // weighted sum of the partition outputs; lane i holds the weight of
    // partition p0 + 32j + i for the current group j of 32
#pragma unroll
    for (int v = 0; v < VEC; ++v) acc[v] = 0.f;
    float c = m1 == -INFINITY ? 0.f : expf(m1 - M) * e1 * invW;
#pragma unroll
    for (int k = 0; k < PRE; ++k) {
        const float ck = __shfl_sync(0xffffffffu, c, k);
#pragma unroll
        for (int v = 0; v < VEC; ++v) acc[v] = fmaf(ck, pre[k][v], acc[v]);
    }
    for (int qb = p0 + PRE; qb < P; qb += PRE) {
        if (((qb - p0) & 31) == 0) {  // next group of 32 partitions
            const int q = qb + lane;
            c = 0.f;
            if (q < P) {
                const float m = ld_stat(ml + q);
                c = m == -INFINITY ? 0.f : expf(m - M) * ld_stat(es + q) * invW;
            }
        }
        float t[PRE][VEC];
#pragma unroll
        for (int k = 0; k < PRE; ++k) {
            if (qb + k < P) {
                load_out(qb + k, t[k]);
            } else {
#pragma unroll
                for (int v = 0; v < VEC; ++v) t[k][v] = 0.f;
            }
        }
#pragma unroll
        for (int k = 0; k < PRE; ++k) {
            const float ck = __shfl_sync(0xffffffffu, c, (qb - p0 + k) & 31);
#pragma unroll
            for (int v = 0; v < VEC; ++v) acc[v] = fmaf(ck, t[k][v], acc[v]);
        }
    }

    // statistics: sequence frame -> absolute ALiBi positions; unused partitions
    // padded (every read of this row's statistics is above, in this warp)
    __syncwarp();
    const float shift = p.alibi ? p.alibi[h] * (float)(len - 1) : 0.f;
    for (int q = lane; q < p.max_parts; q += 32) {
        if (q >= p0 && q < P) {
            if (p.alibi) ml[q] += shift;
        } else {
            ml[q] = -INFINITY;
            es[q] = 0.f;
        }
    }
}

template <typename T, int HEAD, bool L2ONLY>
__device__ __forceinline__ void merge_row_warp(const Params& p, int64_t row, int h, int len, int qn, int qi,
                                               int lane) {
    float acc[HEAD / 32];
    merge_stats_row<HEAD, L2ONLY, false>(p, row * p.num_heads + h, h, len, qn, qi, lane, acc);
    store_row<T, HEAD>(static_cast<T*>(p.out) + (row * p.num_heads + h) * HEAD, acc, lane);
}

// Phase 2 with one warp per (sequence, query token, head) row, for batches of
// many rows with few partitions each (a CTA per row would need several waves
// of mostly idle CTAs).  No shared memory, no block barrier.
template <typename T, int HEAD, bool MQ>
__global__ void __launch_bounds__(kReduceWarpsPerCta * 32) pa_reduce_warp_kernel(const Params p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_launch_dependents();
    pdl_wait_primary();

    const int64_t rid = (int64_t)blockIdx.x * kReduceWarpsPerCta + warp;
    const int64_t nrows = (int64_t)p.num_seqs * (MQ ? p.max_q_len : 1) * p.num_heads;
    if (rid >= nrows) return;
    const int sq = (int)(rid / p.num_heads), h = (int)(rid - (int64_t)sq * p.num_heads);
    const int s = MQ ? sq / p.max_q_len : sq, qi = MQ ? sq - s * p.max_q_len : 0;
    int q0 = s, qn = 1;
    if constexpr (MQ) {
        query_rows(p, s, q0, qn);
        if (qi >= qn) return;
    }
    const int len = clamp_len(p, p.seq_lens[s]);
    merge_row_warp<T, HEAD, false>(p, (int64_t)q0 + qi, h, len, qn, qi, lane);
}

// Phase 2 of one differential (query row, head) by one warp, both maps side by side:
// the first PRE partition outputs of both are loaded with the statistics, so a row
// of up to PRE partitions costs one round trip; then lambda, norm and the output
// row, and the row's statistics as merge_stats_row leaves them.  L2ONLY as there.
template <typename T, int HEAD, bool L2ONLY>
__device__ __forceinline__ void diff_merge_row(const Params& p, int64_t row, int h, int len, int qn, int qi, int lane) {
    constexpr int VEC = HEAD / 32, PRE = HEAD > 128 ? 2 : 4;
    const int hi = len - qn + qi;                       // the query token's position
    const int plen = part_len<true>(p);
    const int P = hi >= 0 ? (hi + plen) / plen : 0;     // partitions holding its keys
    const int p0 = window_lo_at(p, hi) / plen;          // partitions before p0: outside the window
    const int64_t sb = 2 * (row * p.num_heads + h) * p.max_parts;
    const uint64_t pol = l2_policy_evict_first();       // partition outputs: last use
    auto load_out = [&](int map, int q, float (&t)[VEC]) {
        const float* at = p.tmp_out + (sb + (int64_t)map * p.max_parts + q) * HEAD + lane * 4;
#pragma unroll
        for (int c = 0; c < VEC; c += 4) {
            const float4 v = L2ONLY ? __ldcg(reinterpret_cast<const float4*>(at + c * 32))
                                    : ld_global_v4_hint(at + c * 32, pol);
            t[c] = v.x; t[c + 1] = v.y; t[c + 2] = v.z; t[c + 3] = v.w;
        }
    };
    auto ld_stat = [&](const float* a) { return L2ONLY ? __ldcg(a) : *a; };
    float* ml[2] = {p.max_logits + sb, p.max_logits + sb + p.max_parts};
    float* es[2] = {p.exp_sums + sb, p.exp_sums + sb + p.max_parts};

    float pre[2][PRE][VEC];
#pragma unroll
    for (int map = 0; map < 2; ++map)
#pragma unroll
        for (int k = 0; k < PRE; ++k) {
            if (p0 + k < P) {
                load_out(map, p0 + k, pre[map][k]);
            } else {
#pragma unroll
                for (int v = 0; v < VEC; ++v) pre[map][k][v] = 0.f;
            }
        }
    const int q1 = p0 + lane;
    float m1[2], e1[2], M[2], invW[2];
#pragma unroll
    for (int map = 0; map < 2; ++map) {
        m1[map] = q1 < P ? ld_stat(ml[map] + q1) : -INFINITY;
        e1[map] = q1 < P ? ld_stat(es[map] + q1) : 0.f;
    }
#pragma unroll
    for (int map = 0; map < 2; ++map) {
        // global max and weight sum over the row's partitions (lanes, then the warp)
        float m = m1[map], w = m == -INFINITY ? 0.f : e1[map];
        for (int q = q1 + 32; q < P; q += 32) {
            const float mq = ld_stat(ml[map] + q), eq = ld_stat(es[map] + q);
            if (mq == -INFINITY) continue;
            if (mq > m) {
                w = m == -INFINITY ? 0.f : w * expf(m - mq);
                m = mq;
            }
            w += expf(mq - m) * eq;
        }
        float mx = m;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        w = m == -INFINITY ? 0.f : w * expf(m - mx);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
        M[map] = mx;
        invW[map] = w > 0.f ? 1.f / w : 0.f;
    }

    float o[2][VEC];
#pragma unroll
    for (int map = 0; map < 2; ++map) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) o[map][v] = 0.f;
        // lane i holds the weight of partition p0 + 32 j + i of the current group j
        float c = m1[map] == -INFINITY ? 0.f : expf(m1[map] - M[map]) * e1[map] * invW[map];
#pragma unroll
        for (int k = 0; k < PRE; ++k) {
            const float ck = __shfl_sync(0xffffffffu, c, k);
#pragma unroll
            for (int v = 0; v < VEC; ++v) o[map][v] = fmaf(ck, pre[map][k][v], o[map][v]);
        }
        for (int qb = p0 + PRE; qb < P; qb += PRE) {
            if (((qb - p0) & 31) == 0) {
                const int q = qb + lane;
                c = 0.f;
                if (q < P) {
                    const float mq = ld_stat(ml[map] + q);
                    c = mq == -INFINITY ? 0.f : expf(mq - M[map]) * ld_stat(es[map] + q) * invW[map];
                }
            }
            float t[PRE][VEC];
#pragma unroll
            for (int k = 0; k < PRE; ++k) {
                if (qb + k < P) {
                    load_out(map, qb + k, t[k]);
                } else {
#pragma unroll
                    for (int v = 0; v < VEC; ++v) t[k][v] = 0.f;
                }
            }
#pragma unroll
            for (int k = 0; k < PRE; ++k) {
                const float ck = __shfl_sync(0xffffffffu, c, (qb - p0 + k) & 31);
#pragma unroll
                for (int v = 0; v < VEC; ++v) o[map][v] = fmaf(ck, t[k][v], o[map][v]);
            }
        }
    }
    diff_row<T, HEAD>(p, row, h, o[0], o[1], lane);
    // statistics: sequence frame -> absolute ALiBi positions; unused partitions
    // padded (every read of this row's statistics is above, in this warp)
    __syncwarp();
    const float shift = p.alibi ? p.alibi[h] * (float)(len - 1) : 0.f;
    for (int q = lane; q < 2 * p.max_parts; q += 32) {
        const int map = q >= p.max_parts, at = q - map * p.max_parts;
        if (at >= p0 && at < P) {
            if (p.alibi) ml[map][at] += shift;
        } else {
            ml[map][at] = -INFINITY;
            es[map][at] = 0.f;
        }
    }
}

// Phase 2 of differential rows, up to kDiffReduceFewParts partitions: one warp per
// (sequence, query token, head).  (256 x 1000, 4096 rows: 82.5 us for the whole
// call, with two warps per row 87; but with eight partitions 48.8 against 46, so
// pa_diff_reduce_pair_kernel takes those.)
template <typename T, int HEAD, bool MQ>
__global__ void __launch_bounds__(kReduceWarpsPerCta * 32, HEAD > 128 ? 2 : 4) pa_diff_reduce_warp_kernel(const Params p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_launch_dependents();
    pdl_wait_primary();

    const int64_t rid = (int64_t)blockIdx.x * kReduceWarpsPerCta + warp;
    const int64_t nrows = (int64_t)p.num_seqs * (MQ ? p.max_q_len : 1) * p.num_heads;
    if (rid >= nrows) return;
    const int sq = (int)(rid / p.num_heads), h = (int)(rid - (int64_t)sq * p.num_heads);
    const int s = MQ ? sq / p.max_q_len : sq, qi = MQ ? sq - s * p.max_q_len : 0;
    int q0 = s, qn = 1;
    if constexpr (MQ) {
        query_rows(p, s, q0, qn);
        if (qi >= qn) return;
    }
    diff_merge_row<T, HEAD, false>(p, (int64_t)q0 + qi, h, clamp_len(p, p.seq_lens[s]), qn, qi, lane);
}

// Phase 2 of differential rows, more partitions: two warps per (sequence, query
// token, head), one map each (eight partition outputs in flight per map); the
// second hands its row to the first through shared memory.
template <typename T, int HEAD, bool MQ>
__global__ void __launch_bounds__(kReduceWarpsPerCta * 32) pa_diff_reduce_pair_kernel(const Params p) {
    constexpr int VEC = HEAD / 32, ROWS = kReduceWarpsPerCta / 2;
    __shared__ float second[ROWS][HEAD];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, map = warp & 1;
    pdl_launch_dependents();
    pdl_wait_primary();

    const int64_t rid = (int64_t)blockIdx.x * ROWS + (warp >> 1);
    const int64_t nrows = (int64_t)p.num_seqs * (MQ ? p.max_q_len : 1) * p.num_heads;
    const int sq = (int)(rid / p.num_heads), h = (int)(rid - (int64_t)sq * p.num_heads);
    const int s = MQ ? sq / p.max_q_len : sq, qi = MQ ? sq - s * p.max_q_len : 0;
    int q0 = s, qn = 1;
    bool mine = rid < nrows;
    if (MQ && mine) {
        query_rows(p, s, q0, qn);
        mine = qi < qn;
    }
    const int64_t row = (int64_t)q0 + qi;
    float o[VEC];
    if (mine) {
        merge_stats_row<HEAD, false, true>(p, 2 * (row * p.num_heads + h) + map, h, clamp_len(p, p.seq_lens[s]), qn,
                                           qi, lane, o);
        if (map)
#pragma unroll
            for (int v = 0; v < VEC; ++v) second[warp >> 1][lane_col<HEAD>(lane, v)] = o[v];
    }
    __syncthreads();
    if (!mine || map) return;
    float o2[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) o2[v] = second[warp >> 1][lane_col<HEAD>(lane, v)];
    diff_row<T, HEAD>(p, row, h, o, o2, lane);
}

// Phase 2 of differential rows, many partitions: one CTA per (sequence, query
// token, head), half of its warps per map; each thread owns a float4 column of a
// partition row and keeps U of them in flight with its own running max, as
// pa_reduce_kernel does.  The first warp combines them and writes the row.
template <typename T, int HEAD, int WARPS, int U, bool MQ>
__global__ void __launch_bounds__(WARPS * 32) pa_diff_reduce_kernel(const Params p) {
    constexpr int D4 = HEAD / 4;
    constexpr int HALF = WARPS * 16;     // threads of a map
    constexpr int RSTEP = HALF / D4;     // partition rows per round
    constexpr int VEC = HEAD / 32;
    static_assert(HALF % D4 == 0, "whole partition rows");
    __shared__ __align__(16) float part[2][RSTEP][HEAD];
    __shared__ float rowm[2][RSTEP], roww[2][RSTEP];

    const int bid = blockIdx.x;
    const int sq = bid / p.num_heads, h = bid - sq * p.num_heads;
    const int s = MQ ? sq / p.max_q_len : sq, qi = MQ ? sq - s * p.max_q_len : 0;
    const int map = threadIdx.x / HALF, tid = threadIdx.x % HALF, lane = threadIdx.x & 31;
    pdl_launch_dependents();
    pdl_wait_primary();

    int q0 = s, qn = 1;
    if constexpr (MQ) {
        query_rows(p, s, q0, qn);
        if (qi >= qn) return;
    }
    const int len = clamp_len(p, p.seq_lens[s]);
    const int hi = len - qn + qi;                      // the query token's position
    const int plen = part_len<true>(p);
    const int P = hi >= 0 ? (hi + plen) / plen : 0;  // partitions holding its keys
    const int p0 = window_lo_at(p, hi) / plen;     // partitions before p0: outside the window
    const int64_t row = (int64_t)q0 + qi;
    const int64_t sb = (2 * (row * p.num_heads + h) + map) * p.max_parts;
    float* ml = p.max_logits + sb;
    float* es = p.exp_sums + sb;
    const float* tmp = p.tmp_out + sb * HEAD;
    const uint64_t pol = l2_policy_evict_first();  // partition outputs: last use

    const int prow = tid / D4, d4 = tid % D4;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    float M = -INFINITY, W = 0.f;
    for (int qb = p0 + prow; qb < P; qb += RSTEP * U) {
        float mq[U], eq[U];
        float4 t[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int q = qb + u * RSTEP;
            if (q < P) {
                mq[u] = ml[q];
                eq[u] = es[q];
                t[u] = ld_global_v4_hint(tmp + (int64_t)q * HEAD + 4 * d4, pol);
            } else {
                mq[u] = -INFINITY;
                eq[u] = 0.f;
                t[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (mq[u] == -INFINITY) continue;
            if (mq[u] > M) {
                const float sc = (M == -INFINITY) ? 0.f : expf(M - mq[u]);
                a.x *= sc;
                a.y *= sc;
                a.z *= sc;
                a.w *= sc;
                W *= sc;
                M = mq[u];
            }
            const float c = expf(mq[u] - M) * eq[u];
            a.x += c * t[u].x;
            a.y += c * t[u].y;
            a.z += c * t[u].z;
            a.w += c * t[u].w;
            W += c;
        }
    }
    *reinterpret_cast<float4*>(&part[map][prow][4 * d4]) = a;
    if (d4 == 0) {
        rowm[map][prow] = M;
        roww[map][prow] = W;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        float o[2][VEC];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float Mg = -INFINITY, Wg = 0.f;
#pragma unroll
            for (int i = 0; i < RSTEP; ++i) Mg = fmaxf(Mg, rowm[k][i]);
#pragma unroll
            for (int v = 0; v < VEC; ++v) o[k][v] = 0.f;
#pragma unroll
            for (int i = 0; i < RSTEP; ++i) {
                const float c = rowm[k][i] == -INFINITY ? 0.f : expf(rowm[k][i] - Mg);
                Wg = fmaf(c, roww[k][i], Wg);
#pragma unroll
                for (int v = 0; v < VEC; ++v) o[k][v] = fmaf(c, part[k][i][lane_col<HEAD>(lane, v)], o[k][v]);
            }
            const float inv = Wg > 0.f ? 1.f / Wg : 0.f;
#pragma unroll
            for (int v = 0; v < VEC; ++v) o[k][v] *= inv;
        }
        diff_row<T, HEAD>(p, row, h, o[0], o[1], lane);
    }
    // statistics: sequence frame -> absolute ALiBi positions, unused partitions
    // padded (every read of them above happened before the barrier)
    const float shift = p.alibi ? p.alibi[h] * (float)(len - 1) : 0.f;
    for (int q = tid; q < p.max_parts; q += HALF) {
        if (q >= p0 && q < P) {
            if (p.alibi) ml[q] += shift;
        } else {
            ml[q] = -INFINITY;
            es[q] = 0.f;
        }
    }
}

}  // namespace pa
