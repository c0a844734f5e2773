// pa_launch.cuh -- host-side launch of the partition (or v1) kernel and of the
// reduce kernel for one (dtype, head size) family.  Included by the
// per-dtype translation units so they compile in parallel.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

#include "pa_kernels.cuh"

namespace pa {

// What a launch would do, reported instead of launching (see LaunchArgs::query).
struct LaunchOut {
    int occ = 0;        // resident CTAs per SM of the partition kernel
    int64_t grid = 0;   // CTAs of its persistent grid
    bool fused = false; // Phase 2 merge inside the partition kernel (no reduce launch)
};

struct LaunchArgs {
    cudaStream_t stream;
    LaunchOut* query;        // non-null: fill it and launch nothing
    const CUtensorMap* tmk;  // NHD 16-bit only (otherwise unused placeholders)
    const CUtensorMap* tmv;
    int sm_count;
    int64_t tiles_upper;     // upper bound on tiles (persistent grid never exceeds it)
    int group_tiles;         // 1 or 2: n-tiles of 8 query heads
    int layout;
    int head_size;
    int dtype;               // pa_dtype of the query
    void* ev_begin;
    void* ev_end;
};

constexpr int kMaxDevices = 64;

// Launch the partition (or v1) kernel.  *fused reports whether the Phase 2
// merge runs inside it: only with partition counters, a v2 batch that fits in
// one round of the persistent grid (each CTA finishes at most one tile, so at
// most one merge) and at most PA_FUSED_MAX_PARTITIONS partitions per sequence
// (a short merge).  With several rounds the CTA that merges falls behind and
// becomes the last arriver of the next group too, so merges pile up on a few
// CTAs; the separate reduce kernel spreads them over the whole GPU instead.
template <typename T, int HEAD, int NT, int LAYOUT, int KV, bool MQ, bool DIFF = false>
cudaError_t launch_main(const Params& p_in, const LaunchArgs& la, bool* fused) {
    constexpr bool F32 = std::is_same<T, float>::value, WIDE = HEAD > 128;
    constexpr bool FP8X2 = DIFF && !WIDE && NT == 2 && KV != kKvSame;
    constexpr bool F32X2 = DIFF && !WIDE && NT == 2 && F32;
    constexpr int STAGES = FP8X2          ? kStagesFp8x2Diff
                           : F32X2        ? kStagesF32x2Diff
                           : WIDE && F32  ? (NT == 1 ? kStagesF32Wide : kStagesF32Widex2)
                           : WIDE && KV != kKvSame ? (NT == 1 ? kStagesFp8Wide : kStagesFp8Widex2)
                           : WIDE         ? (NT == 1 ? kStages16Wide : kStages16Widex2)
                           : F32          ? (NT == 1 ? kStagesF32 : kStagesF32x2)
                           : KV == kKvE2M1 ? (NT == 1 ? kStagesFp4 : kStagesFp4x2)
                           : KV != kKvSame ? kStagesFp8
                                           : (NT == 1 ? kStages16 : kStages16x2);
    constexpr int NC = FP8X2         ? kConsumerWarps5
                       : F32X2       ? kConsumerWarpsF32x2Diff
                       : WIDE && F32 ? (NT == 1 ? kConsumerWarpsF32Wide : kConsumerWarpsF32Widex2)
                       : WIDE && KV != kKvSame ? (NT == 1 ? kConsumerWarpsFp8Wide : kConsumerWarpsFp8Widex2)
                       : KV == kKvE2M1 ? (NT == 1 ? kConsumerWarpsFp4 : kConsumerWarpsFp4x2)
                       : WIDE ? (NT == 1 ? kConsumerWarps16Wide : kConsumerWarps16Widex2)
                              : ((KV == kKvSame && NT == 1) ? kConsumerWarps5 : kConsumerWarps);
    using C = Cfg<T, HEAD, NT, LAYOUT, STAGES, NC, KV, MQ, DIFF>;
    auto kern = pa_partition_kernel<T, HEAD, NT, LAYOUT, STAGES, NC, KV, MQ, DIFF>;

    static std::atomic<int> occ_cache[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int occ = (dev >= 0 && dev < kMaxDevices) ? occ_cache[dev].load() : 0;
    if (occ <= 0) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
        if (e != cudaSuccess) return e;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kern, C::kThreads, C::kSmemBytes);
        if (e != cudaSuccess) return e;
        if (occ < 1) return cudaErrorInvalidConfiguration;
        if (dev >= 0 && dev < kMaxDevices) occ_cache[dev].store(occ);
    }
    int64_t grid = (int64_t)la.sm_count * occ;
    if (grid > la.tiles_upper) grid = la.tiles_upper;
    if (grid < 1) grid = 1;
    // Equal rounds: the fewest CTAs that keep the number of rounds of the
    // static tile schedule, so that in a uniform batch every CTA gets the same
    // number of tiles instead of a last round that leaves most CTAs idle
    // (1024 tiles: 256 CTAs x 4 instead of 304 CTAs with 112 doing a 4th).
    // tiles_upper is exact for equal lengths and only an upper bound otherwise.
    // The dynamic schedule keeps every resident CTA: its tiles go to whichever
    // CTA is free, so no CTA waits on a fixed share.
    if (!p_in.tile_ctr) {
        const int64_t rounds = (la.tiles_upper + grid - 1) / grid, cut = (la.tiles_upper + rounds - 1) / rounds;
        // 4-bit caches: bound by the instructions of an SM's warps, not by a CTA's stream.  Its CTAs share those, so
        // what counts is the tiles of the busiest SM; a cut that leaves some SMs a CTA more than others
        // can raise them (1024 tiles: 342 CTAs x 3, nine on some SMs; 456 CTAs: seven).
        const int64_t sms = la.sm_count;
        if (KV != kKvE2M1 || (cut + sms - 1) / sms * rounds <= (la.tiles_upper + sms - 1) / sms) grid = cut;
    }
    Params p = p_in;
    p.fused = (!p.v1 && p.counters && p.max_parts <= PA_FUSED_MAX_PARTITIONS &&
               la.tiles_upper <= grid) ? 1 : 0;
    *fused = p.fused != 0;
    if (la.query) {
        la.query->occ = occ;
        la.query->grid = grid;
        la.query->fused = *fused;
        return cudaSuccess;
    }

    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = la.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (la.ev_begin) {
        e = cudaEventRecord(static_cast<cudaEvent_t>(la.ev_begin), la.stream);
        if (e != cudaSuccess) return e;
    }
    e = cudaLaunchKernelEx(&cfg, kern, p, *la.tmk, *la.tmv);
    if (e != cudaSuccess) return e;
    if (la.ev_end) e = cudaEventRecord(static_cast<cudaEvent_t>(la.ev_end), la.stream);
    return e;
}

// Reduce shape by partition count: few partitions need one round of rows,
// long sequences (hundreds of partitions, few (sequence, head) CTAs) want as
// many independent row loads in flight per CTA as possible.
template <typename T, int HEAD, int WARPS, int U, bool MQ>
cudaError_t launch_reduce_shape(const Params& p, const LaunchArgs& la) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)p.num_seqs * p.max_q_len * p.num_heads));
    cfg.blockDim = dim3(WARPS * 32);
    cfg.dynamicSmemBytes = 0;
    cfg.stream = la.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, pa_reduce_kernel<T, HEAD, WARPS, U, MQ>, p);
}

template <typename T, int HEAD, bool MQ>
cudaError_t launch_reduce_warp(const Params& p, const LaunchArgs& la, int64_t rows) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((rows + kReduceWarpsPerCta - 1) / kReduceWarpsPerCta));
    cfg.blockDim = dim3(kReduceWarpsPerCta * 32);
    cfg.dynamicSmemBytes = 0;
    cfg.stream = la.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, pa_reduce_warp_kernel<T, HEAD, MQ>, p);
}

template <typename T, int HEAD, bool MQ>
cudaError_t launch_reduce(const Params& p, const LaunchArgs& la) {
    // Few (sequence, head) rows of many partitions (4 x 28 rows of 196): a
    // wide CTA per row; otherwise one warp per row, so that a batch of
    // thousands of short rows runs in one wave instead of several waves of
    // CTAs that each wait on one round trip.
    const int64_t rows = (int64_t)p.num_seqs * p.max_q_len * p.num_heads;
    if (p.max_parts > 32 && rows <= 2 * (int64_t)la.sm_count)
        return launch_reduce_shape<T, HEAD, 16, 8, MQ>(p, la);
    if (p.max_parts <= kReduceWarpMaxParts) return launch_reduce_warp<T, HEAD, MQ>(p, la, rows);
    return launch_reduce_shape<T, HEAD, 8, 4, MQ>(p, la);
}

template <typename T, int HEAD, int NT, int KV, bool MQ>
cudaError_t launch_layout_mq(const Params& p, const LaunchArgs& la, bool* fused) {
    return la.layout == kNHD ? launch_main<T, HEAD, NT, kNHD, KV, MQ>(p, la, fused)
                             : launch_main<T, HEAD, NT, kSplit, KV, MQ>(p, la, fused);
}

// Single-token decode and several query tokens per sequence are separate
// instantiations, so the common single-token path carries no per-row ranges.
template <typename T, int HEAD, int NT, int KV>
cudaError_t launch_layout(const Params& p, const LaunchArgs& la, bool* fused) {
    return p.query_start ? launch_layout_mq<T, HEAD, NT, KV, true>(p, la, fused)
                         : launch_layout_mq<T, HEAD, NT, KV, false>(p, la, fused);
}

// Whole operation for one (query type, cache type) pair.
template <typename T, int KV = kKvSame>
cudaError_t launch_family(const Params& p, const LaunchArgs& la) {
    cudaError_t e;
    bool fused = false;
    if (la.head_size == 128) {
        e = la.group_tiles == 2 ? launch_layout<T, 128, 2, KV>(p, la, &fused)
                                : launch_layout<T, 128, 1, KV>(p, la, &fused);
    } else {
        e = la.group_tiles == 2 ? launch_layout<T, 64, 2, KV>(p, la, &fused)
                                : launch_layout<T, 64, 1, KV>(p, la, &fused);
    }
    if (e != cudaSuccess || p.v1 || fused || la.query) return e;
    if (p.query_start)
        return la.head_size == 128 ? launch_reduce<T, 128, true>(p, la) : launch_reduce<T, 64, true>(p, la);
    return la.head_size == 128 ? launch_reduce<T, 128, false>(p, la) : launch_reduce<T, 64, false>(p, la);
}

// 4-bit caches: one layout.
template <typename T, int HEAD, bool MQ>
cudaError_t launch_fp4_head(const Params& p, const LaunchArgs& la) {
    bool fused = false;
    const cudaError_t e = la.group_tiles == 2 ? launch_main<T, HEAD, 2, kNHD, kKvE2M1, MQ>(p, la, &fused)
                                              : launch_main<T, HEAD, 1, kNHD, kKvE2M1, MQ>(p, la, &fused);
    if (e != cudaSuccess || p.v1 || fused || la.query) return e;
    return launch_reduce<T, HEAD, MQ>(p, la);
}

template <typename T>
cudaError_t launch_family_fp4(const Params& p, const LaunchArgs& la) {
    if (la.head_size == 128)
        return p.query_start ? launch_fp4_head<T, 128, true>(p, la) : launch_fp4_head<T, 128, false>(p, la);
    return p.query_start ? launch_fp4_head<T, 64, true>(p, la) : launch_fp4_head<T, 64, false>(p, la);
}

// ---------------------------------------------------------------- differential
//
// Measured (GPU time per call, against the KV bytes at the copy rate of 6.8 TB/s):
// 32 x 4096, keys of 64, values of 128, fp16 44.4 us (39.6), fp32 81.4 (79); 4 x
// 100000 bf16, groups of seven, 122.9 (120.6), e4m3 83 (60.3); 32 x 4096 e4m3 with
// four tokens 63.2, with a softcap 68.7 (39.6); 64 ragged sequences, keys of 128, values of 256, bf16
// 152 (140.6), fp32 of those heads 32 x 4096 164 (158).  16-bit caches, and fp32 ones
// up to four rows, are bound by memory, fp8 and fp32 ones of more rows by the
// consumers' chain of a page.

template <typename T, int HEAD, bool MQ>
cudaError_t launch_diff_reduce(const Params& p, const LaunchArgs& la) {
    const int64_t rows = (int64_t)p.num_seqs * p.max_q_len * p.num_heads;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = la.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // few rows of many partitions, or more partitions than a warp should walk: a
    // CTA per row (as launch_reduce)
    if ((p.max_parts > 32 && rows <= 2 * (int64_t)la.sm_count) || p.max_parts > kReduceWarpMaxParts) {
        cfg.gridDim = dim3((unsigned)rows);
        cfg.blockDim = dim3(16 * 32);
        return cudaLaunchKernelEx(&cfg, pa_diff_reduce_kernel<T, HEAD, 16, HEAD == 128 ? 8 : 4, MQ>, p);
    }
    cfg.blockDim = dim3(kReduceWarpsPerCta * 32);
    if (p.max_parts <= kDiffReduceFewParts) {
        cfg.gridDim = dim3((unsigned)((rows + kReduceWarpsPerCta - 1) / kReduceWarpsPerCta));
        return cudaLaunchKernelEx(&cfg, pa_diff_reduce_warp_kernel<T, HEAD, MQ>, p);
    }
    cfg.gridDim = dim3((unsigned)((rows + kReduceWarpsPerCta / 2 - 1) / (kReduceWarpsPerCta / 2)));
    return cudaLaunchKernelEx(&cfg, pa_diff_reduce_pair_kernel<T, HEAD, MQ>, p);
}

template <typename T, int HEAD, int NT, int KV, bool MQ>
cudaError_t launch_diff_layout(const Params& p, const LaunchArgs& la, bool* fused) {
    return la.layout == kNHD ? launch_main<T, HEAD, NT, kNHD, KV, MQ, true>(p, la, fused)
                             : launch_main<T, HEAD, NT, kSplit, KV, MQ, true>(p, la, fused);
}

template <typename T, int HEAD, int KV, bool MQ>
cudaError_t launch_diff_head(const Params& p, const LaunchArgs& la) {
    bool fused = false;
    const cudaError_t e = la.group_tiles == 2 ? launch_diff_layout<T, HEAD, 2, KV, MQ>(p, la, &fused)
                                              : launch_diff_layout<T, HEAD, 1, KV, MQ>(p, la, &fused);
    if (e != cudaSuccess || p.v1 || fused || la.query) return e;
    return launch_diff_reduce<T, HEAD, MQ>(p, la);
}

// Differential attention for one (query type, cache type) pair; la.head_size is
// the value head size, 128 or 256.
template <typename T, int KV, int HEAD>
cudaError_t launch_diff_family(const Params& p, const LaunchArgs& la) {
    return p.query_start ? launch_diff_head<T, HEAD, KV, true>(p, la) : launch_diff_head<T, HEAD, KV, false>(p, la);
}

// One translation unit per (query type, cache kind); kv: kKvSame / kKvE4M3 / kKvE5M2
cudaError_t launch_diff_f32(const Params& p, const LaunchArgs& la);
cudaError_t launch_diff_f16(const Params& p, const LaunchArgs& la);
cudaError_t launch_diff_bf16(const Params& p, const LaunchArgs& la);
cudaError_t launch_diff_f16_fp8(const Params& p, const LaunchArgs& la, int kv);
cudaError_t launch_diff_bf16_fp8(const Params& p, const LaunchArgs& la, int kv);

cudaError_t launch_f32(const Params& p, const LaunchArgs& la);
cudaError_t launch_f16(const Params& p, const LaunchArgs& la);
cudaError_t launch_bf16(const Params& p, const LaunchArgs& la);
cudaError_t launch_f16_fp8(const Params& p, const LaunchArgs& la, int kv);   // kv: kKvE4M3 / kKvE5M2
cudaError_t launch_bf16_fp8(const Params& p, const LaunchArgs& la, int kv);
cudaError_t launch_f16_fp4(const Params& p, const LaunchArgs& la);
cudaError_t launch_bf16_fp4(const Params& p, const LaunchArgs& la);

}  // namespace pa
