// pa_select.cu -- pa_select_tokens: which tokens of a sequence stay within its budget, for
// each kv head.
//
// The threshold is the k-th largest of the scores between the first and the last tokens, by
// radix selection: scores become unsigned keys of the same order, and three histograms of
// 11, 11 and 10 bits (2048 bins in shared memory) fix the key digit by digit.  Then each
// thread takes a run of successive tokens, two prefix sums (of keys equal to the threshold,
// lowest positions first, then of the tokens that stay) give every run its place, and the
// positions come out ascending.  Everything is whole numbers: no order of atomics shows.
//
// One cluster of 1, 2, 4 or 8 CTAs works on a (sequence, kv head), each on a part of the tokens whose
// keys it keeps in shared memory; the CTAs read each other's histograms there.  Little is read
// (four bytes a token) and what bounds the call is the chain of dependent steps, so few steps
// and short ones are what counts (GPU time, 4 kv heads: 32 x 4096 6.5 us, 4 x 100000 16.7).
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <atomic>

#include "pa_cache.h"
#include "pa_host.cuh"
#include "pa_ptx.cuh"

namespace cg = cooperative_groups;

namespace {

constexpr int kBS = PA_BLOCK_SIZE;
constexpr int kThreads = 1024;
constexpr int kBins = 2048;
constexpr int kQuads = 4;       // 16-byte loads of a thread in flight
constexpr uint32_t kStays = 0xffffffffu;  // the key of a token that stays whatever its score: above every score's
constexpr int kCached = 40960;  // keys that a CTA keeps (160 KB); longer parts are read again at every step

struct SelectParams {
    int32_t* kept;
    int32_t* new_seq_lens;
    const float* scores;
    const int32_t* block_tables;
    const int32_t* seq_lens;
    const int32_t* budgets;
    int32_t* dev_error;
    int num_seqs, num_kv_heads, num_blocks, max_seq_len, max_blocks_per_seq, max_budget, sink, recent;
};

// Order of the scores as unsigned numbers; NaN below everything, zeros of both signs the same.
__device__ __forceinline__ uint32_t key_of(float x) {
    if (x != x) return 0;
    const uint32_t u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Sum of v over the threads before this one, and over all of them.  (Two calls in a row take different `warps`, so
// one barrier is enough: no thread writes to one that another still reads.)
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* warps, uint32_t& total) {
    static_assert(kThreads == 1024, "a lane for each warp");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto warp_scan = [&](uint32_t x) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        return x;
    };
    const uint32_t x = warp_scan(v);
    if (lane == 31) warps[warp] = x;
    __syncthreads();
    const uint32_t w = warp_scan(warps[lane]);
    total = __shfl_sync(0xffffffffu, w, 31);
    const uint32_t before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
    return (warp > 0 ? before : 0) + x - v;
}

template <bool CACHED, int RANKS>
__global__ void __launch_bounds__(kThreads) pa_select_kernel(const SelectParams p) {
    extern __shared__ __align__(16) uint32_t keys[];
    __shared__ __align__(16) uint32_t hist[3][kBins];
    __shared__ uint32_t warps[2][kThreads / 32];
    __shared__ uint32_t found[3][2];  // digit of the threshold, how many above it
    __shared__ uint2 counts;          // this CTA's tokens that stay for sure, and those at the threshold
    cg::cluster_group cluster = cg::this_cluster();
    constexpr int ranks = RANKS;
    const int tid = threadIdx.x, rank = RANKS == 1 ? 0 : cluster.block_rank();
    auto sync_all = [&]() {
        if constexpr (RANKS == 1)
            __syncthreads();
        else
            cluster.sync();
    };
    const int unit = blockIdx.x / ranks, seq = unit / p.num_kv_heads, head = unit - seq * p.num_kv_heads;
    for (int i = tid; i < 3 * kBins; i += kThreads) hist[0][i] = 0;
    pa::pdl_launch_dependents();
    pa::pdl_wait_primary();
    int n = p.seq_lens[seq], budget = p.budgets[seq];
    {
        const int n0 = n, b0 = budget;
        n = min(max(n, 0), p.max_seq_len);
        budget = min(max(budget, 0), p.max_budget);
        if ((n != n0 || budget != b0) && tid == 0 && rank == 0 && head == 0 && p.dev_error)
            atomicOr(p.dev_error, PA_DEVERR_SEQ_LEN);
    }
    if (tid == 0 && rank == 0 && head == 0) p.new_seq_lens[seq] = min(n, budget);
    int32_t* kept = p.kept + (int64_t)unit * p.max_budget;
    if (n <= budget) {
        for (int i = rank * kThreads + tid; i < n; i += ranks * kThreads) kept[i] = i;
        return;  // (every CTA of the cluster)
    }
    const int recent = min(p.recent, budget), sink = min(p.sink, budget - recent);
    const int lo = sink, hi = n - recent;  // tokens that their scores decide on
    uint32_t left = (uint32_t)(budget - recent - sink);
    // this CTA's tokens, whole pages
    const int pages = (n + kBS - 1) / kBS, per = (pages + ranks - 1) / ranks;
    const int t0 = min(rank * per * kBS, n), t1 = min((rank + 1) * per * kBS, n), mine = t1 - t0;
    const int32_t* table = p.block_tables + (int64_t)seq * p.max_blocks_per_seq;
    auto read = [&](int t) -> uint32_t {
        const int blk = table[t / kBS];
        if ((unsigned)blk >= (unsigned)p.num_blocks) {
            if (p.dev_error) atomicOr(p.dev_error, PA_DEVERR_BLOCK_ID);
            return 0;
        }
        return key_of(p.scores[((int64_t)blk * p.num_kv_heads + head) * kBS + t % kBS]);
    };
    __syncthreads();  // histograms zeroed
    if (CACHED && left > 0) {
        // the keys, four of a page at a time: the loads of a thread do not wait for each other
        const int quads = (mine + kBS - 1) / kBS * 4;
        for (int i0 = 0; i0 < quads; i0 += kQuads * kThreads) {
            int blk[kQuads];
            float4 x[kQuads];
#pragma unroll
            for (int k = 0; k < kQuads; ++k) {
                const int i = i0 + k * kThreads + tid;
                blk[k] = i < quads ? table[t0 / kBS + i / 4] : 0;
            }
#pragma unroll
            for (int k = 0; k < kQuads; ++k) {
                const int i = i0 + k * kThreads + tid;
                x[k] = make_float4(NAN, NAN, NAN, NAN);
                if (i >= quads) continue;
                if ((unsigned)blk[k] < (unsigned)p.num_blocks)
                    x[k] = *reinterpret_cast<const float4*>(p.scores + ((int64_t)blk[k] * p.num_kv_heads + head) * kBS + i % 4 * 4);
                else if (p.dev_error)
                    atomicOr(p.dev_error, PA_DEVERR_BLOCK_ID);
            }
#pragma unroll
            for (int k = 0; k < kQuads; ++k) {
                const int i = i0 + k * kThreads + tid;
                if (i >= quads) continue;
                uint32_t y[4] = {key_of(x[k].x), key_of(x[k].y), key_of(x[k].z), key_of(x[k].w)};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = t0 + 4 * i + e;
                    if (t >= lo && t < hi)
                        atomicAdd(&hist[0][y[e] >> 21], 1u);
                    else
                        y[e] = kStays;
                }
                *reinterpret_cast<uint4*>(keys + 4 * i) = make_uint4(y[0], y[1], y[2], y[3]);
            }
        }
    }

    uint32_t prefix = 0;  // digits of the threshold that are known, at their places
    if (left > 0) {
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
            const uint32_t known = pass == 0 ? 0 : (pass == 1 ? 0xffe00000u : 0xfffffc00u);
            const uint32_t digits = pass == 2 ? 0x3ffu : 0x7ffu;
            auto add = [&](uint32_t k) {
                if ((k & known) == prefix) atomicAdd(&hist[pass][k >> shift & digits], 1u);
            };
            if constexpr (CACHED) {
                if (pass > 0) {  // (kStays: no score has its first digit)
#pragma unroll 2
                    for (int i = tid; i < (mine + 3) / 4; i += kThreads) {
                        const uint4 v = *reinterpret_cast<const uint4*>(keys + 4 * i);
                        add(v.x);
                        add(v.y);
                        add(v.z);
                        add(v.w);
                    }
                }
            } else {
#pragma unroll 4
                for (int i = max(lo - t0, 0) + tid; i < min(mine, hi - t0); i += kThreads) add(read(t0 + i));
            }
            sync_all();
            // every CTA adds up all histograms: two bins a thread, the highest first
            static_assert(kBins == 2 * kThreads, "two bins a thread");
            uint32_t c[2] = {0, 0}, total;
            const int bin0 = kBins - 2 - 2 * tid;
#pragma unroll
            for (int r = 0; r < ranks; ++r) {
                const uint32_t* at = &hist[pass][bin0];
                const uint2 h = *reinterpret_cast<const uint2*>(RANKS == 1 ? at : cluster.map_shared_rank(at, r));
                c[0] += h.y;
                c[1] += h.x;
            }
            uint32_t above = block_scan(c[0] + c[1], warps[0], total);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (above < left && left <= above + c[i]) {
                    found[pass][0] = (uint32_t)(bin0 + 1 - i);
                    found[pass][1] = above;
                }
                above += c[i];
            }
            __syncthreads();
            prefix |= found[pass][0] << shift;
            left -= found[pass][1];
        }
    }
    // Each thread takes `run` successive tokens of every round of the CTA's: bits of those that stay whatever the
    // ties, and of those at the threshold.  (run: 4, 12, 20 or 28, so that the 16-byte reads of eight lanes lie in
    // all banks.)
    const bool any = budget - recent - sink > 0;
    int run = (mine + kThreads - 1) / kThreads;
    run = run > 20 ? 28 : (run > 12 ? 20 : (run > 4 ? 12 : 4));
    const int rounds = (mine + run * kThreads - 1) / (run * kThreads);
    auto look = [&](int round, uint32_t& sure, uint32_t& ties) {
        const int a = (round * kThreads + tid) * run, count = min(run, mine - a);
        sure = ties = 0;
        if (count <= 0) return;
        if (CACHED && any) {
            for (int i = run - 4; i >= 0; i -= 4) {
                if (i >= count) continue;
                const uint4 v = *reinterpret_cast<const uint4*>(keys + a + i);
                const uint32_t k[4] = {v.x, v.y, v.z, v.w};
                sure <<= 4;
                ties <<= 4;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (k[e] > prefix) sure |= 1u << e;
                    if (k[e] == prefix) ties |= 1u << e;
                }
            }
            sure &= (1u << count) - 1;  // (behind the end: kStays)
            return;
        }
        for (int i = 0; i < count; ++i) {
            const int t = t0 + a + i;
            if (t < lo || t >= hi) {
                sure |= 1u << i;
            } else if (any) {
                const uint32_t k = read(t);
                sure |= (uint32_t)(k > prefix) << i;
                ties |= (uint32_t)(k == prefix) << i;
            }
        }
    };
    // Both counts in one scan: 28 tokens of 1024 threads are less than 2^16.
    static_assert(28 * kThreads < 65536, "two counts to a word");
    uint32_t sure = 0, ties = 0, before = 0, all = 0;
    int turn = 0;
    auto count = [&](int round) {
        look(round, sure, ties);
        turn ^= 1;
        before = block_scan(__popc(ties) << 16 | __popc(sure), warps[turn], all);
    };
    uint32_t place = 0, at_threshold = 0;  // tokens that stay, and ties, of the CTAs before this one, then of this one's rounds
    auto taken = [&](uint32_t n) { return at_threshold < left ? min(n, left - at_threshold) : 0u; };  // of the next n ties
    if constexpr (RANKS > 1) {
        uint32_t all_sure = 0, all_ties = 0;
        for (int round = 0; round < rounds; ++round) {
            count(round);
            all_sure += all & 0xffffu;
            all_ties += all >> 16;
        }
        if (tid == 0) counts = make_uint2(all_sure, all_ties);
        cluster.sync();
        uint2 c[RANKS];
#pragma unroll
        for (int r = 0; r < RANKS; ++r) c[r] = *cluster.map_shared_rank(&counts, r);
#pragma unroll
        for (int r = 0; r < RANKS; ++r) {
            if (r >= rank) continue;
            place += c[r].x + taken(c[r].y);
            at_threshold += c[r].y;
        }
    }
    for (int round = 0; round < rounds; ++round) {
        if (RANKS == 1 || rounds > 1) count(round);
        const uint32_t ties_before = before >> 16, mine_taken = taken(ties_before + __popc(ties)) - taken(ties_before);
        for (uint32_t n = mine_taken; n > 0; --n) {  // the lowest ones
            sure |= ties & (0u - ties);
            ties &= ties - 1;
        }
        int32_t* to = kept + place + (before & 0xffffu) + taken(ties_before);
        const int a = t0 + (round * kThreads + tid) * run;
        for (; sure; sure &= sure - 1) *to++ = a + __ffs(sure) - 1;
        place += (all & 0xffffu) + taken(all >> 16);
        at_threshold += all >> 16;
    }
    if constexpr (RANKS > 1) cluster.sync();  // the counts are read by the others
}

template <bool CACHED, int RANKS>
bool launch(const SelectParams& p, size_t smem, void* stream) {
    auto kern = pa_select_kernel<CACHED, RANKS>;
    if (smem > 16 * 1024) {
        static std::atomic<int> ready[pa::kHostDevices];
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return false;
        if (dev >= pa::kHostDevices || !ready[dev].load()) {
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kCached * 4) != cudaSuccess) return false;
            if (dev < pa::kHostDevices) ready[dev].store(1);
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)p.num_seqs * p.num_kv_heads * RANKS));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = RANKS;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = RANKS > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess;
}

}  // namespace

extern "C" pa_status pa_select_tokens(const pa_select_args* a, void* stream) {
    if (!a) return PA_ERR_INVALID_ARG;
    if (a->num_seqs < 0 || a->num_kv_heads <= 0 || a->num_blocks <= 0 || a->max_seq_len < 0 || a->max_blocks_per_seq < 0 ||
        a->max_budget < 0 || a->sink < 0 || a->recent < 0)
        return PA_ERR_INVALID_ARG;
    if (a->block_size != PA_BLOCK_SIZE || a->max_seq_len > 1 << 30 || a->max_budget > 1 << 30) return PA_ERR_UNSUPPORTED;
    if ((int64_t)a->num_seqs * a->num_kv_heads * 8 > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
    if (a->num_seqs == 0) return PA_OK;
    if ((!a->kept && a->max_budget > 0) || !a->new_seq_lens || !a->scores || !a->block_tables || !a->seq_lens || !a->budgets)
        return PA_ERR_INVALID_ARG;
    if (a->new_seq_lens == a->seq_lens) return PA_ERR_INVALID_ARG;  // read by CTAs that start later
    if ((int64_t)a->max_blocks_per_seq * PA_BLOCK_SIZE < a->max_seq_len) return PA_ERR_INVALID_ARG;
    if (!pa::aligned(a->kept, 4) || !pa::aligned(a->new_seq_lens, 4) || !pa::aligned(a->scores, 16) ||
        !pa::aligned(a->block_tables, 4) || !pa::aligned(a->seq_lens, 4) || !pa::aligned(a->budgets, 4) ||
        !pa::aligned(a->dev_error, 4))
        return PA_ERR_INVALID_ARG;
    SelectParams p = {};
    p.kept = a->kept;
    p.new_seq_lens = a->new_seq_lens;
    p.scores = a->scores;
    p.block_tables = a->block_tables;
    p.seq_lens = a->seq_lens;
    p.budgets = a->budgets;
    p.dev_error = a->dev_error;
    p.num_seqs = a->num_seqs;
    p.num_kv_heads = a->num_kv_heads;
    p.num_blocks = a->num_blocks;
    p.max_seq_len = a->max_seq_len;
    p.max_blocks_per_seq = a->max_blocks_per_seq;
    p.max_budget = a->max_budget;
    p.sink = a->sink;
    p.recent = a->recent;
    int dev = 0, sms = 0;
    if (!pa::device_and_sms(&dev, &sms)) return PA_ERR_LAUNCH;
    // CTAs of a cluster: more while each has over 4096 tokens and all of them take at most half of the SMs (a cluster
    // of eight wants eight free SMs of one part of the GPU: sixteen such clusters ran one after the other,
    // 4 x 100000 36 us, in clusters of four 19)
    const int64_t units = (int64_t)a->num_seqs * a->num_kv_heads;
    int ranks = 1;
    while (ranks < 8 && a->max_seq_len > 4096 * ranks && units * ranks * 4 <= sms) ranks *= 2;
    while (ranks < 8 && (a->max_seq_len + ranks - 1) / ranks + PA_BLOCK_SIZE > kCached) ranks *= 2;
    const int64_t pages = (a->max_seq_len + PA_BLOCK_SIZE - 1) / PA_BLOCK_SIZE, part = (pages + ranks - 1) / ranks * PA_BLOCK_SIZE;
    const size_t smem = (size_t)part * 4;
    const bool ok = part > kCached ? launch<false, 8>(p, 0, stream)
                    : ranks == 1   ? launch<true, 1>(p, smem, stream)
                    : ranks == 2   ? launch<true, 2>(p, smem, stream)
                    : ranks == 4   ? launch<true, 4>(p, smem, stream)
                                   : launch<true, 8>(p, smem, stream);
    return ok ? PA_OK : PA_ERR_LAUNCH;
}
