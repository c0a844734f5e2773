// pa_tables.cu -- pa_build_tables: pages handed out to the sequences of a step
// and the step's slot map, on the GPU.
//
// For sequence s: own = ceil(len / 16) pages before, want = ceil((keep + n) / 16)
// after, pops = max(want - own, 0), pushes = max(own - want, 0).  The exclusive
// sums of pops and pushes over the sequences say which entries of the ring of
// free pages each sequence takes and fills; everything else is one lookup per
// token.  No arithmetic to speak of: the call is bound by its launch and by a
// chain of dependent loads (lengths, scan, ring, table), so it is ONE kernel, in
// which every CTA computes the sums of the whole batch for itself (lengths come
// from L2) and then fills its share of the rows.  The new lengths and the new
// pool state may overwrite the old ones, which other CTAs still read: the last
// CTA to finish writes them.  Measured, back to back on the GPU: 32 sequences of
// one token 4.2 us, 256 with drafts cut and sequences ended 6.7, 128 prompts of
// 16384 tokens (2.1 M rows, 17 MB written: 2.6 us at the copy rate) 8.5; sums by a
// kernel of their own would add a launch and a workspace to each.
#include <cuda_runtime.h>

#include <atomic>

#include "pa_cache.h"
#include "pa_host.cuh"
#include "pa_ptx.cuh"

namespace {

constexpr int kBS = PA_BLOCK_SIZE;
constexpr int kItems = 4;        // sequences per thread and chunk
constexpr int kMaxThreads = 1024;
constexpr int kRowsPerThread = 4;

struct TablesParams {
    int32_t* block_tables;
    const int32_t* seq_lens;
    const int32_t* keep_lens;
    const int32_t* query_start;
    int32_t* free_ring;
    const int32_t* pool_state;
    int32_t* slots;
    int32_t* positions;
    int32_t* new_seq_lens;
    int32_t* new_pool_state;
    int32_t* dev_error;
    int32_t* done_counter;
    int num_seqs, num_tokens, num_blocks, max_seq_len, max_blocks_per_seq;
    int vec;  // slots and positions 16-byte aligned
};

struct Seq {
    int keep, start, n, own, want;  // tokens kept, first row, new tokens, pages before and after
    bool bad;
};

__device__ __forceinline__ Seq load_seq(const TablesParams& p, int s) {
    Seq q;
    const int len = p.seq_lens[s];
    q.keep = p.keep_lens ? p.keep_lens[s] : len;
    const int end = p.query_start ? p.query_start[s + 1] : s + 1;
    q.start = p.query_start ? p.query_start[s] : s;
    q.bad = len < 0 || len > p.max_seq_len || q.keep < 0 || q.keep > len || q.start < 0 || end < q.start ||
            end > p.num_tokens || (s == 0 && q.start != 0) || end - q.start > p.max_seq_len - q.keep;
    q.n = end - q.start;
    if (q.bad) {
        q.keep = q.n = q.own = q.want = 0;
    } else {
        q.own = (int)(((int64_t)len + kBS - 1) / kBS);
        q.want = (int)(((int64_t)q.keep + q.n + kBS - 1) / kBS);
    }
    return q;
}

// Exclusive block-wide sum of v (two 32-bit counts side by side); *total gets
// the sum.  Every thread of the block calls it.
__device__ uint64_t block_scan(uint64_t v, uint64_t* total) {
    __shared__ uint64_t warp_sum[kMaxThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    uint64_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    __syncthreads();  // the last call's sums have been read
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    uint64_t w = lane < warps ? warp_sum[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t x = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += x;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    const uint64_t before = __shfl_sync(0xffffffffu, w, warp == 0 ? 0 : warp - 1);
    return (warp == 0 ? 0 : before) + incl - v;
}

// Last i of [0, n) with a[i] <= x (a rises, a[0] <= x).
__device__ __forceinline__ int last_at_most(const int* a, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kMaxThreads) pa_tables_kernel(const TablesParams p) {
    extern __shared__ int sm[];
    const int chunk = kItems * (int)blockDim.x;
    // of the chunk's sequences: first row, tokens kept, pages before, pages
    // after, ring entries taken / filled before it
    int* start = sm;
    int* keep = start + chunk + 4;  // start[n]: the row behind the chunk's last
    int* own = keep + chunk;
    int* want = own + chunk;
    int* pop0 = want + chunk;
    int* push0 = pop0 + chunk;
    const int tid = threadIdx.x, S = p.num_seqs;

    pa::pdl_launch_dependents();
    pa::pdl_wait_primary();

    // head and count of the pool as they were
    const int head = p.pool_state[0], count = p.pool_state[1], N = p.num_blocks;

    // The sums of a chunk of sequences from `base` on, added to `carry`
    // (pops in the upper half, pushes in the lower); fills the shared arrays.
    auto sum_chunk = [&](int base, uint64_t carry, bool& bad) {
        Seq q[kItems];
        uint64_t mine = 0;
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int s = base + tid * kItems + i;
            if (s < S) {
                q[i] = load_seq(p, s);
                bad |= q[i].bad;
                const int d = q[i].want - q[i].own;
                mine += d > 0 ? (uint64_t)d << 32 : (uint64_t)(-d);
            }
        }
        uint64_t total;
        uint64_t at = carry + block_scan(mine, &total);
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int s = base + tid * kItems + i, j = tid * kItems + i;
            if (s < S) {
                start[j] = q[i].start;
                keep[j] = q[i].keep;
                own[j] = q[i].own;
                want[j] = q[i].want;
                pop0[j] = (int)(at >> 32);
                push0[j] = (int)(at & 0xffffffffu);
                const int d = q[i].want - q[i].own;
                at += d > 0 ? (uint64_t)d << 32 : (uint64_t)(-d);
                if (s == S - 1 || j == chunk - 1) start[j + 1] = q[i].start + q[i].n;
            }
        }
        return carry + total;
    };

    // whole batch: is the step possible?  (One chunk: its arrays stay.)
    bool bad = false;
    uint64_t totals = 0;
    for (int base = 0; base < S; base += chunk) totals = sum_chunk(base, totals, bad);
    bad = __syncthreads_or(bad);
    const int64_t pops = (int64_t)(totals >> 32), pushes = (int64_t)(totals & 0xffffffffu);
    const bool short_pool =
        head < 0 || head >= N || count < 0 || count > N || pops > count || (int64_t)count + pushes > N;
    const bool ok = !bad && !short_pool;
    if (!ok && blockIdx.x == 0 && tid == 0 && p.dev_error)
        atomicOr(p.dev_error, bad ? PA_DEVERR_SEQ_LEN : PA_DEVERR_POOL);

    const bool one_chunk = S <= chunk;
    const int rows = !ok || S == 0 ? 0 : (one_chunk ? start[S] : (p.query_start ? p.query_start[S] : S));  // with a token
    // this CTA's rows: successive ones, so that a thread's next four are mostly
    // of the same sequence or the next
    const int64_t share = ((int64_t)p.num_tokens / kRowsPerThread / gridDim.x + 1) * kRowsPerThread;
    const int64_t first = blockIdx.x * share + tid * kRowsPerThread, end = (blockIdx.x + 1) * share;
    const int step = (int)blockDim.x * kRowsPerThread;

    if (ok) {
        bool bad_id = false;
        uint64_t carry = 0;
        for (int base = 0; base < S; base += chunk) {
            const int n = min(chunk, S - base);
            if (!one_chunk) {  // a further chunk: its sums again
                bool ignored = false;
                __syncthreads();
                carry = sum_chunk(base, carry, ignored);
                __syncthreads();
            }
            const int row0 = start[0];
            const int row1 = start[n];
            // rows [row0, row1): four successive rows per thread
            int j = 0;  // the sequence of the row at hand, within the chunk
            auto page_id = [&](int page, bool first_token) {
                int32_t* entry = p.block_tables + (base + j) * p.max_blocks_per_seq + page;  // below 2^31 entries
                if (page < own[j]) return *entry;
                uint32_t k = (uint32_t)head + (uint32_t)(pop0[j] + page - own[j]);  // both below 2^27
                if (k >= (uint32_t)N) k -= N;
                const int id = p.free_ring[k];
                if (first_token) *entry = id;  // of a new page: always one of this call's
                return id;
            };
            auto slot_at = [&](int id, int off) {
                if ((unsigned)id < (unsigned)N) return id * kBS + off;
                bad_id = true;
                return -1;
            };
            for (int64_t q = first; q < end && q < row1; q += step) {
                if (q + kRowsPerThread <= row0) continue;
                const int t = max((int)q, row0);
                if (!p.query_start)
                    j = t - base;
                else if (start[j + 1] <= t)
                    j += last_at_most(start + j, n - j, t);
                if (p.vec && t == q && t + kRowsPerThread <= start[j + 1]) {  // four tokens of one sequence
                    const int pos = keep[j] + t - start[j], page = pos >> 4, off = pos & 15;
                    const int id = page_id(page, off == 0);
                    const int next = off > kBS - kRowsPerThread ? page_id(page + 1, true) : id;
                    int slot[kRowsPerThread];
#pragma unroll
                    for (int i = 0; i < kRowsPerThread; ++i)
                        slot[i] = off + i < kBS ? slot_at(id, off + i) : slot_at(next, off + i - kBS);
                    *reinterpret_cast<int4*>(p.slots + t) = make_int4(slot[0], slot[1], slot[2], slot[3]);
                    if (p.positions)
                        *reinterpret_cast<int4*>(p.positions + t) = make_int4(pos, pos + 1, pos + 2, pos + 3);
                    continue;
                }
                for (int r = t; r < q + kRowsPerThread && r < row1; ++r) {
                    while (start[j + 1] <= r) ++j;  // ends: start[n] = row1
                    const int pos = keep[j] + r - start[j], off = pos & 15;
                    p.slots[r] = slot_at(page_id(pos >> 4, off == 0), off);
                    if (p.positions) p.positions[r] = pos;
                }
            }
            // pages put back by the chunk's sequences: one entry per thread
            const int last = n - 1;
            const int back0 = push0[0], back1 = push0[last] + max(own[last] - want[last], 0);
            for (int64_t k = back0 + (int64_t)blockIdx.x * blockDim.x + tid; k < back1;
                 k += (int64_t)gridDim.x * blockDim.x) {
                const int j = last_at_most(push0, n, (int)k);
                const int64_t at = ((int64_t)head + count + k) % N;
                p.free_ring[at] = p.block_tables[(int64_t)(base + j) * p.max_blocks_per_seq + want[j] +
                                                 ((int)k - push0[j])];
            }
        }
        if (bad_id && p.dev_error) atomicOr(p.dev_error, PA_DEVERR_BLOCK_ID);
    }
    // padding
    for (int64_t t = rows + (int64_t)blockIdx.x * blockDim.x + tid; t < p.num_tokens;
         t += (int64_t)gridDim.x * blockDim.x) {
        p.slots[t] = -1;
        if (p.positions) p.positions[t] = 0;
    }

    // new lengths and pool state, once every CTA has read the old ones
    bool writes = true;
    if (gridDim.x > 1) {
        __syncthreads();  // this CTA's reads are done
        bool last = false;
        if (tid == 0) {
            last = pa::atom_add_acq_rel_gpu(p.done_counter, 1) == (int)gridDim.x - 1;
            if (last) *p.done_counter = 0;
        }
        writes = __syncthreads_or(last) != 0;
    }
    if (!writes) return;
    for (int s = tid; s < S; s += blockDim.x) {
        if (ok && one_chunk) {
            p.new_seq_lens[s] = keep[s] + start[s + 1] - start[s];
        } else {
            const int len = p.seq_lens[s];
            int now = len;
            if (ok) {
                const int kept = p.keep_lens ? p.keep_lens[s] : len;
                now = kept + (p.query_start ? p.query_start[s + 1] - p.query_start[s] : 1);
            }
            p.new_seq_lens[s] = now;
        }
    }
    if (tid == 0) {
        p.new_pool_state[0] = ok ? (int)(((int64_t)head + pops) % N) : head;
        p.new_pool_state[1] = ok ? (int)(count - pops + pushes) : count;
    }
}

}  // namespace

extern "C" pa_status pa_build_tables(const pa_tables_args* a, void* stream) {
    if (!a) return PA_ERR_INVALID_ARG;
    if (a->num_seqs < 0 || a->num_tokens < 0 || a->num_blocks <= 0 || a->max_seq_len < 0 ||
        a->max_blocks_per_seq < 0)
        return PA_ERR_INVALID_ARG;
    if (a->block_size != PA_BLOCK_SIZE) return PA_ERR_UNSUPPORTED;
    if (a->num_blocks >= 1 << 27) return PA_ERR_UNSUPPORTED;
    // rows and sequences counted past their end, by a thread's step, in 32 bits
    if (a->num_tokens > 1 << 30 || a->num_seqs > 1 << 30) return PA_ERR_UNSUPPORTED;
    if ((int64_t)a->num_seqs * a->max_blocks_per_seq >= (int64_t)1 << 31) return PA_ERR_UNSUPPORTED;
    if ((int64_t)a->max_blocks_per_seq * PA_BLOCK_SIZE < (int64_t)a->max_seq_len) return PA_ERR_INVALID_ARG;
    if (!a->query_start && a->num_tokens < a->num_seqs) return PA_ERR_INVALID_ARG;
    if (!a->free_ring || !a->pool_state || !a->new_pool_state) return PA_ERR_INVALID_ARG;
    if (a->num_seqs > 0 && (!a->block_tables || !a->seq_lens || !a->new_seq_lens)) return PA_ERR_INVALID_ARG;
    if (a->num_tokens > 0 && !a->slots) return PA_ERR_INVALID_ARG;
    const void* all[] = {a->block_tables, a->seq_lens, a->keep_lens, a->query_start, a->free_ring,
                         a->pool_state, a->slots, a->positions, a->new_seq_lens, a->new_pool_state,
                         a->dev_error, a->done_counter};
    for (const void* ptr : all)
        if (!pa::aligned(ptr, 4)) return PA_ERR_INVALID_ARG;

    TablesParams p = {};
    p.block_tables = a->block_tables;
    p.seq_lens = a->seq_lens;
    p.keep_lens = a->keep_lens;
    p.query_start = a->query_start;
    p.free_ring = a->free_ring;
    p.pool_state = a->pool_state;
    p.slots = a->slots;
    p.positions = a->positions;
    p.new_seq_lens = a->new_seq_lens;
    p.new_pool_state = a->new_pool_state;
    p.dev_error = a->dev_error;
    p.done_counter = a->done_counter;
    p.num_seqs = a->num_seqs;
    p.num_tokens = a->num_tokens;
    p.num_blocks = a->num_blocks;
    p.max_seq_len = a->max_seq_len;
    p.max_blocks_per_seq = a->max_blocks_per_seq;
    p.vec = pa::aligned(a->slots, 16) && pa::aligned(a->positions, 16) ? 1 : 0;

    int dev = 0, sm = 0;
    if (!pa::device_and_sms(&dev, &sm)) return PA_ERR_LAUNCH;
    // A small step on one small CTA (32 tokens 4.2 us; 5.0 on 1024 threads, whose
    // barriers take longer), a large one on up to one CTA of 1024 threads per SM.
    const int threads = a->num_seqs <= 1024 && a->num_tokens <= 1024 ? 256 : kMaxThreads;
    int64_t work = a->num_tokens / kRowsPerThread;
    if (a->keep_lens) work += (int64_t)a->num_seqs * a->max_blocks_per_seq / 16;  // pages may come back
    int64_t grid = (work + threads - 1) / threads;
    if (grid > sm) grid = sm;
    if (grid < 1 || !a->done_counter) grid = 1;

    const size_t smem = sizeof(int) * (6 * kItems * threads + 4);  // 96 KB at 1024 threads
    static std::atomic<int> ready[pa::kHostDevices];
    if (dev >= pa::kHostDevices || !ready[dev].load()) {
        if (cudaFuncSetAttribute(pa_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)(sizeof(int) * (6 * kItems * kMaxThreads + 4))) != cudaSuccess)
            return PA_ERR_LAUNCH;
        if (dev < pa::kHostDevices) ready[dev].store(1);
    }
    return pa::launch_pdl(pa_tables_kernel, dim3((unsigned)grid), threads, smem, stream, p) ? PA_OK : PA_ERR_LAUNCH;
}
