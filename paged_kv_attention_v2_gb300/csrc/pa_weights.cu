// pa_weights.cu -- pa_add_weights (pa_weights.cuh): argument checks, tiles, launch; the
// fp32 kernels.
#include <algorithm>
#include <cmath>

#include "pa_weights.cuh"

namespace pa {
bool launch_weights_f32(WeightParams& p, int head_size, int sms, void* stream) {
    return launch_weights<float, kWSame>(p, head_size, sms, stream);
}
}  // namespace pa

extern "C" pa_status pa_add_weights(const pa_weights_args* a, void* stream) {
    if (!a) return PA_ERR_INVALID_ARG;
    if (a->num_seqs < 0 || a->num_heads <= 0 || a->num_kv_heads <= 0 || a->num_blocks <= 0 || a->max_seq_len < 0 ||
        a->max_blocks_per_seq < 0 || a->num_heads % a->num_kv_heads != 0)
        return PA_ERR_INVALID_ARG;
    if (a->dtype != PA_DTYPE_F32 && a->dtype != PA_DTYPE_F16 && a->dtype != PA_DTYPE_BF16) return PA_ERR_INVALID_ARG;
    if (a->layout != PA_LAYOUT_SPLIT && a->layout != PA_LAYOUT_NHD) return PA_ERR_INVALID_ARG;
    const int kv = a->kv_dtype;
    if (kv != PA_KV_SAME && kv != PA_KV_FP8_E4M3 && kv != PA_KV_FP8_E5M2 && kv != PA_KV_FP4_E2M1) return PA_ERR_INVALID_ARG;
    if (!std::isfinite(a->scale) || !std::isfinite(a->softcap) || !std::isfinite(a->k_scale) || !std::isfinite(a->decay) ||
        a->decay < 0.f)
        return PA_ERR_INVALID_ARG;
    if (kv != PA_KV_SAME && a->dtype == PA_DTYPE_F32) return PA_ERR_UNSUPPORTED;
    if (kv == PA_KV_FP4_E2M1 && a->layout != PA_LAYOUT_NHD) return PA_ERR_UNSUPPORTED;
    if (a->block_size != PA_BLOCK_SIZE || (a->head_size != 64 && a->head_size != 128)) return PA_ERR_UNSUPPORTED;
    const int group = a->num_heads / a->num_kv_heads;
    const bool multi = a->query_start != nullptr;
    const int most = multi ? a->max_query_len : 1;
    if (multi && (a->max_query_len < 1 || a->num_query_tokens < 0 || !pa::aligned(a->query_start, 4))) return PA_ERR_INVALID_ARG;
    if ((int64_t)most * group > 16) return PA_ERR_UNSUPPORTED;
    if (a->max_seq_len > 1 << 30) return PA_ERR_UNSUPPORTED;  // positions past a tile's end in 32 bits
    if (a->num_seqs == 0 || a->max_seq_len == 0) return PA_OK;
    if (!a->scores || !a->query || !a->key_cache || !a->block_tables || !a->seq_lens || !a->exp_sums || !a->max_logits)
        return PA_ERR_INVALID_ARG;
    if ((int64_t)a->max_blocks_per_seq * PA_BLOCK_SIZE < a->max_seq_len) return PA_ERR_INVALID_ARG;
    if (!pa::aligned(a->query, 16) || !pa::aligned(a->key_cache, 16) || !pa::aligned(a->scores, 4) ||
        !pa::aligned(a->block_tables, 4) || !pa::aligned(a->seq_lens, 4) || !pa::aligned(a->exp_sums, 4) ||
        !pa::aligned(a->max_logits, 4) || !pa::aligned(a->alibi_slopes, 4) || !pa::aligned(a->dev_error, 4))
        return PA_ERR_INVALID_ARG;
    int dev = 0, sms = 0;
    if (!pa::device_and_sms(&dev, &sms)) return PA_ERR_LAUNCH;

    pa::WeightParams p = {};
    p.scores = a->scores;
    p.query = a->query;
    p.key_cache = a->key_cache;
    p.block_tables = a->block_tables;
    p.seq_lens = a->seq_lens;
    p.query_start = a->query_start;
    p.exp_sums = a->exp_sums;
    p.max_logits = a->max_logits;
    p.alibi = a->alibi_slopes;
    p.relative_max = a->relative_max != 0;
    p.dev_error = a->dev_error;
    p.num_seqs = a->num_seqs;
    p.num_heads = a->num_heads;
    p.num_kv_heads = a->num_kv_heads;
    p.group = group;
    p.num_blocks = a->num_blocks;
    p.max_blocks_per_seq = a->max_blocks_per_seq;
    p.max_seq_len = a->max_seq_len;
    p.max_parts = pa_max_num_partitions(a->max_seq_len);
    p.max_q_len = most;
    p.num_q_rows = multi ? a->num_query_tokens : a->num_seqs;
    // (a window over any length is one of max_seq_len: positions minus the window stay in 32 bits)
    p.window_left = a->sliding_window > 0 ? std::min(a->sliding_window - 1, a->max_seq_len) : -1;
    p.scale = a->scale * (kv != PA_KV_SAME && a->k_scale > 0.f ? a->k_scale : 1.f);
    p.softcap = a->softcap > 0.f ? a->softcap : 0.f;
    p.inv_softcap = a->softcap > 0.f ? 1.f / a->softcap : 0.f;
    p.decay = a->decay;
    const int64_t block_bytes = (int64_t)a->num_kv_heads * a->head_size *
                                (kv == PA_KV_FP4_E2M1 ? 9 : PA_BLOCK_SIZE * (kv != PA_KV_SAME ? 1 : (a->dtype == PA_DTYPE_F32 ? 4 : 2)));
    if (block_bytes > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
    p.block_bytes = (uint32_t)block_bytes;
    const int elem = kv != PA_KV_SAME ? 1 : (a->dtype == PA_DTYPE_F32 ? 4 : 2);
    p.token_step = a->layout == PA_LAYOUT_NHD ? a->head_size * elem : 16;
    p.piece_step = a->layout == PA_LAYOUT_NHD ? 16 : 16 * PA_BLOCK_SIZE;
    // (grid: the CTAs that fit on the GPU once, or for larger batches at most 1 + max_seq_len / 2048 tiles, twice that with rounding, a head)
    if ((int64_t)a->num_seqs * a->num_kv_heads > 0x7fffffffLL / (1 + (a->max_seq_len >> 11)) / 2) return PA_ERR_UNSUPPORTED;
    const int kvk = kv == PA_KV_SAME ? pa::kWSame : kv == PA_KV_FP8_E4M3 ? pa::kWE4M3 : kv == PA_KV_FP8_E5M2 ? pa::kWE5M2 : pa::kWE2M1;
    const bool ok = a->dtype == PA_DTYPE_F32   ? pa::launch_weights_f32(p, a->head_size, sms, stream)
                    : a->dtype == PA_DTYPE_F16 ? pa::launch_weights_f16(p, a->head_size, kvk, sms, stream)
                                               : pa::launch_weights_bf16(p, a->head_size, kvk, sms, stream);
    return ok ? PA_OK : PA_ERR_LAUNCH;
}
