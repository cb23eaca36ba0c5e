// abi_shrink.cu -- the C ABI of 8-bit pools, of decode that sums its attention weights and of eviction:
// argument validation, workspace layout, dispatch.
#include <math.h>

#include "shrink.h"

namespace pkv {

cudaError_t launch_frag_q8_f16(int, int, const FragArgs&, const CUtensorMap&, const CUtensorMap&, cudaStream_t);
cudaError_t launch_frag_q8_bf16(int, int, const FragArgs&, const CUtensorMap&, const CUtensorMap&, cudaStream_t);
cudaError_t launch_frag_scored_f16(int, int, const FragArgs&, const CUtensorMap&, const CUtensorMap&, cudaStream_t);
cudaError_t launch_frag_scored_bf16(int, int, const FragArgs&, const CUtensorMap&, const CUtensorMap&, cudaStream_t);
cudaError_t launch_frag_multi_f16(int, int, const FragArgs&, const CUtensorMap&, const CUtensorMap&, cudaStream_t);
cudaError_t launch_frag_multi_bf16(int, int, const FragArgs&, const CUtensorMap&, const CUtensorMap&, cudaStream_t);
cudaError_t launch_prefill_widened_f16(int, int, const PrefillArgs&, const CUtensorMap&, const CUtensorMap&, cudaStream_t);
cudaError_t launch_prefill_widened_bf16(int, int, const PrefillArgs&, const CUtensorMap&, const CUtensorMap&, cudaStream_t);
cudaError_t frag_multi_ctas_per_sm_f16(int, int, int*);
cudaError_t frag_multi_ctas_per_sm_bf16(int, int, int*);
cudaError_t frag_ctas_per_sm_q8_f16(int, int, int*);
cudaError_t frag_ctas_per_sm_q8_bf16(int, int, int*);
cudaError_t frag_ctas_per_sm_scored_f16(int, int, int*);
cudaError_t frag_ctas_per_sm_scored_bf16(int, int, int*);

cudaError_t frag_ctas_per_sm(int dtype, bool q8, int head_dim, int group, int* out) {
    if (q8) return dtype == PKV_F16 ? frag_ctas_per_sm_q8_f16(head_dim, group, out) : frag_ctas_per_sm_q8_bf16(head_dim, group, out);
    return dtype == PKV_F16 ? frag_ctas_per_sm_scored_f16(head_dim, group, out) : frag_ctas_per_sm_scored_bf16(head_dim, group, out);
}

namespace {
cudaError_t layer_maps(const FragArgs& a, int head_dim, int type, CUtensorMap* tk, CUtensorMap* tv) {
    const long long rows = (long long)a.d.num_blocks * a.d.n_kv * kBlock;
    const cudaError_t err = kv_tensor_map(a.d.k_layer, rows, head_dim, type, PKV_BOX_PANEL, tk);
    return err != cudaSuccess ? err : kv_tensor_map(a.d.v_layer, rows, head_dim, type, PKV_BOX_PANEL, tv);
}
}  // namespace

cudaError_t launch_frag_decode(int dtype, bool q8, int head_dim, int group, const FragArgs& a, cudaStream_t stream) {
    CUtensorMap tk, tv;
    const cudaError_t err = layer_maps(a, head_dim, q8 ? kCodesE4M3 : dtype, &tk, &tv);
    if (err != cudaSuccess) return err;
    if (q8)
        return dtype == PKV_F16 ? launch_frag_q8_f16(head_dim, group, a, tk, tv, stream)
                                : launch_frag_q8_bf16(head_dim, group, a, tk, tv, stream);
    return dtype == PKV_F16 ? launch_frag_scored_f16(head_dim, group, a, tk, tv, stream)
                            : launch_frag_scored_bf16(head_dim, group, a, tk, tv, stream);
}

cudaError_t frag_multi_ctas_per_sm(int dtype, int head_dim, int columns, int* out) {
    return dtype == PKV_F16 ? frag_multi_ctas_per_sm_f16(head_dim, columns, out)
                            : frag_multi_ctas_per_sm_bf16(head_dim, columns, out);
}

cudaError_t launch_frag_multi(int dtype, int head_dim, int columns, const FragArgs& a, cudaStream_t stream) {
    CUtensorMap tk, tv;
    const cudaError_t err = layer_maps(a, head_dim, kCodesE4M3, &tk, &tv);
    if (err != cudaSuccess) return err;
    return dtype == PKV_F16 ? launch_frag_multi_f16(head_dim, columns, a, tk, tv, stream)
                            : launch_frag_multi_bf16(head_dim, columns, a, tk, tv, stream);
}

cudaError_t widened_maps(int dtype, int head_dim, const Q8WidenArgs& w, CUtensorMap* tk, CUtensorMap* tv) {
    const long long rows = (long long)w.num_blocks * w.n_kv * kBlock;
    CUtensorMap codes;  // (only asked for: the widening takes plain addresses)
    cudaError_t err = kv_tensor_map(w.k_codes, rows, head_dim, kCodesE4M3, PKV_BOX_PANEL, &codes);
    if (err == cudaSuccess) err = kv_tensor_map(w.v_codes, rows, head_dim, kCodesE4M3, PKV_BOX_PANEL, &codes);
    if (err == cudaSuccess) err = kv_tensor_map(w.k_out, rows, head_dim, dtype, PKV_BOX_PANEL, tk);
    // (at head_dim 256 each CTA of a pair copies half of a V block's columns)
    return err != cudaSuccess ? err
                              : kv_tensor_map(w.v_out, rows, head_dim, dtype,
                                              head_dim == 256 ? PKV_BOX_BLOCK_HALF : PKV_BOX_BLOCK, tv);
}

cudaError_t launch_prefill_widened(int dtype, int head_dim, int group, const PrefillArgs& a, const CUtensorMap& tk,
                                   const CUtensorMap& tv, cudaStream_t stream) {
    return dtype == PKV_F16 ? launch_prefill_widened_f16(head_dim, group, a, tk, tv, stream)
                            : launch_prefill_widened_bf16(head_dim, group, a, tk, tv, stream);
}

}  // namespace pkv

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

size_t layer_elems(const pkv_cache_desc* d) { return (size_t)d->num_blocks * d->n_kv_heads * d->block_size * d->head_dim; }
size_t layer_scales(const pkv_cache_desc* d) { return (size_t)d->num_blocks * d->n_kv_heads; }
long long pool_rows(const pkv_cache_desc* d) { return (long long)d->num_blocks * d->n_kv_heads * d->block_size; }
int group_of(const pkv_cache_desc* d) { return d->n_q_heads / d->n_kv_heads; }

// A descriptor whose activations are 16-bit.
int validate16(const pkv_cache_desc* d) {
    const int rc = pkv_validate_desc(d);
    if (rc != PKV_OK) return rc;
    return d->dtype == PKV_F32 ? PKV_ERR_UNSUPPORTED : PKV_OK;
}

// Geometry of the fragment kernel. Runs: as many CTAs as the GPU holds at once. Partitions: when every
// (sequence, KV head) pair can have its context cut into a cluster's worth of partitions of at most
// kMaxPartition blocks with no more than one CTA per SM: small calls, where latency counts (8 heads of
// 4,000 tokens: partitions 9.4 us, runs 13.8; at 64 blocks a partition four such sequences take 17.5 us
// against 14.7).
static_assert(pkv::kMaxRuns * sizeof(unsigned int) == PKV_ARRIVAL_BYTES, "one counter a run");

struct FragGeometry {
    int ctas, partition;  // CTAs along x; blocks of a partition, 0 for runs
};

FragGeometry geometry_of(long long pairs, int max_blocks, int sms, int per_sm, int max_runs) {
    FragGeometry geo;
    const long long parts = pairs >= sms ? 1 : sms / pairs < pkv::kMaxCluster ? sms / pairs : pkv::kMaxCluster;
    const int partition = (int)((max_blocks + parts - 1) / parts);
    if (pairs <= sms && partition <= pkv::kMaxPartition) {
        geo.partition = partition < pkv::kMinPartition ? pkv::kMinPartition : partition;
        geo.ctas = pkv::decode_partitions(max_blocks, geo.partition);
    } else {
        geo.partition = 0;
        geo.ctas = sms * per_sm < max_runs ? sms * per_sm : max_runs;
    }
    return geo;
}

cudaError_t frag_geometry(const pkv_cache_desc* d, bool q8, int n_seqs, int max_blocks, FragGeometry* out) {
    int sms = 0, per_sm = 0;
    cudaError_t err = pkv::current_sm_count(&sms);
    if (err == cudaSuccess) err = pkv::frag_ctas_per_sm(d->dtype, q8, d->head_dim, group_of(d), &per_sm);
    if (err != cudaSuccess) return err;
    *out = geometry_of((long long)n_seqs * d->n_kv_heads, max_blocks, sms, per_sm, pkv::kMaxRuns);
    return cudaSuccess;
}

struct FragLayout {
    size_t o, ml, row_ml, z, bytes;  // offsets; the arrival counters lie at 0
};

// Runs: arrival counters (always the same bytes at the front), partials, and for summed weights every
// row's (max, sum) and the logits. Partitions need nothing.
FragLayout frag_layout(const pkv_cache_desc* d, int n_seqs, int max_blocks, const FragGeometry& geo, bool scored) {
    auto up = [](size_t x) { return (x + 15) / 16 * 16; };
    const size_t rows = (size_t)n_seqs * d->n_q_heads;
    if (geo.partition > 0) scored = false;
    const size_t partials = geo.partition > 0 ? 0 : (size_t)geo.ctas * 2 * group_of(d);
    FragLayout l{};
    l.o = partials ? PKV_ARRIVAL_BYTES : 0;
    l.ml = l.o + up(partials * d->head_dim * sizeof(float));
    l.row_ml = l.ml + up(partials * sizeof(float2));
    l.z = l.row_ml + (scored ? up(rows * sizeof(float2)) : 0);
    l.bytes = l.z + (scored ? up(rows * max_blocks * pkv::kBlock * sizeof(float)) : 0);
    return l;
}

size_t frag_workspace(const pkv_cache_desc* d, bool q8, int n_seqs, int max_blocks, bool scored) {
    if (validate16(d) != PKV_OK || n_seqs <= 0 || max_blocks <= 0) return 0;
    FragGeometry geo;
    if (frag_geometry(d, q8, n_seqs, max_blocks, &geo) != cudaSuccess) {
        cudaGetLastError();  // no usable device: report nothing rather than a guess
        return 0;
    }
    return frag_layout(d, n_seqs, max_blocks, geo, scored).bytes;
}

// Shared body of decode over 8-bit pools (q8) and of decode with summed weights (scores).
int frag_decode(bool q8, const pkv_cache_desc* d, int32_t layer, const void* q, const void* k_pool, const void* v_pool,
                const float* k_scales, const float* v_scales, const int32_t* tables, int32_t max_blocks,
                const int32_t* lens, int32_t n_seqs, float scale, void* out, float* scores, int64_t score_stride,
                void* workspace, size_t workspace_bytes, void* stream) {
    int rc = validate16(d);
    if (rc != PKV_OK) return rc;
    if (layer < 0 || layer >= d->n_layers || n_seqs < 0) return PKV_ERR_INVALID_ARG;
    if (n_seqs == 0) return PKV_OK;
    if (max_blocks <= 0 || max_blocks > (1 << 24)) return PKV_ERR_INVALID_ARG;
    if (n_seqs > 65535 || d->n_kv_heads > 65535) return PKV_ERR_UNSUPPORTED;
    if (!q || !k_pool || !v_pool || !tables || !lens || !out) return PKV_ERR_INVALID_ARG;
    if (q8 && (!k_scales || !v_scales || !aligned4(k_scales) || !aligned4(v_scales))) return PKV_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(out) || !aligned16(k_pool) || !aligned16(v_pool)) return PKV_ERR_INVALID_ARG;
    if (scores && (!aligned4(scores) || score_stride < (int64_t)max_blocks * pkv::kBlock)) return PKV_ERR_INVALID_ARG;
    if (pool_rows(d) >= (1LL << 31)) return PKV_ERR_UNSUPPORTED;  // tensor-copy rows are 32-bit
    FragGeometry geo;
    if (frag_geometry(d, q8, n_seqs, max_blocks, &geo) != cudaSuccess) return PKV_ERR_CUDA;
    const FragLayout l = frag_layout(d, n_seqs, max_blocks, geo, scores != nullptr);
    if (l.bytes > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < l.bytes)) return PKV_ERR_INVALID_ARG;

    pkv::FragArgs a;
    const size_t elems = layer_elems(d) * (size_t)layer * (q8 ? 1 : 2);
    char* ws = static_cast<char*>(workspace);
    a.d.q = q;
    a.d.k_layer = static_cast<const char*>(k_pool) + elems;
    a.d.v_layer = static_cast<const char*>(v_pool) + elems;
    a.d.tables = tables;
    a.d.lens = lens;
    a.d.out = out;
    if (geo.partition == 0) {
        a.arrivals = reinterpret_cast<unsigned int*>(ws);
        a.d.part_o = reinterpret_cast<float*>(ws + l.o);
        a.d.part_ml = reinterpret_cast<float*>(ws + l.ml);
    }
    a.d.n_seqs = n_seqs;
    a.d.n_q = d->n_q_heads;
    a.d.n_kv = d->n_kv_heads;
    a.d.num_blocks = d->num_blocks;
    a.d.max_blocks = max_blocks;
    a.d.n_parts = geo.ctas;
    a.partition = geo.partition;
    a.d.scale_log2 = scale * 1.4426950408889634f;
    if (q8) {
        a.k_scales = k_scales + layer_scales(d) * layer;
        a.v_scales = v_scales + layer_scales(d) * layer;
    }
    if (scores && geo.partition > 0) {
        a.scores = scores;
        a.score_stride = score_stride;
    } else if (scores) {
        a.row_ml = reinterpret_cast<float2*>(ws + l.row_ml);
        a.z = reinterpret_cast<float*>(ws + l.z);
    }
    if (pkv::device_status_word(&a.d.status) != cudaSuccess) return PKV_ERR_CUDA;
    cudaError_t err = pkv::launch_frag_decode(d->dtype, q8, d->head_dim, group_of(d), a, static_cast<cudaStream_t>(stream));
    if (err != cudaSuccess) return pkv::launch_status(err);
    pkv::count_launches(1);
    if (scores && geo.partition == 0) {
        pkv::ScoreArgs s;
        s.z = a.z;
        s.row_ml = a.row_ml;
        s.lens = lens;
        s.scores = scores;
        s.stride = score_stride;
        s.n_seqs = n_seqs;
        s.n_kv = d->n_kv_heads;
        s.group = group_of(d);
        s.max_blocks = max_blocks;
        if (pkv::launch_scores(s, static_cast<cudaStream_t>(stream)) != cudaSuccess) return PKV_ERR_CUDA;
        pkv::count_launches(1);
    }
    return PKV_OK;
}

// The most query rows (tokens x heads of the group) that one pass of the chunk kernel over a context holds: as
// many column tiles as have 64 registers of sums a lane.
int wide_columns(const pkv_cache_desc* d) { return d->head_dim < 256 ? 2048 / d->head_dim : 8; }

// Workspace of prefill: arrival counters, the runs' partials, one layer of K and V in 16 bits.
struct ChunkLayout {
    size_t o, ml, k, v, bytes;
};
ChunkLayout chunk_layout(const pkv_cache_desc* d) {
    const size_t partials = (size_t)pkv::kChunkRuns * 2 * wide_columns(d), layer = layer_elems(d) * 2;
    ChunkLayout l;
    l.o = PKV_ARRIVAL_BYTES;
    l.ml = l.o + partials * d->head_dim * sizeof(float);
    l.k = l.ml + partials * sizeof(float2);
    l.v = l.k + layer;
    l.bytes = l.v + layer;
    return l;
}

// Rows of a pass: one column tile of 8, or the most there is room for -- fewer passes, each with more to do. That
// pays from 32 rows on (8 heads x 4 x 128, 20,000 tokens: 24 rows 28.4 us in tiles of 8, 31.5 of 16; 32 rows
// 33.4 and 31.7; 128 rows 97.8 and 76.0) and where the GPU is still full (2 heads x 8 x 128, 1,000 tokens, 128
// rows: 9.0 and 10.1).
int chunk_columns(const pkv_cache_desc* d, int n_seqs, int max_query, int max_blocks) {
    const int group = group_of(d), wide = wide_columns(d), per_pass = wide / group;
    if ((long long)max_query * group < 32) return 8;
    const double passes = (double)n_seqs * ((max_query + per_pass - 1) / per_pass);
    return passes * d->n_kv_heads * max_blocks >= 6000 ? wide : 8;
}

// Whether a chunk is attended to in passes of `columns` rows, each reading the codes again, or widened first and
// handed to the tensor-memory kernel of 16-bit pools. Nanoseconds, for contexts as long as the table is wide:
//   passes  6.5 us (10.5 wide), the context once at 6.5 TB/s, and a pass's work on each token (measured: 3.8, 6.7
//           and 8.5 TB/s of codes at head_dim 64, 128 and 256 in tiles of 8; 2.1 and 5.5 in passes of 32 and 16)
//   widen   8 us, that kernel's waves of 128-key tiles (0.93 us, 1.28 at 256; one CTA of 128 rows an SM, the two of
//           a pair at 256 counted singly) and three bytes a code
// 20,000 tokens, 8 heads x 4 x 128: chunks of 1, 8, 32 and 64 tokens take 19, 32, 76 and 136 us in passes, 168 us
// the other way; 4 x 1,900 tokens, 8 heads x 4 x 64: 2, 16, 32 and 70 tokens 9.5, 22.5, 28.4, 45 against 23.
bool by_passes(const pkv_cache_desc* d, int n_seqs, int n_tokens, int max_query, int max_blocks, int columns, int sms) {
    const double per_pass = columns / group_of(d), row = 2.0 * d->head_dim * d->n_kv_heads;
    const double most = n_seqs * ceil(max_query / per_pass), mean = n_tokens / per_pass + n_seqs * (1 - 1 / per_pass);
    const double passes = most < mean ? most : mean, context = (double)max_blocks * pkv::kBlock;
    const long long ctas = (long long)n_seqs * d->n_kv_heads * (((long long)max_query * group_of(d) + 127) / 128);
    const double waves = (double)((ctas + sms - 1) / sms);
    const bool wide = columns > 8;
    const double rate = d->head_dim == 64 ? (wide ? 2100 : 3800) : d->head_dim == 128 ? (wide ? 5500 : 6700) : 8500;
    return (wide ? 10500 : 6500) + (passes * row / rate + n_seqs * row / 6500) * context <
           8000 + (waves * (d->head_dim == 256 ? 10.0 : 7.3) + n_seqs * row * 3 / 6000.0) * context;
}

}  // namespace

extern "C" {

uint64_t pkv_q8_pool_bytes(const pkv_cache_desc* d) {
    return validate16(d) == PKV_OK ? (uint64_t)d->n_layers * layer_elems(d) : 0;
}

uint64_t pkv_q8_scale_bytes(const pkv_cache_desc* d) {
    return validate16(d) == PKV_OK ? (uint64_t)d->n_layers * layer_scales(d) * sizeof(float) : 0;
}

int pkv_q8_append(const pkv_cache_desc* d, int32_t layer, const void* k, const void* v, const int64_t* slot_mapping,
                  int32_t n_tokens, void* k_codes, void* v_codes, float* k_scales, float* v_scales, void* stream) {
    int rc = validate16(d);
    if (rc != PKV_OK) return rc;
    if (layer < 0 || layer >= d->n_layers || n_tokens < 0) return PKV_ERR_INVALID_ARG;
    if (n_tokens == 0) return PKV_OK;
    if (!k || !v || !slot_mapping || !k_codes || !v_codes || !k_scales || !v_scales) return PKV_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_codes) || !aligned16(v_codes) || !aligned4(k_scales) ||
        !aligned4(v_scales))
        return PKV_ERR_INVALID_ARG;
    // a CTA for every 16 tokens, head, K and V
    if (((long long)n_tokens + 15) / 16 * 2 * d->n_kv_heads >= (1LL << 31)) return PKV_ERR_UNSUPPORTED;
    pkv::Q8AppendArgs a;
    a.k = k;
    a.v = v;
    a.slots = slot_mapping;
    a.k_codes = static_cast<uint8_t*>(k_codes) + layer_elems(d) * layer;
    a.v_codes = static_cast<uint8_t*>(v_codes) + layer_elems(d) * layer;
    a.k_scales = k_scales + layer_scales(d) * layer;
    a.v_scales = v_scales + layer_scales(d) * layer;
    a.n_tok = n_tokens;
    a.n_kv = d->n_kv_heads;
    a.num_blocks = d->num_blocks;
    a.min_exp = pkv::q8_min_exp(d->dtype);
    if (pkv::device_status_word(&a.status) != cudaSuccess) return PKV_ERR_CUDA;
    if (pkv::launch_q8_append(d->dtype, d->head_dim, a, static_cast<cudaStream_t>(stream)) != cudaSuccess)
        return PKV_ERR_CUDA;
    pkv::count_launches(1);
    return PKV_OK;
}

int pkv_q8_copy_blocks(const pkv_cache_desc* d, void* k_codes, void* v_codes, float* k_scales, float* v_scales,
                       const int32_t* pairs, int32_t n_pairs, void* stream) {
    int rc = validate16(d);
    if (rc != PKV_OK) return rc;
    if (n_pairs < 0) return PKV_ERR_INVALID_ARG;
    if (n_pairs == 0) return PKV_OK;
    if (!k_codes || !v_codes || !k_scales || !v_scales || !pairs) return PKV_ERR_INVALID_ARG;
    if (!aligned16(k_codes) || !aligned16(v_codes) || !aligned4(k_scales) || !aligned4(v_scales)) return PKV_ERR_INVALID_ARG;
    if (d->n_layers > 65535) return PKV_ERR_UNSUPPORTED;
    pkv::Q8CopyArgs a;
    a.k_codes = static_cast<uint8_t*>(k_codes);
    a.v_codes = static_cast<uint8_t*>(v_codes);
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.pairs = pairs;
    a.n_pairs = n_pairs;
    a.n_layers = d->n_layers;
    a.n_kv = d->n_kv_heads;
    a.num_blocks = d->num_blocks;
    a.block_bytes = (size_t)d->n_kv_heads * d->block_size * d->head_dim;
    if (pkv::device_status_word(&a.status) != cudaSuccess) return PKV_ERR_CUDA;
    if (pkv::launch_q8_copy(a, static_cast<cudaStream_t>(stream)) != cudaSuccess) return PKV_ERR_CUDA;
    pkv::count_launches(1);
    return PKV_OK;
}

size_t pkv_q8_decode_workspace_bytes(const pkv_cache_desc* d, int32_t n_seqs, int32_t max_blocks_per_seq, int32_t scored) {
    return frag_workspace(d, true, n_seqs, max_blocks_per_seq, scored != 0);
}

int pkv_q8_decode_attention(const pkv_cache_desc* d, int32_t layer, const void* q, const void* k_codes,
                            const void* v_codes, const float* k_scales, const float* v_scales,
                            const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* context_lens,
                            int32_t n_seqs, float scale, void* out, float* scores, int64_t score_stride, void* workspace,
                            size_t workspace_bytes, void* stream) {
    return frag_decode(true, d, layer, q, k_codes, v_codes, k_scales, v_scales, block_tables, max_blocks_per_seq,
                       context_lens, n_seqs, scale, out, scores, score_stride, workspace, workspace_bytes, stream);
}

size_t pkv_scored_workspace_bytes(const pkv_cache_desc* d, int32_t n_seqs, int32_t max_blocks_per_seq) {
    return frag_workspace(d, false, n_seqs, max_blocks_per_seq, true);
}

int pkv_paged_decode_attention_scored(const pkv_cache_desc* d, int32_t layer, const void* q, const void* k_pool,
                                      const void* v_pool, const int32_t* block_tables, int32_t max_blocks_per_seq,
                                      const int32_t* context_lens, int32_t n_seqs, float scale, void* out, float* scores,
                                      int64_t score_stride, void* workspace, size_t workspace_bytes, void* stream) {
    if (n_seqs > 0 && !scores) return PKV_ERR_INVALID_ARG;
    return frag_decode(false, d, layer, q, k_pool, v_pool, nullptr, nullptr, block_tables, max_blocks_per_seq,
                       context_lens, n_seqs, scale, out, scores, score_stride, workspace, workspace_bytes, stream);
}

size_t pkv_q8_prefill_workspace_bytes(const pkv_cache_desc* d) {
    return validate16(d) == PKV_OK ? chunk_layout(d).bytes : 0;
}

int pkv_q8_prefill_attention(const pkv_cache_desc* d, int32_t layer, const void* q, const void* k_codes,
                             const void* v_codes, const float* k_scales, const float* v_scales,
                             const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* context_lens,
                             const int32_t* query_start, int32_t n_seqs, int32_t n_tokens, int32_t max_query_len,
                             float scale, void* out, void* workspace, size_t workspace_bytes, void* stream) {
    int rc = validate16(d);
    if (rc != PKV_OK) return rc;
    if (layer < 0 || layer >= d->n_layers || n_seqs < 0 || n_tokens < 0 || max_query_len < 0 || max_query_len > n_tokens)
        return PKV_ERR_INVALID_ARG;
    if (n_seqs == 0 || max_query_len == 0) return PKV_OK;
    if (max_blocks_per_seq <= 0 || max_blocks_per_seq > (1 << 24)) return PKV_ERR_INVALID_ARG;
    if (n_seqs > 65535 || d->n_kv_heads > 65535 || pool_rows(d) >= (1LL << 31)) return PKV_ERR_UNSUPPORTED;
    if ((long long)max_blocks_per_seq * d->n_kv_heads >= (1LL << 33)) return PKV_ERR_UNSUPPORTED;  // one warp per block and head
    if (!q || !k_codes || !v_codes || !k_scales || !v_scales || !block_tables || !context_lens || !query_start || !out)
        return PKV_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(out) || !aligned16(k_codes) || !aligned16(v_codes) || !aligned4(k_scales) ||
        !aligned4(v_scales))
        return PKV_ERR_INVALID_ARG;
    const ChunkLayout l = chunk_layout(d);
    if (!workspace || !aligned16(workspace) || workspace_bytes < l.bytes) return PKV_ERR_INVALID_ARG;
    char* ws = static_cast<char*>(workspace);
    const uint8_t* k_layer = static_cast<const uint8_t*>(k_codes) + layer_elems(d) * layer;
    const uint8_t* v_layer = static_cast<const uint8_t*>(v_codes) + layer_elems(d) * layer;
    k_scales += layer_scales(d) * layer;
    v_scales += layer_scales(d) * layer;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int group = group_of(d), columns = chunk_columns(d, n_seqs, max_query_len, max_blocks_per_seq);
    const int per_group = columns / group, groups = (max_query_len + per_group - 1) / per_group;
    unsigned int* status = nullptr;
    int sms = 0;
    if (pkv::device_status_word(&status) != cudaSuccess || pkv::current_sm_count(&sms) != cudaSuccess) return PKV_ERR_CUDA;

    // The widened rows' kernel takes the largest product for the largest logit and masks before it scales, so a
    // scale of zero or less (or NaN) goes by passes whatever they cost.
    const long long passes = (long long)n_seqs * groups;
    if (!(scale > 0.f) && passes > (1 << 30)) return PKV_ERR_UNSUPPORTED;  // 32-bit places of the list
    if (!(scale > 0.f) ||
        (passes <= 65535 && by_passes(d, n_seqs, n_tokens, max_query_len, max_blocks_per_seq, columns, sms))) {
        int per_sm = 0;
        if (pkv::frag_multi_ctas_per_sm(d->dtype, d->head_dim, columns, &per_sm) != cudaSuccess) return PKV_ERR_CUDA;
        const FragGeometry geo =
            geometry_of(passes * d->n_kv_heads, max_blocks_per_seq, sms, per_sm, pkv::kChunkRuns);
        pkv::FragArgs a;
        a.d.q = q;
        a.d.k_layer = k_layer;
        a.d.v_layer = v_layer;
        a.d.tables = block_tables;
        a.d.lens = context_lens;
        a.d.out = out;
        a.d.part_o = reinterpret_cast<float*>(ws + l.o);
        a.d.part_ml = reinterpret_cast<float*>(ws + l.ml);
        a.d.status = status;
        a.d.n_seqs = (int)passes;
        a.d.n_q = d->n_q_heads;
        a.d.n_kv = d->n_kv_heads;
        a.d.num_blocks = d->num_blocks;
        a.d.max_blocks = max_blocks_per_seq;
        a.d.n_parts = geo.ctas;
        a.d.scale_log2 = scale * 1.4426950408889634f;
        a.arrivals = reinterpret_cast<unsigned int*>(ws);
        a.k_scales = k_scales;
        a.v_scales = v_scales;
        a.q_start = query_start;
        a.n_tokens = n_tokens;
        a.max_query = max_query_len;
        a.groups = groups;
        a.shift = group == 1 ? 0 : group == 2 ? 1 : group == 4 ? 2 : 3;
        a.partition = geo.partition;
        const cudaError_t err = pkv::launch_frag_multi(d->dtype, d->head_dim, columns, a, st);
        if (err != cudaSuccess) return pkv::launch_status(err);
        pkv::count_launches(1);
        return PKV_OK;
    }

    pkv::Q8WidenArgs w;
    w.k_codes = k_layer;
    w.v_codes = v_layer;
    w.k_scales = k_scales;
    w.v_scales = v_scales;
    w.tables = block_tables;
    w.lens = context_lens;
    w.k_out = ws + l.k;
    w.v_out = ws + l.v;
    w.n_seqs = n_seqs;
    w.n_kv = d->n_kv_heads;
    w.num_blocks = d->num_blocks;
    w.max_blocks = max_blocks_per_seq;
    w.status = status;
    w.v_nan = reinterpret_cast<unsigned int*>(ws);  // (the arrival counters are not used this way)
    // the attention of 16-bit pools over the widened layer, a pool of one layer with the same blocks
    const int per_cta = pkv::prefill_tokens_per_cta(d->dtype, d->head_dim, group);
    pkv::PrefillArgs a;
    a.q = q;
    a.out = out;
    a.k_layer = w.k_out;
    a.v_layer = w.v_out;
    a.tables = block_tables;
    a.lens = context_lens;
    a.q_start = query_start;
    a.status = status;
    a.n_seqs = n_seqs;
    a.n_q = d->n_q_heads;
    a.n_kv = d->n_kv_heads;
    a.num_blocks = d->num_blocks;
    a.max_blocks = max_blocks_per_seq;
    a.n_tokens = n_tokens;
    a.q_tiles = (max_query_len + per_cta - 1) / per_cta;
    a.v_codes = v_layer;
    a.v_nan = w.v_nan;
    a.scale_log2 = scale * 1.4426950408889634f;
    CUtensorMap tk, tv;
    const cudaError_t err = pkv::widened_maps(d->dtype, d->head_dim, w, &tk, &tv);
    if (err != cudaSuccess) return pkv::launch_status(err);
    if (pkv::launch_q8_widen(d->dtype, d->head_dim, w, st) != cudaSuccess) return PKV_ERR_CUDA;
    pkv::count_launches(1);
    if (pkv::launch_prefill_widened(d->dtype, d->head_dim, group, a, tk, tv, st) != cudaSuccess) return PKV_ERR_CUDA;
    pkv::count_launches(1);
    return PKV_OK;
}

size_t pkv_evict_workspace_bytes(const pkv_cache_desc* d, int32_t n_seqs, int32_t max_blocks_per_seq, int32_t q8) {
    if (pkv_validate_desc(d) != PKV_OK || n_seqs <= 0 || max_blocks_per_seq <= 0 || !q8) return 0;
    return 2 * (size_t)d->n_layers * n_seqs * d->n_kv_heads * max_blocks_per_seq * sizeof(float);
}

int pkv_evict_tokens(const pkv_cache_desc* d, void* k_pool, void* v_pool, float* k_scales, float* v_scales,
                     const int32_t* src_tables, const int32_t* dst_tables, int32_t max_blocks_per_seq,
                     const int32_t* context_lens, const int32_t* keep_lens, int32_t n_seqs, int32_t recent,
                     const float* scores, float* new_scores, int64_t score_stride, int32_t* kept, int32_t max_keep,
                     void* workspace, size_t workspace_bytes, void* stream) {
    const bool q8 = k_scales != nullptr || v_scales != nullptr;
    int rc = q8 ? validate16(d) : pkv_validate_desc(d);
    if (rc != PKV_OK) return rc;
    if (n_seqs < 0 || recent < 0 || max_keep < 0) return PKV_ERR_INVALID_ARG;
    if (n_seqs == 0) return PKV_OK;
    if (max_blocks_per_seq <= 0 || max_blocks_per_seq > (1 << 24) || max_keep < 1) return PKV_ERR_INVALID_ARG;
    if (n_seqs > 65535 || d->n_layers > 65535) return PKV_ERR_UNSUPPORTED;
    if (!k_pool || !v_pool || !src_tables || !dst_tables || !context_lens || !keep_lens || !scores || !new_scores || !kept)
        return PKV_ERR_INVALID_ARG;
    if (q8 && (!k_scales || !v_scales || !aligned4(k_scales) || !aligned4(v_scales))) return PKV_ERR_INVALID_ARG;
    if (!aligned16(k_pool) || !aligned16(v_pool) || !aligned4(scores) || !aligned4(new_scores) || !aligned4(kept))
        return PKV_ERR_INVALID_ARG;
    if (score_stride < (int64_t)max_blocks_per_seq * pkv::kBlock) return PKV_ERR_INVALID_ARG;
    const size_t need = pkv_evict_workspace_bytes(d, n_seqs, max_blocks_per_seq, q8);
    if (need > 0 && (!workspace || !aligned4(workspace) || workspace_bytes < need)) return PKV_ERR_INVALID_ARG;

    pkv::EvictArgs a;
    a.k_pool = k_pool;
    a.v_pool = v_pool;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.src = src_tables;
    a.dst = dst_tables;
    a.lens = context_lens;
    a.keep = keep_lens;
    a.scores = scores;
    a.new_scores = new_scores;
    a.kept = kept;
    a.old_scales = static_cast<float*>(workspace);
    a.stride = score_stride;
    a.n_layers = d->n_layers;
    a.n_seqs = n_seqs;
    a.n_kv = d->n_kv_heads;
    a.num_blocks = d->num_blocks;
    a.max_blocks = max_blocks_per_seq;
    a.max_keep = max_keep;
    a.recent = recent;
    a.row_bytes = d->head_dim * (q8 ? 1 : d->dtype == PKV_F32 ? 4 : 2);
    int sms = 0;
    if (pkv::current_sm_count(&sms) != cudaSuccess || pkv::device_status_word(&a.status) != cudaSuccess)
        return PKV_ERR_CUDA;
    // About 8 CTAs an SM share the rows. Column slices (rows moving in place) have 64 bytes at least, or 32
    // while SMs would have none: 32-byte slices of busy grids cost DRAM half its rate (64 triples of 16-bit
    // rows, 2,300 kept: 128-byte slices 98 us, 64 104, 32 142).
    const long long pairs = (long long)n_seqs * d->n_kv_heads;
    auto ctas = [&] { return 2 * pairs * d->n_layers * a.parts; };
    a.parts = 1;
    while (a.parts < 64 && ctas() < 8LL * sms) a.parts *= 2;
    a.slices = a.row_bytes / 64;
    if (2 * pairs * d->n_layers * a.slices < sms) a.slices *= 2;
    if (pairs > 0x7fffffffLL || ctas() > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
    if (pkv::launch_evict(a, static_cast<cudaStream_t>(stream)) != cudaSuccess) return PKV_ERR_CUDA;
    pkv::count_launches(2);
    return PKV_OK;
}

}  // extern "C"
