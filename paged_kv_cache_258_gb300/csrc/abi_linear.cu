// abi_linear.cu -- the C ABI of linear attention and of tables built on the GPU: argument validation, dispatch.
#include "linear.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

size_t layer_floats(const pkv_linear_desc* d) {
    return (size_t)d->n_slots * d->n_v_heads * d->dim_k * d->dim_v;
}

// What decode and prefill check alike; layer's arguments into a. rows: whether there are any tokens.
int linear_args(const pkv_linear_desc* d, int32_t layer, const void* q, const void* k, const void* v,
                const float* log_decay, int64_t decay_stride, float* state, const int32_t* src, const int32_t* dst,
                int32_t n_seqs, float scale, void* out, bool rows, pkv::LinearArgs* a) {
    if ((rows && (!q || !k || !v || !out)) || !state || !src || !dst) return PKV_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(state) || !aligned4(src) ||
        !aligned4(dst))
        return PKV_ERR_INVALID_ARG;
    if (log_decay && (!aligned4(log_decay) || (decay_stride != 0 && decay_stride < d->n_v_heads)))
        return PKV_ERR_INVALID_ARG;
    // a CTA for every sequence, head and 32 columns
    if (n_seqs > 65535 || (long long)n_seqs * d->n_v_heads * (d->dim_v / 32) >= (1LL << 31)) return PKV_ERR_UNSUPPORTED;
    a->q = q;
    a->k = k;
    a->v = v;
    a->out = out;
    a->log_decay = log_decay;
    a->decay_stride = decay_stride;
    a->state = state + layer_floats(d) * layer;
    a->src = src;
    a->dst = dst;
    a->n_seqs = n_seqs;
    a->n_qk = d->n_qk_heads;
    a->n_v = d->n_v_heads;
    a->n_slots = d->n_slots;
    a->scale = scale;
    return pkv::device_status_word(&a->status) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

constexpr int kPiece = 128;          // tokens the tensor-core kernel takes at once
constexpr int kMinShared = 6 * kPiece;  // shortest chunk that is shared out along its length

// Whether a prefill goes by pieces of 128 tokens on the tensor cores or token after token, by what each is estimated to
// take, in microseconds; fp32 has no choice. With units of (sequence, head, 64 columns), dim_k 128 [64]:
//   tokens  2.8 [2.4] and a token of the longest sequence 0.05 + 0.0016 a unit [0.035 + 0.0008], of which 40 to 150
//           count; or over all sequences 0.17 for each million state elements (heads x dim_k x dim_v), at dim_k 128 from
//           six units an SM on 0.135, and 9
//   pieces  bf16 9.4 [7.7] and 1.7 for each piece of the longest sequence but its first, fp16 10.2 [8.2] and 2.4; and where
//           the GPU holds fewer units, 5 [4.2] and for each round of them bf16 4.5 [3.1] and 2.3 [1.9] for each more
//           piece, fp16 6.0 [4.2] and 2.5 [2.2]
// fp16, tokens against pieces: 48 heads x 128 x 128, 16, 32 and 64 tokens 6.6, 9.8 and 16.4 against 10.4; 4 sequences of 16, 32
// and 64 tokens 12.5, 20.9 and 37.4 against 21.6; 32 sequences of 16, 32 and 64 tokens 69, 123 and 227 against 131 (bf16:
// 98). 32 heads x 64 x 64, 32, 64 and 100 tokens 4.2, 6.4 and 8.7 against 7.7 to 8.2; 32 sequences of 16, 32 and 64 tokens
// 14.6, 26.9 and 48.3 against 33 (bf16: 26).
bool by_pieces(const pkv_linear_desc* d, int n_seqs, int n_tokens, int max_query, int sms) {
    if (d->dtype == PKV_F32 || max_query < 2) return false;
    const bool small = d->dim_k == 64, half = d->dtype == PKV_F16;
    const double tokens = n_tokens < (double)n_seqs * max_query ? n_tokens : (double)n_seqs * max_query;
    const double elements = (double)d->n_v_heads * d->dim_k * d->dim_v * 1e-6;
    const double units = (double)n_seqs * d->n_v_heads * (d->dim_v / 64);
    const double some = units < 40 ? 40 : units < 150 ? units : 150;
    const double each = small ? 0.035 + 0.0008 * some : 0.05 + 0.0016 * some;
    const double work = small || units < 6.0 * sms ? 0.17 * tokens * elements : 9 + 0.135 * tokens * elements;
    const double longest = each * max_query;
    double pieces = (small ? (half ? 8.2 : 7.7) : (half ? 10.2 : 9.4)) + (half ? 2.4 : 1.7) * ((max_query - 1) / kPiece);
    if (units > sms) {
        const double rounds = (double)(((long long)units + sms - 1) / sms), more = tokens / n_seqs / kPiece - 1;
        const double first = small ? (half ? 4.2 : 3.1) : (half ? 6.0 : 4.5), next = small ? (half ? 2.2 : 1.9) : (half ? 2.5 : 2.3);
        const double all = (small ? 4.2 : 5.0) + rounds * (first + next * (more > 0 ? more : 0));
        pieces = all > pieces ? all : pieces;
    }
    return pieces < (small ? 2.4 : 2.8) + (work > longest ? work : longest);
}

// How a call's sequences are shared out along their length: in as many segments as the GPU holds CTAs for them, but no more
// than kMaxSegments, each of which reads what all before it leave. dim_k 128 [64], in microseconds: two passes of p / n pieces are
// estimated at 13.5 [10] + 3.1 [2.5] for each piece (fp16 4.1 [3.7]) + 0.25 for each segment, one of p pieces at 6.2 [7.2] + 1.73
// [1.5] (fp16 2.5 [2.25]). Whole against segments, calls behind one another in a graph: 8 heads x 128 x 64, bf16, 768, 1,024, 1,536 and
// 9,005 tokens 16.7, 20.1, 26.8 and 121 against 18.0, 18.4, 19.5 and 30.5, fp16 21.9, 26.8, 36.3 and 169 against 19.4, 19.9, 20.8
// and 34.8; 32 heads x 128 x 128, two segments, 2,048 and 16,384 tokens bf16 35.1 and 219 against 39.7 and 207, fp16 47.2 and 313
// against 48.7 and 283; 16 heads x 64 x 64, bf16, 768 tokens 16.0 against 14.0.
constexpr int kMaxSegments = 32;
struct Segments {
    int n, tokens;
};
Segments segments_of(const pkv_linear_desc* d, int n_seqs, int max_query, int sms) {
    const long long units = (long long)n_seqs * d->n_v_heads * (d->dim_v / 64);
    const int pieces = (max_query + kPiece - 1) / kPiece;
    const Segments whole = {1, pieces * kPiece};
    if (units * 2 > sms || max_query < kMinShared) return whole;
    long long n = sms / units < kMaxSegments ? sms / units : kMaxSegments;
    const int each = (int)((pieces + n - 1) / n);
    n = (pieces + each - 1) / each;
    const bool bf16 = d->dtype == PKV_BF16, small = d->dim_k == 64;
    const double shared = (small ? 10.0 : 13.5) + (small ? (bf16 ? 2.5 : 3.7) : (bf16 ? 3.1 : 4.1)) * each + 0.25 * (double)n;
    if (shared >= (small ? 7.2 : 6.2) + (small ? (bf16 ? 1.5 : 2.25) : (bf16 ? 1.73 : 2.5)) * pieces) return whole;
    return {(int)n, each * kPiece};
}

// Workspace of a shared-out call, in floats: units of 64 columns are at most sms / segments, so sms of them hold all
// that the segments leave, and as many the starts.
struct PrefillLayout {
    size_t start, added, sums, bytes;
};
PrefillLayout prefill_layout(const pkv_linear_desc* d, int sms) {
    const size_t unit = (size_t)d->dim_k * 64, all = unit * (size_t)sms;
    return {0, all, 2 * all, (2 * all + (size_t)sms) * sizeof(float)};
}

}  // namespace

extern "C" {

int pkv_linear_validate_desc(const pkv_linear_desc* d) {
    if (!d || d->n_layers <= 0 || d->n_slots <= 0 || d->n_qk_heads <= 0 || d->n_v_heads <= 0 || d->dim_k <= 0 ||
        d->dim_v <= 0)
        return PKV_ERR_INVALID_ARG;
    if (d->dtype != PKV_F32 && d->dtype != PKV_F16 && d->dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
    if ((d->dim_k != 64 && d->dim_k != 128) || (d->dim_v != 64 && d->dim_v != 128)) return PKV_ERR_UNSUPPORTED;
    if (d->n_v_heads % d->n_qk_heads != 0 || d->n_v_heads > 65535) return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

uint64_t pkv_linear_state_bytes(const pkv_linear_desc* d) {
    return pkv_linear_validate_desc(d) == PKV_OK ? (uint64_t)d->n_layers * layer_floats(d) * sizeof(float) : 0;
}

int pkv_linear_decode(const pkv_linear_desc* d, int32_t layer, const void* q, const void* k, const void* v,
                      const float* log_decay, int64_t decay_stride, float* state, const int32_t* src_slots,
                      const int32_t* dst_slots, int32_t n_seqs, float scale, void* out, void* stream) {
    int rc = pkv_linear_validate_desc(d);
    if (rc != PKV_OK) return rc;
    if (layer < 0 || layer >= d->n_layers || n_seqs < 0) return PKV_ERR_INVALID_ARG;
    if (n_seqs == 0) return PKV_OK;
    pkv::LinearArgs a;
    rc = linear_args(d, layer, q, k, v, log_decay, decay_stride, state, src_slots, dst_slots, n_seqs, scale, out, true, &a);
    if (rc != PKV_OK) return rc;
    a.q_start = nullptr;
    a.n_tokens = n_seqs;
    a.max_query = 1;
    int sms = 0;
    if (pkv::current_sm_count(&sms) != cudaSuccess) return PKV_ERR_CUDA;
    if (pkv::launch_linear_step(d->dtype, d->dim_k, d->dim_v, sms, a, static_cast<cudaStream_t>(stream)) != cudaSuccess)
        return PKV_ERR_CUDA;
    pkv::count_launches(1);
    return PKV_OK;
}

size_t pkv_linear_prefill_workspace_bytes(const pkv_linear_desc* d, int32_t n_seqs, int32_t n_tokens,
                                          int32_t max_query_len) {
    if (pkv_linear_validate_desc(d) != PKV_OK || n_seqs <= 0 || n_tokens <= 0 || max_query_len <= 0) return 0;
    if (d->dtype == PKV_F32 || max_query_len < kMinShared) return 0;
    int sms = 0;
    if (pkv::current_sm_count(&sms) != cudaSuccess) {
        cudaGetLastError();  // no usable device: report nothing rather than a guess
        return 0;
    }
    return prefill_layout(d, sms).bytes;
}

int pkv_linear_prefill(const pkv_linear_desc* d, int32_t layer, const void* q, const void* k, const void* v,
                       const float* log_decay, int64_t decay_stride, float* state, const int32_t* src_slots,
                       const int32_t* dst_slots, const int32_t* query_start, int32_t n_seqs, int32_t n_tokens,
                       int32_t max_query_len, float scale, void* out, void* workspace, size_t workspace_bytes,
                       void* stream) {
    int rc = pkv_linear_validate_desc(d);
    if (rc != PKV_OK) return rc;
    if (layer < 0 || layer >= d->n_layers || n_seqs < 0 || n_tokens < 0 || max_query_len < 0 || max_query_len > n_tokens)
        return PKV_ERR_INVALID_ARG;
    if (n_seqs == 0) return PKV_OK;
    if (n_tokens > 0x7fffff00) return PKV_ERR_UNSUPPORTED;  // (tokens are counted in whole pieces, in 32 bits)
    if (!query_start || !aligned4(query_start)) return PKV_ERR_INVALID_ARG;
    pkv::LinearArgs a;
    rc = linear_args(d, layer, q, k, v, log_decay, decay_stride, state, src_slots, dst_slots, n_seqs, scale, out, n_tokens > 0,
                     &a);
    if (rc != PKV_OK) return rc;
    a.q_start = query_start;
    a.n_tokens = n_tokens;
    a.max_query = max_query_len;
    int sms = 0;
    if (pkv::current_sm_count(&sms) != cudaSuccess) return PKV_ERR_CUDA;
    if (by_pieces(d, n_seqs, n_tokens, max_query_len, sms)) {
        pkv::ChunkArgs c;
        c.l = a;
        c.dv = d->dim_v;
        c.slices = d->dim_v / 64;
        const Segments seg = segments_of(d, n_seqs, max_query_len, sms);
        c.n_segs = seg.n;
        c.seg_tokens = seg.tokens;
        c.take_more = seg.n == 1 && (long long)n_seqs * d->n_v_heads * c.slices > sms;
        if (seg.n > 1) {
            const PrefillLayout lay = prefill_layout(d, sms);
            if (!workspace || !aligned16(workspace) || workspace_bytes < lay.bytes) return PKV_ERR_INVALID_ARG;
            float* ws = static_cast<float*>(workspace);
            c.start = ws + lay.start;
            c.added = ws + lay.added;
            c.sums = ws + lay.sums;
        }
        CUtensorMap tq, tk, tv;
        cudaError_t err = pkv::rows_tensor_map(q, n_tokens, d->n_qk_heads * d->dim_k, d->dtype, kPiece, &tq);
        if (err == cudaSuccess) err = pkv::rows_tensor_map(k, n_tokens, d->n_qk_heads * d->dim_k, d->dtype, kPiece, &tk);
        if (err == cudaSuccess) err = pkv::rows_tensor_map(v, n_tokens, d->n_v_heads * d->dim_v, d->dtype, kPiece, &tv);
        if (err != cudaSuccess) return pkv::launch_status(err);
        const auto launch = d->dtype == PKV_F16 ? pkv::launch_linear_chunk_f16 : pkv::launch_linear_chunk_bf16;
        err = launch(d->dim_k, c, tq, tk, tv, static_cast<cudaStream_t>(stream));
        if (err != cudaSuccess) return PKV_ERR_CUDA;
        pkv::count_launches(seg.n > 1 ? 2 : 1);
        return PKV_OK;
    }
    if (pkv::launch_linear_step(d->dtype, d->dim_k, d->dim_v, sms, a, static_cast<cudaStream_t>(stream)) != cudaSuccess)
        return PKV_ERR_CUDA;
    pkv::count_launches(1);
    return PKV_OK;
}

int pkv_extend_tables(int32_t num_blocks, const int32_t* free_blocks, int32_t n_free, const int32_t* used,
                      int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* context_lens,
                      const int32_t* new_tokens, int32_t n_seqs, int64_t* slot_mapping, int32_t max_tokens,
                      int32_t* query_start, int32_t* new_lens, int32_t* totals, void* stream) {
    if (num_blocks <= 0 || n_free < 0 || n_seqs < 0 || max_tokens < 0) return PKV_ERR_INVALID_ARG;
    if (max_blocks_per_seq <= 0 || max_blocks_per_seq > (1 << 24)) return PKV_ERR_INVALID_ARG;
    if (n_seqs > 65535) return PKV_ERR_UNSUPPORTED;
    if (max_tokens > 0x7ffffffe) return PKV_ERR_UNSUPPORTED;  // (2^31 - 1 is what a sum past it saturates at)
    if ((n_free > 0 && !free_blocks) || !used || !query_start || !totals || (max_tokens > 0 && !slot_mapping))
        return PKV_ERR_INVALID_ARG;
    if (n_seqs > 0 && (!block_tables || !context_lens || !new_lens)) return PKV_ERR_INVALID_ARG;
    if (!aligned4(free_blocks) || !aligned4(used) || !aligned4(block_tables) || !aligned4(context_lens) ||
        !aligned4(new_tokens) || !aligned4(query_start) || !aligned4(new_lens) || !aligned4(totals) ||
        (reinterpret_cast<uintptr_t>(slot_mapping) & 7u) != 0)
        return PKV_ERR_INVALID_ARG;
    pkv::ExtendArgs a;
    a.free_blocks = free_blocks;
    a.used = used;
    a.tables = block_tables;
    a.lens = context_lens;
    a.new_tokens = new_tokens;
    a.slots = slot_mapping;
    a.query_start = query_start;
    a.new_lens = new_lens;
    a.totals = totals;
    a.num_blocks = num_blocks;
    a.n_free = n_free;
    a.max_blocks = max_blocks_per_seq;
    a.n_seqs = n_seqs;
    a.max_tokens = max_tokens;
    if (pkv::device_status_word(&a.status) != cudaSuccess) return PKV_ERR_CUDA;
    int sms = 0, launches = 0;
    if (pkv::current_sm_count(&sms) != cudaSuccess) return PKV_ERR_CUDA;
    if (pkv::launch_extend_tables(a, static_cast<cudaStream_t>(stream), sms, &launches) != cudaSuccess) return PKV_ERR_CUDA;
    pkv::count_launches(launches);
    return PKV_OK;
}

}  // extern "C"
