// Decode-phase PagedAttention entry points (include/pkv.h): argument checks,
// the launch of the bf16-cache kernels (the kernel itself is in
// pkv_decode_kernel.cuh) and the workspace size.
#include "pkv_decode_kernel.cuh"

using namespace pkv;

extern "C" size_t pkv_paged_decode_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                                  int32_t head_dim)
{
    if (num_seqs < 0 || num_seqs > PKV_MAX_SEQS || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
        num_q_heads % num_kv_heads != 0)
        return 0;
    return ws_layout(num_seqs, num_q_heads / num_kv_heads, num_kv_heads, head_dim).total;
}

// What a masked call adds (see DecodeParams): a window and sinks, or a tree over the sequences' new tokens.
struct MaskArgs {
    bool new_tokens = false;  // an attention call: each query needs a key of its own, one query too
    int32_t window = INT32_MAX, sinks = 0;
    const uint32_t *tree = nullptr;
    int32_t tree_words = 0, tree_n = 0;
    const int32_t *tree_lens = nullptr, *tree_cu = nullptr;
};

// Longest sequences of masked calls: a position less a window length or a tile's start stays in 32 bits.
constexpr int64_t kMaskMaxLen = 1 << 30;

static pkv_status check_mask(const MaskArgs &m, bool tree)
{
    if (!tree) return m.window < 1 || m.sinks < 0 ? PKV_EINVAL : PKV_OK;
    if (m.tree_words < 1 || m.tree_n > 32LL * m.tree_words || (reinterpret_cast<uintptr_t>(m.tree) & 3u))
        return PKV_EINVAL;
    return PKV_OK;
}

// (p.len_limit and p.toks are set)
static void set_mask(DecodeParams &p, const MaskArgs &m)
{
    p.lg_toks = ilog2(p.toks);
    p.window = std::min(m.window, std::max(p.len_limit, 1));  // (one as long as the sequences sees all)
    p.sinks = std::min(m.sinks, p.len_limit);
    p.tree = m.tree;
    p.tree_words = m.tree_words;
    p.tree_n = m.tree_n;
    p.tree_lens = m.tree_lens;
    p.tree_cu = m.tree_cu;
}

// Tokens of a sequence that its last n queries see, at most.
static int64_t seen_bound(const MaskArgs *m, int64_t len_limit, int64_t n)
{
    return m ? std::min<int64_t>(len_limit, int64_t(m->window) + m->sinks + n - 1) : len_limit;
}

// The units of a call's list at most (`entries` of them hold work, up to `queries` queries each): unit counts and
// positions in the list are kept in 32 bits.  int8 calls count the units of the CTA that runs them, the others 8 tokens of
// a kv head.  A masked call's list has what its queries see (a window that begins inside a unit, or sinks that end
// inside one: a unit more each).
static int64_t unit_bound(int ct, bool qs, int G, int32_t num_kv_heads, int64_t entries, int64_t len_limit,
                          const MaskArgs *mask, int64_t queries)
{
    const int hg = ct != kI8 || qs ? 1 : head_group(num_kv_heads, G);
    const int toks = ct != kI8 ? 8 : warp_tokens(G, true, qs, qs) * (qs ? 1 : warp_slices(G, hg));
    int64_t units = (len_limit + toks - 1) / toks;
    if (mask) units = std::min(units, (seen_bound(mask, len_limit, queries) + toks - 1) / toks + 2);
    return num_kv_heads / hg * entries * units;
}

// Shared by the entry points of all cache types (ct; k_scale / v_scale: the
// per-kv-head scales of E4M3 caches, scales: those of int8 ones, device arrays).  qn > 1: entry b holds up to qn
// queries that share its K/V stream as qn * G virtual heads of a kv head --
// with row_cnt null, every entry is a sequence with qn new tokens (q / out rows
// b * qn + i; context_lens the sequences' whole lengths); otherwise entry b
// holds row_cnt[b] queries at rows b + i (row_seq[b]: its sequence,
// context_lens[b]: the length its last query sees).  live: the entries that can hold work, where not all do.
static pkv_status decode_call(int ct, bool qs, int32_t qn, const uint16_t *q, const void *k_cache, const void *v_cache,
                              const float *k_scale, const float *v_scale, const int32_t *row_seq,
                              const int32_t *row_cnt, const int32_t *block_tables,
                              int32_t max_blocks_per_seq, const int32_t *context_lens, int32_t num_seqs,
                              int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                              int32_t num_blocks, int32_t max_context_len, float scale, uint16_t *out,
                              void *workspace, size_t workspace_bytes, int32_t num_workers, int32_t *err_word,
                              pkv_stream_t stream, const uint16_t *k_new = nullptr, const uint16_t *v_new = nullptr,
                              int32_t *slot_out = nullptr, const float *scales = nullptr,
                              const int32_t *row0 = nullptr, int64_t live = -1, const MaskArgs *mask = nullptr)
{
    const bool fp8 = ct != kBf16, i8 = ct == kI8;  // fp8: one byte per cached element
    if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0 ||
        head_dim <= 0 || block_size <= 0 || num_blocks <= 0 || max_blocks_per_seq <= 0 || max_context_len < 0 ||
        num_workers < 0 || !std::isfinite(scale))
        return PKV_EINVAL;
    if (num_seqs > PKV_MAX_SEQS || num_workers > PKV_MAX_WORKERS) return PKV_EBOUNDS;
    if (head_dim != 64 && head_dim != 128) return PKV_EUNSUPPORTED;
    if (qn < 1) return PKV_EINVAL;
    const int gq = num_q_heads / num_kv_heads;  // query heads per kv head
    const int G = gq * qn;                      // virtual heads per kv head sharing one K/V stream
    if (G > (ct == kE4m3 ? 8 : 16)) return PKV_EUNSUPPORTED;  // virtual heads per warp: the MMA tile's rows
    if (!is_pow2(block_size) || block_size < (ct == kI8 ? kScaleToks : 8) || block_size > 1024) return PKV_EUNSUPPORTED;
    if (int64_t(num_blocks) * block_size > INT32_MAX) return PKV_EBOUNDS;
    if (num_seqs == 0) return PKV_OK;
    if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !out) return PKV_EINVAL;
    if (ct == kE4m3 && (!k_scale || !v_scale)) return PKV_EINVAL;
    if (ct == kI8 && (!scales || (reinterpret_cast<uintptr_t>(scales) & 7u))) return PKV_EINVAL;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out)) return PKV_EINVAL;
    const int64_t len_limit = std::min<int64_t>(max_context_len, int64_t(max_blocks_per_seq) * block_size);
    const int64_t queries = qs ? 128 / gq : qn;  // of an entry at most
    if (unit_bound(ct, qs, G, num_kv_heads, live < 0 ? num_seqs : live, len_limit, mask, queries) > INT32_MAX)
        return PKV_EBOUNDS;
    if (mask && len_limit > kMaskMaxLen) return PKV_EBOUNDS;
    if (qs && (ct == kE4m3 || !row_cnt || (i8 && !row0))) return PKV_EINVAL;  // query-split entries are chunks of bf16 or int8 calls
    if ((k_new || v_new) && (qs || ct == kI8 || qn != 1 || row_seq || !k_new || !v_new || !aligned16(k_new) ||
                             !aligned16(v_new)))
        return PKV_EINVAL;  // the fused store goes with a decode
    // (query-split entries of int8 calls leave pieces of 16-row blocks whatever their group)
    const WsLayout ws = ws_layout(num_seqs, i8 && qs ? 16 : G, num_kv_heads, head_dim, qs);
    if (!workspace || workspace_bytes < ws.total || !aligned16(workspace)) return PKV_EWORKSPACE;

    DeviceInfo dev;
    if (!current_device_info(&dev)) return PKV_ECUDA;

    LaunchArgs a{};  // every field starts at zero; those a call uses are set below
    DecodeParams &p = a.p;
    uint8_t *wsb = static_cast<uint8_t *>(workspace);
    p.q = q;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.out = out;
    p.ws_count = reinterpret_cast<unsigned long long *>(wsb + ws.count_off);
    p.ws_bal = reinterpret_cast<BalanceState *>(wsb + ws.bal_off);
    p.ws_ml = reinterpret_cast<float *>(wsb + ws.ml_off);
    p.ws_acc = reinterpret_cast<float *>(wsb + ws.acc_off);
    p.err = err_word;
    p.B = num_seqs;
    p.Hq = num_q_heads;
    p.Hkv = num_kv_heads;
    p.bs = block_size;
    p.log2_bs = ilog2(block_size);
    p.NB = num_blocks;
    p.max_blocks = max_blocks_per_seq;
    p.len_limit = int32_t(len_limit);
    p.min_len = !row_cnt && (qn > 1 || (mask && mask->new_tokens)) ? qn : 0;
    // query-split entries of 128 rows run on the tensor-memory CTAs where they can
    const bool tc5 = qs && (i8 || tc5_eligible(head_dim, G, gq, block_size, num_seqs, dev.max_smem_optin));
    p.hg = qs ? 1 : head_group(num_kv_heads, G);
    p.nhg = num_kv_heads / p.hg;
    p.sub = qs ? team_warps(G) : warp_slices(G, p.hg);
    p.toks = warp_tokens(G, fp8, qs, tc5) * (qs ? 1 : p.sub);
    p.boxtok = std::min(p.toks, block_size);
    p.nbox = p.toks / p.boxtok;
    p.lg_nbox = ilog2(p.nbox);
    p.cons = tc5 ? tc5_consumers(ct) : p.hg * p.sub;
    p.nst = 2;
    p.num_workers = 0;
    p.per_segment = 0;
    p.scale_log2 = float(double(scale) * 1.4426950408889634);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.scales = reinterpret_cast<const float2 *>(scales);
    p.row_seq = row_seq;
    p.qn = qn;
    p.gq = gq;
    p.row_cnt = row_cnt;
    p.row0 = row0;
    p.k_new = k_new;
    p.v_new = v_new;
    p.k_cache_w = static_cast<uint8_t *>(const_cast<void *>(k_cache));
    p.v_cache_w = static_cast<uint8_t *>(const_cast<void *>(v_cache));
    p.slot_out = k_new ? slot_out : nullptr;
    p.qstride = row_cnt ? 1 : qn;
    if (mask) set_mask(p, *mask);
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.device = dev.device;
    a.sm_count = dev.sm_count;
    a.max_smem = dev.max_smem_optin;
    a.requested_workers = num_workers;
    // A call with fewer units than SMs (bounded from the host-known lengths) runs one CTA per unit
    // with the fixed split: the CTAs without work would only add set-up and contention
    // (tiny and Qwen2.5-shaped batches: 9.2 -> 7.9 and 17.9 -> 14.1 us per graph-replayed call).
    // Regular CTAs with at most kSegmentUnits units per (entry, head group) run one CTA per segment
    // instead: a few units in one CTA's pipeline cost less than the split-K pieces and merge of a
    // split (per back-to-back call: tiny workload 8.3 -> 7.0 us, Qwen2.5-shaped 14.2 -> 9.0 us).
    if (num_workers == 0) {
        // (a window that begins inside a unit, or sinks that end inside one: a unit more each)
        int64_t per_seg = (len_limit + p.toks - 1) / p.toks;
        if (mask)
            per_seg = std::min(per_seg, (seen_bound(mask, len_limit, queries) + p.toks - 1) / p.toks + 2);
        const int64_t units_max = int64_t(num_seqs) * p.nhg * per_seg;
        if (units_max < dev.sm_count) {
            if ((!qs || i8) && per_seg <= kSegmentUnits && int64_t(num_seqs) * p.nhg <= kMaxSlots) {
                p.per_segment = 1;
                a.requested_workers = num_seqs * p.nhg * p.cons;
            } else {
                a.requested_workers = int32_t(std::max<int64_t>(1, units_max)) * p.cons;
            }
        }
        // int8 caches: also with more units than SMs, as long as every segment has an SM (decode batches of 24 to 140
        // sequences of 130 to 500 tokens, 16 / 8 heads of 128 and 12 / 4 of 64: split 18-27 us, a CTA a segment 10-19;
        // with 16 units a segment the split is as fast, and faster where lengths differ).
        if (i8 && !qs && per_seg <= kSegmentUnits && int64_t(num_seqs) * p.nhg <= dev.sm_count) {
            p.per_segment = 1;
            a.requested_workers = num_seqs * p.nhg * p.cons;
        }
        // int8 caches, few segments: a segment's pieces are counted in and folded one after another (about half a
        // microsecond each), its units streamed by as many CTAs as it has pieces, so the sum of both is least at a
        // number of pieces that grows with the root of the units.  Measured on 10 batches of 1 to 16 sequences of
        // 600 to 32000 tokens, num_workers swept: the best number lies between 1.1 and 2.2 sqrt(units), 1.6 within
        // 15 % of it everywhere; one sequence of 3500 tokens 66.6 -> 27.5 us, of 32000 79 -> 54 us, two of 12000
        // 47.7 -> 32.5 us.
        if (i8 && !qs && !p.per_segment) {
            const int64_t pieces = int64_t(std::ceil(1.6 * std::sqrt(double(per_seg))));
            const int64_t ctas = std::min<int64_t>(units_max, int64_t(num_seqs) * p.nhg * pieces);
            if (ctas < dev.sm_count) a.requested_workers = int32_t(std::max<int64_t>(1, ctas)) * p.cons;
        }
    }
    a.stream = reinterpret_cast<cudaStream_t>(stream);

    LaunchFn fn = mask && ct == kE4m3 ? pick_mask_fp8(head_dim, G)
                  : mask && ct == kI8 ? (qs ? pick_mask_i8_tc5(head_dim)
                                            : G > 8 ? pick_mask_i8_wide(head_dim, G) : pick_mask_i8(head_dim, G))
                  : mask ? (G > 8 ? pick_mask_wide(head_dim, G) : pick_mask(head_dim, G))
                  : ct == kE4m3 ? pick_decode_fp8(head_dim, G)
                  : ct == kI8 ? (qs ? pick_decode_i8_tc5(head_dim)
                                    : G > 8 ? pick_decode_i8_wide(head_dim, G) : pick_decode_i8(head_dim, G))
                  : tc5  ? pick_decode_tc5(head_dim)
                  : qs   ? pick_decode_qs(head_dim, G)
                  : G > 8 ? pick_decode_wide(head_dim, G)
                         : (head_dim == 64 ? pick_group<64, kBf16, false>(G) : pick_group<128, kBf16, false>(G));
    if (!fn) return PKV_EUNSUPPORTED;
    if (ws.count_clear) {  // counters outside the fixed region start at zero (see WsLayout)
        const cudaError_t ce = cudaMemsetAsync(p.ws_count, 0, ws.count_bytes, a.stream);
        if (ce != cudaSuccess) {
            cudaGetLastError();
            return cuda_fail("cudaMemsetAsync (arrival counters)", ce);
        }
    }
    return fn(a);
}

extern "C" pkv_status pkv_paged_decode(const uint16_t *q, const uint16_t *k_cache, const uint16_t *v_cache,
                                       const int32_t *block_tables, int32_t max_blocks_per_seq,
                                       const int32_t *context_lens, int32_t num_seqs, int32_t num_q_heads,
                                       int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                       int32_t num_blocks, int32_t max_context_len, float scale, uint16_t *out,
                                       void *workspace, size_t workspace_bytes, int32_t num_workers,
                                       int32_t *err_word, pkv_stream_t stream)
{
    return decode_call(kBf16, false, 1, q, k_cache, v_cache, nullptr, nullptr, nullptr, nullptr, block_tables,
                       max_blocks_per_seq, context_lens, num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                       num_blocks, max_context_len, scale, out, workspace, workspace_bytes, num_workers, err_word,
                       stream);
}

extern "C" pkv_status pkv_paged_decode_store(const uint16_t *q, const uint16_t *k_new, const uint16_t *v_new,
                                             uint16_t *k_cache, uint16_t *v_cache, const int32_t *block_tables,
                                             int32_t max_blocks_per_seq, const int32_t *context_lens,
                                             int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                             int32_t head_dim, int32_t block_size, int32_t num_blocks,
                                             int32_t max_context_len, float scale, uint16_t *out,
                                             int32_t *slot_mapping, void *workspace, size_t workspace_bytes,
                                             int32_t num_workers, int32_t *err_word, pkv_stream_t stream)
{
    if (num_seqs > 0 && (!k_new || !v_new)) return PKV_EINVAL;
    return decode_call(kBf16, false, 1, q, k_cache, v_cache, nullptr, nullptr, nullptr, nullptr, block_tables,
                       max_blocks_per_seq, context_lens, num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                       num_blocks, max_context_len, scale, out, workspace, workspace_bytes, num_workers, err_word,
                       stream, k_new, v_new, slot_mapping);
}

extern "C" pkv_status pkv_paged_decode_store_fp8(const uint16_t *q, const uint16_t *k_new, const uint16_t *v_new,
                                                 uint8_t *k_cache, uint8_t *v_cache, const float *k_scale,
                                                 const float *v_scale, const int32_t *block_tables,
                                                 int32_t max_blocks_per_seq, const int32_t *context_lens,
                                                 int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                                 int32_t head_dim, int32_t block_size, int32_t num_blocks,
                                                 int32_t max_context_len, float scale, uint16_t *out,
                                                 int32_t *slot_mapping, void *workspace, size_t workspace_bytes,
                                                 int32_t num_workers, int32_t *err_word, pkv_stream_t stream)
{
    if (num_seqs > 0 && (!k_new || !v_new)) return PKV_EINVAL;
    return decode_call(kE4m3, false, 1, q, k_cache, v_cache, k_scale, v_scale, nullptr, nullptr, block_tables,
                       max_blocks_per_seq, context_lens, num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                       num_blocks, max_context_len, scale, out, workspace, workspace_bytes, num_workers, err_word,
                       stream, k_new, v_new, slot_mapping);
}

extern "C" pkv_status pkv_paged_decode_fp8(const uint16_t *q, const uint8_t *k_cache, const uint8_t *v_cache,
                                           const float *k_scale, const float *v_scale, const int32_t *block_tables,
                                           int32_t max_blocks_per_seq, const int32_t *context_lens,
                                           int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                           int32_t head_dim, int32_t block_size, int32_t num_blocks,
                                           int32_t max_context_len, float scale, uint16_t *out, void *workspace,
                                           size_t workspace_bytes, int32_t num_workers, int32_t *err_word,
                                           pkv_stream_t stream)
{
    return decode_call(kE4m3, false, 1, q, k_cache, v_cache, k_scale, v_scale, nullptr, nullptr, block_tables,
                       max_blocks_per_seq, context_lens,
                       num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, max_context_len, scale,
                       out, workspace, workspace_bytes, num_workers, err_word, stream);
}

extern "C" pkv_status pkv_paged_decode_i8(const uint16_t *q, const int8_t *k_cache, const int8_t *v_cache,
                                          const float *scales, const int32_t *block_tables,
                                          int32_t max_blocks_per_seq, const int32_t *context_lens, int32_t num_seqs,
                                          int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                          int32_t block_size, int32_t num_blocks, int32_t max_context_len,
                                          float scale, uint16_t *out, void *workspace, size_t workspace_bytes,
                                          int32_t num_workers, int32_t *err_word, pkv_stream_t stream)
{
    return decode_call(kI8, false, 1, q, k_cache, v_cache, nullptr, nullptr, nullptr, nullptr, block_tables,
                       max_blocks_per_seq, context_lens, num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                       num_blocks, max_context_len, scale, out, workspace, workspace_bytes, num_workers, err_word,
                       stream, nullptr, nullptr, nullptr, scales);
}

// ------------------------------------------------------------------ several query rows per sequence
namespace pkv {

// Whether the num_seqs + 1 offsets never decrease.  Every block looks at all of them (every thread of it calls this):
// a search over offsets that do would miss some of them, and the rows of the others could overlap.
__device__ __forceinline__ bool offsets_in_order(const int32_t *__restrict__ cu, int32_t num_seqs)
{
    bool ok = true;
    for (int32_t b = threadIdx.x; b < num_seqs; b += blockDim.x) ok &= __ldg(cu + b) <= __ldg(cu + b + 1);
    return __syncthreads_and(ok) != 0;
}

// Query row r = cu_seqlens_q[b] + i of sequence b (n = cu_seqlens_q[b+1] -
// cu_seqlens_q[b] new tokens, L = context_lens[b] in the cache) sits at
// position L - n + i: it sees the L - n + i + 1 keys before it.  The rows of
// a sequence are cut into chunks of up to `chunk` consecutive queries that share
// one K/V stream; a chunk is entry r of the decode kernel, r the row of its
// first query: row_seq[r] = b, row_cnt[r] = its query count, row_len[r] = the
// keys its last query sees.  Rows that start no chunk get row_cnt = 0 and
// row_len = 0 (no work, no output).  One thread per row finds its sequence by
// binary search over cu_seqlens_q, so every row gets a sequence in
// [0, num_seqs) even when the offsets are inconsistent; such rows (not inside
// their sequence's range, n > L, offsets not starting at 0) are entries of
// their own or their chunk's with length 0 (zero output) and set
// PKV_ERR_CONTEXT_RANGE.  Offsets that decrease anywhere make every row one
// of them: the search sees only some of such offsets.  With cu_seqlens_q null,
// every sequence has new_per_seq rows (row r belongs to sequence r / new_per_seq).  More than max_new rows of a
// sequence (what a tree's masks hold) are inconsistent too.
__global__ void expand_rows_kernel(const int32_t *__restrict__ cu_seqlens_q, int32_t new_per_seq,
                                   const int32_t *__restrict__ context_lens, int32_t num_seqs, int32_t num_rows,
                                   int32_t chunk, int32_t max_new, int32_t *__restrict__ row_seq,
                                   int32_t *__restrict__ row_len, int32_t *__restrict__ row_cnt, int32_t *err)
{
    griddep_launch_dependents();
    griddep_wait();
    const bool ordered = !cu_seqlens_q || offsets_in_order(cu_seqlens_q, num_seqs);
    const int32_t r = blockIdx.x * blockDim.x + threadIdx.x;
    if (r >= num_rows) return;
    int32_t lo = 0, r0 = 0, r1 = 0;
    if (cu_seqlens_q) {
        int32_t hi = num_seqs;  // the last b with cu_seqlens_q[b] <= r
        while (hi - lo > 1) {
            const int32_t mid = (lo + hi) >> 1;
            if (__ldg(cu_seqlens_q + mid) <= r)
                lo = mid;
            else
                hi = mid;
        }
        r0 = __ldg(cu_seqlens_q + lo);
        r1 = __ldg(cu_seqlens_q + lo + 1);
    } else {
        lo = min(r / new_per_seq, num_seqs - 1);
        r0 = lo * new_per_seq;
        r1 = r0 + new_per_seq;
    }
    const int32_t L = __ldg(context_lens + lo);
    const int32_t n = r1 - r0, i = r - r0;
    const bool inside = ordered && r0 <= r && r < r1;
    const bool ok = (!cu_seqlens_q || __ldg(cu_seqlens_q) == 0) && inside && n <= L && n <= max_new && r1 <= num_rows;
    if (!ok) flag_error(err, PKV_ERR_CONTEXT_RANGE);
    int32_t cnt = 1, len = 0;  // a row outside its sequence's range: an entry of its own, zero output
    if (inside) {
        cnt = i % chunk == 0 ? min(min(chunk, n - i), num_rows - r) : 0;  // never past the last row
        len = ok && cnt > 0 ? L - n + i + cnt : 0;
    }
    row_seq[r] = lo;
    row_len[r] = len;
    row_cnt[r] = cnt;
}

// The same for query-split int8 calls, whose entries are numbered without gaps to speak of: sequence b's chunks
// are entries cu_seqlens_q[b] / chunk + b on (room for the ceil(n / chunk) chunks of its n rows; entries that are no
// chunk have row_cnt = 0), num_rows / chunk + num_seqs of them.  One thread per entry and per row: the entry's
// thread finds its sequence by binary search and writes the entry (row0: the row of its first query), the row's
// thread checks that the row lies in a consistent sequence and else writes zeros to its output (every row's, when the
// offsets decrease anywhere).
__global__ void expand_entries_kernel(const int32_t *__restrict__ cu_seqlens_q, int32_t new_per_seq,
                                      const int32_t *__restrict__ context_lens, int32_t num_seqs, int32_t num_rows,
                                      int32_t num_entries, int32_t chunk, int32_t max_new, int32_t len_limit,
                                      int32_t row_values, int32_t *__restrict__ row_seq, int32_t *__restrict__ row_len,
                                      int32_t *__restrict__ row_cnt, int32_t *__restrict__ row0,
                                      uint16_t *__restrict__ out, int32_t *err)
{
    griddep_launch_dependents();
    griddep_wait();
    const bool ordered = !cu_seqlens_q || offsets_in_order(cu_seqlens_q, num_seqs);
    const int32_t x = blockIdx.x * blockDim.x + threadIdx.x;
    auto start = [&](int32_t b) { return cu_seqlens_q ? __ldg(cu_seqlens_q + b) : b * new_per_seq; };
    // the last b whose key is at most v (keys of consistent offsets are non-decreasing)
    auto find = [&](int32_t v, bool entries) {
        int32_t lo = 0, hi = num_seqs;
        while (hi - lo > 1) {
            const int32_t mid = (lo + hi) >> 1;
            if ((entries ? max(start(mid), 0) / chunk + mid : start(mid)) <= v)
                lo = mid;
            else
                hi = mid;
        }
        return lo;
    };
    auto consistent = [&](int32_t b, int32_t r0, int32_t r1) {
        const int32_t L = __ldg(context_lens + b);
        return ordered && start(0) == 0 && r0 >= 0 && r0 <= r1 && r1 <= num_rows && r1 - r0 <= L &&
               r1 - r0 <= max_new && L <= len_limit;
    };
    if (x < num_entries) {
        const int32_t b = find(x, true), r0 = start(b), r1 = start(b + 1);
        const int32_t i = x - (max(r0, 0) / chunk + b);
        int32_t cnt = 0, len = 0;
        if (i >= 0 && consistent(b, r0, r1) && int64_t(i) * chunk < r1 - r0) {
            cnt = min(chunk, r1 - r0 - i * chunk);
            len = __ldg(context_lens + b) - (r1 - r0) + i * chunk + cnt;
        }
        row_seq[x] = b;
        row_len[x] = len;
        row_cnt[x] = cnt;
        row0[x] = cnt > 0 ? r0 + i * chunk : 0;
    }
    if (x < num_rows) {
        const int32_t b = find(x, false), r0 = start(b), r1 = start(b + 1);
        if (!(r0 <= x && x < r1 && consistent(b, r0, r1))) {
            flag_error(err, PKV_ERR_CONTEXT_RANGE);
            uint4 *o = reinterpret_cast<uint4 *>(out + int64_t(x) * row_values);
            for (int32_t k = 0; k < row_values / 8; ++k) o[k] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
}

inline size_t rows_bytes(int32_t num_rows) { return align256(size_t(num_rows) * 4); }

// Queries per warp: as many as keep its qg * G virtual heads within the rows
// of the MMA tile it uses: 8 for a regular CTA (same-n entries), 16 for a
// query-split one.  A query-split entry holds the queries of all team_warps
// warps of its CTA.
inline int32_t chunk_queries(int32_t num_q_heads, int32_t num_kv_heads, int32_t rows = 8)
{
    return std::max(1, rows / (num_q_heads / num_kv_heads));
}

inline int32_t qs_queries(int32_t num_q_heads, int32_t num_kv_heads)
{
    return chunk_queries(num_q_heads, num_kv_heads, 16);
}

inline int32_t entry_queries(int32_t num_q_heads, int32_t num_kv_heads)
{
    const int32_t qg = qs_queries(num_q_heads, num_kv_heads);
    return qg * team_warps(qg * (num_q_heads / num_kv_heads));
}

}  // namespace pkv

extern "C" size_t pkv_paged_attention_workspace_size(int32_t num_rows, int32_t num_q_heads, int32_t num_kv_heads,
                                                     int32_t head_dim)
{
    const size_t base = pkv_paged_decode_workspace_size(num_rows, num_q_heads, num_kv_heads, head_dim);
    if (base == 0) return 0;
    // decode workspace: same-n calls (entries of n <= qg queries, n * G virtual heads), or one
    // chunk entry per row (qg * G virtual heads a warp, on a regular or a query-split CTA); then the
    // three row arrays
    const int32_t gq = num_q_heads / num_kv_heads, qg = qs_queries(num_q_heads, num_kv_heads);
    size_t dec = std::max(base, ws_layout(num_rows, gq * qg, num_kv_heads, head_dim, true).total);
    for (int32_t qn = 2; qn <= qg; ++qn)
        dec = std::max(dec, ws_layout(num_rows, gq * qn, num_kv_heads, head_dim).total);
    return align256(dec) + 3 * rows_bytes(num_rows);
}

// What a query-split int8 call of this many entries takes: pieces of 16-row blocks whatever the group, then four
// arrays of the entries.
static size_t i8_entries_bytes(int32_t entries, int32_t num_kv_heads, int32_t head_dim)
{
    return align256(ws_layout(entries, 16, num_kv_heads, head_dim, true).total) + align256(size_t(entries) * 16);
}

extern "C" size_t pkv_paged_attention_i8_workspace_size(int32_t num_rows, int32_t num_q_heads, int32_t num_kv_heads,
                                                        int32_t head_dim)
{
    const size_t base = pkv_paged_attention_workspace_size(num_rows, num_q_heads, num_kv_heads, head_dim);
    if (base == 0 || num_q_heads / num_kv_heads > 16) return base;
    return std::max(base, i8_entries_bytes(num_rows, num_kv_heads, head_dim));  // (at most an entry a row)
}

// Shared by the bf16 and the int8 entry points (scales: the latter's).
static pkv_status attention_call(int ct, const uint16_t *q, const void *k_cache, const void *v_cache,
                                 const float *scales, const int32_t *block_tables, int32_t max_blocks_per_seq,
                                 const int32_t *cu_seqlens_q, const int32_t *context_lens, int32_t num_seqs,
                                 int32_t num_rows, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                 int32_t block_size, int32_t num_blocks, int32_t max_context_len, float scale,
                                 uint16_t *out, int32_t new_per_seq, void *workspace, size_t workspace_bytes,
                                 int32_t num_workers, int32_t *err_word, pkv_stream_t stream,
                                 const MaskArgs *mask = nullptr)
{
    if (num_seqs < 0 || num_rows < 0 || new_per_seq < 0) return PKV_EINVAL;
    if (num_rows == 0) return PKV_OK;
    if (num_seqs == 0 || !context_lens || (new_per_seq == 0 && !cu_seqlens_q)) return PKV_EINVAL;
    if (new_per_seq > 0 && int64_t(num_seqs) * new_per_seq != num_rows) return PKV_EINVAL;
    if (num_kv_heads <= 0 || num_q_heads <= 0 || num_q_heads % num_kv_heads != 0) return PKV_EINVAL;
    if (ct == kI8 || mask) {  // decode_call's refusals that need no more than the arguments: a refused call writes nothing
        if (head_dim <= 0 || block_size <= 0 || num_blocks <= 0 || max_blocks_per_seq <= 0 || max_context_len < 0 ||
            num_workers < 0 || !std::isfinite(scale))
            return PKV_EINVAL;
        if ((head_dim != 64 && head_dim != 128) || num_q_heads / num_kv_heads > 16 || !is_pow2(block_size) ||
            block_size < (ct == kI8 ? kScaleToks : 8) || block_size > 1024)
            return PKV_EUNSUPPORTED;
        if (num_workers > PKV_MAX_WORKERS || int64_t(num_blocks) * block_size > INT32_MAX) return PKV_EBOUNDS;
        if (!q || !k_cache || !v_cache || (ct == kI8 && !scales) || !block_tables || !out || !aligned16(q) ||
            !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
            (reinterpret_cast<uintptr_t>(scales) & 7u))
            return PKV_EINVAL;
    }
    const int64_t len_max = std::min<int64_t>(max_context_len, int64_t(max_blocks_per_seq) * std::max(block_size, 0));
    if (mask && len_max > kMaskMaxLen) return PKV_EBOUNDS;
    const int32_t max_new = mask && mask->tree ? int32_t(std::min<int64_t>(32LL * mask->tree_words, INT32_MAX)) : INT32_MAX;
    const size_t need = pkv_paged_attention_workspace_size(num_rows, num_q_heads, num_kv_heads, head_dim);
    if (mask && workspace_bytes < pkv_paged_attention_i8_workspace_size(num_rows, num_q_heads, num_kv_heads, head_dim))
        return PKV_EWORKSPACE;
    if (need == 0) return num_rows > PKV_MAX_SEQS ? PKV_EBOUNDS : PKV_EINVAL;
    if (!workspace || workspace_bytes < need || !aligned16(workspace)) return PKV_EWORKSPACE;
    // Up to qg queries of a sequence fit one regular CTA warp's MMA tile (qg * G <= 16 virtual heads):
    // the CTA's warps split the K/V tokens, as in decode.  Longer runs of new tokens go to query-split
    // CTAs, whose warps split an entry of up to 8 * qg queries and share every K/V tile.
    const int32_t qg = qs_queries(num_q_heads, num_kv_heads);
    if (new_per_seq > (mask ? 0 : 1) && new_per_seq <= qg)
        // every sequence's n new tokens share its K/V stream: read once, n * G virtual heads
        return decode_call(ct, false, new_per_seq, q, k_cache, v_cache, nullptr, nullptr, nullptr, nullptr,
                           block_tables, max_blocks_per_seq, context_lens, num_seqs, num_q_heads, num_kv_heads,
                           head_dim, block_size, num_blocks, max_context_len, scale, out, workspace,
                           workspace_bytes, num_workers, err_word, stream, nullptr, nullptr, nullptr, scales,
                           nullptr, -1, mask);
    // chunks of a sequence's queries, one entry per row; few new tokens per sequence on average (at
    // most two regular chunks): chunks of qg on regular CTAs, else chunks of 8 * qg on query-split ones.
    // The row arrays sit after the decode workspace.
    // (Query-split int8 entries, and those of masked calls, fill the tensor-memory tile: as many whole queries as 128
    // rows hold.)
    const int32_t tile = 128 / std::min(num_q_heads / num_kv_heads, 128);
    // (Masked calls over bf16 caches: mask_tile_kernel reads the keys once, at any number of new tokens, and its results
    // repeat bit for bit.  With two parts to a weight, 64 sequences of 512-4096, 16 / 8 heads of 128: 12 nodes each 120 us
    // against 224 on regular CTAs, 1 to 4 nodes 116 against 118, under a window of 1024 60 against 65; two sequences of 9
    // nodes 26 against 159; but 256 sequences of 50-300 with 1 to 4 nodes 63 against 55.)
    const bool few = int64_t(num_rows) <= 2 * int64_t(qg) * num_seqs;
    bool qs = (mask && ct == kBf16) || !few;
    if (ct == kI8 && !qs && int64_t(num_rows) > int64_t(qg) * num_seqs) {
        // Between one and two chunks a sequence: regular CTAs read the keys twice, but take larger calls as fast; in
        // calls of few tiles their list, one entry a row, most of them empty, costs more (16 new tokens, 16 / 8 heads
        // of 128: 5 sequences of 200 tokens 48 -> 16 us, of 2000 59 -> 40 us, 32 of 300 43 -> 38 us; 64 of 2000 would
        // take 111 us against 106).
        DeviceInfo dev;
        if (!current_device_info(&dev)) return PKV_ECUDA;
        const int64_t tiles = int64_t(num_seqs) * num_kv_heads *
                              ((seen_bound(mask, len_max, 2 * qg) + kTc5Keys - 1) / kTc5Keys);
        qs = tiles < 8 * int64_t(dev.sm_count) && num_rows / tile + num_seqs <= num_rows;
    }
    // (entries of a query-split int8 call; without room for their pieces the call takes regular CTAs)
    const int64_t entries = int64_t(num_rows) / tile + num_seqs;
    if (ct == kI8 && qs)
        qs = entries <= num_rows && workspace_bytes >= i8_entries_bytes(int32_t(entries), num_kv_heads, head_dim);
    const int32_t chunk = !qs ? qg : ct == kI8 || mask ? tile : entry_queries(num_q_heads, num_kv_heads);
    uint8_t *wsb = static_cast<uint8_t *>(workspace);
    int64_t live = -1;
    if (ct == kI8 || mask) {  // the rest of decode_call's refusals, before the list is laid out
        const int G = num_q_heads / num_kv_heads * qg, hg = head_group(num_kv_heads, G);
        live = std::min<int64_t>(num_rows, int64_t(num_rows) / chunk + num_seqs);
        if (mask && qs && ct == kBf16) {  // (a segment's list counts a few units more there)
            if (live * num_kv_heads * ((seen_bound(mask, len_max, tile) + kMtKeys - 1) / kMtKeys + 8) > INT32_MAX)
                return PKV_EBOUNDS;
        } else if (unit_bound(ct, qs, G, num_kv_heads, live, len_max, mask, chunk) > INT32_MAX) {
            return PKV_EBOUNDS;
        }
        DeviceInfo dev;
        if (!current_device_info(&dev)) return PKV_ECUDA;
        const bool i8 = ct == kI8;
        if (!qs && cta_layout(head_dim, G, i8 ? 1 : 2, hg, warp_slices(G, hg), 2, num_rows, false, false,
                              one_q_buffer_ok(G, i8, false, false) ? 1 : 2, i8).total > uint32_t(dev.max_smem_optin))
            return PKV_EUNSUPPORTED;
        if (qs && !i8) {
            const int32_t n = mask_tile_entries(num_seqs, num_rows, new_per_seq, tile);
            if (!mask_tile_fits(head_dim, n, new_per_seq == 0, dev.max_smem_optin)) return PKV_EUNSUPPORTED;
            DecodeParams p{};
            p.q = q;
            p.block_tables = block_tables;
            p.context_lens = context_lens;
            p.out = out;
            p.err = err_word;
            p.Hq = num_q_heads;
            p.Hkv = num_kv_heads;
            p.gq = num_q_heads / num_kv_heads;
            p.bs = block_size;
            p.log2_bs = ilog2(block_size);
            p.NB = num_blocks;
            p.max_blocks = max_blocks_per_seq;
            p.len_limit = int32_t(len_max);
            p.scale_log2 = float(double(scale) * 1.4426950408889634);
            p.toks = kMtKeys;
            set_mask(p, *mask);
            // (few new tokens: two parts to a weight, as on the regular CTAs that take such calls without masks.  One part:
            // 12 nodes each 115 us, so 120; 1 to 4 nodes 112, so 116, under a window 55, so 60; 256 short sequences 50, so
            // 63.  Long runs with two parts: 32-node trees 106 us, so 110; 64-token chunks 61, so 67; prompts 50, so 59.)
            return mask_tile_call(p, k_cache, v_cache, cu_seqlens_q, num_seqs, num_rows, new_per_seq, max_new, few,
                                  head_dim, wsb, num_workers, reinterpret_cast<cudaStream_t>(stream));
        }
    }
    if (ct == kI8 && qs) {
        const size_t dec_bytes = i8_entries_bytes(int32_t(entries), num_kv_heads, head_dim) -
                                 align256(size_t(entries) * 16);
        int32_t *row_seq = reinterpret_cast<int32_t *>(wsb + dec_bytes), *row_len = row_seq + entries,
                *row_cnt = row_len + entries, *row0 = row_cnt + entries;
        const int32_t len_limit = int32_t(len_max);
        const cudaError_t e = launch_pdl(expand_entries_kernel, dim3((num_rows + 255) / 256), dim3(256), 0,
                                         reinterpret_cast<cudaStream_t>(stream),
                                         new_per_seq > 0 ? nullptr : cu_seqlens_q, new_per_seq, context_lens, num_seqs,
                                         num_rows, int32_t(entries), chunk, max_new, len_limit,
                                         num_q_heads * head_dim, row_seq, row_len, row_cnt, row0, out, err_word);
        if (e != cudaSuccess) {
            cudaGetLastError();
            return cuda_fail("expand_entries_kernel launch", e);
        }
        const pkv_status st = launch_status("expand_entries_kernel launch");
        if (st != PKV_OK) return st;
        return decode_call(ct, true, qg, q, k_cache, v_cache, nullptr, nullptr, row_seq, row_cnt, block_tables,
                           max_blocks_per_seq, row_len, int32_t(entries), num_q_heads, num_kv_heads, head_dim, block_size,
                           num_blocks, max_context_len, scale, out, workspace, dec_bytes, num_workers, err_word, stream,
                           nullptr, nullptr, nullptr, scales, row0, live, mask);
    }
    const size_t dec_bytes = need - 3 * rows_bytes(num_rows);
    int32_t *row_seq = reinterpret_cast<int32_t *>(wsb + dec_bytes);
    int32_t *row_len = reinterpret_cast<int32_t *>(wsb + dec_bytes + rows_bytes(num_rows));
    int32_t *row_cnt = reinterpret_cast<int32_t *>(wsb + dec_bytes + 2 * rows_bytes(num_rows));
    const cudaError_t e = launch_pdl(expand_rows_kernel, dim3((num_rows + 255) / 256), dim3(256), 0,
                                     reinterpret_cast<cudaStream_t>(stream), new_per_seq > 0 ? nullptr : cu_seqlens_q,
                                     new_per_seq, context_lens, num_seqs, num_rows, chunk, max_new, row_seq,
                                     row_len, row_cnt, err_word);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return cuda_fail("expand_rows_kernel launch", e);
    }
    const pkv_status st = launch_status("expand_rows_kernel launch");
    if (st != PKV_OK) return st;
    return decode_call(ct, qs, qg, q, k_cache, v_cache, nullptr, nullptr, row_seq, row_cnt, block_tables,
                       max_blocks_per_seq, row_len, num_rows, num_q_heads, num_kv_heads, head_dim, block_size,
                       num_blocks, max_context_len, scale, out, workspace, dec_bytes, num_workers, err_word, stream,
                       nullptr, nullptr, nullptr, scales, nullptr, live, mask);
}

extern "C" pkv_status pkv_paged_attention(const uint16_t *q, const uint16_t *k_cache, const uint16_t *v_cache,
                                          const int32_t *block_tables, int32_t max_blocks_per_seq,
                                          const int32_t *cu_seqlens_q, const int32_t *context_lens, int32_t num_seqs,
                                          int32_t num_rows, int32_t num_q_heads, int32_t num_kv_heads,
                                          int32_t head_dim, int32_t block_size, int32_t num_blocks,
                                          int32_t max_context_len, float scale, uint16_t *out, int32_t new_per_seq,
                                          void *workspace, size_t workspace_bytes, int32_t num_workers,
                                          int32_t *err_word, pkv_stream_t stream)
{
    return attention_call(kBf16, q, k_cache, v_cache, nullptr, block_tables, max_blocks_per_seq, cu_seqlens_q,
                          context_lens, num_seqs, num_rows, num_q_heads, num_kv_heads, head_dim, block_size,
                          num_blocks, max_context_len, scale, out, new_per_seq, workspace, workspace_bytes,
                          num_workers, err_word, stream);
}

extern "C" pkv_status pkv_paged_attention_i8(const uint16_t *q, const int8_t *k_cache, const int8_t *v_cache,
                                             const float *scales, const int32_t *block_tables,
                                             int32_t max_blocks_per_seq, const int32_t *cu_seqlens_q,
                                             const int32_t *context_lens, int32_t num_seqs, int32_t num_rows,
                                             int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                             int32_t block_size, int32_t num_blocks, int32_t max_context_len,
                                             float scale, uint16_t *out, int32_t new_per_seq, void *workspace,
                                             size_t workspace_bytes, int32_t num_workers, int32_t *err_word,
                                             pkv_stream_t stream)
{
    return attention_call(kI8, q, k_cache, v_cache, scales, block_tables, max_blocks_per_seq, cu_seqlens_q,
                          context_lens, num_seqs, num_rows, num_q_heads, num_kv_heads, head_dim, block_size,
                          num_blocks, max_context_len, scale, out, new_per_seq, workspace, workspace_bytes,
                          num_workers, err_word, stream);
}

// ------------------------------------------------------------------ sliding windows with sinks, trees
extern "C" pkv_status pkv_paged_decode_window(
    const uint16_t *q, const uint16_t *k_cache, const uint16_t *v_cache, const int32_t *block_tables,
    int32_t max_blocks_per_seq, const int32_t *context_lens, int32_t num_seqs, int32_t num_q_heads,
    int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t num_blocks, int32_t max_context_len,
    float scale, int32_t window, int32_t sinks, uint16_t *out, void *workspace, size_t workspace_bytes,
    int32_t num_workers, int32_t *err_word, pkv_stream_t stream)
{
    MaskArgs m;
    m.window = window;
    m.sinks = sinks;
    if (const pkv_status st = check_mask(m, false); st != PKV_OK) return st;
    return decode_call(kBf16, false, 1, q, k_cache, v_cache, nullptr, nullptr, nullptr, nullptr, block_tables,
                       max_blocks_per_seq, context_lens, num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                       num_blocks, max_context_len, scale, out, workspace, workspace_bytes, num_workers, err_word,
                       stream, nullptr, nullptr, nullptr, nullptr, nullptr, -1, &m);
}

extern "C" pkv_status pkv_paged_decode_window_fp8(
    const uint16_t *q, const uint8_t *k_cache, const uint8_t *v_cache, const float *k_scale, const float *v_scale,
    const int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *context_lens, int32_t num_seqs,
    int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t num_blocks,
    int32_t max_context_len, float scale, int32_t window, int32_t sinks, uint16_t *out, void *workspace,
    size_t workspace_bytes, int32_t num_workers, int32_t *err_word, pkv_stream_t stream)
{
    MaskArgs m;
    m.window = window;
    m.sinks = sinks;
    if (const pkv_status st = check_mask(m, false); st != PKV_OK) return st;
    return decode_call(kE4m3, false, 1, q, k_cache, v_cache, k_scale, v_scale, nullptr, nullptr, block_tables,
                       max_blocks_per_seq, context_lens, num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                       num_blocks, max_context_len, scale, out, workspace, workspace_bytes, num_workers, err_word,
                       stream, nullptr, nullptr, nullptr, nullptr, nullptr, -1, &m);
}

extern "C" pkv_status pkv_paged_decode_window_i8(
    const uint16_t *q, const int8_t *k_cache, const int8_t *v_cache, const float *scales,
    const int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *context_lens, int32_t num_seqs,
    int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t num_blocks,
    int32_t max_context_len, float scale, int32_t window, int32_t sinks, uint16_t *out, void *workspace,
    size_t workspace_bytes, int32_t num_workers, int32_t *err_word, pkv_stream_t stream)
{
    MaskArgs m;
    m.window = window;
    m.sinks = sinks;
    if (const pkv_status st = check_mask(m, false); st != PKV_OK) return st;
    return decode_call(kI8, false, 1, q, k_cache, v_cache, nullptr, nullptr, nullptr, nullptr, block_tables,
                       max_blocks_per_seq, context_lens, num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                       num_blocks, max_context_len, scale, out, workspace, workspace_bytes, num_workers, err_word,
                       stream, nullptr, nullptr, nullptr, scales, nullptr, -1, &m);
}

extern "C" pkv_status pkv_paged_attention_window(
    const uint16_t *q, const uint16_t *k_cache, const uint16_t *v_cache, const int32_t *block_tables,
    int32_t max_blocks_per_seq, const int32_t *cu_seqlens_q, const int32_t *context_lens, int32_t num_seqs,
    int32_t num_rows, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
    int32_t num_blocks, int32_t max_context_len, float scale, int32_t window, int32_t sinks, uint16_t *out,
    int32_t new_per_seq, void *workspace, size_t workspace_bytes, int32_t num_workers, int32_t *err_word,
    pkv_stream_t stream)
{
    MaskArgs m;
    m.new_tokens = true;
    m.window = window;
    m.sinks = sinks;
    if (const pkv_status st = check_mask(m, false); st != PKV_OK) return st;
    return attention_call(kBf16, q, k_cache, v_cache, nullptr, block_tables, max_blocks_per_seq, cu_seqlens_q,
                          context_lens, num_seqs, num_rows, num_q_heads, num_kv_heads, head_dim, block_size,
                          num_blocks, max_context_len, scale, out, new_per_seq, workspace, workspace_bytes,
                          num_workers, err_word, stream, &m);
}

extern "C" pkv_status pkv_paged_attention_window_i8(
    const uint16_t *q, const int8_t *k_cache, const int8_t *v_cache, const float *scales,
    const int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *cu_seqlens_q,
    const int32_t *context_lens, int32_t num_seqs, int32_t num_rows, int32_t num_q_heads, int32_t num_kv_heads,
    int32_t head_dim, int32_t block_size, int32_t num_blocks, int32_t max_context_len, float scale, int32_t window,
    int32_t sinks, uint16_t *out, int32_t new_per_seq, void *workspace, size_t workspace_bytes, int32_t num_workers,
    int32_t *err_word, pkv_stream_t stream)
{
    MaskArgs m;
    m.new_tokens = true;
    m.window = window;
    m.sinks = sinks;
    if (const pkv_status st = check_mask(m, false); st != PKV_OK) return st;
    return attention_call(kI8, q, k_cache, v_cache, scales, block_tables, max_blocks_per_seq, cu_seqlens_q,
                          context_lens, num_seqs, num_rows, num_q_heads, num_kv_heads, head_dim, block_size,
                          num_blocks, max_context_len, scale, out, new_per_seq, workspace, workspace_bytes,
                          num_workers, err_word, stream, &m);
}

extern "C" pkv_status pkv_paged_attention_tree(
    const uint16_t *q, const uint16_t *k_cache, const uint16_t *v_cache, const int32_t *block_tables,
    int32_t max_blocks_per_seq, const int32_t *cu_seqlens_q, const int32_t *context_lens, int32_t num_seqs,
    int32_t num_rows, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
    int32_t num_blocks, int32_t max_context_len, float scale, const int32_t *tree_mask, int32_t mask_words,
    uint16_t *out, int32_t new_per_seq, void *workspace, size_t workspace_bytes, int32_t num_workers,
    int32_t *err_word, pkv_stream_t stream)
{
    if (num_rows > 0 && !tree_mask) return PKV_EINVAL;
    MaskArgs m;
    m.new_tokens = true;
    m.tree = reinterpret_cast<const uint32_t *>(tree_mask);
    m.tree_words = mask_words;
    m.tree_n = new_per_seq;
    m.tree_lens = context_lens;
    m.tree_cu = cu_seqlens_q;
    if (const pkv_status st = check_mask(m, true); st != PKV_OK) return st;
    return attention_call(kBf16, q, k_cache, v_cache, nullptr, block_tables, max_blocks_per_seq, cu_seqlens_q,
                          context_lens, num_seqs, num_rows, num_q_heads, num_kv_heads, head_dim, block_size,
                          num_blocks, max_context_len, scale, out, new_per_seq, workspace, workspace_bytes,
                          num_workers, err_word, stream, &m);
}

extern "C" pkv_status pkv_paged_attention_tree_i8(
    const uint16_t *q, const int8_t *k_cache, const int8_t *v_cache, const float *scales,
    const int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *cu_seqlens_q,
    const int32_t *context_lens, int32_t num_seqs, int32_t num_rows, int32_t num_q_heads, int32_t num_kv_heads,
    int32_t head_dim, int32_t block_size, int32_t num_blocks, int32_t max_context_len, float scale,
    const int32_t *tree_mask, int32_t mask_words, uint16_t *out, int32_t new_per_seq, void *workspace,
    size_t workspace_bytes, int32_t num_workers, int32_t *err_word, pkv_stream_t stream)
{
    if (num_rows > 0 && !tree_mask) return PKV_EINVAL;
    MaskArgs m;
    m.new_tokens = true;
    m.tree = reinterpret_cast<const uint32_t *>(tree_mask);
    m.tree_words = mask_words;
    m.tree_n = new_per_seq;
    m.tree_lens = context_lens;
    m.tree_cu = cu_seqlens_q;
    if (const pkv_status st = check_mask(m, true); st != PKV_OK) return st;
    return attention_call(kI8, q, k_cache, v_cache, scales, block_tables, max_blocks_per_seq, cu_seqlens_q,
                          context_lens, num_seqs, num_rows, num_q_heads, num_kv_heads, head_dim, block_size,
                          num_blocks, max_context_len, scale, out, new_per_seq, workspace, workspace_bytes,
                          num_workers, err_word, stream, &m);
}
