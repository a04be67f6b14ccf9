// Masked attention for several new tokens per sequence on the 5th-generation tensor cores: sliding windows with sinks
// and trees of drafted tokens over bf16 caches, but for calls whose sequences' new tokens all fit one pass of the decode
// kernel (see attention_call).
//
// An entry is up to 128 / gq consecutive queries of a sequence; with the gq query heads of a kv head they are the up to
// 128 rows of a tile (row r: query r / gq, head r % gq).  A unit is 64 keys of an (entry, kv head) segment; the unit
// list leaves out what no query of the entry sees (seen_units).  Per unit
//     S = Q K^T  (128 x 64, fp32 in tensor memory),   P = 2^(c S - m),   O += P V  (128 x D, fp32 in tensor memory)
// with m the row's running max, moved only when a score passes it by kRescaleSlack (O is then scaled in place), and
// out = O / l at the segment's end, l the fp32 sum of the weights.  P enters the product as bf16, the operand type of V:
// in calls of few new tokens as two parts (TWO), bf16(p) and bf16 of what that leaves, in the columns that the scores had
// (2^-16 of a weight at most, as the decode kernel's); in longer ones as one (2^-8), as the tensor-memory CTAs take it in
// calls without masks (see attention_call).
//
// Why this shape: one unit's chain of copy, product, softmax and product has far more latency than work, so two CTAs
// share an SM, each with its own segments, half the tensor memory (two score buffers of 64 columns and the output: 256
// columns) and half the shared memory; a row belongs to one thread, so the softmax needs no word between threads.  K
// and V tiles of 64 keys come through one ring of slots in the order the products use them (K0 K1 V0 K2 V1 ...), from
// any page size, a copy for each page and 64-dim half; Q is one copy of a box of queries x heads.
//
// Warps: 0-3 softmax (thread t is row t of the tile and TMEM lane t), 4 issues the products (one thread), 5 the copies
// of K and V.  Ordering (unit k of the CTA's list, buffer k % 2): copy landed -> full[slot]; scores -> sfull[k % 2] and
// the K slot free (commits); weights written, over their scores -> pfull[k % 2][half] (4 warps); output product ->
// odone[k % 2] and the V slot free; a segment's Q landed -> qready (its copy is issued once the last scores that read
// the one before are in).  S(k) is issued when P(k - 2) V is done, P(k - 1) V after S(k), or before it where unit k
// opens a segment.  The weights go out 32 keys at a time, so that the first half's product runs beside the second
// half's exponentials (32-node trees of 64 sequences, one call after another on the same inputs, 106.4 us, so 104.7).
// Every barrier's next phase needs its waiter's own next step, so none runs two phases ahead; the softmax warps, which
// see only some V tiles, look at their barrier after the unit's scores, which come behind the slot's item before.
//
// The list is cut into equal slices, one a CTA.  Slices, and with them the sums' order, depend on the list and the grid
// alone: the results repeat bit for bit.  Pieces of a segment that lies in several slices are merged
//   - by the CTA that completes it (MERGE).  A piece costs its CTA two meetings of its warps, a fence and a counter,
//     and the last one a trip through L2 for every other piece, so bounds move to a segment's start or end that is near;
//   - or, where segments are few and their pieces many, by a second kernel (mask_merge_kernel): the merges of one CTA
//     would come one after another (25 nodes over one sequence of 30000 tokens, 38 pieces a segment: 125 us, so
//     43 us; of four sequences of 512-4096 34 us, so 26).  With many segments the second kernel's start would cost more
//     than the merges do (64 sequences: 64-token chunks 66 us, so 78; 32-node trees 110 and 120).
// Where segments are short, slices end at their starts and there is nothing to merge.  The copying warp walks the list
// and hands each segment to the others in shared memory (MtDesc), the next one before it copies the last unit of this
// one.
//
// What bounds it (64 sequences of 512-4096, 16 / 8 heads of 128, 1.95 GHz; calls whose inputs come from memory; the steps
// above and at the constants are from calls at other stages): 32-node trees, 596 MB, 110 us of 87.7 at the copy rate;
// 64-token chunks under a window of 1024, 62.7 us of 45; whole prompts of 1-2048 tokens under a window of 512, 54 us of
// 15 at the products' rate.  A unit takes a CTA 2000-2200 cycles: softmax 1000, a wait of 500-900 for the next scores,
// which share one tensor pipe with the other CTA's products and wait for the output product that reads the same columns,
// masks and instruction fetch 400.  Tensor memory holds no third score buffer at head_dim 128.  A segment's end costs
// 5000 to 7000 cycles: its last product, 128 rows of 256 bytes, the first unit's masks.  Where segments are not cut,
// slices are uneven: a bound moves to its segment's start, and the fullest of 304 CTAs has 51 to 57 places of the list in
// the chunks (mean 36.8) and 52 to 54 in the prompts (mean 41.9).
#include "pkv_decode_kernel.cuh"

namespace pkv {

constexpr int kMtSoftmaxWarps = 4;
constexpr int kMtThreads = 32 * (kMtSoftmaxWarps + 2);
constexpr uint32_t kMtSlab = kMtKeys * 128;   // one 64-dim half of a K or V tile: 64 rows of 128 bytes
constexpr uint32_t kMtQSlab = 128 * 128;      // one 64-dim half of Q
constexpr uint32_t kMtCols = 256, kMtOCol = 128;
constexpr int kMtMaxSlots = 8, kMtDescs = 4;
// A slice of the unit list is at least this long: a piece costs its CTA and its merge about as much as a few units.
constexpr int kMtMinSlice = 4;
// What a segment's start and end cost, in units (see MtSeg).
constexpr int kMtSegCost = 4;
// A slice's bound this near to a segment's start or end, in units, moves there: MERGE (none: 73 us the 64-token chunks
// under a 1024 window, 6 or 8: 66), and where a second kernel merges.
constexpr int kMtSnap = 8, kMtSnapFew = 1;
// Segments of at most this many units are not cut: bounds move to their starts.  More where there is a segment for
// every CTA (the 64-token chunks, 17 units a segment: 65.5 us, so 63.3).
constexpr int kMtWhole = 12, kMtWholeMany = 20;
// CTAs over segments from which on a second kernel merges.
constexpr int kMtFew = 4;

struct TileParams {
    DecodeParams p;       // B: entries, context_lens: by sequence, nst: ring slots, seg_cost, num_workers unused
    const int32_t *cu;    // offsets of the sequences' rows (null: per_seq rows each)
    int32_t num_seqs, num_rows, per_seq;
    int32_t tile;         // queries of an entry
    int32_t per_entry;    // null cu: entries of a sequence
    int32_t max_new;
    int32_t snap;         // see kMtSnap, kMtWhole
    bool ctr_by_row;      // arrival counters by the entry's first row, not by entry
    bool two;             // weights as two bf16 parts, not one (see the head of the file)
    int32_t merge;        // 1: the CTA that completes a segment merges it; 2: a second kernel does; 0: nothing to merge
};

// A segment's part in the CTA's slice, as the softmax warps and the issuing one see it: units u .. u + len - 1 of the n
// of entry b and kv head g (len 0: no more), the segment's start in the list, whether it is the slice's first (see
// mt_piece), and what its entry says.
struct alignas(16) MtDesc {
    int32_t b, g, u, n, len, x0, first, L, cnt, row0, base;
};

struct MtLayout {
    uint32_t off_q, off_bar, off_desc, off_bound, off_tmp, off_scan, off_seq, total;
};

__host__ __device__ inline MtLayout mt_layout(int D, int nslots, int B, bool seqs, bool merge)
{
    MtLayout l;
    uint32_t o = uint32_t(nslots) * uint32_t(kMtKeys * D * 2);
    l.off_q = o;
    o += 128u * uint32_t(D) * 2u;
    l.off_bar = o;
    o += uint32_t(2 * kMtMaxSlots + 12 + 2 * kMtDescs) * 8u;
    l.off_desc = o;
    o += uint32_t(kMtDescs * sizeof(MtDesc));
    l.off_bound = o;
    o += merge ? (kMaxSlots + 1) * 4u : 0u;
    l.off_tmp = o;
    o += 40u * 4u;
    l.off_scan = o;
    o += uint32_t(B + 1) * 4u;
    l.off_seq = o;
    o += seqs ? uint32_t(B) * 2u : 0u;
    l.total = o;
    return l;
}

struct MtSmem {
    uint64_t *full, *empty, *sfull, *pfull, *odone, *qready, *drain, *team;
    uint64_t *dfull, *dempty;  // [kMtDescs] a descriptor written by the copying warp, done with by the others
    struct MtDesc *desc;
    const int32_t *scan;
    const uint16_t *seq;  // entry -> sequence (null: entry / per_entry)
};

// The ring's items: K of a CTA's unit k is item 0 or 2k - 1, V of it 2k + 2 (the item before the last one stays empty).
__device__ __forceinline__ uint32_t mt_kitem(uint32_t k) { return k == 0 ? 0u : 2u * k - 1u; }
__device__ __forceinline__ uint32_t mt_vitem(uint32_t k) { return 2u * k + 2u; }

// A sequence's rows and context length, and whether they fit each other.
struct MtRows {
    int32_t r0, r1, L;
    bool ok;
};

__device__ __forceinline__ MtRows mt_rows(const TileParams &tp, int32_t b)
{
    MtRows r;
    r.r0 = tp.cu ? __ldg(tp.cu + b) : b * tp.per_seq;
    r.r1 = tp.cu ? __ldg(tp.cu + b + 1) : r.r0 + tp.per_seq;
    r.L = __ldg(tp.p.context_lens + b);
    r.ok = r.r0 >= 0 && r.r0 <= r.r1 && r.r1 <= tp.num_rows && r.r1 - r.r0 <= r.L && r.r1 - r.r0 <= tp.max_new &&
           r.L <= tp.p.len_limit;
    return r;
}

// Entry e: its sequence, its queries (cnt of them from row row0 on; 0: no entry), the length its last one sees and the
// sequence's first new position.  Sequence b's entries are numbered from cu[b] / tile + b on (there is room for
// ceil(n / tile) of them), or from b * per_entry on.
struct MtEntry {
    int32_t seq, L, cnt, row0, base;
    bool bad;  // its sequence has rows that do not fit
};

__device__ __forceinline__ MtEntry mt_entry(const TileParams &tp, int32_t e, int32_t seq)
{
    const MtRows r = mt_rows(tp, seq);
    MtEntry en;
    en.seq = seq;
    const int32_t i = tp.cu ? e - (max(r.r0, 0) / tp.tile + seq) : e - seq * tp.per_entry;
    en.cnt = r.ok && i >= 0 && (long long)i * tp.tile < r.r1 - r.r0 ? min(tp.tile, r.r1 - r.r0 - i * tp.tile) : 0;
    en.bad = !r.ok && r.r0 != r.r1;
    en.row0 = r.r0 + i * tp.tile;
    en.base = r.L - (r.r1 - r.r0);
    en.L = en.base + i * tp.tile + en.cnt;
    return en;
}

// List position x < nhg * scan[B]: its entry b, kv head g, place u in the segment and the segment's length n (as
// walker_locate, in 32 bits and without a division).
__device__ __forceinline__ Walker mt_locate(const DecodeParams &p, const int32_t *scan, int32_t x)
{
    int lo = 0, hi = p.B;  // nhg * scan[lo] <= x < nhg * scan[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.nhg * scan[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    Walker w;
    w.b = lo;
    w.n = scan[lo + 1] - scan[lo];
    const int32_t rem = x - p.nhg * scan[lo];
    w.g = int32_t(__fdividef(float(rem), float(w.n)));  // off by one at most (g < nhg is small)
    w.u = rem - w.g * w.n;
    if (w.u < 0) {
        --w.g;
        w.u += w.n;
    } else if (w.u >= w.n) {
        ++w.g;
        w.u -= w.n;
    }
    return w;
}

// A segment's part in a slice of the list: units u .. u + len - 1 of the n of (b, g).  In the list a segment counts
// p.seg_cost more than its units, before the first: what its start and end cost a CTA, so that slices of many short
// segments take no longer than those of few long ones.  x0: the segment's start in the list, next: its end or the
// slice's.  (List positions stay in 32 bits: see attention_call.)
struct MtSeg {
    int32_t b, g, u, n, len, x0, next;
};

// The order in which a CTA takes its slice [lo, hi): from its last segment's start (or lo) on, then from lo; the part of
// a segment that goes on in the next slice is then there early, and the piece that completes a segment comes amid the
// run, not at its end.
struct MtRange {
    int32_t lo, hi, rot;
};

// The first segment from list position x on (in that order) that has units of its own; false: none.
__device__ __forceinline__ bool mt_seg(const DecodeParams &p, const int32_t *scan, const MtRange &r, int32_t x, MtSeg &s)
{
    for (;;) {
        if (x >= r.hi) {
            if (r.rot <= r.lo) return false;
            x = r.lo;
        }
        const Walker w = mt_locate(p, scan, x);
        const int32_t end = min(w.n, w.u + (r.hi - x));
        s.b = w.b;
        s.g = w.g;
        s.n = w.n - p.seg_cost;
        s.u = max(w.u - p.seg_cost, 0);
        s.len = max(end - p.seg_cost, 0) - s.u;
        s.x0 = x - w.u;
        s.next = s.x0 + end;
        if (s.len > 0) return true;
        x = s.next;
        if (x == r.rot && r.rot > r.lo) return false;
    }
}

// The segment after s; false: s was the last.
__device__ __forceinline__ bool mt_next(const DecodeParams &p, const int32_t *scan, const MtRange &r, const MtSeg &s,
                                        MtSeg &n)
{
    if (r.rot > r.lo && s.next == r.rot) return false;
    return mt_seg(p, scan, r, s.next, n);
}

// The slices: nsl of T list positions.
struct MtSlices {
    int32_t T, nsl, each, rest, snap;
    float inv;
};

// One slice a CTA, none much shorter than kMtMinSlice.
__device__ __forceinline__ MtSlices mt_slices(const TileParams &tp, int32_t T, int ctas)
{
    MtSlices q{T, min(ctas, max(1, T / (kMtMinSlice + tp.p.seg_cost))), 0, 0, tp.snap, 0.f};
    q.each = T / q.nsl;
    q.rest = T - q.each * q.nsl;
    q.inv = 1.0f / float(q.nsl);
    return q;
}

// Where slice i begins (i = nsl: the list's end).
__device__ __forceinline__ int32_t mt_bound(const DecodeParams &p, const int32_t *scan, const MtSlices &q, int i)
{
    if (i >= q.nsl) return q.T;
    int32_t x = q.each * i + min(int32_t(float(q.rest * i) * q.inv), q.rest);  // (grows with i, as it should)
    if (i > 0) {
        const Walker w = mt_locate(p, scan, x);
        if (w.u - p.seg_cost <= q.snap)
            x -= w.u;
        else if (w.n - w.u <= q.snap)
            x += w.n - w.u;
    }
    return x;
}

// Slice that holds list position x, from slice s on (mostly that one or the next).
__device__ __forceinline__ int mt_slice_of(const int32_t *bound, int nsl, int s, int32_t x)
{
    for (int i = 0; i < 4; ++i) {
        if (bound[s] > x)
            --s;
        else if (bound[s + 1] <= x)
            ++s;
        else
            return s;
    }
    int lo = 0, hi = nsl;  // bound[lo] <= x < bound[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (bound[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// The largest of three.
__device__ __forceinline__ float mt_max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// A segment's piece of a slice, as tc5_piece_tile, with the entry's first row in the entry's place: entries that have
// rows have different first rows, in the list's order, so a workspace for num_rows entries does, however many sequences
// have no rows.
__device__ __forceinline__ long long mt_piece(const TileParams &tp, int slice, bool slice_first, int32_t row0, int g)
{
    return slots_by_slice(tp.num_rows, tp.p.nhg) ? 2LL * slice + (slice_first ? 0 : 1)
                                                 : slice + (long long)row0 * tp.p.nhg + g;
}

// 32 bytes to a 16-byte aligned place (one store where it is 32-byte aligned).
__device__ __forceinline__ void store32(uint16_t *dst, const uint32_t (&v)[8], bool wide)
{
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]), "r"(v[1]),
                     "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(dst)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4 *>(dst)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}

// 16 columns of a row's output.
__device__ __forceinline__ void mt_store16(uint16_t *dst, const float (&a)[16], bool wide)
{
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = pack_bf16x2(a[2 * i], a[2 * i + 1]);
    store32(dst, v, wide);
}

// A row's output, l > 0 its weights' sum, from the unnormalised sums in tensor memory at `o`.  (A rolled loop: code that
// runs once a segment comes at the pace of its instruction fetch.)
template <int D>
__device__ __forceinline__ void mt_output(float l, uint32_t o, uint16_t *out)
{
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    const bool wide = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += 16) {
        uint32_t r[16];
        tmem_ld16(o + uint32_t(c0), r);
        float a[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) a[j] = __uint_as_float(r[j]) * inv;
        if (out) mt_store16(out + c0, a, wide);
    }
}

// The same where its segment, which starts at list position x0, has other pieces: those that the slices sf..sl but `own`
// left join the row's own state (m, l):
//     M = max m_i,  l = sum 2^(m_i - M) l_i,  out = sum 2^(m_i - M) acc_i / l,
// summed in slice order, products rounded before they are added: the result does not depend on which piece came last.
// Every load is a trip to the other pieces' SMs' side of L2 and nothing else hides it, so (m, l) come four pieces at a
// time and sums, 32 columns a step, a piece ahead.
template <int D>
__device__ __forceinline__ void mt_merge(const TileParams &tp, const int32_t *bound, int sf, int sl, int own, int32_t x0,
                                         int g, int32_t row0, int row, float m, float l, uint32_t o, uint16_t *out)
{
    const DecodeParams &p = tp.p;
    const float2 *ml = reinterpret_cast<const float2 *>(p.ws_ml);
    auto next = [&](int sk) {  // the next slice that is not empty (an empty one left nothing)
        do ++sk;
        while (sk <= sl && bound[sk + 1] <= bound[sk]);
        return sk;
    };
    auto tile_of = [&](int sk) { return mt_piece(tp, sk, x0 <= bound[sk], row0, g); };
    auto state = [&](int sk) { return sk == own || sk > sl ? make_float2(m, l) : __ldcg(ml + tile_of(sk) * 128 + row); };
    const bool wide = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
    const int s0 = next(sf - 1);
    struct Piece {
        float4 v[8];
        float2 st;
    };
    // piece sk's columns c0 .. c0 + 31 (the own one's stay in tensor memory until they are due)
    auto load = [&](Piece &q, int sk, int c0) {
        q.st = state(sk);
        if (sk == own) return;
        const float4 *src = reinterpret_cast<const float4 *>(p.ws_acc + tile_of(sk) * 128 * D) + row;
#pragma unroll
        for (int j = 0; j < 8; ++j) q.v[j] = __ldcg(src + (c0 / 4 + j) * 128);
    };
    Piece q, ahead;
    load(q, s0, 0);
    float M = -INFINITY, L = 0.f;
#pragma unroll 1
    for (int sk = s0; sk <= sl;) {
        float2 st[4];
        bool in[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            st[j] = state(sk);
            in[j] = sk <= sl;
            if (in[j]) sk = next(sk);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float mn = fmaxf(M, st[j].x), at = mn == -INFINITY ? 0.f : mn;
            if (in[j]) {
                L = __fadd_rn(__fmul_rn(L, ex2(M - at)), __fmul_rn(ex2(st[j].x - at), st[j].y));
                M = mn;
            }
        }
    }
    const float at = M == -INFINITY ? 0.f : M, inv = L == 0.f ? 0.f : 1.0f / L;
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += 32) {
        float a[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) a[j] = 0.f;
#pragma unroll 1
        for (int sk = s0; sk <= sl;) {
            const int nk = next(sk);
            const bool step = nk > sl;  // the columns' last piece
            if (!step || c0 + 32 < D) load(ahead, step ? s0 : nk, step ? c0 + 32 : c0);
            const float f = ex2(q.st.x - at) * inv;
            if (sk == own) {
                uint32_t r[32];
                tmem_ld32(o + uint32_t(c0), r);
#pragma unroll
                for (int j = 0; j < 32; ++j) a[j] = __fadd_rn(a[j], __fmul_rn(f, __uint_as_float(r[j])));
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    a[4 * j] = __fadd_rn(a[4 * j], __fmul_rn(f, q.v[j].x));
                    a[4 * j + 1] = __fadd_rn(a[4 * j + 1], __fmul_rn(f, q.v[j].y));
                    a[4 * j + 2] = __fadd_rn(a[4 * j + 2], __fmul_rn(f, q.v[j].z));
                    a[4 * j + 3] = __fadd_rn(a[4 * j + 3], __fmul_rn(f, q.v[j].w));
                }
            }
            q = ahead;
            sk = nk;
        }
        if (out) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float w[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) w[j] = a[16 * h + j];
                mt_store16(out + c0 + 16 * h, w, wide);
            }
        }
    }
}

// Which of the 64 tokens from tok0 on, drafted ones among them, query qi of the entry sees (x, y; none: qi >= cnt), and
// which some query does (z, w).  The rows of one warp are a part of the queries, so a warp looks at all of them, a lane
// at every 32nd, and a row takes its own from the lane that has it: one trip for the masks (a second one for the
// entry's: 256 short sequences of 1 to 4 nodes 58.4 us, so 50.0).
__device__ __forceinline__ uint4 mt_tree_sees(const DecodeParams &p, int32_t tok0, int32_t L, int32_t cnt, int32_t row0,
                                              int32_t base, int qi, int lane)
{
    uint4 s = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
    for (int i0 = 0; i0 < cnt; i0 += 32) {
        uint32_t a = 0u, b = 0u;
        if (i0 + lane < cnt) {
            const uint32_t *mask = p.tree + (long long)(row0 + i0 + lane) * p.tree_words;
            a = row_sees(p, tok0, L - cnt + i0 + lane, base, mask);
            b = row_sees(p, tok0 + 32, L - cnt + i0 + lane, base, mask);
        }
        const uint32_t x = __shfl_sync(kFull, a, qi & 31), y = __shfl_sync(kFull, b, qi & 31);
        if (qi >> 5 == i0 >> 5) {
            s.x = x;
            s.y = y;
        }
        s.z |= a;
        s.w |= b;
    }
    s.z = __reduce_or_sync(kFull, s.z);
    s.w = __reduce_or_sync(kFull, s.w);
    return s;
}

// The softmax warps (see the head of the file).
template <int D, bool MERGE, bool TWO>
__device__ void mt_softmax(const TileParams &tp, const CUtensorMap *qmap, const MtSmem &m, uint8_t *ring, uint8_t *qop,
                           uint32_t tmem, int32_t *bound, int *sh, const MtSlices &sl, uint32_t gen)
{
    const DecodeParams &p = tp.p;
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const uint32_t tlane = tmem + (uint32_t(32 * warp) << 16), ns = uint32_t(p.nst);
    const int qi = t / p.gq, qh = t - qi * p.gq;
    // the row's factor stays positive whatever the scale's sign: the scores take the sign, or are zeros
    const float c = p.scale_log2 == 0.f ? 1.f : fabsf(p.scale_log2);
    const uint32_t sflip = p.scale_log2 < 0.f ? 0x80000000u : 0u, skeep = p.scale_log2 == 0.f ? 0u : 0xffffffffu;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (mbar_wait_bounded(bar, parity)) return true;
        if (lane == 0) flag_error(p.err, PKV_ERR_WAIT_TIMEOUT);
        return false;
    };
    [[maybe_unused]] uint32_t meets = 0;
    [[maybe_unused]] bool bounded = false;
    [[maybe_unused]] auto meet = [&]() {  // of the four warps
        __syncwarp();
        if (lane == 0) mbar_arrive(m.team);
        return wait(m.team, meets++ & 1u);
    };
    // a segment's Q: rows past the entry's queries are others', or zeros past the last row (their results go nowhere)
    auto copy_q = [&](const MtDesc &e) {
        mbar_arrive_expect_tx(m.qready, uint32_t(tp.tile * p.gq * D * 2));
#pragma unroll
        for (int h = 0; h < D / 64; ++h) tma_load_3d(qop + h * kMtQSlab, qmap, 64 * h, e.g * p.gq, e.row0, m.qready);
    };
    uint32_t k = 0;  // unit of the CTA
    if (!wait(&m.dfull[0], 0u)) return;
    if (t == 0 && m.desc[0].len > 0) copy_q(m.desc[0]);
    for (uint32_t j = 0;; ++j) {
        const MtDesc &sg = m.desc[j % kMtDescs], &nsg = m.desc[(j + 1) % kMtDescs];
        const int32_t len = sg.len;
        if (len == 0) break;
        const int32_t L = sg.L, cnt = sg.cnt, row0 = sg.row0, base = sg.base, u0 = sg.u;  // (the rest is read when needed)
        const SeenUnits su = seen_units(p, L, cnt);
        const bool row_ok = qi < cnt;
        const int32_t pos = L - cnt + qi;  // the row's query
        // token units that every query sees whole
        const int32_t all0 = (max(L - p.window, 0) + kMtKeys - 1) / kMtKeys;
        const int32_t all1 = (p.tree ? min(L - cnt + 1, base) : L - cnt + 1) / kMtKeys;
        [[maybe_unused]] auto ctr = [&]() { return p.ws_count + (long long)(tp.ctr_by_row ? row0 : sg.b) * p.Hkv + sg.g; };
        [[maybe_unused]] unsigned long long arrived = 0;
        float mrun = -INFINITY, lrun = 0.f;
        for (int i = 0; i < len; ++i, ++k) {
            const int32_t tu = su.token_unit(u0 + i), tok0 = tu * kMtKeys;
            const bool all = tu >= all0 && tu < all1;
            uint32_t v0 = 0xffffffffu, v1 = 0xffffffffu, e0 = v0, e1 = v0;  // the keys that the row sees, that any query does
            if (!all) {
                if (p.tree && tok0 + kMtKeys > base) {
                    const uint4 s = mt_tree_sees(p, tok0, L, cnt, row0, base, qi, lane);
                    v0 = s.x;
                    v1 = s.y;
                    e0 = s.z;
                    e1 = s.w;
                } else {
                    v0 = row_ok ? row_sees(p, tok0, pos, base, nullptr) : 0u;
                    v1 = row_ok ? row_sees(p, tok0 + 32, pos, base, nullptr) : 0u;
                    e0 = entry_sees(p, tok0, L, cnt);
                    e1 = entry_sees(p, tok0 + 32, L, cnt);
                }
            }
            if (!wait(&m.sfull[k & 1u], (k >> 1) & 1u)) return;
            tc_fence_after();
            if (i == len - 1) {  // the segment's last scores are in
                if (!wait(&m.dfull[(j + 1) % kMtDescs], ((j + 1) / kMtDescs) & 1u)) return;
                if (t == 0 && nsg.len > 0) copy_q(nsg);
                if constexpr (MERGE)  // looked at once the weights are out: whether this piece completes the segment
                    if (t == 0 && len < sg.n) arrived = *reinterpret_cast<volatile unsigned long long *>(ctr());
            }
            const uint32_t sbuf = tlane + (k & 1u) * kMtKeys;
            uint32_t r[kMtKeys];
            tmem_ld64(sbuf, r);
            if (sflip != 0u || skeep == 0u) {
#pragma unroll
                for (int j = 0; j < kMtKeys; ++j) r[j] = (r[j] ^ sflip) & skeep;
            }
            if (!all) {
#pragma unroll
                for (int j = 0; j < kMtKeys; ++j)
                    r[j] = ((j < 32 ? v0 : v1) >> (j & 31)) & 1u ? r[j] : 0xff800000u;
            }
            float mx4[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) mx4[j] = __uint_as_float(r[j]);
#pragma unroll
            for (int j = 4; j < kMtKeys - 4; j += 8)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mx4[i] = mt_max3(mx4[i], __uint_as_float(r[j + i]), __uint_as_float(r[j + 4 + i]));
#pragma unroll
            for (int i = 0; i < 4; ++i) mx4[i] = fmaxf(mx4[i], __uint_as_float(r[kMtKeys - 4 + i]));
            const float mx = fmaxf(mt_max3(mx4[0], mx4[1], mx4[2]), mx4[3]) * c;
            float alpha = 1.0f;
            bool resc = false;
            if (mx > mrun + kRescaleSlack) {  // also the row's first unit with a key (mrun = -inf)
                if (mrun != -INFINITY) {
                    alpha = ex2(mrun - mx);
                    lrun *= alpha;
                    resc = true;
                }
                mrun = mx;
            }
            if (__any_sync(kFull, resc)) {  // O's rows scaled in place once P(k - 1) V is in
                if (!wait(&m.odone[(k - 1) & 1u], ((k - 1) >> 1) & 1u)) return;
                tc_fence_after();
#pragma unroll 1
                for (int cc = 0; cc < D; cc += 16) {
                    uint32_t o[16];
                    tmem_ld16(tlane + kMtOCol + cc, o);
#pragma unroll
                    for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
                    tmem_st16(tlane + kMtOCol + cc, o);
                }
            }
            const float mneg = mrun == -INFINITY ? 0.f : -mrun;
            const uint64_t c2 = f32x2(c, c), m2 = f32x2(mneg, mneg);
            uint64_t ps[2] = {0ull, 0ull};
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // 32 keys at a time: the first half's output product runs beside the second
                uint32_t w[kMtKeys / 4], rest[TWO ? kMtKeys / 4 : 1];
#pragma unroll
                for (int j = 0; j < kMtKeys / 4; ++j) {
                    const int e = 32 * h + 2 * j;
                    const float2 x =
                        f32x2_parts(fma2(f32x2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), c2, m2));
                    const float p0 = ex2(x.x), p1 = ex2(x.y);
                    ps[j & 1] = add2(ps[j & 1], f32x2(p0, p1));
                    w[j] = pack_bf16x2(p0, p1);
                    if constexpr (TWO)
                        rest[j] = pack_bf16x2(p0 - __uint_as_float(w[j] << 16), p1 - __uint_as_float(w[j] & 0xffff0000u));
                }
                if (h == 0 && (e0 & e1) != 0xffffffffu) {
                    // V rows that no query sees may hold anything, and 0 * NaN is NaN: zeros there, once they have landed.
                    // (Not before the scores are in: only those tell that the slot's item before this one has landed, and a
                    // barrier two phases behind would pass for one that is done.  Here rather than right after them the
                    // tile has had more time to land: 64-token chunks 60.6 us, so 59.5.)
                    const uint32_t item = mt_vitem(k);
                    if (!wait(&m.full[item % ns], (item / ns) & 1u)) return;
                    uint8_t *v = ring + (item % ns) * uint32_t(kMtKeys * D * 2);
                    for (int j = t; j < kMtKeys * (D / 8); j += 32 * kMtSoftmaxWarps) {
                        const int r = (j >> 3) & (kMtKeys - 1);
                        if (!(((r < 32 ? e0 : e1) >> (r & 31)) & 1u))
                            *reinterpret_cast<uint4 *>(v + j * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();  // for the tensor core
                }
                tmem_st16(sbuf + uint32_t(16 * h), w);
                if constexpr (TWO) tmem_st16(sbuf + uint32_t(kMtKeys / 2 + 16 * h), rest);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&m.pfull[2 * (k & 1u) + h]);
            }
            const float2 pa = f32x2_parts(ps[0]), pb = f32x2_parts(ps[1]);
            lrun += (pa.x + pa.y) + (pb.x + pb.y);
        }
        // The segment's part here ends, with the last output product.
        uint16_t *orow = row_ok ? p.out + ((long long)(row0 + qi) * p.Hq + (long long)sg.g * p.gq + qh) * D : nullptr;
        [[maybe_unused]] const int slice = int(blockIdx.x);
        bool done = len == sg.n;
        if constexpr (MERGE)
            if (!done) {
                if (!bounded) {  // all slices' bounds, where a CTA's first piece asks for them
                    for (int i = t; i <= sl.nsl; i += 32 * kMtSoftmaxWarps) bound[i] = mt_bound(p, m.scan, sl, i);
                    bounded = true;
                }
                // Every other piece counted in: this one stays where it is and the others join it.
                if (t == 0) {
                    sh[1] = uint32_t(arrived >> 32) == gen && uint32_t(arrived) + uint32_t(len) == uint32_t(sg.n);
                    __threadfence();
                }
                if (!meet()) return;
                done = sh[1] != 0;
                if (done && t == 0) atomicExch(ctr(), 0ull);  // the counter at rest again
            }
        if (!wait(&m.odone[(k - 1) & 1u], ((k - 1) >> 1) & 1u)) return;
        tc_fence_after();
        if (!done) {
            // a piece: (m, l, O) of every row into the slice's piece tile
            const long long tile = mt_piece(tp, slice, sg.first != 0, row0, sg.g);
            float4 *dst = reinterpret_cast<float4 *>(p.ws_acc + tile * 128 * D) + t;
#pragma unroll 1
            for (int cc = 0; cc < D; cc += 32) {
                uint32_t o[32];
                tmem_ld32(tlane + kMtOCol + cc, o);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    dst[(cc / 4 + j) * 128] = make_float4(__uint_as_float(o[4 * j]), __uint_as_float(o[4 * j + 1]),
                                                          __uint_as_float(o[4 * j + 2]), __uint_as_float(o[4 * j + 3]));
            }
            reinterpret_cast<float2 *>(p.ws_ml)[tile * 128 + t] = make_float2(mrun, lrun);
            if constexpr (MERGE) {
                // the whole piece is written before it is counted in (the counting thread's fence carries all of them)
                if (!meet()) return;
                if (t == 0) {
                    __threadfence();
                    sh[1] = arrive_last(ctr(), gen, uint32_t(len), uint32_t(sg.n), p.err);
                }
                if (!meet()) return;
                done = sh[1] != 0;
            }
        }
        if (len == sg.n) {
            mt_output<D>(lrun, tlane + kMtOCol, orow);
        } else if constexpr (MERGE) {
            if (done) {
                __threadfence();
                mt_merge<D>(tp, bound, mt_slice_of(bound, sl.nsl, slice, sg.x0 + p.seg_cost),
                            mt_slice_of(bound, sl.nsl, slice, sg.x0 + p.seg_cost + sg.n - 1), slice, sg.x0, sg.g, row0, t,
                            mrun, lrun, tlane + kMtOCol, orow);
            }
            if (!meet()) return;  // sh[1] is read before it is written again
        }
        tc_fence_before();  // the reads of O come before the next segment's first product overwrites it
        __syncwarp();
        if (lane == 0) mbar_arrive(&m.dempty[j % kMtDescs]);
    }
    tc_fence_before();
}

// The issuing warp, lane 0.  One thread's chain of instructions per unit, so addresses and descriptors are kept and
// moved on, not made anew (made anew, with a division for the slots: 3100 cycles a unit, the CTA's longest chain).
template <int D, bool TWO>
__device__ void mt_products(const DecodeParams &p, const MtSmem &m, uint32_t ring, uint32_t qop, uint32_t tmem)
{
    constexpr uint32_t IS = idesc_bf16_f32(128, kMtKeys, false), IP = idesc_bf16_f32(128, D, true);
    constexpr uint32_t kSlot16 = kMtKeys * D * 2 / 16;  // descriptors count 16 bytes
    const uint32_t ns = uint32_t(p.nst);
    const uint32_t empty = smem_u32(m.empty), sfull = smem_u32(m.sfull), odone = smem_u32(m.odone);
    const uint64_t qdesc = smem_desc_sw128(qop, 16, 1024), kdesc = smem_desc_sw128(ring, 16, 1024),
                   vdesc = smem_desc_sw128(ring, kMtSlab, 1024);
    bool dead = false;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        dead = !mbar_test_wait(smem_u32(bar), parity) && !mbar_wait_lean<false>(bar, parity);
        return !dead;
    };
    uint32_t ks = 0, kph = 0, vs = 2 % ns, vph = 2 / ns;  // slots of the next K and V item, their parities
    uint32_t segs = 0;
    // scores of unit k (b = k % 2, ph: parity of the buffer's use)
    auto scores = [&](uint32_t k, uint32_t b, uint32_t ph, bool first) {
        if (!wait(m.full + ks, kph)) return false;
        if (first && !wait(m.qready, segs++ & 1u)) return false;
        if (k >= 2 && !wait(m.odone + b, ph ^ 1u)) return false;
        tc_fence_after();
        const uint64_t kd = kdesc + ks * kSlot16;
        const uint32_t d = tmem + b * kMtKeys;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
            tc_mma_bf16(d, qdesc + ((i >> 2) * kMtQSlab + (i & 3) * 32) / 16, kd + ((i >> 2) * kMtSlab + (i & 3) * 32) / 16,
                        IS, i > 0);
        tc_commit_at(sfull + 8 * b);
        tc_commit_at(empty + 8 * ks);
        ks += k == 0 ? 1 : 2;
        if (ks >= ns) {
            ks -= ns;
            kph ^= 1u;
        }
        return true;
    };
    auto output = [&](uint32_t b, uint32_t ph, bool first) {
        if (!wait(m.pfull + 2 * b, ph) || !wait(m.full + vs, vph)) return false;
        tc_fence_after();
        const uint64_t vd = vdesc + vs * kSlot16;
        const uint32_t pa = tmem + b * kMtKeys, d = tmem + kMtOCol;
#pragma unroll
        for (int i = 0; i < kMtKeys / 16; ++i) {
            if (i == kMtKeys / 32) {
                if (!wait(m.pfull + 2 * b + 1, ph)) return false;
                tc_fence_after();
            }
            tc_mma_bf16_ta(d, pa + uint32_t(8 * i), vd + uint32_t(i) * (2048 / 16), IP, i > 0 || !first);
            if constexpr (TWO)
                tc_mma_bf16_ta(d, pa + uint32_t(kMtKeys / 2 + 8 * i), vd + uint32_t(i) * (2048 / 16), IP, true);
        }
        tc_commit_at(odone + 8 * b);
        tc_commit_at(empty + 8 * vs);
        vs += 2;
        if (vs >= ns) {
            vs -= ns;
            vph ^= 1u;
        }
        return true;
    };
    uint32_t k = 0;
    bool first_prev = false, owed = false;  // unit k - 1 opened its segment, its output product is to be issued
    auto pay = [&]() {
        if (owed && !dead) output((k - 1) & 1u, ((k - 1) >> 1) & 1u, first_prev);
        owed = false;
    };
    for (uint32_t j = 0; !dead; ++j) {
        const uint32_t d = j % kMtDescs;
        if (!wait(m.dfull + d, (j / kMtDescs) & 1u)) break;
        const int32_t len = m.desc[d].len;
        mbar_arrive(&m.dempty[d]);
        pay();
        if (len == 0) break;
        for (int32_t i = 0; i < len && !dead; ++i, ++k) {
            if (!scores(k, k & 1u, (k >> 1) & 1u, i == 0)) break;
            pay();
            first_prev = i == 0;
            owed = true;
        }
    }
    if (dead) flag_error(p.err, PKV_ERR_WAIT_TIMEOUT);
    tc_commit(m.drain);  // every product issued has completed before the tensor memory is freed
}

// The copying warp: it walks the CTA's slice, describes its segments and copies their K and V.  Lane = (box of the
// unit, 64-dim half): nbox * D / 64 <= 16 lanes copy.
template <int D>
__device__ void mt_copies(const TileParams &tp, const MtSmem &m, uint8_t *ring, const CUtensorMap *kmap,
                          const CUtensorMap *vmap, const MtSlices &sl)
{
    constexpr int PARTS = D / 64;
    const DecodeParams &p = tp.p;
    const int lane = threadIdx.x & 31;
    const uint64_t policy = policy_evict_first();
    const uint32_t ns = uint32_t(p.nst), slot_bytes = uint32_t(kMtKeys * D * 2);
    const uint32_t box_bytes = uint32_t(p.boxtok) * 128u;
    // the slice's bounds, and its last segment's start or its own
    int32_t x = 0;
    if (lane < 2) x = mt_bound(p, m.scan, sl, int(blockIdx.x) + lane);
    MtRange rg{__shfl_sync(kFull, x, 0), __shfl_sync(kFull, x, 1), 0};
    rg.rot = rg.lo < rg.hi ? max(rg.lo, rg.hi - 1 - mt_locate(p, m.scan, rg.hi - 1).u) : rg.lo;
    struct Seg {
        MtSeg s;
        MtEntry e;
    };
    auto entry = [&](Seg &x) { x.e = mt_entry(tp, x.s.b, m.seq ? int32_t(m.seq[x.s.b]) : x.s.b / tp.per_entry); };
    bool dead = false;
    uint32_t told = 0;  // descriptors written
    auto tell = [&](const Seg &x, bool end) {
        const uint32_t d = told % kMtDescs;
        if (told >= kMtDescs && !mbar_wait_bounded(&m.dempty[d], (told / kMtDescs - 1) & 1u)) {
            dead = true;
            return;
        }
        if (lane == 0) {
            m.desc[d] = MtDesc{x.s.b, x.s.g, x.s.u, x.s.n, end ? 0 : x.s.len, x.s.x0, x.s.x0 <= rg.lo,
                               x.e.L, x.e.cnt, x.e.row0, x.e.base};
            mbar_arrive(&m.dfull[d]);
        }
        ++told;
    };
    // 32 boxes' table entries at a time, one a lane, loaded a batch ahead: at which block of the sequence's table the
    // box's rows are, and which rows of it (-1: nobody sees it).  Nothing waits for the table's entry here.
    struct Boxes {
        int32_t blk, in;
    };
    auto batch = [&](const Seg &x, int32_t i0) {  // from the segment part's unit i0 on
        Boxes q{0, -1};
        const int32_t i = i0 + (lane >> p.lg_nbox);
        if (i < x.s.len) {
            const int32_t pos = seen_units(p, x.e.L, x.e.cnt).token_unit(x.s.u + i) * kMtKeys + (lane & (p.nbox - 1)) * p.boxtok;
            if (pos < x.e.L && (pos < p.sinks || pos + p.boxtok > window_start(p, x.e.L, x.e.cnt))) {
                // pos < L, which fits the table (longer sequences have no entries)
                q.blk = __ldg(p.block_tables + (long long)x.e.seq * p.max_blocks + (pos >> p.log2_bs));
                q.in = pos & (p.bs - 1);
            }
        }
        return q;
    };
    auto rows = [&](const Boxes &q) {  // the cache rows, -1 where nothing is copied
        if (q.in < 0) return -1;
        if (q.blk >= 0 && q.blk < p.NB) return q.blk * p.bs + q.in;
        flag_error(p.err, PKV_ERR_BLOCK_RANGE);
        return -1;
    };
    uint32_t top = 0;  // items issued, by number
    uint32_t ks = 0, kph = 0, vs = 2 % ns, vph = 2 / ns;  // slots of the next K and V item, their parities
    // one tile into slot s: rows by lane (a unit's box j in lane j), head g
    auto load = [&](const CUtensorMap *map, uint32_t item, uint32_t s, uint32_t ph, int32_t row, int32_t g) {
        if (item >= ns && !mbar_wait_bounded(&m.empty[s], ph ^ 1u)) {
            dead = true;
            return;
        }
        const uint32_t boxes = __popc(__ballot_sync(kFull, lane < p.nbox && row >= 0));
        if (lane == 0) mbar_arrive_expect_tx(&m.full[s], boxes * PARTS * box_bytes);
        __syncwarp();
        const int part = lane & (PARTS - 1), box = lane / PARTS;
        const int32_t mine = __shfl_sync(kFull, row, box);
        if (box < p.nbox && mine >= 0)
            tma_load_4d(ring + s * slot_bytes + uint32_t(part) * kMtSlab + uint32_t(box) * box_bytes, map, 0, mine, part, g,
                        &m.full[s], policy);
        top = max(top, item + 1);
    };
    auto load_k = [&](uint32_t k, int32_t row, int32_t g) {
        load(kmap, mt_kitem(k), ks, kph, row, g);
        ks += k == 0 ? 1 : 2;
        if (ks >= ns) {
            ks -= ns;
            kph ^= 1u;
        }
    };
    auto load_v = [&](uint32_t k, int32_t row, int32_t g) {
        load(vmap, mt_vitem(k), vs, vph, row, g);
        vs += 2;
        if (vs >= ns) {
            vs -= ns;
            vph ^= 1u;
        }
    };
    uint32_t k = 0;
    int32_t vrow = -1, vg = 0;
    Seg cur{}, nxt{};
    bool more = rg.lo < rg.hi && mt_seg(p, m.scan, rg, rg.rot, cur.s);
    if (more) entry(cur);
    tell(cur, !more);
    Boxes first = batch(cur, 0);
    while (more && !dead) {
        const int32_t len = cur.s.len, per = 32 >> p.lg_nbox;  // units of a batch
        int32_t at = rows(first);
        Boxes ahead = batch(cur, per);
        more = mt_next(p, m.scan, rg, cur.s, nxt.s);  // the next segment, told at once, its first boxes looked up
        if (more) entry(nxt);
        tell(nxt, !more);
        if (more) first = batch(nxt, 0);
        for (int32_t i = 0; i < len && !dead; ++i, ++k) {
            if (i > 0 && (i & (per - 1)) == 0) {
                at = rows(ahead);
                ahead = batch(cur, i + per);
            }
            const int32_t row = __shfl_sync(kFull, at, (((i & (per - 1)) << p.lg_nbox) + lane) & 31);  // lane j: box j's row
            load_k(k, row, cur.s.g);
            if (k > 0 && !dead) load_v(k - 1, vrow, vg);
            vrow = row;
            vg = cur.s.g;
        }
        cur = nxt;
    }
    if (k > 0 && !dead) load_v(k - 1, vrow, vg);
    if (dead && lane == 0) flag_error(p.err, PKV_ERR_WAIT_TIMEOUT);
    // every copy this warp started lands before the CTA can retire
    for (uint32_t i = top > ns ? top - ns : 0u; i < top; ++i)
        if (dead || i + 2 != top) mbar_wait_bounded(&m.full[i % ns], (i / ns) & 1u);  // (the item that stays empty)
}

// Zeros to the rows of inconsistent sequences and to rows of none, each CTA a share; flagged.
__device__ __noinline__ void mt_zero_rows(const TileParams &tp, int32_t values)
{
    const DecodeParams &p = tp.p;
    bool ok = true;
    if (tp.cu) {
        for (int32_t b = threadIdx.x; b < tp.num_seqs; b += kMtThreads) ok &= __ldg(tp.cu + b) <= __ldg(tp.cu + b + 1);
        ok &= __ldg(tp.cu) == 0;
    }
    ok = __syncthreads_and(ok) != 0;
    // rows [a, b) of the output: this CTA's share where all CTAs come here, else all of them
    auto zero = [&](long long a, long long b, bool shared) {
        uint4 *o = reinterpret_cast<uint4 *>(p.out + a * values);
        const long long n = (b - a) * values / 8, step = shared ? (long long)gridDim.x * kMtThreads : kMtThreads;
        for (long long i = (shared ? (long long)blockIdx.x * kMtThreads : 0) + threadIdx.x; i < n; i += step)
            o[i] = make_uint4(0u, 0u, 0u, 0u);
        if (threadIdx.x == 0) flag_error(p.err, PKV_ERR_CONTEXT_RANGE);
    };
    if (!ok) return zero(0, tp.num_rows, true);
    const int32_t end = tp.cu ? __ldg(tp.cu + tp.num_seqs) : tp.num_rows;
    if (end < tp.num_rows) zero(end, tp.num_rows, true);
    for (int32_t b = blockIdx.x; b < tp.num_seqs; b += gridDim.x) {
        const MtRows r = mt_rows(tp, b);
        if (!r.ok && r.r0 < min(r.r1, tp.num_rows)) zero(r.r0, min(r.r1, tp.num_rows), false);
    }
}

// The entries' sequences and the prefix of their list lengths, by all NT threads, each a run of entries; zeros for rows
// that get no other output (values > 0: of a row).
template <int NT>
__device__ __forceinline__ void mt_setup(const TileParams &tp, int32_t *scan, uint16_t *seq, int32_t *tmp, int32_t values)
{
    const DecodeParams &p = tp.p;
    const int t = threadIdx.x, lane = t & 31, wid = t >> 5;
    const int per = (p.B + NT - 1) / NT;
    const int lo = min(p.B, t * per), hi = min(p.B, lo + per);
    bool trouble = false;  // offsets out of order, rows of no sequence, or a sequence whose rows and length do not fit
    int32_t s = 0;
    if (tp.cu) {
        for (int32_t b = t; b < tp.num_seqs; b += NT) trouble |= __ldg(tp.cu + b) > __ldg(tp.cu + b + 1);
        if (t == 0) trouble |= __ldg(tp.cu) != 0 || __ldg(tp.cu + tp.num_seqs) != tp.num_rows;
        if (lo < hi) {  // the last sequence whose entries start at lo or before
            int32_t a = 0, b = tp.num_seqs;
            while (b - a > 1) {
                const int32_t mid = (a + b) >> 1;
                if (__ldg(tp.cu + mid) / tp.tile + mid <= lo)
                    a = mid;
                else
                    b = mid;
            }
            s = a;
        }
    }
    int32_t sum = 0;
    for (int i = lo; i < hi; ++i) {
        if (tp.cu) {
            while (s + 1 < tp.num_seqs && __ldg(tp.cu + s + 1) / tp.tile + s + 1 <= i) ++s;
            seq[i] = uint16_t(s);
        } else {
            s = i / tp.per_entry;
        }
        const MtEntry e = mt_entry(tp, i, s);
        trouble |= e.bad;
        const int32_t n = e.cnt > 0 ? seen_units(p, e.L, e.cnt).n + p.seg_cost : 0;
        scan[i] = n;
        sum += n;
    }
    if (__syncthreads_or(trouble)) {
        if (values > 0) mt_zero_rows(tp, values);
        bool ok = true;
        if (tp.cu) {
            for (int32_t b = t; b < tp.num_seqs; b += NT) ok &= __ldg(tp.cu + b) <= __ldg(tp.cu + b + 1);
            ok &= __ldg(tp.cu) == 0;
        }
        if (!__syncthreads_and(ok)) {
            for (int i = t; i <= p.B; i += NT) scan[i] = 0;
            __syncthreads();
            return;
        }
    }
    int32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t v = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) tmp[wid] = incl;
    __syncthreads();
    int32_t run = incl - sum;
    for (int i = 0; i < wid; ++i) run += tmp[i];
    for (int i = lo; i < hi; ++i) {
        const int32_t n = scan[i];
        scan[i] = run;
        run += n;
    }
    if (lo < hi && hi == p.B) scan[p.B] = run;
    __syncthreads();
}

template <int D, bool MERGE, bool TWO>
__global__ void __launch_bounds__(kMtThreads, 2)
    mask_tile_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const __grid_constant__ TileParams tp)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    const DecodeParams &p = tp.p;
    const MtLayout lay = mt_layout(D, p.nst, p.B, tp.cu != nullptr, tp.merge == 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t *scan = reinterpret_cast<int32_t *>(smem + lay.off_scan);
    MtSmem m;
    m.full = reinterpret_cast<uint64_t *>(smem + lay.off_bar);
    m.empty = m.full + kMtMaxSlots;
    m.sfull = m.empty + kMtMaxSlots;
    m.pfull = m.sfull + 2;
    m.odone = m.pfull + 4;
    m.qready = m.odone + 2;
    m.drain = m.qready + 1;
    m.team = m.drain + 1;
    m.dfull = m.team + 1;
    m.dempty = m.dfull + kMtDescs;
    m.desc = reinterpret_cast<MtDesc *>(smem + lay.off_desc);
    m.scan = scan;
    m.seq = tp.cu ? reinterpret_cast<uint16_t *>(smem + lay.off_seq) : nullptr;
    int32_t *bound = reinterpret_cast<int32_t *>(smem + lay.off_bound);  // MERGE
    int *sh = reinterpret_cast<int *>(smem + lay.off_tmp);  // [0] tensor-memory address, [1] a segment is complete, [8..] scan
    if (threadIdx.x == 0) {
        prefetch_tensormap(&qmap);
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
        for (int i = 0; i < p.nst; ++i) {
            mbar_init(&m.full[i], 1);
            mbar_init(&m.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&m.sfull[i], 1);
            mbar_init(&m.pfull[2 * i], kMtSoftmaxWarps);
            mbar_init(&m.pfull[2 * i + 1], kMtSoftmaxWarps);
            mbar_init(&m.odone[i], 1);
        }
        for (int i = 0; i < kMtDescs; ++i) {
            mbar_init(&m.dfull[i], 1);
            mbar_init(&m.dempty[i], kMtSoftmaxWarps + 1);
        }
        mbar_init(m.qready, 1);
        mbar_init(m.drain, 1);
        mbar_init(m.team, kMtSoftmaxWarps);
        fence_barrier_init();
    }
    if (warp == kMtSoftmaxWarps) tmem_alloc(reinterpret_cast<uint32_t *>(sh), kMtCols);
    __syncthreads();  // a next kernel's CTA on this SM takes its tensor memory after this one
    griddep_launch_dependents();
    griddep_wait();
    uint32_t epoch = 0;
    if constexpr (MERGE) {
        epoch = __ldcg(&p.ws_bal->epoch);
        const uint32_t stamp = __ldcg(&p.ws_bal->stamp);
        if (threadIdx.x == 0 && blockIdx.x == 0 && stamp != (epoch ^ kEpochMagic) && !(epoch == 0u && stamp == 0u))
            flag_error(p.err, PKV_ERR_WORKSPACE);
    }
    const uint32_t gen = epoch + 1u;  // this call's tag of the arrival counters (see BalanceState)
    mt_setup<kMtThreads>(tp, scan, const_cast<uint16_t *>(m.seq), sh + 8, p.Hq * D);
    const int32_t T = p.nhg * scan[p.B];
    const MtSlices sl = mt_slices(tp, T, int(gridDim.x));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uint32_t(sh[0]);
    uint8_t *qop = smem + lay.off_q;
    if (int(blockIdx.x) < sl.nsl) {
        if (warp < kMtSoftmaxWarps) {
            mt_softmax<D, MERGE, TWO>(tp, &qmap, m, smem, qop, tmem, bound, sh, sl, gen);
        } else if (warp == kMtSoftmaxWarps) {
            if (lane == 0) mt_products<D, TWO>(p, m, smem_u32(smem), smem_u32(qop), tmem);
            __syncwarp();
            if (!mbar_wait_bounded(m.drain, 0u) && lane == 0) flag_error(p.err, PKV_ERR_WAIT_TIMEOUT);
        } else {
            mt_copies<D>(tp, m, smem, &kmap, &vmap, sl);
        }
    }
    tc_fence_before();
    __syncthreads();  // every tensor-memory access of the CTA is done
    if (warp == kMtSoftmaxWarps) {
        tc_fence_after();
        tmem_dealloc(tmem, kMtCols);
    }
    // count this CTA in (it read the control block long ago); the last one leaves the block ready for the next call
    if (MERGE && threadIdx.x == 0) {
        __threadfence();
        if (atomicAdd(&p.ws_bal->done, 1u) == gridDim.x - 1) {
            p.ws_bal->done = 0u;
            p.ws_bal->epoch = epoch + 1u;
            p.ws_bal->stamp = (epoch + 1u) ^ kEpochMagic;
        }
    }
}

// Merges the pieces of the segments that lie in several of the `ctas` slices, in slice order:
//     M = max m_i,  l = sum 2^(m_i - M) l_i,  out = sum 2^(m_i - M) acc_i / l.
// CTA (x, y): four columns, from 4 x on, of the 128 rows of segment y (entry y / nhg), a thread a row, eight pieces'
// loads in flight.
constexpr int kMtMergeThreads = 128;

template <int D>
__global__ void __launch_bounds__(kMtMergeThreads) mask_merge_kernel(const __grid_constant__ TileParams tp, int ctas)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    const DecodeParams &p = tp.p;
    int32_t *tmp = reinterpret_cast<int32_t *>(smem), *bound = tmp + 8, *scan = bound + kMaxSlots + 1;
    uint16_t *seq = tp.cu ? reinterpret_cast<uint16_t *>(scan + p.B + 1) : nullptr;
    griddep_launch_dependents();
    griddep_wait();
    mt_setup<kMtMergeThreads>(tp, scan, seq, tmp, 0);
    const int b = int(blockIdx.y) / p.nhg, g = int(blockIdx.y) - b * p.nhg, row = threadIdx.x;
    const int32_t n = scan[b + 1] - scan[b];
    if (n == 0) return;
    const MtSlices sl = mt_slices(tp, p.nhg * scan[p.B], ctas);
    const int32_t x0 = p.nhg * scan[b] + g * n, first = x0 + p.seg_cost, last = x0 + n - 1;
    // the slices that hold its units: from about where they would be without moved bounds
    int sf = min(max(first / max(sl.each, 1) - 2, 0), sl.nsl - 1);
    while (sf > 0 && mt_bound(p, scan, sl, sf) > first) --sf;
    while (mt_bound(p, scan, sl, sf + 1) <= first) ++sf;
    for (int i = sf + row; i <= sl.nsl; i += kMtMergeThreads) {
        bound[i] = mt_bound(p, scan, sl, i);
        if (bound[i] > last) break;
    }
    __syncthreads();
    int end = sf;
    while (bound[end + 1] <= last) ++end;
    if (end == sf) return;  // one piece: its output is written
    const MtEntry e = mt_entry(tp, b, seq ? int32_t(seq[b]) : b / tp.per_entry);
    const int qi = row / p.gq, c4 = int(blockIdx.x);
    float M = -INFINITY, L = 0.f, a[4] = {0.f, 0.f, 0.f, 0.f};
    for (int s0 = sf; s0 <= end; s0 += 8) {
        float2 st[8];
        float4 v[8];
        bool in[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int s = min(s0 + k, end);
            in[k] = s0 + k <= end && bound[s + 1] > bound[s];  // (an empty slice left nothing)
            const long long tile = mt_piece(tp, s, x0 <= bound[s], e.row0, g);
            st[k] = __ldcg(reinterpret_cast<const float2 *>(p.ws_ml) + tile * 128 + row);
            v[k] = __ldcg(reinterpret_cast<const float4 *>(p.ws_acc + tile * 128 * D) + c4 * 128 + row);
        }
        float mn = M;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (in[k]) mn = fmaxf(mn, st[k].x);
        const float at = mn == -INFINITY ? 0.f : mn, r = ex2(M - at);
        L *= r;
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] *= r;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (in[k]) {
                const float f = ex2(st[k].x - at);
                L = fmaf(f, st[k].y, L);
                a[0] = fmaf(f, v[k].x, a[0]);
                a[1] = fmaf(f, v[k].y, a[1]);
                a[2] = fmaf(f, v[k].z, a[2]);
                a[3] = fmaf(f, v[k].w, a[3]);
            }
        M = mn;
    }
    if (qi >= e.cnt) return;
    const float inv = L == 0.f ? 0.f : 1.0f / L;
    uint16_t *out = p.out + ((long long)(e.row0 + qi) * p.Hq + (long long)g * p.gq + (row - qi * p.gq)) * D + 4 * c4;
    *reinterpret_cast<uint2 *>(out) = make_uint2(pack_bf16x2(a[0] * inv, a[1] * inv), pack_bf16x2(a[2] * inv, a[3] * inv));
}

// Q as [num_rows][Hq][D], a box of `tile` queries x gq heads x 64 dims landing as 128-byte-swizzled rows.
static bool encode_q_map(CUtensorMap *map, const TileParams &tp, int D)
{
    EncodeTiledFn enc = encode_tiled_fn();
    if (!enc) {
        record_cuda_error("cuTensorMapEncodeTiled", "driver entry point unavailable");
        return false;
    }
    const cuuint64_t dims[3] = {cuuint64_t(D), cuuint64_t(tp.p.Hq), cuuint64_t(tp.num_rows)};
    const cuuint64_t strides[2] = {cuuint64_t(D) * 2, cuuint64_t(tp.p.Hq) * D * 2};
    const cuuint32_t box[3] = {64u, cuuint32_t(tp.p.gq), cuuint32_t(tp.tile)}, estr[3] = {1u, 1u, 1u};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t *>(tp.p.q), dims, strides, box,
                           estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r == CUDA_SUCCESS) return true;
    char msg[64];
    std::snprintf(msg, sizeof msg, "CUresult %d", int(r));
    record_cuda_error("cuTensorMapEncodeTiled", msg);
    return false;
}

template <int D, bool MERGE, bool TWO>
static pkv_status launch_kernel(const TileParams &tp, const CUtensorMap &qmap, const CUtensorMap &kmap, const CUtensorMap &vmap,
                                int device, int grid, uint32_t smem, cudaStream_t stream)
{
    auto kern = mask_tile_kernel<D, MERGE, TWO>;
    if (!ensure_smem_attribute<D, MERGE, kBf16, TWO, true, true>(kern, device, smem)) return PKV_ECUDA;
    const cudaError_t e = launch_pdl(kern, dim3(grid), dim3(kMtThreads), smem, stream, qmap, kmap, vmap, tp);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return cuda_fail("mask_tile_kernel launch", e);
    }
    return launch_status("mask_tile_kernel launch");
}

template <int D>
static pkv_status launch_tile(TileParams &tp, const void *k_cache, const void *v_cache, const DeviceInfo &dev,
                              int32_t num_workers, cudaStream_t stream)
{
    DecodeParams &p = tp.p;
    // Two CTAs an SM (their shared memory: what the SM has, less the 1 KiB a CTA the system keeps) with at least four
    // slots each, or one with more where the list of entries is too long for that.
    const uint32_t half = uint32_t((dev.max_smem_optin + 1024) / 2 - 1024), all = uint32_t(dev.max_smem_optin);
    auto depth = [&](uint32_t room) {
        int n = kMtMaxSlots;
        while (n > 0 && mt_layout(D, n, p.B, tp.cu != nullptr, tp.merge == 1).total > room) --n;
        return n;
    };
    int ctas = 2, n = depth(half);
    if (n < 4) {
        ctas = 1;
        n = depth(all);
    }
    if (n < 3) return PKV_EUNSUPPORTED;
    p.nst = n;
    p.seg_cost = kMtSegCost;
    const uint32_t total = mt_layout(D, n, p.B, tp.cu != nullptr, tp.merge == 1).total;
    int grid = std::min(dev.sm_count * ctas, kMaxSlots);
    if (num_workers > 0) grid = std::min((num_workers + team_warps(16) - 1) / team_warps(16), kMaxSlots);
    CUtensorMap qmap, kmap, vmap;
    const int64_t rows = int64_t(p.NB) * p.bs;
    if (!encode_q_map(&qmap, tp, D) ||
        !cached_cache_map(&kmap, dev.device, k_cache, false, D, p.Hkv, rows, 1, p.boxtok, 1) ||
        !cached_cache_map(&vmap, dev.device, v_cache, false, D, p.Hkv, rows, 1, p.boxtok, 1))
        return PKV_ECUDA;
    auto fn = tp.merge == 1 ? (tp.two ? launch_kernel<D, true, true> : launch_kernel<D, true, false>)
                            : (tp.two ? launch_kernel<D, false, true> : launch_kernel<D, false, false>);
    const pkv_status st = fn(tp, qmap, kmap, vmap, dev.device, grid, total, stream);
    if (st != PKV_OK || tp.merge != 2) return st;
    const size_t bytes = size_t(8 + kMaxSlots + 1 + p.B + 1) * 4 + size_t(p.B) * 2;  // (few segments: a few KiB)
    const cudaError_t em = launch_pdl(mask_merge_kernel<D>, dim3(D / 4, unsigned(p.B * p.nhg)), dim3(kMtMergeThreads), bytes,
                                      stream, tp, grid);
    if (em != cudaSuccess) {
        cudaGetLastError();
        return cuda_fail("mask_merge_kernel launch", em);
    }
    return launch_status("mask_merge_kernel launch");
}

int32_t mask_tile_entries(int32_t num_seqs, int32_t num_rows, int32_t per_seq, int32_t tile)
{
    const int64_t n = per_seq > 0 ? int64_t(num_seqs) * ((per_seq + tile - 1) / tile) : int64_t(num_rows) / tile + num_seqs;
    return int32_t(std::min<int64_t>(n, INT32_MAX));
}

bool mask_tile_fits(int D, int32_t entries, bool ragged, int max_smem)
{
    return mt_layout(D, 3, entries, ragged, true).total <= uint32_t(max_smem);
}

pkv_status mask_tile_call(DecodeParams &p, const void *k_cache, const void *v_cache, const int32_t *cu, int32_t num_seqs,
                          int32_t num_rows, int32_t per_seq, int32_t max_new, bool two_parts, int32_t head_dim,
                          uint8_t *workspace, int32_t num_workers, cudaStream_t stream)
{
    DeviceInfo dev;
    if (!current_device_info(&dev)) return PKV_ECUDA;
    TileParams tp{};
    tp.cu = per_seq > 0 ? nullptr : cu;
    tp.num_seqs = num_seqs;
    tp.num_rows = num_rows;
    tp.per_seq = per_seq;
    tp.tile = 128 / p.gq;
    tp.per_entry = per_seq > 0 ? (per_seq + tp.tile - 1) / tp.tile : 0;
    tp.max_new = max_new;
    tp.two = two_parts;
    p.B = mask_tile_entries(num_seqs, num_rows, per_seq, tp.tile);
    const WsLayout ws = ws_layout(num_rows, 16, p.Hkv, head_dim, true);  // (see mt_piece)
    p.ws_ml = reinterpret_cast<float *>(workspace + ws.ml_off);
    p.ws_acc = reinterpret_cast<float *>(workspace + ws.acc_off);
    p.hg = 1;
    p.nhg = p.Hkv;
    p.boxtok = std::min(kMtKeys, p.bs);
    p.nbox = kMtKeys / p.boxtok;
    p.lg_nbox = ilog2(p.nbox);
    const int64_t seen = std::min<int64_t>(p.len_limit, int64_t(p.window) + p.sinks + tp.tile);
    const int64_t segments = int64_t(p.B) * p.nhg;
    const int ctas = 2 * dev.sm_count;
    if ((seen + kMtKeys - 1) / kMtKeys + 2 <= (segments >= ctas ? kMtWholeMany : kMtWhole)) {
        tp.merge = 0;
        tp.snap = INT32_MAX / 2;
    } else if (segments * kMtFew <= ctas) {
        tp.merge = 2;
        tp.snap = kMtSnapFew;
    } else {
        tp.merge = 1;
        tp.snap = kMtSnap;
        p.ws_bal = reinterpret_cast<BalanceState *>(workspace + ws.bal_off);
        // Counters in the fixed region where it has one for every segment (by entry, or, with many sequences that have no
        // rows, by row), else in the one behind it, which starts at zero (see WsLayout; the clearing costs 2 us).
        tp.ctr_by_row = segments > int64_t(kFixedCounters);
        const bool clear = tp.ctr_by_row && size_t(num_rows) * size_t(p.Hkv) > kFixedCounters;
        p.ws_count = reinterpret_cast<unsigned long long *>(
            workspace + (clear ? ws.count_off : align256(sizeof(BalanceState))));
        if (clear) {
            const cudaError_t e =
                cudaMemsetAsync(p.ws_count, 0, size_t(num_rows) * size_t(p.Hkv) * sizeof(unsigned long long), stream);
            if (e != cudaSuccess) {
                cudaGetLastError();
                return cuda_fail("cudaMemsetAsync (arrival counters)", e);
            }
        }
    }
    tp.p = p;
    return head_dim == 64 ? launch_tile<64>(tp, k_cache, v_cache, dev, num_workers, stream)
                          : launch_tile<128>(tp, k_cache, v_cache, dev, num_workers, stream);
}

}  // namespace pkv
