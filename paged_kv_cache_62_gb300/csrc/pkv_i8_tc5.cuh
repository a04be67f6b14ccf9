// The tensor-memory query-split CTA over int8 caches: what differs from the bf16 one (see the comment at
// Tc5Smem in pkv_decode_kernel.cuh).  Included by the translation unit that instantiates it.
//
// A unit's stage holds the codes of its K and V tile as the copies wrote them.  Four converting warps turn each
// tile into f16 rows in the operands' shared-memory layout (128-byte-swizzled 64-dim slabs): a code is exact
// in f16, and so are the query rows, brought to one power of two each, so both products see what the cache
// holds and the scales enter in fp32 in the softmax warps.  f16 weights round by at most 2^-11.
// One operand buffer each for K and V is enough: the buffer of K is free as soon as the scores are computed,
// that of V as soon as the output product is done, and both are refilled while the softmax warps work.
//
// The eight softmax warps are two groups of four, one thread a row, and the units of a segment go to them in
// turn: group w takes the units j with j % 2 == w, with score buffer w, its own running max and sum, and its own
// output accumulator.  Two tiles are then in work at any time without a word between the groups until the
// segment ends, where their states are put together as split-K pieces are.  Tensor memory (512 columns): two
// score buffers (each later its tile's weights in the first 64 columns), two outputs; Q is a shared-memory
// operand.
//
// What bounds it: the straight-line instructions between a unit's loops.  Three kinds of warps run different code
// on the SM and a line of it is gone from the nearest instruction cache when a warp comes round to it a unit
// later, so the passes over the keys are loops of 16 keys, waits are short
// (mbar_wait_lean), and the exchange between two threads of a row that the bf16 CTA makes every unit is gone.
// Measured: 64 new tokens of each of 64 sequences of 512-4096 (16 / 8 heads of 128) 155 us, 517 TFLOP/s, 2.3 TB/s
// of codes; 3100 cycles a 128-key tile, of which its shared-memory traffic alone needs 1790 (copies in 256,
// converters 256 read and 512 written, scores 512, outputs 256).  One group of warps over both halves of the keys,
// as in the bf16 CTA: 179 us; straight-line passes: 283 us; two converting warps: 326 us; warp-level tiles: 535 us.
// A segment's end takes 9500 cycles (the next Q 3400, outputs 2300, counting 2100) and comes at the pace of its
// instruction fetch: 180 instructions less there took 8 us off.
//
// Ordering: codes and scales landed -> full[s]; K operand written -> kready (4 warps), read -> kfree
// (tcgen05.commit); V likewise vready, vfree; scales prepared -> dready[s]; stage released -> empty[s] (4
// converting warps, 8 softmax warps, and the warp that issues output products); scores -> sfull[w]; weights ->
// pfull[w] (4 warps); output product done -> odone[w]; a segment's Q written -> qready (8 warps: after the last scores of
// the segment before it are in); all softmax warps met -> team.  A group passes the end of a segment only with the other, so no barrier runs
// two phases ahead of a waiter.
#pragma once

#include "pkv_decode_kernel.cuh"
#include "pkv_i8_codes.cuh"

namespace pkv {

constexpr uint32_t kTc5I8OCol = 256;  // the outputs' first tensor-memory column
// Head room of the f16 weights (see kI8Head in pkv_i8_tile.cuh: largest 2^14, a row's max at 2^6 or more).
constexpr float kI8TcHead = 6.0f;

// Instruction descriptor of tcgen05.mma kind::f16 with f16 A and B, fp32 accumulators (see idesc_bf16_f32).
__host__ __device__ constexpr uint32_t idesc_f16_f32(int m, int n, bool b_mn_major)
{
    return (1u << 4) | (b_mn_major ? (1u << 16) : 0u) | (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}

// Codes of one tile (128 rows of D bytes at `raw`, as the copies swizzle them) into an f16 operand at `dst`.
// A thread takes 16 codes of a row at a time (piece i of PER): one 16-byte load, two 16-byte stores, several
// rows' loads in flight.  At D = 128 the threads of the row's upper half take the neighbouring row instead: the
// eight threads of a quarter-warp then read and write eight different bank groups (a row's pieces 0-3 and
// its neighbour's 4-7; even chunks of one slab and odd ones of the other).
template <int D>
__device__ __forceinline__ void tc5_convert_tile(const uint8_t *raw, uint8_t *dst, int t)
{
    constexpr int PER = D / 16;                        // 16-code pieces of a row
    constexpr int ROWS = 32 * kTc5ConvertWarps / PER;  // rows the threads cover at a time
    constexpr int BATCH = 4;
    static_assert(ROWS % 8 == 0 && 128 % (ROWS * BATCH) == 0, "the swizzle key of a thread's rows stays");
    const int i = t % PER, r0 = (t / PER) ^ (D == 128 ? i >> 2 : 0);
    const int key = r0 & 7, c = 2 * (i & 3);
    const uint4 *src = reinterpret_cast<const uint4 *>(raw + r0 * D) + (i ^ (D == 128 ? key : (r0 >> 1) & 3));
    uint8_t *base = dst + (i >> 2) * kTc5SlabBytes + r0 * 128;
    uint4 *lo = reinterpret_cast<uint4 *>(base + ((c ^ key) << 4));
    uint4 *hi = reinterpret_cast<uint4 *>(base + (((c + 1) ^ key) << 4));
#pragma unroll 1  // three instruction streams share the SM's instruction cache
    for (int it = 0; it < 128 / ROWS; it += BATCH) {
        uint4 w[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) w[k] = src[(it + k) * ROWS * D / 16];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            uint4 a, b;
            i8x4_to_f16x2x2<0x4140, 0x4342>(w[k].x, a.x, a.y);
            i8x4_to_f16x2x2<0x4140, 0x4342>(w[k].y, a.z, a.w);
            i8x4_to_f16x2x2<0x4140, 0x4342>(w[k].z, b.x, b.y);
            i8x4_to_f16x2x2<0x4140, 0x4342>(w[k].w, b.z, b.w);
            lo[(it + k) * ROWS * 8] = a;
            hi[(it + k) * ROWS * 8] = b;
        }
    }
}

// Whether a scale block's scales (K scale, V scale) are of ordinary size; one whose scales are not is dealt with
// in the operands (tc5_mark_block), the scales that the softmax takes being 1.
__device__ __forceinline__ bool tc5_plain(float2 s)
{
    return s.x > 0.f && s.x < INFINITY && s.y >= kMinVScale && s.y <= kMaxVScale;
}

// mode 1: zeros, mode 2: NaN, into scale block g of an operand: each converting thread over what it wrote there
// itself (see tc5_convert_tile).
template <int D>
__device__ __noinline__ void tc5_mark_block(uint8_t *dst, int g, int mode, int t)
{
    constexpr int PER = D / 16, ROWS = 32 * kTc5ConvertWarps / PER;
    const int i = t % PER, r0 = (t / PER) ^ (D == 128 ? i >> 2 : 0);
    const int row = r0 + g * kScaleToks / ROWS * ROWS, key = r0 & 7, c = 2 * (i & 3);
    if (row / kScaleToks != g) return;
    const uint32_t v = mode == 2 ? 0x7fff7fffu : 0u;
    uint8_t *base = dst + (i >> 2) * kTc5SlabBytes + row * 128;
    *reinterpret_cast<uint4 *>(base + ((c ^ key) << 4)) = make_uint4(v, v, v, v);
    *reinterpret_cast<uint4 *>(base + (((c + 1) ^ key) << 4)) = make_uint4(v, v, v, v);
}

// The converting warps: their thread t.  K runs a unit ahead of V: the scores of unit j + 1 can then be computed
// while the softmax warps work on unit j, and V's buffer, free only when the output product of unit j - 1 is
// done, holds nothing else back.
template <int D, bool MASK>
__device__ void tc5_convert_warps(const DecodeParams &p, const CtaLayout &lay, const Tc5Smem &m, uint8_t *stage0, int t)
{
    const int lane = t & 31;
    uint8_t *kdst = m.vbase, *vdst = m.vbase + kTc5KConv * 2u * lay.kv_bytes;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (mbar_wait_lean(bar, parity)) return true;
        if (lane == 0) flag_error(p.err, PKV_ERR_WAIT_TIMEOUT);
        return false;
    };
    int s = 0, sv = 0;  // stages of unit j (K) and j - 1 (V)
    uint32_t ph = 0;
    bool more = true;
    unsigned vzero = 0u, vzero_next = 0u;  // scale blocks of zeros in V of units j - 1 and j
    for (uint32_t j = 0;; ++j) {
        vzero = vzero_next;
        if (more) {
            if (!wait(&m.full[s], ph)) break;
            more = m.metas[s].b >= 0;
            const uint32_t kb = j % kTc5KConv;
            if (j >= kTc5KConv && !wait(&m.kfree[kb], ((j / kTc5KConv) - 1) & 1u)) break;
            if (more) {
                constexpr int kGroups = kTc5Keys / kScaleToks;
                const float2 sc = m.scales[s * kGroups + (lane & (kGroups - 1))];
                const bool plain = tc5_plain(sc);
                if (t < 32) {
                    if (lane < kGroups) {
                        // a K or V scale of zero: zeros there; a V scale below kMinVScale counts as zero; a NaN, an
                        // infinity or a V scale above kMaxVScale: NaN scores
                        const bool ko = sc.x > 0.f && sc.x < INFINITY, vo = sc.y >= kMinVScale && sc.y <= kMaxVScale;
                        float lv = vo ? __log2f(sc.y) : 0.f;
                        if (__any_sync((1u << kGroups) - 1u, !vo)) {
                            // a V scale of zero takes the smallest log2 of the unit's blocks (see kZeroLog)
                            bool seen;
                            if constexpr (MASK)
                                seen = (entry_sees(p, m.metas[s].tu * kTc5Keys + lane * kScaleToks, m.metas[s].L,
                                                   m.metas[s].cnt) & 0xffffu) != 0u;
                            else
                                seen = lane * kScaleToks < m.metas[s].L - m.metas[s].u * kTc5Keys;
                            float low = vo && seen ? lv : INFINITY;
#pragma unroll
                            for (int o = 1; o < kGroups; o <<= 1)
                                low = fminf(low, __shfl_xor_sync((1u << kGroups) - 1u, low, o));
                            if (!vo) lv = low < INFINITY ? low : kZeroLog;
                        }
                        m.prep[s * kGroups + lane] = make_float4(ko ? sc.x : 1.f, lv, ex2(-lv), 0.f);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&m.dready[s]);
                }
                uint8_t *kop = kdst + kb * 2u * lay.kv_bytes;
                tc5_convert_tile<D>(stage0 + uint32_t(s) * lay.stage_bytes, kop, t);
                // blocks to mark (the same in every warp)
                const bool kz = sc.x == 0.f, vz = sc.y >= 0.f && sc.y < kMinVScale;
                vzero_next = 0u;
                if (const unsigned odd = __ballot_sync(kFull, !plain) & ((1u << kGroups) - 1u)) {
                    const bool ko = sc.x > 0.f && sc.x < INFINITY, vo = sc.y >= kMinVScale && sc.y <= kMaxVScale;
                    const unsigned bad = __ballot_sync(kFull, !((ko || kz) && (vo || vz)));
                    const unsigned zero = __ballot_sync(kFull, kz);
                    vzero_next = odd & ~bad & __ballot_sync(kFull, vz);
                    for (unsigned o = odd & (bad | zero); o; o &= o - 1) {
                        const int g = __ffs(o) - 1;
                        tc5_mark_block<D>(kop, g, bad >> g & 1u ? 2 : 1, t);
                    }
                }
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) {  // after the last unit: tells the other warps the end
                mbar_arrive(&m.kready[kb]);
                if (!more && t < 32) mbar_arrive(&m.dready[s]);
            }
        }
        if (j > 0) {
            const uint32_t u = j - 1, vb = u % kTc5VConv;
            if (u >= kTc5VConv && !wait(&m.vfree[vb], ((u / kTc5VConv) - 1) & 1u)) break;
            uint8_t *vop = vdst + vb * 2u * lay.kv_bytes;
            tc5_convert_tile<D>(stage0 + uint32_t(sv) * lay.stage_bytes + lay.kv_bytes, vop, t);
            for (unsigned o = vzero; o; o &= o - 1) tc5_mark_block<D>(vop, __ffs(o) - 1, 1, t);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&m.vready[vb]);
                mbar_arrive(&m.empty[sv]);
            }
            if (++sv == p.nst) sv = 0;
        }
        if (!more) break;
        if (++s == p.nst) {
            s = 0;
            ph ^= 1u;
        }
    }
}

// The two issuing warps, lane 0 each: one the scores of every unit, as soon as its K operand is written, its
// score buffer free (the output product of unit k - 2, which read its weights there, done) and, at a segment's
// first unit, its Q written; the other (output) the output products, as soon as a unit's weights and V operand are
// written.  An issue blocks while the tensor core works through earlier products (8 products of 128 x 128 x 16
// take about 1000 cycles here, shared memory being busy with the conversions), so one thread for both would be the
// longest chain in the CTA.  Their waits suspend them: they take no issue slots from the warps they share a
// scheduler with.
template <int D>
__device__ void tc5_mma_warp_i8(const DecodeParams &p, const Tc5Smem &m, uint32_t tmem, bool output)
{
    constexpr uint32_t IS = idesc_f16_f32(128, kTc5Keys, false), IP = idesc_f16_f32(128, D, true);
    constexpr uint32_t kOperand = uint32_t(kTc5Keys * D * 2);  // bytes of an operand buffer
    static_assert(kTc5KConv == 1 && kTc5VConv == 1, "one descriptor each");
    const uint64_t kdesc = smem_desc_sw128(m.v_addr, 16, 1024),
                   vdesc = smem_desc_sw128(m.v_addr + kOperand, kTc5SlabBytes, 1024),
                   qdesc = smem_desc_sw128(m.v_addr + 2u * kOperand, 16, 1024);
    const int lane = threadIdx.x & 31;
    if (lane == 0) {
        bool dead = false;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            dead = !mbar_wait_lean<false>(bar, parity);
            return !dead;
        };
        int s = 0;  // stage of unit k
        uint32_t ph = 0;
        if (!output) {
            uint32_t segs = 0;  // segments begun
            for (uint32_t k = 0;; ++k) {
                if (!wait(&m.kready[0], k & 1u)) break;
                if (m.metas[s].b < 0) break;
                if ((m.metas[s].flags & kFirst) && !wait(m.qready, segs++ & 1u)) break;
                if (k >= 2 && !wait(&m.odone[k & 1u], ((k >> 1) - 1) & 1u)) break;
                tc_fence_after();
                // (rolled: a short loop is fetched once; descriptors count 16 bytes)
                uint64_t at = 0;
#pragma unroll 1
                for (int ks = 0; ks < D / 16; ++ks) {
                    tc_mma_bf16(tmem + (k & 1u) * 128u, qdesc + at, kdesc + at, IS, ks > 0);
                    at += (ks & 3) == 3 ? kTc5SlabBytes / 16 - 6 : 2;
                }
                tc_commit(&m.sfull[k & 1u]);
                tc_commit(&m.kfree[0]);
                if (++s == p.nst) s = 0;
            }
        } else {
            uint32_t fresh = 3u;  // bit w: group w has no output yet in this segment
            for (uint32_t k = 0;; ++k) {
                if (!wait(&m.dready[s], ph)) break;
                if (m.metas[s].b < 0) break;
                if (m.metas[s].flags & kFirst) fresh = 3u;
                mbar_arrive(&m.empty[s]);
                const uint32_t w = k & 1u;
                if (!wait(&m.pfull[w], (k >> 1) & 1u) || !wait(&m.vready[0], w)) break;
                tc_fence_after();
                uint32_t pa = tmem + w * 128u;  // the weights, over the unit's scores
                uint64_t vd = vdesc;
                bool more = !(fresh >> w & 1u);
                fresh &= ~(1u << w);
#pragma unroll 1
                for (int ks = 0; ks < kTc5Keys / 16; ++ks) {
                    tc_mma_bf16_ta(tmem + kTc5I8OCol + w * 128u, pa, vd, IP, more);
                    pa += 8;
                    vd += 2048 / 16;
                    more = true;
                }
                tc_commit(&m.odone[w]);
                tc_commit(&m.vfree[0]);
                if (++s == p.nst) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        if (dead) flag_error(p.err, PKV_ERR_WAIT_TIMEOUT);
        tc_commit(m.drain);  // every product issued has completed before the tensor memory is freed
    }
    __syncwarp();
    if (!mbar_wait_bounded(m.drain, 0u) && lane == 0) flag_error(p.err, PKV_ERR_WAIT_TIMEOUT);
}

// The pieces of one (entry, kv head) segment, merged by the CTA whose piece completed its unit count: thread
// (row, half) folds its half of the row's columns over the pieces left by the non-empty slices sf..sl, in slice
// order, and writes the row's output if it is one of the entry's queries.
template <int D>
__device__ __noinline__ void tc5_merge_i8(const DecodeParams &p, const long long *bound, int sf, int sl, long long x0,
                                          int g, int b, int row, int half, uint16_t *out)
{
    constexpr int C = 32;  // columns at a time: the eight loads of two pieces each in flight together
    const float2 *ml = reinterpret_cast<const float2 *>(p.ws_ml);
    auto tile_of = [&](int sk) { return tc5_piece_tile(p, sk, !(sk == sf && x0 != bound[sf]), b, g); };
    auto next = [&](int sk) {  // the next slice that is not empty (an empty one left nothing)
        do ++sk;
        while (sk <= sl && bound[sk + 1] <= bound[sk]);
        return sk;
    };
#pragma unroll 1
    for (int c0 = half * (D / 2); c0 < (half + 1) * (D / 2); c0 += C) {
        float M = -INFINITY, L = 0.f, a[C];
#pragma unroll
        for (int e = 0; e < C; ++e) a[e] = 0.f;
#pragma unroll 1
        for (int sk = sf; sk <= sl;) {
            const int s2 = next(sk);
            const bool two = s2 <= sl;  // else the piece once more, with weight 0
            const long long t1 = tile_of(sk), t2 = tile_of(two ? s2 : sk);
            const float2 m1 = __ldcg(ml + t1 * 128 + row);
            float2 m2 = __ldcg(ml + t2 * 128 + row);
            const float4 *p1 = reinterpret_cast<const float4 *>(p.ws_acc + t1 * 128 * D) + (c0 / 4) * 128 + row;
            const float4 *p2 = reinterpret_cast<const float4 *>(p.ws_acc + t2 * 128 * D) + (c0 / 4) * 128 + row;
            float4 v[C / 4], w[C / 4];
#pragma unroll
            for (int k = 0; k < C / 4; ++k) v[k] = __ldcg(p1 + k * 128);
#pragma unroll
            for (int k = 0; k < C / 4; ++k) w[k] = __ldcg(p2 + k * 128);
            if (!two) m2.x = -INFINITY;
            const float Mn = fmaxf(M, fmaxf(m1.x, m2.x)), at = Mn == -INFINITY ? 0.f : Mn;
            const float r = ex2(M - at), f1 = ex2(m1.x - at), f2 = ex2(m2.x - at);
            M = Mn;
            L = fmaf(f1, m1.y, fmaf(f2, m2.y, L * r));
#pragma unroll
            for (int k = 0; k < C / 4; ++k) {
                a[4 * k] = fmaf(f1, v[k].x, fmaf(f2, w[k].x, a[4 * k] * r));
                a[4 * k + 1] = fmaf(f1, v[k].y, fmaf(f2, w[k].y, a[4 * k + 1] * r));
                a[4 * k + 2] = fmaf(f1, v[k].z, fmaf(f2, w[k].z, a[4 * k + 2] * r));
                a[4 * k + 3] = fmaf(f1, v[k].w, fmaf(f2, w[k].w, a[4 * k + 3] * r));
            }
            sk = two ? next(s2) : s2;
        }
        const float inv = L > 0.f || L != L ? 1.0f / L : 0.f;
        if (out) {
#pragma unroll
            for (int k = 0; k < C / 8; ++k)
                *reinterpret_cast<uint4 *>(out + c0 + 8 * k) = make_uint4(
                    pack_bf16x2(a[8 * k] * inv, a[8 * k + 1] * inv),
                    pack_bf16x2(a[8 * k + 2] * inv, a[8 * k + 3] * inv),
                    pack_bf16x2(a[8 * k + 4] * inv, a[8 * k + 5] * inv),
                    pack_bf16x2(a[8 * k + 6] * inv, a[8 * k + 7] * inv));
        }
    }
}

// The softmax warps: group w = warp / 4, thread row r = 32 (warp % 4) + lane (TMEM lane r) of the entry's tile,
// query r / gq, head r % gq.  x_j = kc s_j + lv with s_j the score of key j's codes, kc the row's factor times the
// K scale of its block and lv = log2 of the V scale; weights 2^(x_j - m); the row's sum takes them over the V
// scale (2^-lv).
template <int D, bool MASK>
__device__ void tc5_softmax_warps_i8(const DecodeParams &p, const CtaLayout &lay, const Tc5Smem &m, uint32_t tmem,
                                     float2 *xch, const long long *bound, const int32_t *scan, int *sh,
                                     const float *wts, int nslots, uint32_t gen, int wp, bool adaptive)
{
    constexpr int kGroups = kTc5Keys / kScaleToks;
    constexpr int DH = D / 2;
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int wg = warp >> 2, row = 32 * (warp & 3) + lane;
    const uint32_t tlane = tmem + (uint32_t(32 * (warp & 3)) << 16);
    const uint32_t sbuf = tlane + uint32_t(wg) * 128u, obuf = tlane + kTc5I8OCol;
    const int qi = row / p.gq, qh = row - qi * p.gq;
    const int home = sh[0];
    uint8_t *qop = m.vbase + (kTc5KConv + kTc5VConv) * 2u * lay.kv_bytes;
    int s = 0, shift = 0, u_first = 0;
    uint32_t ph = 0, j = 0, j_first = 0, teams = 0;
    float mrun = -INFINITY, lrun = 0.f, crow = 0.f, cnext = 0.f;
    bool row_ok = false;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (mbar_wait_lean(bar, parity)) return true;
        if (lane == 0) flag_error(p.err, PKV_ERR_WAIT_TIMEOUT);
        return false;
    };
    auto meet = [&]() {  // of the eight warps
        __syncwarp();
        if (lane == 0) mbar_arrive(m.team);
        return wait(m.team, teams++ & 1u);
    };
    // A segment's Q as a shared-memory operand: this thread's half of its row's dims (half = wg), f16 times the
    // power of two that brings the row's largest |q| to [2^14, 2^15), found with the row's other thread; zeros for
    // rows that are not queries.  The half row's loads are all in flight together: a memory round trip under full
    // load is a microsecond.  False if a wait gave up.
    uint32_t *qmax = reinterpret_cast<uint32_t *>(xch + 256);
    auto write_q = [&](const UnitMeta &sg) {
        const uint4 *src = reinterpret_cast<const uint4 *>(
            p.q + ((long long)(sg.row0 + qi) * p.Hq + (long long)sg.g * p.gq + qh) * D + wg * DH);
        uint4 v[DH / 8];
#pragma unroll
        for (int k = 0; k < DH / 8; ++k) v[k] = qi < sg.cnt ? __ldg(src + k) : make_uint4(0u, 0u, 0u, 0u);
        // (two values at a time, as bf16: a NaN wins)
        __nv_bfloat162 top = __float2bfloat162_rn(0.f);
#pragma unroll
        for (int k = 0; k < DH / 8; ++k) {
            const uint32_t u[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                top = __hmax2_nan(top, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&u[e])));
        }
        const uint32_t tb = *reinterpret_cast<const uint32_t *>(&top);
        uint32_t mx = max(tb & 0x7fffu, (tb >> 16) & 0x7fffu);
        qmax[wg * 128 + row] = mx;
        if (!meet()) return false;
        mx = max(mx, qmax[(1 - wg) * 128 + row]);
        float mul;
        const float c = p.scale_log2;
        // the row's factor stays positive, whatever the scale's sign (a masked key is -inf times it)
        cnext = fabsf(c) * q_pow2(mx, mul);
        if (c <= 0.f) mul = c < 0.f ? -mul : 0.f;
        if (c == 0.f) cnext = 1.f;
#pragma unroll
        for (int k = 0; k < DH / 8; ++k) {
            const int ch = wg * (DH / 8) + k;  // 8-dim chunk of the row
            uint32_t u[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                u[e] = f16x2_of(__uint_as_float(u[e] << 16) * mul, __uint_as_float(u[e] & 0xffff0000u) * mul);
            *reinterpret_cast<uint4 *>(qop + (ch >> 3) * kTc5SlabBytes + row * 128 + (((ch & 7) ^ (row & 7)) << 4)) =
                make_uint4(u[0], u[1], u[2], u[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(m.qready);
        return true;
    };
    // One round per unit; round 0 has none and only writes the first segment's Q, as the last unit of a segment
    // writes the next one's (the code stands once: the instruction caches are the short resource here).
    UnitMeta mt;
    mt.flags = kLast;
    for (bool begun = false;; begun = true) {
        bool own = false;
        if (begun) {
            if (!wait(&m.dready[s], ph)) break;
            mt = m.metas[s];
            if (mt.b < 0) break;
            if (mt.flags & kFirst) {
                row_ok = qi < mt.cnt;
                shift = (mt.cnt - 1) - qi;  // the row's query sees this many fewer of the entry's last keys
                mrun = -INFINITY;
                lrun = 0.f;
                u_first = mt.u;
                j_first = j;
                crow = cnext;
            }
            own = int(j & 1u) == wg;
            if (own) {
                const float4 *prep = m.prep + s * kGroups;
                const int tok0 = (MASK ? mt.tu : mt.u) * kTc5Keys;
                const int lim = row_ok ? min(kTc5Keys, mt.L - tok0 - shift) : 0;  // visible keys of the tile
                // masked calls: the keys that the row sees, 32 a word
                uint32_t vis[MASK ? kTc5Keys / 32 : 1] = {};
                if constexpr (MASK) {
                    const uint32_t *mask = p.tree ? p.tree + (long long)(mt.row0 + qi) * p.tree_words : nullptr;
                    if (row_ok && (mt.flags & kWhole)) {
#pragma unroll
                        for (int i = 0; i < kTc5Keys / 32; ++i) vis[i] = 0xffffffffu;
                    } else if (row_ok) {
#pragma unroll 1
                        for (int w = 0; w < kTc5Keys / 32; ++w) {
                            const uint32_t v = row_sees(p, tok0 + 32 * w, mt.L - 1 - shift, mt.base, mask);
#pragma unroll
                            for (int i = 0; i < kTc5Keys / 32; ++i) vis[i] = i == w ? v : vis[i];
                        }
                    }
                }
                // the scores of 32 keys, two scale blocks: -inf at or past the row's bound
                auto scores32 = [&](int g, float (&y)[32]) {
                    uint32_t r[32];
                    tmem_ld32(sbuf + uint32_t(kScaleToks * g), r);
#pragma unroll
                    for (int i = 0; i < 32; ++i) y[i] = __uint_as_float(r[i]);
                    if constexpr (MASK) {
                        const uint32_t v = g & 4 ? (g & 2 ? vis[3] : vis[2]) : (g & 2 ? vis[1] : vis[0]);
                        if (v != 0xffffffffu) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) y[i] = (v >> i) & 1u ? y[i] : -INFINITY;
                        }
                        return;
                    }
                    const int left = lim - kScaleToks * g;
                    if (left < 32) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) y[i] = i < left ? y[i] : -INFINITY;
                    }
                };
                if (!wait(&m.sfull[wg], (j >> 1) & 1u)) break;
                tc_fence_after();
                float mx = -INFINITY;
#pragma unroll 1
                for (int g = 0; g < kGroups; g += 2) {
                    float y[32];
                    scores32(g, y);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float4 sc = prep[g + h];
                        float m2[2] = {y[16 * h], y[16 * h + 1]};
#pragma unroll
                        for (int i = 2; i < kScaleToks; ++i) m2[i & 1] = fmaxf(m2[i & 1], y[16 * h + i]);
                        mx = fmaxf(mx, fmaf(fmaxf(m2[0], m2[1]), fmaxf(sc.x * crow, 0x1p-126f), sc.y));
                    }
                }
                mx -= kI8TcHead;
                // fmaxf passes NaN over: a row that has seen a key of a marked block takes some max all the same (a
                // piece whose max is -inf counts as empty)
                bool sees = lim > 0;
                if constexpr (MASK) sees = (vis[0] | vis[1] | vis[2] | vis[3]) != 0u;
                if (mx == -INFINITY && sees) mx = 0.f;
                float alpha = 1.0f;
                bool resc = false;
                if (mx > mrun + kRescaleSlack) {  // also the row's first tile with a key (mrun = -inf)
                    if (mrun != -INFINITY) {
                        alpha = ex2(mrun - mx);
                        lrun *= alpha;
                        resc = true;
                    }
                    mrun = mx;
                }
                // the group's output scaled in place once its last product is in (a row that keeps its max: alpha 1)
                if (__any_sync(kFull, resc)) {
                    if (!wait(&m.odone[wg], ((j >> 1) - 1) & 1u)) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 16) {
                        uint32_t r[16];
                        tmem_ld16(obuf + uint32_t(wg * 128 + c0), r);
#pragma unroll
                        for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
                        tmem_st16(obuf + uint32_t(wg * 128 + c0), r);
                    }
                }
                const float mneg = mrun == -INFINITY ? 0.f : -mrun;
                // (the weights of blocks g and g + 1, 16 columns, go over scores read already: blocks up to g / 2 + 1)
#pragma unroll 1
                for (int g = 0; g < kGroups; g += 2) {
                    float y[32];
                    scores32(g, y);
                    uint32_t w[16];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float4 sc = prep[g + h];
                        const float kc = fmaxf(sc.x * crow, 0x1p-126f), bias = sc.y + mneg;  // kc: never zero
                        float ps[2] = {0.f, 0.f};
#pragma unroll
                        for (int k = 0; k < kScaleToks / 2; ++k) {
                            const float p0 = ex2(fmaf(y[16 * h + 2 * k], kc, bias));
                            const float p1 = ex2(fmaf(y[16 * h + 2 * k + 1], kc, bias));
                            ps[k & 1] += p0 + p1;
                            w[8 * h + k] = f16x2_of(p0, p1);
                        }
                        lrun = fmaf(ps[0] + ps[1], sc.z, lrun);
                    }
                    tmem_st16(sbuf + uint32_t(8 * g), w);
                }
                tmem_wait_st();
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) {
                if (own) mbar_arrive(&m.pfull[wg]);
                mbar_arrive(&m.empty[s]);  // its meta and scales are read
            }
        }
        if (mt.flags & kLast) {
            // the segment's part in this slice ends.  First the next one's Q, once the last scores are in (they
            // read this one's), so that its first scores run during what follows
            const uint32_t wl = j & 1u;
            if (begun && !own && !wait(&m.sfull[wl], (j >> 1) & 1u)) break;
            {
                const int sn = !begun ? 0 : s + 1 == p.nst ? 0 : s + 1;
                if (!wait(&m.mready[sn], begun && sn == 0 ? ph ^ 1u : ph)) break;
                if (m.metas[sn].b >= 0 && !write_q(m.metas[sn])) break;
            }
            if (!begun) continue;
            // both groups' outputs are final; the states are put together
            if (!wait(&m.odone[wl], (j >> 1) & 1u)) break;
            if (j > j_first && !wait(&m.odone[wl ^ 1u], ((j - 1) >> 1) & 1u)) break;
            tc_fence_after();
            xch[wg * 128 + row] = make_float2(mrun, lrun);
            if (!meet()) break;
            const float2 o0 = xch[row], o1 = xch[128 + row];
            const float M = fmaxf(o0.x, o1.x);
            const float f0 = o0.x == -INFINITY ? 0.f : ex2(o0.x - M), f1 = o1.x == -INFINITY ? 0.f : ex2(o1.x - M);
            const float L = f0 * o0.y + f1 * o1.y;
            const bool has0 = j > j_first || wl == 0u, has1 = j > j_first || wl == 1u;
            const int piece = mt.u - u_first + 1;
            const bool whole = piece == mt.n;  // the whole segment ran here: output; else a piece
            const float inv = !whole ? 1.0f : (L > 0.f || L != L ? 1.0f / L : 0.f);
            const float g0 = has0 ? f0 * inv : 0.f, g1 = has1 ? f1 * inv : 0.f;
            uint16_t *orow =
                p.out + ((long long)(mt.row0 + qi) * p.Hq + (long long)mt.g * p.gq + qh) * D;
            const long long x0 = (long long)p.nhg * scan[mt.b] + (long long)mt.g * mt.n;
            const long long tile = tc5_piece_tile(p, mt.slice, u_first > 0 || x0 == bound[mt.slice], mt.b, mt.g);
            float4 *dst = reinterpret_cast<float4 *>(p.ws_acc + tile * 128 * D) + row;
#pragma unroll 1
            for (int c0 = wg * DH; c0 < (wg + 1) * DH; c0 += 16) {
                uint32_t r0[16], r1[16];
                tmem_ld16(obuf + (has0 ? 0u : 128u) + uint32_t(c0), r0);  // (a group without an output: the other's,
                tmem_ld16(obuf + (has1 ? 128u : 0u) + uint32_t(c0), r1);  // times zero)
                float v[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = fmaf(g0, __uint_as_float(r0[i]), g1 * __uint_as_float(r1[i]));
                if (whole) {
                    if (row_ok) {
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            *reinterpret_cast<uint4 *>(orow + c0 + 8 * k) =
                                make_uint4(pack_bf16x2(v[8 * k], v[8 * k + 1]), pack_bf16x2(v[8 * k + 2], v[8 * k + 3]),
                                           pack_bf16x2(v[8 * k + 4], v[8 * k + 5]),
                                           pack_bf16x2(v[8 * k + 6], v[8 * k + 7]));
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        dst[(c0 / 4 + k) * 128] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                }
            }
            tc_fence_before();  // the reads of O come before the next segment's first products overwrite it
            if (!whole && wg == 0) reinterpret_cast<float2 *>(p.ws_ml)[tile * 128 + row] = make_float2(M, L);
            // the outputs (and the exchanged states) are read, a piece is written: the counting thread's fence at
            // device scope carries all threads' stores (fences are cumulative)
            if (!meet()) break;
            if (!whole) {
                if (t == 0) {
                    __threadfence();
                    sh[5] = arrive_last(p.ws_count + ((long long)mt.b * p.Hkv + mt.g) * p.sub, gen, uint32_t(piece),
                                        uint32_t(mt.n), p.err);
                }
                if (!meet()) break;
                if (sh[5]) {
                    __threadfence();
                    tc5_merge_i8<D>(p, bound, slice_of(bound, nslots, x0), slice_of(bound, nslots, x0 + mt.n - 1), x0,
                                    mt.g, mt.b, row, wg, row_ok ? orow : nullptr);
                }
            }
        }
        if ((mt.flags & kSliceEnd) && adaptive && t == 0) {
            // balance record for the next call (as the regular consumers leave it)
            const bool mine = mt.slice == home;
            const float us =
                float(global_ns() - *reinterpret_cast<const volatile unsigned long long *>(sh + 2)) * 1e-3f;
            p.ws_bal->weight[wp][mt.slice] = mine ? wts[mt.slice] : 0.f;
            p.ws_bal->elapsed[wp][mt.slice] = mine ? fmaxf(us, 1e-3f) : 0.f;
            p.ws_bal->tag[wp][mt.slice] = gen ^ kTableMagic;
        }
        ++j;
        if (++s == p.nst) {
            s = 0;
            ph ^= 1u;
        }
    }
    tc_fence_before();
}

}  // namespace pkv
