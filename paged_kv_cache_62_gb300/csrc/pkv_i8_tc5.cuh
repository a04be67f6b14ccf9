// The tensor-memory query-split CTA over int8 caches: what differs from the bf16 one (see the comment at
// Tc5Smem in pkv_decode_kernel.cuh).  Included by the translation unit that instantiates it.
//
// A unit's stage holds the codes of its K and V tile as the copies wrote them.  The converting warps turn each
// tile into f16 rows in the operands' shared-memory layout (128-byte-swizzled 64-dim slabs): a code is exact
// in f16, and so are the query rows, brought to one power of two each, so both products see what the cache
// holds and the scales enter in fp32 in the softmax warps.  f16 weights round by at most 2^-11.
// One operand buffer each for K and V is enough: the buffer of K is free as soon as the scores are computed,
// that of V as soon as the output product is done, and both are refilled while the softmax warps work on the
// tile, which takes longer.
// Ordering: codes and scales landed -> full[s]; K operand written -> kready, read -> kfree
// (tcgen05.commit); V likewise vready, vfree; scales prepared -> dready[s]; stage released -> empty[s] (the
// converting and the softmax warps).  The other barriers are the bf16 CTA's.
#pragma once

#include "pkv_decode_kernel.cuh"
#include "pkv_i8_codes.cuh"

namespace pkv {

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

// What the softmax takes of a scale block (K scale s_k, V scale s_v): (s_k, lv = log2 s_v, 2^-lv).  A block
// whose scales are not of ordinary size is dealt with in the operands (tc5_mark_block), with scales of 1 here.
__device__ __forceinline__ bool tc5_plain(float2 s)
{
    return s.x > 0.f && s.x < INFINITY && s.y >= kMinVScale && s.y <= kMaxVScale;
}

// mode 1: zeros, mode 2: NaN, into the 16 rows of scale block g of an operand (all converting warps).
template <int D>
__device__ __noinline__ void tc5_mark_block(uint8_t *dst, int g, int mode, int t)
{
    constexpr int N = kScaleToks * D / 8;  // 16-byte pieces
    const uint32_t v = mode == 2 ? 0x7fff7fffu : 0u;
    for (int i = t; i < N; i += 32 * kTc5ConvertWarps) {
        const int slab = i / (kScaleToks * 8), r = i - slab * (kScaleToks * 8);
        *reinterpret_cast<uint4 *>(dst + slab * kTc5SlabBytes + g * (kScaleToks * 128) + r * 16) = make_uint4(v, v, v, v);
    }
}

// The converting warps: their thread t.  K runs a unit ahead of V: the scores of unit j + 1 can then be computed
// while the softmax warps work on unit j, and V's buffer, free only when the output product of unit j - 1 is
// done, holds nothing else back.
template <int D>
__device__ void tc5_convert_warps(const DecodeParams &p, const CtaLayout &lay, const Tc5Smem &m, uint8_t *stage0, int t)
{
    const int lane = t & 31;
    uint8_t *kdst = m.vbase, *vdst = m.vbase + kTc5KConv * 2u * lay.kv_bytes;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (mbar_wait_bounded(bar, parity)) return true;
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
                        const float lv = vo ? __log2f(sc.y) : 0.f;
                        m.prep[s * kGroups + lane] = make_float4(ko ? sc.x : 1.f, lv, ex2(-lv), 0.f);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&m.dready[s]);
                }
                uint8_t *kop = kdst + kb * 2u * lay.kv_bytes;
                tc5_convert_tile<D>(stage0 + uint32_t(s) * lay.stage_bytes, kop, t);
                // blocks to mark (the same in every warp): bits 0-7 zeros in K, 8-15 zeros in V, 16-23 NaN in K
                const bool kz = sc.x == 0.f, vz = sc.y >= 0.f && sc.y < kMinVScale;
                const bool bad = !plain && !((kz || (sc.x > 0.f && sc.x < INFINITY)) && (vz || (sc.y >= kMinVScale && sc.y <= kMaxVScale)));
                const unsigned odd = __ballot_sync(kFull, !plain) & ((1u << kGroups) - 1u);
                if (odd) {
                    const unsigned mk = __ballot_sync(kFull, kz && !bad), mv = __ballot_sync(kFull, vz && !bad),
                                   mn = __ballot_sync(kFull, bad);
                    vzero_next = odd & mv;
                    named_barrier(3, 32 * kTc5ConvertWarps);  // the rows below were just written by all of them
                    for (unsigned o = odd; o; o &= o - 1) {
                        const int g = __ffs(o) - 1;
                        if ((mk | mn) >> g & 1u) tc5_mark_block<D>(kop, g, mn >> g & 1u ? 2 : 1, t);
                    }
                } else {
                    vzero_next = 0u;
                }
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&m.kready[kb]);  // after the last unit: tells the issuing warp the end
        }
        if (j > 0) {
            const uint32_t u = j - 1, vb = u % kTc5VConv;
            if (u >= kTc5VConv && !wait(&m.vfree[vb], ((u / kTc5VConv) - 1) & 1u)) break;
            uint8_t *vop = vdst + vb * 2u * lay.kv_bytes;
            tc5_convert_tile<D>(stage0 + uint32_t(sv) * lay.stage_bytes + lay.kv_bytes, vop, t);
            if (vzero) {
                named_barrier(3, 32 * kTc5ConvertWarps);
                for (unsigned o = vzero; o; o &= o - 1) tc5_mark_block<D>(vop, __ffs(o) - 1, 1, t);
            }
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

// Lane 0 issues every product of the CTA, each as soon as its inputs are ready (as tc5_mma_warp).
template <int D>
__device__ void tc5_mma_warp_i8(const DecodeParams &p, const Tc5Smem &m, uint32_t tmem)
{
    constexpr uint32_t IS = idesc_f16_f32(128, kTc5Keys, false), IP = idesc_f16_f32(128, D, true);
    constexpr uint32_t kOperand = uint32_t(kTc5Keys * D * 2);  // bytes of an operand buffer
    const uint32_t kaddr = m.v_addr, vaddr = m.v_addr + kTc5KConv * kOperand;
    const int lane = threadIdx.x & 31;
    bool dead = false;
    if (lane == 0) {
        int s = 0;                 // stage of unit ns
        uint32_t ns = 0, npv = 0;  // next unit to score, next unit to multiply by V
        uint32_t segs = 0;         // segments begun (Q tiles used)
        bool have = false, ended = false;
        int flags = 0;
        bool first_of[2] = {false, false};
        uint64_t t0 = 0;           // when a run of polls without progress was first timed
        uint32_t idle = 0;         // polls without progress (the timer is read every 1024 of them)
        for (;;) {
            bool progress = false;
            if (!ended && ns < npv + 2) {
                if (!have && mbar_test_wait(smem_u32(&m.kready[ns % kTc5KConv]), (ns / kTc5KConv) & 1u)) {
                    have = true;
                    flags = m.metas[s].flags;
                    if (m.metas[s].b < 0) ended = true;
                }
                if (have && !ended) {
                    const bool qok = !(flags & kFirst) || mbar_test_wait(smem_u32(m.qready), segs & 1u);
                    const bool bok = ns < 2 || mbar_test_wait(smem_u32(&m.odone[ns & 1u]), ((ns >> 1) - 1) & 1u);
                    if (qok && bok) {
                        if (flags & kFirst) ++segs;
                        tc_fence_after();
                        const uint32_t qa = tmem + kTc5QCol + ((segs - 1) & 1u) * 64u;
                        const uint32_t ka = kaddr + (ns % kTc5KConv) * kOperand;
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks)
                            tc_mma_bf16_ta(tmem + (ns & 1u) * 128u, qa + uint32_t(8 * ks),
                                           smem_desc_sw128(ka + uint32_t(ks >> 2) * kTc5SlabBytes + uint32_t(ks & 3) * 32u,
                                                           16, 1024), IS, ks > 0);
                        tc_commit(&m.sfull[ns & 1u]);
                        tc_commit(&m.kfree[ns % kTc5KConv]);
                        first_of[ns & 1u] = (flags & kFirst) != 0;
                        ++ns;
                        have = false;
                        if (++s == p.nst) s = 0;
                        progress = true;
                    }
                }
            }
            if (npv < ns && mbar_test_wait(smem_u32(&m.pfull[npv & 1u]), (npv >> 1) & 1u) &&
                mbar_test_wait(smem_u32(&m.vready[npv % kTc5VConv]), (npv / kTc5VConv) & 1u)) {
                tc_fence_after();
                const uint32_t va = vaddr + (npv % kTc5VConv) * kOperand;
                const uint32_t pa = tmem + (npv & 1u) * 128u;  // the weights, over the unit's scores
#pragma unroll
                for (int ks = 0; ks < kTc5Keys / 16; ++ks)
                    tc_mma_bf16_ta(tmem + kTc5OCol, pa + uint32_t(64 * (ks >> 2) + 8 * (ks & 3)),
                                   smem_desc_sw128(va + uint32_t(ks) * 2048u, kTc5SlabBytes, 1024), IP,
                                   !(first_of[npv & 1u] && ks == 0));
                tc_commit(&m.odone[npv & 1u]);
                tc_commit(&m.vfree[npv % kTc5VConv]);
                ++npv;
                progress = true;
            }
            if (ended && npv == ns) break;
            if (progress) {
                idle = 0;
                t0 = 0;
            } else if ((++idle & 1023u) == 0) {
                const uint64_t now = global_ns();
                if (t0 == 0) {
                    t0 = now;
                } else if (now - t0 > kWaitLimitNs) {
                    dead = true;
                    break;
                }
            }
        }
        if (dead) flag_error(p.err, PKV_ERR_WAIT_TIMEOUT);
        tc_commit(m.drain);  // every product issued has completed before the tensor memory is freed
    }
    __syncwarp();
    if (!mbar_wait_bounded(m.drain, 0u) && lane == 0) flag_error(p.err, PKV_ERR_WAIT_TIMEOUT);
}

}  // namespace pkv
