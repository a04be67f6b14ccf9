// One warp tile of the decode kernel over int8 caches.  Included by the translation units that
// instantiate the kernel for them, after pkv_decode_kernel.cuh.
//
// A cached value is code * scale with one scale per kScaleToks = 16 tokens and kv head, one for K and one
// for V, so a 16-token sub-tile of the MMA tile has one (K scale s_k, V scale s_v) pair, and with lv = log2 s_v
//     x_j = (q . code_j) * (scale * s_k) + lv,   p_j = 2^(x_j - m),
//     o += sum_j p_j codeV_j,   l += (sum_j p_j) / s_v,   out = o / l:
// the weights take the V scale along and the sum divides it out, so both products see plain codes and m, the
// running max of the x_j, keeps the weights in the f16 range whatever the scales.  The products run in f16 with
// fp32 accumulators: codes are exact, a query row too once it is brought to one power of two (see q_pow2), and a
// weight rounds by at most 2^-11 of itself.
//
// The widening of the codes is what the consumers spend most on.  One byte permute makes 1152 + code in f16 (see
// i8x4_biased); the 1152 is taken off in the products, not from every pair of codes: the score accumulators start
// at -1152 sum q (computed once a segment), and a product with -1152 for a matrix takes 1152 sum p off the
// output of every sub-tile.  Next to a subtraction per pair that saves 128 of about 590 instructions a tile;
// what the detour costs is fp32 rounding at 1152 times a sub-tile's weights, 2^-13.8 of a code each time.  16-row
// tiles subtract from V's codes (their two halves would need twice the products).
//
// What bounds it: the consumers' latency, two warps a scheduler with few independent chains.  64 sequences of
// 512-4096 (16 / 8 heads of 128): 58.2 us = 5.15 TB/s (0.76 of the copy rate; 61.6 us with a subtraction per pair of
// codes); 4 new tokens of each (16-row tiles) 68.8 us; 256 sequences of 1-32768, whose long segments hide it,
// 217 us = 6.46 TB/s (0.95).
#pragma once

#include "pkv_decode_kernel.cuh"
#include "pkv_i8_codes.cuh"

namespace pkv {

// Head room of the weights: they stay <= 2^(kI8Head + kRescaleSlack) = 2^14 (f16 holds up to 65504), and the
// largest of a row is at least 2^kI8Head when its max last moved, so the f16 subnormal step of 2^-24 is
// 2^-30 of it.
constexpr float kI8Head = 6.0f;

// -1152 times the sum of the thread's rows of Q (f16 fragments; rows g and g + 8), as a product with -1152
// for every key: what the biased codes add to a score.
template <int KS, int HR>
__device__ __forceinline__ void q_bias(const uint32_t (&qa)[KS][2 * HR], float (&qb)[HR])
{
    float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
        mma_f16_16816(t, qa[ks][0], HR == 2 ? qa[ks][2 % (2 * HR)] : 0u, qa[ks][1], HR == 2 ? qa[ks][3 % (2 * HR)] : 0u,
                      0xe480e480u, 0xe480e480u);
#pragma unroll
    for (int hr = 0; hr < HR; ++hr) qb[hr] = t[2 * hr];
}

// What a tile takes of a scale block's pair (s_k, s_v).  Scales of ordinary size (plain) as they are; a V scale of
// zero or below kMinVScale counts as zero: the block's V codes are taken as zeros (vzero); a NaN, an infinity or a
// V scale above kMaxVScale makes the block's scores NaN.
__device__ __forceinline__ I8Scales i8_scales(float2 s)
{
    I8Scales r;
    r.plain = s.y >= kMinVScale && s.y <= kMaxVScale;
    r.vzero = s.y >= 0.f && s.y < kMinVScale;
    r.k = r.plain || r.vzero ? s.x : __uint_as_float(0x7fc00000u);
    r.lv = r.plain ? __log2f(s.y) : 0.f;
    r.iv = ex2(-r.lv);
    return r;
}

__device__ __forceinline__ void i8_zero_log(I8Scales &s, float lv)
{
    s.lv = lv;
    s.iv = ex2(-lv);
}

// A query row's power of two (see q_pow2): the row's four threads (r4 = 0..3) look at their own dims.
template <int D>
__device__ __forceinline__ float q_row_scale(const uint16_t *qr, bool live, int r4, float &mul)
{
    uint32_t mx = 0u;
    if (live) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            const uint2 w = *reinterpret_cast<const uint2 *>(qr + 16 * ks + 4 * r4);
            mx = max(max(mx, max(w.x & 0x7fffu, (w.x >> 16) & 0x7fffu)), max(w.y & 0x7fffu, (w.y >> 16) & 0x7fffu));
        }
    }
    mx = max(mx, __shfl_xor_sync(kFull, mx, 1));
    mx = max(mx, __shfl_xor_sync(kFull, mx, 2));
    return q_pow2(mx, mul);
}

template <int D, int HR_, bool TAIL>
__device__ __forceinline__ void attend_tile_i8(uint32_t kb, uint32_t vb, const LaneOffsets<D, kI8, false> &off,
                                               const uint32_t (&qa)[Tc<D, kI8, false, HR_>::KS][2 * HR_],
                                               const float (&rowf)[HR_], const float (&qb)[HR_],
                                               const I8Scales (&sc)[2], const int (&lim)[HR_], int valid,
                                               float (&m)[HR_], float (&l)[HR_],
                                               float (&o)[Tc<D, kI8, false, HR_>::MT][HR_][4], int lane)
{
    using T = Tc<D, kI8, false, HR_>;
    constexpr int NT = T::NT, HR = T::HR;
    static_assert(NT == 2, "two 16-token sub-tiles, one pair of scales each");
    constexpr uint32_t kMinus1152 = 0xe480e480u;  // f16 pair
    const int r4 = lane & 3;
    auto a1 = [&](int ks) { return HR == 2 ? qa[ks][2 % (2 * HR)] : 0u; };
    auto a3 = [&](int ks) { return HR == 2 ? qa[ks][3 % (2 * HR)] : 0u; };
    float sa[NT][2][4];  // [sub-tile][n-tile][fragment]
#pragma unroll
    for (int st = 0; st < NT; ++st)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) sa[st][nt][e] = qb[e >> 1 < HR ? e >> 1 : 0];
#pragma unroll
    for (int i = 0; i < T::NCP; ++i) {
#pragma unroll
        for (int st = 0; st < NT; ++st) {
            uint32_t r0, r1, r2, r3;
            ldsm_x4(kb + off.at(st, i), r0, r1, r2, r3);
            // chunk 2i (r0, r2) is k-step 2i, chunk 2i + 1 (r1, r3) k-step 2i + 1; a register holds codes
            // 4 r4 .. 4 r4 + 3 of a token (tokens 0-7 in r0, r1; 8-15 in r2, r3)
            uint32_t b[4][2];
            i8x4_biased<0x4140, 0x4342>(r0, b[0][0], b[0][1]);
            i8x4_biased<0x4140, 0x4342>(r1, b[1][0], b[1][1]);
            i8x4_biased<0x4140, 0x4342>(r2, b[2][0], b[2][1]);
            i8x4_biased<0x4140, 0x4342>(r3, b[3][0], b[3][1]);
            mma_f16_16816(sa[st][0], qa[2 * i][0], a1(2 * i), qa[2 * i][1], a3(2 * i), b[0][0], b[0][1]);
            mma_f16_16816(sa[st][1], qa[2 * i][0], a1(2 * i), qa[2 * i][1], a3(2 * i), b[2][0], b[2][1]);
            mma_f16_16816(sa[st][0], qa[2 * i + 1][0], a1(2 * i + 1), qa[2 * i + 1][1], a3(2 * i + 1), b[1][0],
                          b[1][1]);
            mma_f16_16816(sa[st][1], qa[2 * i + 1][0], a1(2 * i + 1), qa[2 * i + 1][1], a3(2 * i + 1), b[3][0],
                          b[3][1]);
        }
    }
    // the thread's scores (see attend_tile), log2 of the V scale added; a sub-tile without a token has no
    // scales, its scores are masked
    float x[HR][NT * 4];
#pragma unroll
    for (int hr = 0; hr < HR; ++hr)
#pragma unroll
        for (int st = 0; st < NT; ++st) {
            const float f = rowf[hr] * sc[st].k;
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    x[hr][4 * st + 2 * nt + e] = 16 * st + 8 * nt + 2 * r4 + e < lim[hr]
                                                     ? fmaf(sa[st][nt][2 * hr + e], f, sc[st].lv)
                                                     : -INFINITY;
        }
    float mx[HR];
    bool grow = false;
#pragma unroll
    for (int hr = 0; hr < HR; ++hr) {
        mx[hr] = x[hr][0];
#pragma unroll
        for (int k = 1; k < NT * 4; ++k) mx[hr] = fmaxf(mx[hr], x[hr][k]);
        mx[hr] = fmaxf(mx[hr], __shfl_xor_sync(kFull, mx[hr], 1));
        mx[hr] = fmaxf(mx[hr], __shfl_xor_sync(kFull, mx[hr], 2)) - kI8Head;
        grow |= mx[hr] > m[hr] + kRescaleSlack;
    }
    if (__any_sync(kFull, grow)) {
#pragma unroll
        for (int hr = 0; hr < HR; ++hr) {
            const float mn = fmaxf(m[hr], mx[hr]);
            const float alpha = mn == -INFINITY ? 1.0f : ex2(m[hr] - mn);
            l[hr] *= alpha;
            m[hr] = mn;
            const float a0 = __shfl_sync(kFull, alpha, 8 * r4), a1v = __shfl_sync(kFull, alpha, 8 * r4 + 4);
#pragma unroll
            for (int mt = 0; mt < T::MT; ++mt) {
                o[mt][hr][0] *= a0;
                o[mt][hr][1] *= a1v;
                o[mt][hr][2] *= a0;
                o[mt][hr][3] *= a1v;
            }
        }
    }
    uint32_t pb[HR][NT][2];
#pragma unroll
    for (int hr = 0; hr < HR; ++hr) {
        const float mr = m[hr] == -INFINITY ? 0.f : m[hr];
#pragma unroll
        for (int st = 0; st < NT; ++st) {
            float pr[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) pr[k] = ex2(x[hr][4 * st + k] - mr);
            // (a sub-tile without a token has no scales either)
            if (!TAIL || 16 * st < valid) l[hr] = fmaf((pr[0] + pr[1]) + (pr[2] + pr[3]), sc[st].iv, l[hr]);
#pragma unroll
            for (int c = 0; c < 2; ++c) pb[hr][st][c] = f16x2_of(pr[2 * c], pr[2 * c + 1]);
        }
    }
#pragma unroll
    for (int st = 0; st < NT; ++st) {
        if (TAIL && 16 * st >= valid) break;  // no token
        uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
        if constexpr (TAIL) {
            const int v0 = sc[st].vzero ? 0 : valid - 16 * st;
            keep0 = (2 * r4 < v0 ? 0x0000ffffu : 0u) | (2 * r4 + 1 < v0 ? 0xffff0000u : 0u);
            keep1 = (2 * r4 + 8 < v0 ? 0x0000ffffu : 0u) | (2 * r4 + 9 < v0 ? 0xffff0000u : 0u);
        }
#pragma unroll
        for (int i = 0; i < T::NCP; ++i) {
            uint32_t r0, r1, r2, r3;
            ldsm_x4_t(vb + off.at(st, i), r0, r1, r2, r3);
            if constexpr (TAIL) {
                r0 &= keep0;
                r1 &= keep0;
                r2 &= keep1;
                r3 &= keep1;
            }
            // a register holds (token 2 r4: dims 2g, 2g + 1 | token 2 r4 + 1: the same) of a 16-dim chunk: the
            // permute pairs the two tokens of a dim
            uint32_t a[4][2];
            if constexpr (HR == 1) {
                i8x4_biased<0x4240, 0x4341>(r0, a[0][0], a[0][1]);
                i8x4_biased<0x4240, 0x4341>(r1, a[1][0], a[1][1]);
                i8x4_biased<0x4240, 0x4341>(r2, a[2][0], a[2][1]);
                i8x4_biased<0x4240, 0x4341>(r3, a[3][0], a[3][1]);
            } else {
                i8x4_to_f16x2x2<0x4240, 0x4341>(r0, a[0][0], a[0][1]);
                i8x4_to_f16x2x2<0x4240, 0x4341>(r1, a[1][0], a[1][1]);
                i8x4_to_f16x2x2<0x4240, 0x4341>(r2, a[2][0], a[2][1]);
                i8x4_to_f16x2x2<0x4240, 0x4341>(r3, a[3][0], a[3][1]);
            }
#pragma unroll
            for (int hr = 0; hr < HR; ++hr) {
                mma_f16_16816(o[2 * i][hr], a[0][0], a[0][1], a[2][0], a[2][1], pb[hr][st][0], pb[hr][st][1]);
                mma_f16_16816(o[2 * i + 1][hr], a[1][0], a[1][1], a[3][0], a[3][1], pb[hr][st][0], pb[hr][st][1]);
                if constexpr (HR == 1) {
                    mma_f16_16816(o[2 * i][hr], kMinus1152, kMinus1152, kMinus1152, kMinus1152, pb[hr][st][0],
                                  pb[hr][st][1]);
                    mma_f16_16816(o[2 * i + 1][hr], kMinus1152, kMinus1152, kMinus1152, kMinus1152, pb[hr][st][0],
                                  pb[hr][st][1]);
                }
            }
        }
    }
}

template <int D, int G>
__device__ __noinline__ void merge_pieces_i8(const DecodeParams &p, const long long *bound, int sf, int sl,
                                             long long x0, int g, int h, int b, int kvh, int nvh, int lane)
{
    constexpr int PER = D / 32;                                   // output values per lane
    constexpr int HB = G < 8 ? G : 8;                             // heads merged together
    constexpr int BATCH = 64 / (HB * PER) < 8 ? 64 / (HB * PER) : 8;  // pieces whose values are in flight
    using Vec = typename std::conditional<PER == 4, float4, float2>::type;
    const float2 *ml = reinterpret_cast<const float2 *>(p.ws_ml);
#pragma unroll 1
    for (int h0 = 0; h0 < nvh; h0 += HB) {
        float M[HB], L[HB], a[HB][PER];
#pragma unroll
        for (int i = 0; i < HB; ++i) {
            M[i] = -INFINITY;
            L[i] = 0.f;
#pragma unroll
            for (int e = 0; e < PER; ++e) a[i][e] = 0.f;
        }
#pragma unroll 1
        for (int s0 = sf; s0 <= sl; s0 += 32) {
            const int s = s0 + lane;
            const bool use = s <= sl && bound[s + 1] > bound[s];  // empty slices left nothing
            const int sk = use ? s : sf;
            const int slot = int(((slots_by_slice(p.B, p.nhg) ? 2LL * sk + ((sk == sf && x0 != bound[sf]) ? 1 : 0)
                                                              : sk + (long long)b * p.nhg + g) * p.hg + h));
            float2 st[HB];
#pragma unroll
            for (int i = 0; i < HB; ++i) st[i] = __ldcg(ml + (long long)slot * G + min(h0 + i, G - 1));
            const int n = min(32, sl - s0 + 1);
            float w[HB];  // the lane's piece's weight
#pragma unroll
            for (int i = 0; i < HB; ++i) {
                float mx = use ? st[i].x : -INFINITY;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
                mx = fmaxf(mx, M[i]);
                // a head without a valid token in any piece so far keeps its zero state
                const float r = mx == -INFINITY ? 1.0f : ex2(M[i] - mx);
                w[i] = use && st[i].x != -INFINITY ? ex2(st[i].x - mx) : 0.f;
                L[i] = L[i] * r + warp_sum(use ? w[i] * st[i].y : 0.f);
#pragma unroll
                for (int e = 0; e < PER; ++e) a[i][e] *= r;
                M[i] = mx;
            }
#pragma unroll 1
            for (int k = 0; k < n; k += BATCH) {
                Vec v[BATCH][HB];
#pragma unroll
                for (int j = 0; j < BATCH; ++j) {
                    const long long sj = __shfl_sync(kFull, slot, min(k + j, n - 1));
#pragma unroll
                    for (int i = 0; i < HB; ++i)
                        v[j][i] = __ldcg(reinterpret_cast<const Vec *>(
                            p.ws_acc + (sj * G + min(h0 + i, G - 1)) * D + lane * PER));
                }
#pragma unroll
                for (int j = 0; j < BATCH; ++j)
#pragma unroll
                    for (int i = 0; i < HB; ++i) {
                        const float wj = __shfl_sync(kFull, w[i], min(k + j, n - 1));
                        const float f = k + j < n ? wj : 0.f;
                        const float *x = reinterpret_cast<const float *>(&v[j][i]);
#pragma unroll
                        for (int e = 0; e < PER; ++e) a[i][e] = fmaf(f, x[e], a[i][e]);
                    }
            }
        }
#pragma unroll
        for (int i = 0; i < HB; ++i) {
            const int hh = h0 + i;
            if (hh >= nvh) break;
            const float inv = 1.0f / L[i];
            uint16_t *o = p.out + ((int64_t(b) * p.qstride + hh / p.gq) * p.Hq + int64_t(kvh) * p.gq + hh % p.gq) * D +
                          lane * PER;
            if constexpr (PER == 4)
                *reinterpret_cast<uint2 *>(o) = make_uint2(pack_bf16x2(a[i][0] * inv, a[i][1] * inv),
                                                           pack_bf16x2(a[i][2] * inv, a[i][3] * inv));
            else
                *reinterpret_cast<uint32_t *>(o) = pack_bf16x2(a[i][0] * inv, a[i][1] * inv);
        }
    }
}

}  // namespace pkv
