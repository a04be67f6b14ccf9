// Rotary positions with one or several axes, and the store of the rotated rows.
//
// With f_i the rotary frequencies, a(i) the position axis that frequency i follows and p_a the row's
// position on axis a, the angle of pair i is t_i = p_a(i) f_i and the pair (x, y) becomes
//     (x cos t - y sin t,  y cos t + x sin t).
// Pair i is (dims i, i + rot / 2) or, interleaved, (dims 2i, 2i + 1); dims from rot on pass through.
//
// The angle is reduced exactly: f_i / 2 pi is held as a 64-bit fraction of a turn, so position times
// frequency modulo one turn is one wrapping 64-bit integer product, whatever the position's size (the
// fraction's last place, 2^-64, times 2^31 is 2^-33 turns); its upper 32 bits go to sincospif.  An fp32
// product would lose the angle's low bits to its whole turns (2^-24 of 32768 radians is 2e-3).
//
// Memory-bound: a row is read once and written once.  One warp takes a token (or, when there are few tokens,
// a part of its heads): it makes the token's rot / 2 cosines and sines, two or so a lane, while the first rows'
// loads are on their way, passes them through shared memory (no barrier but the warp's own), and then turns 16
// dims of a head per lane and step, two 16-byte loads and stores.  A lane keeps its place within the head, so
// its eight cosines and sines stay in registers for all heads.  16384 rows of 16 + 2 x 8 heads of 128 on three axes,
// 269 MB: 47.1 us = 5.7 TB/s, 0.84 of the copy rate (a CTA a token group with a barrier after the cosines: 61 us);
// 64 rows: 3.1 us, a launch and two dependent loads.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "pkv_device.cuh"
#include "pkv_host.h"

namespace pkv {

constexpr int kRopeMaxHalf = 128;  // rot / 2 at most (head_dim <= 256)

struct RopeParams {
    const uint16_t *q, *k, *v;
    uint16_t *q_out, *k_out, *v_out;  // k_out / v_out: rows by slot (slots not null) or by token
    long long q_stride, k_stride, v_stride, qo_stride, ko_stride, vo_stride;
    const int32_t *positions, *freq_axis, *slots;
    const float *inv_freq;
    int32_t axes, T, Hq, Hkv, D, rot, parts;
    long long num_slots;
    int32_t *err;
};

// inv_freq / 2 pi modulo 1 as a 64-bit fraction of a turn: the float's 24-bit significand times 1 / 2 pi in
// 128 fractional bits, shifted by the float's exponent.
__device__ __forceinline__ uint64_t turn_fraction(float f)
{
    constexpr uint64_t kHi = 0x28be60db9391054aull, kLo = 0x7f09d5f47d4d3770ull;  // 2^128 / 2 pi
    const uint32_t bits = __float_as_uint(f);
    const int E = int((bits >> 23) & 255u);
    const uint64_t m = (bits & 0x7fffffu) | (E > 0 ? 0x800000u : 0u);  // f = m 2^(max(E, 1) - 150)
    const uint64_t p0 = m * kLo, t = m * kHi, c = __umul64hi(m, kLo);
    const uint64_t p1 = t + c;
    const uint64_t p2 = __umul64hi(m, kHi) + (p1 < t ? 1u : 0u);  // m 2^128 / 2 pi = p2 : p1 : p0
    const int shift = 214 - max(E, 1);                            // f / 2 pi in 64 fractional bits: >> shift
    uint64_t F;
    if (shift >= 192)
        F = 0;
    else if (shift >= 128)
        F = p2 >> (shift - 128);
    else if (shift > 64)
        F = (p1 >> (shift - 64)) | (p2 << (128 - shift));
    else if (shift == 64)
        F = p1;
    else if (shift > 0)
        F = (p0 >> shift) | (p1 << (64 - shift));
    else
        F = p0 << min(-shift, 63);
    return (bits >> 31) ? 0ull - F : F;
}

__device__ __forceinline__ float2 turn_cos_sin(uint64_t F, int32_t pos)
{
    const uint64_t phase = F * uint64_t(int64_t(pos));
    float s, c;
    sincospif(float(int32_t(uint32_t(phase >> 32))) * 0x1p-31f, &s, &c);  // half turns in [-1, 1)
    return make_float2(c, s);
}

// Two 8-value vectors of one head turned in place: pairs (a[e], b[e]) with cs[e] (ADJ: pairs of neighbours
// within a, cs[0..3], and within b, cs[4..7]).
template <bool ADJ>
__device__ __forceinline__ void turn16(uint4 &a, uint4 &b, const float2 *cs)
{
    uint32_t ua[4] = {a.x, a.y, a.z, a.w}, ub[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float a0 = __uint_as_float(ua[j] << 16), a1 = __uint_as_float(ua[j] & 0xffff0000u);
        const float b0 = __uint_as_float(ub[j] << 16), b1 = __uint_as_float(ub[j] & 0xffff0000u);
        if constexpr (ADJ) {
            const float2 ca = cs[j], cb = cs[4 + j];
            ua[j] = pack_bf16x2(a0 * ca.x - a1 * ca.y, a1 * ca.x + a0 * ca.y);
            ub[j] = pack_bf16x2(b0 * cb.x - b1 * cb.y, b1 * cb.x + b0 * cb.y);
        } else {
            const float2 c0 = cs[2 * j], c1 = cs[2 * j + 1];
            ua[j] = pack_bf16x2(a0 * c0.x - b0 * c0.y, a1 * c1.x - b1 * c1.y);
            ub[j] = pack_bf16x2(b0 * c0.x + a0 * c0.y, b1 * c1.x + a1 * c1.y);
        }
    }
    a = make_uint4(ua[0], ua[1], ua[2], ua[3]);
    b = make_uint4(ub[0], ub[1], ub[2], ub[3]);
}

constexpr int kRopeWarps = 2;  // warps (token parts) a CTA: small ones, whose last warp holds little back

template <bool ADJ>
__global__ void __launch_bounds__(32 * kRopeWarps) rope_kernel(const RopeParams p)
{
    __shared__ __align__(16) float2 cs_all[kRopeWarps][kRopeMaxHalf];
    constexpr int B = 3;  // pieces of a lane in flight
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t w = int64_t(blockIdx.x) * kRopeWarps + (threadIdx.x >> 5);
    const int t = int(w / p.parts), part = int(w - int64_t(t) * p.parts);
    if (t >= p.T) return;  // warps do not meet after this
    float2 *cs = cs_all[threadIdx.x >> 5];
    const int half = p.rot >> 1, per = p.D >> 4, turned = p.rot >> 4;  // 16-dim pieces of a head, those that turn
    const int hpw = 32 / per;                                           // heads a step takes
    const int hl = lane / per, c = lane - hl * per;                     // the lane's head of a step, its piece
    const int heads = p.Hq + p.Hkv + (p.v ? p.Hkv : 0), turning = p.Hq + p.Hkv;
    const int64_t slot = p.slots ? int64_t(__ldg(p.slots + t)) : int64_t(t);
    const bool drop = p.slots && (slot < 0 || slot >= p.num_slots);
    if (p.slots && (slot < -1 || slot >= p.num_slots) && lane == 0) flag_error(p.err, PKV_ERR_SLOT_RANGE);
    const bool mine = hl < hpw;
    // the piece of head h (q heads, k heads, v heads): false where nothing is written
    auto place = [&](int h, const uint16_t *&src, uint16_t *&dst) {
        if (!mine || h >= heads) return false;
        if (h < p.Hq) {
            src = p.q + t * p.q_stride + int64_t(h) * p.D;
            dst = p.q_out + t * p.qo_stride + int64_t(h) * p.D;
            return true;
        }
        if (drop) return false;
        if (h < turning) {
            src = p.k + t * p.k_stride + int64_t(h - p.Hq) * p.D;
            dst = p.k_out + slot * p.ko_stride + int64_t(h - p.Hq) * p.D;
        } else {
            src = p.v + t * p.v_stride + int64_t(h - turning) * p.D;
            dst = p.v_out + slot * p.vo_stride + int64_t(h - turning) * p.D;
        }
        return true;
    };
    // a turning piece of pairs of halves lies in two places of the head
    auto d0 = [&](int h) { return c < turned && !ADJ && h < turning ? 8 * c : 16 * c; };
    auto d1 = [&](int h) { return c < turned && !ADJ && h < turning ? half + 8 * c : 16 * c + 8; };
    uint4 a[B], b[B];
    auto load = [&](int h0) {
#pragma unroll
        for (int k = 0; k < B; ++k) {
            const int h = h0 + k * hpw * p.parts;
            const uint16_t *src;
            uint16_t *dst;
            if (place(h, src, dst)) {
                a[k] = *reinterpret_cast<const uint4 *>(src + d0(h));
                b[k] = *reinterpret_cast<const uint4 *>(src + d1(h));
            }
        }
    };
    const int h0 = part * hpw + hl, step = B * hpw * p.parts;
    load(h0);
    for (int i = lane; i < half; i += 32) {
        int ax = p.freq_axis ? __ldg(p.freq_axis + i) : 0;
        if (ax < 0 || ax >= p.axes) {
            flag_error(p.err, PKV_ERR_AXIS_RANGE);
            ax = 0;
        }
        cs[i] = turn_cos_sin(turn_fraction(__ldg(p.inv_freq + i)), __ldg(p.positions + int64_t(ax) * p.T + t));
    }
    __syncwarp();
    float2 mycs[8];
    if (c < turned) {
#pragma unroll
        for (int e = 0; e < 8; ++e) mycs[e] = cs[8 * c + e];
    }
    for (int h1 = h0; h1 < heads; h1 += step) {
#pragma unroll
        for (int k = 0; k < B; ++k) {
            const int h = h1 + k * hpw * p.parts;
            const uint16_t *src;
            uint16_t *dst;
            if (place(h, src, dst)) {
                if (c < turned && h < turning) turn16<ADJ>(a[k], b[k], mycs);
                *reinterpret_cast<uint4 *>(dst + d0(h)) = a[k];
                *reinterpret_cast<uint4 *>(dst + d1(h)) = b[k];
            }
        }
        load(h1 + step);
    }
}

// ------------------------------------------------------------------ with a norm
// A q or k head x becomes x / sqrt(mean x^2 + eps) * w before the turn; the layout is the one above, the D / 16 lanes of
// a head add up their squares with shuffles.  Memory-bound in principle; what stands between is the warps that registers
// leave room for and the instructions a piece takes.  So cosines and sines stay in shared memory and weights in the
// nearest cache, a lane has two pieces in flight, products are two to an instruction (f32x2), offsets have 32 bits, and
// the common head sizes have instances of their own (PER).  16384 rows of 16 + 2 x 8 heads of 128, 269 MB: 48.7 us = 5.5 TB/s,
// 0.81 of the copy rate; on the way there: the kernel above with factors in registers and three pieces in flight 73 us
// (168 registers a thread), with weights from memory 62.6 us, rows through shared memory by bulk copies 58 us (16 warps
// an SM), two products an instruction 52.3 us.  64 rows: 3.3 us.
constexpr int kNormPieces = 2;  // pieces of a lane in flight (1: 48.8-50.4 us, 3: 49.6-57 us)
// CTAs an SM that registers have to leave room for: 12 for pairs of halves (8: 49.5 us, 14: 51.5 us); pairs of
// neighbours and unusual head sizes take more registers (1531 rows of 14 + 2 heads of 80: 5.9 us, with 12 7.7 us).
__host__ __device__ constexpr int norm_ctas(bool adj, int per) { return adj || per == 0 ? 8 : 12; }

__device__ __forceinline__ void unpack8(uint4 v, uint64_t (&x)[4])
{
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = f32x2(__uint_as_float(u[j] << 16), __uint_as_float(u[j] & 0xffff0000u));
}
__device__ __forceinline__ uint4 pack8(const uint64_t (&x)[4])
{
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = f32x2_parts(x[j]);
        u[j] = pack_bf16x2(f.x, f.y);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

struct NormParams {
    RopeParams r;
    const float *qw, *kw;  // [D] or null: ones
    float eps;
};

// PER: 16-dim pieces of a head (0: p.D / 16, any number).
template <bool ADJ, int PER>
__global__ void __launch_bounds__(32 * kRopeWarps, norm_ctas(ADJ, PER)) norm_rope_kernel(const __grid_constant__ NormParams np)
{
    // pairs of halves: cosines, then sines; of neighbours: (cos, cos) and (-sin, sin) of each
    __shared__ __align__(16) float cs_all[kRopeWarps][(ADJ ? 4 : 2) * kRopeMaxHalf];
    const RopeParams &p = np.r;
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t wi = int64_t(blockIdx.x) * kRopeWarps + (threadIdx.x >> 5);
    const int t = int(wi / p.parts), part = int(wi - int64_t(t) * p.parts);
    if (t >= p.T) return;  // warps do not meet after this
    float *cs = cs_all[threadIdx.x >> 5];
    const int D = PER ? 16 * PER : p.D;
    const int half = p.rot >> 1, per = PER ? PER : p.D >> 4, turned = p.rot >> 4;  // 16-dim pieces of a head, those that turn
    const int hpw = 32 / per;                                           // heads a step takes
    const int hl = lane / per, c = lane - hl * per;                     // the lane's head of a step, its piece
    const int heads = p.Hq + p.Hkv + (p.v ? p.Hkv : 0), turning = p.Hq + p.Hkv;
    const bool mine = PER != 0 || hl < hpw, turn = c < turned, pow2 = (per & (per - 1)) == 0;
    const int64_t slot = p.slots ? int64_t(__ldg(p.slots + t)) : int64_t(t);
    const bool drop = p.slots && (slot < 0 || slot >= p.num_slots);
    if (p.slots && (slot < -1 || slot >= p.num_slots) && lane == 0) flag_error(p.err, PKV_ERR_SLOT_RANGE);
    // the lane's dims of a head: a turning piece of pairs of halves lies in two places (v heads do not turn, but move the
    // same way)
    const int e0 = turn && !ADJ ? 8 * c : 16 * c, e1 = turn && !ADJ ? half + 8 * c : 16 * c + 8;
    // (from every row's place as if it were the first of the token's heads: head h is h D on from there; a token's heads
    // have less than 2^30 elements)
    const uint16_t *qs = p.q + t * p.q_stride, *ks = p.k + t * p.k_stride - p.Hq * D, *vs = p.v + t * p.v_stride - turning * D;
    uint16_t *qd = p.q_out + t * p.qo_stride, *kd = p.k_out + slot * p.ko_stride - p.Hq * D,
             *vd = p.v_out + slot * p.vo_stride - turning * D;
    const int last = mine ? (drop ? p.Hq : heads) : 0;  // the lane's heads with something to write end here
    auto load = [&](int h, uint4 &a, uint4 &b) {
        if (h >= last) return;
        const uint16_t *src = (h < p.Hq ? qs : h < turning ? ks : vs) + h * D;
        a = *reinterpret_cast<const uint4 *>(src + e0);
        b = *reinterpret_cast<const uint4 *>(src + e1);
    };
    const int step = hpw * p.parts;
    int h = part * hpw + hl;
    uint4 a[kNormPieces] = {}, b[kNormPieces] = {};
#pragma unroll
    for (int k = 0; k < kNormPieces; ++k) load(h + k * step, a[k], b[k]);
    for (int i = lane; i < half; i += 32) {
        int ax = p.freq_axis ? __ldg(p.freq_axis + i) : 0;
        if (ax < 0 || ax >= p.axes) {
            flag_error(p.err, PKV_ERR_AXIS_RANGE);
            ax = 0;
        }
        const float2 v = turn_cos_sin(turn_fraction(__ldg(p.inv_freq + i)), __ldg(p.positions + int64_t(ax) * p.T + t));
        if constexpr (ADJ) {
            *reinterpret_cast<float2 *>(cs + 2 * i) = make_float2(v.x, v.x);
            *reinterpret_cast<float2 *>(cs + 2 * kRopeMaxHalf + 2 * i) = make_float2(-v.y, v.y);
        } else {
            cs[i] = v.x;
            cs[kRopeMaxHalf + i] = v.y;
        }
    }
    __syncwarp();
    const float invd = 1.0f / float(D);
    // a piece at head g: normed, turned, stored; its registers take the piece kNormPieces steps on meanwhile
    auto piece = [&](int g, uint4 &ra, uint4 &rb) {
        uint64_t x[4], y[4];
        const uint4 va = ra, vb = rb;
        unpack8(va, x);
        unpack8(vb, y);
        load(g + kNormPieces * step, ra, rb);
        uint64_t s2 = mul2(x[0], x[0]), t2 = mul2(y[0], y[0]);
#pragma unroll
        for (int j = 1; j < 4; ++j) {
            s2 = fma2(x[j], x[j], s2);
            t2 = fma2(y[j], y[j], t2);
        }
        const float2 sp = f32x2_parts(s2), tp = f32x2_parts(t2);
        float ss = (sp.x + sp.y) + (tp.x + tp.y);
        if (PER != 0 || pow2) {
#pragma unroll
            for (int o = 1; o < per; o <<= 1) ss += __shfl_xor_sync(kFull, ss, o);
        } else {
            float all = 0.f;
            for (int i = 0; i < per; ++i) all += __shfl_sync(kFull, ss, hl * per + i);
            ss = all;
        }
        if (g >= last) return;
        uint16_t *dst = (g < p.Hq ? qd : g < turning ? kd : vd) + g * D;
        if (g >= turning) {
            *reinterpret_cast<uint4 *>(dst + e0) = va;
            *reinterpret_cast<uint4 *>(dst + e1) = vb;
            return;
        }
        const float r = rsqrtf(fmaf(ss, invd, np.eps));
        const uint64_t r2 = f32x2(r, r);
        const float *w = g < p.Hq ? np.qw : np.kw;
        auto scale = [&](uint64_t (&z)[4], int e) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint64_t w0 = r2, w1 = r2;
                if (w) {
                    const ulonglong2 u = __ldg(reinterpret_cast<const ulonglong2 *>(w + e) + j);
                    w0 = mul2(u.x, r2);
                    w1 = mul2(u.y, r2);
                }
                z[2 * j] = mul2(z[2 * j], w0);
                z[2 * j + 1] = mul2(z[2 * j + 1], w1);
            }
        };
        scale(x, e0);
        scale(y, e1);
        if (turn) {
            if constexpr (ADJ) {
                auto turn4 = [&](uint64_t (&z)[4], int f) {  // frequencies f .. f + 3
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const ulonglong2 cc = *(reinterpret_cast<const ulonglong2 *>(cs + 2 * f) + j);
                        const ulonglong2 sn = *(reinterpret_cast<const ulonglong2 *>(cs + 2 * kRopeMaxHalf + 2 * f) + j);
                        const float2 z0 = f32x2_parts(z[2 * j]), z1 = f32x2_parts(z[2 * j + 1]);
                        z[2 * j] = fma2(z[2 * j], cc.x, mul2(f32x2(z0.y, z0.x), sn.x));
                        z[2 * j + 1] = fma2(z[2 * j + 1], cc.y, mul2(f32x2(z1.y, z1.x), sn.y));
                    }
                };
                turn4(x, 8 * c);
                turn4(y, 8 * c + 4);
            } else {
                constexpr uint64_t kMinus = 0x8000000080000000ull;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const ulonglong2 cc = *(reinterpret_cast<const ulonglong2 *>(cs + 8 * c) + j);
                    const ulonglong2 sn = *(reinterpret_cast<const ulonglong2 *>(cs + kRopeMaxHalf + 8 * c) + j);
                    uint64_t u = x[2 * j];
                    x[2 * j] = fma2(u, cc.x, mul2(y[2 * j], sn.x) ^ kMinus);
                    y[2 * j] = fma2(y[2 * j], cc.x, mul2(u, sn.x));
                    u = x[2 * j + 1];
                    x[2 * j + 1] = fma2(u, cc.y, mul2(y[2 * j + 1], sn.y) ^ kMinus);
                    y[2 * j + 1] = fma2(y[2 * j + 1], cc.y, mul2(u, sn.y));
                }
            }
        }
        *reinterpret_cast<uint4 *>(dst + e0) = pack8(x);
        *reinterpret_cast<uint4 *>(dst + e1) = pack8(y);
    };
    // (the lanes stay together: they add up across a head)
    for (; h - hl < heads; h += kNormPieces * step)
#pragma unroll
        for (int k = 0; k < kNormPieces; ++k)
            if (h + k * step - hl < heads) piece(h + k * step, a[k], b[k]);
}

// Warps a token.  Few tokens: several, each with a part of the heads (as many as leave every lane a piece), until the SMs
// have eight warps each.
static int rope_parts(const RopeParams &p, int sm_count)
{
    const int heads = p.Hq + p.Hkv + (p.v ? p.Hkv : 0), hpw = 32 / (p.D / 16);
    const int most = (heads + hpw - 1) / hpw;
    return int(std::min<int64_t>(most, std::max<int64_t>(1, int64_t(sm_count) * 8 / p.T)));
}

static pkv_status rope_call(RopeParams &p, int interleaved, pkv_stream_t stream)
{
    DeviceInfo dev;
    if (!current_device_info(&dev)) return PKV_ECUDA;
    p.parts = rope_parts(p, dev.sm_count);
    const int64_t grid = (int64_t(p.T) * p.parts + kRopeWarps - 1) / kRopeWarps;
    const cudaError_t e = launch_pdl(interleaved ? rope_kernel<true> : rope_kernel<false>, dim3(unsigned(grid)),
                                     dim3(32 * kRopeWarps), 0, reinterpret_cast<cudaStream_t>(stream), p);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return cuda_fail("rope_kernel launch", e);
    }
    return launch_status("rope_kernel launch");
}

// The norm of a call that has one.
struct Norm {
    const float *qw, *kw;
    float eps;
};

static pkv_status norm_call(const RopeParams &r, const Norm &n, int interleaved, pkv_stream_t stream)
{
    DeviceInfo dev;
    if (!current_device_info(&dev)) return PKV_ECUDA;
    NormParams np{r, n.qw, n.kw, n.eps};
    RopeParams &p = np.r;
    p.parts = rope_parts(p, dev.sm_count);
    const int64_t grid = (int64_t(p.T) * p.parts + kRopeWarps - 1) / kRopeWarps;
    auto pick = [&](auto adj) {
        constexpr bool ADJ = decltype(adj)::value;
        return p.D == 128  ? norm_rope_kernel<ADJ, 8>
               : p.D == 64 ? norm_rope_kernel<ADJ, 4> : p.D == 256 ? norm_rope_kernel<ADJ, 16> : norm_rope_kernel<ADJ, 0>;
    };
    const cudaError_t e = launch_pdl(interleaved ? pick(std::true_type{}) : pick(std::false_type{}), dim3(unsigned(grid)),
                                     dim3(32 * kRopeWarps), 0, reinterpret_cast<cudaStream_t>(stream), np);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return cuda_fail("norm_rope_kernel launch", e);
    }
    return launch_status("norm_rope_kernel launch");
}

// Checks shared by the two entry points; the sizes are nonnegative afterwards.
static pkv_status rope_check(const uint16_t *q, int64_t q_stride, const uint16_t *k, int64_t k_stride,
                             const uint16_t *q_out, int64_t qo_stride, int32_t num_tokens, int32_t num_q_heads,
                             int32_t num_kv_heads, int32_t head_dim, int32_t rot_dim, const int32_t *positions,
                             int32_t num_axes, const float *inv_freq)
{
    if (num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || rot_dim <= 0 ||
        rot_dim > head_dim || num_axes <= 0)
        return PKV_EINVAL;
    if (head_dim % 16 != 0 || head_dim > 2 * kRopeMaxHalf || rot_dim % 16 != 0) return PKV_EUNSUPPORTED;
    if ((int64_t(num_q_heads) + 2 * int64_t(num_kv_heads)) * head_dim > INT32_MAX / 2) return PKV_EBOUNDS;
    if (num_tokens == 0) return PKV_OK;
    if (!q || !k || !q_out || !positions || !inv_freq) return PKV_EINVAL;
    if (!aligned16(q) || !aligned16(k) || !aligned16(q_out)) return PKV_EINVAL;
    const int64_t qrow = int64_t(num_q_heads) * head_dim, krow = int64_t(num_kv_heads) * head_dim;
    if (q_stride < qrow || qo_stride < qrow || k_stride < krow || q_stride % 8 != 0 || qo_stride % 8 != 0 ||
        k_stride % 8 != 0)
        return PKV_EINVAL;
    return PKV_OK;
}

}  // namespace pkv

using namespace pkv;

static bool norm_ok(const Norm &n)
{
    return std::isfinite(n.eps) && n.eps > 0.f && aligned16(n.qw) && aligned16(n.kw);  // (null is aligned)
}

static pkv_status rope_impl(const Norm *norm, const uint16_t *q, int64_t q_stride, const uint16_t *k, int64_t k_stride,
                            const int32_t *positions, int32_t num_axes, const float *inv_freq,
                            const int32_t *freq_axis, int32_t num_tokens, int32_t num_q_heads,
                            int32_t num_kv_heads, int32_t head_dim, int32_t rot_dim, int32_t interleaved,
                            uint16_t *q_out, int64_t q_out_stride, uint16_t *k_out, int64_t k_out_stride,
                            int32_t *err_word, pkv_stream_t stream)
{
    const pkv_status st = rope_check(q, q_stride, k, k_stride, q_out, q_out_stride, num_tokens, num_q_heads,
                                     num_kv_heads, head_dim, rot_dim, positions, num_axes, inv_freq);
    if (st != PKV_OK || num_tokens == 0) return st;
    if (!k_out || !aligned16(k_out) || k_out_stride < int64_t(num_kv_heads) * head_dim || k_out_stride % 8 != 0)
        return PKV_EINVAL;
    RopeParams p{};
    p.q = q;
    p.k = k;
    p.q_out = q_out;
    p.k_out = k_out;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.qo_stride = q_out_stride;
    p.ko_stride = k_out_stride;
    p.positions = positions;
    p.freq_axis = freq_axis;
    p.inv_freq = inv_freq;
    p.axes = num_axes;
    p.T = num_tokens;
    p.Hq = num_q_heads;
    p.Hkv = num_kv_heads;
    p.D = head_dim;
    p.rot = rot_dim;
    p.err = err_word;
    if (norm) return norm_call(p, *norm, interleaved, stream);
    return rope_call(p, interleaved, stream);
}

static pkv_status rope_store_impl(const Norm *norm, const uint16_t *q, int64_t q_stride, const uint16_t *k,
                                  int64_t k_stride, const uint16_t *v, int64_t v_stride, const int32_t *positions,
                                  int32_t num_axes, const float *inv_freq, const int32_t *freq_axis,
                                  const int32_t *slot_mapping, int32_t num_tokens, int32_t num_q_heads,
                                  int32_t num_kv_heads, int32_t head_dim, int32_t rot_dim, int32_t interleaved,
                                  uint16_t *q_out, int64_t q_out_stride, uint16_t *k_cache, uint16_t *v_cache,
                                  int32_t num_blocks, int32_t block_size, int32_t *err_word, pkv_stream_t stream)
{
    if (num_blocks <= 0 || block_size <= 0) return PKV_EINVAL;
    const pkv_status st = rope_check(q, q_stride, k, k_stride, q_out, q_out_stride, num_tokens, num_q_heads,
                                     num_kv_heads, head_dim, rot_dim, positions, num_axes, inv_freq);
    if (st != PKV_OK || num_tokens == 0) return st;
    const int64_t krow = int64_t(num_kv_heads) * head_dim;
    if (!v || !slot_mapping || !k_cache || !v_cache || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) ||
        v_stride < krow || v_stride % 8 != 0)
        return PKV_EINVAL;
    RopeParams p{};
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_out = q_out;
    p.k_out = k_cache;
    p.v_out = v_cache;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.qo_stride = q_out_stride;
    p.ko_stride = krow;
    p.vo_stride = krow;
    p.positions = positions;
    p.freq_axis = freq_axis;
    p.slots = slot_mapping;
    p.inv_freq = inv_freq;
    p.axes = num_axes;
    p.T = num_tokens;
    p.Hq = num_q_heads;
    p.Hkv = num_kv_heads;
    p.D = head_dim;
    p.rot = rot_dim;
    p.num_slots = int64_t(num_blocks) * block_size;
    p.err = err_word;
    if (norm) return norm_call(p, *norm, interleaved, stream);
    return rope_call(p, interleaved, stream);
}

extern "C" pkv_status pkv_rope(const uint16_t *q, int64_t q_stride, const uint16_t *k, int64_t k_stride,
                               const int32_t *positions, int32_t num_axes, const float *inv_freq,
                               const int32_t *freq_axis, int32_t num_tokens, int32_t num_q_heads,
                               int32_t num_kv_heads, int32_t head_dim, int32_t rot_dim, int32_t interleaved,
                               uint16_t *q_out, int64_t q_out_stride, uint16_t *k_out, int64_t k_out_stride,
                               int32_t *err_word, pkv_stream_t stream)
{
    return rope_impl(nullptr, q, q_stride, k, k_stride, positions, num_axes, inv_freq, freq_axis, num_tokens,
                     num_q_heads, num_kv_heads, head_dim, rot_dim, interleaved, q_out, q_out_stride, k_out,
                     k_out_stride, err_word, stream);
}

extern "C" pkv_status pkv_qk_norm_rope(const uint16_t *q, int64_t q_stride, const uint16_t *k, int64_t k_stride,
                                       const float *q_weight, const float *k_weight, float eps,
                                       const int32_t *positions, int32_t num_axes, const float *inv_freq,
                                       const int32_t *freq_axis, int32_t num_tokens, int32_t num_q_heads,
                                       int32_t num_kv_heads, int32_t head_dim, int32_t rot_dim, int32_t interleaved,
                                       uint16_t *q_out, int64_t q_out_stride, uint16_t *k_out, int64_t k_out_stride,
                                       int32_t *err_word, pkv_stream_t stream)
{
    const Norm n{q_weight, k_weight, eps};
    if (!norm_ok(n)) return PKV_EINVAL;
    return rope_impl(&n, q, q_stride, k, k_stride, positions, num_axes, inv_freq, freq_axis, num_tokens,
                     num_q_heads, num_kv_heads, head_dim, rot_dim, interleaved, q_out, q_out_stride, k_out,
                     k_out_stride, err_word, stream);
}

extern "C" pkv_status pkv_rope_store(const uint16_t *q, int64_t q_stride, const uint16_t *k, int64_t k_stride,
                                     const uint16_t *v, int64_t v_stride, const int32_t *positions, int32_t num_axes,
                                     const float *inv_freq, const int32_t *freq_axis, const int32_t *slot_mapping,
                                     int32_t num_tokens, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                     int32_t rot_dim, int32_t interleaved, uint16_t *q_out, int64_t q_out_stride,
                                     uint16_t *k_cache, uint16_t *v_cache, int32_t num_blocks, int32_t block_size,
                                     int32_t *err_word, pkv_stream_t stream)
{
    return rope_store_impl(nullptr, q, q_stride, k, k_stride, v, v_stride, positions, num_axes, inv_freq, freq_axis,
                           slot_mapping, num_tokens, num_q_heads, num_kv_heads, head_dim, rot_dim, interleaved, q_out,
                           q_out_stride, k_cache, v_cache, num_blocks, block_size, err_word, stream);
}

extern "C" pkv_status pkv_qk_norm_rope_store(const uint16_t *q, int64_t q_stride, const uint16_t *k, int64_t k_stride,
                                             const uint16_t *v, int64_t v_stride, const float *q_weight,
                                             const float *k_weight, float eps, const int32_t *positions,
                                             int32_t num_axes, const float *inv_freq, const int32_t *freq_axis,
                                             const int32_t *slot_mapping, int32_t num_tokens, int32_t num_q_heads,
                                             int32_t num_kv_heads, int32_t head_dim, int32_t rot_dim,
                                             int32_t interleaved, uint16_t *q_out, int64_t q_out_stride,
                                             uint16_t *k_cache, uint16_t *v_cache, int32_t num_blocks,
                                             int32_t block_size, int32_t *err_word, pkv_stream_t stream)
{
    const Norm n{q_weight, k_weight, eps};
    if (!norm_ok(n)) return PKV_EINVAL;
    return rope_store_impl(&n, q, q_stride, k, k_stride, v, v_stride, positions, num_axes, inv_freq, freq_axis,
                           slot_mapping, num_tokens, num_q_heads, num_kv_heads, head_dim, rot_dim, interleaved, q_out,
                           q_out_stride, k_cache, v_cache, num_blocks, block_size, err_word, stream);
}
