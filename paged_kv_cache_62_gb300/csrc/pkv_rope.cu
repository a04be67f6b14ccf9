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
//
// With a norm (NORM), a q or k head x becomes x / sqrt(mean x^2 + eps) * w before the turn: the D / 16 lanes that
// hold a head add up their squares with shuffles, and the row's factor and the weights join the turn's products, so
// the head makes no second trip through registers.
#include <algorithm>
#include <cmath>

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
    const float *qw, *kw;  // NORM: weights of a q and a k head (null: ones)
    float eps;
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

// The same for a head that is normed first: a and b times r and the weights at wa and wb (null: ones); turned or not.
template <bool ADJ>
__device__ __forceinline__ void norm_turn16(uint4 &a, uint4 &b, const float2 *cs, bool turn, float r, const float *wa,
                                            const float *wb)
{
    const uint32_t ua[4] = {a.x, a.y, a.z, a.w}, ub[4] = {b.x, b.y, b.z, b.w};
    float x[8], y[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = __uint_as_float(ua[j] << 16) * r;
        x[2 * j + 1] = __uint_as_float(ua[j] & 0xffff0000u) * r;
        y[2 * j] = __uint_as_float(ub[j] << 16) * r;
        y[2 * j + 1] = __uint_as_float(ub[j] & 0xffff0000u) * r;
    }
    if (wa) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float4 u = __ldg(reinterpret_cast<const float4 *>(wa) + j);
            const float4 v = __ldg(reinterpret_cast<const float4 *>(wb) + j);
            x[4 * j] *= u.x;
            x[4 * j + 1] *= u.y;
            x[4 * j + 2] *= u.z;
            x[4 * j + 3] *= u.w;
            y[4 * j] *= v.x;
            y[4 * j + 1] *= v.y;
            y[4 * j + 2] *= v.z;
            y[4 * j + 3] *= v.w;
        }
    }
    if (turn) {
#pragma unroll
        for (int e = 0; e < (ADJ ? 4 : 8); ++e) {
            if constexpr (ADJ) {
                const float p = x[2 * e], q = y[2 * e];
                x[2 * e] = p * cs[e].x - x[2 * e + 1] * cs[e].y;
                x[2 * e + 1] = x[2 * e + 1] * cs[e].x + p * cs[e].y;
                y[2 * e] = q * cs[4 + e].x - y[2 * e + 1] * cs[4 + e].y;
                y[2 * e + 1] = y[2 * e + 1] * cs[4 + e].x + q * cs[4 + e].y;
            } else {
                const float p = x[e];
                x[e] = p * cs[e].x - y[e] * cs[e].y;
                y[e] = y[e] * cs[e].x + p * cs[e].y;
            }
        }
    }
    a = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    b = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
}

__device__ __forceinline__ float squares(uint4 a)
{
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float lo = __uint_as_float(u[j] << 16), hi = __uint_as_float(u[j] & 0xffff0000u);
        s0 = fmaf(lo, lo, s0);
        s1 = fmaf(hi, hi, s1);
    }
    return s0 + s1;
}

constexpr int kRopeWarps = 2;  // warps (token parts) a CTA: small ones, whose last warp holds little back

template <bool ADJ, bool NORM>
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
    uint4 a[B] = {}, b[B] = {};
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
    const bool pow2 = (per & (per - 1)) == 0;
    for (int h1 = h0; NORM ? h1 - hl < heads : h1 < heads; h1 += step) {  // (NORM: the lanes stay together)
        float rs[B];
        if constexpr (NORM) {
            float ss[B];
#pragma unroll
            for (int k = 0; k < B; ++k) ss[k] = squares(a[k]) + squares(b[k]);
            if (pow2) {
                for (int o = 1; o < per; o <<= 1)
#pragma unroll
                    for (int k = 0; k < B; ++k) ss[k] += __shfl_xor_sync(kFull, ss[k], o);
            } else {
                float all[B] = {};
                for (int i = 0; i < per; ++i)
#pragma unroll
                    for (int k = 0; k < B; ++k) all[k] += __shfl_sync(kFull, ss[k], hl * per + i);
#pragma unroll
                for (int k = 0; k < B; ++k) ss[k] = all[k];
            }
#pragma unroll
            for (int k = 0; k < B; ++k) rs[k] = rsqrtf(fmaf(ss[k], 1.0f / float(p.D), p.eps));
        }
#pragma unroll
        for (int k = 0; k < B; ++k) {
            const int h = h1 + k * hpw * p.parts;
            const uint16_t *src;
            uint16_t *dst;
            if (place(h, src, dst)) {
                if constexpr (NORM) {
                    if (h < turning) {
                        const float *w = h < p.Hq ? p.qw : p.kw;
                        norm_turn16<ADJ>(a[k], b[k], mycs, c < turned, rs[k], w ? w + d0(h) : nullptr, w + d1(h));
                    }
                } else if (c < turned && h < turning)
                    turn16<ADJ>(a[k], b[k], mycs);
                *reinterpret_cast<uint4 *>(dst + d0(h)) = a[k];
                *reinterpret_cast<uint4 *>(dst + d1(h)) = b[k];
            }
        }
        load(h1 + step);
    }
}

static pkv_status rope_call(RopeParams &p, int interleaved, pkv_stream_t stream, bool norm = false)
{
    DeviceInfo dev;
    if (!current_device_info(&dev)) return PKV_ECUDA;
    // few tokens: several warps a token, each with a part of the heads (as many as leave every lane a piece), until
    // the SMs have eight warps each
    const int heads = p.Hq + p.Hkv + (p.v ? p.Hkv : 0), hpw = 32 / (p.D / 16);
    const int most = (heads + hpw - 1) / hpw;
    p.parts = int(std::min<int64_t>(most, std::max<int64_t>(1, int64_t(dev.sm_count) * 8 / p.T)));
    const int64_t grid = (int64_t(p.T) * p.parts + kRopeWarps - 1) / kRopeWarps;
    auto kern = norm ? (interleaved ? rope_kernel<true, true> : rope_kernel<false, true>)
                     : (interleaved ? rope_kernel<true, false> : rope_kernel<false, false>);
    const cudaError_t e = launch_pdl(kern, dim3(unsigned(grid)), dim3(32 * kRopeWarps), 0,
                                     reinterpret_cast<cudaStream_t>(stream), p);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return cuda_fail("rope_kernel launch", e);
    }
    return launch_status("rope_kernel launch");
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

// The norm of a call that has one.
struct Norm {
    const float *qw, *kw;
    float eps;
};

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
    if (norm) {
        p.qw = norm->qw;
        p.kw = norm->kw;
        p.eps = norm->eps;
    }
    return rope_call(p, interleaved, stream, norm != nullptr);
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
    if (norm) {
        p.qw = norm->qw;
        p.kw = norm->kw;
        p.eps = norm->eps;
    }
    return rope_call(p, interleaved, stream, norm != nullptr);
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
