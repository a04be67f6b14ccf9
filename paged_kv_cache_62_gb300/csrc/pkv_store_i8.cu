// Stores and page copies of the int8 cache with a scale per block of 16 tokens and kv head.
//
// pkv_kv_store_i8: for every scale block that the call's new rows reach, with a = the largest |x| of the
//   block's new rows (per kv head, K and V apart) and s the block's scale so far:
//     s' = a * fl(1 / 127)         if the call writes the block's first row, else max(s, a * fl(1 / 127));
//     code(x) = x / s' rounded to nearest even, for the new rows;
//     code'   = code * s / s' rounded to nearest even, for the earlier rows, where s' > s.
//   Every quotient is rounded once, as if it were exact: an approximate quotient gives the integer, or next to
//   a tie its neighbour, and an exact fused residual tells (see quantise8_i8 and exact_code).
// pkv_copy_blocks_i8: block dst of the two code arrays and of the scales becomes a copy of block src.
//
// The store gives one warp a (scale block, kv head, K or V): the block's maximum, its scale and its codes need no
// atomics and no second launch, and the result does not depend on the order in which warps run.  The rows are read
// twice, the second time from L1: 16 rows of 128 values held in registers would leave half the warps on an SM.
// Prompts: 22k rows of 8 heads of 128, 137 MB, in 30.9 us = 4.4 TB/s, 0.65 of the copy rate; with a division a value
// 73 us, with the rows in registers 52 us.  No one resource holds them: instructions issue in 66 % of the cycles
// (15 a value and lane, half of them the rounding and its check), and a warp's longest wait is for the rows, its two
// passes over them one after the other.  A decode step's 64 rows take 2.9 us, a launch and its dependent loads; a
// step that grows every block's scale 4.5 us with one earlier row to requantise a block and 12 us with fourteen
// (one code at a time, out of line: rare in a real run, where a block's maximum grows ever more seldom).
// The copies are memory-bound: 120 pages of 256 tokens, 126 MB, in 20.6 us = 6.1 TB/s, 0.90 of the copy rate.
#include <algorithm>

#include "pkv_device.cuh"
#include "pkv_host.h"

namespace pkv {

constexpr int kSB = PKV_I8_BLOCK;  // tokens a scale block holds
constexpr int kStoreThreads = 256;
constexpr float kRound = 12582912.0f;  // 1.5 * 2^23: adding it rounds a small float to an integer, ties to even

struct StoreI8Params {
    const uint16_t *k, *v;
    long long k_stride, v_stride;  // elements between rows
    const int32_t *block_tables, *cu_seqlens, *context_lens;
    int32_t max_blocks, new_per_seq, slots_per_seq, num_seqs, num_tokens;
    int8_t *k_cache, *v_cache;
    float *scales;  // [NB * bs / kSB][Hkv][2]
    int32_t num_blocks, block_size, log2_bs, Hkv;
    int32_t *err;
};

// (hi + lo) / s rounded to the nearest integer, ties to even, exactly (|lo| <= half an ulp of hi, s > 0, the
// quotient at most 127.5): t is the rounding of an approximate quotient q (off by less than 2^-16), which is
// wrong only next to a tie b = t +- 1/2, and there the sign of hi + lo - b s decides: b has 8 bits and s 24, so
// hi - b s is exact where it is small.
__device__ __forceinline__ int exact_code(float hi, float lo, float s, float inv)
{
    const float q = hi * inv, t = rintf(q);
    const float half = q >= t ? 0.5f : -0.5f;
    const float e = __fadd_rn(__fmaf_rn(-(t + half), s, hi), lo);
    const int ti = int(t), away = half > 0.f ? ti + 1 : ti - 1;
    const bool past = half > 0.f ? e > 0.f : e < 0.f;
    const int c = past ? away : (e == 0.f && (ti & 1) ? away : ti);
    return max(-127, min(127, c));
}

// Eight bf16 values over s as int8 codes (element e in byte e), exactly: t = x * inv rounded (inv is 1 / s
// rounded) is the code or, next to a tie, its neighbour, and the residual x - t s, exact in fp32, tells: the code
// is t where its magnitude stays below s / 2.  (With bf16 rows near-ties are no rarity: 127 x / a has few bits
// for many x and a.  Checking the residual leaves the corrections to the few that rounded the wrong way.)
__device__ __forceinline__ uint2 quantise8_i8(const uint4 w, float s, float inv)
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    uint32_t c[8];
    float far = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float x = __uint_as_float(e & 1 ? u[e >> 1] & 0xffff0000u : u[e >> 1] << 16);
        const float r = __fmaf_rn(x, inv, kRound);  // its low byte is the code
        far = fmaxf(far, fabsf(__fmaf_rn(kRound - r, s, x)));
        c[e] = __float_as_uint(r);
    }
    const float half = 0.5f * s;
    if (far >= half) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x = __uint_as_float(e & 1 ? u[e >> 1] & 0xffff0000u : u[e >> 1] << 16);
            const float d = __fmaf_rn(kRound - __uint_as_float(c[e]), s, x);
            if (fabsf(d) > half || (fabsf(d) == half && (c[e] & 1u))) c[e] += d > 0.f ? 1u : ~0u;
        }
    }
    auto pack = [&](int i) {
        return __byte_perm(__byte_perm(c[i], c[i + 1], 0x0040), __byte_perm(c[i + 2], c[i + 3], 0x0040), 0x5410);
    };
    return make_uint2(pack(0), pack(4));
}

// The earlier rows' eight codes from scale s0 to scale s.
__device__ __noinline__ uint2 requantise8_i8(uint2 w, float s0, float s)
{
    const float lift = s < 0x1p-100f ? 0x1p+110f : 1.0f;  // keeps 1 / s and the residuals in range
    s *= lift;
    const float inv = __fdiv_rn(1.0f, s);
#pragma unroll 1
    for (int e = 0; e < 8; ++e) {
        const float c = float(int(int8_t(w.x & 0xffu)));
        const float hi = __fmul_rn(c, s0), lo = __fmaf_rn(c, s0, -hi);
        w.x = (w.x >> 8) | (w.y << 24);
        w.y = (w.y >> 8) | (uint32_t(exact_code(hi * lift, lo * lift, s, inv)) << 24);
    }
    return w;
}

// Eight bf16 values times 2^110 (a block of tiny values, see kv_store_i8_kernel).
__device__ __forceinline__ uint4 lifted(uint4 w)
{
    uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        u[i] = pack_bf16x2(__uint_as_float(u[i] << 16) * 0x1p+110f, __uint_as_float(u[i] & 0xffff0000u) * 0x1p+110f);
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// One CTA (or, for few slots, a few: blockIdx.y) per slot of the block list; its warps take the (kv head, K or V)
// pairs of the slot's scale block.  Slots: with new_per_seq each sequence has slots_per_seq of them (as many blocks
// as n rows can reach); with offsets sequence b has those from cu[b] / 16 + 2 b on, which leaves room for the
// floor((n + 14) / 16) + 1 blocks that n rows can reach, so a slot finds its sequence by a search over the offsets
// and no prefix over blocks is needed.
template <int D>
__global__ void __launch_bounds__(kStoreThreads, 5) kv_store_i8_kernel(const StoreI8Params p)
{
    constexpr int LR = D / 8;        // lanes per row (16 bytes of bf16 each)
    constexpr int RPL = 32 / LR;     // rows per load of the warp
    constexpr int NV = kSB / RPL;    // loads that cover the block's rows
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    int32_t b, i, r0, n, L;
    if (p.cu_seqlens) {
        // The search below sees only some of the offsets, so CTA x also looks whether offset x decreases (there are
        // at least two CTAs a sequence).
        bool down = false;
        if (threadIdx.x == 0 && int(blockIdx.x) < p.num_seqs)
            down = __ldg(p.cu_seqlens + blockIdx.x) > __ldg(p.cu_seqlens + blockIdx.x + 1);
        // the last b with cu[b] / 16 + 2 b <= slot, by 32-way steps
        int lo = 0, width = p.num_seqs;
        while (width > 1) {
            const int step = (width + 31) / 32;
            const int c = lo + lane * step;
            const bool le = lane * step < width &&
                            (max(0, __ldg(p.cu_seqlens + c)) >> 4) + 2 * (long long)c <= (long long)blockIdx.x;
            const unsigned m = __ballot_sync(kFull, le);
            const int k = m ? 31 - __clz(m) : 0;
            lo += k * step;
            width = min(step, width - k * step);
        }
        b = lo;
        r0 = __ldg(p.cu_seqlens + b);
        L = __ldg(p.context_lens + b);
        const int32_t r1 = __ldg(p.cu_seqlens + b + 1);
        const int32_t before = __ldg(p.cu_seqlens + max(b - 1, 0)), after = __ldg(p.cu_seqlens + min(b + 2, p.num_seqs));
        i = int32_t(blockIdx.x) - ((max(0, r0) >> 4) + 2 * b);
        n = r1 - r0;
        if (down) flag_error(p.err, PKV_ERR_CONTEXT_RANGE);
        if (r0 < 0 || r1 < r0 || r1 > p.num_tokens || (b == 0 && r0 != 0) || before > r0 || r1 > after) {
            if (threadIdx.x == 0) flag_error(p.err, PKV_ERR_CONTEXT_RANGE);
            return;
        }
    } else {
        b = int32_t(blockIdx.x) / p.slots_per_seq;
        i = int32_t(blockIdx.x) - b * p.slots_per_seq;
        n = p.new_per_seq;
        r0 = b * n;
        L = __ldg(p.context_lens + b);
    }
    if (n == 0 || i < 0 || (L == 0 && !p.cu_seqlens)) return;  // no rows, or a padding sequence
    if (L < n || L > int64_t(p.max_blocks) * p.block_size) {
        if (threadIdx.x == 0 && i == 0) flag_error(p.err, PKV_ERR_CONTEXT_RANGE);
        return;
    }
    const int32_t p0 = L - n;                       // position of the first new row
    const int64_t base64 = int64_t(p0 & ~(kSB - 1)) + int64_t(i) * kSB;  // position of this block's first row
    if (base64 >= L) return;
    const int32_t base = int32_t(base64);
    const int32_t first = max(p0 - base, 0), last = min(L - base, kSB);  // new rows of the block
    const int32_t phys = __ldg(p.block_tables + int64_t(b) * p.max_blocks + (base >> p.log2_bs));
    const int row = lane / LR, col = (lane - row * LR) * 8;
    const int64_t src0 = int64_t(r0) + (base - p0);  // input row of the block's row 0 (may lie before the input)
    if (phys < 0 || phys >= p.num_blocks) {
        if (threadIdx.x == 0) flag_error(p.err, PKV_ERR_BLOCK_RANGE);
        return;
    }
    const int64_t crow = int64_t(phys) * p.block_size + (base & (p.block_size - 1));  // cache row of the block

    for (int w = warp + int(blockIdx.y) * nwarps; w < 2 * p.Hkv; w += nwarps * int(gridDim.y)) {
        const int which = w & 1, h = w >> 1;
        const uint16_t *x = (which ? p.v : p.k) + int64_t(h) * D + col;
        const int64_t stride = which ? p.v_stride : p.k_stride;
        int8_t *codes = (which ? p.v_cache : p.k_cache) + (crow * p.Hkv + h) * D + col;
        float *sp = p.scales + ((crow / kSB) * p.Hkv + h) * 2 + which;
        const float s0 = first > 0 ? *sp : 0.f;
        // the block's largest magnitude; two bf16 a lane-word, compared as such (a NaN wins, infinities are seen)
        __nv_bfloat162 top = __float2bfloat162_rn(0.f);
#pragma unroll
        for (int j0 = 0; j0 < NV; j0 += 4) {  // four loads in flight a thread: 40 warps an SM
            uint4 in[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = (j0 + j) * RPL + row;
                in[j] = make_uint4(0u, 0u, 0u, 0u);
                if (r >= first && r < last) in[j] = __ldg(reinterpret_cast<const uint4 *>(x + (src0 + r) * stride));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t u[4] = {in[j].x, in[j].y, in[j].z, in[j].w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    top = __hmax2_nan(top, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&u[e])));
            }
        }
        const uint32_t tb = *reinterpret_cast<const uint32_t *>(&top);
        const uint32_t mx = __reduce_max_sync(kFull, max(tb & 0x7fffu, (tb >> 16) & 0x7fffu));
        // an infinity or NaN makes the block's scale NaN (and a NaN scale stays until the block starts anew)
        float s = mx >= 0x7f80u ? __uint_as_float(0x7fc00000u) : __fmul_rn(__uint_as_float(mx << 16), 1.0f / 127.0f);
        if (first > 0) s = s0 >= s ? s0 : (s0 < s ? s : __uint_as_float(0x7fc00000u));
        const bool fine = s > 0.f;  // not zero, not NaN
        const bool tiny = fine && s < 0x1p-100f;  // lifted by 2^110: 1 / s and the residuals stay in range
        const float sq = !fine ? 1.0f : tiny ? s * 0x1p+110f : s, inv = __fdiv_rn(1.0f, sq);
        if (first > 0 && s > s0) {  // the scale grew: the earlier rows move to it
#pragma unroll 1
            for (int r = row; r < first; r += RPL) {
                uint2 *at = reinterpret_cast<uint2 *>(codes + int64_t(r) * p.Hkv * D);
                *at = requantise8_i8(*at, s0, s);
            }
        }
        // the rows once more, from L1: holding them in registers would halve the warps an SM has in flight
        const int rf = first + ((row - first) & (RPL - 1));
        const uint16_t *xr = x + (src0 + rf) * stride;
        int8_t *cr = codes + int64_t(rf) * p.Hkv * D;
#pragma unroll 2
        for (int r = rf; r < last; r += RPL, xr += RPL * stride, cr += int64_t(RPL) * p.Hkv * D) {
            uint4 w = __ldg(reinterpret_cast<const uint4 *>(xr));
            if (tiny) w = lifted(w);
            *reinterpret_cast<uint2 *>(cr) = fine ? quantise8_i8(w, sq, inv) : make_uint2(0u, 0u);
        }
        __syncwarp();  // every lane has read the old scale
        if (lane == 0) *sp = s;
    }
}

// Page copies: chunks of 32 KiB of one page of one code array, and one chunk for the page's scales; a
// persistent grid walks them with eight 16-byte loads in flight a thread (as copy_blocks_kernel).
constexpr int kCopyI8Threads = 256;
constexpr int kCopyI8Vecs = 8;
constexpr int64_t kCopyI8Chunk = kCopyI8Threads * kCopyI8Vecs;

__global__ void __launch_bounds__(kCopyI8Threads) copy_blocks_i8_kernel(uint4 *__restrict__ k_cache,
                                                                      uint4 *__restrict__ v_cache,
                                                                      uint2 *__restrict__ scales,
                                                                      const int32_t *__restrict__ pairs,
                                                                      int32_t num_pairs, int32_t num_blocks,
                                                                      int64_t block_vecs, int64_t block_scales,
                                                                      int32_t chunks, int32_t *err)
{
    griddep_launch_dependents();
    griddep_wait();
    const int32_t per = 2 * chunks + 1;
    const int64_t total = int64_t(num_pairs) * per;
    for (int64_t c = blockIdx.x; c < total; c += gridDim.x) {
        const int32_t i = int32_t(c / per), part = int32_t(c - int64_t(i) * per);
        const int32_t src = __ldg(pairs + 2 * i), dst = __ldg(pairs + 2 * i + 1);
        if (src < 0 || src >= num_blocks || dst < 0 || dst >= num_blocks) {
            if (threadIdx.x == 0 && part == 0) flag_error(err, PKV_ERR_BLOCK_RANGE);
            continue;
        }
        if (src == dst) continue;
        if (part == 2 * chunks) {
            const uint2 *from = scales + src * block_scales;
            uint2 *to = scales + dst * block_scales;
            for (int64_t v = threadIdx.x; v < block_scales; v += kCopyI8Threads) to[v] = __ldcg(from + v);
            continue;
        }
        uint4 *base = part >= chunks ? v_cache : k_cache;
        const uint4 *from = base + int64_t(src) * block_vecs;
        uint4 *to = base + int64_t(dst) * block_vecs;
        const int64_t v0 = int64_t(part >= chunks ? part - chunks : part) * kCopyI8Chunk + threadIdx.x;
        uint4 x[kCopyI8Vecs];
#pragma unroll
        for (int j = 0; j < kCopyI8Vecs; ++j)
            if (v0 + int64_t(j) * kCopyI8Threads < block_vecs) x[j] = __ldcg(from + v0 + int64_t(j) * kCopyI8Threads);
#pragma unroll
        for (int j = 0; j < kCopyI8Vecs; ++j)
            if (v0 + int64_t(j) * kCopyI8Threads < block_vecs) to[v0 + int64_t(j) * kCopyI8Threads] = x[j];
    }
}

}  // namespace pkv

using namespace pkv;

extern "C" pkv_status pkv_kv_store_i8(const uint16_t *k, const uint16_t *v, int64_t k_stride, int64_t v_stride,
                                      const int32_t *block_tables, int32_t max_blocks_per_seq,
                                      const int32_t *cu_seqlens, const int32_t *context_lens, int32_t num_seqs,
                                      int32_t num_tokens, int32_t new_per_seq, int8_t *k_cache, int8_t *v_cache,
                                      float *scales, int32_t num_blocks, int32_t block_size, int32_t num_kv_heads,
                                      int32_t head_dim, int32_t *err_word, pkv_stream_t stream)
{
    if (num_seqs < 0 || num_tokens < 0 || new_per_seq < 0 || max_blocks_per_seq <= 0 || num_blocks <= 0 ||
        num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0)
        return PKV_EINVAL;
    if (head_dim != 64 && head_dim != 128) return PKV_EUNSUPPORTED;
    if (!is_pow2(block_size) || block_size < kSB || block_size > 1024) return PKV_EUNSUPPORTED;
    if (int64_t(num_blocks) * block_size > INT32_MAX || int64_t(num_kv_heads) * head_dim > INT32_MAX / 2)
        return PKV_EBOUNDS;
    if (num_tokens == 0) return PKV_OK;
    if (num_seqs == 0 || (new_per_seq == 0 && !cu_seqlens)) return PKV_EINVAL;
    if (new_per_seq > 0 && int64_t(num_seqs) * new_per_seq != num_tokens) return PKV_EINVAL;
    if (!k || !v || !block_tables || !context_lens || !k_cache || !v_cache || !scales) return PKV_EINVAL;
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) ||
        (reinterpret_cast<uintptr_t>(scales) & 7u))
        return PKV_EINVAL;
    const int64_t row = int64_t(num_kv_heads) * head_dim;
    if (k_stride < row || v_stride < row || k_stride % 8 != 0 || v_stride % 8 != 0) return PKV_EINVAL;
    StoreI8Params p{};
    p.k = k;
    p.v = v;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.block_tables = block_tables;
    p.cu_seqlens = new_per_seq > 0 ? nullptr : cu_seqlens;
    p.context_lens = context_lens;
    p.max_blocks = max_blocks_per_seq;
    p.new_per_seq = new_per_seq;
    p.slots_per_seq = new_per_seq > 0 ? (new_per_seq + kSB - 2) / kSB + 1 : 0;
    p.num_seqs = num_seqs;
    p.num_tokens = num_tokens;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.scales = scales;
    p.num_blocks = num_blocks;
    p.block_size = block_size;
    p.log2_bs = ilog2(block_size);
    p.Hkv = num_kv_heads;
    p.err = err_word;
    const int64_t grid = new_per_seq > 0 ? int64_t(num_seqs) * p.slots_per_seq
                                         : int64_t(num_tokens) / kSB + 2 * int64_t(num_seqs);
    if (grid > INT32_MAX) return PKV_EBOUNDS;
    // Few slots (a decode step): small CTAs with one (kv head, K or V) a warp, several a slot, so that the step takes
    // one warp's latency (64 rows of 8 kv heads: 4.8 -> 2.8 us).  Many: one CTA a slot, whose warps share the search
    // for its sequence (22k prompt rows: 30.9 us against 31.5 with the others).
    DeviceInfo dev;
    if (!current_device_info(&dev)) return PKV_ECUDA;
    const bool few = grid < 4 * int64_t(dev.sm_count);
    const int threads = std::min(64 * num_kv_heads, few ? 128 : kStoreThreads);
    const int parts = few ? (64 * num_kv_heads + threads - 1) / threads : 1;
    if (parts > 65535) return PKV_EBOUNDS;
    const cudaError_t e = launch_pdl(head_dim == 64 ? kv_store_i8_kernel<64> : kv_store_i8_kernel<128>,
                                     dim3(unsigned(grid), unsigned(parts)), dim3(threads), 0,
                                     reinterpret_cast<cudaStream_t>(stream), p);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return cuda_fail("kv_store_i8_kernel launch", e);
    }
    return launch_status("kv_store_i8_kernel launch");
}

extern "C" pkv_status pkv_copy_blocks_i8(int8_t *k_cache, int8_t *v_cache, float *scales, const int32_t *pairs,
                                         int32_t num_pairs, int32_t num_blocks, int32_t block_size,
                                         int32_t num_kv_heads, int32_t head_dim, int32_t *err_word,
                                         pkv_stream_t stream)
{
    if (num_pairs < 0 || num_blocks <= 0 || block_size <= 0 || num_kv_heads <= 0 || head_dim <= 0)
        return PKV_EINVAL;
    if (block_size % kSB != 0) return PKV_EUNSUPPORTED;
    if (int64_t(num_blocks) * block_size > INT32_MAX || int64_t(num_kv_heads) * head_dim > INT32_MAX / 2)
        return PKV_EBOUNDS;
    if (num_pairs == 0) return PKV_OK;
    if (!k_cache || !v_cache || !scales || !pairs) return PKV_EINVAL;
    if (!aligned16(k_cache) || !aligned16(v_cache) || (reinterpret_cast<uintptr_t>(scales) & 7u)) return PKV_EINVAL;
    DeviceInfo dev;
    if (!current_device_info(&dev)) return PKV_ECUDA;
    const int64_t block_vecs = int64_t(block_size) * num_kv_heads * head_dim / 16;  // block_size % 16 == 0
    const int64_t block_scales = int64_t(block_size / kSB) * num_kv_heads;
    const int64_t chunks = (block_vecs + kCopyI8Chunk - 1) / kCopyI8Chunk;
    if (chunks > INT32_MAX / 4) return PKV_EBOUNDS;
    const int64_t grid = std::min<int64_t>(int64_t(num_pairs) * (2 * chunks + 1), int64_t(dev.sm_count) * 8);
    const cudaError_t e = launch_pdl(copy_blocks_i8_kernel, dim3(unsigned(grid)), dim3(kCopyI8Threads), 0,
                                     reinterpret_cast<cudaStream_t>(stream), reinterpret_cast<uint4 *>(k_cache),
                                     reinterpret_cast<uint4 *>(v_cache), reinterpret_cast<uint2 *>(scales), pairs,
                                     num_pairs, num_blocks, block_vecs, block_scales, int32_t(chunks), err_word);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return cuda_fail("copy_blocks_i8_kernel launch", e);
    }
    return launch_status("copy_blocks_i8_kernel launch");
}
