// Kernels around the paged latent cache: rotary positions, the write of new rows
// (bf16, or e4m3 with one power-of-two scale per page), and the fork, free, copy
// and compaction of pages (include/mla_cache.h).
//
// All of them move bytes: their floor is the data read once and written once,
// and for the small calls the launch.  A decode kernel reads the cache, the table
// and the lengths before its own wait on the previous grid.  It reads what these
// calls wrote, because a call's last kernel lets no dependent grid start before its end and, where it writes
// any of these, ends with a device-wide fence; a kernel of the call before it (the
// check, a plan) lets the next one start early, but every CTA of that one begins with a wait
// for its end.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <cstdint>

#include "mla_cache.h"
#include "schedule.cuh"
#include "sm100_ptx.cuh"

namespace mla {

constexpr int kRopePairs = 32;
constexpr int kMoveThreads = 256;

// ------------------------------------------------------------------ e4m3
// Two e4m3 values of (lo, hi), lo in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t h2_of_e4m3x2(uint32_t v) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(v)));
    return r;
}
__device__ __forceinline__ __half2 as_h2(uint32_t v) { return *reinterpret_cast<__half2*>(&v); }
__device__ __forceinline__ uint32_t as_u32(__half2 v) { return *reinterpret_cast<uint32_t*>(&v); }

// Exponent e of the power-of-two scale of a largest magnitude amax (its bits;
// finite, > 0): the least e with amax <= 448 * 2^e.  448 = 1.75 * 2^8.
__host__ __device__ __forceinline__ int e4m3_scale_exp(uint32_t amax_bits) {
    return static_cast<int>(amax_bits >> 23) - 127 - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
}
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }

constexpr uint32_t kInfBits = 0x7f800000u;
constexpr int kMinScaleExp = -100, kMaxScaleExp = 119;

// ------------------------------------------------------------------ rotation
// cos and sin (times the amplitude) of pair i at a position.  The angle in
// turns is a product of 53-bit numbers, so its fraction is good to 2^-53 of the
// whole turns: 1e-7 turns are not reached below 2^29 turns.  Rounded to fp32 alone that fraction
// would move a small cosine by 1e-7; what the rounding leaves turns the pair once more, to first order.
__device__ __forceinline__ float2 rope_cos_sin(const double* turns, float amplitude, int pos, int i) {
    const double t = static_cast<double>(pos) * turns[i];
    const double half = 2.0 * (t - rint(t));  // half turns
    const float f = static_cast<float>(half);
    const float rest = static_cast<float>(half - f) * 3.14159265f;
    float s, c;
    sincospif(f, &s, &c);
    return make_float2(fmaf(-s, rest, c) * amplitude, fmaf(c, rest, s) * amplitude);
}
__device__ __forceinline__ void rotate(float& a, float& b, float2 cs) {
    const float x = a * cs.x - b * cs.y, y = a * cs.y + b * cs.x;
    a = x;
    b = y;
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        f[2 * e] = __uint_as_float(w[e] << 16);
        f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

struct RopeParams {
    const void* x;
    const int32_t* positions;
    void* out;
    int64_t xt, xh, ot, oh;  // strides in values
    int T, h, offset, transpose;
    int tpc, hpc;            // tokens and heads per CTA
    int per_row, rows_pass;  // units per row, rows per pass of the CTA's threads
    mla_rope_table table;
};

// 8 consecutive columns, as loaded.
template <typename E>
struct Chunk8;
template <>
struct Chunk8<__nv_bfloat16> {
    uint4 v;
    __device__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
    __device__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = v; }
    __device__ void get(float (&f)[8]) const { unpack8(v, f); }
    __device__ void set(const float (&f)[8]) { v = pack8(f); }
};
template <>
struct Chunk8<float> {
    float4 a, b;
    __device__ void load(const float* p) {
        a = *reinterpret_cast<const float4*>(p);
        b = *reinterpret_cast<const float4*>(p + 4);
    }
    __device__ void store(float* p) const {
        *reinterpret_cast<float4*>(p) = a;
        *reinterpret_cast<float4*>(p + 4) = b;
    }
    __device__ void get(float (&f)[8]) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    __device__ void set(const float (&f)[8]) {
        a = make_float4(f[0], f[1], f[2], f[3]);
        b = make_float4(f[4], f[5], f[6], f[7]);
    }
};

// A CTA takes tpc tokens x hpc heads.  A thread owns one unit of a row (8 columns; in
// the half layout's rotary part 16, whose pairs lie 32 columns apart) and walks
// the rows with it, kRopeUnroll of them in flight, so that nothing is divided per
// unit.  The first rows are on their way while the angles of the CTA's
// tokens are computed, once, into shared memory for every head.  Bound by the
// bytes of x and out; small calls by the launch.  B200, 4099 tokens x 128 heads x 192
// bf16 columns (403 MB, 61.5 us at the copy rate), half layout: 111 us with a division
// per unit and the angles first; 97 us without, 4 rows in flight per thread and 3 CTAs
// per SM; 84 us with 4 CTAs; 76.3 us with 2 rows and 6 CTAs, as it is (1 row and
// 8 CTAs 78.2, 2 and 8 84.4; 64 or 256 instead of 128 rows per CTA 77.9 and 92.1).
constexpr int kRopeUnroll = 2;
constexpr int kRopeMaxTokens = 16;
template <typename E, bool kInterleaved>
__global__ void __launch_bounds__(kMoveThreads, sizeof(E) == 2 ? 6 : 4) mla_rope_kernel(const __grid_constant__ RopeParams p) {
    __shared__ float2 cs[kRopeMaxTokens][kRopePairs];
    constexpr int kRot = kInterleaved ? 8 : 4;  // units of the rotary part
    const int t0 = blockIdx.x * p.tpc, h0 = blockIdx.y * p.hpc;
    const int nt = min(p.tpc, p.T - t0), nh = min(p.hpc, p.h - h0);
    const int rows = nt * nh;
    const int r0 = threadIdx.x / p.per_row, u = threadIdx.x - r0 * p.per_row;
    const bool rot = u < kRot;
    // rotary units first, then the columns around them
    const int off8 = p.offset / 8;
    const int col = 8 * (rot ? off8 + u : u - kRot < off8 ? u - kRot : u - kRot + 8);
    const E* x = static_cast<const E*>(p.x) + (int64_t)t0 * p.xt + (int64_t)h0 * p.xh + col;
    E* out = static_cast<E*>(p.out) + (int64_t)t0 * p.ot + (int64_t)h0 * p.oh + col;
    const int mine = r0 < p.rows_pass ? rows : 0;  // (the last threads of the block may own no unit)
    Chunk8<E> v[kRopeUnroll], v2[kInterleaved ? 1 : kRopeUnroll];
    auto load = [&](int base) {
#pragma unroll
        for (int i = 0; i < kRopeUnroll; ++i) {
            const int row = base + r0 + i * p.rows_pass;
            if (row < mine) {
                const int t = p.tpc == 1 ? 0 : row / nh;
                const E* s = x + t * p.xt + (row - t * nh) * p.xh;
                v[i].load(s);
                if constexpr (!kInterleaved)
                    if (rot) v2[i].load(s + kRopePairs);
            }
        }
    };
    load(0);
    for (int i = threadIdx.x; i < nt * kRopePairs; i += blockDim.x) {
        const int t = i / kRopePairs, k = i % kRopePairs;
        float2 c = rope_cos_sin(p.table.turns, p.table.amplitude, p.positions[t0 + t], k);
        if (p.transpose) c.y = -c.y;
        cs[t][k] = c;
    }
    __syncthreads();
    for (int base = 0; base < rows; base += kRopeUnroll * p.rows_pass) {
        if (base > 0) load(base);
#pragma unroll
        for (int i = 0; i < kRopeUnroll; ++i) {
            const int row = base + r0 + i * p.rows_pass;
            if (row >= mine) continue;
            const int t = p.tpc == 1 ? 0 : row / nh;
            E* d = out + t * p.ot + (row - t * nh) * p.oh;
            if (rot) {
                const float2* c = cs[t] + u * (kInterleaved ? 4 : 8);
                float a[8];
                v[i].get(a);
                if constexpr (kInterleaved) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) rotate(a[2 * k], a[2 * k + 1], c[k]);
                } else {
                    float b[8];
                    v2[i].get(b);
#pragma unroll
                    for (int k = 0; k < 8; ++k) rotate(a[k], b[k], c[k]);
                    v2[i].set(b);
                    v2[i].store(d + kRopePairs);
                }
                v[i].set(a);
            }
            v[i].store(d);
        }
    }
}

inline void launch_rope(const mla_rope_dims& d, const mla_rope_table& table, const void* x, const int32_t* positions, void* out,
                        cudaStream_t stream) {
    RopeParams p = {};
    p.x = x;
    p.positions = positions;
    p.out = out;
    p.xt = d.x_token_stride;
    p.xh = d.x_head_stride;
    p.ot = d.out_token_stride;
    p.oh = d.out_head_stride;
    p.T = d.tokens;
    p.h = d.num_heads;
    p.offset = d.offset;
    p.transpose = d.transpose;
    p.table = table;
    // units per row (at most kMoveThreads: rows are at most 2048 values wide), and
    // rows that one pass of the CTA's threads covers
    p.per_row = (table.interleaved ? 8 : 4) + (x == out ? 0 : (d.width - 2 * kRopePairs) / 8);
    p.rows_pass = kMoveThreads / p.per_row;
    // Enough rows per CTA for a few rounds of loads (the angles are computed once for
    // all of them), but no fewer CTAs than fill the device.
    const int64_t all = (int64_t)d.tokens * d.num_heads;
    const int64_t share = all / (2 * 148) > 1 ? all / (2 * 148) : 1;
    const int want = (int)min((int64_t)128, max((int64_t)p.rows_pass, share));
    p.hpc = min(d.num_heads, want);
    p.tpc = min(min(kRopeMaxTokens, d.tokens), max(1, want / p.hpc));
    const dim3 grid((d.tokens + p.tpc - 1) / p.tpc, (d.num_heads + p.hpc - 1) / p.hpc);
    const int threads = (p.rows_pass * p.per_row + 31) / 32 * 32;
    if (d.dtype == MLA_DTYPE_BF16) {
        if (table.interleaved) mla_rope_kernel<__nv_bfloat16, true><<<grid, threads, 0, stream>>>(p);
        else mla_rope_kernel<__nv_bfloat16, false><<<grid, threads, 0, stream>>>(p);
    } else {
        if (table.interleaved) mla_rope_kernel<float, true><<<grid, threads, 0, stream>>>(p);
        else mla_rope_kernel<float, false><<<grid, threads, 0, stream>>>(p);
    }
}

// ------------------------------------------------------------------ pool and books
struct CachePool {
    uint8_t* kv;
    float* scales;  // e4m3 pools
    int num_blocks;
    int page_bytes;
};
struct CacheBooks {
    int32_t* bt;
    int32_t* lens;
    int32_t* refs;
    int32_t* status;
    int batch, max_blocks, num_blocks;
};
__device__ __forceinline__ void raise(int32_t* status, int bit) {
    if (status != nullptr) atomicOr(status, bit);
}

// Sums over the block, for block sizes that are multiples of 32 up to 1024:
// the sum before this thread, and the total.  `tot` is 33 ints of shared memory.
__device__ __forceinline__ int block_exclusive(int v, int* tot, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // an earlier call's readers are done
    if (lane == 31) tot[warp] = x;
    __syncthreads();
    if (warp == 0) {
        const int own = lane < warps ? tot[lane] : 0;
        int w = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        tot[lane] = w - own;
        if (lane == 31) tot[32] = w;
    }
    __syncthreads();
    *total = tot[32];
    return tot[warp] + x - v;
}

// ------------------------------------------------------------------ append
struct AppendParams {
    const __nv_bfloat16* c_kv;
    const __nv_bfloat16* k_pe;
    int64_t c_stride, pe_stride;
    const int32_t* off;
    const int32_t* bt;
    const int32_t* lens;
    CachePool pool;
    int32_t* status;
    int batch, max_blocks, tokens, rotate;
    mla_rope_table rope;
};

// Pages that request b's new rows touch; 0, with *bad set, where they do not fit.
struct NewRows {
    int start, L, first, pages;  // position of the first new row, length, row in c_kv, pages
};
__device__ __forceinline__ NewRows new_rows(const AppendParams& p, int b, bool* bad) {
    NewRows r;
    const int lo = p.off[b], hi = p.off[b + 1];
    const int64_t n = (int64_t)hi - lo;
    r.L = p.lens[b];
    r.first = lo;
    r.pages = 0;
    r.start = 0;
    if (lo < 0 || hi > p.tokens || n < 0 || n > r.L || !seqlen_in_range(r.L, p.max_blocks)) {
        *bad = true;
        return r;
    }
    r.start = r.L - (int)n;
    if (n > 0) r.pages = pages_of(r.L) - r.start / kPage;
    return r;
}

__device__ __forceinline__ float finite_or_nan(float x) { return fabsf(x) <= FLT_MAX ? x : __int_as_float(0x7fffffff); }
__device__ __forceinline__ uint2 quant8(const float (&f)[8], float inv) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = e4m3x2(finite_or_nan(f[2 * e] * inv), finite_or_nan(f[2 * e + 1] * inv));
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}
// The same of eight finite bf16 values (a finite value times a power of two that
// brings the largest to 448 stays finite).
__device__ __forceinline__ uint2 quant8_finite(const uint4& v, float inv) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = e4m3x2(__uint_as_float(w[e] << 16) * inv, __uint_as_float(w[e] & 0xffff0000u) * inv);
    return make_uint2(o[0] | o[1] << 16, o[2] | o[3] << 16);
}
__device__ __forceinline__ uint32_t amax_of(uint32_t amax, float x) {
    const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
    return b < kInfBits ? max(amax, b) : amax;
}

// One CTA per touched page: it holds the page's new rows in registers (per thread
// kLatRows pieces of 8 latent columns and 4 RoPE pairs for a full page; two such CTAs
// fit an SM), so the scale costs no second read of them.  The CTA finds its
// (request, page) by a scan over the requests' page counts.
// A single token per request is a chain of dependent reads (offsets and lengths,
// table, row) and the fence: 128 requests 5.4 us on B200.  Prompts are bound by the two
// rounds of CTAs and by the conversions: 32,900 rows to e4m3 (57 MB read and written) 16.9 us,
// of it the angles 2 us and the fence 1.2 (18.4 with a check per value; the loop over pages
// past the grid costs 0.35); to bf16 16.1 us.
constexpr int kAppendThreads = 512;
constexpr int kLatRows = kPage * (kDv / 8) / kAppendThreads;  // 8
static_assert(kPage * 8 == kAppendThreads, "one RoPE unit per thread");
// Page `nth` of request b's new ones.
template <bool kQ8>
__device__ __forceinline__ void append_page(const AppendParams& p, int b, int nth, uint32_t* warp_max) {
    const int tid = threadIdx.x;
    bool bad = false;
    const NewRows nr = new_rows(p, b, &bad);
    const int page = nr.start / kPage + nth;
    const int phys = p.bt[(size_t)b * p.max_blocks + page];
    if ((unsigned)phys >= (unsigned)p.pool.num_blocks) {
        if (tid == 0) raise(p.status, MLA_STATUS_BAD_BLOCK_TABLE);
        return;
    }
    const int r0 = max(nr.start - page * kPage, 0), r1 = min(nr.L - page * kPage, kPage);
    const int64_t src0 = (int64_t)nr.first + (page * kPage - nr.start);  // source row of page row 0
    uint8_t* dst = p.pool.kv + (size_t)phys * p.pool.page_bytes;

    // latent: piece tid % 64 of rows r0 + tid / 64 + 8 k;  RoPE: unit tid % 8 of row r0 + tid / 8
    const int lc = tid & 63, lr = tid >> 6, pu = tid & 7, pr = tid >> 3;
    uint4 lat[kLatRows];
    float pe[8];
#pragma unroll
    for (int k = 0; k < kLatRows; ++k) {
        const int r = r0 + lr + 8 * k;
        if (r < r1) lat[k] = *reinterpret_cast<const uint4*>(p.c_kv + (src0 + r) * p.c_stride + lc * 8);
    }
    const bool inter = !p.rotate || p.rope.interleaved;
    const int rr = r0 + pr;
    if (rr < r1) {
        const __nv_bfloat16* s = p.k_pe + (src0 + rr) * p.pe_stride;
        uint4 raw;
        if (inter) {
            raw = *reinterpret_cast<const uint4*>(s + pu * 8);
        } else {  // pairs 4 pu .. 4 pu + 3: columns c and c + 32
            const uint2 lo = *reinterpret_cast<const uint2*>(s + pu * 4);
            const uint2 hi = *reinterpret_cast<const uint2*>(s + kRopePairs + pu * 4);
            raw = make_uint4(lo.x, lo.y, hi.x, hi.y);
        }
        unpack8(raw, pe);
        if (p.rotate) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 c = rope_cos_sin(p.rope.turns, p.rope.amplitude, page * kPage + rr, pu * 4 + i);
                // (selected, not indexed: both layouts keep the values in registers)
                float a = inter ? pe[2 * i] : pe[i], z = inter ? pe[2 * i + 1] : pe[i + 4];
                rotate(a, z, c);
                if (inter) {
                    pe[2 * i] = a;
                    pe[2 * i + 1] = z;
                } else {
                    pe[i] = a;
                    pe[i + 4] = z;
                }
            }
        }
    }
    float inv = 1.f;
    bool finite = true;
    if constexpr (kQ8) {
        // Largest magnitude as bits, non-finite values included: they are the
        // largest, and where there is none the finite maximum is at hand.
        uint32_t two = 0;  // of the low and the high halves
#pragma unroll
        for (int k = 0; k < kLatRows; ++k) {
            if (r0 + lr + 8 * k >= r1) continue;
            two = __vmaxu2(two, __vmaxu2(__vmaxu2(lat[k].x & 0x7fff7fffu, lat[k].y & 0x7fff7fffu),
                                         __vmaxu2(lat[k].z & 0x7fff7fffu, lat[k].w & 0x7fff7fffu)));
        }
        uint32_t top = max(two << 16, two & 0xffff0000u);
        if (rr < r1)
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(pe[i]) & 0x7fffffffu);
        top = __reduce_max_sync(0xffffffffu, top);
        if ((tid & 31) == 0) warp_max[tid >> 5] = top;
        const float held = r0 > 0 ? p.pool.scales[phys] : 0.f;  // (read by all before thread 0 writes it)
        __syncthreads();
        uint32_t amax = 0;
#pragma unroll
        for (int w = 0; w < kAppendThreads / 32; ++w) amax = max(amax, warp_max[w]);
        finite = amax < kInfBits;
        if (!finite) {  // (seldom)
            uint32_t fin = 0;
            for (int k = 0; k < kLatRows; ++k) {
                if (r0 + lr + 8 * k >= r1) continue;
                float f[8];
                unpack8(lat[k], f);
                for (int i = 0; i < 8; ++i) fin = amax_of(fin, f[i]);
            }
            if (rr < r1)
                for (int i = 0; i < 8; ++i) fin = amax_of(fin, pe[i]);
            fin = __reduce_max_sync(0xffffffffu, fin);
            __syncthreads();
            if ((tid & 31) == 0) warp_max[tid >> 5] = fin;
            __syncthreads();
            amax = 0;
            for (int w = 0; w < kAppendThreads / 32; ++w) amax = max(amax, warp_max[w]);
        }
        const int e = amax == 0 ? kMinScaleExp : min(max(e4m3_scale_exp(amax), kMinScaleExp), kMaxScaleExp);
        const float scale = fmaxf(pow2f(e), held);
        inv = 1.f / scale;
        if (r0 > 0 && scale > held) {
            // The page's earlier rows move to the larger scale.
            const float f = held / scale;
            uint2* rows = reinterpret_cast<uint2*>(dst);
            for (int i = tid; i < r0 * (kDqk / 8); i += kAppendThreads) {
                const uint2 v = rows[i];
                const uint32_t w[4] = {v.x & 0xffffu, v.x >> 16, v.y & 0xffffu, v.y >> 16};
                uint32_t o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 h = __half22float2(as_h2(h2_of_e4m3x2(w[k])));
                    o[k] = e4m3x2(h.x * f, h.y * f);
                }
                rows[i] = make_uint2(o[0] | o[1] << 16, o[2] | o[3] << 16);
            }
        }
        if (tid == 0) p.pool.scales[phys] = scale;
    }
#pragma unroll
    for (int k = 0; k < kLatRows; ++k) {
        const int r = r0 + lr + 8 * k;
        if (r >= r1) continue;
        if constexpr (kQ8) {
            uint2 v;
            if (finite) {
                v = quant8_finite(lat[k], inv);
            } else {
                float f[8];
                unpack8(lat[k], f);
                v = quant8(f, inv);
            }
            *reinterpret_cast<uint2*>(dst + r * kDqk + lc * 8) = v;
        } else {
            *reinterpret_cast<uint4*>(dst + (r * kDqk + lc * 8) * 2) = lat[k];
        }
    }
    if (rr < r1) {
        if constexpr (kQ8) {
            const uint2 v = quant8(pe, inv);
            uint8_t* d = dst + rr * kDqk + kDv;
            if (inter) {
                *reinterpret_cast<uint2*>(d + pu * 8) = v;
            } else {
                *reinterpret_cast<uint32_t*>(d + pu * 4) = v.x;
                *reinterpret_cast<uint32_t*>(d + kRopePairs + pu * 4) = v.y;
            }
        } else {
            const uint4 v = pack8(pe);
            __nv_bfloat16* d = reinterpret_cast<__nv_bfloat16*>(dst) + rr * kDqk + kDv;
            if (inter) {
                *reinterpret_cast<uint4*>(d + pu * 8) = v;
            } else {
                *reinterpret_cast<uint2*>(d + pu * 4) = make_uint2(v.x, v.y);
                *reinterpret_cast<uint2*>(d + kRopePairs + pu * 4) = make_uint2(v.z, v.w);
            }
        }
    }
}

// Finds page number `want` of all requests' new ones: job[0], job[1] = its request and place there (job[0]
// stays -1: there is none), job[2] = the number of pages looked at, job[3] = want.  CTA 0 looks at every request, for the status.
__device__ __forceinline__ void append_find(const AppendParams& p, int want, int* tot, int* job) {
    const int tid = threadIdx.x;
    if (tid == 0) job[0] = -1;
    int before = 0;
    for (int base = 0; base < p.batch; base += kAppendThreads) {
        const int b = base + tid;
        bool bad = false;
        int pages = 0;
        if (b < p.batch) pages = new_rows(p, b, &bad).pages;
        if (bad) raise(p.status, MLA_STATUS_BAD_ROW);
        int total;
        const int mine = before + block_exclusive(pages, tot, &total);
        if (want >= mine && want < mine + pages) {
            job[0] = b;
            job[1] = want - mine;
        }
        before += total;
        if (blockIdx.x != 0 && want < before) break;
    }
    if (tid == 0) {
        job[2] = before;
        job[3] = want;
    }
    __syncthreads();
}

template <bool kQ8>
__global__ void __launch_bounds__(kAppendThreads, 2) mla_cache_append_kernel(const __grid_constant__ AppendParams p) {
    __shared__ int tot[33];
    __shared__ int job[4];
    __shared__ uint32_t warp_max[kAppendThreads / 32];
    // Every page has a CTA while the offsets do not fall.  Where they do, requests that are in
    // order may name the same rows, and more pages than there are CTAs: CTA 0 writes those one after the other.
    for (int want = blockIdx.x;;) {
        append_find(p, want, tot, job);
        if (job[0] >= 0) append_page<kQ8>(p, job[0], job[1], warp_max);
        if (blockIdx.x != 0) break;
        want = max(job[3] + 1, (int)gridDim.x);
        if (want >= job[2]) break;
        __syncthreads();
    }
    __threadfence();
}

inline void launch_append(const AppendParams& p, cudaStream_t stream) {
    // n new rows touch at most n pages, and at most n / 64 + 2; and the requests' rows are
    // `tokens` in all, if their offsets do not fall
    const int64_t most = min((int64_t)p.tokens, (int64_t)p.tokens / kPage + 2 * (int64_t)p.batch);
    if (p.pool.scales != nullptr) mla_cache_append_kernel<true><<<(unsigned)most, kAppendThreads, 0, stream>>>(p);
    else mla_cache_append_kernel<false><<<(unsigned)most, kAppendThreads, 0, stream>>>(p);
}

// ------------------------------------------------------------------ page moves
// A CTA moves slices of pages, two 16-byte loads in flight per thread; 288 threads cut
// a page (36,864 or 73,728 bytes) into 4 or 8 whole slices.  Bound by the bytes, each
// read and written once; a compaction that moves 182 MB takes 29.5 us (6.2 TB/s).
constexpr int kCopyThreads = 288;
constexpr int kSliceBytes = 2 * kCopyThreads * 16;
static_assert(kPage * kDqk % kSliceBytes == 0, "whole slices");
inline int page_slices(int page_bytes) { return page_bytes / kSliceBytes; }

__device__ __forceinline__ void copy_slice(const CachePool& pool, int src, int dst, int slice) {
    const uint8_t* s = pool.kv + (size_t)src * pool.page_bytes;
    uint8_t* d = pool.kv + (size_t)dst * pool.page_bytes;
    const int a = slice * kSliceBytes + threadIdx.x * 16, b = a + kCopyThreads * 16;
    const uint4 va = *reinterpret_cast<const uint4*>(s + a);
    const uint4 vb = *reinterpret_cast<const uint4*>(s + b);
    *reinterpret_cast<uint4*>(d + a) = va;
    *reinterpret_cast<uint4*>(d + b) = vb;
    if (slice == 0 && threadIdx.x == 0 && pool.scales != nullptr) pool.scales[dst] = pool.scales[src];
}

__global__ void __launch_bounds__(kCopyThreads)
    mla_cache_copy_kernel(const CachePool pool, const int32_t* src, const int32_t* dst, int32_t* status) {
    const int s = src[blockIdx.x], d = dst[blockIdx.x];
    if (s < 0) return;
    if (s >= pool.num_blocks || (unsigned)d >= (unsigned)pool.num_blocks) {
        if (threadIdx.x == 0) raise(status, MLA_STATUS_BAD_BLOCK_TABLE);
        return;
    }
    copy_slice(pool, s, d, blockIdx.y);
    __threadfence();
}
inline void launch_copy_pages(const CachePool& pool, int n, const int32_t* src, const int32_t* dst, int32_t* status,
                              cudaStream_t stream) {
    mla_cache_copy_kernel<<<dim3(n, page_slices(pool.page_bytes)), kCopyThreads, 0, stream>>>(pool, src, dst, status);
}

// The second kernel of a call, launched as a programmatic dependent of the first: its
// launch overlaps the first one's run.
template <typename... P, typename... A>
inline void launch_after(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);  // (an error is the caller's to collect)
}

// A page that a row holds although its count says that it is free, while a call works.
constexpr int kHeldUncounted = INT32_MIN;

// ------------------------------------------------------------------ fork
constexpr int kForkMax = 1024;
constexpr int kBookThreads = 1024;
constexpr int kBookUnroll = 4;
// workspace words of fork i
enum ForkWord { kForkOk = 0, kForkSrc = 1, kForkDst = 2, kForkWords = 3 };
__host__ __device__ inline size_t fork_workspace_words(int n) { return (size_t)kForkWords * n; }

// One CTA decides every fork, in order: checks the rows, ranks the forks that need
// a page and hands them the lowest free ones.  Which pages are free depends on every
// fork before, so one block settles it; a chain of short reads and block scans, 6.8 us on B200 for
// 24 forks in 350 pages and 8.8 us for 192 in 5,200, while the copy kernel is being launched.
__global__ void __launch_bounds__(kBookThreads)
    mla_cache_fork_plan_kernel(const CacheBooks k, int n, const int32_t* parents, const int32_t* children, int32_t* ws) {
    __shared__ __align__(16) int child_s[kForkMax];
    __shared__ int fresh[kForkMax];
    __shared__ int tot[33];
    griddep_launch_dependents();  // (the copies wait for this grid's end)
    const int i = threadIdx.x;
    const int parent = i < n ? parents[i] : -1, child = i < n ? children[i] : -1;
    child_s[i] = i < n ? child : -1;  // (kForkMax threads)
    __syncthreads();
    bool ok = i < n && (unsigned)parent < (unsigned)k.batch && (unsigned)child < (unsigned)k.batch;
    if (ok) {  // not named before: four rows at a time
        bool again = false;
        const int4* c4 = reinterpret_cast<const int4*>(child_s);
#pragma unroll 4
        for (int j = 0; j < i / 4; ++j) {
            const int4 c = c4[j];
            again |= c.x == child || c.y == child || c.z == child || c.w == child;
        }
        for (int j = i & ~3; j < i; ++j) again |= child_s[j] == child;
        ok = !again;
    }
    int L = 0;
    if (ok) {
        L = k.lens[parent];
        ok = seqlen_in_range(L, k.max_blocks) && k.lens[child] == 0;
    }
    if (i < n && !ok) raise(k.status, MLA_STATUS_BAD_ROW);
    const int last = L / kPage;
    int src = -1, lost = -1, lost_count = 0;
    if (ok && L % kPage != 0) {
        src = k.bt[(size_t)parent * k.max_blocks + last];
        if ((unsigned)src >= (unsigned)k.num_blocks) {
            raise(k.status, MLA_STATUS_BAD_BLOCK_TABLE);
            ok = false;
            src = -1;
        } else if (const int count = k.refs[src]; count <= 0) {
            // held, but free by its count: not copied, and not given out below
            raise(k.status, MLA_STATUS_BAD_REF_COUNT);
            ok = false;
            if (count != kHeldUncounted) {
                lost = src;
                lost_count = count;
                k.refs[src] = kHeldUncounted;
            }
            src = -1;
        }
    }
    int need;
    const int rank = block_exclusive(src >= 0 ? 1 : 0, tot, &need);
    // the lowest `need` free pages
    int found = 0;
    for (int base = 0; base < k.num_blocks && found < need; base += kBookThreads * kBookUnroll) {
        // thread t takes kBookUnroll consecutive pages, so that ranks rise with pages
        int at[kBookUnroll], cnt = 0;
#pragma unroll
        for (int u = 0; u < kBookUnroll; ++u) {
            const int page = base + i * kBookUnroll + u;
            at[u] = page < k.num_blocks && k.refs[page] == 0 ? 1 : 0;
            cnt += at[u];
        }
        int total;
        int r = found + block_exclusive(cnt, tot, &total);
#pragma unroll
        for (int u = 0; u < kBookUnroll; ++u) {
            if (at[u] && r < need) fresh[r] = base + i * kBookUnroll + u;
            r += at[u];
        }
        found += total;
    }
    __syncthreads();
    if (lost >= 0) k.refs[lost] = lost_count;
    int dst = -1;
    if (src >= 0) {
        if (rank < found) {
            dst = fresh[rank];
        } else {
            raise(k.status, MLA_STATUS_NO_FREE_PAGE);
            ok = false;
        }
    }
    if (i < n) {
        ws[kForkWords * i + kForkOk] = ok ? 1 : 0;
        ws[kForkWords * i + kForkSrc] = ok ? src : -1;
        ws[kForkWords * i + kForkDst] = dst;
        if (ok && L > 0) {
            k.lens[child] = L;
            if (dst >= 0) {
                k.bt[(size_t)child * k.max_blocks + last] = dst;
                k.refs[dst] = 1;
            }
        }
    }
}

// CTA (i, s): slice s of fork i's page, or (the last s) its table row.  4.5 us for 24
// forks of e4m3 pages, 8 us for 192 of bf16 pages (28 MB).
__global__ void __launch_bounds__(kCopyThreads)
    mla_cache_fork_kernel(const CacheBooks k, const CachePool pool, const int32_t* parents, const int32_t* children,
                          const int32_t* ws) {
    griddep_wait();  // the plan
    const int32_t* w = ws + kForkWords * blockIdx.x;
    if (!w[kForkOk]) return;
    if (blockIdx.y + 1 < gridDim.y) {
        if (w[kForkSrc] >= 0) copy_slice(pool, w[kForkSrc], w[kForkDst], blockIdx.y);
    } else {
        const int parent = parents[blockIdx.x], child = children[blockIdx.x];
        const int full = k.lens[child] / kPage;
        for (int j = threadIdx.x; j < full; j += kCopyThreads) {
            const int page = k.bt[(size_t)parent * k.max_blocks + j];
            k.bt[(size_t)child * k.max_blocks + j] = page;
            if ((unsigned)page >= (unsigned)k.num_blocks) raise(k.status, MLA_STATUS_BAD_BLOCK_TABLE);
            else if (atomicAdd(k.refs + page, 1) <= 0) raise(k.status, MLA_STATUS_BAD_REF_COUNT);
        }
    }
    __threadfence();
}
inline void launch_fork(const CacheBooks& k, const CachePool& pool, int n, const int32_t* parents, const int32_t* children,
                        int32_t* ws, cudaStream_t stream) {
    mla_cache_fork_plan_kernel<<<1, kBookThreads, 0, stream>>>(k, n, parents, children, ws);
    launch_after(mla_cache_fork_kernel, dim3(n, page_slices(pool.page_bytes) + 1), kCopyThreads, stream, k, pool, parents, children,
                 (const int32_t*)ws);
}

// ------------------------------------------------------------------ free
// A CTA per row: one counter per page, returned by atomics (whole numbers, so their
// order does not matter).  Bound by the launch: 24 rows 5.5 us.
__global__ void __launch_bounds__(kMoveThreads) mla_cache_free_kernel(const CacheBooks k, const int32_t* rows) {
    __shared__ int len;
    const int row = rows[blockIdx.x];
    if ((unsigned)row >= (unsigned)k.batch) {
        if (threadIdx.x == 0) raise(k.status, MLA_STATUS_BAD_ROW);
        return;
    }
    if (threadIdx.x == 0) len = atomicExch(k.lens + row, 0);  // a row named twice is empty the second time
    __syncthreads();
    if (!seqlen_in_range(len, k.max_blocks) && threadIdx.x == 0) raise(k.status, MLA_STATUS_BAD_SEQLEN);
    const int pages = pages_of(clamp_seqlen(len, k.max_blocks));
    int32_t* bt = k.bt + (size_t)row * k.max_blocks;
    for (int j = threadIdx.x; j < pages; j += kMoveThreads) {
        const int page = bt[j];
        bt[j] = -1;
        if ((unsigned)page >= (unsigned)k.num_blocks) {
            raise(k.status, MLA_STATUS_BAD_BLOCK_TABLE);
        } else if (atomicSub(k.refs + page, 1) <= 0) {
            atomicAdd(k.refs + page, 1);
            raise(k.status, MLA_STATUS_BAD_REF_COUNT);
        }
    }
    __threadfence();
}
inline void launch_free(const CacheBooks& k, int n, const int32_t* rows, cudaStream_t stream) {
    mla_cache_free_kernel<<<n, kMoveThreads, 0, stream>>>(k, rows);
}

// ------------------------------------------------------------------ compact
// workspace: live, moves, then the destinations (free pages before `live`, rising)
// and the sources (pages in use behind it, rising) one after the other, then for
// each page behind `live` its place in that list (-1: not in use).
enum CompactWord { kCompactLive = 0, kCompactMoves = 1, kCompactList = 4 };
inline size_t compact_workspace_words(int num_blocks) { return kCompactList + 2 * (size_t)num_blocks; }

// The table against the counts, before anything moves: a page that a row holds although its count
// says that it is free would be written over.  Its count is marked, and the plan takes it for
// one in use (and puts the 0 back).  Whoever finds it writes the same mark, so the order does
// not matter.  CTA (x, y) takes every gridDim.y-th piece of kCheckEntries entries of row x: several to a row only while
// rows alone do not fill the device, and none costs more than its length's read where a wide table is mostly empty.  It
// lengthens a compaction on B200 by 1.2 us (of 64 rows, 40 in use); the plan's launch overlaps it.
constexpr int kCheckEntries = 4 * kMoveThreads;
__global__ void __launch_bounds__(kMoveThreads) mla_cache_check_kernel(const CacheBooks k) {
    griddep_launch_dependents();  // (the plan waits for this grid's end)
    const int b = blockIdx.x, L = k.lens[b];
    if (blockIdx.y == 0 && threadIdx.x == 0 && !seqlen_in_range(L, k.max_blocks)) raise(k.status, MLA_STATUS_BAD_SEQLEN);
    const int end = pages_of(clamp_seqlen(L, k.max_blocks));
    const int32_t* bt = k.bt + (size_t)b * k.max_blocks;
    for (int64_t first = (int64_t)blockIdx.y * kCheckEntries; first < end; first += (int64_t)gridDim.y * kCheckEntries) {
        int page[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t j = first + i * kMoveThreads + threadIdx.x;
            page[i] = j < end ? bt[j] : -1;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if ((unsigned)page[i] < (unsigned)k.num_blocks && k.refs[page[i]] <= 0) {
                k.refs[page[i]] = kHeldUncounted;
                raise(k.status, MLA_STATUS_BAD_REF_COUNT);
            }
        }
    }
    __threadfence();
}

// As many free pages lie before `live` as pages in use behind it (live counts
// both those in use before it and those behind), so one running count over the
// pages that move or are moved to numbers both lists.  A warp owns a run of
// consecutive pages, 32 at a time, and a lane keeps which of its pages are in use as
// bits, so the counts are read once up to 65,536 pages (again for more), and
// only the warps' totals meet across the block.  8.3 us on B200 for 10,500 pages (two rounds
// of loads, three block scans); 16 loads in flight instead of 8 measured the same.
constexpr int kPlanBits = 64;
__global__ void __launch_bounds__(kBookThreads) mla_cache_compact_plan_kernel(const CacheBooks k, int32_t* ws) {
    __shared__ int tot[33];
    griddep_launch_dependents();  // (the moves wait for this grid's end)
    griddep_wait();               // the check
    const int nb = k.num_blocks, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int span = kBookThreads * kPlanBits;
    // pages per lane and round, in eights: eight loads are in flight at a time
    const int per = nb < span ? ((nb + kBookThreads - 1) / kBookThreads + 7) / 8 * 8 : kPlanBits;
    auto in_use = [&](int base, bool last) -> uint64_t {  // last: marks become 0 again
        const int first = base + warp * 32 * per + lane;
        uint64_t bits = 0;
        for (int u = 0; u < per; u += 8) {
            int v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = first + 32 * (u + i) < nb ? k.refs[first + 32 * (u + i)] : 0;
            uint32_t b = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                b |= (v[i] > 0 || v[i] == kHeldUncounted ? 1u : 0u) << i;
                if (last && v[i] == kHeldUncounted) k.refs[first + 32 * (u + i)] = 0;
            }
            bits |= (uint64_t)b << u;
        }
        return bits;
    };
    int mine = 0;
    uint64_t bits = 0;
    for (int base = 0; base < nb; base += kBookThreads * per) {
        bits = in_use(base, nb <= kBookThreads * per);
        mine += __popcll(bits);
    }
    int live;
    block_exclusive(mine, tot, &live);
    int32_t* list = ws + kCompactList;
    int32_t* place = list + nb;
    int before = 0;
    for (int base = 0; base < nb; base += kBookThreads * per) {
        if (nb > kBookThreads * per) bits = in_use(base, true);
        const int first = base + warp * 32 * per + lane;
        // pages that move or are moved to
        uint64_t at = 0;
#pragma unroll 8
        for (int u = 0; u < per; ++u) {
            const int page = first + 32 * u;
            if (page < nb && (bool)((bits >> u) & 1) == (page >= live)) at |= 1ull << u;
        }
        int total;
        const int r = before + block_exclusive(__popcll(at), tot, &total);
        int run = __shfl_sync(0xffffffffu, r, 0);  // of the warp's first page
#pragma unroll 8
        for (int u = 0; u < per; ++u) {
            const int page = first + 32 * u;
            const bool hit = (at >> u) & 1;
            const unsigned hits = __ballot_sync(0xffffffffu, hit);
            const int rank = run + __popc(hits & ((1u << lane) - 1));
            if (hit) list[rank] = page;
            if (page < nb && page >= live) place[page] = hit ? rank : -1;
            run += __popc(hits);
        }
        before += total;
    }
    if (threadIdx.x == 0) {
        ws[kCompactLive] = live;
        ws[kCompactMoves] = before / 2;
    }
}

// Moves the pages, then renames them in the tables of the rows in use.  7 CTAs per SM are
// resident; 8, 16, 24 or 32 per SM in the grid: 52.8, 49.4, 48.3, 48.7 us for the books,
// the plan and 182 MB of moves (16 and 24 with the check: 52.2, 51.3; 19 MB of bf16 pages 17.9 both).
__global__ void __launch_bounds__(kCopyThreads)
    mla_cache_compact_kernel(const CacheBooks k, const CachePool pool, const int32_t* ws, int shift) {
    griddep_wait();  // the plan
    const int live = ws[kCompactLive], moves = ws[kCompactMoves];
    const int32_t* list = ws + kCompactList;
    const int32_t* place = list + k.num_blocks;
    // A unit is move u >> shift, slice u & (slices - 1) of its 4 or 8; the next unit's pages
    // are looked up while this one's bytes are on their way.
    const int64_t units = (int64_t)moves << shift;
    int64_t u = blockIdx.x;
    int dst = 0, src = 0;
    if (u < units) {
        dst = list[u >> shift];
        src = list[moves + (u >> shift)];
    }
    while (u < units) {
        const int64_t next = u + gridDim.x;
        int dst2 = 0, src2 = 0;
        if (next < units) {
            dst2 = list[next >> shift];
            src2 = list[moves + (next >> shift)];
        }
        const int s = (int)(u & ((1 << shift) - 1));
        copy_slice(pool, src, dst, s);
        if (s == 0 && threadIdx.x == 0) {
            k.refs[dst] = k.refs[src];
            k.refs[src] = 0;
        }
        u = next;
        dst = dst2;
        src = src2;
    }
    for (int b = blockIdx.x; b < k.batch; b += gridDim.x) {
        const int pages = pages_of(clamp_seqlen(k.lens[b], k.max_blocks));
        int32_t* bt = k.bt + (size_t)b * k.max_blocks;
        for (int j = threadIdx.x; j < pages; j += kCopyThreads) {
            const int page = bt[j];
            if ((unsigned)page >= (unsigned)k.num_blocks) {
                raise(k.status, MLA_STATUS_BAD_BLOCK_TABLE);
            } else if (page >= live) {
                const int at = place[page];
                if (at >= moves) bt[j] = list[at - moves];
                else raise(k.status, MLA_STATUS_BAD_REF_COUNT);
            }
        }
    }
    __threadfence();
}
inline void launch_compact(const CacheBooks& k, const CachePool& pool, int32_t* ws, cudaStream_t stream) {
    const int slices = page_slices(pool.page_bytes);
    const int pieces = (k.max_blocks + kCheckEntries - 1) / kCheckEntries;
    mla_cache_check_kernel<<<dim3(k.batch, min(pieces, max(1, 148 * 8 / k.batch))), kMoveThreads, 0, stream>>>(k);
    launch_after(mla_cache_compact_plan_kernel, dim3(1), kBookThreads, stream, k, ws);
    const int64_t most = max((int64_t)k.batch, (int64_t)(k.num_blocks / 2) * slices);
    launch_after(mla_cache_compact_kernel, dim3((unsigned)min((int64_t)148 * 24, max(most, (int64_t)1))), kCopyThreads, stream, k, pool,
                 (const int32_t*)ws, slices == 4 ? 2 : 3);
}

}  // namespace mla
