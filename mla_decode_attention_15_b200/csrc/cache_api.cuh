// C ABI of include/mla_cache.h: argument checks, tensor maps and launches of the
// cache's operators and of decode over the 8-bit cache.  Included once, at the
// end of mla_decode_api.cu, whose helpers it uses.
#pragma once

namespace {

constexpr int kCacheAbiVersion = 1;

// ------------------------------------------------------------------ 8-bit decode
// Query groups of 16 columns, or of 32 where a request has more; several
// groups walk each range of pages side by side where the device has an SM for
// each.
int make_plan_q8(const mla_decode_dims* d, Plan* pl) {
    int rc = validate_dims(d);
    if (rc != MLA_OK) return rc;
    pl->gr.N = d->num_heads * d->s_q;
    pl->gr.NG = pl->gr.N <= 16 ? 16 : 32;
    pl->gr.Hg = (pl->gr.N + pl->gr.NG - 1) / pl->gr.NG;
    if ((int64_t)d->batch * pl->gr.Hg * ((int64_t)d->max_blocks_per_seq + kQ8ItemOverhead) >= (int64_t)INT32_MAX)
        return MLA_ERR_UNSUPPORTED;
    int sms = 0;
    rc = resolve_ctas(d, &sms);
    if (rc != MLA_OK) return rc;
    pl->pair = false;
    pl->shift = kPageShift;
    pl->overhead = kQ8ItemOverhead;
    if (pl->gr.Hg > 1 && sms >= pl->gr.Hg) {
        pl->G = sms / pl->gr.Hg;
        pl->BG = d->batch;
        pl->plan_Hg = 1;
        pl->share = pl->gr.Hg;
    } else {
        pl->G = sms;
        pl->BG = d->batch * pl->gr.Hg;
        pl->plan_Hg = pl->gr.Hg;
        pl->share = 1;
    }
    pl->ctas = pl->G * pl->share;
    pl->slots = max_slots(pl->G) * pl->share;
    return MLA_OK;
}

bool q8_plan_in_kernel(int32_t flags, const Plan& pl) {
    return (flags & MLA_FLAG_INLINE_PLAN) &&
           pl.BG <= (pl.gr.NG == 16 ? Q8Cfg<16>::kInlinePlanMaxBG : Q8Cfg<32>::kInlinePlanMaxBG);
}

// Pool [num_blocks][64][576] bytes as 3-D (col, token, page); box = cols x 64 tokens.
int make_q8_map(CUtensorMap* m, const void* kv, int num_blocks, int cols) {
    auto enc = get_encode_fn();
    if (!enc) return MLA_ERR_CUDA;
    cuuint64_t dims[3] = {(cuuint64_t)kQ8Row, (cuuint64_t)kPage, (cuuint64_t)num_blocks};
    cuuint64_t strides[2] = {(cuuint64_t)kQ8Row, (cuuint64_t)kQ8PageBytes};
    cuuint32_t box[3] = {(cuuint32_t)cols, (cuuint32_t)kPage, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(kv), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, cols == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? MLA_OK : MLA_ERR_CUDA;
}

template <int NG>
int launch_q8(const Plan& pl, const Q8Params& p, const CUtensorMap& kvm, const CUtensorMap& rm, cudaStream_t stream) {
    using C = Q8Cfg<NG>;
    static bool done[kMaxDevices] = {};
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return MLA_ERR_CUDA;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!done[dev]) {
            if (cudaFuncSetAttribute(mla_decode_q8_kernel<NG>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kAlloc) !=
                cudaSuccess) {
                cudaGetLastError();
                return MLA_ERR_CUDA;
            }
            // setmaxnreg.inc waits until the registers it asks for are free in
            // the CTA: the split must fit the launch as compiled
            cudaFuncAttributes fa;
            if (cudaFuncGetAttributes(&fa, mla_decode_q8_kernel<NG>) != cudaSuccess) return MLA_ERR_CUDA;
            if (C::kSplitRegs && fa.numRegs * 4 < C::kRegsIssue + C::kRegsQ + 2 * C::kRegsSoftmax) return MLA_ERR_UNSUPPORTED;
            done[dev] = true;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(pl.ctas);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kAlloc;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, mla_decode_q8_kernel<NG>, kvm, rm, p) != cudaSuccess) {
        cudaGetLastError();
        return MLA_ERR_CUDA;
    }
    return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

// ------------------------------------------------------------------ cache
bool aligned4(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool status_ok(const int32_t* s) { return (reinterpret_cast<uintptr_t>(s) & 3u) == 0; }

int validate_cache(const mla_cache_dims* d) {
    if (d == nullptr) return MLA_ERR_INVALID_ARG;
    if (d->batch < 1 || d->max_blocks_per_seq < 1 || d->num_blocks < 1) return MLA_ERR_INVALID_ARG;
    if (d->page_size != kPage || d->row_width != kDqk || (d->dtype != MLA_CACHE_BF16 && d->dtype != MLA_CACHE_E4M3))
        return MLA_ERR_UNSUPPORTED;
    // a table entry's index, and a length in tokens, fit 32 bits
    if ((int64_t)d->batch * d->max_blocks_per_seq >= (int64_t)INT32_MAX || d->max_blocks_per_seq > INT32_MAX / kPage)
        return MLA_ERR_UNSUPPORTED;
    return MLA_OK;
}
// A pool and, for an 8-bit one, its scales.
bool pool_ok(const mla_cache_dims* d, const void* kv, const float* scales) {
    return aligned16(kv) && (d->dtype == MLA_CACHE_BF16 ? scales == nullptr : aligned16(scales));
}

CachePool pool_of(const mla_cache_dims* d, void* kv, float* scales) {
    CachePool c;
    c.kv = static_cast<uint8_t*>(kv);
    c.scales = scales;
    c.num_blocks = d->num_blocks;
    c.page_bytes = kPage * kDqk * (d->dtype == MLA_CACHE_E4M3 ? 1 : 2);
    return c;
}
CacheBooks books_of(const mla_cache_dims* d, int32_t* bt, int32_t* lens, int32_t* refs, int32_t* status) {
    CacheBooks k;
    k.bt = bt;
    k.lens = lens;
    k.refs = refs;
    k.status = status;
    k.batch = d->batch;
    k.max_blocks = d->max_blocks_per_seq;
    k.num_blocks = d->num_blocks;
    return k;
}

int launched() { return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA; }

}  // namespace

extern "C" {

int mla_cache_version(void) { return kCacheAbiVersion; }

size_t mla_decode_q8_schedule_bytes(const mla_decode_dims* dims) {
    Plan pl;
    if (make_plan_q8(dims, &pl) != MLA_OK) return 0;
    return (size_t)schedule_words(pl.G, pl.BG) * sizeof(int32_t);
}

size_t mla_decode_q8_workspace_bytes(const mla_decode_dims* dims) {
    Plan pl;
    if (make_plan_q8(dims, &pl) != MLA_OK) return 0;
    return workspace_bytes_of(pl);
}

int mla_decode_q8_get_schedule(const mla_decode_dims* dims, const int32_t* cache_seqlens, void* schedule, void* stream) {
    Plan pl;
    int rc = make_plan_q8(dims, &pl);
    if (rc != MLA_OK) return rc;
    if (!aligned16(cache_seqlens) || !aligned16(schedule)) return MLA_ERR_INVALID_ARG;
    return launch_schedule(pl, dims->batch, dims->max_blocks_per_seq, cache_seqlens, schedule,
                           static_cast<cudaStream_t>(stream));
}

int mla_decode_q8_get_schedule_host(const mla_decode_dims* dims, const int32_t* seqlens, void* schedule_host) {
    int rc = validate_dims(dims);
    if (rc != MLA_OK) return rc;
    if (dims->num_sms <= 0 || seqlens == nullptr || schedule_host == nullptr) return MLA_ERR_INVALID_ARG;
    Plan pl;
    rc = make_plan_q8(dims, &pl);
    if (rc != MLA_OK) return rc;
    host_plan(pl, dims->batch, dims->max_blocks_per_seq, seqlens, schedule_host);
    return MLA_OK;
}

int mla_decode_q8_fwd(const mla_decode_dims* dims, void* schedule, void* workspace, const void* q, const void* kv_cache,
                      const float* kv_scales, const int32_t* block_table, const int32_t* cache_seqlens,
                      float softmax_scale, void* out, float* lse, void* stream) {
    Plan pl;
    int rc = make_plan_q8(dims, &pl);
    if (rc != MLA_OK) return rc;
    if (!aligned16(schedule) || !aligned16(workspace) || !aligned16(q) || !aligned16(kv_cache) || !aligned16(kv_scales) ||
        !aligned16(block_table) || !aligned16(cache_seqlens) || !aligned16(out) || !aligned16(lse))
        return MLA_ERR_INVALID_ARG;
    if (!std::isfinite(softmax_scale)) return MLA_ERR_INVALID_ARG;
    CUtensorMap kvm, rm;
    rc = make_q8_map(&kvm, kv_cache, dims->num_blocks, 128);
    if (rc != MLA_OK) return rc;
    rc = make_q8_map(&rm, kv_cache, dims->num_blocks, 64);
    if (rc != MLA_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool in_kernel = q8_plan_in_kernel(dims->flags, pl);
    if ((dims->flags & MLA_FLAG_INLINE_PLAN) && !in_kernel) {
        rc = launch_schedule(pl, dims->batch, dims->max_blocks_per_seq, cache_seqlens, schedule, st);
        if (rc != MLA_OK) return rc;
    }
    Q8Params p = {};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.kv_scales = kv_scales;
    p.sched = static_cast<const int32_t*>(schedule);
    p.plan_out = in_kernel ? static_cast<int32_t*>(schedule) : nullptr;
    p.block_table = block_table;
    p.seqlens = cache_seqlens;
    p.kv = static_cast<const uint8_t*>(kv_cache);
    p.out = out;
    p.out_f32 = (dims->flags & MLA_FLAG_FP32_OUT) ? 1 : 0;
    p.lse = lse;
    p.opart = static_cast<float*>(workspace);
    p.lpart = p.opart + (size_t)pl.slots * pl.gr.NG * kDv;
    p.status = const_cast<int32_t*>(p.sched) + kHdrStatus;
    p.s_q = dims->s_q;
    p.heads = dims->num_heads;
    p.N = pl.gr.N;
    p.num_blocks = dims->num_blocks;
    p.max_blocks = dims->max_blocks_per_seq;
    p.causal = dims->causal;
    p.G = pl.G;
    p.BG = pl.BG;
    p.Hg = pl.plan_Hg;
    p.share = pl.share;
    p.overhead = pl.overhead;
    p.slots_cap = (int)pl.slots;
    p.scale_log2 = (float)((double)softmax_scale * 1.4426950408889634);
    p.test_stall = (dims->flags & MLA_FLAG_TEST_STALL) ? 1 : 0;
    p.run_rows = pl.gr.NG;
    p.kv_groups = 1;
    rc = pl.gr.NG == 16 ? launch_q8<16>(pl, p, kvm, rm, st) : launch_q8<32>(pl, p, kvm, rm, st);
    if (rc != MLA_OK) return rc;
    if (dims->flags & MLA_FLAG_NO_COMBINE) return MLA_OK;
    return launch_combine<kDv>(mla_colmap(dims, pl), pl, schedule, workspace, out, lse, dims->flags, in_kernel, st);
}

int mla_decode_q8_combine(const mla_decode_dims* dims, const void* schedule, const void* workspace, void* out, float* lse,
                          void* stream) {
    Plan pl;
    int rc = make_plan_q8(dims, &pl);
    if (rc != MLA_OK) return rc;
    if (!aligned16(schedule) || !aligned16(workspace) || !aligned16(out) || !aligned16(lse))
        return MLA_ERR_INVALID_ARG;
    return launch_combine<kDv>(mla_colmap(dims, pl), pl, schedule, workspace, out, lse, dims->flags,
                               q8_plan_in_kernel(dims->flags, pl), static_cast<cudaStream_t>(stream));
}

int mla_rope_init(const mla_rope_config* c, mla_rope_table* t) {
    if (c == nullptr || t == nullptr) return MLA_ERR_INVALID_ARG;
    if (!std::isfinite(c->theta) || c->theta <= 1.0 || !std::isfinite((float)c->amplitude) || c->reserved != 0 ||
        c->scaling < MLA_ROPE_NONE || c->scaling > MLA_ROPE_YARN || (c->interleaved != 0 && c->interleaved != 1))
        return MLA_ERR_INVALID_ARG;
    if (c->scaling != MLA_ROPE_NONE && !(std::isfinite(c->factor) && c->factor > 0.0)) return MLA_ERR_INVALID_ARG;
    const double kTwoPi = 6.283185307179586476925286766559;
    const int d = 2 * kRopePairs;
    double low = 0, high = 0;
    if (c->scaling == MLA_ROPE_YARN) {
        if (!std::isfinite(c->beta_fast) || !std::isfinite(c->beta_slow) || c->beta_fast <= 0 || c->beta_slow <= 0 ||
            c->original_max_position < 1)
            return MLA_ERR_INVALID_ARG;
        // the (real-valued) pair whose wavelength turns beta times within the original length
        auto pair_of = [&](double beta) {
            return d * std::log(c->original_max_position / (beta * kTwoPi)) / (2 * std::log(c->theta));
        };
        low = std::fmax(std::floor(pair_of(c->beta_fast)), 0.0);
        high = std::fmin(std::ceil(pair_of(c->beta_slow)), d - 1.0);
    }
    double turns[kRopePairs];
    for (int i = 0; i < kRopePairs; ++i) {
        double f = std::pow(c->theta, -2.0 * i / d);
        if (c->scaling == MLA_ROPE_LINEAR) f /= c->factor;
        if (c->scaling == MLA_ROPE_YARN) {
            const double r = std::fmin(std::fmax((i - low) / std::fmax(high - low, 0.001), 0.0), 1.0);
            f = f * (1.0 - r) + f / c->factor * r;
        }
        turns[i] = f / kTwoPi;
        // the angle of every position is a number
        if (!std::isfinite(turns[i] * 2147483648.0)) return MLA_ERR_INVALID_ARG;
    }
    for (int i = 0; i < kRopePairs; ++i) t->turns[i] = turns[i];
    t->amplitude = (float)c->amplitude;
    t->interleaved = c->interleaved;
    return MLA_OK;
}

int mla_rope_apply(const mla_rope_dims* d, const mla_rope_table* table, const void* x, const int32_t* positions, void* out,
                   void* stream) {
    if (d == nullptr || table == nullptr) return MLA_ERR_INVALID_ARG;
    if (d->tokens < 0 || d->num_heads < 1 || d->num_heads > 65535 || d->width < 2 * kRopePairs || d->width > 2048 || d->width % 8 != 0 ||
        d->offset < 0 || d->offset % 8 != 0 || d->offset + 2 * kRopePairs > d->width ||
        (d->transpose != 0 && d->transpose != 1))
        return MLA_ERR_INVALID_ARG;
    if (d->dtype != MLA_DTYPE_BF16 && d->dtype != MLA_DTYPE_FP32) return MLA_ERR_UNSUPPORTED;
    const int64_t st[4] = {d->x_token_stride, d->x_head_stride, d->out_token_stride, d->out_head_stride};
    for (int i = 0; i < 4; ++i)
        if (st[i] < 0 || st[i] % 8 != 0) return MLA_ERR_INVALID_ARG;
    // rows of out are apart: heads within a token and tokens, or tokens within a head and heads
    const int64_t T = d->tokens, h = d->num_heads, w = d->width, ts = st[2], hs = st[3];
    const bool by_token = (h == 1 || hs >= w) && (T <= 1 || ts >= (h - 1) * hs + w);
    const bool by_head = (T <= 1 || ts >= w) && (h == 1 || hs >= (T - 1) * ts + w);
    if (!by_token && !by_head) return MLA_ERR_INVALID_ARG;
    if (x == out && (st[0] != st[2] || st[1] != st[3])) return MLA_ERR_INVALID_ARG;
    if (d->tokens == 0) return MLA_OK;
    if (!aligned16(x) || !aligned16(out) || !aligned4(positions)) return MLA_ERR_INVALID_ARG;
    launch_rope(*d, *table, x, positions, out, static_cast<cudaStream_t>(stream));
    return launched();
}

int mla_cache_append(const mla_cache_dims* d, int32_t tokens, const void* c_kv, int64_t c_stride, const void* k_pe,
                     int64_t pe_stride, const int32_t* new_offsets, const mla_rope_table* table,
                     const int32_t* block_table, const int32_t* cache_seqlens, void* kv_cache, float* kv_scales,
                     int32_t* status, void* stream) {
    int rc = validate_cache(d);
    if (rc != MLA_OK) return rc;
    if (tokens < 0 || c_stride < kDv || c_stride % 8 != 0 || pe_stride < 2 * kRopePairs || pe_stride % 8 != 0)
        return MLA_ERR_INVALID_ARG;
    if (!aligned4(new_offsets) || !aligned4(block_table) || !aligned4(cache_seqlens) || !status_ok(status) ||
        !pool_ok(d, kv_cache, kv_scales))
        return MLA_ERR_INVALID_ARG;
    if (tokens == 0) return MLA_OK;
    if (!aligned16(c_kv) || !aligned16(k_pe)) return MLA_ERR_INVALID_ARG;
    AppendParams p = {};
    p.c_kv = static_cast<const __nv_bfloat16*>(c_kv);
    p.k_pe = static_cast<const __nv_bfloat16*>(k_pe);
    p.c_stride = c_stride;
    p.pe_stride = pe_stride;
    p.off = new_offsets;
    p.bt = block_table;
    p.lens = cache_seqlens;
    p.pool = pool_of(d, kv_cache, kv_scales);
    p.status = status;
    p.batch = d->batch;
    p.max_blocks = d->max_blocks_per_seq;
    p.tokens = tokens;
    p.rotate = table != nullptr;
    if (table) p.rope = *table;
    launch_append(p, static_cast<cudaStream_t>(stream));
    return launched();
}

size_t mla_cache_fork_workspace_bytes(int32_t n) {
    return n < 1 || n > kForkMax ? 0 : fork_workspace_words(n) * sizeof(int32_t);
}

int mla_cache_fork(const mla_cache_dims* d, int32_t n, const int32_t* parents, const int32_t* children,
                   int32_t* block_table, int32_t* cache_seqlens, int32_t* ref_counts, void* kv_cache, float* kv_scales,
                   void* workspace, int32_t* status, void* stream) {
    int rc = validate_cache(d);
    if (rc != MLA_OK) return rc;
    if (n < 1 || n > kForkMax) return MLA_ERR_INVALID_ARG;
    if (!aligned4(parents) || !aligned4(children) || !aligned4(block_table) || !aligned4(cache_seqlens) ||
        !aligned4(ref_counts) || !aligned16(workspace) || !status_ok(status) || !pool_ok(d, kv_cache, kv_scales))
        return MLA_ERR_INVALID_ARG;
    launch_fork(books_of(d, block_table, cache_seqlens, ref_counts, status), pool_of(d, kv_cache, kv_scales), n, parents,
                children, static_cast<int32_t*>(workspace), static_cast<cudaStream_t>(stream));
    return launched();
}

int mla_cache_free(const mla_cache_dims* d, int32_t n, const int32_t* rows, int32_t* block_table, int32_t* cache_seqlens,
                   int32_t* ref_counts, int32_t* status, void* stream) {
    int rc = validate_cache(d);
    if (rc != MLA_OK) return rc;
    if (n < 1) return MLA_ERR_INVALID_ARG;
    if (!aligned4(rows) || !aligned4(block_table) || !aligned4(cache_seqlens) || !aligned4(ref_counts) ||
        !status_ok(status))
        return MLA_ERR_INVALID_ARG;
    launch_free(books_of(d, block_table, cache_seqlens, ref_counts, status), n, rows, static_cast<cudaStream_t>(stream));
    return launched();
}

int mla_cache_copy_pages(const mla_cache_dims* d, int32_t n, const int32_t* src, const int32_t* dst, void* kv_cache,
                         float* kv_scales, int32_t* status, void* stream) {
    int rc = validate_cache(d);
    if (rc != MLA_OK) return rc;
    if (n < 0) return MLA_ERR_INVALID_ARG;
    if (!status_ok(status) || !pool_ok(d, kv_cache, kv_scales)) return MLA_ERR_INVALID_ARG;
    if (n == 0) return MLA_OK;
    if (!aligned4(src) || !aligned4(dst)) return MLA_ERR_INVALID_ARG;
    launch_copy_pages(pool_of(d, kv_cache, kv_scales), n, src, dst, status, static_cast<cudaStream_t>(stream));
    return launched();
}

size_t mla_cache_compact_workspace_bytes(const mla_cache_dims* d) {
    if (validate_cache(d) != MLA_OK) return 0;
    return compact_workspace_words(d->num_blocks) * sizeof(int32_t);
}

int mla_cache_compact(const mla_cache_dims* d, int32_t* block_table, const int32_t* cache_seqlens, int32_t* ref_counts,
                      void* kv_cache, float* kv_scales, void* workspace, int32_t* status, void* stream) {
    int rc = validate_cache(d);
    if (rc != MLA_OK) return rc;
    if (!aligned4(block_table) || !aligned4(cache_seqlens) || !aligned4(ref_counts) || !aligned16(workspace) ||
        !status_ok(status) || !pool_ok(d, kv_cache, kv_scales))
        return MLA_ERR_INVALID_ARG;
    launch_compact(books_of(d, block_table, const_cast<int32_t*>(cache_seqlens), ref_counts, status),
                   pool_of(d, kv_cache, kv_scales), static_cast<int32_t*>(workspace), static_cast<cudaStream_t>(stream));
    return launched();
}

}  // extern "C"
