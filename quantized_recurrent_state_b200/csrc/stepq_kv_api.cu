// C ABI of the quantised key-value cache (include/stepq.h): geometry, argument
// checks and launches.
#include <cmath>
#include <new>

#include "../../include/stepq.h"
#include "stepq_host.h"
#include "stepq_kv.cuh"

using stepq::check_ptr;
using stepq::check_rows;
using stepq::cuda_fail;
using stepq::fail;
using stepq::NvtxRange;

struct stepq_kv {
    stepq::KvGeo g{};
    stepq::ErrorWord err;
    int device = 0;
    // ceil(2^(30 + l) / page_tokens), l = ceil(log2 page_tokens) >= 4: exact quotients of numbers below 2^30
    uint32_t div_mul = 0;
    int div_shift = 0;
    int blocks[2][2] = {};  // of an attend call, by tiles of rows and terms of q
    uint32_t polls = 1u << 22, phantom_tx = 0;
};

extern "C" int stepq_kv_create(int bits, int n_heads, int d, int page_tokens, int n_pages, stepq_kv **out) {
    if (!out) return fail(STEPQ_EINVAL, "kv_create: null argument");
    if (bits != 4 && bits != 8) return fail(STEPQ_EINVAL, "kv_create: width %d (4 or 8)", bits);
    if (d != 64 && d != 128 && d != 256) return fail(STEPQ_EINVAL, "kv_create: d %d (64, 128 or 256)", d);
    if (n_heads < 1 || n_heads > 4096) return fail(STEPQ_EINVAL, "kv_create: n_heads %d", n_heads);
    if (page_tokens < 16 || page_tokens > 65536 || page_tokens % 16)
        return fail(STEPQ_EINVAL, "kv_create: page_tokens %d (a multiple of 16, at most 65536)", page_tokens);
    if (n_pages < 1) return fail(STEPQ_EINVAL, "kv_create: n_pages %d", n_pages);
    const stepq::KvGeo g{bits, n_heads, d, page_tokens, n_pages, nullptr};
    if (g.page_bytes() > 0x7fffffff) return fail(STEPQ_EINVAL, "kv_create: a page of %lld bytes", (long long)g.page_bytes());
    int dev = 0, major = 0, minor = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if ((e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
        return cuda_fail(e, "cudaDeviceGetAttribute");
    if (major < 10) return fail(STEPQ_ECUDA, "kv_create: device %d is sm_%d%d; this library is built for sm_100a", dev, major, minor);
    stepq_kv *kv = new (std::nothrow) stepq_kv;
    if (!kv) return fail(STEPQ_ENOMEM, "kv_create: out of memory");
    kv->g = g;
    int l = 4;
    while ((1 << l) < page_tokens) ++l;
    kv->div_mul = (uint32_t)(((1ull << (30 + l)) + page_tokens - 1) / page_tokens);
    kv->div_shift = l - 2;
    kv->device = dev;
    if ((e = stepq::kv_prepare(g, sms, kv->blocks)) != cudaSuccess) {
        delete kv;
        return cuda_fail(e, "kv_create: kernel setup");
    }
    if ((e = kv->err.create()) != cudaSuccess) {
        kv->err.destroy();
        delete kv;
        return cuda_fail(e, "cudaMalloc(error word)");
    }
    kv->g.err = kv->err.device();
    *out = kv;
    return STEPQ_OK;
}

extern "C" void stepq_kv_free(stepq_kv *kv) {
    if (!kv) return;
    {
        const stepq::DeviceScope dev(kv->device);
        kv->err.destroy();
    }
    delete kv;
}

extern "C" size_t stepq_kv_bytes(const stepq_kv *kv) { return kv ? (size_t)kv->g.page_bytes() * kv->g.n_pages : 0; }

extern "C" int stepq_kv_append(stepq_kv *kv, void *cache, int dtype, int n_tokens, const void *k, const void *v,
                               int64_t k_stride, int64_t v_stride, const int64_t *places, void *stream) {
    NvtxRange nvtx_range("stepq_kv_append");
    if (!kv) return fail(STEPQ_EINVAL, "kv_append: null cache handle");
    int rc = stepq::check_dtype(dtype, "kv_append");
    if (rc) return rc;
    if (n_tokens < 0) return fail(STEPQ_EINVAL, "kv_append: n_tokens %d", n_tokens);
    if ((rc = check_ptr(cache, 128, "cache"))) return rc;
    if (n_tokens == 0) return STEPQ_OK;
    const long long width = (long long)kv->g.H * kv->g.d;
    if ((rc = check_rows(k, dtype, k_stride, width, "k")) || (rc = check_rows(v, dtype, v_stride, width, "v")) ||
        (rc = check_ptr(places, 8, "places")))
        return rc;
    const stepq::DeviceScope dev(kv->device);
    if (dev.error() != cudaSuccess) return cuda_fail(dev.error(), "cudaSetDevice");
    const stepq::KvAppendArgs a{kv->g, static_cast<uint8_t *>(cache), {k, v}, {k_stride, v_stride}, places, n_tokens,
                                kv->div_mul, kv->div_shift};
    const cudaError_t e = stepq::launch_kv_append(dtype, a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? STEPQ_OK : cuda_fail(e, "kv_append launch");
}

static int check_table(const stepq_kv *kv, const void *cache, int n_seq, const int32_t *page_table, int max_pages,
                       const int32_t *lens, const char *what) {
    int rc;
    if (n_seq < 0) return fail(STEPQ_EINVAL, "%s: n_seq %d", what, n_seq);
    if (max_pages < 1 || (long long)max_pages * kv->g.page_tokens > (1ll << 30))
        return fail(STEPQ_EINVAL, "%s: max_pages %d", what, max_pages);
    if ((rc = check_ptr(cache, 128, "cache"))) return rc;
    if (n_seq == 0) return STEPQ_OK;
    if ((rc = check_ptr(page_table, 4, "page_table")) || (rc = check_ptr(lens, 4, "lens"))) return rc;
    return STEPQ_OK;
}

extern "C" int stepq_kv_read(stepq_kv *kv, const void *cache, int n_seq, const int32_t *page_table, int max_pages,
                             const int32_t *lens, const int32_t *cu_seqlens, int64_t n_rows, int dtype, void *k,
                             void *v, int64_t k_stride, int64_t v_stride, void *stream) {
    NvtxRange nvtx_range("stepq_kv_read");
    if (!kv) return fail(STEPQ_EINVAL, "kv_read: null cache handle");
    int rc = stepq::check_dtype(dtype, "kv_read");
    if (rc || (rc = check_table(kv, cache, n_seq, page_table, max_pages, lens, "kv_read"))) return rc;
    if (n_rows < 0) return fail(STEPQ_EINVAL, "kv_read: n_rows %lld", (long long)n_rows);
    if (n_seq == 0) return STEPQ_OK;
    if ((rc = check_ptr(cu_seqlens, 4, "cu_seqlens"))) return rc;
    const long long width = (long long)kv->g.H * kv->g.d;
    if (n_rows > 0 && ((rc = check_rows(k, dtype, k_stride, width, "k")) || (rc = check_rows(v, dtype, v_stride, width, "v"))))
        return rc;
    const stepq::DeviceScope dev(kv->device);
    if (dev.error() != cudaSuccess) return cuda_fail(dev.error(), "cudaSetDevice");
    const stepq::KvReadArgs a{kv->g, static_cast<const uint8_t *>(cache), page_table, lens, cu_seqlens, n_seq, max_pages,
                              n_rows, {k, v}, {k_stride, v_stride}, kv->div_mul, kv->div_shift};
    const cudaError_t e = stepq::launch_kv_read(dtype, a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? STEPQ_OK : cuda_fail(e, "kv_read launch");
}

extern "C" size_t stepq_kv_attend_workspace_bytes(const stepq_kv *kv, int n_seq, int n_tok, int n_q_heads, int max_pages) {
    if (!kv || n_seq < 0 || n_tok < 1 || n_q_heads < 1 || n_q_heads % kv->g.H || max_pages < 1) return 0;
    // two pieces a block: sums, (references, total)
    const int nr = stepq::kv_split(kv->g, n_tok, n_q_heads).nr;
    const int blocks = kv->blocks[nr - 1][0] > kv->blocks[nr - 1][1] ? kv->blocks[nr - 1][0] : kv->blocks[nr - 1][1];
    return (size_t)blocks * 2 * 8 * nr * (kv->g.d + 4) * sizeof(float);
}

extern "C" int stepq_kv_attend(stepq_kv *kv, const void *cache, int n_seq, const int32_t *page_table, int max_pages,
                               const int32_t *lens, int dtype, int n_tok, int n_q_heads, const void *q, int64_t q_stride,
                               float scale, void *o, int64_t o_stride, float *lse, void *workspace, void *stream) {
    NvtxRange nvtx_range("stepq_kv_attend");
    if (!kv) return fail(STEPQ_EINVAL, "kv_attend: null cache handle");
    int rc = stepq::check_dtype(dtype, "kv_attend");
    if (rc || (rc = check_table(kv, cache, n_seq, page_table, max_pages, lens, "kv_attend"))) return rc;
    if (n_tok < 1) return fail(STEPQ_EINVAL, "kv_attend: n_tok %d", n_tok);
    if (n_q_heads < 1 || n_q_heads % kv->g.H)
        return fail(STEPQ_EINVAL, "kv_attend: %d query heads are no multiple of the cache's %d", n_q_heads, kv->g.H);
    if ((long long)n_tok * n_q_heads > (1ll << 24)) return fail(STEPQ_EINVAL, "kv_attend: %d tokens of %d heads", n_tok, n_q_heads);
    if (!std::isfinite(scale) || !(scale > 0.0f)) return fail(STEPQ_EINVAL, "kv_attend: scale %g", scale);
    if (n_seq == 0) return STEPQ_OK;
    const long long width = (long long)n_q_heads * kv->g.d;
    if ((rc = check_rows(q, dtype, q_stride, width, "q")) || (rc = check_rows(o, dtype, o_stride, width, "o")) ||
        (rc = check_ptr(workspace, 16, "workspace")))
        return rc;
    if (lse && (rc = check_ptr(lse, 4, "lse"))) return rc;
    const stepq::DeviceScope dev(kv->device);
    if (dev.error() != cudaSuccess) return cuda_fail(dev.error(), "cudaSetDevice");
    const stepq::KvSplit k = stepq::kv_split(kv->g, n_tok, n_q_heads);
    const int blocks = kv->blocks[k.nr - 1][dtype == STEPQ_FP32 ? 1 : 0];
    float *const part = static_cast<float *>(workspace);
    const stepq::KvAttendArgs a{kv->g, static_cast<const uint8_t *>(cache), page_table, lens, n_seq, max_pages, n_tok,
                                n_q_heads, dtype, q, o, q_stride, o_stride, scale, lse,
                                part, reinterpret_cast<float4 *>(part + (size_t)blocks * 2 * 8 * k.nr * kv->g.d),
                                blocks, k.row_tiles, kv->div_mul, kv->div_shift,
                                kv->g.page_tokens % 64 == 0 ? 64 : kv->g.page_tokens % 32 == 0 ? 32 : 16,
                                kv->polls, kv->phantom_tx};
    const cudaError_t e = stepq::launch_kv_attend(a, k.nr, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? STEPQ_OK : cuda_fail(e, "kv_attend launch");
}

extern "C" int stepq_kv_set_wait_limit(stepq_kv *kv, uint32_t polls, uint32_t phantom_bytes) {
    if (!kv) return fail(STEPQ_EINVAL, "kv_set_wait_limit: null cache handle");
    if (phantom_bytes >= (1u << 16)) return fail(STEPQ_EINVAL, "kv_set_wait_limit: phantom_bytes %u", phantom_bytes);
    kv->polls = polls ? polls : (1u << 22);
    kv->phantom_tx = phantom_bytes;
    return STEPQ_OK;
}

extern "C" int stepq_kv_check(stepq_kv *kv, void *stream) {
    if (!kv) return fail(STEPQ_EINVAL, "kv_check: null cache handle");
    const stepq::DeviceScope dev(kv->device);
    cudaError_t e = dev.error();
    int word = 0;
    if (e == cudaSuccess) e = kv->err.take(static_cast<cudaStream_t>(stream), word);
    if (e != cudaSuccess) return cuda_fail(e, "kv_check");
    if (!word) return STEPQ_OK;
    return fail(STEPQ_EDEVICE, "device error word 0x%x (%s%s%s)", word,
                (word & stepq::kErrKvPlace) ? "place, page or output row out of range " : "",
                (word & stepq::kErrKvLen) ? "length above the page table's " : "",
                (word & stepq::kErrKvWait) ? "copy wait gave up " : "");
}
