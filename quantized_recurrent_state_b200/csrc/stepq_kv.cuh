// Geometry and launch arguments of the quantised key-value cache
// (stepq_kv.cu, stepq_kv_attend.cu), shared with the C ABI that fills them.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace stepq {

constexpr int kErrKvPlace = 1;  // device error word: a place, page or output row out of range
constexpr int kErrKvLen = 2;    // a length above max_pages * page_tokens
constexpr int kErrKvWait = 4;   // a wait for a copy gave up

struct KvGeo {
    int bits, H, d, page_tokens, n_pages;
    int *err;
    __host__ __device__ int row_bytes() const { return d * bits / 8; }
    __host__ __device__ int64_t head_bytes() const { return (int64_t)page_tokens * (2 * row_bytes() + 8); }
    __host__ __device__ int64_t page_bytes() const { return head_bytes() * H; }
};

struct KvAppendArgs {
    KvGeo g;
    uint8_t *cache;
    const void *x[2];       // k, v
    int64_t stride[2];
    const int64_t *places;
    int n_tokens;
    uint32_t div_mul;       // n / page_tokens = umulhi(n, div_mul) >> div_shift for n < 2^30
    int div_shift;
};

struct KvReadArgs {
    KvGeo g;
    const uint8_t *cache;
    const int32_t *table, *lens, *cu;
    int n_seq, max_pages;
    int64_t n_rows;
    void *x[2];
    int64_t stride[2];
    uint32_t div_mul;
    int div_shift;
};

struct KvAttendArgs {
    KvGeo g;
    const uint8_t *cache;
    const int32_t *table, *lens;
    int n_seq, max_pages, n_tok, Hq, dtype;
    const void *q;
    void *o;
    int64_t qs, os;
    float scale;
    float *lse;
    float *part;            // pieces of units: sums [block][2][row][d]
    float4 *meta;           // and (score reference, total, scale reference, -) [block][2][row]
    int blocks, row_tiles;
    uint32_t div_mul;
    int div_shift;
    int seg;                // tokens of a copy: divides a page and a stage of 64, at least 16
    uint32_t polls;         // before a wait gives up
    uint32_t phantom_tx;    // bytes a stage waits for that never arrive (0: none; the test of that)
};

// dtype 0 fp32, 1 fp16, 2 bf16
cudaError_t launch_kv_append(int dtype, const KvAppendArgs &a, cudaStream_t st);
cudaError_t launch_kv_read(int dtype, const KvReadArgs &a, cudaStream_t st);

// How a call is cut up: rows of query heads and tokens that share a cache head, eight to an MMA column tile, nr (1 or 2)
// tiles to a unit of work.
struct KvSplit {
    int nr, row_tiles;
};
KvSplit kv_split(const KvGeo &g, int n_tok, int Hq);
// Blocks that the current device holds at once, [nr - 1][0: 16-bit queries, 1: fp32], and the kernels' shared memory set; once
// per cache.
cudaError_t kv_prepare(const KvGeo &g, int n_sms, int (*blocks)[2]);
cudaError_t launch_kv_attend(const KvAttendArgs &a, int nr, cudaStream_t st);

}  // namespace stepq
