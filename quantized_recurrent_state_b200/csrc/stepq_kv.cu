// Quantising keys and values into the paged cache as they are written, and
// reading sequences back (definitions: include/stepq.h).
//
// Both kernels move each byte once: a thread takes twice eight neighbouring values of a row (two 16-byte loads of a 16-bit
// type), one in each half, so d / 16 lanes share a row, a place or page and a scale are looked up once for 16 values, and the
// row's maximum is log2(d / 16) shuffles.  A block works on the keys or the values
// of one head; the heads of the same tokens are neighbouring blocks, whose rows lie side by side outside the cache.
// Bytes in flight hide the latency.  Writing: one row a thread and many threads (6,144 tokens, 8 heads of 128, 8 bits, bf16: 15.2 us,
// 38 MB; two and four rows, whose registers leave fewer warps, 16.4 and 23 us).  Reading, where a row is 16 bytes a
// thread behind three dependent loads: eight rows at once (31,000 such tokens: 45 us, 192 MB, 4.3 TB/s; with 256 threads a block 46 us, and four and two rows
// 47 and 66 us; 512 threads 52 us).  Bound by those latencies and HBM at large sizes, by the launch at small ones (70 tokens of 4 heads of 64 written: 2.1 us;
// 70 sequences of up to 300 read: 7.4 us, four rows 8.9).
#include <float.h>

#include "stepq_delta.cuh"
#include "stepq_dev.cuh"
#include "stepq_kv.cuh"

namespace stepq {

namespace {

constexpr int kThreads = 128, kReadRows = 8;

template <int D, int BITS, class T>
__global__ void __launch_bounds__(kThreads) k_kv_append(KvAppendArgs a) {
    constexpr int LANES = D / 16, PASS = kThreads / LANES, QMAX = (1 << (BITS - 1)) - 1;
    const KvGeo &g = a.g;
    const uint32_t tile = blockIdx.x / (2u * g.H), hw = blockIdx.x - tile * 2u * g.H;
    const int which = hw >= (uint32_t)g.H, h = hw - which * g.H, part = threadIdx.x % LANES;
    const int64_t t = (int64_t)tile * PASS + threadIdx.x / LANES;
    if (t >= a.n_tokens) return;
    const int64_t place = __ldg(a.places + t);
    const T *src = static_cast<const T *>(a.x[which]) + t * a.stride[which] + h * D + part * 8;
    float x[2][8];
#pragma unroll
    for (int c = 0; c < 2; ++c) load_vec<8>(src + c * (D / 2), x[c]);
    uint8_t *const head = a.cache + (int64_t)h * g.head_bytes();
    const uint32_t page_bytes = (uint32_t)g.page_bytes();      // below 2 GiB
    // rows are whole groups of lanes of one warp (32 is a multiple of LANES), which take the same way
    const unsigned lane0 = (threadIdx.x & 31) / LANES * LANES;
    const unsigned group = (LANES == 32 ? 0xffffffffu : ((1u << (LANES & 31)) - 1u)) << lane0;
    // magnitudes compared as their bits: a NaN is above infinity, and both mark the row
    int m = 0;
#pragma unroll
    for (int e = 0; e < 16; ++e) m = max(m, __float_as_int(x[e / 8][e % 8]) & 0x7fffffff);
#pragma unroll
    for (int s = LANES / 2; s > 0; s >>= 1) m = max(m, __shfl_xor_sync(group, m, s));
    // (asked here, so that the row's loads do not wait for its place)
    if (place < 0 || place >= (int64_t)g.n_pages * g.page_tokens) {
        if (place != -1 && part == 0 && hw == 0) atomicOr(g.err, kErrKvPlace);
        return;
    }
    const bool finite = m < 0x7f800000;
    // a row of zeros has the scale 0: it reads back the same as under any other, and attention must not take it for a large one
    float r = __int_as_float(m) / (float)QMAX;
    if (r < FLT_MIN) r = 0.0f;
    const float inv = r > 0.0f ? 1.0f / r : 0.0f;
    const int64_t page = place < (1 << 30) ? (int64_t)(__umulhi((uint32_t)place, a.div_mul) >> a.div_shift)
                                           : place / g.page_tokens;
    const int at = (int)(place - page * g.page_tokens);
    uint8_t *base = head + (uint64_t)page * page_bytes;
    uint8_t *dst = base + (uint32_t)(which * g.page_tokens + at) * (uint32_t)(D * BITS / 8) + part * BITS;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        uint32_t u[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            // 1.5 * 2^23 + the code's offset + the product, rounded once: the nearest integer to the exact product, ties
            // to even (the constant is even); |product| <= qmax (1 + 2^-22), so it needs no clamp
            const float y = fmaf(x[c][e], inv, 12582912.0f + (float)(QMAX + 1));
            u[e] = finite ? __float_as_uint(y) : (uint32_t)(QMAX + 1);
        }
        if constexpr (BITS == 8) {
            auto four = [&](int e) {
                return __byte_perm(__byte_perm(u[e], u[e + 1], 0x0040), __byte_perm(u[e + 2], u[e + 3], 0x0040), 0x5410);
            };
            *reinterpret_cast<uint2 *>(dst + c * (D * BITS / 16)) = make_uint2(four(0), four(4));
        } else {
            uint32_t w = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) w |= (u[e] & 0xfu) << (4 * e);
            *reinterpret_cast<uint32_t *>(dst + c * (D * BITS / 16)) = w;
        }
    }
    if (part == 0)
        *reinterpret_cast<float *>(base + (uint32_t)g.page_tokens * (2u * (D * BITS / 8) + 4u * which) + 4u * at) =
            finite ? r : __int_as_float(0x7fffffff);
}

template <int D, int BITS, class T>
__global__ void __launch_bounds__(kThreads) k_kv_read(KvReadArgs a, int tiles) {
    constexpr int LANES = D / 16, PASS = kThreads / LANES, ZERO = 1 << (BITS - 1);
    const KvGeo &g = a.g;
    const uint32_t tile = blockIdx.x / (2u * g.H), hw = blockIdx.x - tile * 2u * g.H;
    const int which = hw >= (uint32_t)g.H, h = hw - which * g.H, part = threadIdx.x % LANES;
    const int s = (int)(tile / tiles), t0 = (int)(tile % tiles) * (PASS * kReadRows) + threadIdx.x / LANES;
    const int len = __ldg(a.lens + s);
    if (t0 >= len) return;
    if (len > (int64_t)a.max_pages * g.page_tokens) {
        if (part == 0 && hw == 0) atomicOr(g.err, kErrKvLen);
        return;
    }
    const int64_t first = __ldg(a.cu + s);
    const uint8_t *const head = a.cache + (int64_t)h * g.head_bytes();
    const uint32_t page_bytes = (uint32_t)g.page_bytes();      // below 2 GiB
    const int32_t *table = a.table + (int64_t)s * a.max_pages;
    uint32_t w[kReadRows][2][BITS == 8 ? 2 : 1];
    float r[kReadRows];
    bool ok[kReadRows];
#pragma unroll
    for (int i = 0; i < kReadRows; ++i) {
        const int t = t0 + i * PASS;
        ok[i] = false;
        if (t >= len) continue;
        const int p = (int)(__umulhi((uint32_t)t, a.div_mul) >> a.div_shift), page = __ldg(table + p), at = t - p * g.page_tokens;
        ok[i] = page >= 0 && page < g.n_pages && first + t >= 0 && first + t < a.n_rows;
        if (!ok[i]) {
            if (part == 0 && hw == 0) atomicOr(g.err, kErrKvPlace);
            continue;
        }
        const uint8_t *base = head + (uint64_t)(uint32_t)page * page_bytes;
        const uint8_t *src = base + (uint32_t)(which * g.page_tokens + at) * (uint32_t)(D * BITS / 8) + part * BITS;
        r[i] = __ldg(reinterpret_cast<const float *>(base + (uint32_t)g.page_tokens * (2u * (D * BITS / 8) + 4u * which) + 4u * at));
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if constexpr (BITS == 8) {
                const uint2 y = __ldg(reinterpret_cast<const uint2 *>(src + c * (D / 2)));
                w[i][c][0] = y.x;
                w[i][c][1] = y.y;
            } else {
                w[i][c][0] = __ldg(reinterpret_cast<const unsigned int *>(src + c * (D / 4)));
            }
        }
    }
    T *dst = static_cast<T *>(a.x[which]) + h * D + part * 8;
#pragma unroll
    for (int i = 0; i < kReadRows; ++i) {
        if (!ok[i]) continue;
        T *to = dst + (first + t0 + i * PASS) * a.stride[which];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                // 2^23 + u has the code in its low bits
                float2 y;
                if constexpr (BITS == 8) {
                    y.x = __uint_as_float(__byte_perm(w[i][c][e / 4], 0x4b000000u, 0x7440 + e % 4));
                    y.y = __uint_as_float(__byte_perm(w[i][c][e / 4], 0x4b000000u, 0x7440 + e % 4 + 1));
                } else {
                    y.x = __uint_as_float(((w[i][c][0] >> (4 * e)) & 0xfu) | 0x4b000000u);
                    y.y = __uint_as_float(((w[i][c][0] >> (4 * e + 4)) & 0xfu) | 0x4b000000u);
                }
                const float zero = -(8388608.0f + (float)ZERO);
                y = mul2(add2(y, make_float2(zero, zero)), make_float2(r[i], r[i]));
                x[e] = y.x;
                x[e + 1] = y.y;
            }
            if constexpr (sizeof(T) == 2) {
                store_vec<8>(to + c * (D / 2), x);
            } else {
                *reinterpret_cast<float4 *>(to + c * (D / 2)) = make_float4(x[0], x[1], x[2], x[3]);
                *reinterpret_cast<float4 *>(to + c * (D / 2) + 4) = make_float4(x[4], x[5], x[6], x[7]);
            }
        }
    }
}

// f<D, BITS, T>() for the run-time geometry
template <class F>
cudaError_t dispatch(const KvGeo &g, int dtype, F f) {
    auto by_type = [&](auto d, auto b) {
        if (dtype == 0) return f(d, b, float());
        if (dtype == 1) return f(d, b, __half());
        return f(d, b, __nv_bfloat16());
    };
    auto by_bits = [&](auto d) {
        return g.bits == 8 ? by_type(d, std::integral_constant<int, 8>()) : by_type(d, std::integral_constant<int, 4>());
    };
    if (g.d == 64) return by_bits(std::integral_constant<int, 64>());
    if (g.d == 128) return by_bits(std::integral_constant<int, 128>());
    return by_bits(std::integral_constant<int, 256>());
}

}  // namespace

cudaError_t launch_kv_append(int dtype, const KvAppendArgs &a, cudaStream_t st) {
    const int64_t tile = kThreads / (a.g.d / 16), blocks = (a.n_tokens + tile - 1) / tile;
    if (blocks * 2 * a.g.H > 0x7fffffff) return cudaErrorInvalidValue;
    const unsigned grid = (unsigned)(blocks * 2 * a.g.H);
    return dispatch(a.g, dtype, [&](auto d, auto b, auto t) {
        k_kv_append<decltype(d)::value, decltype(b)::value, decltype(t)><<<grid, kThreads, 0, st>>>(a);
        return cudaGetLastError();
    });
}

cudaError_t launch_kv_read(int dtype, const KvReadArgs &a, cudaStream_t st) {
    const int64_t tile = kThreads / (a.g.d / 16) * kReadRows, tiles = ((int64_t)a.max_pages * a.g.page_tokens + tile - 1) / tile;
    if (tiles * a.n_seq > 0x7fffffff || tiles * a.n_seq * 2 * a.g.H > 0x7fffffff) return cudaErrorInvalidValue;
    const unsigned grid = (unsigned)(tiles * a.n_seq * 2 * a.g.H);
    return dispatch(a.g, dtype, [&](auto d, auto b, auto t) {
        k_kv_read<decltype(d)::value, decltype(b)::value, decltype(t)><<<grid, kThreads, 0, st>>>(a, (int)tiles);
        return cudaGetLastError();
    });
}

}  // namespace stepq
