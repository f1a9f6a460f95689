// Quantising keys and values into the paged cache as they are written, and
// reading sequences back (definitions: include/stepq.h).
//
// Both kernels move each byte once: a thread takes eight neighbouring values
// of a row (one 16-byte load of a 16-bit type), d / 8 lanes share a row, and the
// row's maximum is log2(d / 8) shuffles.  HBM-bound at large sizes,
// launch-bound at small ones.
#include <float.h>

#include "stepq_delta.cuh"
#include "stepq_kv.cuh"

namespace stepq {

namespace {

constexpr int kThreads = 256;

template <int D, int BITS, class T>
__global__ void __launch_bounds__(kThreads) k_kv_append(KvAppendArgs a) {
    constexpr int LANES = D / 8, QMAX = (1 << (BITS - 1)) - 1;
    const KvGeo &g = a.g;
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int part = (int)(id % LANES);
    const int64_t row = id / LANES;                         // [token][k, v][head]
    const int h = (int)(row % g.H), which = (int)(row / g.H % 2);
    const int64_t t = row / g.H / 2;
    // rows are whole groups of lanes of one warp (kThreads and 32 are multiples of LANES)
    const unsigned lane0 = (threadIdx.x & 31) / LANES * LANES;
    const unsigned group = (LANES == 32 ? 0xffffffffu : ((1u << (LANES & 31)) - 1u)) << lane0;
    if (t >= a.n_tokens) return;
    const int64_t place = a.places[t];
    if (place < 0 || place >= (int64_t)g.n_pages * g.page_tokens) {
        if (place != -1 && part == 0) atomicOr(g.err, kErrKvPlace);
        return;
    }
    float x[8];
    load_vec<8>(static_cast<const T *>(a.x[which]) + t * a.stride[which] + h * D + part * 8, x);
    float m = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float y = fabsf(x[e]);
        m = y <= FLT_MAX ? fmaxf(m, y) : INFINITY;          // a NaN counts as an infinity
    }
#pragma unroll
    for (int s = LANES / 2; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(group, m, s));
    float r = m / (float)QMAX;
    if (r < FLT_MIN) r = 1.0f;
    const bool finite = m <= FLT_MAX;
    const float inv = 1.0f / r;
    uint32_t u[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        // 1.5 * 2^23 + the product, rounded once: the nearest integer to the exact product, ties to even
        const int z = __float_as_int(fmaf(x[e], inv, 12582912.0f)) - 0x4B400000;
        u[e] = finite ? (uint32_t)(min(max(z, -QMAX), QMAX) + QMAX + 1) : (uint32_t)(QMAX + 1);
    }
    const int64_t page = place / g.page_tokens;
    const int at = (int)(place - page * g.page_tokens);
    uint8_t *dst = a.cache + g.codes_at(page, h, which) + (int64_t)at * (D * BITS / 8) + part * BITS;
    if constexpr (BITS == 8) {
        *reinterpret_cast<uint2 *>(dst) = make_uint2(u[0] | u[1] << 8 | u[2] << 16 | u[3] << 24,
                                                     u[4] | u[5] << 8 | u[6] << 16 | u[7] << 24);
    } else {
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) w |= u[e] << (4 * e);
        *reinterpret_cast<uint32_t *>(dst) = w;
    }
    if (part == 0)
        *reinterpret_cast<float *>(a.cache + g.scales_at(page, h, which) + 4 * (int64_t)at) =
            finite ? r : __int_as_float(0x7fffffff);
}

// A block takes kReadTokens tokens of one sequence, all heads, keys and values.
constexpr int kReadTokens = 16;

template <int D, int BITS, class T>
__global__ void __launch_bounds__(kThreads) k_kv_read(KvReadArgs a, int tiles) {
    constexpr int LANES = D / 8, ZERO = 1 << (BITS - 1);
    const KvGeo &g = a.g;
    const int s = (int)(blockIdx.x / tiles), t0 = (int)(blockIdx.x % tiles) * kReadTokens;
    const int len = a.lens[s];
    if (t0 >= len) return;
    if (len > (int64_t)a.max_pages * g.page_tokens) {
        if (threadIdx.x == 0) atomicOr(g.err, kErrKvLen);
        return;
    }
    const int page = a.table[(int64_t)s * a.max_pages + t0 / g.page_tokens];
    const int64_t first = (int64_t)a.cu[s] + t0;
    const int n = min(kReadTokens, len - t0);
    if (page < 0 || page >= g.n_pages || first < 0 || first + n > a.n_rows) {
        if (threadIdx.x == 0) atomicOr(g.err, kErrKvPlace);
        return;
    }
    const int at0 = t0 % g.page_tokens;
    for (int id = threadIdx.x; id < n * 2 * g.H * LANES; id += kThreads) {
        const int part = id % LANES, row = id / LANES;
        const int h = row % g.H, which = row / g.H % 2, t = row / g.H / 2;
        const uint8_t *src = a.cache + g.codes_at(page, h, which) + (int64_t)(at0 + t) * (D * BITS / 8) + part * BITS;
        const float r = __ldg(reinterpret_cast<const float *>(a.cache + g.scales_at(page, h, which)) + at0 + t);
        uint32_t w[BITS == 8 ? 2 : 1];
        if constexpr (BITS == 8) {
            const uint2 y = __ldg(reinterpret_cast<const uint2 *>(src));
            w[0] = y.x;
            w[1] = y.y;
        } else {
            w[0] = __ldg(reinterpret_cast<const unsigned int *>(src));
        }
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t u = BITS == 8 ? (w[e / 4] >> (8 * (e % 4))) & 0xffu : (w[0] >> (4 * e)) & 0xfu;
            x[e] = r * (float)((int)u - ZERO);
        }
        T *dst = static_cast<T *>(a.x[which]) + (first + t) * a.stride[which] + h * D + part * 8;
        if constexpr (sizeof(T) == 2) {
            store_vec<8>(dst, x);
        } else {
            *reinterpret_cast<float4 *>(dst) = make_float4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<float4 *>(dst + 4) = make_float4(x[4], x[5], x[6], x[7]);
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
    const int64_t threads = (int64_t)a.n_tokens * 2 * a.g.H * (a.g.d / 8);
    const int64_t blocks = (threads + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    return dispatch(a.g, dtype, [&](auto d, auto b, auto t) {
        k_kv_append<decltype(d)::value, decltype(b)::value, decltype(t)><<<(unsigned)blocks, kThreads, 0, st>>>(a);
        return cudaGetLastError();
    });
}

cudaError_t launch_kv_read(int dtype, const KvReadArgs &a, cudaStream_t st) {
    const int64_t tiles = (int64_t)a.max_pages * (a.g.page_tokens / kReadTokens);
    if (tiles * a.n_seq > 0x7fffffff) return cudaErrorInvalidValue;
    return dispatch(a.g, dtype, [&](auto d, auto b, auto t) {
        k_kv_read<decltype(d)::value, decltype(b)::value, decltype(t)>
            <<<(unsigned)(tiles * a.n_seq), kThreads, 0, st>>>(a, (int)tiles);
        return cudaGetLastError();
    });
}

}  // namespace stepq
