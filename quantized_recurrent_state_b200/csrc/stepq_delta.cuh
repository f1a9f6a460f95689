// Launch arguments of the served-layer gated delta rule (stepq_delta.cu,
// stepq_delta_chunk.cu), shared with the C ABI that fills them, and the
// conversions of the token types.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace stepq {

// device error word
constexpr int kErrSeq = 32;    // a sequence's token range is not within the batch
constexpr int kErrRange = 64;  // the chunked form left the range of its operands

struct DeltaArgs {
    float *S;               // slots: [n_slots][n_layers][H][D][D]; else [n_seq][H][D][D]
    const int32_t *slots;   // null: state s belongs to sequence s
    const uint8_t *fresh;   // null: every sequence continues from its state
    const int32_t *cu;      // [n_seq + 1]; null: sequence s has the tokens [s n_tok, (s + 1) n_tok)
    int n_slots, n_layers, layer;
    int n_seq, n_tok, n_tokens;
    int H, Hk;
    const void *q, *k, *v;
    void *o;
    const float *alpha, *beta;
    int64_t qs, ks, vs, os;  // token strides in elements
    int check_gates;         // 1: a gate outside (0, 1] sets kErrGateRange
    int *err;
};

// dtype 0 fp32, 1 fp16, 2 bf16 (the ABI's STEPQ_FP32, STEPQ_FP16, STEPQ_BF16)
cudaError_t launch_delta_seq(int D, int dtype, bool rows, const DeltaArgs &a, cudaStream_t st);
// d = 128, per-head gates, fp16 or bf16 tokens
cudaError_t launch_delta_chunk(int dtype, const DeltaArgs &a, cudaStream_t st);

#ifdef __CUDACC__
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <class T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// N consecutive values (N sizeof(T) a multiple of 4, p aligned to the smaller of that and 16 bytes)
template <int N, class T>
__device__ __forceinline__ void load_vec(const T *p, float (&x)[N]) {
    constexpr int B = N * (int)sizeof(T), V = B < 16 ? B : 16, PER = V / (int)sizeof(T);
    static_assert(B % V == 0 && (V == 4 || V == 8 || V == 16), "vector width");
#pragma unroll
    for (int c = 0; c < B / V; ++c) {
        union {
            uint4 u4;
            uint2 u2;
            uint32_t u1;
            T e[PER];
        } raw;
        if constexpr (V == 16) raw.u4 = __ldg(reinterpret_cast<const uint4 *>(p) + c);
        else if constexpr (V == 8) raw.u2 = __ldg(reinterpret_cast<const uint2 *>(p) + c);
        else raw.u1 = __ldg(reinterpret_cast<const unsigned int *>(p) + c);
#pragma unroll
        for (int e = 0; e < PER; ++e) x[c * PER + e] = to_f32(raw.e[e]);
    }
}
template <int N, class T>
__device__ __forceinline__ void store_vec(T *p, const float (&x)[N]) {
    constexpr int B = N * (int)sizeof(T);
    static_assert(B == 8 || B == 16, "vector width");
    union {
        uint4 u4;
        uint2 u2;
        T e[N];
    } raw;
#pragma unroll
    for (int e = 0; e < N; ++e) raw.e[e] = from_f32<T>(x[e]);
    if constexpr (B == 16) *reinterpret_cast<uint4 *>(p) = raw.u4;
    else *reinterpret_cast<uint2 *>(p) = raw.u2;
}

// The state of sequence s, value head h; null where it is to be skipped.
__device__ __forceinline__ float *delta_state(const DeltaArgs &a, int s, int h, int D, int bad_slot) {
    size_t at;
    if (a.slots) {
        const int slot = a.slots[s];
        if (slot < 0 || slot >= a.n_slots) {
            if (slot != -1) atomicOr(a.err, bad_slot);
            return nullptr;
        }
        at = (size_t)slot * a.n_layers + a.layer;
    } else {
        at = (size_t)s;
    }
    return a.S + (at * a.H + h) * (size_t)(D * D);
}

// Token range of sequence s; false where it is not within the batch.
__device__ __forceinline__ bool delta_range(const DeltaArgs &a, int s, int &first, int &count) {
    if (!a.cu) {
        first = s * a.n_tok;
        count = a.n_tok;
        return true;
    }
    const int c0 = a.cu[s], c1 = a.cu[s + 1];
    first = c0;
    count = c1 - c0;
    if (c0 >= 0 && c1 >= c0 && c1 <= a.n_tokens) return true;
    atomicOr(a.err, kErrSeq);
    return false;
}
#endif

}  // namespace stepq
