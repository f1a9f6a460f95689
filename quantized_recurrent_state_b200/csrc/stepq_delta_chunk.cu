// The gated delta rule over a ragged batch in chunks of 64 tokens on the fifth-generation tensor
// cores: d = 128, per-head gates, bfloat16 or fp16 tokens, fp32 states.
//
// With gamma_t the running product of the gates in a chunk, Gamma_ts = gamma_t / gamma_s and S the
// state before it; k'_t = k_t / ks_t and q'_t = q_t / qs_t, ks_t and qs_t powers of two that bring
// the row's largest value to [1, 2); u'_t = ks_t u_t:
//   X = (I + N)^-1,  N_ts = beta_t ks_t^2 Gamma_ts k'_t.k'_s (s < t)
//   U' = X R,        R_t = beta_t ks_t (v_t - gamma_t ks_t S^T k'_t)
//   O_t = qs_t (gamma_t S^T q'_t + sum_s A_ts u'_s),  A_ts = Gamma_ts q'_t.k'_s (s <= t)
//   S  <- gamma_C S + K'^T diag(gamma_C / gamma) U'
// Every Gamma is at most 1, so nothing overflows however fast a gate decays.
//
// Precision: q' and k' are exact fp16 operands (bfloat16 tokens: to 2^-25 of the row's largest value).  Gates are multiplied
// up in fp32, 64 of them at most.  fp32 operands (S, R, U', X) enter as the sum of two fp16 values, 2^-22 of the value: each value
// column's S, and its R and U', are scaled by a power of two taken from an upper bound, which may be 2^13 too large before a bit is
// lost.  Accumulators are fp32, S is held in fp32.  The readout uses the leading terms alone for bfloat16
// outputs (2^-12 of a term against their own 2^-9) and both terms for fp16.  X stays below 2^5 while beta |k|^2 <= 2, where the recurrence
// does not grow.  An operand that leaves fp16 is the sum of infinity and its opposite, which every product takes on to U' as
// NaN; a U' beyond fp16 from tokens and a state that are numbers sets kErrRange.
//
// One block per (sequence, head) walks the chunks; blocks of heads that share k and q are neighbours.  The
// chain S -> R -> U' -> S is serial, so the block is split by what it waits for:
//   warps 0-7  (state)   thread = value column j and half of the key rows: S in registers; R, U', S as operands;
//                        thread 0 issues the products that need them
//   warps 8-15 (prepare) two groups of four warps, a group to every other chunk: loads, scales, gates, [K; Q] K^T, X, A,
//                        and the chunk's output.  What a group prepares is mostly latency (loads, barriers, the
//                        substitution), so two chunks at a time.
// The register file is split 168 : 88 between them (2 x 168 + 2 x 88 = 4 x 128 in each quarter of the SM).
// The value columns j are the lanes of every product (W^T = S^T K'^T and so on), so what a
// product leaves in a thread's lane is what the thread feeds to the next one.
//
// Tensor memory columns: S^T terms 0-127 (hi, lo, two values a column), later diag(gamma_C / gamma) U' (0-63) and U'
// (64-127); W^T 128-191 and R terms 192-255, later the state's increment; Y^T = S^T Q'^T 256-319; U'^T 320-383, later
// A U'; [K; Q] K^T 384-511, one for each group.
//
// Bound: latency, not HBM (14 %) nor the tensor pipe (23 %).  A chunk of a head takes 9,000 cycles: S to operands 1,700, W 700,
// R 1,600, U' 900, the increment 900, S 550, the rest hand-overs; a group's preparation takes 13,000 for every other chunk.  The SM
// issues 52 % of the time, 24,000 warp instructions a chunk.  2,048 tokens of one prompt and 48 heads 173 us; 16 prompts of up
// to 2,048 tokens 572 us (floor 107: 0.7 GB); 37 prompts of up to 130 tokens and 32 heads 148 us.
// C = 64: X costs C^2 a token and the hand-overs 1 / C; 64 rows of K and 64 of Q fill the 128 rows of one product.
//
// Sequences of at most 12 tokens go token by token in the same launch (short_sequence): their state is all they cost, and a
// launch of their own for a ragged batch measured more (64 sequences of two to four tokens 83 to 98 us, as chunks 176).
//
// Every wait is bounded: a wait that gives up ends its warp's or group's part and sets kErrWait; what waits for that
// part gives up in turn.
#include <type_traits>

#include "stepq_dev.cuh"
#include "stepq_delta.cuh"
#include "stepq_prefill.cuh"
#include "stepq_tc16.cuh"

namespace stepq {

namespace {

constexpr int D = 128, C = 64, NS = 256, NP = 128, NT = NS + 2 * NP;
constexpr uint32_t kPolls = 1u << 20;
constexpr uint32_t TSH = 0, TSL = 64, TFH = 0, TFL = 32, TUH = 64, TUL = 96, TW = 128, TRH = 192, TRL = 224, TD = 128, TY = 256,
                   TU = 320, TG = 384;
constexpr uint32_t kHalf = 128 * 128;   // bytes of 64 columns of [K; Q]
constexpr int SN = C + 4;               // row stride of the fp32 scratch matrix
constexpr int kTopS = 13, kTopR = 6;    // the scaled bounds of S and R are 2^kTop
constexpr float kHalfMax = 65504.0f, kFloatMax = 3.402823466e38f;

template <class T>
struct Smem {
    static constexpr int AT = std::is_same<T, __half>::value ? 2 : 1;   // terms of A (and of S and U' in the readout)
    alignas(1024) uint8_t kq[2][2 * kHalf];    // [buffer][column half][K rows, Q rows][128 bytes]
    alignas(1024) uint8_t x[2][2 * C * 128];   // X, two terms
    alignas(1024) uint8_t a[2][AT * C * 128];  // A
    alignas(16) T v[2][C * D];                 // V, later the chunk's output
    alignas(16) float n[2][C * SN];            // by group: N below the diagonal, its inverse in place
    alignas(16) float gk[2][C], bk[2][C];      // gamma ks, beta ks
    alignas(16) float f[2][C];                 // gamma_C / gamma
    alignas(16) float go[2][C], qs[2][C];      // gamma qs, qs
    alignas(16) float ks[2][C], be[2][C];      // by group: ks, beta ks^2
    alignas(16) float al[2][C], up[2][C], down[2][C];   // the gate; the product of its half chunk's up to it, and after it
    float gl[2], mb[2], mg[2];                 // gamma_C, the largest beta ks, the largest gamma ks
    int finite[2];                             // the chunk's keys are numbers and its gates in range
    float smx[2][D], vmx[2][D], umx[2][D];     // largest |S|, |v|, |u'| of a lane, by half
    float ss[2][D], sr[2][D];                  // a lane's scales of the S and R terms
    alignas(8) uint64_t full[2], vfull[2], ready[2], empty[2], sput, rput, uput[2], w, u, d, z[2], out, g[2], drain[3];
    uint32_t taddr;
};

__device__ __forceinline__ void mbar_init_n(uint64_t *bar, uint32_t n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(tc::smem_addr(bar)), "r"(n) : "memory");
}
// A warp's wait: the same answer in every lane.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, kPolls));
}
// 16 bytes of global memory into shared memory, or zeros.
__device__ __forceinline__ void copy16(void *dst, const void *src, bool take) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_addr(dst)), "l"(src), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 pair_of(const uint32_t *v, int i) {
    return make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
}
// The power of two that brings `bound` (>= 0) to at most 2^top (bounds below 2^-86 as 2^-86), and its inverse.
__device__ __forceinline__ void scale_for(float bound, int top, float &s, float &inv) {
    const int e = min(max((int)(__float_as_uint(bound) >> 23), 41), 240) + 1 - top;
    s = __uint_as_float((uint32_t)e << 23);
    inv = __uint_as_float((uint32_t)(254 - e) << 23);
}
// The exponent of the power of two at or below x >= 0 (0, infinity, NaN: of 1), its inverse a normal number, too.
__device__ __forceinline__ int exponent_of(float x) {
    const int e = (int)(__float_as_uint(x) >> 23);
    return e == 0 || e == 255 ? 127 : min(e, 253);
}
// The larger of both, NaN where one is.
__device__ __forceinline__ float max_nan(float x, float y) {
    float z;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
    return z;
}
template <class T>
struct Pair;
template <>
struct Pair<__half> {
    using type = __half2;
};
template <>
struct Pair<__nv_bfloat16> {
    using type = __nv_bfloat162;
};
__device__ __forceinline__ __half2 lows(__half2 x, __half2 y) { return __lows2half2(x, y); }
__device__ __forceinline__ __half2 highs(__half2 x, __half2 y) { return __highs2half2(x, y); }
__device__ __forceinline__ __nv_bfloat162 lows(__nv_bfloat162 x, __nv_bfloat162 y) { return __lows2bfloat162(x, y); }
__device__ __forceinline__ __nv_bfloat162 highs(__nv_bfloat162 x, __nv_bfloat162 y) { return __highs2bfloat162(x, y); }
__device__ __forceinline__ float2 to_f32x2(__half2 x) { return __half22float2(x); }
__device__ __forceinline__ float2 to_f32x2(__nv_bfloat162 x) { return __bfloat1622float2(x); }

// A sequence of at most kShort tokens, token by token: a warp has 8 value columns, lane 4 g + c rows [16 g, 16 g + 16) of two.
// A chunk costs a block about 12 us however few tokens it has (64 sequences of 32 heads: up to 4 tokens 176 us in chunks).
constexpr int kShort = 12;
template <class T>
__device__ __forceinline__ void short_sequence(const DeltaArgs &a, float *Sg, bool fresh, int first, int count, int h, int hk) {
    const int lane = threadIdx.x & 31, row0 = (lane >> 2) * 16, col0 = 8 * (threadIdx.x >> 5) + 2 * (lane & 3);
    Sg += (size_t)row0 * D + col0;
    float2 S[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) S[r] = fresh ? make_float2(0.f, 0.f) : *reinterpret_cast<const float2 *>(Sg + (size_t)r * D);
    auto sum = [&](float2 x) {   // over the eight groups of rows
#pragma unroll
        for (int m = 4; m < 32; m <<= 1) {
            x.x += __shfl_xor_sync(0xffffffffu, x.x, m);
            x.y += __shfl_xor_sync(0xffffffffu, x.y, m);
        }
        return x;
    };
    bool good = true;
#pragma unroll 1
    for (int i = 0; i < count; ++i) {
        const size_t t = (size_t)(first + i);
        float k[16], q[16], v[2];
        load_vec<16>(static_cast<const T *>(a.k) + t * a.ks + hk * D + row0, k);
        load_vec<16>(static_cast<const T *>(a.q) + t * a.qs + hk * D + row0, q);
        load_vec<2>(static_cast<const T *>(a.v) + t * a.vs + h * D + col0, v);
        const float al = __ldg(a.alpha + t * a.H + h), bt = __ldg(a.beta + t * a.H + h);
        good = good && al > 0.0f && al <= 1.0f;
        float2 u = make_float2(0.f, 0.f), o = u;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            S[r] = mul2(S[r], make_float2(al, al));
            u = fma2(make_float2(k[r], k[r]), S[r], u);
        }
        u = sum(u);
        u = make_float2(bt * (v[0] - u.x), bt * (v[1] - u.y));
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            S[r] = fma2(make_float2(k[r], k[r]), u, S[r]);
            o = fma2(make_float2(q[r], q[r]), S[r], o);
        }
        o = sum(o);
        if (lane < 4) {
            T *dst = static_cast<T *>(a.o) + t * a.os + h * D + col0;
            *reinterpret_cast<typename Pair<T>::type *>(dst) = typename Pair<T>::type(from_f32<T>(o.x), from_f32<T>(o.y));
        }
    }
    if (!good) atomicOr(a.err, kErrGateRange);
    if (count > 0 || fresh)
#pragma unroll
        for (int r = 0; r < 16; ++r) *reinterpret_cast<float2 *>(Sg + (size_t)r * D) = S[r];
}

template <class T>
__global__ void __launch_bounds__(NT, 1) k_delta_chunk(DeltaArgs a) {
    extern __shared__ __align__(1024) uint8_t raw[];
    using Sm = Smem<T>;
    using T2 = typename Pair<T>::type;
    constexpr bool TWO = Sm::AT == 2;
    Sm &sm = *reinterpret_cast<Sm *>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int s = blockIdx.x / a.H, h = blockIdx.x % a.H, hk = h / (a.H / a.Hk);
    int first, count;
    if (!delta_range(a, s, first, count)) return;
    float *Sg = delta_state(a, s, h, D, kErrBadSlot);
    if (!Sg) return;
    const bool fresh = a.fresh && a.fresh[s];
    if (count <= kShort) {
        short_sequence<T>(a, Sg, fresh, first, count, h, hk);
        return;
    }
    const int chunks = (count + C - 1) / C;

    if (tid == 0) {
        for (int b = 0; b < 2; ++b) {
            mbar_init_n(&sm.full[b], NP);
            mbar_init_n(&sm.vfull[b], NP);
            mbar_init_n(&sm.ready[b], NP);
            mbar_init_n(&sm.empty[b], NS);
            mbar_init_n(&sm.uput[b], NS);
            mbar_init_n(&sm.z[b], 1);
            mbar_init_n(&sm.g[b], 1);
        }
        for (uint64_t *b : {&sm.sput, &sm.rput}) mbar_init_n(b, NS);
        mbar_init_n(&sm.out, NP);
        for (uint64_t *b : {&sm.w, &sm.u, &sm.d, &sm.drain[0], &sm.drain[1], &sm.drain[2]}) mbar_init_n(b, 1);
        fence_mbar_init();
    }
    if (warp == 0) tc::alloc(&sm.taddr, 512);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tm = sm.taddr;
    bool ok = true;

    if (warp < NS / 32) {
        // ---- state ----
        asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
        const int hh = warp >> 2, j = 32 * (warp & 3) + lane;   // key rows [64 hh, 64 hh + 64), value column
        const uint32_t quad = tm + ((uint32_t)(32 * (warp & 3)) << 16);
        float2 S[32];
        T2 v[16];
        float sS, smax = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            S[i].x = fresh ? 0.0f : Sg[(size_t)(64 * hh + 2 * i) * D + j];
            S[i].y = fresh ? 0.0f : Sg[(size_t)(64 * hh + 2 * i + 1) * D + j];
            smax = max_nan(smax, max_nan(fabsf(S[i].x), fabsf(S[i].y)));
        }
        sm.smx[hh][j] = smax;
        tc16::group_and(1, NS, true);
        // what the column has taken in so far are numbers: if u' is none, it has left the range of its operands
        bool finite = sm.smx[0][j] <= kFloatMax && sm.smx[1][j] <= kFloatMax;
        // S as operand of chunk c, and the chunk's V into registers
        auto put = [&](int c, float bound) {
            const int b = c & 1;
            float inv;
            scale_for(bound, kTopS, sS, inv);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) tc16::split2(mul2(S[16 * p + i], both(inv)), hi[i], lo[i]);
                tc16::st16(quad + TSH + 32 * hh + 16 * p, hi);
                tc16::st16(quad + TSL + 32 * hh + 16 * p, lo);
            }
            ok = warp_wait(&sm.full[b], (c >> 1) & 1) && warp_wait(&sm.vfull[b], (c >> 1) & 1) && ok;
            const T *src = sm.v[b] + 32 * hh * D + j;
            T2 m = __habs2(T2(src[0], src[D]));
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                v[i] = T2(src[2 * i * D], src[(2 * i + 1) * D]);
                m = __hmax2_nan(m, __habs2(v[i]));
            }
            const float2 mf = to_f32x2(m);
            sm.vmx[hh][j] = max_nan(mf.x, mf.y);
            tc16::st_wait();
            tc::fence_before();
            mbar_arrive(&sm.sput);
        };
        // The products, by warp 0 once every thread's operands are in place: one elected lane, operands from values that the
        // compiler knows to be the same in all lanes (otherwise each of them is moved to the uniform registers by itself, 110
        // cycles an instruction).  A descriptor's address field counts 16 bytes.
        const uint32_t tmu = __shfl_sync(0xffffffffu, tm, 0);
        const uint64_t dk = tc16::kmajor(tc::smem_addr(sm.kq)), dx = tc16::kmajor(tc::smem_addr(sm.x)),
                       da = tc16::kmajor(tc::smem_addr(sm.a)), dn = tc16::desc(tc::smem_addr(sm.kq), kHalf, 1024);
        constexpr uint32_t id = tc16::idesc(128, C, false), id_mn = tc16::idesc(128, D, true);
        auto issue_w = [&](int b, uint32_t ph, uint32_t ph2) {    // W^T = S^T K'^T
            if (!warp_wait(&sm.sput, ph) || !warp_wait(&sm.full[b], ph2)) return false;
            tc::fence_after();
            const uint64_t kq = dk + b * (2 * kHalf >> 4);
            if (tc16::elect()) {
#pragma unroll
                for (int m = 0; m < 16; ++m)
                    tc16::mma_ts(tmu + TW, tmu + (m < 8 ? TSH : TSL) + 8 * (m & 7), kq + ((((m >> 2) & 1) * kHalf + (m & 3) * 32) >> 4), id, m);
                tc::commit(&sm.w);
            }
            __syncwarp();
            return true;
        };
        auto issue_yu = [&](int b, uint32_t ph, uint32_t ph2, bool fresh_y) {
            // Y^T = S^T Q'^T, where the last chunk's output has been read
            if (!fresh_y && !warp_wait(&sm.out, ph ^ 1)) return false;
            tc::fence_after();
            const uint64_t q = dk + ((b * 2 * kHalf + C * 128) >> 4), xb = dx + b * (2 * C * 128 >> 4);
            if (tc16::elect()) {
#pragma unroll
                for (int m = 0; m < 8 * Sm::AT; ++m)
                    tc16::mma_ts(tmu + TY, tmu + (m < 8 ? TSH : TSL) + 8 * (m & 7), q + ((((m >> 2) & 1) * kHalf + (m & 3) * 32) >> 4), id, m);
            }
            __syncwarp();
            // U'^T = R^T X^T
            if (!warp_wait(&sm.rput, ph) || !warp_wait(&sm.ready[b], ph2)) return false;
            tc::fence_after();
            if (tc16::elect()) {
#pragma unroll
                for (int m = 0; m < 12; ++m)
                    tc16::mma_ts(tmu + TU, tmu + (m < 8 ? TRH : TRL) + 8 * (m & 3),
                                 xb + (((m >= 4 && m < 8 ? C * 128 : 0) + (m & 3) * 32) >> 4), id, m);
                tc::commit(&sm.u);
            }
            __syncwarp();
            return true;
        };
        auto issue_dz = [&](int b, uint32_t ph2) {
            if (!warp_wait(&sm.uput[b], ph2)) return false;
            tc::fence_after();
            const uint64_t kn = dn + b * (2 * kHalf >> 4), ab = da + b * (Sm::AT * C * 128 >> 4);
            if (tc16::elect()) {
                // the increment of S^T: K's rows along the summed index
#pragma unroll
                for (int m = 0; m < 8; ++m)
                    tc16::mma_ts(tmu + TD, tmu + (m < 4 ? TFH : TFL) + 8 * (m & 3), kn + ((m & 3) * 2048 >> 4), id_mn, m);
                tc::commit(&sm.d);
                // (A U')^T
#pragma unroll
                for (int m = 0; m < (TWO ? 12 : 4); ++m)
                    tc16::mma_ts(tmu + TU, tmu + (m >= 4 && m < 8 ? TUL : TUH) + 8 * (m & 3),
                                 ab + (((m >= 8 ? C * 128 : 0) + (m & 3) * 32) >> 4), id, m);
                tc::commit(&sm.z[b]);
            }
            __syncwarp();
            return true;
        };
        float bound = fmaxf(sm.smx[0][j], sm.smx[1][j]);
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            const int b = __shfl_sync(0xffffffffu, c & 1, 0);
            const uint32_t ph = b, ph2 = (c >> 1) & 1;
            put(c, bound);
            if (warp == 0) ok = issue_w(b, ph, ph2) && ok;
            // R from W^T and V
            ok = ok && warp_wait(&sm.sput, ph) && warp_wait(&sm.w, ph);
            if (!ok) break;
            tc::fence_after();
            float sR;
            const float before = fmaxf(sm.smx[0][j], sm.smx[1][j]);
            finite = finite && sm.finite[b] && sm.vmx[0][j] <= kFloatMax && sm.vmx[1][j] <= kFloatMax;
            {
                uint32_t w[32], hi[16], lo[16];
                tc::ld32(quad + TW + 32 * hh, w);
                float iR;
                // |S^T k'| <= 128 * 2 * max |S|
                scale_for(sm.mb[b] * fmaf(sm.mg[b] * 256.0f, before, fmaxf(sm.vmx[0][j], sm.vmx[1][j])), kTopR, sR, iR);
                if (hh == 0) {
                    sm.ss[b][j] = sS;
                    sm.sr[b][j] = sR;
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 g = *reinterpret_cast<const float2 *>(&sm.gk[b][32 * hh + 2 * i]);
                    const float2 bt = *reinterpret_cast<const float2 *>(&sm.bk[b][32 * hh + 2 * i]);
                    const float2 y = fma2(g, mul2(pair_of(w, i), both(-sS)), to_f32x2(v[i]));
                    tc16::split2(mul2(y, mul2(bt, both(iR))), hi[i], lo[i]);
                }
                tc16::st16(quad + TRH + 16 * hh, hi);
                tc16::st16(quad + TRL + 16 * hh, lo);
                tc16::st_wait();
            }
            tc::fence_before();
            mbar_arrive(&sm.rput);
            if (warp == 0) ok = issue_yu(b, ph, ph2, c == 0) && ok;
            // U' and diag(gamma_C / gamma) U'
            ok = ok && warp_wait(&sm.u, ph);
            if (!ok) break;
            tc::fence_after();
            float um = 0.0f;
            {
                uint32_t u[32], hi[16], lo[16];
                tc::ld32(quad + TU + 32 * hh, u);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 x = pair_of(u, i);
                    um = max_nan(um, max_nan(fabsf(x.x), fabsf(x.y)));
                    tc16::split2(mul2(x, *reinterpret_cast<const float2 *>(&sm.f[b][32 * hh + 2 * i])), hi[i], lo[i]);
                }
                tc16::st16(quad + TFH + 16 * hh, hi);
                tc16::st16(quad + TFL + 16 * hh, lo);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    if constexpr (TWO) tc16::split2(pair_of(u, i), hi[i], lo[i]);
                    else hi[i] = tc16::pack2(pair_of(u, i));
                }
                tc16::st16(quad + TUH + 16 * hh, hi);
                if constexpr (TWO) tc16::st16(quad + TUL + 16 * hh, lo);
                sm.umx[hh][j] = um;
                if (finite && !(um <= kHalfMax)) atomicOr(a.err, kErrRange);
                tc16::st_wait();
            }
            tc::fence_before();
            mbar_arrive(&sm.uput[b]);
            if (warp == 0) ok = issue_dz(b, ph2) && ok;
            // S
            ok = ok && warp_wait(&sm.uput[b], ph2) && warp_wait(&sm.d, ph);
            if (!ok) break;
            tc::fence_after();
            const float last = sm.gl[b];
            um = fmaxf(sm.umx[0][j], sm.umx[1][j]);
            float m0 = 0.0f, m1 = 0.0f;
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                uint32_t x[32];
                tc::ld32(quad + TD + 64 * hh + 32 * p, x);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float2 &y = S[16 * p + i];
                    y = fma2(pair_of(x, i), both(sR), mul2(y, both(last)));
                    m0 = fmaxf(m0, fabsf(y.x));
                    m1 = fmaxf(m1, fabsf(y.y));
                }
            }
            sm.smx[hh][j] = fmaxf(m0, m1);
            mbar_arrive(&sm.empty[b]);
            // U' as an operand stands where S goes
            ok = warp_wait(&sm.z[b], ph2);
            if (!ok) break;
            bound = fmaf(last, before, 128.0f * sR * um);   // |K'^T u'| <= 64 * 2 * max |u'|
        }
        if (ok) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                Sg[(size_t)(64 * hh + 2 * i) * D + j] = S[i].x;
                Sg[(size_t)(64 * hh + 2 * i + 1) * D + j] = S[i].y;
            }
        }
    } else {
        // ---- prepare ----
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        const int gp = (warp - NS / 32) >> 2, p = tid - NS - gp * NP, pw = p >> 5;   // group, thread and warp of the group
        const int bar = 2 + gp, b = gp;                                              // a group's chunks use its buffers
        const uint32_t quad = tm + ((uint32_t)(32 * pw) << 16);
        const int r0 = p >> 4, i8 = p & 15;                                          // 16 lanes to a row: rows r0 + 8 i
        const T *gq = static_cast<const T *>(a.q) + (size_t)hk * D, *gk = static_cast<const T *>(a.k) + (size_t)hk * D;
        const T *gv = static_cast<const T *>(a.v) + (size_t)h * D;
        float *const n = sm.n[gp], *const ks = sm.ks[gp], *const be = sm.be[gp], *const gate = sm.al[gp], *const up = sm.up[gp], *const down = sm.down[gp];
        bool gates_ok = true;
        // warp 3: a chunk's gates, two tokens a lane, 16 lanes a half: gamma and gamma_C / gamma, products of the gates up to
        // and after a token
        float al[2] = {1.0f, 1.0f}, bt[2] = {0.0f, 0.0f}, total = 1.0f;
        float2 gam, fin;
        auto load_gates = [&](int c) {
            if (pw == 3) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int t = c * C + 2 * lane + e;
                    al[e] = t < count ? __ldg(a.alpha + (size_t)(first + t) * a.H + h) : 1.0f;
                    bt[e] = t < count ? __ldg(a.beta + (size_t)(first + t) * a.H + h) : 0.0f;
                }
            }
        };
        auto running = [&]() {
            gates_ok = gates_ok && al[0] > 0.0f && al[0] <= 1.0f && al[1] > 0.0f && al[1] <= 1.0f;
            float p = al[0] * al[1], q = p;
#pragma unroll
            for (int m = 1; m < 16; m <<= 1) {
                const float y = __shfl_up_sync(0xffffffffu, p, m, 16), z = __shfl_down_sync(0xffffffffu, q, m, 16);
                if ((lane & 15) >= m) p *= y;
                if ((lane & 15) + m < 16) q *= z;
            }
            float before = __shfl_up_sync(0xffffffffu, p, 1, 16), after = __shfl_down_sync(0xffffffffu, q, 1, 16);
            if ((lane & 15) == 0) before = 1.0f;
            if ((lane & 15) == 15) after = 1.0f;
            const float h0 = __shfl_sync(0xffffffffu, p, 15), h1 = __shfl_sync(0xffffffffu, p, 31);
            const float2 u = make_float2(before * al[0], p), w = make_float2(al[1] * after, after);
            total = h0 * h1;
            gam = lane < 16 ? u : mul2(u, both(h0));
            fin = lane < 16 ? mul2(w, both(h1)) : w;
            // the group is done with its last chunk's
            *reinterpret_cast<float2 *>(&gate[2 * lane]) = make_float2(al[0], al[1]);
            *reinterpret_cast<float2 *>(&up[2 * lane]) = u;
            *reinterpret_cast<float2 *>(&down[2 * lane]) = w;
        };
        // K and Q rows as they are into their operand places (16-bit types all), zeros behind the last token; 64 rows keep
        // a row's place in its group of eight
        const uint32_t at0 = (i8 >> 3) * kHalf + tc16::sw_off(r0, (i8 & 7) * 8);
        auto load_kq = [&](int c) {
            const int cc = min(C, count - c * C);
            const T *k = gk + (size_t)(first + c * C + r0) * a.ks + i8 * 8, *q = gq + (size_t)(first + c * C + r0) * a.qs + i8 * 8;
            uint8_t *dst = sm.kq[b] + at0;
#pragma unroll 2
            for (int i = 0; i < 8; ++i) {
                const bool in = r0 + 8 * i < cc;
                copy16(dst, in ? k : gk, in);
                copy16(dst + C * 128, in ? q : gq, in);
                dst += 8 * 128;
                k += 8 * a.ks;
                q += 8 * a.qs;
            }
            cp_async_commit();
        };
        auto load_v = [&](int c) {
            const int cc = min(C, count - c * C);
            const T *v = gv + (size_t)(first + c * C + r0) * a.vs + i8 * 8;
            T *dst = sm.v[b] + r0 * D + i8 * 8;
#pragma unroll 2
            for (int i = 0; i < 8; ++i) {
                const bool in = r0 + 8 * i < cc;
                copy16(dst + 8 * i * D, in ? v : gv, in);
                v += 8 * a.vs;
            }
            // arrives when this thread's copies have landed
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tc::smem_addr(&sm.vfull[b])) : "memory");
        };
        load_gates(gp);
#pragma unroll 1
        for (int c = gp; c < chunks + 2; c += 2) {
            const int done = c - 2;              // the group's last chunk, whose output comes before the next one's loads
            const bool more = c < chunks;
            const uint32_t ph2 = (c >> 1) & 1;
            if (pw == 3 && more) running();
            if (done >= 0) {
                // its last product is done: K, Q, X, A have been read, Y^T and (A U')^T are there
                ok = warp_wait(&sm.uput[b], ph2 ^ 1) && warp_wait(&sm.z[b], ph2 ^ 1);
                tc::fence_after();
            }
            if (ok && more) load_kq(c);
            if (done >= 0) {
                const int cc = min(C, count - done * C);
                // O to rows of V's buffer, and from there to global memory
                {
                    const int j = 32 * pw + lane;
                    const float sS = sm.ss[b][j], sR = sm.sr[b][j];
#pragma unroll 1
                    for (int t0 = 0; t0 < C; t0 += 16) {
                        float4 g[4], q[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            g[i] = *reinterpret_cast<const float4 *>(&sm.go[b][t0 + 4 * i]);
                            q[i] = *reinterpret_cast<const float4 *>(&sm.qs[b][t0 + 4 * i]);
                        }
                        uint32_t y[16], z[16];
                        tc16::ld16x2(quad + TY + t0, y, quad + TU + t0, z);
                        if (t0 + 16 == C) {
                            tc::fence_before();
                            mbar_arrive(&sm.out);
                        }
                        T *dst = sm.v[b] + t0 * D + j;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 g4 = g[i / 2], q4 = q[i / 2];
                            const float2 g2 = i & 1 ? make_float2(g4.z, g4.w) : make_float2(g4.x, g4.y);
                            const float2 q2 = i & 1 ? make_float2(q4.z, q4.w) : make_float2(q4.x, q4.y);
                            const float2 o = fma2(g2, mul2(pair_of(y, i), both(sS)), mul2(q2, mul2(pair_of(z, i), both(sR))));
                            dst[2 * i * D] = from_f32<T>(o.x);
                            dst[(2 * i + 1) * D] = from_f32<T>(o.y);
                        }
                    }
                }
                ok = tc16::group_and(bar, NP, ok);
                if (!ok) break;
                {
                    T *dst = static_cast<T *>(a.o) + (size_t)(first + done * C) * a.os + h * D + i8 * 8;
                    uint4 y[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = *reinterpret_cast<const uint4 *>(sm.v[b] + (r0 + 8 * i) * D + i8 * 8);
                    dst += r0 * a.os;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (r0 + 8 * i < cc) *reinterpret_cast<uint4 *>(dst) = y[i];
                        dst += 8 * a.os;
                    }
                }
            }
            if (!more) break;
            load_v(c);                           // a thread's copies of V go where it alone has read the output
            // this thread's own copies: rows scaled to a largest value in [1, 2), as fp16
            asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll 1
            for (int i0 = 0; i0 < 8; i0 += 4) {   // pieces of four rows r0 + 8 i of K and of Q at a time
                uint8_t *at = sm.kq[b] + at0 + i0 * 8 * 128;
                uint4 rw[8];
                T2 m[4];
#pragma unroll
                for (int i = 0; i < 8; ++i) rw[i] = *reinterpret_cast<const uint4 *>(at + (i & 1) * C * 128 + (i >> 1) * 8 * 128);
                auto most = [](const uint4 &x) {
                    const T2 *pr = reinterpret_cast<const T2 *>(&x);
                    return __hmax2_nan(__hmax2_nan(__habs2(pr[0]), __habs2(pr[1])), __hmax2_nan(__habs2(pr[2]), __habs2(pr[3])));
                };
#pragma unroll
                for (int i = 0; i < 4; ++i) {     // (of K, of Q)
                    const T2 k = most(rw[2 * i]), q = most(rw[2 * i + 1]);
                    m[i] = __hmax2_nan(lows(k, q), highs(k, q));
                }
#pragma unroll
                for (int w = 8; w > 0; w >>= 1)
#pragma unroll
                    for (int i = 0; i < 4; ++i) m[i] = __hmax2_nan(m[i], __shfl_xor_sync(0xffffffffu, m[i], w));
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const T2 *pr = reinterpret_cast<const T2 *>(&rw[i]);
                    const float2 mf = to_f32x2(m[i >> 1]);
                    const int e = exponent_of(i & 1 ? mf.y : mf.x);
                    const float2 inv = both(__uint_as_float((uint32_t)(254 - e) << 23));
                    uint4 out;
                    out.x = tc16::pack2(mul2(to_f32x2(pr[0]), inv));
                    out.y = tc16::pack2(mul2(to_f32x2(pr[1]), inv));
                    out.z = tc16::pack2(mul2(to_f32x2(pr[2]), inv));
                    out.w = tc16::pack2(mul2(to_f32x2(pr[3]), inv));
                    *reinterpret_cast<uint4 *>(at + (i & 1) * C * 128 + (i >> 1) * 8 * 128) = out;
                    // (a key that is not finite has the scale NaN)
                    if (i8 == 0)
                        (i & 1 ? sm.qs[b] : ks)[r0 + 8 * (i0 + (i >> 1))] =
                            __uint_as_float(i & 1 || mf.x <= kFloatMax ? (uint32_t)e << 23 : 0x7fffffffu);
                }
            }
            tc::fence_smem_to_async();
            ok = tc::mbar_wait(&sm.empty[b], ph2 ^ 1, kPolls);   // the state is done with the last chunk's gates
            ok = tc16::group_and(bar, NP, ok);
            if (!ok) break;
            if (pw == 0) {   // [K; Q] K^T
                const uint64_t kq = tc16::kmajor(tc::smem_addr(sm.kq)) + __shfl_sync(0xffffffffu, b, 0) * (2 * kHalf >> 4);
                const uint32_t dst = __shfl_sync(0xffffffffu, tm + TG + C * gp, 0);
                tc::fence_after();
                if (tc16::elect()) {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {
                        const uint64_t at = kq + (((kk >> 2) * kHalf + (kk & 3) * 32) >> 4);
                        tc16::mma_ss(dst, at, at, tc16::idesc(128, C, false), kk);
                    }
                    tc::commit(&sm.g[gp]);
                }
                __syncwarp();
            }
            if (pw == 3) {   // the token's factors
                const float2 bb = make_float2(bt[0], bt[1]);
                const float2 kk = *reinterpret_cast<const float2 *>(&ks[2 * lane]);
                const float2 qq = *reinterpret_cast<const float2 *>(&sm.qs[b][2 * lane]);
                const float2 gkk = mul2(gam, kk), bkk = mul2(bb, kk);
                *reinterpret_cast<float2 *>(&be[2 * lane]) = mul2(bkk, kk);
                *reinterpret_cast<float2 *>(&sm.gk[b][2 * lane]) = gkk;
                *reinterpret_cast<float2 *>(&sm.bk[b][2 * lane]) = bkk;
                *reinterpret_cast<float2 *>(&sm.f[b][2 * lane]) = fin;
                *reinterpret_cast<float2 *>(&sm.go[b][2 * lane]) = mul2(gam, qq);
                float mb = fmaxf(fabsf(bkk.x), fabsf(bkk.y)), mg = fmaxf(fabsf(gkk.x), fabsf(gkk.y));
#pragma unroll
                for (int w = 16; w > 0; w >>= 1) {
                    mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, w));
                    mg = fmaxf(mg, __shfl_xor_sync(0xffffffffu, mg, w));
                }
                const bool numbers = __all_sync(0xffffffffu, gates_ok && kk.x == kk.x && kk.y == kk.y);
                if (lane == 0) {
                    sm.finite[b] = numbers;
                    sm.gl[b] = total;
                    sm.mb[b] = mb;
                    sm.mg[b] = mg;
                }
            }
            mbar_arrive(&sm.full[b]);
            if (c + 2 < chunks) {   // the next chunk's gates into registers, its rows into L2
                load_gates(c + 2);
                const int t = (c + 2) * C + (p >> 1), half = (p & 1) * (D / 2);
                if (t < count) {
                    const size_t tok = (size_t)(first + t);
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(gk + tok * a.ks + half) : "memory");
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(gq + tok * a.qs + half) : "memory");
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(gv + tok * a.vs + half) : "memory");
                }
            }
            ok = warp_wait(&sm.full[b], ph2) && warp_wait(&sm.g[gp], ph2);
            tc::fence_after();
            // A row of Gamma o [K; Q] K^T a lane.  Right of the diagonal: N is not read there, A is 0.  Gamma_ts is the product of
            // the gates between, column after column to the left of the diagonal (at most 32 roundings, whatever gates came
            // before; the difference of logarithms of gamma loses what a run of strong gates adds to both); over the
            // middle of the chunk, up_t down_s, each at most 1.
            {
                const int t = (32 * pw + lane) & 63;
                const bool is_n = pw < 2;
                const float row = is_n ? be[t] : 1.0f;
#pragma unroll 1
                for (int s0 = 0; s0 < C; s0 += 32) {
                    if (s0 > 0 && !(pw & 1)) {     // right of the diagonal for every row of the warp
                        if (!is_n) {
#pragma unroll
                            for (int e = 0; e < 32; e += 8)
#pragma unroll
                                for (int m = 0; m < Sm::AT; ++m)
                                    *reinterpret_cast<uint4 *>(sm.a[b] + m * C * 128 + tc16::sw_off(t, s0 + e)) = make_uint4(0, 0, 0, 0);
                        }
                        continue;
                    }
                    uint32_t g[32];
                    tc::ld32(quad + TG + C * gp + s0, g);
                    float2 x[16];
                    if (s0 == 0 && (pw & 1)) {     // the first half for every row of the second
                        const float2 far = both(row * up[t]);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            x[i] = mul2(mul2(far, *reinterpret_cast<const float2 *>(&down[2 * i])), pair_of(g, i));
                    } else {
                        float y = row;
#pragma unroll
                        for (int i = 15; i >= 0; --i) {
                            const float2 a2 = *reinterpret_cast<const float2 *>(&gate[s0 + 2 * i]);
                            float2 w = make_float2(0.0f, 0.0f);
                            if (s0 + 2 * i + 1 <= t) {
                                w.y = y;
                                y *= a2.y;
                            }
                            if (s0 + 2 * i <= t) {
                                w.x = y;
                                y *= a2.x;
                            }
                            x[i] = mul2(w, pair_of(g, i));
                        }
                    }
                    if (is_n) {
#pragma unroll
                        for (int i = 0; i < 16; i += 2)
                            *reinterpret_cast<float4 *>(&n[t * SN + s0 + 2 * i]) = make_float4(x[i].x, x[i].y, x[i + 1].x, x[i + 1].y);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t hi[4], lo[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if constexpr (TWO) tc16::split2(x[4 * e + i], hi[i], lo[i]);
                                else hi[i] = tc16::pack2(x[4 * e + i]);
                            }
                            uint8_t *dst = sm.a[b] + tc16::sw_off(t, s0 + 8 * e);
                            *reinterpret_cast<uint4 *>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                            if constexpr (TWO) *reinterpret_cast<uint4 *>(dst + C * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                        }
                    }
                }
            }
            tc::fence_before();
            ok = tc16::group_and(bar, NP, ok);
            if (!ok) break;
            // (I + N)^-1 in place: the diagonal blocks of 16 by substitution, a warp a block, a column a lane
            {
                const int d0 = 16 * pw, col = lane & 15;
                float x[16];
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    float y0 = r == col ? 1.0f : 0.0f, y1 = 0.0f;
#pragma unroll
                    for (int m = 0; m + 1 < r; m += 2) {
                        const float2 nn = *reinterpret_cast<const float2 *>(&n[(d0 + r) * SN + d0 + m]);
                        y0 = fmaf(-nn.x, x[m], y0);
                        y1 = fmaf(-nn.y, x[m + 1], y1);
                    }
                    if (r & 1) y0 = fmaf(-n[(d0 + r) * SN + d0 + r - 1], x[r - 1], y0);
                    x[r] = y0 + y1;
                }
                __syncwarp();
                if (lane < 16) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) n[(d0 + r) * SN + d0 + col] = x[r];
                }
            }
            tc16::group_and(bar, NP, true);
            // pairs of blocks of M rows at u0 (upper) and u0 + M (lower): the block below the diagonal becomes
            // -X_lower (N X_upper), the product in brackets in the unused top right quarter; a warp does 16 x 8 TILES of it,
            // operands as two fp16 terms, three products
            auto join = [&](auto m_, auto tiles_, int u0, int row, int col) {
                constexpr int M = decltype(m_)::value, TILES = decltype(tiles_)::value;
                const int g = lane >> 2, q = 2 * (lane & 3);
                auto product = [&](const float *l, const float *r, float *out, float sign) {
                    float acc[TILES][4];
#pragma unroll
                    for (int y = 0; y < TILES; ++y) acc[y][0] = acc[y][1] = acc[y][2] = acc[y][3] = 0.0f;
#pragma unroll
                    for (int k = 0; k < M; k += 16) {
                        uint32_t ah[4], al_[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            tc16::split2(*reinterpret_cast<const float2 *>(l + (row + g + 8 * (i & 1)) * SN + k + q + 8 * (i >> 1)), ah[i], al_[i]);
#pragma unroll
                        for (int y = 0; y < TILES; ++y) {
                            uint32_t bh[2], bl[2];
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const float *x = r + (k + q + 8 * i) * SN + col + 8 * y + g;
                                tc16::split2(make_float2(x[0], x[SN]), bh[i], bl[i]);
                            }
                            tc16::mma_sync(acc[y], ah, bh);
                            tc16::mma_sync(acc[y], ah, bl);
                            tc16::mma_sync(acc[y], al_, bh);
                        }
                    }
#pragma unroll
                    for (int y = 0; y < TILES; ++y) {
                        float *o = out + (row + g) * SN + col + 8 * y + q;
                        *reinterpret_cast<float2 *>(o) = make_float2(sign * acc[y][0], sign * acc[y][1]);
                        *reinterpret_cast<float2 *>(o + 8 * SN) = make_float2(sign * acc[y][2], sign * acc[y][3]);
                    }
                    tc16::group_and(bar, NP, true);
                };
                float *below = n + (u0 + M) * SN + u0, *right = n + u0 / 2 * SN + C / 2;
                product(below, n + u0 * SN + u0, right, 1.0f);
                product(n + (u0 + M) * SN + u0 + M, right, below, -1.0f);
            };
            join(std::integral_constant<int, 16>(), std::integral_constant<int, 1>(), pw & 2 ? 32 : 0, 0, 8 * (pw & 1));
            join(std::integral_constant<int, 32>(), std::integral_constant<int, 2>(), 0, 16 * (pw >> 1), 16 * (pw & 1));
            {   // X as operand, zeros right of the diagonal
                const int t = p & 63, s0 = 32 * (p >> 6);
                float4 y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = *reinterpret_cast<const float4 *>(&n[t * SN + s0 + 4 * i]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 y4 = y[2 * e + i / 2];
                        float2 x = i & 1 ? make_float2(y4.z, y4.w) : make_float2(y4.x, y4.y);
                        const int ss = s0 + 8 * e + 2 * i;
                        if (ss > t) x.x = 0.0f;
                        if (ss + 1 > t) x.y = 0.0f;
                        tc16::split2(x, hi[i], lo[i]);
                    }
                    uint8_t *dst = sm.x[b] + tc16::sw_off(t, s0 + 8 * e);
                    *reinterpret_cast<uint4 *>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(dst + C * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
            tc::fence_smem_to_async();
            mbar_arrive(&sm.ready[b]);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (!gates_ok) atomicOr(a.err, kErrGateRange);
    }
    // A product may still be in flight only after a wait gave up: let it end (bounded) before its memory is given
    // back.  A commit covers what its own thread has issued.
    if (!__syncthreads_and(ok) && (warp & 3) == 0 && (warp == 0 || warp >= NS / 32) && tc16::elect()) {
        if (warp == 0) atomicOr(a.err, kErrWait);
        uint64_t *bar = &sm.drain[warp == 0 ? 0 : warp == NS / 32 ? 1 : 2];
        tc::commit(bar);
        if (!tc::mbar_wait(bar, 0, kPolls)) atomicOr(a.err, kErrTmemDrain);
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 0) tc::dealloc(tm, 512);
}

template <class T>
cudaError_t launch(const DeltaArgs &a, cudaStream_t st) {
    static_assert(NT / 32 * 8 == D, "a warp to every eight value columns");
    static_assert(sizeof(Smem<T>) <= 227 * 1024, "shared memory of a block");
    const long long blocks = (long long)a.n_seq * a.H;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    auto *kern = k_delta_chunk<T>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem<T>));
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)blocks, NT, sizeof(Smem<T>), st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_chunk(int dtype, const DeltaArgs &a, cudaStream_t st) {
    return dtype == 2 ? launch<__nv_bfloat16>(a, st) : launch<__half>(a, st);
}

}  // namespace stepq
