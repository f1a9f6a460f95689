// The gated delta rule over a ragged batch in chunks of 64 tokens on the fifth-generation tensor
// cores: d = 128, per-head gates, bfloat16 or fp16 tokens, fp32 states.
//
// With gamma_t the running product of the gates in a chunk, Gamma_ts = gamma_t / gamma_s and
// S_0 the state before it:
//   N_ts = beta_t Gamma_ts k_t.k_s (s < t),  T = (I + N)^-1 diag(beta)
//   U = T (V - diag(gamma) K S_0)
//   O = diag(gamma) Q S_0 + A U,  A_ts = Gamma_ts q_t.k_s (s <= t)
//   S_C = gamma_C S_0 + K^T diag(gamma_C / gamma) U
// Every Gamma is at most 1, so nothing overflows however fast a gate decays.
//
// One block per (sequence, head) walks the chunks; blocks of heads that share k and q are neighbours.  The
// chain S_0 -> U -> S_C is serial, so the block is split by what it waits for:
//   warps 0-7  (state)  thread = value column j and half of the key rows: S in 64 registers, fp32.
//   warps 8-11 (prepare) the next chunk: loads, gates, K K^T and Q K^T, the triangular inverse, A.
// All products are tcgen05 with the value columns j in the lanes (W^T = S^T K^T and so on), so what
// one product leaves in a thread's lane is what the thread feeds to the next one.
//
// Precision: bfloat16 tokens are exact operands; fp32 operands (S, U, T, V - gamma K S) enter as the sum of
// two bfloat16 values (2^-18 of the value is left out), accumulators are fp32.  The readout uses the leading term
// alone for bfloat16 outputs (2^-9 of a term, as the output's own rounding) and both for fp16.  fp16 tokens are the
// sum of two bfloat16 values exactly.
//
// Tensor memory: S^T terms 0-127 (hi, lo, two values a column), W^T | Y^T 128-255 and later the state's
// increment, the right side's terms 256-319 and later U's, U^T 320-383 and later A U, (U f)^T terms 384-447,
// [K; Q] K^T 448-511.  All 512 columns, one block per SM.
//
// Every wait is bounded: a wait that gives up sets kErrWait, its group leaves the loop together, and the other
// group's waits run out in turn.
#include <type_traits>

#include "stepq_dev.cuh"
#include "stepq_delta.cuh"
#include "stepq_prefill.cuh"
#include "stepq_tc16.cuh"

namespace stepq {

namespace {

constexpr int D = 128, C = 64, NS = 256, NP = 128, NT = NS + NP;
constexpr uint32_t kPolls = 1u << 22;
constexpr uint32_t TSH = 0, TSL = 64, TWY = 128, TR = 256, TU = 320, TF = 384, TG = 448;
constexpr uint32_t kHalf = 128 * 128;   // bytes of 64 columns of [K; Q]
constexpr uint32_t kTerm = 2 * kHalf;   // bytes of one term of [K; Q]
constexpr int SN = C + 4;               // row stride of the fp32 scratch matrices

// KT: bfloat16 terms of a token value (1: bfloat16 tokens, 2: fp16 tokens).  VB: buffers of V.
template <int KT>
struct Smem {
    static constexpr int VB = 3 - KT;
    alignas(1024) uint8_t kq[2][KT * kTerm];   // [buffer][term][column half][K rows, Q rows][128 bytes]
    alignas(1024) uint8_t t[2][2 * C * 128];   // T, two terms
    alignas(1024) uint8_t a[2][KT * C * 128];  // A, KT terms
    alignas(16) uint16_t v[VB][C * D];
    alignas(16) float n[C * SN];               // N, its inverse in place
    alignas(16) float gam[2][C], f[2][C];
    alignas(16) float lg[C], beta[C];
    alignas(8) uint64_t full[2], ready[2], empty[2], v_free, wy, u, d, z, g, drain[2];
    uint32_t taddr;
};

__device__ __forceinline__ void mbar_init_n(uint64_t *bar, uint32_t n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(tc::smem_addr(bar)), "r"(n) : "memory");
}

// 16 bytes of global memory into shared memory, or zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool take) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}

template <int KT, class T>
__global__ void __launch_bounds__(NT, 1) k_delta_chunk(DeltaArgs a) {
    extern __shared__ __align__(1024) uint8_t raw[];
    using Sm = Smem<KT>;
    Sm &sm = *reinterpret_cast<Sm *>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int s = blockIdx.x / a.H, h = blockIdx.x % a.H, hk = h / (a.H / a.Hk);
    int first, count;
    if (!delta_range(a, s, first, count)) return;
    float *Sg = delta_state(a, s, h, D, kErrBadSlot);
    if (!Sg) return;
    const bool fresh = a.fresh && a.fresh[s];
    if (count == 0) {
        if (fresh)
            for (int e = tid; e < D * D / 4; e += NT) reinterpret_cast<float4 *>(Sg)[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        return;
    }
    const int chunks = (count + C - 1) / C;

    if (tid == 0) {
        for (int b = 0; b < 2; ++b) {
            mbar_init_n(&sm.full[b], NP);
            mbar_init_n(&sm.ready[b], NP);
            mbar_init_n(&sm.empty[b], NS);
        }
        mbar_init_n(&sm.v_free, NS);
        for (uint64_t *b : {&sm.wy, &sm.u, &sm.d, &sm.z, &sm.g, &sm.drain[0], &sm.drain[1]}) mbar_init_n(b, 1);
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
        const int hh = warp >> 2, j = 32 * (warp & 3) + lane;   // key rows [64 hh, 64 hh + 64), value column
        const uint32_t quad = tm + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t kq0 = tc::smem_addr(sm.kq), t0 = tc::smem_addr(sm.t), a0 = tc::smem_addr(sm.a);
        float S[64];
#pragma unroll
        for (int i = 0; i < 64; ++i) S[i] = fresh ? 0.0f : Sg[(size_t)(64 * hh + i) * D + j];
        auto put_state = [&]() {
            uint32_t hi[32], lo[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) tc16::split2(S[2 * i], S[2 * i + 1], hi[i], lo[i]);
            tc16::st32(quad + TSH + 32 * hh, hi);
            tc16::st32(quad + TSL + 32 * hh, lo);
            tc16::st_wait();
            tc::fence_before();
        };
        // W^T = S^T K^T and Y^T = S^T Q^T: the rows of [K; Q] are the 128 columns
        auto issue_wy = [&](int c) {
            const int b = c & 1;
            if (!tc::mbar_wait(&sm.full[b], (c >> 1) & 1, kPolls)) return false;
            tc::fence_after();
            const uint32_t kq = kq0 + b * KT * kTerm;
            for (int p = 0; p < (KT == 1 ? 2 : 3); ++p) {
                const uint32_t sa = tm + (p == 1 ? TSL : TSH), kb = kq + (p == 2 ? kTerm : 0u);
                const uint32_t id = tc16::idesc(128, KT == 1 && p == 1 ? C : 2 * C, false);
                for (int kk = 0; kk < 8; ++kk)
                    tc16::mma_ts(tm + TWY, sa + 8 * kk, tc16::kmajor(kb + (kk >> 2) * kHalf + (kk & 3) * 32), id, p || kk);
            }
            tc::commit(&sm.wy);
            return true;
        };
        put_state();
        ok = tc16::group_and(1, NS, ok);
        if (tid == 0) {
            tc::fence_after();
            ok = issue_wy(0);
        }
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            const int b = c & 1, cc = min(C, count - c * C), vb = Sm::VB == 2 ? b : 0;
            const uint32_t ph = c & 1;
            // V and the gates are in place where the products are, but this thread has to see them itself
            ok = tc::mbar_wait(&sm.full[b], (c >> 1) & 1, kPolls) && ok;
            ok = tc::mbar_wait(&sm.wy, ph, kPolls) && ok;
            tc::fence_after();
            uint32_t y[32];
            {
                uint32_t w[32], hi[16], lo[16];
                tc::ld32(quad + TWY + 32 * hh, w);
                tc::ld32(quad + TWY + C + 32 * hh, y);
                const T *v = reinterpret_cast<const T *>(sm.v[vb]) + 32 * hh * D + j;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float r[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int t = 2 * i + e;
                        const float x = fmaf(-sm.gam[b][32 * hh + t], __uint_as_float(w[t]), to_f32(v[t * D]));
                        r[e] = 32 * hh + t < cc ? x : 0.0f;
                    }
                    tc16::split2(r[0], r[1], hi[i], lo[i]);
                }
                tc16::st16(quad + TR + 16 * hh, hi);
                tc16::st16(quad + TR + 32 + 16 * hh, lo);
                tc16::st_wait();
            }
            if constexpr (KT == 2) mbar_arrive(&sm.v_free);
            tc::fence_before();
            ok = tc16::group_and(1, NS, ok);
            if (!ok) break;
            if (tid == 0) {   // U^T = R^T T^T
                ok = tc::mbar_wait(&sm.ready[b], (c >> 1) & 1, kPolls);
                tc::fence_after();
                const uint32_t id = tc16::idesc(128, C, false);
                if (ok) {
                    for (int p = 0; p < 3; ++p)
                        for (int kk = 0; kk < 4; ++kk)
                            tc16::mma_ts(tm + TU, tm + TR + (p == 2 ? 32 : 0) + 8 * kk,
                                         tc16::kmajor(t0 + b * 2 * C * 128 + (p == 1 ? C * 128 : 0) + kk * 32), id, p || kk);
                    tc::commit(&sm.u);
                }
            }
            ok = tc::mbar_wait(&sm.u, ph, kPolls) && ok;
            tc::fence_after();
            {
                uint32_t u[32], hi[16], lo[16];
                tc::ld32(quad + TU + 32 * hh, u);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 f = *reinterpret_cast<const float2 *>(&sm.f[b][32 * hh + 2 * i]);
                    tc16::split2(f.x * __uint_as_float(u[2 * i]), f.y * __uint_as_float(u[2 * i + 1]), hi[i], lo[i]);
                }
                tc16::st16(quad + TF + 16 * hh, hi);
                tc16::st16(quad + TF + 32 + 16 * hh, lo);
#pragma unroll
                for (int i = 0; i < 16; ++i) tc16::split2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]), hi[i], lo[i]);
                tc16::st16(quad + TR + 16 * hh, hi);
                if constexpr (KT == 2) tc16::st16(quad + TR + 32 + 16 * hh, lo);
                tc16::st_wait();
            }
            tc::fence_before();
            ok = tc16::group_and(1, NS, ok);
            if (!ok) break;
            if (tid == 0) {
                tc::fence_after();
                // the increment of S^T: (U f)^T K, K's rows along the summed index
                const uint32_t kq = kq0 + b * KT * kTerm;
                uint32_t id = tc16::idesc(128, D, true);
                for (int p = 0; p < KT + 1; ++p)
                    for (int kk = 0; kk < 4; ++kk)
                        tc16::mma_ts(tm + TWY, tm + TF + (p == 1 ? 32 : 0) + 8 * kk,
                                     tc16::desc(kq + (p == 2 ? kTerm : 0u) + kk * 2048, kHalf, 1024), id, p || kk);
                tc::commit(&sm.d);
                // (A U)^T
                id = tc16::idesc(128, C, false);
                for (int p = 0; p < (KT == 1 ? 1 : 3); ++p)
                    for (int kk = 0; kk < 4; ++kk)
                        tc16::mma_ts(tm + TU, tm + TR + (p == 1 ? 32 : 0) + 8 * kk,
                                     tc16::kmajor(a0 + b * KT * C * 128 + (p == 2 ? C * 128 : 0) + kk * 32), id, p || kk);
                tc::commit(&sm.z);
            }
            ok = tc::mbar_wait(&sm.d, ph, kPolls) && ok;
            tc::fence_after();
            const float last = sm.gam[b][C - 1];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                uint32_t x[32];
                tc::ld32(quad + TWY + 64 * hh + 32 * p, x);
#pragma unroll
                for (int i = 0; i < 32; ++i) S[32 * p + i] = fmaf(last, S[32 * p + i], __uint_as_float(x[i]));
            }
            if (c + 1 < chunks) put_state();
            else tc::fence_before();
            ok = tc16::group_and(1, NS, ok);
            if (!ok) break;
            if (tid == 0 && c + 1 < chunks) {
                tc::fence_after();
                ok = issue_wy(c + 1);
            }
            ok = tc::mbar_wait(&sm.z, ph, kPolls) && ok;
            tc::fence_after();
            {
                uint32_t z[32];
                tc::ld32(quad + TU + 32 * hh, z);
                T *o = static_cast<T *>(a.o) + (size_t)(first + c * C + 32 * hh) * a.os + h * D + j;
#pragma unroll
                for (int t = 0; t < 32; ++t)
                    if (32 * hh + t < cc)
                        o[(size_t)t * a.os] = from_f32<T>(fmaf(sm.gam[b][32 * hh + t], __uint_as_float(y[t]), __uint_as_float(z[t])));
            }
            tc::fence_before();
            mbar_arrive(&sm.empty[b]);
        }
        if (tc16::group_and(1, NS, ok)) {
#pragma unroll
            for (int i = 0; i < 64; ++i) Sg[(size_t)(64 * hh + i) * D + j] = S[i];
        } else if (tid == 0) {
            atomicOr(a.err, kErrWait);
        }
    } else {
        // ---- prepare ----
        const int p = tid - NS, pw = p >> 5;
        const uint32_t quad = tm + ((uint32_t)(32 * pw) << 16);
        const T *gq = static_cast<const T *>(a.q) + (size_t)hk * D, *gk = static_cast<const T *>(a.k) + (size_t)hk * D;
        const T *gv = static_cast<const T *>(a.v) + (size_t)h * D;
        bool gates_ok = true;
        // the rows of a chunk into L2, ahead of their loads
        auto prefetch = [&](int c) {
            const int cc = min(C, count - c * C);
            for (int e = p; e < 3 * cc; e += NP) {
                const size_t tok = (size_t)(first + c * C + e / 3);
                const T *src = e % 3 == 0 ? gk + tok * a.ks : e % 3 == 1 ? gq + tok * a.qs : gv + tok * a.vs;
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(D * 2) : "memory");
            }
        };
        prefetch(0);
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            const int b = c & 1, cc = min(C, count - c * C), vb = Sm::VB == 2 ? b : 0;
            ok = tc::mbar_wait(&sm.empty[b], ((c >> 1) & 1) ^ 1, kPolls) && ok;
            if constexpr (KT == 2) ok = tc::mbar_wait(&sm.v_free, (c & 1) ^ 1, kPolls) && ok;
            ok = tc16::group_and(2, NP, ok);
            if (!ok) break;
            if (c + 1 < chunks) prefetch(c + 1);
            const size_t tok0 = (size_t)(first + c * C);
            {   // 16 lanes a row of 128 values
                const int i8 = p & 15;
                const uint32_t kq = tc::smem_addr(sm.kq[b]) + (i8 >> 3) * kHalf, vs = tc::smem_addr(sm.v[vb]);
#pragma unroll 4
                for (int r = p >> 4; r < C; r += NP / 16) {
                    const bool in = r < cc;
                    const size_t tok = in ? tok0 + r : tok0;
                    const T *k = gk + tok * a.ks + i8 * 8, *q = gq + tok * a.qs + i8 * 8, *v = gv + tok * a.vs + i8 * 8;
                    const uint32_t off = tc16::sw_off(r, (i8 & 7) * 8);   // K and Q rows: 64 rows keep r % 8
                    copy16(vs + (r * D + i8 * 8) * 2, v, in);
                    if constexpr (KT == 1) {
                        copy16(kq + off, k, in);
                        copy16(kq + C * 128 + off, q, in);
                    } else {
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                            if (in) load_vec<8>(m ? q : k, x);
                            uint4 hi, lo;
                            tc16::split2(x[0], x[1], hi.x, lo.x);
                            tc16::split2(x[2], x[3], hi.y, lo.y);
                            tc16::split2(x[4], x[5], hi.z, lo.z);
                            tc16::split2(x[6], x[7], hi.w, lo.w);
                            uint8_t *dst = sm.kq[b] + (i8 >> 3) * kHalf + m * C * 128 + off;
                            *reinterpret_cast<uint4 *>(dst) = hi;
                            *reinterpret_cast<uint4 *>(dst + kTerm) = lo;
                        }
                    }
                }
            }
            if (pw == 0) {   // gates: two tokens a lane; log2 of the running products
                float l2[2], bt[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int t = 2 * lane + e;
                    l2[e] = 0.0f;
                    bt[e] = 0.0f;
                    if (t < cc) {
                        const float al = __ldg(a.alpha + (tok0 + t) * a.H + h);
                        gates_ok = gates_ok && al > 0.0f && al <= 1.0f;
                        l2[e] = log2f(al);
                        bt[e] = __ldg(a.beta + (tok0 + t) * a.H + h);
                    }
                }
                float sum = l2[0] + l2[1];
#pragma unroll
                for (int m = 1; m < 32; m <<= 1) {
                    const float y = __shfl_up_sync(0xffffffffu, sum, m);
                    if (lane >= m) sum += y;
                }
                const float total = __shfl_sync(0xffffffffu, sum, 31), mid = sum - l2[1];
                *reinterpret_cast<float2 *>(&sm.lg[2 * lane]) = make_float2(mid, sum);
                *reinterpret_cast<float2 *>(&sm.beta[2 * lane]) = make_float2(bt[0], bt[1]);
                *reinterpret_cast<float2 *>(&sm.gam[b][2 * lane]) = make_float2(exp2f(mid), exp2f(sum));
                *reinterpret_cast<float2 *>(&sm.f[b][2 * lane]) = make_float2(exp2f(total - mid), exp2f(total - sum));
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            tc::fence_smem_to_async();
            mbar_arrive(&sm.full[b]);
            ok = tc::mbar_wait(&sm.full[b], (c >> 1) & 1, kPolls);
            if (p == 0 && ok) {   // [K; Q] K^T
                tc::fence_after();
                const uint32_t kq = tc::smem_addr(sm.kq[b]), id = tc16::idesc(128, C, false);
                for (int m = 0; m < KT * KT; ++m)
                    for (int kk = 0; kk < 8; ++kk) {
                        const uint32_t at = (kk >> 2) * kHalf + (kk & 3) * 32;
                        tc16::mma_ss(tm + TG, tc16::kmajor(kq + (m >> 1) * kTerm + at), tc16::kmajor(kq + (m & 1) * kTerm + at), id, m || kk);
                    }
                tc::commit(&sm.g);
            }
            ok = tc::mbar_wait(&sm.g, c & 1, kPolls) && ok;
            tc::fence_after();
            {
                const int t = p & 63;
                const float lt = sm.lg[t], bt = sm.beta[t];
#pragma unroll 1
                for (int s0 = 0; s0 < C; s0 += 32) {
                    uint32_t g[32];
                    tc::ld32(quad + TG + s0, g);
                    const bool none = s0 > (t | 31);   // right of the diagonal for the whole warp
                    if (p < C) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            float x[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int ss = s0 + e + i;
                                x[i] = !none && ss < t ? bt * exp2f(lt - sm.lg[ss]) * __uint_as_float(g[e + i]) : 0.0f;
                            }
                            *reinterpret_cast<float4 *>(&sm.n[t * SN + s0 + e]) = make_float4(x[0], x[1], x[2], x[3]);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            float x[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const int ss = s0 + e + i;
                                x[i] = !none && ss <= t ? exp2f(lt - sm.lg[ss]) * __uint_as_float(g[e + i]) : 0.0f;
                            }
                            uint4 hi, lo;
                            tc16::split2(x[0], x[1], hi.x, lo.x);
                            tc16::split2(x[2], x[3], hi.y, lo.y);
                            tc16::split2(x[4], x[5], hi.z, lo.z);
                            tc16::split2(x[6], x[7], hi.w, lo.w);
                            uint8_t *dst = sm.a[b] + tc16::sw_off(t, s0 + e);
                            *reinterpret_cast<uint4 *>(dst) = hi;
                            if constexpr (KT == 2) *reinterpret_cast<uint4 *>(dst + C * 128) = lo;
                        }
                    }
                }
            }
            tc::fence_before();
            ok = tc16::group_and(2, NP, ok);
            if (!ok) break;
            // (I + N)^-1: the diagonal blocks of 16 by substitution, a column a lane
            {
                const int r0 = 16 * pw, col = lane & 15;
                float x[16];
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    float y0 = r == col ? 1.0f : 0.0f, y1 = 0.0f;
#pragma unroll
                    for (int m = 0; m + 1 < r; m += 2) {
                        const float2 nn = *reinterpret_cast<const float2 *>(&sm.n[(r0 + r) * SN + r0 + m]);
                        y0 = fmaf(-nn.x, x[m], y0);
                        y1 = fmaf(-nn.y, x[m + 1], y1);
                    }
                    if (r & 1) y0 = fmaf(-sm.n[(r0 + r) * SN + r0 + r - 1], x[r - 1], y0);
                    x[r] = y0 + y1;
                }
                __syncwarp();
                if (lane < 16) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) sm.n[(r0 + r) * SN + r0 + col] = x[r];
                }
            }
            tc16::group_and(2, NP, true);
            // pairs of blocks of M rows at r0 (upper) and r0 + M (lower): the block below the diagonal is
            // -X_lower N X_upper, in N's place; thread: R rows x 4 columns of it.
            auto join = [&](auto m_, auto r_, int r0, int at) {
                constexpr int M = decltype(m_)::value, R = decltype(r_)::value;
                const int row = at / (M / 4) * R, col = at % (M / 4) * 4;
                float acc[R][4];
                auto product = [&](const float *l, const float *r) {
#pragma unroll
                    for (int i = 0; i < R; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
#pragma unroll 4
                    for (int k = 0; k < M; k += 4) {
                        float4 lv[R];
#pragma unroll
                        for (int i = 0; i < R; ++i) lv[i] = *reinterpret_cast<const float4 *>(l + (row + i) * SN + k);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float4 rv = *reinterpret_cast<const float4 *>(r + (k + e) * SN + col);
#pragma unroll
                            for (int i = 0; i < R; ++i) {
                                const float w = e == 0 ? lv[i].x : e == 1 ? lv[i].y : e == 2 ? lv[i].z : lv[i].w;
                                acc[i][0] = fmaf(w, rv.x, acc[i][0]);
                                acc[i][1] = fmaf(w, rv.y, acc[i][1]);
                                acc[i][2] = fmaf(w, rv.z, acc[i][2]);
                                acc[i][3] = fmaf(w, rv.w, acc[i][3]);
                            }
                        }
                    }
                };
                auto put = [&](float sign) {
#pragma unroll
                    for (int i = 0; i < R; ++i)
                        *reinterpret_cast<float4 *>(&sm.n[(r0 + M + row + i) * SN + r0 + col]) =
                            make_float4(sign * acc[i][0], sign * acc[i][1], sign * acc[i][2], sign * acc[i][3]);
                };
                const float *nb = &sm.n[(r0 + M) * SN + r0];
                product(nb, &sm.n[r0 * SN + r0]);
                tc16::group_and(2, NP, true);   // every read of the block is done
                put(1.0f);
                tc16::group_and(2, NP, true);
                product(&sm.n[(r0 + M) * SN + r0 + M], nb);
                tc16::group_and(2, NP, true);
                put(-1.0f);
                tc16::group_and(2, NP, true);
            };
            join(std::integral_constant<int, 16>(), std::integral_constant<int, 1>(), p < 64 ? 0 : 32, p & 63);
            join(std::integral_constant<int, 32>(), std::integral_constant<int, 2>(), 0, p);
            // T = X diag(beta), two terms, zeros right of the diagonal
            {
                const int t = p & 63;
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int s0 = 32 * (p >> 6) + 8 * m;
                    float x[8];
#pragma unroll
                    for (int i = 0; i < 8; i += 4) {
                        const float4 y = *reinterpret_cast<const float4 *>(&sm.n[t * SN + s0 + i]);
                        const float4 bt = *reinterpret_cast<const float4 *>(&sm.beta[s0 + i]);
                        x[i] = s0 + i <= t ? y.x * bt.x : 0.0f;
                        x[i + 1] = s0 + i + 1 <= t ? y.y * bt.y : 0.0f;
                        x[i + 2] = s0 + i + 2 <= t ? y.z * bt.z : 0.0f;
                        x[i + 3] = s0 + i + 3 <= t ? y.w * bt.w : 0.0f;
                    }
                    uint4 hi, lo;
                    tc16::split2(x[0], x[1], hi.x, lo.x);
                    tc16::split2(x[2], x[3], hi.y, lo.y);
                    tc16::split2(x[4], x[5], hi.z, lo.z);
                    tc16::split2(x[6], x[7], hi.w, lo.w);
                    uint8_t *dst = sm.t[b] + tc16::sw_off(t, s0);
                    *reinterpret_cast<uint4 *>(dst) = hi;
                    *reinterpret_cast<uint4 *>(dst + C * 128) = lo;
                }
            }
            tc::fence_smem_to_async();
            mbar_arrive(&sm.ready[b]);
            // beta and the gates' logarithms are rewritten by the next chunk: after every thread's reads
            tc16::group_and(2, NP, true);
        }
        if (!gates_ok) atomicOr(a.err, kErrGateRange);
        if (!ok && p == 0) atomicOr(a.err, kErrWait);
    }
    // A product may still be in flight only after a wait gave up: let it end (bounded) before its memory is given
    // back.  A commit covers what its own thread has issued.
    if (!__syncthreads_and(ok) && (tid == 0 || tid == NS)) {
        uint64_t *bar = &sm.drain[tid == 0 ? 0 : 1];
        tc::commit(bar);
        if (!tc::mbar_wait(bar, 0, kPolls)) atomicOr(a.err, kErrTmemDrain);
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 0) tc::dealloc(tm, 512);
}

template <int KT, class T>
cudaError_t launch(const DeltaArgs &a, cudaStream_t st) {
    const long long blocks = (long long)a.n_seq * a.H;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    auto *kern = k_delta_chunk<KT, T>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem<KT>));
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)blocks, NT, sizeof(Smem<KT>), st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_chunk(int dtype, const DeltaArgs &a, cudaStream_t st) {
    static_assert(sizeof(Smem<1>) <= 227 * 1024 && sizeof(Smem<2>) <= 227 * 1024, "shared memory of a block");
    return dtype == 2 ? launch<1, __nv_bfloat16>(a, st) : launch<2, __half>(a, st);
}

}  // namespace stepq
