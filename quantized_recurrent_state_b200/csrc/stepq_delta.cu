// The gated delta rule token by token on fp32 states (the form of a single
// decoded token, of a few drafted ones, and of the prompts the chunked kernel
// does not take).
//
//   S' = Diag(alpha) S;  u = beta (v - S'^T k);  S = S' + k u^T;  o = S^T q
//
// Columns of S are independent given k, q and the gates, so a warp takes 16
// value columns of one state and needs no other warp: lane 4 g + c holds rows
// [g RT, g RT + RT) of columns 4 c .. 4 c + 3 (RT = D / 8, 64 values at D = 128) in
// registers, reads them once, runs all tokens and writes them once.  The sums
// over the rows are RT fma per lane and column, then three shuffle levels over
// the eight row groups; each level halves the columns that a lane still adds up, so
// it sends 2 + 1 + 1 values.
//
// Bound: HBM, each state read and written once (8 D^2 bytes), as long as there are few tokens: 70 requests of 48 heads at D = 128,
// one token each, 74 us, 5.9 TB/s (65 us of it in the kernel, whose 12 warps an SM have 6,144 16-byte loads in
// flight).  One request is bound by the launch and the host's call (13 us).  From about four tokens on the shuffles count, which are latency: with
// several tokens the next one's rows are loaded before the current one's sums (MANY, up to 242 registers instead of 168;
// 17 requests of 32 heads with four fp32 tokens and gates per key row: 28 to 32 us against a floor of 12).  A warp for
// 16 columns, not a block for a state: no barrier, and 48 states of one request are 384 warps.
#include "stepq_dev.cuh"
#include "stepq_delta.cuh"
#include "stepq_prefill.cuh"

namespace stepq {

namespace {

constexpr int kWarps = 2;  // per block: 48 states of one request already fill the SMs

// Sum of x over the lanes of equal lane % 4; every lane gets all four.
__device__ __forceinline__ void sum_groups(float (&x)[4], int lane) {
    const unsigned full = 0xffffffffu;
    const bool up = lane & 16;
    const float s0 = up ? x[0] : x[2], s1 = up ? x[1] : x[3];
    float a = (up ? x[2] : x[0]) + __shfl_xor_sync(full, s0, 16);
    float b = (up ? x[3] : x[1]) + __shfl_xor_sync(full, s1, 16);
    const bool odd = lane & 8;
    const float s2 = odd ? a : b;
    float c = (odd ? b : a) + __shfl_xor_sync(full, s2, 8);
    c += __shfl_xor_sync(full, c, 4);
    // column 2 up + odd is in c: collect the four from lanes of (up, odd)
    const int base = lane & 7;
    x[0] = __shfl_sync(full, c, base);
    x[1] = __shfl_sync(full, c, base + 8);
    x[2] = __shfl_sync(full, c, base + 16);
    x[3] = __shfl_sync(full, c, base + 24);
}

template <int D, class T, bool ROWS>
struct TokenRow {
    static constexpr int RT = D / 8;
    float k[RT], q[RT], v[4], alpha[ROWS ? RT : 1], beta;
    __device__ __forceinline__ void load(const DeltaArgs &a, size_t t, int h, int hk, int row0, int col0) {
        load_vec<RT>(static_cast<const T *>(a.k) + t * a.ks + hk * D + row0, k);
        load_vec<RT>(static_cast<const T *>(a.q) + t * a.qs + hk * D + row0, q);
        load_vec<4>(static_cast<const T *>(a.v) + t * a.vs + h * D + col0, v);
        if constexpr (ROWS) load_vec<RT>(a.alpha + (t * a.H + h) * D + row0, alpha);
        else alpha[0] = __ldg(a.alpha + t * a.H + h);
        beta = __ldg(a.beta + t * a.H + h);
    }
};

template <int D, class T, bool ROWS, bool MANY>
__global__ void __launch_bounds__(32 * kWarps) k_delta_seq(DeltaArgs a) {
    constexpr int RT = D / 8, PARTS = D / 16;
    const int lane = threadIdx.x & 31;
    const long long item = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int part = (int)(item % PARTS);
    const long long sh = item / PARTS;
    if (sh >= (long long)a.n_seq * a.H) return;
    const int s = (int)(sh / a.H), h = (int)(sh % a.H), hk = h / (a.H / a.Hk);
    const int row0 = (lane >> 2) * RT, col0 = 16 * part + 4 * (lane & 3);
    int first, count;
    if (!delta_range(a, s, first, count)) return;
    float *Sg = delta_state(a, s, h, D, kErrBadSlot);
    if (!Sg) return;
    Sg += (size_t)row0 * D + col0;
    const bool fresh = a.fresh && a.fresh[s];
    if (count == 0 && !fresh) return;

    float4 S[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
        S[r] = fresh ? make_float4(0.f, 0.f, 0.f, 0.f) : *reinterpret_cast<const float4 *>(Sg + (size_t)r * D);

    auto token = [&](const TokenRow<D, T, ROWS> &x, size_t t) {
        float u[4] = {0.f, 0.f, 0.f, 0.f};
        bool good = true;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const float al = x.alpha[ROWS ? r : 0];
            if (ROWS || r == 0) good = good && al > 0.0f && al <= 1.0f;
            S[r].x *= al; S[r].y *= al; S[r].z *= al; S[r].w *= al;
            u[0] = fmaf(x.k[r], S[r].x, u[0]);
            u[1] = fmaf(x.k[r], S[r].y, u[1]);
            u[2] = fmaf(x.k[r], S[r].z, u[2]);
            u[3] = fmaf(x.k[r], S[r].w, u[3]);
        }
        if (a.check_gates && !good) atomicOr(a.err, kErrGateRange);
        sum_groups(u, lane);
#pragma unroll
        for (int c = 0; c < 4; ++c) u[c] = x.beta * (x.v[c] - u[c]);
        float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            S[r].x = fmaf(x.k[r], u[0], S[r].x);
            S[r].y = fmaf(x.k[r], u[1], S[r].y);
            S[r].z = fmaf(x.k[r], u[2], S[r].z);
            S[r].w = fmaf(x.k[r], u[3], S[r].w);
            o[0] = fmaf(x.q[r], S[r].x, o[0]);
            o[1] = fmaf(x.q[r], S[r].y, o[1]);
            o[2] = fmaf(x.q[r], S[r].z, o[2]);
            o[3] = fmaf(x.q[r], S[r].w, o[3]);
        }
        sum_groups(o, lane);
        if (lane < 4) store_vec<4>(static_cast<T *>(a.o) + t * a.os + h * D + col0, o);
    };

    TokenRow<D, T, ROWS> x;
    if constexpr (MANY) {
        // the next token's rows are fetched while this one is worked on
        if (count > 0) x.load(a, (size_t)first, h, hk, row0, col0);
#pragma unroll 1
        for (int i = 0; i < count; ++i) {
            TokenRow<D, T, ROWS> next;
            next.load(a, (size_t)(first + min(i + 1, count - 1)), h, hk, row0, col0);
            token(x, (size_t)(first + i));
            x = next;
        }
    } else {
        x.load(a, (size_t)first, h, hk, row0, col0);
        token(x, (size_t)first);
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) *reinterpret_cast<float4 *>(Sg + (size_t)r * D) = S[r];
}

template <int D, class T>
cudaError_t launch_d(bool rows, const DeltaArgs &a, cudaStream_t st) {
    const long long warps = (long long)a.n_seq * a.H * (D / 16);
    const long long blocks = (warps + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    const bool many = a.cu || a.n_tok > 1;
    auto *kern = rows ? (many ? k_delta_seq<D, T, true, true> : k_delta_seq<D, T, true, false>)
                      : (many ? k_delta_seq<D, T, false, true> : k_delta_seq<D, T, false, false>);
    kern<<<(unsigned)blocks, 32 * kWarps, 0, st>>>(a);
    return cudaGetLastError();
}

template <class T>
cudaError_t launch_t(int D, bool rows, const DeltaArgs &a, cudaStream_t st) {
    switch (D) {
        case 16: return launch_d<16, T>(rows, a, st);
        case 32: return launch_d<32, T>(rows, a, st);
        case 64: return launch_d<64, T>(rows, a, st);
        case 128: return launch_d<128, T>(rows, a, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_delta_seq(int D, int dtype, bool rows, const DeltaArgs &a, cudaStream_t st) {
    if (dtype == 0) return launch_t<float>(D, rows, a, st);
    if (dtype == 1) return launch_t<__half>(D, rows, a, st);
    return launch_t<__nv_bfloat16>(D, rows, a, st);
}

}  // namespace stepq
