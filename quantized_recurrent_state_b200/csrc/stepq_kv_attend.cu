// Attention of the newest tokens over the quantised cache (definitions:
// include/stepq.h).
//
// Bound: HBM, the codes and scales of the sequence read once (d bits / 4 + 8
// bytes a token and head).  The codes never become floating-point rows in memory: each
// lane loads its own 16-byte pieces of them straight into the registers that the
// tensor cores read (mma.sync m16n8k16; one query row per column, so a group of eight
// query heads or drafted tokens fills a tile; the fifth-generation instruction needs
// 128 rows and its operands in shared memory, which eight rows cannot pay for).
//   S^T = K q^T    A: 16 tokens x 16 of d, B: q, in shared memory in fragment order
//   O^T += V^T P^T A: 16 of d x 16 tokens, B: P, moved from the C to the B layout
//                  by two 8 x 8 transposes
// The index summed over may be permuted at will, so a lane's codes need not be
// neighbours in the fragment's order: a lane takes contiguous bytes, q is stored to
// match.  Codes become fp16 exactly (1024 + u has the code in its low bits, 1024 + 16 u in the next four; one
// subtraction or fma leaves z.  Leaving the constant in and taking it off the score instead saves 32 of 350 instructions a tile
// but costs the score eight bits where a few channels stand out and the other codes are small).  The row scales stay outside
// the products: r_k multiplies the score, r_v the weight.
//
// The weight p r_v has to fit fp16, whatever r_v is, while the sum of p wants p near 1 at the largest score.  So a row has two
// references: one of the scores, near the largest, which p = 2^(s - ref) is taken against, and an integer power of two for the value
// scales on top of it, which the weight p r_v is multiplied by: 2^7 exactly at the largest.  Both stay where they are until a weight would
// exceed 2^15 or a p 2^16: sums are fp32; a move costs six shuffles a row and the rescaling, a vote otherwise.  fp16 weights carry
// up to 2^-11 of themselves as rounding error, or 2^-32 of the largest's where that is more (fp16 ends at 2^-25); fp32 outputs take
// them as sums of two fp16 values, the second held 2^11 times as large (2^-22 of the weight, or 2^-43 of the largest's), and q
// likewise without that factor (2^-22 of a value, or 2^-39 of the row's largest).  (One reference for both, the largest s + log2 r_v,
// was 1 to 3 % faster, and lost the tokens that it pushed below 2^-126 beside value rows of 1e35 and more.)
//
// Work is cut evenly: all stages of 64 tokens of all (sequence, cache head, tile of rows) units lie in one line, and block i of
// as many as the GPU holds at once takes the i-th piece of it, whatever the lengths are (they are on the device, and each
// block finds its place by a scan of them).  A unit that ends up in several blocks leaves their sums, references and totals in
// the workspace, two places a block; a second kernel joins them in order, so results do not depend on timing.
//
// The cache comes in by bulk copies of whole rows of a page into a ring of stages, issued by a fifth warp that runs ahead
// across units.  Each of the other four warps works on its own 16 tokens of every stage with its own reference, total and sums,
// joined in a fixed order at the end of a unit.
//
// Every wait is bounded.  A warp whose wait gives up goes to the unit's end, where the four agree on whether to go on, and the
// copying warp stays until its copies have landed: shared memory is not given back under them.
//
// Measured: 70 requests of up to 8,192 tokens, 8 cache heads of 128, 8 bits, 32 query heads: 131 to 139 us, 0.66 GB, 5 TB/s (the stages
// alone run at the copy's rate; the start of a block costs 6 us, the end of a unit 3 to 4, the join 7).  One request of
// 131,072 tokens at 4 bits: 50 us against 22: 4-bit codes cost 350 instructions a tile of 16 tokens, and the SM issues 59 % of the
// time.  16 requests of up to 20,000 tokens, two heads of 256: 54.5 us against 29.  Few short ones: 14 us, launch and host.
#include <float.h>

#include <type_traits>

#include "stepq_delta.cuh"
#include "stepq_dev.cuh"
#include "stepq_kv.cuh"
#include "stepq_tc16.cuh"

namespace stepq {

namespace {

constexpr int kWarps = 4, kTile = 16, kMaxBlocks = 1024;
constexpr int kStep = kWarps * kTile;    // tokens of a stage
// The largest weight and p that do not move the references; log2 of the largest just after a move.  fp16 ends at 2^16 above and
// 2^-25 below, so a weight is lost 2^32 below the largest.
constexpr float kMost = 32768.0f, kMostP = 65536.0f;
constexpr int kLift = 7;
constexpr int kLiftQ = 15;               // the queries' largest value is below 2^15: their small values stay above fp16's end, too
constexpr float kNone = -1e30f;          // reference of a row that has seen nothing
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// (x & mask) | magic in one instruction: both constants in registers (two immediates would take two)
__device__ __forceinline__ uint32_t pick(uint32_t x, uint32_t mask, uint32_t magic) {
    uint32_t y;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(y) : "r"(x), "r"(mask), "r"(magic));
    return y;
}
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t bits_of(__half2 x) { return *reinterpret_cast<uint32_t *>(&x); }
__device__ __forceinline__ __half2 half2_of(uint32_t x) { return *reinterpret_cast<__half2 *>(&x); }
// (1024 + u) pairs -> u - zero
__device__ __forceinline__ uint32_t minus(uint32_t x, uint32_t c) { return bits_of(__hsub2(half2_of(x), half2_of(c))); }

// Bytes of a code row that one lane loads: PER of them (a quarter of a K row, an eighth of a V row), in pieces of V
// bytes, piece n of lane i of LANES at byte (n LANES + i) V.
template <int PER>
struct Piece {
    static constexpr int V = PER < 16 ? PER : 16, N = PER / V, W = PER / 4;
    template <int LANES>
    static __device__ __forceinline__ void load(const uint8_t *row, int i, uint32_t (&w)[W]) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const uint8_t *p = row + (n * LANES + i) * V;
            if constexpr (V == 16) {
                const uint4 y = *reinterpret_cast<const uint4 *>(p);
                w[4 * n] = y.x; w[4 * n + 1] = y.y; w[4 * n + 2] = y.z; w[4 * n + 3] = y.w;
            } else if constexpr (V == 8) {
                const uint2 y = *reinterpret_cast<const uint2 *>(p);
                w[0] = y.x; w[1] = y.y;
            } else {
                w[0] = *reinterpret_cast<const uint32_t *>(p);
            }
        }
    }
};

template <int BITS, int D, int NR>
struct Geo {
    static constexpr int RB = D * BITS / 8;              // bytes of a code row
    using K = Piece<RB / 4>;
    using V = Piece<RB / 8>;
    static constexpr int CW = 32 / BITS;                 // codes in a word
    static constexpr int KS = D / 16;                    // K steps of the scores, and 16-column tiles of the sums
    static constexpr int R = 8 * NR;                     // rows of a block
    static constexpr int STAGE = kStep * (2 * RB + 8);   // bytes of a stage: segments as in a page, K codes, V codes, scales
    static constexpr int STAGES = STAGE > 20480 ? 2 : STAGE > 10240 ? 3 : STAGE > 5120 ? 5 : 6;
    static constexpr int SUM1 = KS * NR * 4 * 33;        // the sums of a warp in fragment order, 33 floats for 32 lanes
    static constexpr int SUM = 2 * SUM1 * 4;             // bytes of those of two warps
    static constexpr int SMEM(int terms) { return STAGES * STAGE + SUM + terms * KS * NR * 256; }
    // place of q element dd in the fragments: step, register, half, lane quarter
    static __device__ __forceinline__ int q_at(int dd, int r, int &plane_words) {
        constexpr int CV = K::V * CW / 4;                // codes of a piece
        const int piece = dd / (4 * CV), c = dd / CV % 4, idx = piece * CV + dd % CV;
        int ks, reg, half;
        if constexpr (BITS == 8) {
            ks = idx / 4; reg = idx / 2 % 2; half = idx % 2;
        } else {
            ks = idx / 8 * 2 + idx % 4 / 2; reg = idx % 2; half = idx / 4 % 2;   // codes m and m + 4 of a word are a pair
        }
        plane_words = KS * NR * 32 * 2;
        return ((((ks * NR + r / 8) * 32 + (r % 8) * 4 + c) * 2) + reg) * 2 + half;
    }
    // place of (row r, value column c) among the sums in fragment order: the idx-th of a lane's columns is half idx % 2
    // (rows g or g + 8) of tile idx / 2
    static __device__ __forceinline__ int sum_at(int r, int c) {
        constexpr int CV = V::V * CW / 4;                // codes of a piece
        const int g = c / CV % 8, idx = c / (8 * CV) * CV + c % CV;
        return ((idx / 2 * NR + r / 8) * 4 + 2 * (idx % 2) + (r & 1)) * 33 + g * 4 + r % 8 / 2;
    }
};

// The line of stages.  A sequence of n tokens has ceil(n / 64) of them for each of its units.
struct Line {
    long long total;   // stages of all units
    int per;           // stages of a block
};
__device__ __forceinline__ int stages_of(const KvAttendArgs &a, int s) {
    const int len = a.lens[s];
    if (len <= 0 || len > (int64_t)a.max_pages * a.g.page_tokens) return 0;
    return (len + kStep - 1) / kStep;
}
__device__ __forceinline__ Line line_of(const KvAttendArgs &a, int lane) {
    long long n = 0;
    for (int i = lane; i < a.n_seq; i += 32) n += stages_of(a, i);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) n += __shfl_xor_sync(0xffffffffu, n, w);
    n *= a.g.H * a.row_tiles;
    return {n, (int)((n + a.blocks - 1) / a.blocks)};
}
// A place in the line, and the piece of a unit that starts there.
struct Place {
    int s = -1, stages = 0;      // sequence, its stages a unit
    long long base = 0, end = 0; // its stages in the line
    int unit = 0, first = 0;     // unit of the sequence, stage of the unit
};
__device__ __forceinline__ Place place_of(const KvAttendArgs &a, long long w, int lane) {
    Place p;
    const int units = a.g.H * a.row_tiles;
    long long before = 0;
    for (int i0 = 0; i0 < a.n_seq; i0 += 32) {
        const long long own = i0 + lane < a.n_seq ? (long long)units * stages_of(a, i0 + lane) : 0;
        long long upto = own;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, upto, m);
            if (lane >= m) upto += y;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, before + upto > w);
        if (hit) {
            const int l = __ffs(hit) - 1;
            p.s = i0 + l;
            p.end = before + __shfl_sync(0xffffffffu, upto, l);
            p.base = p.end - __shfl_sync(0xffffffffu, own, l);
            p.stages = (int)((p.end - p.base) / units);
            p.unit = (int)((w - p.base) / p.stages);
            p.first = (int)((w - p.base) % p.stages);
            return p;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
    return p;
}
// The start of the next unit.
__device__ __forceinline__ void next_unit(const KvAttendArgs &a, Place &p) {
    p.first = 0;
    if (p.base + (long long)(++p.unit) * p.stages < p.end) return;
    p.unit = 0;
    p.base = p.end;
    do p.stages = stages_of(a, ++p.s);
    while (p.stages == 0);
    p.end = p.base + (long long)a.g.H * a.row_tiles * p.stages;
}
__device__ __forceinline__ void put_out(const KvAttendArgs &a, int64_t at, float y) {
    if (a.dtype == 0) static_cast<float *>(a.o)[at] = y;
    else if (a.dtype == 1) static_cast<__half *>(a.o)[at] = __float2half_rn(y);
    else static_cast<__nv_bfloat16 *>(a.o)[at] = __float2bfloat16_rn(y);
}
// Natural logarithm of 2^m l.
__device__ __forceinline__ float log_sum(float m, float l) { return l == 0.0f ? -INFINITY : fmaf(m, kLn2, logf(l)); }
// The value scales' reference k (an integer within [-60, 126]) as the factor of the weights, and what undoes it at the end.
__device__ __forceinline__ float factor_of(int k) { return __uint_as_float((uint32_t)(127 + kLift - k) << 23); }
__device__ __forceinline__ float undo_of(int k) { return __uint_as_float((uint32_t)(127 - kLift + k) << 23); }
__device__ __forceinline__ int k_of(float factor) { return 127 + kLift - (int)(__float_as_uint(factor) >> 23); }
__device__ __forceinline__ int scale_ref(float x) { return (int)fminf(fmaxf(ceilf(x), -60.0f), 126.0f); }
__device__ __forceinline__ void bar_workers() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory"); }

// Blocks an SM that the compiler is held to with two terms, whose independent sums it would otherwise run side by side in the
// registers of a block: those of one term have as many without being told.
template <int BITS, int D, int NR, int TERMS>
__global__ void __launch_bounds__(32 * kWarps + 32, TERMS == 1 ? 0 : NR * D > 256 ? 1 : NR * D > 128 ? 2 : NR * D > 64 ? 3 : 4) k_kv_attend(KvAttendArgs a) {
    using G = Geo<BITS, D, NR>;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t *const ring = smem;                                                 // [STAGES] stages
    float *const sum = reinterpret_cast<float *>(smem + G::STAGES * G::STAGE);  // [2][SUM1]
    __half *qf = reinterpret_cast<__half *>(smem + G::STAGES * G::STAGE + G::SUM);   // [TERMS][KS][NR][32][2] half pairs
    __shared__ float qe[G::R];                           // score factor of the row
    __shared__ float wref[kWarps][G::R], wtot[kWarps][G::R];
    __shared__ float wsc[kWarps][G::R];
    __shared__ uint64_t full[G::STAGES], empty[G::STAGES];
    const KvGeo &g = a.g;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, lg = lane >> 2, lc = lane & 3;
    const int group = a.Hq / g.H, rows = a.n_tok * group;
    // every block is resident at once, so the joining kernel's may take what is left of the SMs and wait there
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Line line = line_of(a, lane);
    const long long w0 = (long long)blockIdx.x * line.per, w1 = min(line.total, w0 + line.per);
    if (w0 >= w1) return;
    if (threadIdx.x == 0) {
        for (int b = 0; b < G::STAGES; ++b) {
            mbar_init(&full[b], 1);
            mbar_init(&empty[b], kWarps);
        }
        fence_mbar_init();
    }
    __syncthreads();
    Place at = place_of(a, w0, lane);
    if (warp == kWarps) {
        // ---- copies ---- a lane takes a.seg tokens of a stage, which lie in one page: seg divides pages and stages.  One
        // copy where that is the page (its rows and scales are neighbours), four otherwise.
        const uint32_t page_bytes = (uint32_t)g.page_bytes(), v_off = (uint32_t)(g.page_tokens * G::RB);
        const uint32_t codes = (uint32_t)(a.seg * G::RB), scales = (uint32_t)(a.seg * 4);
        const int off = lane * a.seg;
        bool bad_page = false, in_time = true;
        int b = 0;
        uint32_t round = 0;
        for (long long w = w0; w < w1 && in_time;) {
            const int n = (int)min(w1 - w, (long long)(at.stages - at.first)), len = a.lens[at.s];
            const int32_t *table = a.table + (int64_t)at.s * a.max_pages;
            const uint8_t *const head = a.cache + (int64_t)(at.unit / a.row_tiles) * g.head_bytes();
            auto lookup = [&](int t, int &row) {
                const int i = (int)(__umulhi((uint32_t)t, a.div_mul) >> a.div_shift);
                row = t - i * g.page_tokens;
                return __ldg(table + i);
            };
            int t0 = at.first * kStep;
            const int end = min(len, (at.first + n) * kStep);
            int row = 0, page = off < kStep && t0 + off < end ? lookup(t0 + off, row) : 0;
            for (; t0 < end; t0 += kStep) {
                const bool mine = off < kStep && t0 + off < end;
                const int now = page, now_row = row;
                if (off < kStep && t0 + kStep + off < end) page = lookup(t0 + kStep + off, row);   // ahead of its use
                in_time = __all_sync(0xffffffffu, mbar_wait_bounded(&empty[b], (round & 1) ^ 1, a.polls));
                if (!in_time) break;
                const uint32_t lanes = __popc(__ballot_sync(0xffffffffu, mine));
                if (lane == 0) mbar_arrive_expect(&full[b], lanes * 2 * (codes + scales) + a.phantom_tx);
                __syncwarp();
                if (mine) {
                    const bool in = (uint32_t)now < (uint32_t)g.n_pages;
                    bad_page = bad_page || !in;
                    const uint8_t *base = head + (uint64_t)(in ? (uint32_t)now : 0u) * page_bytes;
                    const uint8_t *src = base + (uint32_t)(now_row * G::RB), *sc = base + 2 * v_off + 4 * now_row;
                    uint8_t *dst = ring + b * G::STAGE + lane * 2 * (codes + scales);   // as in a page of seg tokens
                    if (a.seg == g.page_tokens) {
                        bulk_g2s(dst, base, 2 * (codes + scales), &full[b]);
                    } else {
                        bulk_g2s(dst, src, codes, &full[b]);
                        bulk_g2s(dst + codes, src + v_off, codes, &full[b]);
                        bulk_g2s(dst + 2 * codes, sc, scales, &full[b]);
                        bulk_g2s(dst + 2 * codes + scales, sc + 4 * g.page_tokens, scales, &full[b]);
                    }
                }
                if (++b == G::STAGES) {
                    b = 0;
                    ++round;
                }
            }
            w += n;
            if (w < w1) next_unit(a, at);
        }
        if (bad_page) atomicOr(g.err, kErrKvPlace);
        if (lane == 0) {
            // stage i was last filled in this turn of the ring, or in the one before
            for (int i = 0; i < G::STAGES; ++i)
                if (i < b || round > 0) in_time = mbar_wait_bounded(&full[i], (i < b ? round : round - 1) & 1, a.polls) && in_time;
            if (!in_time) atomicOr(g.err, kErrKvWait);
        }
        return;
    }

    // where this lane's rows and scales stand in a stage
    // 4-bit codes in bits 0-3 / 4-7 of both halves of a word as fp16 pairs: (1024 + u) - 1032, (1024 + 16 u) / 16 - 72
    const uint32_t lo_mask = 0x000f000fu, hi_mask = 0x00f000f0u, magic = 0x64006400u;
    auto low = [&](uint32_t x) { return minus(pick(x, lo_mask, magic), 0x64086408u); };
    auto high = [&](uint32_t x) {
        return bits_of(__hfma2(half2_of(pick(x, hi_mask, magic)), half2_of(0x2c002c00u), half2_of(0xd480d480u)));
    };
    const int seg_at = warp * kTile / a.seg * a.seg * (2 * G::RB + 8), seg_row = warp * kTile % a.seg;
    const int k_at = seg_at + (seg_row + lg) * G::RB, v_at = seg_at + (a.seg + seg_row + 2 * lc) * G::RB;
    const int s_at = seg_at + 2 * a.seg * G::RB + 4 * (seg_row + lg);
    bool ok = true;
    int b = 0;
    uint32_t round = 0;
#pragma unroll 1
    for (long long w = w0; w < w1;) {
    const int s = at.s, len = a.lens[s], n = (int)min(w1 - w, (long long)(at.stages - at.first));
    const int h = at.unit / a.row_tiles, r0 = at.unit % a.row_tiles * G::R, nrow = min(G::R, rows - r0);
    const int begin = at.first * kStep, end = min(len, (at.first + n) * kStep);

    // q rows as fp16 fragments, scaled by a power of two to below 2^kLiftQ
    constexpr int QR = G::R / kWarps;
    float qx[QR][D / 32];
#pragma unroll
    for (int y = 0; y < QR; ++y) {
        const int r = warp + y * kWarps;
        if (r < nrow) {
            const int i = (r0 + r) / group, hq = h * group + (r0 + r) % group;
            const int64_t from = ((int64_t)s * a.n_tok + i) * a.qs + (int64_t)hq * D + lane;
#pragma unroll
            for (int e = 0; e < D / 32; ++e)
                qx[y][e] = a.dtype == 0   ? static_cast<const float *>(a.q)[from + e * 32]
                           : a.dtype == 1 ? to_f32(static_cast<const __half *>(a.q)[from + e * 32])
                                          : to_f32(static_cast<const __nv_bfloat16 *>(a.q)[from + e * 32]);
        } else {
#pragma unroll
            for (int e = 0; e < D / 32; ++e) qx[y][e] = 0.0f;
        }
    }
#pragma unroll
    for (int y0 = 0; y0 < QR; ++y0) {
        const int r = warp + y0 * kWarps;
        const float (&x)[D / 32] = qx[y0];
        float m = 0.0f;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) m = fmaxf(m, fabsf(x[e]));
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
        int ex = 0;
        if (m > 0.0f && m <= FLT_MAX) frexpf(m, &ex);
        if (ex > -100) ex -= kLiftQ;                     // (the score factor below has to stay a normal number)
        // 2^-ex in two factors, each of which is a normal number
        const int e1 = ex / 2, e2 = ex - e1;
        const float f1 = ldexpf(1.0f, -e1), f2 = ldexpf(1.0f, -e2);
        int plane;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {
            const float y = x[e] * f1 * f2;
            const int at = G::q_at(e * 32 + lane, r, plane);
            const __half hi = __float2half_rn(y);
            qf[at] = hi;
            if constexpr (TERMS == 2) qf[2 * plane + at] = __float2half_rn(y - __half2float(hi));
        }
        if (lane == 0) qe[r] = ldexpf(a.scale * kLog2e, ex);
    }
    bar_workers();

    float ref[2 * NR], total[2 * NR], lift[2 * NR];
    float fac[2 * NR];                                   // of the value scales' reference
    int limit[2 * NR];                                   // first token that the row does not see
    float acc[G::KS][NR][4];
#pragma unroll
    for (int j = 0; j < 2 * NR; ++j) {
        const int r = 8 * (j / 2) + 2 * lc + j % 2;
        ref[j] = 0.0f;                                   // set by the first tile
        fac[j] = factor_of(0);
        total[j] = 0.0f;
        lift[j] = qe[r];
        limit[j] = r < nrow ? len - a.n_tok + 1 + (r0 + r) / group : 0;   // a row without a query sees nothing
    }
    const int clear = len - a.n_tok + 1 + r0 / group;    // tokens below it are seen by every row
#pragma unroll
    for (int mt = 0; mt < G::KS; ++mt)
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) acc[mt][nr][0] = acc[mt][nr][1] = acc[mt][nr][2] = acc[mt][nr][3] = 0.0f;

    bool first = true;
#pragma unroll 1
    for (int t0 = begin + warp * kTile; t0 - warp * kTile < end; t0 += kStep) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&full[b], round & 1, a.polls));
        if (!ok) break;
        const uint8_t *const stage = ring + b * G::STAGE;
        uint64_t *const done = &empty[b];
        if (++b == G::STAGES) {
            b = 0;
            ++round;
        }
        if (t0 >= end) {                                 // the unit's last stage
            if (lane == 0) mbar_arrive(done);
            continue;
        }
        uint32_t kw[2][G::K::W], vw[4][G::V::W];
        float rk[2], rv[2];
        {
            const uint8_t *kr = stage + k_at;
            const float *sc = reinterpret_cast<const float *>(stage + s_at);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                G::K::template load<4>(kr + 8 * i * G::RB, lc, kw[i]);
                rk[i] = sc[8 * i];
                rv[i] = sc[a.seg + 8 * i];
            }
        }
        // scores of 16 tokens (rows lg, lg + 8 of the tile) by R query rows
        float sc[NR][4];
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) sc[nr][0] = sc[nr][1] = sc[nr][2] = sc[nr][3] = 0.0f;
        const uint2 *qs = reinterpret_cast<const uint2 *>(qf) + lane;
        auto score = [&](int ks, const uint32_t (&f)[4]) {
#pragma unroll
            for (int p = 0; p < TERMS; ++p)
#pragma unroll
                for (int nr = 0; nr < NR; ++nr) {
                    const uint2 b = qs[((p * G::KS + ks) * NR + nr) * 32];
                    mma16816(sc[nr], f, b.x, b.y);
                }
        };
#pragma unroll
        for (int w = 0; w < G::K::W; ++w) {
            if constexpr (BITS == 8) {
                uint32_t f[4];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    f[i] = minus(__byte_perm(kw[i][w], 0x64646464u, 0x4140), 0x64806480u);
                    f[2 + i] = minus(__byte_perm(kw[i][w], 0x64646464u, 0x4342), 0x64806480u);
                }
                score(w, f);
            } else {
                uint32_t f[2][4];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int m = 0; m < 2; ++m) {        // codes 2 m and 2 m + 4, 2 m + 1 and 2 m + 5 of the word
                        const uint32_t y = kw[i][w] >> (8 * m);
                        f[m][i] = low(y);
                        f[m][2 + i] = high(y);
                    }
                score(2 * w, f[0]);
                score(2 * w + 1, f[1]);
            }
        }
        {
            const uint8_t *vr = stage + v_at;
#pragma unroll
            for (int i = 0; i < 4; ++i) G::V::template load<8>(vr + ((i & 1) + 8 * (i >> 1)) * G::RB, lg, vw[i]);
        }
        // the score less its reference
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 y = fma2(make_float2(sc[nr][2 * i], sc[nr][2 * i + 1]),
                                      mul2(make_float2(rk[i], rk[i]), make_float2(lift[2 * nr], lift[2 * nr + 1])),
                                      make_float2(-ref[2 * nr], -ref[2 * nr + 1]));
                sc[nr][2 * i] = y.x;
                sc[nr][2 * i + 1] = y.y;
            }
        const bool masked = t0 + kTile > clear;
        if (masked) {
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (t0 + lg + 8 * (e >> 1) >= limit[2 * nr + (e & 1)]) sc[nr][e] = -INFINITY;
        }
        float p[NR][4], wgt[NR][4];
        auto weigh = [&]() {                             // true: a weight or a p is too large for the references
            bool far = false;
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 p2 = make_float2(ex2(sc[nr][2 * i]), ex2(sc[nr][2 * i + 1]));
                    float2 w = mul2(mul2(p2, make_float2(rv[i], rv[i])), make_float2(fac[2 * nr], fac[2 * nr + 1]));
                    if (masked) {                        // nothing of a masked row, whatever its scale
                        if (sc[nr][2 * i] == -INFINITY) w.x = 0.0f;
                        if (sc[nr][2 * i + 1] == -INFINITY) w.y = 0.0f;
                    }
                    far = far || p2.x > kMostP || p2.y > kMostP || w.x > kMost || w.y > kMost;
                    p[nr][2 * i] = p2.x;
                    p[nr][2 * i + 1] = p2.y;
                    wgt[nr][2 * i] = w.x;
                    wgt[nr][2 * i + 1] = w.y;
                }
            return far;
        };
        if (first || __any_sync(0xffffffffu, weigh())) {
            // A row of zeros (r_v = 0) and one marked NaN count as 2^-60, so that they do not move the others' weights down.
            const float lr[2] = {fmaxf(lg2(rv[0]), -60.0f), fmaxf(lg2(rv[1]), -60.0f)};
#pragma unroll
            for (int j = 0; j < 2 * NR; ++j) {
                const float s0 = sc[j / 2][j & 1], s1 = sc[j / 2][2 + (j & 1)];
                float ms = fmaxf(s0, s1), mw = fmaxf(s0 + lr[0], s1 + lr[1]);
#pragma unroll
                for (int w = 4; w < 32; w <<= 1) {
                    ms = fmaxf(ms, __shfl_xor_sync(0xffffffffu, ms, w));
                    mw = fmaxf(mw, __shfl_xor_sync(0xffffffffu, mw, w));
                }
                // the row's own need, whatever its neighbours': down only while there are no sums (a row that sees nothing in its first
                // tile sees nothing at all).  The largest weight becomes 2^7 exactly, so that fp16 takes nothing from it (one token
                // that outweighs the rest is the common case); the score's reference is then within 1 of the largest score.
                const float was = (float)k_of(fac[j]);
                float by = 0.0f;
                int k = first ? 0 : (int)was;
                if (first ? mw > -INFINITY : ms > 8.0f || mw - was > 8.0f) {
                    const float most = first ? mw : fmaxf(mw, was);   // against the score's reference as it was
                    k = scale_ref(most - (first ? ms : fmaxf(ms, 0.0f)));
                    by = ref[j] + (most - (float)k) - ref[j];
                }
                const float f = first ? 1.0f : ex2(-by), fa = first ? 1.0f : ex2(was - (float)k - by);
                ref[j] += by;
                fac[j] = factor_of(k);
                sc[j / 2][j & 1] = s0 - by;
                sc[j / 2][2 + (j & 1)] = s1 - by;
                total[j] *= f;
#pragma unroll
                for (int mt = 0; mt < G::KS; ++mt) {
                    acc[mt][j / 2][j & 1] *= fa;
                    acc[mt][j / 2][2 + (j & 1)] *= fa;
                }
            }
            weigh();
        }
        uint32_t pb[TERMS][NR][2];
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float w0 = wgt[nr][2 * i], w1 = wgt[nr][2 * i + 1];
                total[2 * nr] += p[nr][2 * i];
                total[2 * nr + 1] += p[nr][2 * i + 1];
                const __half2 hi = __floats2half2_rn(w0, w1);
                pb[0][nr][i] = transpose8(bits_of(hi));
                if constexpr (TERMS == 2) {
                    const float2 back = __half22float2(hi);
                    pb[1][nr][i] = transpose8(bits_of(__floats2half2_rn((w0 - back.x) * 2048.0f, (w1 - back.y) * 2048.0f)));
                }
            }
        // sums; the weights' second terms are 2^11 times what they stand for, their codes 2^-11 (exact).  The instruction cuts off
        // what it adds to a larger sum, so for fp32 a tile is summed by itself and added rounded (2 to 9 %: 16 requests of 20,000 tokens, two
        // heads of 256, 8 bits, 88 us for 84; d = 128 52.5 for 51).
        auto add = [&](int mt, const uint32_t (&f)[4]) {
            if constexpr (TERMS == 1) {
#pragma unroll
                for (int nr = 0; nr < NR; ++nr) mma16816(acc[mt][nr], f, pb[0][nr][0], pb[0][nr][1]);
            } else {
                uint32_t g[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) g[i] = bits_of(__hmul2(half2_of(f[i]), half2_of(0x10001000u)));
#pragma unroll
                for (int nr = 0; nr < NR; ++nr) {
                    float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    mma16816(x, f, pb[0][nr][0], pb[0][nr][1]);
                    mma16816(x, g, pb[1][nr][0], pb[1][nr][1]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[mt][nr][e] += x[e];
                }
            }
        };
#pragma unroll
        for (int w = 0; w < G::V::W; ++w) {
            if constexpr (BITS == 8) {
                uint32_t f[2][4];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t lo = __byte_perm(vw[2 * i][w], vw[2 * i + 1][w], 0x5140);
                    const uint32_t hi = __byte_perm(vw[2 * i][w], vw[2 * i + 1][w], 0x7362);
                    f[0][2 * i] = minus(__byte_perm(lo, 0x64646464u, 0x4140), 0x64806480u);
                    f[0][2 * i + 1] = minus(__byte_perm(lo, 0x64646464u, 0x4342), 0x64806480u);
                    f[1][2 * i] = minus(__byte_perm(hi, 0x64646464u, 0x4140), 0x64806480u);
                    f[1][2 * i + 1] = minus(__byte_perm(hi, 0x64646464u, 0x4342), 0x64806480u);
                }
                add(2 * w, f[0]);
                add(2 * w + 1, f[1]);
            } else {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t f[2][4];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t y = __byte_perm(vw[2 * i][w], vw[2 * i + 1][w], half ? 0x7632 : 0x5410);
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            const uint32_t z = y >> (8 * m);
                            f[m][2 * i] = low(z);
                            f[m][2 * i + 1] = high(z);
                        }
                    }
                    add(4 * w + 2 * half, f[0]);
                    add(4 * w + 2 * half + 1, f[1]);
                }
            }
        }
        first = false;
        // only here: a load that has been issued but not used yet may still read the stage after the arrival
        __syncwarp();
        if (lane == 0) mbar_arrive(done);
    }
    // join the warps: totals and references first, then the sums, (0 + 2) + (1 + 3)
#pragma unroll
    for (int j = 0; j < 2 * NR; ++j) {
        total[j] += __shfl_xor_sync(0xffffffffu, total[j], 4);
        total[j] += __shfl_xor_sync(0xffffffffu, total[j], 8);
        total[j] += __shfl_xor_sync(0xffffffffu, total[j], 16);
        if (lg == 0) {
            const int r = 8 * (j / 2) + 2 * lc + j % 2;
            wref[warp][r] = total[j] == 0.0f ? kNone : ref[j];
            wtot[warp][r] = total[j];
            wsc[warp][r] = (float)k_of(fac[j]);
        }
    }
    ok = tc16::group_and(1, 32 * kWarps, ok);            // all four stop, or none
#pragma unroll
    for (int j = 0; j < 2 * NR; ++j) {
        const int r = 8 * (j / 2) + 2 * lc + j % 2;
        float m = wref[0][r];
#pragma unroll
        for (int y = 1; y < kWarps; ++y) m = fmaxf(m, wref[y][r]);
        float top = wref[0][r] - m + wsc[0][r];
#pragma unroll
        for (int y = 1; y < kWarps; ++y) top = fmaxf(top, wref[y][r] - m + wsc[y][r]);
        const float f = ex2(wref[warp][r] - m + wsc[warp][r] - (float)scale_ref(top));
#pragma unroll
        for (int mt = 0; mt < G::KS; ++mt) {
            acc[mt][j / 2][j & 1] *= f;
            acc[mt][j / 2][2 + (j & 1)] *= f;
        }
    }
    auto pass = [&](float *to, const float *from) {      // this warp's sums, plus `from`, to `to`
#pragma unroll
        for (int mt = 0; mt < G::KS; ++mt)
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int c = ((mt * NR + nr) * 4 + e) * 33 + lane;
                    if (from) acc[mt][nr][e] += from[c];
                    if (to) to[c] = acc[mt][nr][e];
                }
    };
    if (warp >= 2) pass(sum + (warp - 2) * G::SUM1, nullptr);
    bar_workers();
    if (warp < 2) pass(warp == 1 ? sum + G::SUM1 : nullptr, sum + warp * G::SUM1);
    bar_workers();
    if (warp == 0) pass(sum, sum + G::SUM1);
    bar_workers();
    const bool whole = n == at.stages;
    for (int r = warp; r < nrow; r += kWarps) {
        float m = wref[0][r], l = 0.0f;
#pragma unroll
        for (int y = 1; y < kWarps; ++y) m = fmaxf(m, wref[y][r]);
#pragma unroll
        for (int y = 0; y < kWarps; ++y) l += ex2(wref[y][r] - m) * wtot[y][r];
        float top = wref[0][r] - m + wsc[0][r];
#pragma unroll
        for (int y = 1; y < kWarps; ++y) top = fmaxf(top, wref[y][r] - m + wsc[y][r]);
        const int k = scale_ref(top);
        const float undo = undo_of(k);
        const int64_t tok = (int64_t)s * a.n_tok + (r0 + r) / group;
        const int hq = h * group + (r0 + r) % group;
        const int64_t place = ((int64_t)blockIdx.x * 2 + (at.first == 0 ? 1 : 0)) * G::R + r;   // if not whole
        for (int c = lane; c < D; c += 32) {
            const float y = sum[G::sum_at(r, c)];
            if (whole) put_out(a, tok * a.os + (int64_t)hq * D + c, l == 0.0f ? 0.0f : y / l * undo);
            else a.part[place * D + c] = y;
        }
        if (lane == 0) {
            if (!whole) a.meta[place] = make_float4(m, l, (float)k, 0.0f);
            else if (a.lse) a.lse[tok * a.Hq + hq] = log_sum(m, l);
        }
    }
    if (!ok) break;
    w += n;
    if (w < w1) next_unit(a, at);
    }
    if (!ok && lane == 0) atomicOr(g.err, kErrKvWait);
}

// Joins the pieces of a row that several blocks worked on, in their order: a block a row.  Factors of all pieces first, then
// groups of D / 4 threads take every (4 kJoin / D)-th piece, and the groups' sums are added in order.  Rows of empty
// sequences are written here.
constexpr int kJoin = 256;
template <int D>
__global__ void __launch_bounds__(kJoin) k_kv_join(KvAttendArgs a, int R) {
    constexpr int L = D / 4, GROUPS = kJoin / L;
    __shared__ float f[kMaxBlocks], red[3][kJoin / 32];
    __shared__ __align__(16) float sum[GROUPS][D];
    const KvGeo &g = a.g;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int group = a.Hq / g.H, rows = a.n_tok * group;
    const int rr = (int)(blockIdx.x % rows);
    const int64_t sh = blockIdx.x / rows;
    const int h = (int)(sh % g.H), s = (int)(sh / g.H);
    const int len = a.lens[s], stages = stages_of(a, s);
    const Line line = line_of(a, lane);
    long long before = 0;
    for (int i = lane; i < s; i += 32) before += stages_of(a, i);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) before += __shfl_xor_sync(0xffffffffu, before, w);
    const long long w0 = before * g.H * a.row_tiles + (long long)(h * a.row_tiles + rr / R) * stages;
    // before any return: what follows this kernel relies on the blocks' work, too
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t tok = (int64_t)s * a.n_tok + rr / group;
    const int hq = h * group + rr % group;
    if (stages == 0) {
        if (len > 0 && tid == 0) atomicOr(g.err, kErrKvLen);   // a length above the page table's
        if (len == 0 && tid < D) put_out(a, tok * a.os + (int64_t)hq * D + tid, 0.0f);
        if (len == 0 && tid == 0 && a.lse) a.lse[tok * a.Hq + hq] = -INFINITY;
        return;
    }
    const int b0 = (int)(w0 / line.per), pieces = (int)((w0 + stages - 1) / line.per) - b0 + 1;
    if (pieces == 1) return;                             // written by its block
    // the first piece begins a unit, the others do not
    auto place = [&](int p) { return ((int64_t)(b0 + p) * 2 + (p == 0 ? 1 : 0)) * R + rr % R; };
    float m = kNone;
    for (int p = tid; p < pieces; p += kJoin) m = fmaxf(m, a.meta[place(p)].x);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
    if (lane == 0) red[0][warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoin / 32; ++w) m = fmaxf(m, red[0][w]);
    float l = 0.0f, top = -60.0f;
    for (int p = tid; p < pieces; p += kJoin) {
        const float4 x = a.meta[place(p)];
        l += ex2(x.x - m) * x.y;
        f[p] = x.x - m + x.z;                            // log2 of the piece's sums against the largest score
        top = fmaxf(top, f[p]);
    }
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) {
        l += __shfl_xor_sync(0xffffffffu, l, w);
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
    }
    if (lane == 0) {
        red[1][warp] = l;
        red[2][warp] = top;
    }
    __syncthreads();
    l = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoin / 32; ++w) {
        l += red[1][w];
        top = fmaxf(top, red[2][w]);
    }
    const int k = scale_ref(top);
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int p = tid / L; p < pieces; p += GROUPS) {
        const float4 x = *reinterpret_cast<const float4 *>(a.part + place(p) * D + tid % L * 4);
        const float w = ex2(f[p] - (float)k);
        y.x += w * x.x;
        y.y += w * x.y;
        y.z += w * x.z;
        y.w += w * x.w;
    }
    *reinterpret_cast<float4 *>(&sum[tid / L][tid % L * 4]) = y;
    __syncthreads();
    if (tid < D) {
        float z = 0.0f;
#pragma unroll
        for (int w = 0; w < GROUPS; ++w) z += sum[w][tid];
        put_out(a, tok * a.os + (int64_t)hq * D + tid, l == 0.0f ? 0.0f : z / l * undo_of(k));
    }
    if (tid == 0 && a.lse) a.lse[tok * a.Hq + hq] = log_sum(m, l);
}

template <int BITS, int D, int NR, int TERMS>
cudaError_t launch_one(const KvAttendArgs &a, cudaStream_t st) {
    using G = Geo<BITS, D, NR>;
    const int64_t rows = (int64_t)a.n_seq * a.n_tok * a.Hq;
    if (rows > 0x7fffffff) return cudaErrorInvalidValue;
    constexpr int smem = G::SMEM(TERMS);
    static_assert(smem <= 226 * 1024, "shared memory of a block");
    auto *kern = k_kv_attend<BITS, D, NR, TERMS>;
    kern<<<a.blocks, 32 * kWarps + 32, smem, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // launched while the pieces are still being made: it waits for them itself
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)rows);
    cfg.blockDim = dim3(kJoin);
    cfg.stream = st;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_kv_join<D>, a, G::R);
}

template <int BITS, int D>
cudaError_t launch_d(const KvAttendArgs &a, int nr, cudaStream_t st) {
    if (a.dtype == 0) return nr == 1 ? launch_one<BITS, D, 1, 2>(a, st) : launch_one<BITS, D, 2, 2>(a, st);
    return nr == 1 ? launch_one<BITS, D, 1, 1>(a, st) : launch_one<BITS, D, 2, 1>(a, st);
}

}  // namespace

KvSplit kv_split(const KvGeo &g, int n_tok, int Hq) {
    KvSplit k;
    const int64_t rows = (int64_t)n_tok * (Hq / g.H);
    k.nr = rows <= 8 ? 1 : 2;
    k.row_tiles = (int)((rows + 8 * k.nr - 1) / (8 * k.nr));
    return k;
}

namespace {
template <int BITS, int D, int NR, int TERMS>
cudaError_t blocks_of(int *per_sm) {
    constexpr int smem = Geo<BITS, D, NR>::SMEM(TERMS);
    auto *kern = k_kv_attend<BITS, D, NR, TERMS>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    return e == cudaSuccess ? cudaOccupancyMaxActiveBlocksPerMultiprocessor(per_sm, kern, 32 * kWarps + 32, smem) : e;
}
template <int BITS, int D>
cudaError_t prepare_d(int (*per_sm)[2]) {
    cudaError_t e = blocks_of<BITS, D, 1, 1>(&per_sm[0][0]);
    if (e == cudaSuccess) e = blocks_of<BITS, D, 1, 2>(&per_sm[0][1]);
    if (e == cudaSuccess) e = blocks_of<BITS, D, 2, 1>(&per_sm[1][0]);
    if (e == cudaSuccess) e = blocks_of<BITS, D, 2, 2>(&per_sm[1][1]);
    return e;
}
}  // namespace

cudaError_t kv_prepare(const KvGeo &g, int n_sms, int (*blocks)[2]) {
    cudaError_t e;
    if (g.bits == 8) e = g.d == 64 ? prepare_d<8, 64>(blocks) : g.d == 128 ? prepare_d<8, 128>(blocks) : prepare_d<8, 256>(blocks);
    else e = g.d == 64 ? prepare_d<4, 64>(blocks) : g.d == 128 ? prepare_d<4, 128>(blocks) : prepare_d<4, 256>(blocks);
    for (int i = 0; i < 4; ++i) {
        int &n = blocks[i / 2][i % 2];
        n = n * n_sms < 1 ? 1 : n * n_sms > kMaxBlocks ? kMaxBlocks : n * n_sms;
    }
    return e;
}

cudaError_t launch_kv_attend(const KvAttendArgs &a, int nr, cudaStream_t st) {
    if (a.g.bits == 8) {
        if (a.g.d == 64) return launch_d<8, 64>(a, nr, st);
        if (a.g.d == 128) return launch_d<8, 128>(a, nr, st);
        return launch_d<8, 256>(a, nr, st);
    }
    if (a.g.d == 64) return launch_d<4, 64>(a, nr, st);
    if (a.g.d == 128) return launch_d<4, 128>(a, nr, st);
    return launch_d<4, 256>(a, nr, st);
}

}  // namespace stepq
