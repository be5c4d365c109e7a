// k_dequant_gemm.hip -- int8 x int8 GEMM with a scale for each row of A
// (token) and of B (output channel), an optional bias and a float output:
// C[m][n] = T(fp32(acc) * scale_a[m] * scale_b[n] + bias[n]).
//
// acc is exact in int32 (K <= 131056), so the result does not depend on how
// K is cut; its conversion to binary32 rounds once when |acc| > 2^24, then
// each product and the sum round once, and T (binary16, bfloat16) once.
#include "kv_common.hpp"
#include "launch.hpp"

namespace qg {

namespace {

struct DqArgs {
    const uint8_t *A;
    const uint8_t *B;
    int64_t lda, ldb;
    const float *scale_a, *scale_b, *bias;
    void *C;
    int64_t ldc;
    int M, N, K;
    int tiles_m, tiles_n;
};

// 16-byte chunk swizzle of 128-byte LDS rows: a fragment read gives lane L
// row L & 15 and chunk 4 h + (L >> 4); XOR-ing the chunk with row bits 1..3
// spreads the 16 lanes of each read cycle over the 16 bank groups.
// Rows of 256 bytes span all groups, so every row takes its own.
template <int KB>
__device__ __forceinline__ int swz(int row) { return KB == 128 ? (row >> 1) & 7 : row & 15; }

// four adjacent results of one row
template <int DT>
__device__ __forceinline__ void store4(const DqArgs &p, int m, int n, const float (&y)[4])
{
    if (m >= p.M)
        return;
    const bool vec = n + 3 < p.N && (p.ldc & 3) == 0;
    if constexpr (DT == DT_F32) {
        float *dst = (float *)p.C + (int64_t)m * p.ldc + n;
        if (vec) {
            *(v4f *)dst = (v4f){y[0], y[1], y[2], y[3]};
        } else {
            for (int e = 0; e < 4; ++e)
                if (n + e < p.N)
                    dst[e] = y[e];
        }
    } else {
        uint16_t *dst = (uint16_t *)p.C + (int64_t)m * p.ldc + n;
        const v2u w = {pack2<DT>(y[0], y[1]), pack2<DT>(y[2], y[3])};
        if (vec) {
            *(v2u *)dst = w;
        } else {
            for (int e = 0; e < 4; ++e)
                if (n + e < p.N)
                    dst[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
        }
    }
}

template <int N>
__device__ __forceinline__ void wait_and_barrier()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// BM x BN output tile per workgroup of KG groups of 4 waves (2 x 2).  K goes
// in stages of 128 KG bytes through a ring of NS stages in LDS, filled by
// direct-to-LDS buffer loads NS - 1 stages ahead, one barrier per stage; each
// group multiplies its 128 bytes of a stage, and the groups' sums are joined
// in LDS at the end.  These sizes give a compute unit one tile or none, so two
// groups of waves stand in for a second workgroup (512x8192x8192: 56.7 us with
// two, 59.6 with one), and four for the smallest sizes.  What is left is bound by how fast one unit's few stages
// in flight come in: 65x8192x8192 (64x64 tiles) 27 us, without its products
// 22, without its loads 17; 333x4107x4112 (128x64 tiles) 18.3 us, 0.61 POP/s,
// the matrix cores 11% busy.
template <int DT, int BM, int BN, int WM, int NS, int KG>
__global__ __launch_bounds__(256 * KG) void k_dq_tile(DqArgs p)
{
    constexpr int KB = 128 * KG;
    constexpr int kStage = (BM + BN) * KB;
    constexpr int CPR = KB / 16, RPL = 1024 / KB;        // chunks per row, rows per load
    constexpr int LA = BM / 32, LB = BN / 32;            // loads per wave per stage
    constexpr int WN = 4 / WM;                           // waves of a group: WM x WN
    constexpr int TM = BM / WM / 16, TN = BN / WN / 16;  // 16x16 tiles per wave
    __shared__ __attribute__((aligned(1024))) uint8_t lds[NS * kStage];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int kg = wave >> 2, wm = (wave & 3) / WN, wn = (wave & 3) % WN;
    const int t = xcd_remap(blockIdx.x, gridDim.x);
    const int tm = t % p.tiles_m, tn = t / p.tiles_m;
    const int m0 = tm * BM, n0 = tn * BN;
    const int nkt = (p.K + KB - 1) / KB;

    // a load fills RPL rows of KB bytes; lane L fetches chunk (L % CPR) ^ swz
    // of row L / CPR.  Rows past the operand re-read its last row (their
    // results are not stored); bytes past K read as zeros.
    const uint8_t *abase = p.A + (int64_t)m0 * p.lda;
    const uint8_t *bbase = p.B + (int64_t)n0 * p.ldb;
    const int am = min(BM, p.M - m0) - 1, bn = min(BN, p.N - n0) - 1;
    const uint32_t abytes = (uint32_t)(am * p.lda + p.K), bbytes = (uint32_t)(bn * p.ldb + p.K);
    uint32_t sa[LA], sb[LB];
    int ca[LA], cb[LB];
#pragma unroll
    for (int i = 0; i < LA; ++i) {
        const int r = (wave * LA + i) * RPL + lane / CPR;
        ca[i] = ((lane % CPR) ^ swz<KB>(r)) << 4;
        sa[i] = (uint32_t)(min(r, am) * p.lda) + ca[i];
    }
#pragma unroll
    for (int i = 0; i < LB; ++i) {
        const int r = (wave * LB + i) * RPL + lane / CPR;
        cb[i] = ((lane % CPR) ^ swz<KB>(r)) << 4;
        sb[i] = (uint32_t)(min(r, bn) * p.ldb) + cb[i];
    }
    auto issue = [&](int slot, int kt) __attribute__((always_inline)) {
        uint8_t *st = lds + slot * kStage;
        const int k0 = min(kt * KB, p.K);  // past the end nothing is read
#pragma unroll
        for (int i = 0; i < LA; ++i)
            buffer_load_lds16(abase, abytes, k0 + ca[i] < p.K ? sa[i] + k0 : 0xFFFFFFF0u, 0,
                              st + (wave * LA + i) * 1024);
#pragma unroll
        for (int i = 0; i < LB; ++i)
            buffer_load_lds16(bbase, bbytes, k0 + cb[i] < p.K ? sb[i] + k0 : 0xFFFFFFF0u, 0,
                              st + BM * KB + (wave * LB + i) * 1024);
    };

    v4i acc[TN][TM];
    for (int j = 0; j < TN; ++j)
        for (int i = 0; i < TM; ++i)
            acc[j][i] = (v4i){0, 0, 0, 0};

    for (int s = 0; s < NS - 1; ++s)
        issue(s, s);
    const int arow = wm * (BM / WM) + (lane & 15), brow = wn * (BN / WN) + (lane & 15);
    const int c0 = lane >> 4;
    int slot = 0;
    for (int kt = 0; kt < nkt; ++kt) {
        wait_and_barrier<(NS - 2) * (LA + LB)>();
        issue(slot == 0 ? NS - 1 : slot - 1, kt + NS - 1);
        const uint8_t *st = lds + slot * kStage;
        slot = slot == NS - 1 ? 0 : slot + 1;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = 8 * kg + 4 * h + c0;
            v4i af[TM], bf[TN];
#pragma unroll
            for (int i = 0; i < TM; ++i)
                af[i] = *(const v4i *)(st + (arow + 16 * i) * KB + ((c ^ swz<KB>(arow)) << 4));
#pragma unroll
            for (int j = 0; j < TN; ++j)
                bf[j] = *(const v4i *)(st + BM * KB + (brow + 16 * j) * KB +
                                       ((c ^ swz<KB>(brow)) << 4));
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int i = 0; i < TM; ++i)
                    acc[j][i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(bf[j], af[i], acc[j][i], 0, 0, 0);
        }
    }
    // loads of stages past the last must land before the workgroup ends
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

    // the groups' sums: group j % KG finishes column block j
    if constexpr (KG > 1) {
        static_assert(TN * TM * 4 * KG * 1024 <= NS * kStage, "the ring takes the sums");
        v4i(*sums)[KG][4][TM][64] = (v4i(*)[KG][4][TM][64])lds;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < TN; ++j)
            if (j % KG != kg)
#pragma unroll
                for (int i = 0; i < TM; ++i)
                    sums[j][kg][wave & 3][i][lane] = acc[j][i];
        __syncthreads();
#pragma unroll
        for (int j = 0; j < TN; ++j)
            if (j % KG == kg)
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int o = 1; o < KG; ++o) {
                        const v4i x = sums[j][(kg + o) % KG][wave & 3][i][lane];
                        for (int e = 0; e < 4; ++e)
                            acc[j][i][e] += x[e];
                    }
    }

    // lane: row m0 + .. + lane % 16, columns 4 (lane / 16) + e of each tile
#pragma unroll
    for (int j = 0; j < TN; ++j) {
        if (KG > 1 && j % KG != kg)
            continue;
        const int n = n0 + wn * (BN / WN) + 16 * j + 4 * c0;
        float sbv[4], bv[4];
        for (int e = 0; e < 4; ++e) {
            const int nn = min(n + e, p.N - 1);
            sbv[e] = p.scale_b ? p.scale_b[nn] : 1.0f;
            bv[e] = p.bias ? p.bias[nn] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int m = m0 + wm * (BM / WM) + 16 * i + (lane & 15);
            const float sav = p.scale_a ? p.scale_a[min(m, p.M - 1)] : 1.0f;
            float y[4];
            for (int e = 0; e < 4; ++e)
                y[e] = scale_and_bias(acc[j][i][e], sav, sbv[e], bv[e]);
            store4<DT>(p, m, n, y);
        }
    }
}

// A few tokens (up to 16 TB per grid row): the weights' bytes bound the call.
// The memory wants whole kilobytes of a row per load and about 64 KB in
// flight per compute unit, the matrix operands one lane per weight row, so
// the weights pass through LDS: one workgroup of 8 waves per compute unit
// walks a strided list of 16-column groups, in units of 16 rows x 4 KB of K
// that alternate between two 64 KB slots.  Wave w multiplies bytes 512 w ..
// 512 w + 511 of a unit's rows; its activations stay in registers while K <=
// 8192.  One barrier per unit: after it this unit's bytes are there for every
// wave and the other slot is free, so the next unit's loads go out at once.
// A finished group's 8 partial sums are added by one wave behind that
// barrier, and its results wait in LDS until the end (a store would sit in
// the count that the next unit's wait drains).  Measured: 16x28672x8192 to
// bfloat16 43 us, 236 MB, 5.5 TB/s.
namespace stream {
constexpr int kWaves = 8, kSteps = 8;
constexpr int kChunk = kWaves * kSteps * 64;   // bytes of K per unit (4 KB)
constexpr int kSlot = 16 * kChunk;             // 64 KB
constexpr int kPieces = kChunk / 1024;
constexpr int kLoads = 16 * kPieces / kWaves;  // per wave per unit
constexpr int kHeld = 2;                       // chunks whose activations stay in registers
constexpr int kMaxGroups = 16;
constexpr int kRed = 2 * kSlot;                           // v4i [2][kWaves][64]
constexpr int kPrm = kRed + 2 * kWaves * 64 * 16;         // float [2][kMaxGroups * 16]
constexpr int kOut = kPrm + 2 * kMaxGroups * 16 * 4;      // results, 64 lanes x 4 values each
constexpr int kLds = 160 * 1024;
template <int DT>
constexpr int kOutBytes = 64 * 4 * kElemBytes<DT>;
// groups of a workgroup: its results wait in LDS
template <int DT, int TB>
constexpr int max_groups()
{
    const int n = (kLds - kOut) / (kOutBytes<DT> * TB);
    return n < kMaxGroups ? n : kMaxGroups;
}
}  // namespace stream

typedef __attribute__((address_space(3))) void lds_void_t;
typedef __attribute__((address_space(1))) void glb_void_t;

template <int DT, int TB>
__global__ __launch_bounds__(512, 1) void k_dq_stream(DqArgs p)
{
    using namespace stream;
    constexpr int MAXG = max_groups<DT, TB>();
    static_assert(MAXG >= 7, "LDS budget");
    __shared__ __attribute__((aligned(16))) uint8_t lds[kLds];
    v4i(*red)[kWaves][64] = (v4i(*)[kWaves][64])(lds + kRed);
    float(*prm)[kMaxGroups * 16] = (float(*)[kMaxGroups * 16])(lds + kPrm);

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, g = lane >> 4;
    const int tok = blockIdx.y * 16 * TB + col;  // token of block 0; block b adds 16 b
    const int nch = (p.K + kChunk - 1) / kChunk;
    const int ngroups = (p.N + 15) / 16;
    const int ng = (ngroups - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
    const int nunits = ng * nch;
    auto group_of = [&](int i) { return (int)blockIdx.x + i * (int)gridDim.x; };

    // weights of unit u: wave w loads rows 2 w and 2 w + 1, a kilobyte per
    // load, lane L the granule L ^ row (the fragment reads below then hit
    // different banks); past the end of a row in-bounds bytes of it, which
    // meet zero activations, and past the last row that row, never stored
    auto issue = [&](int u) __attribute__((always_inline)) {
        const int i = u / nch, c = u - i * nch;
        uint8_t *slot = lds + (u & 1) * kSlot;
#pragma unroll
        for (int q = 0; q < kLoads; ++q) {
            const int r = 2 * wave + q / kPieces, piece = q % kPieces;
            const int n = min(group_of(i) * 16 + r, p.N - 1);
            const int kb = min(c * kChunk + piece * 1024 + ((lane ^ r) << 4), p.K - 16);
            __builtin_amdgcn_global_load_lds((const glb_void_t *)(p.B + (int64_t)n * p.ldb + kb),
                                             (lds_void_t *)(slot + (r * kPieces + piece) * 1024), 16,
                                             0, 0);
        }
    };
    // activations of chunk c: zeros past the end of K
    auto load_acts = [&](int c, v4i(&x)[kSteps], int b) __attribute__((always_inline)) {
        const uint8_t *row = p.A + (int64_t)min(tok + 16 * b, p.M - 1) * p.lda;
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
            x[s] = *(const v4i *)(row + min(c * kChunk + (wave * kSteps + s) * 64 + 16 * g, p.K - 16));
    };
    auto drop_past_k = [&](int c, v4i(&x)[kSteps]) __attribute__((always_inline)) {
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int keep = c * kChunk + (wave * kSteps + s) * 64 + 16 * g < p.K ? -1 : 0;
            for (int e = 0; e < 4; ++e)
                x[s][e] &= keep;
        }
    };

    issue(0);
    // this lane's factors: its tokens' here, its columns' through LDS
    float sa[TB];
#pragma unroll
    for (int b = 0; b < TB; ++b)
        sa[b] = p.scale_a ? p.scale_a[min(tok + 16 * b, p.M - 1)] : 1.0f;
    if (tid < ng * 16) {
        const int n = min(group_of(tid >> 4) * 16 + (tid & 15), p.N - 1);
        prm[0][tid] = p.scale_b ? p.scale_b[n] : 1.0f;
        prm[1][tid] = p.bias ? p.bias[n] : 0.0f;
    }
    v4i held[kHeld][TB][kSteps];
    const bool hold = nch <= kHeld;
    if (hold) {
#pragma unroll
        for (int c = 0; c < kHeld; ++c)
            if (c < nch)
#pragma unroll
                for (int b = 0; b < TB; ++b) {
                    load_acts(c, held[c][b], b);
                    drop_past_k(c, held[c][b]);
                }
    } else {
#pragma unroll
        for (int b = 0; b < TB; ++b)
            load_acts(0, held[0][b], b);
    }

    int rd[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
        rd[s] = (col * kPieces + (wave >> 1)) * 1024 + ((((wave & 1) * 32 + 4 * s + g) ^ col) << 4);

    v4i acc[TB];
    auto consume = [&](int slot, const v4i(&x)[TB][kSteps]) __attribute__((always_inline)) {
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const v4i w = *(const v4i *)(lds + slot * kSlot + rd[s]);
#pragma unroll
            for (int b = 0; b < TB; ++b)
                acc[b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w, x[b][s], acc[b], 0, 0, 0);
        }
    };
    // waves 2 i and 2 i + 1 (two token blocks) or wave i finish group i
    auto reduce = [&](int i) __attribute__((always_inline)) {
        const int b = TB == 2 ? wave & 1 : 0;
        if ((TB == 2 ? wave >> 1 : wave) != i % (kWaves / TB))
            return;
        const int rb = TB == 2 ? b : i & 1;
        v4i sum = red[rb][0][lane];
#pragma unroll
        for (int v = 1; v < kWaves; ++v) {
            const v4i x = red[rb][v][lane];
            for (int e = 0; e < 4; ++e)
                sum[e] += x[e];
        }
        const v4f sb = *(const v4f *)&prm[0][i * 16 + 4 * g];
        const v4f bias = *(const v4f *)&prm[1][i * 16 + 4 * g];
        float y[4];
        for (int e = 0; e < 4; ++e)
            y[e] = scale_and_bias(sum[e], TB == 2 && b ? sa[TB - 1] : sa[0], sb[e], bias[e]);
        uint8_t *dst = lds + kOut + (i * TB + b) * kOutBytes<DT> + lane * 4 * kElemBytes<DT>;
        if constexpr (DT == DT_F32)
            *(v4f *)dst = (v4f){y[0], y[1], y[2], y[3]};
        else
            *(v2u *)dst = (v2u){pack2<DT>(y[0], y[1]), pack2<DT>(y[2], y[3])};
    };
    // one unit: its weights are in slot u & 1, its activations in `now`;
    // `next` takes the next unit's when they are not held
    auto unit = [&](int u, v4i(&now)[TB][kSteps], v4i(&next)[TB][kSteps]) __attribute__((always_inline)) {
        // this wave's loads are done and its LDS work too, then every wave's
        __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) expcnt(7) lgkmcnt(0)
        asm volatile("s_barrier" ::: "memory");
        if (u + 1 < nunits) {
            issue(u + 1);
            if (!hold)
#pragma unroll
                for (int b = 0; b < TB; ++b)
                    load_acts((u + 1) % nch, next[b], b);
        }
        const int i = u / nch, c = u - i * nch;
        if (!hold)
#pragma unroll
            for (int b = 0; b < TB; ++b)
                drop_past_k(c, now[b]);
        if (c == 0 && i > 0) {
            reduce(i - 1);
            // two token blocks use both halves of the buffer: its readers
            // finish before this group's sums overwrite it
            if (TB == 2)
                asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        }
        if (c == 0)
#pragma unroll
            for (int b = 0; b < TB; ++b)
                acc[b] = (v4i){0, 0, 0, 0};
        consume(u & 1, now);
        if (c == nch - 1)
#pragma unroll
            for (int b = 0; b < TB; ++b)
                red[TB == 2 ? b : i & 1][wave][lane] = acc[b];
    };
    if (nch == 1) {
        for (int u = 0; u < nunits; ++u)
            unit(u, held[0], held[1]);
    } else {
        // an even number of units per pass of the loop body; with two held
        // chunks unit u takes chunk u & 1, otherwise the buffers alternate
        for (int u = 0; u < nunits; u += 2) {
            unit(u, held[0], held[1]);
            if (u + 1 < nunits)
                unit(u + 1, held[1], held[0]);
        }
    }
    __builtin_amdgcn_s_waitcnt(0x0070);
    asm volatile("s_barrier" ::: "memory");
    reduce(ng - 1);
    __syncthreads();

    // a lane's 4 values: token lane % 16, columns 4 (lane / 16) ..
    for (int j = wave; j < ng * TB; j += kWaves) {
        const int i = j / TB, m = tok + 16 * (j % TB), n = group_of(i) * 16 + 4 * g;
        const uint8_t *src = lds + kOut + j * kOutBytes<DT> + lane * 4 * kElemBytes<DT>;
        if (m >= p.M)
            continue;
        const bool vec = n + 3 < p.N && (p.ldc & 3) == 0;
        if constexpr (DT == DT_F32) {
            float *dst = (float *)p.C + (int64_t)m * p.ldc + n;
            const v4f y = *(const v4f *)src;
            if (vec) {
                *(v4f *)dst = y;
            } else {
                for (int e = 0; e < 4; ++e)
                    if (n + e < p.N)
                        dst[e] = y[e];
            }
        } else {
            uint16_t *dst = (uint16_t *)p.C + (int64_t)m * p.ldc + n;
            const v2u y = *(const v2u *)src;
            if (vec) {
                *(v2u *)dst = y;
            } else {
                for (int e = 0; e < 4; ++e)
                    if (n + e < p.N)
                        dst[e] = (uint16_t)(y[e >> 1] >> (16 * (e & 1)));
            }
        }
    }
}

template <int DT, int TB>
hipError_t run_stream(const DqArgs &a, int cus, hipStream_t s)
{
    // one workgroup per compute unit, unless its results would not fit; the
    // grid rows of more tokens share the units (a multiple of 8, so that the
    // workgroups of one column set sit on one XCD) and its L2
    const int ngroups = (a.N + 15) / 16, rows = (a.M + 16 * TB - 1) / (16 * TB);
    constexpr int MAXG = stream::max_groups<DT, TB>();
    int grid = rows > 1 ? (cus / rows) & ~7 : cus;
    if (grid < 8)
        grid = 8;
    if (grid * MAXG < ngroups)
        grid = (ngroups + MAXG - 1) / MAXG;
    if (grid > ngroups)
        grid = ngroups;
    hipLaunchKernelGGL((k_dq_stream<DT, TB>), dim3(grid, rows), dim3(512), 0, s, a);
    return hipGetLastError();
}

template <int DT, int BM, int BN, int WM, int NS, int KG>
hipError_t run_tile(DqArgs a, hipStream_t s)
{
    a.tiles_m = (a.M + BM - 1) / BM;
    a.tiles_n = (a.N + BN - 1) / BN;
    hipLaunchKernelGGL((k_dq_tile<DT, BM, BN, WM, NS, KG>), dim3(a.tiles_m * a.tiles_n), dim3(256 * KG), 0, s, a);
    return hipGetLastError();
}

template <int DT>
hipError_t run_dequant(const DequantDesc &d, hipStream_t s)
{
    DqArgs a{};
    a.A = (const uint8_t *)d.A;
    a.B = (const uint8_t *)d.B;
    a.lda = d.lda;
    a.ldb = d.ldb;
    a.scale_a = d.scale_a;
    a.scale_b = d.scale_b;
    a.bias = d.bias;
    a.C = d.C;
    a.ldc = d.ldc;
    a.M = (int)d.M;
    a.N = (int)d.N;
    a.K = (int)d.K;
    // the ring kernel's conditions are those of the other int8 GEMMs
    GemmDesc g{d.A, d.lda, d.B, d.ldb, (const int32_t *)d.bias, nullptr, nullptr, d.C, d.ldc, d.M,
               d.N, d.K, d.cus, nullptr, 0, false, 0, 0, d.scale_a, d.scale_b};
    if (dma_gemm_fits(g, false))
        return launch_s8s8_dequant_dma(g, DT, s);
    if (d.M <= 16)
        return run_stream<DT, 1>(a, d.cus, s);
    const auto tiles = [&](int bm, int bn) {
        return ((d.M + bm - 1) / bm) * ((d.N + bn - 1) / bn);
    };
    // Few small tiles: the length of the walk along K decides, so four groups
    // of waves share it (us, against the two kernels below): 739x160x8048 13.2
    // and 20.4 with 64x32 tiles, 128x1024x8192 11.8 and 15.7, 100x1000x2064 5.3
    // and 6.4; 60x1984x5760 10.3 and 14.5 with the weight stream, 64x4096x1024
    // 4.4 and 9.2, 17x512x16384 16.7 and 17.6.  A second round on the chip costs
    // more: 160x2238x4368 16.6 and 13.1.
    if (tiles(32, 32) <= 256)
        return run_tile<DT, 32, 32, 2, 4, 4>(a, s);
    if (d.M <= 64)
        return run_stream<DT, 2>(a, d.cus, s);
    // The tile by what fills the chip's 256 compute units (us, weights from
    // memory, HIP graph; M x N x K):
    //   256 tiles of 128x128 fill it: 512x8192x8192 56.7, with one group of
    //   waves 59.6
    //   128x64 where 64x64 would need a second round: 333x4107x4112 21.6
    //   against 26.7; 512x4096x4096 20.9 against 24.5.  From 129 to 255 tiles of
    //   128x128 it has more than 256 itself and takes two rounds, which has not
    //   been measured against one of 128x128
    //   64x64: 256x4096x4096 12.9 against 17.2 with 128x64
    //   64x32 when even those leave half of it idle: 70x2900x2064 6.7
    //   against 7.9 with 64x64
    //   128x128 that more than fill it: two workgroups of one group each share a
    //   unit, 1024x8192x2064 38.2 against 42.6, 2048x8192x4112 115 against 136
    if (tiles(128, 128) > 256)
        return run_tile<DT, 128, 128, 2, 2, 1>(a, s);
    if (tiles(128, 128) == 256)
        return run_tile<DT, 128, 128, 2, 2, 2>(a, s);
    if (tiles(64, 64) > 256)
        return run_tile<DT, 128, 64, 2, 3, 2>(a, s);
    if (tiles(64, 64) > 128)
        return run_tile<DT, 64, 64, 2, 3, 2>(a, s);
    return run_tile<DT, 64, 32, 2, 4, 2>(a, s);
}

}  // namespace

hipError_t launch_s8s8_dequant(const DequantDesc &d, hipStream_t s)
{
    if (d.dtype == DT_F32)
        return run_dequant<DT_F32>(d, s);
    if (d.dtype == DT_F16)
        return run_dequant<DT_F16>(d, s);
    return run_dequant<DT_BF16>(d, s);
}

}  // namespace qg
