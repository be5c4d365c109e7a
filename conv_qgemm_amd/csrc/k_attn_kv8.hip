// k_attn_kv8.hip -- attention of new queries over the paged int8 cache.
//
// For one query row (a new token and a query head) with scores
// x_j = scale * q . k_j over the tokens it sees: one pass over the cache with
// the running maximum m and sum l of the softmax (in powers of two: x is
// taken times log2 e), out = sum_j 2^(x_j - m) v_j / l.
//
// Codes times scales.  A code is exact in binary16 and in bfloat16, so keys
// enter the matrix product as codes and a block's scale multiplies its
// scores.  A block's value scale s joins the weight: the product takes
// w_j = 2^(x_j + log2 s_j - y) with codes, where y is the row's running maximum
// of x_j + log2 s_j over the tokens that it sees, and l collects w_j * (R / s)
// with R = 2^(y - m).  So w stays within [0, 1] and the row's largest term is
// near 1: what a weight loses to binary16's range is small beside the row's own
// terms, whatever scales other rows or hidden tokens have.  (One R for a wave,
// at least every scale met, was 1.5% faster on a prompt but let a row vanish
// beside a later block's scale.)
//
// The product K Q^T leaves token x row tiles in the layout that the second
// product, V^T W^T, takes its weights in (a lane holds 4 tokens of one row
// from every 16; the sum over tokens may run in any order as long as V's
// fragments use the same one), so weights go from one product to the next in
// registers.
#include <type_traits>

#include "kv_common.hpp"

#include "attn_weights.hpp"
#include "launch.hpp"

namespace qg {

namespace {

typedef __attribute__((address_space(3))) void lds_void_t;
typedef __attribute__((address_space(1))) void glb_void_t;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttnArgs {
    AttnDesc d;
    int group;   // query heads per cache head
    int splits;  // parts a sequence is cut into
    int extra;   // find_item
    bool one_tile;  // 16-row kernel: no sequence has more than 16 rows, item b is sequence b
    int shares;  // then: workgroups per cache head that share all sequences' tiles, or 0
    int few;     // sequences of up to this many rows take the 16-row kernel
    float c2;    // scale * log2 e
    int block_shift;      // log2 of the block size
    unsigned num_blocks;
    float *po, *pm, *pl;  // partial results of the parts
    uint8_t *images;      // widened tiles (k_attn_widen), or null
    int max_tiles;        // of a sequence
    int seq0, seq1;       // the sequences that they are of
};

// A widened tile in memory: what k_attn_rows_many keeps of it in LDS, byte for
// byte: 32 keys, 32 values, the scales of its two runs of 16 tokens.
constexpr int kImageTokens = 32;
constexpr int image_bytes(int D) { return 4 * kImageTokens * D + 64; }

template <int DT>
struct Frag;
template <>
struct Frag<DT_F16> {
    typedef v8h type;
};
template <>
struct Frag<DT_BF16> {
    typedef v8bf type;
};

template <int DT>
__device__ __forceinline__ v4f mfma16(v4i a, v4i b, v4f c)
{
    typedef typename Frag<DT>::type F;
    if constexpr (DT == DT_F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(F, a),
                                                      __builtin_bit_cast(F, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(F, a),
                                                       __builtin_bit_cast(F, b), c, 0, 0, 0);
}

// a signed byte of w as binary32: one instruction with the byte selected in
// its operand (the compiler extracts the byte first)
template <int I>
__device__ __forceinline__ float byte_f(int w)
{
    float f;
    if constexpr (I == 0)
        asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_0" : "=v"(f) : "v"(w));
    else if constexpr (I == 1)
        asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_1" : "=v"(f) : "v"(w));
    else if constexpr (I == 2)
        asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_2" : "=v"(f) : "v"(w));
    else
        asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_3" : "=v"(f) : "v"(w));
    return f;
}

// two integers of at most 8 bits as two 16-bit floats (exact in both types)
template <int DT>
__device__ __forceinline__ int pack_codes(float a, float b)
{
    if constexpr (DT == DT_F16)
        return __builtin_bit_cast(int, __builtin_amdgcn_cvt_pkrtz(a, b));
    else
        return (int)__builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}

// the two 16-bit floats of a dword as binary32
template <int DT>
__device__ __forceinline__ float low_f(unsigned w)
{
    if constexpr (DT == DT_F16)
        return (float)__builtin_bit_cast(v2h, w)[0];
    else
        return __uint_as_float(w << 16);
}
template <int DT>
__device__ __forceinline__ float high_f(unsigned w)
{
    if constexpr (DT == DT_F16)
        return (float)__builtin_bit_cast(v2h, w)[1];
    else
        return __uint_as_float(w & 0xFFFF0000u);
}

// p less one of the two binary16 numbers of w, in one instruction (the
// compiler widens first)
__device__ __forceinline__ float less_low(float p, unsigned w)
{
    float r;
    asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel:[0,0,0] op_sel_hi:[1,0,0]" : "=v"(r) : "v"(w), "v"(p));
    return r;
}
__device__ __forceinline__ float less_high(float p, unsigned w)
{
    float r;
    asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "=v"(r) : "v"(w), "v"(p));
    return r;
}

// 8 codes (two dwords) -> one fragment in their order
template <int DT>
__device__ __forceinline__ v4i widen8(int w0, int w1)
{
    v4i r;
    r[0] = pack_codes<DT>(byte_f<0>(w0), byte_f<1>(w0));
    r[1] = pack_codes<DT>(byte_f<2>(w0), byte_f<3>(w0));
    r[2] = pack_codes<DT>(byte_f<0>(w1), byte_f<1>(w1));
    r[3] = pack_codes<DT>(byte_f<2>(w1), byte_f<3>(w1));
    return r;
}

// byte I of 8 dwords -> one fragment
template <int DT, int I>
__device__ __forceinline__ v4i widen_col(const int (&w)[8])
{
    v4i r;
    for (int j = 0; j < 4; ++j)
        r[j] = pack_codes<DT>(byte_f<I>(w[2 * j]), byte_f<I>(w[2 * j + 1]));
    return r;
}

// the larger of x in lanes that differ in bit 4, or bit 5, of their number
__device__ __forceinline__ float max_of_16s(float x)
{
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}
__device__ __forceinline__ float max_of_halves(float x)
{
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}

// Shares: sequences cut into parts of about one length, one workgroup for each,
// so that none is left with a long sequence while others have ended.  A part
// has up to the shares' mean of tiles of 64 tokens (each sequence at most 16
// rows); the parts number at most shares + sequences.
constexpr int kMinShare = 8;  // tiles: two per wave
constexpr int kMaxShareSeqs = 4096;

struct Seq {
    int t0, n, len;  // first new token, new tokens, length
    int tiles;
};
__device__ __forceinline__ Seq seq_info(const AttnArgs &a, int b)
{
    const AttnDesc &d = a.d;
    Seq s;
    s.t0 = max(d.b.cu[b], 0);
    s.n = (int)min((int64_t)d.b.cu[b + 1], d.b.tokens) - s.t0;
    s.len = max(0, min(min(d.b.len[b], d.b.max_kv), d.c.table_cols * d.c.block_size));
    s.tiles = s.n > 0 ? (s.len + 63) / 64 : 0;
    return s;
}

__device__ __forceinline__ int parts_of(int tiles, int share) { return (tiles + share - 1) / share; }

// The parts' order: the longer ones first for up to kOrdered sequences, where
// few parts share a compute unit, otherwise by sequence.
constexpr int kOrdered = 64;
struct Parts {
    int n;        // sequences per thread
    int share;    // tiles of a part, at most
    int own;      // parts of the thread's sequences, t * n ..
    int length;   // tiles of a part, if n is 1
    Seq s;        // the last of the thread's sequences
};
__device__ __forceinline__ int length_of(int tiles, int parts) { return parts > 0 ? (tiles + parts - 1) / parts : 0; }

// `sums` are 4 ints in LDS; ends with a barrier behind their writing.
__device__ __forceinline__ Parts count_parts(const AttnArgs &a, int *sums)
{
    const int tid = threadIdx.x, S = a.d.b.seqs;
    Parts p;
    p.n = (S + 255) / 256;
    const int first = tid * p.n, last = min(first + p.n, S);
    p.s = {0, 0, 0, 0};
    int x = 0;
    for (int b = first; b < last; ++b) {
        p.s = seq_info(a, b);
        x += p.s.tiles;
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1)
        x += __shfl_xor(x, o);
    if ((tid & 63) == 0)
        sums[tid >> 6] = x;
    __syncthreads();
    const int total = (sums[0] + sums[1]) + (sums[2] + sums[3]);
    p.share = max(kMinShare, (total + a.shares - 1) / a.shares);
    p.own = 0;
    if (p.n == 1)
        p.own = parts_of(p.s.tiles, p.share);
    else
        for (int b = first; b < last; ++b)
            p.own += parts_of(seq_info(a, b).tiles, p.share);
    p.length = length_of(p.s.tiles, p.own);
    return p;
}

// A part's sequence (-1: there is no such part), the part's number there, and
// how many parts the sequence has.
struct Part {
    int seq, index, parts;
    Seq s;
};
__device__ __forceinline__ Part find_part(const AttnArgs &a, int part)
{
    __shared__ int sums[8];
    __shared__ Part found;
    __shared__ __attribute__((aligned(8))) int2 lengths[kOrdered];
    __shared__ int quarter[4][kOrdered];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, S = a.d.b.seqs;
    if (tid == 0)
        found.seq = -1;
    Parts p = count_parts(a, sums);
    int before = 0;
    if (S <= kOrdered) {
        if (tid < kOrdered)
            lengths[tid] = {p.length, p.own};
        __syncthreads();
        // the waves count a quarter each of what comes before sequence `lane`
        const int length = lengths[lane].x;
#pragma unroll 8
        for (int j = wave; j < S; j += 4) {
            const int2 o = lengths[j];
            before += o.x > length || (o.x == length && j < lane) ? o.y : 0;
        }
        quarter[wave][lane] = before;
        __syncthreads();
        before = (quarter[0][lane] + quarter[1][lane]) + (quarter[2][lane] + quarter[3][lane]);
    } else {
        int x = p.own;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int y = __shfl_up(x, o);
            x += lane >= o ? y : 0;
        }
        if (lane == 63)
            sums[4 + wave] = x;
        __syncthreads();
        before = x - p.own;
#pragma unroll
        for (int w = 0; w < 3; ++w)
            before += w < wave ? sums[4 + w] : 0;
    }
    if (part >= before && part < before + p.own) {
        int b = tid * p.n, k = p.own;
        if (p.n > 1)
            for (;; before += k, ++b) {
                p.s = seq_info(a, b);
                k = parts_of(p.s.tiles, p.share);
                if (part < before + k)
                    break;
            }
        found = {b, part - before, k, p.s};
    }
    __syncthreads();
    return found;
}

// 16 rows of one cache head per workgroup (rows are new tokens x the query
// heads of the cache head, heads first): decoding, where the cache's bytes
// bound the call.  The four waves take tiles of 64 tokens in turn, straight
// from memory into the matrix operands (a lane reads KD contiguous bytes of
// its token's key, and VD bytes of four tokens' values), with the next tile's
// bytes on their way while one is multiplied and the block numbers one tile
// further ahead; they join their sums in LDS at the end.
//
// A second product takes what the rounding of a weight to 16 bits left, or the
// weights' rounding would be as large as the result's own: the matrix cores
// idle here anyway.
//
// SHARES: a workgroup per part; k_attn_join adds up sequences of several.
//
// Measured: 64 sequences of 2048 to 8192 tokens, 64 / 8 heads of 128, 128 us,
// 674 MB, 5.3 TB/s (long reads reach 5.5); one of 131071, 32 / 8 heads, in 32
// parts 51 us, 5.3 TB/s, and 4 us for their join.
template <int DT, int D, bool SHARES>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void k_attn_rows16(AttnArgs a)
{
    constexpr int WAVES = 4;
    constexpr int KD = D / 4;    // bytes of a key per lane group
    constexpr int KS = D / 32;   // MFMA steps over d
    constexpr int VD = D / 16;   // values per lane and token, and 16-row tiles of out^T
    constexpr int VW = VD / 4;   // dwords of them
    constexpr float kSlack = 8.0f;  // a maximum may lag by 2^8 before the sums are rescaled
    const AttnDesc &d = a.d;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, g = lane >> 4;
    const int G = a.group, H = d.c.heads, bs = d.c.block_size;
    const int head = SHARES ? blockIdx.x : blockIdx.y;
    int split = blockIdx.z;
    __shared__ float sm[WAVES][16], sl[WAVES][16];
    __shared__ __attribute__((aligned(16))) float so[WAVES][16][D];
    int seq, row0 = 0, parts = a.splits, part = 0;
    Seq cur;
    if constexpr (SHARES) {
        // The first shares go to compute units of their own, the next ones
        // beside them: the longest of these beside the shortest of those.
        part = blockIdx.y < a.shares ? a.shares - 1 - (int)blockIdx.y : blockIdx.y;
        const Part p = find_part(a, part);
        seq = __builtin_amdgcn_readfirstlane(p.seq);
        if (seq < 0)
            return;
        split = __builtin_amdgcn_readfirstlane(p.index);
        parts = __builtin_amdgcn_readfirstlane(p.parts);
        cur = {__builtin_amdgcn_readfirstlane(p.s.t0), __builtin_amdgcn_readfirstlane(p.s.n),
               __builtin_amdgcn_readfirstlane(p.s.len), __builtin_amdgcn_readfirstlane(p.s.tiles)};
    } else if (a.one_tile) {
        seq = blockIdx.x;
        cur = seq_info(a, seq);
    } else {
        const Item it = find_item(d.b.cu, d.b.len, d.b.seqs, d.b.tokens, blockIdx.x, G, 16, a.extra);
        seq = it.seq;
        row0 = it.index * 16;
        cur.t0 = it.t0;
        cur.n = it.t1 - it.t0;
        cur.len = max(0, min(min(it.len, d.b.max_kv), d.c.table_cols * bs));
    }
    const int t0 = cur.t0, n = cur.n, len = cur.len;
    if (row0 >= n * G || n * G > a.few)
        return;
    const int first = len - n;  // place of the first new token
    const int row = row0 + r16;
    const bool live = row < n * G;
    const int tok = live ? row / G : n - 1;
    const int hq = head * G + (live ? row - tok * G : 0);
    // tokens this row sees, and the most and least that the tile's rows do
    const int sees = !live ? 0 : d.causal ? max(0, min(len, first + tok + 1)) : len;
    const int last_tok = min(n - 1, (row0 + 15) / G);
    const int most = d.causal ? max(0, min(len, first + last_tok + 1)) : len;
    const int least = d.causal ? max(0, min(len, first + row0 / G + 1)) : len;
    const int tiles = (most + 63) / 64;
    const int per = (tiles + parts - 1) / parts;
    const int tile0 = split * per, tile1 = min(tiles, tile0 + per);

    // queries: lane group g holds d = g KD .. g KD + KD - 1 of its row
    v4i qf[KS];
    {
        const uint16_t *q = (const uint16_t *)d.Q + (int64_t)(t0 + tok) * d.ldq + hq * D + g * KD;
#pragma unroll
        for (int s = 0; s < KS; ++s)
            qf[s] = *(const v4i *)(q + 8 * s);
    }

    v4f o[VD];
#pragma unroll
    for (int t = 0; t < VD; ++t)
        o[t] = (v4f){0, 0, 0, 0};
    float m = kNothing, y = kNothing, l = 0.0f, R = 1.0f, log2R = 0.0f;

    // a tile's four runs of 16 tokens; runs past the last token re-read the
    // last one (its weights are masked).  Lane 4 k + s looks after run s.
    const int32_t *table = d.c.table + seq * d.c.ld_table;
    const int last_run = (most - 1) & ~15;
    auto run_place = [&](int tile, int s) __attribute__((always_inline)) {
        return min(tile * 64 + 16 * s, last_run);
    };
    auto block_of = [&](int tile) __attribute__((always_inline)) {
        return table[run_place(tile, lane & 3) >> a.block_shift];
    };
    struct Tile {
        v4i k[4][KD / 16];
        int v[4][4][VW];
        float ks, vs;  // lane s: the scales of run s
    };
    const uint32_t klane = r16 * D + g * KD, vlane = 4 * g * D + r16 * VD;
    auto fetch = [&](Tile &x, int tile, int blk_v) __attribute__((always_inline)) {
        const unsigned b = (unsigned)blk_v < a.num_blocks ? (unsigned)blk_v : 0;
        const int64_t mine = (int64_t)b * H + head;
        x.ks = d.c.ks[mine];
        x.vs = d.c.vs[mine];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int64_t bh = (int64_t)(unsigned)__builtin_amdgcn_readlane((int)b, s) * H + head;
            const int64_t base = ((bh << a.block_shift) + (run_place(tile, s) & (bs - 1))) * D;
            const int8_t *kp = d.c.k + base, *vp = d.c.v + base;
#pragma unroll
            for (int i = 0; i < KD / 16; ++i)
                x.k[s][i] = *(const v4i *)(kp + (klane + 16 * i));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (VW == 1) {
                    x.v[s][i][0] = *(const int *)(vp + (vlane + i * D));
                } else if constexpr (VW == 2) {
                    const v2u w = *(const v2u *)(vp + (vlane + i * D));
                    x.v[s][i][0] = (int)w[0];
                    x.v[s][i][1] = (int)w[1];
                } else {
                    const v4i w = *(const v4i *)(vp + (vlane + i * D));
                    for (int e = 0; e < 4; ++e)
                        x.v[s][i][e] = w[e];
                }
            }
        }
    };

    auto attend = [&](auto masked_tag, const Tile &tl, int tile) __attribute__((always_inline)) {
        constexpr bool MASKED = decltype(masked_tag)::value;
        // scores of 16 tokens x 16 rows: lane holds tokens 4 g + e of row r16
        v4f x[4];
        float mt = -INFINITY, yt = -INFINITY, kc[4], vs[4], log2s[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            kc[s] = score_factor(__int_as_float(__builtin_amdgcn_readlane(__float_as_int(tl.ks), s)), a.c2);
            vs[s] = held_scale(__int_as_float(__builtin_amdgcn_readlane(__float_as_int(tl.vs), s)));
            log2s[s] = __builtin_amdgcn_logf(vs[s]);
            x[s] = (v4f){0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const v4i w = tl.k[s][k / 2];
                x[s] = mfma16<DT>(widen8<DT>(w[2 * (k & 1)], w[2 * (k & 1) + 1]), qf[k], x[s]);
            }
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            if constexpr (MASKED) {
                const int j0 = tile * 64 + 16 * s + 4 * g;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[s][e] = j0 + e < sees ? x[s][e] : -INFINITY;
            }
            const float mu = fmaxf(fmaxf(x[s][0], x[s][1]), fmaxf(x[s][2], x[s][3]));
            mt = fmaxf(mt, mu * kc[s]);
            yt = fmaxf(yt, __builtin_fmaf(mu, kc[s], log2s[s]));
        }
        mt = max_of_halves(max_of_16s(mt));
        yt = max_of_halves(max_of_16s(yt));
        // the sums are rescaled when a row's maximum has grown past the slack
        const bool up_m = mt > m + kSlack, up_y = yt > y + kSlack;
        if (__builtin_amdgcn_ballot_w64(up_m || up_y) != 0) {
            const float m1 = up_m ? mt : m, y1 = up_y ? yt : y, f = __builtin_amdgcn_exp2f(y - y1);
            l *= __builtin_amdgcn_exp2f(m - m1);
            m = m1;
            y = y1;
            log2R = y - m;
            R = __builtin_amdgcn_exp2f(log2R);
#pragma unroll
            for (int t = 0; t < VD; ++t)
                for (int e = 0; e < 4; ++e)
                    o[t][e] *= f;
        }
        v4i wf[2], wr[2];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            // weights take 2^lv (value scale / R, lifted), sums take it back
            const float lv = run_shift(log2s[s], log2R);
            const float back = run_back(R, __builtin_amdgcn_rcpf(vs[s]));
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                p[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[s][e], kc[s], lv - m));
            l = __builtin_fmaf((p[0] + p[1]) + (p[2] + p[3]), back, l);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const unsigned w = pack2<DT>(p[2 * e], p[2 * e + 1]);
                wf[s >> 1][2 * (s & 1) + e] = (int)w;
                wr[s >> 1][2 * (s & 1) + e] =
                    (int)pack2<DT>(p[2 * e] - low_f<DT>(w), p[2 * e + 1] - high_f<DT>(w));
            }
        }
        // out^T tile t: rows d = r VD + t for r = 0 .. 15
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
#pragma unroll
            for (int w = 0; w < VW; ++w) {
                int c8[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    c8[i] = tl.v[2 * hh + (i >> 2)][i & 3][w];
                auto add = [&](auto byte) __attribute__((always_inline)) {
                    constexpr int B = decltype(byte)::value;
                    const v4i vf = widen_col<DT, B>(c8);
                    o[4 * w + B] = mfma16<DT>(vf, wf[hh], o[4 * w + B]);
                    o[4 * w + B] = mfma16<DT>(vf, wr[hh], o[4 * w + B]);
                };
                add(std::integral_constant<int, 0>{});
                add(std::integral_constant<int, 1>{});
                add(std::integral_constant<int, 2>{});
                add(std::integral_constant<int, 3>{});
            }
        }
    };

    const int start = tile0 + wave;
    if (start < tile1) {
        Tile ta, tb;
        int blk = block_of(start);
        fetch(ta, start, blk);
        blk = block_of(start + WAVES);
        // The queries are here: said with the builtin, so that the compiler
        // does not wait for them inside the loop, which would wait for the
        // tiles on their way.
        __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) expcnt(7) lgkmcnt(0)
        auto turn = [&](Tile &now, Tile &next, int tile) __attribute__((always_inline)) {
            // past the last tile this fetches the last run again
            fetch(next, tile + WAVES, blk);
            blk = block_of(tile + 2 * WAVES);
            if (tile * 64 + 64 <= least && row0 + 16 <= n * G)
                attend(std::false_type{}, now, tile);
            else
                attend(std::true_type{}, now, tile);
        };
        for (int tile = start;;) {
            turn(ta, tb, tile);
            if ((tile += WAVES) >= tile1)
                break;
            turn(tb, ta, tile);
            if ((tile += WAVES) >= tile1)
                break;
        }
    }
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);

    // ---- join the waves: lane holds out[row r16][d = (4 g + e) VD + t] / R ----
    if (g == 0) {
        sm[wave][r16] = m;
        sl[wave][r16] = l;
    }
    const float f = R * 0x1p-6f;
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int t = 0; t < VD; t += 4)
            *(v4f *)&so[wave][r16][(4 * g + e) * VD + t] =
                (v4f){o[t][e] * f, o[t + 1][e] * f, o[t + 2][e] * f, o[t + 3][e] * f};
    __syncthreads();
    for (int i = tid; i < 16 * (D / 4); i += 256) {
        const int r = i / (D / 4), c = (i % (D / 4)) * 4;
        if (row0 + r >= n * G)
            break;
        float mm = fmaxf(fmaxf(sm[0][r], sm[1][r]), fmaxf(sm[2][r], sm[3][r]));
        float ll = 0.0f;
        v4f oo = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const float e2 = __builtin_amdgcn_exp2f(sm[w][r] - mm);
            ll = __builtin_fmaf(e2, sl[w][r], ll);
            const v4f x = *(const v4f *)&so[w][r][c];
            for (int e = 0; e < 4; ++e)
                oo[e] = __builtin_fmaf(e2, x[e], oo[e]);
        }
        const int tk = (row0 + r) / G, h = head * G + (row0 + r) - tk * G;
        const int64_t orow = (int64_t)(t0 + tk) * d.q_heads + h;
        if (parts == 1) {
            const float inv = ll > 0.0f ? 1.0f / ll : 0.0f;
            const v2u w = {pack2<DT>(oo[0] * inv, oo[1] * inv), pack2<DT>(oo[2] * inv, oo[3] * inv)};
            *(v2u *)((uint16_t *)d.out + (int64_t)(t0 + tk) * d.ldo + h * D + c) = w;
            if (c == 0 && d.lse)
                d.lse[orow] = (mm + __builtin_amdgcn_logf(ll)) * kLn2;
        } else {
            const int64_t prow = SHARES ? ((int64_t)part * H + head) * 16 + r
                                        : (int64_t)split * d.b.tokens * d.q_heads + orow;
            *(v4f *)(a.po + prow * D + c) = oo;
            if (c == 0) {
                a.pm[prow] = mm;
                a.pl[prow] = ll;
            }
        }
    }
}

template <int DT>
__device__ __forceinline__ v16f mfma32(v4i a, v4i b, v16f c)
{
    typedef typename Frag<DT>::type F;
    if constexpr (DT == DT_F16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(F, a),
                                                      __builtin_bit_cast(F, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(F, a),
                                                       __builtin_bit_cast(F, b), c, 0, 0, 0);
}

// Swizzle of 16-byte chunks in LDS rows that are read 32 rows at a time at
// one chunk (lane & 31 the row): the 16 lanes of a read cycle share bit 5 of
// the lane and the parity of bits 2..4, so their rows differ in bits 0, 1
// and (3, 4).  Rows of 256 bytes and more take all four bits; two rows of
// 128 bytes share the 64 banks, their bit 0 already tells them apart, and so
// do bits 0 and 1 of four rows of 64 bytes.
template <int ROW_BYTES>
__device__ __forceinline__ int swz32(int row)
{
    if constexpr (ROW_BYTES >= 256)
        return (row & 3) | (((row >> 3) & 3) << 2);
    else if constexpr (ROW_BYTES == 128)
        return ((row >> 1) & 1) | (((row >> 3) & 3) << 1);
    else
        return (row >> 3) & 3;
}

// ---- tiles of TK (64 or 32) tokens in 16 bits ----
//   * keys: rows of D values by token, in the type of the queries;
//   * values: rows of TK tokens by d, binary16 (the weights that they meet are
//     binary16 too: 11 bits where bfloat16 has 8), the tokens of a row in the
//     order in which a lane's weights sit in its registers: chunk 2 u + h of
//     a row holds tokens 16 u + 4 h + 0..3 and 16 u + 8 + 4 h + 0..3;
//   * 16-byte chunks of a row swizzled by swz32;
//   * per run of 16 tokens: score factor, log2 of the value scale, its
//     reciprocal.
// Widen: WAVES waves bring a tile from the cache into LDS, each TPW tokens.
template <int DT, int D, int WAVES, int TK>
struct Widen {
    static constexpr int KROW = D * 2, VROW = TK * 2, kK = TK * KROW;
    static constexpr int TPW = TK / WAVES;      // 8 or 16 tokens, within one run of 16
    static constexpr int KBL = TPW * D / 64;    // bytes of keys per lane
    static constexpr int KLPT = D / KBL;        // lanes per token
    static constexpr int LPQ = 64 / (TPW / 4);  // lanes per quad of tokens
    static constexpr int VBL = D / LPQ;         // values per lane and token
    typedef typename std::conditional<VBL == 2, uint16_t, int>::type vword;
    static constexpr int VWN = VBL <= 4 ? 1 : VBL / 4;

    const AttnArgs &a;
    const int32_t *table;
    int lane, wtok, run, head, last_run;
    int kreg[KBL / 4];
    vword vreg[4][VWN];
    float scale_k, scale_v;

    __device__ __forceinline__ Widen(const AttnArgs &args, int seq, int h, int most)
        : a(args), table(args.d.c.table + seq * args.d.c.ld_table), lane(threadIdx.x & 63),
          wtok(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * TPW), run(wtok >> 4), head(h),
          last_run((most - 1) & ~15)
    {
    }
    // runs past the last token re-read the last one
    __device__ __forceinline__ int place_of(int tile) const
    {
        return min(tile * TK + 16 * run, last_run) + (wtok & 15);
    }
    // a vector load (`lane >> 6` is 0), so that nothing waits on the scalar
    // counter that the LDS reads use too
    __device__ __forceinline__ int block_of(int tile) const
    {
        return table[(place_of(tile) >> a.block_shift) + (lane >> 6)];
    }
    __device__ __forceinline__ void fetch(int tile, int blk_v)
    {
        const KvCache &c = a.d.c;
        const unsigned b = (unsigned)__builtin_amdgcn_readfirstlane(blk_v);
        const int64_t bh = (int64_t)(b < a.num_blocks ? b : 0) * c.heads + head;
        const int64_t base = ((bh << a.block_shift) + (place_of(tile) & (c.block_size - 1))) * D;
        scale_k = c.ks[bh + (lane >> 6)];
        scale_v = c.vs[bh + (lane >> 6)];
        const int8_t *kp = c.k + base, *vp = c.v + base;
        const uint32_t kl = lane * KBL, vl = 4 * (lane / LPQ) * D + (lane % LPQ) * VBL;
        if constexpr (KBL == 8) {
            const v2u w = *(const v2u *)(kp + kl);
            kreg[0] = (int)w[0];
            kreg[1] = (int)w[1];
        } else {
#pragma unroll
            for (int i = 0; i < KBL / 16; ++i) {
                const v4i w = *(const v4i *)(kp + kl + 16 * i);
                for (int e = 0; e < 4; ++e)
                    kreg[4 * i + e] = w[e];
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int i = 0; i < VWN; ++i)
                vreg[k][i] = *(const vword *)(vp + vl + k * D + 4 * i);
    }
    // what fetch brought, into a tile's LDS; scl: its scales [TK / 16][4]
    __device__ __forceinline__ void stash(uint8_t *tile_lds, float *scl)
    {
        const int tk = wtok + lane / KLPT;
        uint8_t *kr = tile_lds + tk * KROW;
#pragma unroll
        for (int i = 0; i < KBL / 8; ++i) {
            const int c = (lane % KLPT) * (KBL / 8) + i;
            *(v4i *)(kr + ((c ^ swz32<KROW>(tk)) << 4)) = widen8<DT>(kreg[2 * i], kreg[2 * i + 1]);
        }
        const int quad = ((wtok & 15) >> 2) + lane / LPQ;  // quad of the run
        const int c = 2 * run + (quad & 1);
        uint8_t *vr = tile_lds + kK + ((quad >> 1) & 1) * 8;
        auto put = [&](auto byte, int w) __attribute__((always_inline)) {
            constexpr int B = decltype(byte)::value;
            const int dd = (lane % LPQ) * VBL + 4 * w + B;
            v2u x;
            x[0] = pack_codes<DT_F16>(byte_f<B>((int)vreg[0][w]), byte_f<B>((int)vreg[1][w]));
            x[1] = pack_codes<DT_F16>(byte_f<B>((int)vreg[2][w]), byte_f<B>((int)vreg[3][w]));
            *(v2u *)(vr + dd * VROW + ((c ^ swz32<VROW>(dd)) << 4)) = x;
        };
#pragma unroll
        for (int w = 0; w < VWN; ++w) {
            put(std::integral_constant<int, 0>{}, w);
            put(std::integral_constant<int, 1>{}, w);
            if constexpr (VBL >= 4) {
                put(std::integral_constant<int, 2>{}, w);
                put(std::integral_constant<int, 3>{}, w);
            }
        }
        // every wave of a run writes the same scales
        const float sv = held_scale(scale_v);
        if (lane == 0)
            *(v4f *)(scl + 4 * run) = (v4f){score_factor(scale_k, a.c2), __builtin_amdgcn_logf(sv),
                                            __builtin_amdgcn_rcpf(sv), 0.0f};
    }
};

// Widened tiles to memory, once for all of the workgroups that will read
// them: one workgroup per tile, cache head and sequence.
template <int DT, int D>
__global__ __launch_bounds__(256) void k_attn_widen(AttnArgs a)
{
    constexpr int TK = kImageTokens, kTile = 4 * TK * D;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kTile + 64];
    const AttnDesc &d = a.d;
    const int seq = a.seq0 + (int)blockIdx.z, head = blockIdx.y, tile = blockIdx.x;
    const int n = (int)min((int64_t)d.b.cu[seq + 1], d.b.tokens) - max(d.b.cu[seq], 0);
    const int len = max(0, min(min(d.b.len[seq], d.b.max_kv), d.c.table_cols * d.c.block_size));
    if ((int64_t)n * a.group <= a.few || tile * TK >= len)
        return;
    Widen<DT, D, 4, TK> w(a, seq, head, len);
    w.fetch(tile, w.block_of(tile));
    w.stash(lds, (float *)(lds + kTile));
    __syncthreads();
    uint8_t *out = a.images + (((int64_t)blockIdx.z * a.max_tiles + tile) * d.c.heads + head) * image_bytes(D);
    for (int i = threadIdx.x * 16; i < kTile + 64; i += 256 * 16)
        *(v4i *)(out + i) = *(const v4i *)(lds + i);
}

// Many rows per cache head: WAVES waves of 32 rows each walk the same tiles of
// TK tokens through two buffers in LDS, one barrier per tile.  K Q^T (32
// tokens x 32 rows per matrix instruction) leaves a lane one row and half of
// the tokens, so a row's maximum takes one exchange between lane halves and
// its sum none until the end.
//
// READY: the tiles come widened (k_attn_widen) by direct-to-LDS loads, for
// prompts whose many workgroups would each widen the same tile.  Workgroups of
// 4 waves share a compute unit and drift apart, so that one's matrix products
// run beside another's softmax, where 8 waves that meet at one barrier stay in
// step; tiles of 32 tokens leave room for three (D = 128) or four (64).
// Otherwise 8 waves widen each tile of 64 once for 256 rows.
//
// Measured: a prompt of 8192 tokens, 32 / 8 heads of 128, causal, READY: 555 to
// 585 us by board (14 of them k_attn_widen), 550 GFLOP, 0.94 to 0.99 PFLOP/s.
// The matrix cores are busy 53% of the cycles, the softmax's and the scales'
// vector work most of the rest (alone it takes 219 us), and the clock settles
// at 1.8 GHz; a large bfloat16 product on this card reaches 1.41 PFLOP/s.
constexpr int kReadyWaves = 4;
// waves per SIMD that the registers are shared out for
constexpr int min_waves(int D, bool ready) { return D == 256 ? 1 : !ready ? 2 : D == 128 ? 3 : 4; }
template <int DT, int D, int WAVES, bool READY>
__global__ __launch_bounds__(WAVES * 64, min_waves(D, READY)) void k_attn_rows_many(AttnArgs a)
{
    constexpr int TK = READY ? kImageTokens : 64, NT = TK / 32, NU = TK / 16;
    constexpr int ROWS = WAVES * 32;
    constexpr int KROW = D * 2, VROW = TK * 2;
    constexpr int KS = D / 16;   // matrix steps over d
    constexpr int DT32 = D / 32; // 32-row tiles of out^T
    constexpr int kK = TK * KROW, kTile = kK + D * VROW;
    constexpr int kBuf = kTile + 1024;  // a tile and its scales, whole kilobytes
    // A weight's rounding to binary16 is an eighth of the rounding of a
    // bfloat16 result but as large as that of a binary16 one (error against 64
    // bits 0.00037, the result's own rounding 0.00021): there a second product
    // takes its rest.  It costs a binary16 prompt of 8192 tokens 190 us (837
    // instead of 647 on one board; 776 on another, bfloat16 584).
    constexpr bool REST = DT == DT_F16;
    constexpr float kSlack = 8.0f;  // a maximum may lag by 2^8 before the sums are rescaled
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kBuf];

    const AttnDesc &d = a.d;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r32 = lane & 31, h = lane >> 5;
    const int G = a.group, H = d.c.heads, bs = d.c.block_size;
    // A tile's heads are neighbours in the grid.  The last rows see the most
    // tokens: they start first.
    const int back = (gridDim.x - 1 - blockIdx.x) / H, split = blockIdx.y;
    const int head = (gridDim.x - 1 - blockIdx.x) - back * H;

    const Item it = find_item(d.b.cu, d.b.len, d.b.seqs, d.b.tokens, back, G, ROWS, a.extra);
    const int t0 = it.t0, n = it.t1 - t0, row0 = it.index * ROWS;
    if (row0 >= n * G || n * G <= a.few)
        return;
    if (READY && (it.seq < a.seq0 || it.seq >= a.seq1))
        return;
    const int len = max(0, min(min(it.len, d.b.max_kv), d.c.table_cols * bs));
    const int first = len - n;
    auto sees_of = [&](int row) {  // tokens that a row of the sequence sees
        return row >= n * G ? 0 : d.causal ? max(0, min(len, first + row / G + 1)) : len;
    };
    const int most = sees_of(min(row0 + ROWS, n * G) - 1);
    const int tiles = (most + TK - 1) / TK;
    const int per = (tiles + a.splits - 1) / a.splits;
    const int tile0 = split * per, tile1 = min(tiles, tile0 + per);

    // this wave's rows
    const int wrow0 = row0 + wave * 32;
    const int wmost = wrow0 < n * G ? sees_of(min(wrow0 + 32, n * G) - 1) : 0;
    const int wleast = wrow0 + 32 <= n * G ? sees_of(wrow0) : 0;  // tiles below need no mask
    const int row = wrow0 + r32;
    const int sees = sees_of(row);
    const int tok = min(row, n * G - 1) / G, hq = head * G + min(row, n * G - 1) - tok * G;
    v4i qf[KS];
    {
        const uint16_t *q = (const uint16_t *)d.Q + (int64_t)(t0 + tok) * d.ldq + hq * D + 8 * h;
#pragma unroll
        for (int s = 0; s < KS; ++s)
            qf[s] = *(const v4i *)(q + 16 * s);
    }

    v16f o[DT32];
#pragma unroll
    for (int t = 0; t < DT32; ++t)
        for (int e = 0; e < 16; ++e)
            o[t][e] = 0.0f;
    float m = kNothing, y = kNothing, l = 0.0f, R = 1.0f, log2R = 0.0f;

    // LDS offsets of this lane's fragments: chunk 2 s + h of row r32 (and of
    // rows 32, 64, .. further, which swizzle alike) is at place ^ 32 s
    const int kplace = r32 * KROW + ((h ^ swz32<KROW>(r32)) << 4);
    const int vplace = r32 * VROW + ((h ^ swz32<VROW>(r32)) << 4);

    auto attend = [&](auto masked_tag, int tile, int buf) __attribute__((always_inline)) {
        constexpr bool MASKED = decltype(masked_tag)::value;
        const uint8_t *sk = lds + buf * kBuf, *sv = sk + kK;
        const float *scl = (const float *)(sk + kTile);
        v4f sc[NU];  // of a run: score factor, log2 of the value scale, its reciprocal
#pragma unroll
        for (int u = 0; u < NU; ++u)
            sc[u] = *(const v4f *)(scl + 4 * u);
        // fragments are read one step ahead of their products; the first ones
        // of the values go out before the softmax
        auto read_k = [&](int s, v4i(&f)[NT]) __attribute__((always_inline)) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
                f[t] = *(const v4i *)(sk + (kplace ^ (s << 5)) + t * 32 * KROW);
        };
        auto read_v = [&](int u, v4i(&f)[DT32]) __attribute__((always_inline)) {
#pragma unroll
            for (int t = 0; t < DT32; ++t)
                f[t] = *(const v4i *)(sv + (vplace ^ (u << 5)) + t * 32 * VROW);
        };
        v4i wf[NU], wr[NU], kf[2][NT], vf[2][DT32];
        v16f x[NT];
        read_k(0, kf[0]);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            if (s + 1 < KS)
                read_k(s + 1, kf[(s + 1) & 1]);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const v16f zero = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
                x[t] = mfma32<DT>(kf[s & 1][t], qf[s], s == 0 ? zero : x[t]);
            }
        }
        read_v(0, vf[0]);
        if constexpr (MASKED) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int j = tile * TK + 32 * t + 8 * (e >> 2) + 4 * h + (e & 3);
                    x[t][e] = j < sees ? x[t][e] : -INFINITY;
                }
        }
        float mt = -INFINITY, yt = -INFINITY;
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            float mu = x[u >> 1][8 * (u & 1)];
#pragma unroll
            for (int e = 1; e < 8; ++e)
                mu = fmaxf(mu, x[u >> 1][8 * (u & 1) + e]);
            mt = fmaxf(mt, mu * sc[u][0]);
            yt = fmaxf(yt, __builtin_fmaf(mu, sc[u][0], sc[u][1]));
        }
        mt = max_of_halves(mt);
        yt = max_of_halves(yt);
        // the sums are rescaled when a row's maximum has grown past the slack
        const bool up_m = mt > m + kSlack, up_y = yt > y + kSlack;
        if (__builtin_amdgcn_ballot_w64(up_m || up_y) != 0) {
            const float m1 = up_m ? mt : m, y1 = up_y ? yt : y, f = __builtin_amdgcn_exp2f(y - y1);
            l *= __builtin_amdgcn_exp2f(m - m1);
            m = m1;
            y = y1;
            log2R = y - m;
            R = __builtin_amdgcn_exp2f(log2R);
#pragma unroll
            for (int t = 0; t < DT32; ++t)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    o[t][e] *= f;
        }
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            // weights take 2^b (value scale / R, lifted), sums take it back
            const float b = run_shift(sc[u][1], log2R) - m;
            const float back = run_back(R, sc[u][2]);
            float p[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                p[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[u >> 1][8 * (u & 1) + e], sc[u][0], b));
            const float sum = ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
            l = __builtin_fmaf(sum, back, l);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const unsigned w = pack2<DT_F16>(p[2 * e], p[2 * e + 1]);
                wf[u][e] = (int)w;
                if constexpr (REST)
                    wr[u][e] = (int)pack2<DT_F16>(less_low(p[2 * e], w), less_high(p[2 * e + 1], w));
            }
        }
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            if (u + 1 < NU)
                read_v(u + 1, vf[(u + 1) & 1]);
#pragma unroll
            for (int t = 0; t < DT32; ++t)
                o[t] = mfma32<DT_F16>(vf[u & 1][t], wf[u], o[t]);
            if constexpr (REST)
#pragma unroll
                for (int t = 0; t < DT32; ++t)
                    o[t] = mfma32<DT_F16>(vf[u & 1][t], wr[u], o[t]);
        }
    };
    // the tile's bytes are there (this wave's loads), its LDS work is done,
    // then the other waves'
    auto meet = [&]() __attribute__((always_inline)) {
        __builtin_amdgcn_s_waitcnt(READY ? 0x0070 : 0xC07F);  // [vmcnt(0)] lgkmcnt(0)
        asm volatile("s_barrier" ::: "memory");
    };
    // tiles that all of the wave's rows see whole, then the others (two loops:
    // with both forms in one, the compiler keeps two copies of the sums);
    // every wave passes the same number of barriers
    auto walk = [&](auto before, auto after) __attribute__((always_inline)) {
        const int whole = max(tile0, min(tile1, wleast / TK));
        int tile = tile0;
        for (; tile < whole; ++tile) {
            before(tile);
            attend(std::false_type{}, tile, (tile - tile0) & 1);
            after(tile);
        }
        for (; tile < tile1; ++tile) {
            before(tile);
            if (tile * TK < wmost)
                attend(std::true_type{}, tile, (tile - tile0) & 1);
            after(tile);
        }
    };
    if (tile0 < tile1) {
        if constexpr (READY) {
            const int64_t step = (int64_t)H * image_bytes(D);
            const uint8_t *img = a.images + ((int64_t)(it.seq - a.seq0) * a.max_tiles * H + head) * image_bytes(D);
            auto load = [&](int tile) __attribute__((always_inline)) {
                const uint8_t *src = img + tile * step;
                uint8_t *dst = lds + ((tile - tile0) & 1) * kBuf;
#pragma unroll
                for (int i = 0; i < (kTile / 1024 + WAVES - 1) / WAVES; ++i) {
                    const int off = (i * WAVES + wave) * 1024;
                    if (kTile / 1024 % WAVES != 0 && off >= kTile)
                        break;
                    buffer_load_lds16(src, kTile, lane * 16, off, dst + off);
                }
                if (wave == 0 && lane < 4 * NU)
                    __builtin_amdgcn_global_load_lds((const glb_void_t *)(src + kTile + lane * 4),
                                                     (lds_void_t *)(dst + kTile), 4, 0, 0);
            };
            load(tile0);
            meet();
            walk(
                [&](int tile) __attribute__((always_inline)) {
                    if (tile + 1 < tile1)
                        load(tile + 1);
                },
                [&](int) __attribute__((always_inline)) { meet(); });
        } else {
            Widen<DT, D, WAVES, TK> w(a, it.seq, head, most);
            w.fetch(tile0, w.block_of(tile0));
            w.stash(lds, (float *)(lds + kTile));
            int next = w.block_of(tile0 + 1);
            __syncthreads();
            // past the last tile this fetches the last one again
            walk(
                [&](int tile) __attribute__((always_inline)) {
                    w.fetch(tile + 1, next);
                    next = w.block_of(tile + 2);
                },
                [&](int tile) __attribute__((always_inline)) {
                    uint8_t *dst = lds + ((tile + 1 - tile0) & 1) * kBuf;
                    w.stash(dst, (float *)(dst + kTile));
                    meet();
                });
        }
    }

    // lane: row r32 of 32, d = 32 t + 8 (e / 4) + 4 h + e % 4
    l += __shfl_xor(l, 32);
    if (row >= n * G)
        return;
    const int64_t orow = (int64_t)(t0 + tok) * d.q_heads + hq;
    const float f = R * 0x1p-6f;
    if (a.splits == 1) {
        const float inv = l > 0.0f ? f / l : 0.0f;
        uint16_t *dst = (uint16_t *)d.out + (int64_t)(t0 + tok) * d.ldo + hq * D + 4 * h;
#pragma unroll
        for (int t = 0; t < DT32; ++t)
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                const v2u w = {pack2<DT>(o[t][e] * inv, o[t][e + 1] * inv),
                               pack2<DT>(o[t][e + 2] * inv, o[t][e + 3] * inv)};
                *(v2u *)(dst + 32 * t + 2 * e) = w;
            }
        if (h == 0 && d.lse)
            d.lse[orow] = (m + __builtin_amdgcn_logf(l)) * kLn2;
    } else {
        const int64_t prow = (int64_t)split * d.b.tokens * d.q_heads + orow;
        float *dst = a.po + prow * D + 4 * h;
#pragma unroll
        for (int t = 0; t < DT32; ++t)
#pragma unroll
            for (int e = 0; e < 16; e += 4)
                *(v4f *)(dst + 32 * t + 2 * e) =
                    (v4f){o[t][e] * f, o[t][e + 1] * f, o[t][e + 2] * f, o[t][e + 3] * f};
        if (h == 0) {
            a.pm[prow] = m;
            a.pl[prow] = l;
        }
    }
}

// Joins the parts of split sequences: one workgroup per row, 256 threads as
// 256 / (D / 4) groups that each sum every so many parts (few rows over many
// parts would wait for one load after the other), then add up in LDS.
constexpr int kMaxSplits = 256;
template <int DT, int D>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a)
{
    constexpr int LANES = D / 4, PARTS = 256 / LANES;
    __shared__ float sw[kMaxSplits], sred[4];
    __shared__ __attribute__((aligned(16))) v4f so[PARTS][LANES];
    const AttnDesc &d = a.d;
    const int tid = threadIdx.x, c = tid % LANES, part = tid / LANES;
    const int64_t rows = d.b.tokens * d.q_heads, row = blockIdx.x;
    const float pm = tid < a.splits ? a.pm[tid * rows + row] : -INFINITY;
    const float pl = tid < a.splits ? a.pl[tid * rows + row] : 0.0f;
    float mm = pm;
#pragma unroll
    for (int i = 1; i < 64; i <<= 1)
        mm = fmaxf(mm, __shfl_xor(mm, i));
    if ((tid & 63) == 0)
        sred[tid >> 6] = mm;
    __syncthreads();
    mm = fmaxf(fmaxf(sred[0], sred[1]), fmaxf(sred[2], sred[3]));
    const float w = __builtin_amdgcn_exp2f(pm - (mm == -INFINITY ? 0.0f : mm));
    sw[tid] = w;
    float ll = w * pl;
#pragma unroll
    for (int i = 1; i < 64; i <<= 1)
        ll += __shfl_xor(ll, i);
    __syncthreads();
    if ((tid & 63) == 0)
        sred[tid >> 6] = ll;
    v4f oo = {0, 0, 0, 0};
    const float *po = a.po + row * D + 4 * c;
#pragma unroll 8
    for (int s = part; s < a.splits; s += PARTS) {
        const v4f x = *(const v4f *)(po + s * rows * D);
        const float f = sw[s];
        for (int e = 0; e < 4; ++e)
            oo[e] = __builtin_fmaf(f, x[e], oo[e]);
    }
    so[part][c] = oo;
    __syncthreads();
    if (part != 0)
        return;
#pragma unroll
    for (int p = 1; p < PARTS; ++p) {
        const v4f x = so[p][c];
        for (int e = 0; e < 4; ++e)
            oo[e] += x[e];
    }
    ll = (sred[0] + sred[1]) + (sred[2] + sred[3]);
    const float inv = ll > 0.0f ? 1.0f / ll : 0.0f;
    const int tok = (int)(row / d.q_heads), h = (int)(row - (int64_t)tok * d.q_heads);
    const v2u y = {pack2<DT>(oo[0] * inv, oo[1] * inv), pack2<DT>(oo[2] * inv, oo[3] * inv)};
    *(v2u *)((uint16_t *)d.out + (int64_t)tok * d.ldo + h * D + 4 * c) = y;
    if (c == 0 && d.lse)
        d.lse[row] = (mm + __builtin_amdgcn_logf(ll)) * kLn2;
}

// Joins the parts of sequences of several and writes the rows of those of no
// tokens: a workgroup per sequence and cache head, its waves a row at a time.
template <int DT, int D>
__global__ __launch_bounds__(256) void k_attn_join_parts(AttnArgs a)
{
    constexpr int LANES = D / 4, GROUPS = 64 / LANES;
    __shared__ int sums[8];
    const AttnDesc &d = a.d;
    const int tid = threadIdx.x, lane = tid & 63, c = lane % LANES, group = lane / LANES;
    const int seq = blockIdx.y, head = blockIdx.x;
    const Seq me = seq_info(a, seq);
    const Parts p = count_parts(a, sums);
    const int parts = parts_of(me.tiles, p.share), length = length_of(me.tiles, parts);
    if (parts == 1)
        return;
    // the parts before this sequence's
    int x = 0;
    if (p.n == 1)
        x = d.b.seqs <= kOrdered && p.length != length ? (p.length > length ? p.own : 0)
            : tid < seq                                ? p.own
                                                       : 0;
    else
        for (int b = tid * p.n; b < min(seq, (tid + 1) * p.n); ++b)
            x += parts_of(seq_info(a, b).tiles, p.share);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1)
        x += __shfl_xor(x, o);
    if (lane == 0)
        sums[4 + (tid >> 6)] = x;
    __syncthreads();
    const int before = (sums[4] + sums[5]) + (sums[6] + sums[7]);
    const int64_t stride = d.c.heads * 16;
    for (int r = tid >> 6; r < min(16, me.n * a.group); r += 4) {
        const int tok = me.t0 + r / a.group, h = head * a.group + r % a.group;
        const int64_t part0 = ((int64_t)before * d.c.heads + head) * 16 + r;
        float pm[kMaxSplits / 64], mm = -INFINITY, ll = 0.0f;
#pragma unroll
        for (int j = 0; j < kMaxSplits / 64; ++j) {
            pm[j] = lane + 64 * j < parts ? a.pm[part0 + (lane + 64 * j) * stride] : -INFINITY;
            mm = fmaxf(mm, pm[j]);
        }
#pragma unroll
        for (int i = 1; i < 64; i <<= 1)
            mm = fmaxf(mm, __shfl_xor(mm, i));
        v4f oo = {0, 0, 0, 0};
        const float *po = a.po + part0 * D + 4 * c;
#pragma unroll
        for (int j = 0; j < kMaxSplits / 64; ++j) {
            const int n = min(parts - 64 * j, 64);
            if (n <= 0)
                break;
            const float w = __builtin_amdgcn_exp2f(pm[j] - (mm == -INFINITY ? 0.0f : mm));
            if (lane < n)
                ll = __builtin_fmaf(w, a.pl[part0 + (lane + 64 * j) * stride], ll);
#pragma unroll 8
            for (int s = 0; s < n; s += GROUPS) {
                const int k = s + group;
                const float f = __shfl(w, k < n ? k : 0);
                if (k < n) {
                    const v4f x = *(const v4f *)(po + (k + 64 * j) * stride * D);
                    for (int e = 0; e < 4; ++e)
                        oo[e] = __builtin_fmaf(f, x[e], oo[e]);
                }
            }
        }
#pragma unroll
        for (int i = 1; i < 64; i <<= 1)
            ll += __shfl_xor(ll, i);
#pragma unroll
        for (int i = LANES; i < 64; i <<= 1)
            for (int e = 0; e < 4; ++e)
                oo[e] += __shfl_xor(oo[e], i);
        if (group == 0) {
            const float inv = ll > 0.0f ? 1.0f / ll : 0.0f;
            const v2u y = {pack2<DT>(oo[0] * inv, oo[1] * inv), pack2<DT>(oo[2] * inv, oo[3] * inv)};
            *(v2u *)((uint16_t *)d.out + (int64_t)tok * d.ldo + h * D + 4 * c) = y;
            if (c == 0 && d.lse)
                d.lse[(int64_t)tok * d.q_heads + h] = (mm + __builtin_amdgcn_logf(ll)) * kLn2;
        }
    }
}

// sequences of up to this many rows (new tokens x query heads per cache head)
// take the 16-row kernel
constexpr int kFew = 32;
// Up to 16 rows per sequence and several sequences: parts (k_attn_rows16,
// SHARES) where sequences would be cut anyway, and for a cache of so many
// tokens, from where unlike lengths cost more than the look-up and the join
// (us, head size 128, with and without parts):
//   64 / 8 heads: 64 sequences of 2048 to 8192 tokens 128 and 148, 64 of 5120
//   126 and 122, 32 of 5120 64 and 60
//   32 / 8 heads: one of 131071 and 63 of 100 66 and 1610; 64 of 768 to 3000
//   51 and 56, 64 of 1875 50 and 46; 32 of 512 to 2048 29 and 24
// 256 shares, one per compute unit: 512 of them 156 instead of 153, 1024 160
// (64 sequences of 2048 to 8192, not yet in order of length).
constexpr int kShares = 256;
constexpr int kShareTokens = 4096;
// Tiles are widened to memory first for sequences of at least so many rows,
// and of no fewer rows than cached tokens (us, one sequence, new tokens +
// cached before, query heads / cache heads; with and without):
//   4096 + 0, 32 / 8: D 64 114 and 137, D 128 174 and 193; D 256, 16 / 4 268 and 284
//   256 + 500, 32 / 8, D 128: 28 and 33
//   512 + 8000, 32 / 8, D 128: 129 and 115
constexpr int kReadyRows = 1024;
// They take twice a 16-bit cache's bytes, every sequence as long as max_kv.  Of
// several, one prompt among decoding steps would make nearly all of that
// padding: past 64 MB the new tokens must be a quarter of the padded ones (one
// of 8192 and 127 decoding: 1120 us and no workspace, 1065 and 4.1 GB).  The
// workspace has room for 1 GB, which slices of the sequences use in turn (64
// prompts of 4096 to 16384 in 5 slices).
constexpr int64_t kSmallImages = (int64_t)1 << 26;  // bytes
constexpr int64_t kMaxImages = (int64_t)1 << 30;

struct Plan {
    int64_t top;    // rows of a sequence, at most
    bool many;      // some sequence may take the many-row kernel
    bool ready;     // its tiles come widened
    int rows;       // rows of its workgroups
    int max_tiles;
    int slice;      // sequences whose widened tiles there is room for at a time
    int64_t images; // bytes of them
    int splits;
    int shares;
    int64_t part_rows;  // rows of parts
    int64_t bytes;  // workspace
};

// Everything that the sizes of a call decide.
Plan plan(int64_t tokens, int seqs, int max_q, int max_kv, int q_heads, int kv_heads, int D)
{
    Plan p{};
    const int64_t group = q_heads / kv_heads;
    p.top = (max_q < tokens ? max_q : tokens) * group;
    p.many = p.top > kFew;
    p.max_tiles = (int)(((int64_t)max_kv + kImageTokens - 1) / kImageTokens);
    const int64_t image = (int64_t)p.max_tiles * kv_heads * image_bytes(D);  // of a sequence
    p.ready = max_kv > 0 && p.top >= kReadyRows && p.top >= max_kv && image <= kMaxImages && seqs <= 65535 &&
              (seqs == 1 || seqs * image <= kSmallImages || (int64_t)seqs * max_kv <= 4 * tokens);
    if (p.ready) {
        p.slice = seqs > kMaxImages / image ? (int)(kMaxImages / image) : seqs;
        p.images = p.slice * image;
    }
    p.rows = p.ready ? 32 * kReadyWaves : D == 256 ? 128 : 256;
    // Parts per sequence: enough workgroups for the chip, each of 512 tokens
    // or more.  Few rows: one workgroup per compute unit keeps enough bytes in
    // flight, and each start and join costs several microseconds (one
    // sequence of 131071 tokens, 32 / 8 heads: 256 workgroups 56 us, 512 59,
    // 1024 63, 2048 72).
    const int64_t wgs = (p.top <= 16 ? seqs : tokens * group / (p.many ? p.rows : 16) + seqs) * kv_heads;
    const int64_t most = (int64_t)max_kv / 512;
    const int64_t want = ((p.many ? 512 : 256) + wgs - 1) / wgs;
    int64_t n = want < most ? want : most;
    if (n > kMaxSplits)
        n = kMaxSplits;
    p.splits = n < 1 ? 1 : (int)n;
    if (p.top <= 16 && seqs > 1 && (p.splits > 1 || max_kv >= kShareTokens) && seqs <= kMaxShareSeqs &&
        (int64_t)seqs * kv_heads <= kMaxShareSeqs && (int64_t)seqs * max_kv < (int64_t)1 << 36) {
        p.splits = 1;
        p.shares = kShares / kv_heads;
        p.shares = p.shares < 1 ? 1 : p.shares > kMaxSplits ? kMaxSplits : p.shares;
    }
    p.part_rows = p.shares ? (int64_t)(p.shares + seqs) * kv_heads * 16
                           : p.splits == 1 ? 0 : p.splits * tokens * q_heads;
    p.bytes = p.images + p.part_rows * (D + 2) * 4;
    return p;
}

template <int DT, int D>
void launch_rows(const AttnArgs &a, const Plan &p, bool any_few, hipStream_t s)
{
    const AttnDesc &d = a.d;
    const int64_t rows = d.b.tokens * a.group;
    if (p.many) {
        const dim3 grid((unsigned)((rows / p.rows + (int64_t)a.extra * d.b.seqs) * d.c.heads),
                        (unsigned)a.splits);
        if (p.ready) {
            for (AttnArgs b = a; b.seq0 < d.b.seqs; b.seq0 = b.seq1) {
                b.seq1 = b.seq0 + p.slice < d.b.seqs ? b.seq0 + p.slice : d.b.seqs;
                hipLaunchKernelGGL((k_attn_widen<DT, D>),
                                   dim3((unsigned)p.max_tiles, (unsigned)d.c.heads, (unsigned)(b.seq1 - b.seq0)),
                                   dim3(256), 0, s, b);
                hipLaunchKernelGGL((k_attn_rows_many<DT, D, kReadyWaves, true>), grid,
                                   dim3(64 * kReadyWaves), 0, s, b);
            }
        } else {
            constexpr int WAVES = D == 256 ? 4 : 8;
            hipLaunchKernelGGL((k_attn_rows_many<DT, D, WAVES, false>), grid, dim3(WAVES * 64), 0, s, a);
        }
    }
    if (p.shares) {
        hipLaunchKernelGGL((k_attn_rows16<DT, D, true>), dim3((unsigned)d.c.heads, (unsigned)(p.shares + d.b.seqs)),
                           dim3(256), 0, s, a);
        hipLaunchKernelGGL((k_attn_join_parts<DT, D>),
                           dim3((unsigned)d.c.heads, (unsigned)d.b.seqs), dim3(256), 0, s, a);
        return;
    }
    if (any_few) {
        const dim3 grid((unsigned)(a.one_tile ? d.b.seqs : rows / 16 + (int64_t)a.extra * d.b.seqs),
                        (unsigned)d.c.heads, (unsigned)a.splits);
        hipLaunchKernelGGL((k_attn_rows16<DT, D, false>), grid, dim3(256), 0, s, a);
    }
    if (a.splits > 1)
        hipLaunchKernelGGL((k_attn_join<DT, D>), dim3((unsigned)(d.b.tokens * d.q_heads)), dim3(256),
                           0, s, a);
}

template <int DT>
hipError_t run_attn(const AttnArgs &a, const Plan &p, hipStream_t s)
{
    const AttnDesc &d = a.d;
    // Sequences of more than `few` rows take the many-row kernel.  When every
    // sequence has max_q new tokens only one of the two can have work.
    const bool any_few = !p.many || d.b.tokens != (int64_t)d.b.max_q * d.b.seqs;
    if (d.c.head_dim == 64)
        launch_rows<DT, 64>(a, p, any_few, s);
    else if (d.c.head_dim == 128)
        launch_rows<DT, 128>(a, p, any_few, s);
    else
        launch_rows<DT, 256>(a, p, any_few, s);
    return hipGetLastError();
}

}  // namespace

int64_t attn_workspace_bytes(int64_t tokens, int seqs, int max_q, int max_kv, int q_heads,
                             int kv_heads, int head_dim)
{
    return plan(tokens, seqs, max_q, max_kv, q_heads, kv_heads, head_dim).bytes;
}

hipError_t launch_attn_kv8(const AttnDesc &d, hipStream_t s)
{
    const Plan p = plan(d.b.tokens, d.b.seqs, d.b.max_q, d.b.max_kv, d.q_heads, d.c.heads,
                        d.c.head_dim);
    AttnArgs a{};
    a.d = d;
    a.group = d.q_heads / d.c.heads;
    a.splits = p.splits;
    a.shares = p.shares;
    a.extra = 1;
    a.few = kFew;
    a.one_tile = p.top <= 16;
    a.c2 = d.scale < 2.0e38f ? d.scale * kLog2e : 3.4e38f;  // finite
    a.block_shift = __builtin_ctz((unsigned)d.c.block_size);
    a.num_blocks = (unsigned)d.c.num_blocks;
    a.images = (uint8_t *)d.workspace;
    a.max_tiles = p.max_tiles;
    a.po = (float *)((uint8_t *)d.workspace + p.images);
    a.pm = a.po + p.part_rows * d.c.head_dim;
    a.pl = a.pm + p.part_rows;
    return d.dtype == DT_F16 ? run_attn<DT_F16>(a, p, s) : run_attn<DT_BF16>(a, p, s);
}

}  // namespace qg
