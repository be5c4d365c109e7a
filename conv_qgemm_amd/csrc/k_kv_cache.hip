// k_kv_cache.hip -- writing new keys and values to the paged int8 cache, with
// the position rotation on the way, and reading cached values back.
//
// Rotation: a pair (a, b) of a head at position p becomes (a c - b s,
// b c + a s) with the cosine c and sine s of the pair's angle at p, each
// operation rounded to binary32 by itself, so that the result does not
// depend on how the compiler contracts it.
//
// Coding: one scale per (block of the cache, head), that of the largest
// value the block holds: scale' = max(scale, max |x| / 127).  A scale only
// grows while a block fills, so tokens that are there already are recoded
// (code * scale / scale', rounded) only when a new value exceeds all earlier
// ones.  One workgroup owns a (block, head) of a call, so there are no
// atomics and the result does not depend on any order.
#include "kv_common.hpp"
#include "launch.hpp"

namespace qg {

namespace {

constexpr int kThreads = 256;

struct AppendArgs {
    AppendDesc d;
    int extra;        // find_item
    int block_shift;  // log2 of the block size
    int kv_wgs;       // workgroups that write keys and values; the rest rotate queries
    int q_tokens;     // tokens per workgroup that rotates queries
    int unit_shift;   // log2 of the units of 16 values of a head
};

// The sequence of token t, for the wave's first token by a search of the
// whole wave (64 candidates per step), then walking on.
__device__ __forceinline__ int first_seq(const int32_t *cu, int seqs, int t)
{
    const int lane = threadIdx.x & 63;
    int lo = 0, stride = 1;
    while (64 * stride < seqs)
        stride *= 64;
    for (;; stride /= 64) {
        const int b = lo + lane * stride;
        const int below = __builtin_popcountll(
            __builtin_amdgcn_ballot_w64(b < seqs && cu[min(b, seqs - 1)] <= t));
        lo += max(below - 1, 0) * stride;
        if (stride == 1)
            return lo;
    }
}
__device__ __forceinline__ int seq_of(const int32_t *cu, int seqs, int t, int seq)
{
    while (seq + 1 < seqs && cu[seq + 1] <= t)
        ++seq;
    return seq;
}

// The 16 values that one unit of a head's row covers: two runs of 8, which
// are the two halves of 8 pairs (rotation by halves), 8 pairs (interleaved),
// or unrotated values.
__device__ __forceinline__ void unit_places(int u, int rot, bool inter, int &e0, int &e1)
{
    if (u * 16 < rot && !inter) {
        e0 = u * 8;
        e1 = u * 8 + rot / 2;
    } else {
        e0 = u * 16;
        e1 = u * 16 + 8;
    }
}

// x0, x1: the unit's two runs; cs: row of the table for the token's position
__device__ __forceinline__ void rotate_unit(float (&x0)[8], float (&x1)[8], int u, int rot,
                                            bool inter, const float *cs)
{
#pragma clang fp contract(off)
    if (u * 16 >= rot)
        return;
    float c[8], s[8];
    load8<DT_F32>(cs + u * 8, c);
    load8<DT_F32>(cs + rot / 2 + u * 8, s);
    if (inter) {
        for (int i = 0; i < 4; ++i) {
            const float a = x0[2 * i], b = x0[2 * i + 1];
            x0[2 * i] = a * c[i] - b * s[i];
            x0[2 * i + 1] = b * c[i] + a * s[i];
            const float a1 = x1[2 * i], b1 = x1[2 * i + 1];
            x1[2 * i] = a1 * c[4 + i] - b1 * s[4 + i];
            x1[2 * i + 1] = b1 * c[4 + i] + a1 * s[4 + i];
        }
    } else {
        for (int i = 0; i < 8; ++i) {
            const float a = x0[i], b = x1[i];
            x0[i] = a * c[i] - b * s[i];
            x1[i] = b * c[i] + a * s[i];
        }
    }
}

__device__ __forceinline__ v2u pack8_codes(const float (&f)[8])
{
    v2u w;
    w[0] = pack4_i8((int)f[0], (int)f[1], (int)f[2], (int)f[3]);
    w[1] = pack4_i8((int)f[4], (int)f[5], (int)f[6], (int)f[7]);
    return w;
}

// One unit per thread at a time: the registers of more would cost the keys'
// and values' workgroups of the same kernel their places on the chip.
template <int DT>
__device__ void rotate_queries(const AppendArgs &a, int wg)
{
    constexpr int EB = kElemBytes<DT>;
    const AppendDesc &d = a.d;
    const int D = d.c.head_dim, us = a.unit_shift, um = (1 << us) - 1;
    const int per_tok = d.q_heads << us;  // units
    const int tok0 = wg * a.q_tokens;
    const int units = (int)min((int64_t)a.q_tokens, d.b.tokens - tok0) * per_tok;
    const int seq0 = first_seq(d.b.cu, d.b.seqs, tok0);
    const float inv = 1.0f / (float)per_tok;
    for (int i = threadIdx.x; i < units; i += kThreads) {
        // i / per_tok: by the reciprocal, then put right
        int dt = (int)((float)i * inv);
        dt -= dt * per_tok > i;
        dt += (dt + 1) * per_tok <= i;
        const int r = i - dt * per_tok;
        const int t = tok0 + dt, h = r >> us, u = r & um;
        int e0, e1;
        unit_places(u, d.rot_dim, d.interleaved, e0, e1);
        const uint8_t *src = (const uint8_t *)d.Q + (t * d.ldq + (int64_t)h * D) * EB;
        uint8_t *dst = (uint8_t *)d.Q_out + (t * d.ldqo + (int64_t)h * D) * EB;
        float x0[8], x1[8];
        load8<DT>(src + e0 * EB, x0);
        load8<DT>(src + e1 * EB, x1);
        if (d.rot_dim) {
            const int seq = seq_of(d.b.cu, d.b.seqs, t, seq0);
            const int64_t pos = (int64_t)d.b.len[seq] - d.b.cu[seq + 1] + t;
            rotate_unit(x0, x1, u, d.rot_dim, d.interleaved,
                        d.cos_sin + max((int64_t)0, min(pos, d.max_pos - 1)) * d.rot_dim);
        }
        store8<DT>(dst + e0 * EB, x0);
        store8<DT>(dst + e1 * EB, x1);
    }
}

// The codes of 8 values: x / sc rounded half away from zero (|x / sc| <= 127
// up to rounding, by the choice of sc), without a division for scales within
// [2^-100, 2^100].  Adding x * (1 / sc) to 1.5 * 2^23 in one rounding leaves
// the nearest whole number in the low bits, its two's complement low byte the
// code.  The product with the correctly rounded reciprocal is within 127 *
// 2^-24 of x / sc and the correctly rounded quotient within 2^-18 of that, so
// unless the product lies within 2^-14 of a half (about one value in 8000)
// the whole number next to both is the same; then, and for other scales, the
// codes come from the division.
__device__ __forceinline__ v2u code8(const float (&x)[8], float sc, float rsc, bool fast)
{
    constexpr float kWhole = 0x1.8p23f;
    v2u w = {0, 0};
    float off = 0.0f, s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        s[e] = __builtin_fmaf(x[e], rsc, kWhole);
        off = fmaxf(off, fabsf(__builtin_fmaf(x[e], rsc, kWhole - s[e])));
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const unsigned lo = __builtin_amdgcn_perm(__float_as_uint(s[4 * q + 1]), __float_as_uint(s[4 * q]),
                                                  0x0C0C0400u);
        const unsigned hi = __builtin_amdgcn_perm(__float_as_uint(s[4 * q + 3]), __float_as_uint(s[4 * q + 2]),
                                                  0x04000C0Cu);
        w[q] = lo | hi;
    }
    if (!(fast && off <= 0.5f - 0x1p-14f)) {
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] = sc > 0.0f ? code_of_quotient(x[e], sc) : 0.0f;
        w = pack8_codes(f);
    }
    return w;
}

// A workgroup takes a block of one head, keys and values (BOTH) or one of
// them, U units of 16 values of each per thread, held in registers between
// the pass that finds the largest value and the coding: every value is read
// once and every code written once.  The workgroups past those of the blocks
// rotate queries, so that a step is one launch.  Bound by memory when there
// are many tokens (6 prompts of up to 4099 tokens, 16 heads of 64, binary16,
// queries included: 43 us, 182 MB, 4.2 TB/s; a 1 GiB copy reaches 5.1), by three
// dependent loads (sums, block number, scale) when there are few (48 new
// tokens: 6.5 us).
template <int DT, int U, bool BOTH>
__global__ __launch_bounds__(kThreads) void k_append(AppendArgs a)
{
    constexpr int EB = kElemBytes<DT>;
    constexpr int KV = BOTH ? 2 : 1;
    __shared__ float red[KV][kThreads / 64];
    const AppendDesc &d = a.d;
    if ((int)blockIdx.x >= a.kv_wgs) {
        rotate_queries<DT>(a, blockIdx.x - a.kv_wgs);
        return;
    }
    const int H = d.c.heads, D = d.c.head_dim, bs = d.c.block_size;
    const int us = a.unit_shift, um = (1 << us) - 1;
    const int job = BOTH ? (int)blockIdx.x : (int)blockIdx.x >> 1;
    const int item = job / H, h = job - item * H;
    const Item it = find_item(d.b.cu, d.b.len, d.b.seqs, d.b.tokens, item, 1, bs, a.extra);
    const int n = it.t1 - it.t0, pos0 = it.len - n;
    if (n <= 0 || pos0 < 0)
        return;
    const int col = (pos0 >> a.block_shift) + it.index;
    // this block's new tokens: places p0 .. p1 - 1, token t0 + (col bs + p - pos0)
    const int64_t before = (int64_t)col * bs - pos0;
    const int p0 = (int)max(-before, (int64_t)0), p1 = (int)min(n - before, (int64_t)bs);
    if (p1 <= p0 || col >= d.c.table_cols)
        return;
    const int blk = d.c.table[it.seq * d.c.ld_table + col];
    const int tok = it.t0 + (int)before + p0;  // the token of place p0
    const int units = (p1 - p0) << us;

    // which of keys (0) and values (1) pass v is
    auto which = [&](int v) __attribute__((always_inline)) { return BOTH ? v : (int)(blockIdx.x & 1); };
    float x0[KV][U][8], x1[KV][U][8], amax[KV];
#pragma unroll
    for (int v = 0; v < KV; ++v) {
        const bool is_v = which(v);
        const int64_t ld = is_v ? d.ldv : d.ldk;
        const uint8_t *src = (const uint8_t *)(is_v ? d.V : d.K) + (tok * ld + (int64_t)h * D) * EB;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int i = min((int)threadIdx.x + k * kThreads, units - 1);  // the last one again
            const int p = i >> us, u = i & um;
            int e0, e1;
            unit_places(u, is_v ? 0 : d.rot_dim, d.interleaved, e0, e1);
            const uint8_t *row = src + p * ld * EB;
            load8<DT>(row + e0 * EB, x0[v][k]);
            load8<DT>(row + e1 * EB, x1[v][k]);
        }
    }
    // the values are on their way: the block they go to, only now
    if ((unsigned)blk >= (uint64_t)d.c.num_blocks)
        return;
    const int64_t bh = (int64_t)blk * H + h;
    float old[KV];
#pragma unroll
    for (int v = 0; v < KV; ++v)
        old[v] = p0 > 0 ? (which(v) ? d.c.vs : d.c.ks)[bh] : 0.0f;
#pragma unroll
    for (int v = 0; v < KV; ++v) {
        amax[v] = 0.0f;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (!which(v) && d.rot_dim) {
                const int i = min((int)threadIdx.x + k * kThreads, units - 1);
                const int p = i >> us, u = i & um;
                const int64_t pos = min((int64_t)col * bs + p0 + p, d.max_pos - 1);
                rotate_unit(x0[v][k], x1[v][k], u, d.rot_dim, d.interleaved, d.cos_sin + pos * d.rot_dim);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
                amax[v] = fmaxf(amax[v], fmaxf(fabsf(x0[v][k][e]), fabsf(x1[v][k][e])));
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1)
            amax[v] = fmaxf(amax[v], __shfl_xor(amax[v], o));
        if ((threadIdx.x & 63) == 0)
            red[v][threadIdx.x >> 6] = amax[v];
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < KV; ++v) {
        const bool is_v = which(v);
#pragma unroll
        for (int w = 0; w < kThreads / 64; ++w)
            amax[v] = fmaxf(amax[v], red[v][w]);
        const float need = amax[v] / 127.0f;
        const float sc = fmaxf(old[v], need < 0x1p-100f ? 0.0f : need);
        if (threadIdx.x == 0)
            (is_v ? d.c.vs : d.c.ks)[bh] = sc;
        const bool fast = sc >= 0x1p-100f && sc <= 0x1p100f;
        const float rsc = fast ? 1.0f / sc : 0.0f;
        int8_t *dst = (is_v ? d.c.v : d.c.k) + (bh << a.block_shift) * D;
        const int rot = is_v ? 0 : d.rot_dim;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int i = (int)threadIdx.x + k * kThreads;
            if (i >= units)
                break;
            const int p = i >> us, u = i & um;
            int e0, e1;
            unit_places(u, rot, d.interleaved, e0, e1);
            int8_t *row = dst + (p0 + p) * D;
            const v2u c0 = code8(x0[v][k], sc, rsc, fast), c1 = code8(x1[v][k], sc, rsc, fast);
            if (e1 == e0 + 8 && (u * 16 >= rot || d.interleaved)) {
                *(v4i *)(row + e0) = (v4i){(int)c0[0], (int)c0[1], (int)c1[0], (int)c1[1]};
            } else {
                *(v2u *)(row + e0) = c0;
                *(v2u *)(row + e1) = c1;
            }
        }
        // earlier tokens of the block: recoded when its scale grew
        if (p0 > 0 && sc > old[v]) {
            const float ratio = old[v] / sc;
            for (int i = threadIdx.x; i < p0 * D / 4; i += kThreads) {
                const int w = ((const int *)dst)[i];
                int q[4];
                for (int e = 0; e < 4; ++e)
                    q[e] = (int)code_of_quotient((float)(int8_t)(w >> (8 * e)) * ratio, 1.0f);
                ((unsigned *)dst)[i] = pack4_i8(q[0], q[1], q[2], q[3]);
            }
        }
    }
}

// `tokens` tokens per workgroup; blockIdx.y: keys or values.  A thread takes
// 16 codes and its neighbours the next, so reads and writes are whole lines.
// Memory bounds it: 85 667 tokens of 8 heads of 128 to bfloat16, 526 MB, in
// 130 us (4.0 TB/s).
template <int DT>
__global__ __launch_bounds__(kThreads) void k_read(KvCache c, KvBatch b, int tokens, int block_shift,
                                                   void *K_out, void *V_out)
{
    constexpr int EB = kElemBytes<DT>;
    const int H = c.heads, D = c.head_dim, bs = c.block_size, upr = D / 16;
    const int per_tok = H * upr, tok0 = blockIdx.x * tokens;
    const int seq0 = first_seq(b.cu, b.seqs, tok0);
    const bool is_v = blockIdx.y;
    for (int i = threadIdx.x; i < tokens * per_tok; i += kThreads) {
        const int dt = i / per_tok, r = i - dt * per_tok;
        const int t = tok0 + dt;
        if (t >= b.tokens)
            return;
        const int h = r / upr, u = r - h * upr;
        const int seq = seq_of(b.cu, b.seqs, t, seq0);
        const int64_t pos = (int64_t)b.len[seq] + t - b.cu[seq];
        const int64_t col = pos >> block_shift;
        if (pos < 0 || col >= c.table_cols)
            continue;
        const int blk = c.table[seq * c.ld_table + col];
        if ((unsigned)blk >= (uint64_t)c.num_blocks)
            continue;
        const int64_t row = (int64_t)blk * H + h;
        const float sc = (is_v ? c.vs : c.ks)[row];
        const v4i w = *(const v4i *)((is_v ? c.v : c.k) +
                                     ((row << block_shift) + (pos & (bs - 1))) * D + u * 16);
        uint8_t *out = (uint8_t *)(is_v ? V_out : K_out) + ((int64_t)tok0 * per_tok + i) * 16 * EB;
        for (int k = 0; k < 2; ++k) {
            float x[8];
            for (int e = 0; e < 8; ++e)
                x[e] = (float)(int8_t)((unsigned)w[2 * k + (e >> 2)] >> (8 * (e & 3))) * sc;
            store8<DT>(out + k * 8 * EB, x);
        }
    }
}

template <int DT>
void run_append(AppendArgs a, int64_t items, int64_t q_wgs, hipStream_t s)
{
    // units of what one workgroup takes of a block of one head; up to 512 of
    // them it takes keys and values together
    const int upr = a.d.c.head_dim / 16;
    const int rows = a.d.c.block_size < a.d.b.max_q ? a.d.c.block_size : a.d.b.max_q;
    const int units = rows * upr;
    a.kv_wgs = (int)(items * a.d.c.heads * (units <= 2 * kThreads ? 1 : 2));
    const dim3 grid((unsigned)(a.kv_wgs + q_wgs)), block(kThreads);
    if (units <= kThreads)
        hipLaunchKernelGGL((k_append<DT, 1, true>), grid, block, 0, s, a);
    else if (units <= 2 * kThreads)
        hipLaunchKernelGGL((k_append<DT, 2, true>), grid, block, 0, s, a);
    else if (units <= 4 * kThreads)
        hipLaunchKernelGGL((k_append<DT, 4, false>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((k_append<DT, 8, false>), grid, block, 0, s, a);
}

// tokens per workgroup whose units fill its threads once
int tokens_per_wg(int units_per_token)
{
    return units_per_token >= kThreads ? 1 : kThreads / units_per_token;
}

}  // namespace

hipError_t launch_kv_append(const AppendDesc &d, hipStream_t s)
{
    AppendArgs a{};
    a.d = d;
    a.extra = d.b.max_q == 1 ? 1 : 2;
    a.block_shift = __builtin_ctz((unsigned)d.c.block_size);
    a.unit_shift = __builtin_ctz((unsigned)d.c.head_dim) - 4;
    const int64_t items = d.b.tokens / d.c.block_size + (int64_t)a.extra * d.b.seqs;
    a.q_tokens = tokens_per_wg(d.q_heads * (d.c.head_dim / 16));
    const int64_t q_wgs = d.Q ? (d.b.tokens + a.q_tokens - 1) / a.q_tokens : 0;
    if (d.dtype == DT_F32)
        run_append<DT_F32>(a, items, q_wgs, s);
    else if (d.dtype == DT_F16)
        run_append<DT_F16>(a, items, q_wgs, s);
    else
        run_append<DT_BF16>(a, items, q_wgs, s);
    return hipGetLastError();
}

hipError_t launch_kv_read(const KvCache &c, const KvBatch &b, void *K_out, void *V_out, int dtype,
                          hipStream_t s)
{
    const int tokens = tokens_per_wg(c.heads * (c.head_dim / 16));
    const int shift = __builtin_ctz((unsigned)c.block_size);
    const dim3 grid((unsigned)((b.tokens + tokens - 1) / tokens), 2), block(kThreads);
    if (dtype == DT_F32)
        hipLaunchKernelGGL(k_read<DT_F32>, grid, block, 0, s, c, b, tokens, shift, K_out, V_out);
    else if (dtype == DT_F16)
        hipLaunchKernelGGL(k_read<DT_F16>, grid, block, 0, s, c, b, tokens, shift, K_out, V_out);
    else
        hipLaunchKernelGGL(k_read<DT_BF16>, grid, block, 0, s, c, b, tokens, shift, K_out, V_out);
    return hipGetLastError();
}

}  // namespace qg
