// kivi_pool_rows.cu -- attention of new tokens over a pool's pages, 16 rows
// (token, head of one kv head) at a time, split over the cache's length.
//
// Scores.  A key group (32 tokens of one channel d) decodes to z_d + s_d c,
// c in 0..3.  With c' = c - 1 in {-1, 0, 1, 2}, s_d c' is exact in fp16, so
//   q . x^ = sum_d q_d (s_d c'_d) + sum_d q_d (z_d + s_d)
// takes exact products only: the first sum on the matrix units over the 32
// tokens, the second once per group (z and s are two more columns), as the
// first one's initial accumulator.  Outlier key channels (100 times the
// others) would otherwise cost the scores their accuracy.  Queries are fp16
// there, bf16 ones scaled by a power of two per row (exact).
// Values decode to fp16(z + s c), one rounding; probabilities are fp16
// (relative 2^-11, absolute 2^-25 against a maximum of at least 2^-8), sums
// and outputs fp32.  Tokens not yet coded take the same products in their own
// type, straight from their rows.
//
// A warp owns 16 rows and a range of the work: the (sequence, row tile, kv
// head) segments lie one after another, 1 per key group and kRawWeight per 32
// uncoded tokens, and the total is cut into equal ranges (so no sequence
// length leaves a warp idle).  A segment inside one range is finished by its
// warp; the others leave partial (max, sum, output) rows, at most two per
// warp, which pool_join_kernel adds in a fixed order.
// The 24*D-byte group blocks come through a per-warp ring of cp.async stages;
// fragments are decoded in registers: the codes of the block are ordered so
// that one masked word is two codes of a fragment register.
#include <cuda_runtime.h>

#include "kivi_code.cuh"
#include "kivi_pool.cuh"

namespace kivi {
namespace {

constexpr int kRowWarps = 4;        // warps per CTA
constexpr int kRowCtas = 3;         // CTAs per SM (168 registers a thread)
constexpr int kRowStages = 4;       // group blocks in flight per warp
constexpr int kRawWeight = 2;       // cost of 32 uncoded tokens, in groups
constexpr float kLazy = 8.0f;       // the running maximum follows when exceeded by 2^8

// ---- fragments ------------------------------------------------------------------
template <int DT>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1)
{
    if constexpr (DT == KIVI_BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ __half2 as_h2(uint32_t u)
{
    __half2 r;
    memcpy(&r, &u, 4);
    return r;
}
__device__ __forceinline__ uint32_t as_u(__half2 h)
{
    uint32_t r;
    memcpy(&r, &h, 4);
    return r;
}
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    uint32_t r;
    if constexpr (DT == KIVI_BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        memcpy(&r, &v, 4);
    } else {
        const __half2 v = __floats2half2_rn(a, b);
        memcpy(&r, &v, 4);
    }
    return r;
}
__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// The two codes of pair i of word w plus 2^(10 - 2k), as fp16 pairs (k = i % 5:
// a code at mantissa bits 2k, 2k + 1 of a number with exponent 10 - 2k counts
// ones).  Pairs 5 to 7 are read from the word shifted right by 10.
__device__ __forceinline__ uint32_t code_bits(uint32_t w, uint32_t w10, int i)
{
    const int k = i < 5 ? i : i - 5;
    const uint32_t mask = 0x00030003u << (2 * k);
    const uint32_t one = (uint32_t)((25 - 2 * k) << 10) * 0x10001u;
    return ((i < 5 ? w : w10) & mask) | one;
}
// Minus that offset, plus `less`, as an fp16 pair (exact).
__device__ __forceinline__ __half2 code_offset(int i, int less)
{
    const int k = i < 5 ? i : i - 5;
    const __half h = __float2half_rn(-(float)((1 << (10 - 2 * k)) + less));
    return __half2half2(h);
}

struct Seg {
    int e, rt, h;          // entry, row tile, kv head
    long long base, C;     // where the segment starts, its weight
};

// The segment that contains position pos of the split.
__device__ __forceinline__ Seg find_segment(const AttnTab &t, const AttnCall &c, long long pos)
{
    int lo = 0, hi = t.nb - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.off[mid] <= pos) lo = mid;
        else hi = mid - 1;
    }
    Seg s;
    s.e = lo;
    const int raw = (t.r[lo] + 31) / 32 + (t.nk[lo] + 31) / 32;
    s.C = max(1, t.ng[lo] + raw * kRawWeight);
    const int si = (int)((pos - t.off[lo]) / s.C);
    s.base = t.off[lo] + si * s.C;
    s.rt = si / c.v.H;
    s.h = si - s.rt * c.v.H;
    return s;
}

__device__ __forceinline__ long long range_at(long long w, long long tot, long long warps)
{
    return (long long)((unsigned long long)(w * tot) / (unsigned long long)warps);   // w * tot < 2^63, see launch_pool_rows
}

template <int D>
struct RowsSmem {
    static constexpr int RING = kRowStages * 24 * D;   // also the staging of 32 uncoded value rows
    static constexpr int FIRST = RING;                 // per channel: first new token whose value is not finite
    static constexpr int PER_WARP = RING + D * 4;
    static constexpr int BYTES = kRowWarps * PER_WARP;
    static_assert(32 * D * 2 <= RING, "value rows are staged in the ring");
};

// Partial result of a segment: 16 rows of D floats, then 16 (max, sum) pairs.
template <int D>
constexpr int kPartFloats = 16 * D + 32;

template <int D>
__device__ __forceinline__ int chunk_at(int t, int c)
{
    return (t * (D / 8) + (c ^ (t & 7))) * 16;
}

// Running softmax of the lane's two rows (lane/4 and lane/4 + 8) and their
// output columns 8c + 2cs, + 1.
template <int D>
struct State {
    float o[D / 8][4];
    float m[2], l[2];
};

// Scores S (4 tiles of 8 tokens; already in units of log2) to probabilities in
// place, moving the running maximum when a row exceeds it by 2^kLazy.
template <int D>
__device__ __forceinline__ void softmax_step(State<D> &st, float (&S)[4][4])
{
    float mx[2] = {fmaxf(S[0][0], S[0][1]), fmaxf(S[0][2], S[0][3])};
#pragma unroll
    for (int j = 1; j < 4; ++j) {
        mx[0] = fmaxf(mx[0], fmaxf(S[j][0], S[j][1]));
        mx[1] = fmaxf(mx[1], fmaxf(S[j][2], S[j][3]));
    }
    const bool grow = mx[0] > st.m[0] + kLazy || mx[1] > st.m[1] + kLazy;
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
            const float m = fmaxf(st.m[r], mx[r]);
            // A row that has seen nothing keeps a scale of 0 (its sums are 0).
            const float f = st.m[r] == -INFINITY ? 0.0f : ex2(st.m[r] - m);
            st.m[r] = m;
            st.l[r] *= f;
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                st.o[c][2 * r] *= f;
                st.o[c][2 * r + 1] *= f;
            }
        }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const float m = st.m[r] == -INFINITY ? 0.0f : st.m[r];
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            S[j][2 * r] = ex2(S[j][2 * r] - m);
            S[j][2 * r + 1] = ex2(S[j][2 * r + 1] - m);
            sum += S[j][2 * r] + S[j][2 * r + 1];
        }
        st.l[r] += sum;
    }
}

// One segment's items [i0, i1): groups below ng, then blocks of 32 residual
// tokens, then blocks of 32 new tokens.
template <int D, int DT>
__device__ __forceinline__ void run_items(const AttnCall &c, const AttnTab &t, const Seg &sg, int i0, int i1,
                                          uint8_t *sm, State<D> &st)
{
    using L = PageLayout<D>;
    constexpr int KU = D / 32, NC = D / 8, KW = L::KW;
    const int lane = threadIdx.x & 31, tq = lane >> 2, cs = lane & 3;
    const int e = sg.e, n = t.n[e], ng = t.ng[e], r_res = t.r[e], nk = t.nk[e], seq = t.seq[e];
    const PoolView &v = c.v;
#pragma unroll
    for (int k = 0; k < NC; ++k) st.o[k][0] = st.o[k][1] = st.o[k][2] = st.o[k][3] = 0.0f;
    st.m[0] = st.m[1] = -INFINITY;
    st.l[0] = st.l[1] = 0.0f;
    int *first = (int *)(sm + RowsSmem<D>::FIRST);
    for (int d = lane; d < D; d += 32) first[d] = 0x7fffffff;

    // The lane's rows: new token tok[k] and its head.
    int tok[2];
    const uint16_t *qp[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int row = 16 * sg.rt + tq + 8 * k;
        tok[k] = row / c.group;
        const bool real = tok[k] < n;
        const int hq = sg.h * c.group + row - tok[k] * c.group;
        qp[k] = real ? c.q.p + (long long)(t.row0[e] + tok[k]) * c.q.ts + hq * c.q.hs : nullptr;
        if (!real) tok[k] = -1;
    }
    uint32_t qa[KU][4], qb[KU][4];
    auto load_q = [&]() {
#pragma unroll
        for (int u = 0; u < KU; ++u) {
            const uint4 z = make_uint4(0, 0, 0, 0);
            *(uint4 *)qa[u] = qp[0] ? *(const uint4 *)(qp[0] + 32 * u + 8 * cs) : z;
            *(uint4 *)qb[u] = qp[1] ? *(const uint4 *)(qp[1] + 32 * u + 8 * cs) : z;
        }
    };

    // ---- coded groups ----
    const int g1 = min(i1, ng);
    if (i0 < g1) {
        load_q();
        float sc[2] = {c.scale, c.scale};
        if constexpr (DT == KIVI_BF16) {
            // fp16 queries: each row times 2^k with its largest magnitude
            // brought to [2^13, 2^14).
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                uint32_t(&q)[KU][4] = r ? qb : qa;
                float mx = 0.0f;
#pragma unroll
                for (int u = 0; u < KU; ++u)
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(q[u][w] << 16)),
                                             fabsf(__uint_as_float(q[u][w] & 0xffff0000u))));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                int k = 13 - ((int)(__float_as_uint(mx) >> 23) - 127);
                k = mx > 0.0f && mx < INFINITY ? max(-110, min(110, k)) : 0;
                const float f = __uint_as_float((uint32_t)(127 + k) << 23);
                sc[r] = c.scale * __uint_as_float((uint32_t)(127 - k) << 23);
#pragma unroll
                for (int u = 0; u < KU; ++u)
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        q[u][w] = pack2<KIVI_F16>(__uint_as_float(q[u][w] << 16) * f,
                                                  __uint_as_float(q[u][w] & 0xffff0000u) * f);
            }
        }
        const uint32_t ring = (uint32_t)__cvta_generic_to_shared(sm);
        const long long head_bytes = (long long)v.gpp * L::GB;
        const int *table = v.table + (long long)seq * v.max_pages;
        int next_page = table[i0 / v.gpp];
        auto issue = [&](int g) {
            if (g < g1) {
                const uint8_t *blk = v.packed + ((long long)next_page * v.H + sg.h) * head_bytes + (g % v.gpp) * L::GB;
                const uint32_t to = ring + (uint32_t)((g - i0) % kRowStages) * L::GB;
#pragma unroll
                for (int k = 0; k < L::GB / 512; ++k)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + (k * 32 + lane) * 16),
                                 "l"(blk + (k * 32 + lane) * 16)
                                 : "memory");
                if (g + 1 < g1) next_page = table[(g + 1) / v.gpp];
            }
            cp_async_commit();
        };
        for (int k = 0; k < kRowStages - 1; ++k) issue(i0 + k);
#pragma unroll 1
        for (int g = i0; g < g1; ++g) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kRowStages - 2) : "memory");
            __syncwarp();
            issue(g + kRowStages - 1);   // into the stage that the last iteration has read
            const uint8_t *blk = sm + ((g - i0) % kRowStages) * L::GB;
            // Bias of the group: columns of even tq hold z, of odd tq s, so a
            // lane's two columns add up to it.
            float b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int u = 0; u < KU; ++u) {
                uint32_t z[4];
                *(uint4 *)z = *(const uint4 *)(blk + ((tq & 1) ? L::KS : L::KZ) + u * 64 + cs * 16);
                mma<KIVI_F16>(b, qa[u][0], qb[u][0], qa[u][1], qb[u][1], z[0], z[1]);
                mma<KIVI_F16>(b, qa[u][2], qb[u][2], qa[u][3], qb[u][3], z[2], z[3]);
            }
            float S[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                S[j][0] = S[j][1] = b[0] + b[1];
                S[j][2] = S[j][3] = b[2] + b[3];
            }
            {
                uint32_t kw[L::WPL];
#pragma unroll
                for (int q = 0; q < L::WPL / 4; ++q)
                    *(uint4 *)(kw + 4 * q) = *(const uint4 *)(blk + L::KC + (q * 32 + lane) * 16);
#pragma unroll
                for (int u = 0; u < KU; ++u) {
                    uint32_t s[4];
                    *(uint4 *)s = *(const uint4 *)(blk + L::KS + u * 64 + cs * 16);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t w = kw[j * KW + u / 2], w10 = w >> 10;
                        uint32_t f[4];
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            const int i = 4 * (u % 2) + p;
                            f[p] = as_u(__hmul2(__hadd2(as_h2(code_bits(w, w10, i)), code_offset(i, 1)), as_h2(s[p])));
                        }
                        mma<KIVI_F16>(S[j], qa[u][0], qb[u][0], qa[u][1], qb[u][1], f[0], f[1]);
                        mma<KIVI_F16>(S[j], qa[u][2], qb[u][2], qa[u][3], qb[u][3], f[2], f[3]);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                S[j][0] *= sc[0];
                S[j][1] *= sc[0];
                S[j][2] *= sc[1];
                S[j][3] *= sc[1];
            }
            softmax_step<D>(st, S);
            uint32_t vw[L::WPL];
#pragma unroll
            for (int q = 0; q < L::WPL / 4; ++q)
                *(uint4 *)(vw + 4 * q) = *(const uint4 *)(blk + L::VC + (q * 32 + lane) * 16);
#pragma unroll
            for (int mm = 0; mm < 2; ++mm) {
                const uint32_t a0 = pack2<KIVI_F16>(S[2 * mm][0], S[2 * mm][1]);
                const uint32_t a1 = pack2<KIVI_F16>(S[2 * mm][2], S[2 * mm][3]);
                const uint32_t a2 = pack2<KIVI_F16>(S[2 * mm + 1][0], S[2 * mm + 1][1]);
                const uint32_t a3 = pack2<KIVI_F16>(S[2 * mm + 1][2], S[2 * mm + 1][3]);
#pragma unroll
                for (int jh = 0; jh < KW; ++jh) {
                    uint4 sz[2][2];   // [token half][group]: scales x, z of even group .. w of odd
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const uint4 q = *(const uint4 *)(blk + L::VM + page_vm_offset<D>(2 * mm + hf, cs, 2 * jh));
                        sz[hf][0] = make_uint4(q.x, q.y, 0, 0);
                        sz[hf][1] = make_uint4(q.z, q.w, 0, 0);
                    }
                    const uint32_t w0 = vw[(2 * mm) * KW + jh], w1 = vw[(2 * mm + 1) * KW + jh];
                    const uint32_t x0 = w0 >> 10, x1 = w1 >> 10;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint4 p0 = sz[0][i / 4], p1 = sz[1][i / 4];
                        const uint32_t f0 = as_u(__hfma2(__hadd2(as_h2(code_bits(w0, x0, i)), code_offset(i, 0)),
                                                         as_h2(p0.x), as_h2(p0.y)));
                        const uint32_t f1 = as_u(__hfma2(__hadd2(as_h2(code_bits(w1, x1, i)), code_offset(i, 0)),
                                                         as_h2(p1.x), as_h2(p1.y)));
                        mma<KIVI_F16>(st.o[8 * jh + i], a0, a1, a2, a3, f0, f1);
                    }
                }
            }
        }
        cp_async_wait_all();
        __syncwarp();
    }

    // ---- uncoded tokens, 32 at a time ----
    const int nres = (r_res + 31) / 32;
    if (i1 > ng) {
        load_q();
        // The last new token that a row of the tile sees.
        const int last_row = min(16 * sg.rt + 15, n * c.group - 1);
        const int last_tok = min(nk - 1, last_row / c.group), first_tok = 16 * sg.rt / c.group;
#pragma unroll 1
        for (int it = max(i0, ng); it < i1; ++it) {
            const bool is_new = it - ng >= nres;
            const int t0 = 32 * (is_new ? it - ng - nres : it - ng);
            if (is_new && t0 > last_tok) break;
            const int cnt = min(32, is_new ? nk - t0 : r_res - t0);
            const uint16_t *kp, *vp;
            long long kts, vts;
            if (is_new) {
                kp = c.k.p + (long long)(t.row0[e] + t0) * c.k.ts + sg.h * c.k.hs;
                vp = c.nv.p + (long long)(t.row0[e] + t0) * c.nv.ts + sg.h * c.nv.hs;
                kts = c.k.ts;
                vts = c.nv.ts;
            } else {
                const long long at = (((long long)seq * v.H + sg.h) * v.R + t0) * D;
                kp = v.resK + at;
                vp = v.resV + at;
                kts = vts = D;
            }
            // Values to shared memory (rows past the end: zeros).
#pragma unroll
            for (int k = 0; k < D / 8; ++k) {
                const int q = k * 32 + lane, row = q / (D / 8), ch = q % (D / 8);
                const uint32_t to = (uint32_t)__cvta_generic_to_shared(sm) + chunk_at<D>(row, ch);
                const int bytes = row < cnt ? 16 : 0;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to),
                             "l"(vp + (row < cnt ? row : 0) * vts + ch * 8), "r"(bytes)
                             : "memory");
            }
            cp_async_commit();
            float S[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                S[j][0] = S[j][1] = S[j][2] = S[j][3] = 0.0f;
                const int row = tq + 8 * j;
                const bool real = row < cnt;
#pragma unroll
                for (int u = 0; u < KU; ++u) {
                    uint32_t f[4] = {0, 0, 0, 0};
                    if (real) *(uint4 *)f = *(const uint4 *)(kp + row * kts + 32 * u + 8 * cs);
                    mma<DT>(S[j], qa[u][0], qb[u][0], qa[u][1], qb[u][1], f[0], f[1]);
                    mma<DT>(S[j], qa[u][2], qb[u][2], qa[u][3], qb[u][3], f[2], f[3]);
                }
            }
            const bool masked = is_new && t0 + cnt - 1 > first_tok;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int col = 8 * j + 2 * cs + (k & 1);
                    const bool seen = col < cnt && (!is_new || t0 + col <= tok[k >> 1]);
                    S[j][k] = seen ? S[j][k] * c.scale : -INFINITY;
                }
            softmax_step<D>(st, S);
            cp_async_wait_all();
            __syncwarp();
            if (masked) {
                // Some rows do not see some of these tokens: their probability
                // is 0, and 0 times a value that is not finite would still
                // spoil the row.  Such values leave the product; a row that
                // sees one becomes NaN in that channel at the end.
                constexpr uint32_t kExp = DT == KIVI_BF16 ? 0x7f80u : 0x7c00u;
#pragma unroll 1
                for (int k = 0; k < D / 8; ++k) {
                    const int q = k * 32 + lane, row = q / (D / 8), ch = q % (D / 8);
                    uint16_t *x = (uint16_t *)(sm + chunk_at<D>(row, ch));
                    uint32_t w[4];
                    *(uint4 *)w = *(const uint4 *)x;
                    bool bad = false;
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        bad = bad || (w[z] & kExp) == kExp || ((w[z] >> 16) & kExp) == kExp;
                    if (bad)
                        for (int z = 0; z < 8; ++z)
                            if ((x[z] & kExp) == kExp) {
                                atomicMin(first + ch * 8 + z, t0 + row);
                                x[z] = 0;
                            }
                }
                __syncwarp();
            }
#pragma unroll
            for (int mm = 0; mm < 2; ++mm) {
                const uint32_t a0 = pack2<DT>(S[2 * mm][0], S[2 * mm][1]);
                const uint32_t a1 = pack2<DT>(S[2 * mm][2], S[2 * mm][3]);
                const uint32_t a2 = pack2<DT>(S[2 * mm + 1][0], S[2 * mm + 1][1]);
                const uint32_t a3 = pack2<DT>(S[2 * mm + 1][2], S[2 * mm + 1][3]);
#pragma unroll
                for (int k = 0; k < NC; k += 2) {
                    // Matrices: token halves of channel tiles k and k + 1.
                    const int row = 16 * mm + (lane & 15), ch = k + (lane >> 4);
                    uint32_t f[4];
                    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                                 : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3])
                                 : "r"((uint32_t)__cvta_generic_to_shared(sm) + chunk_at<D>(row, ch))
                                 : "memory");
                    mma<DT>(st.o[k], a0, a1, a2, a3, f[0], f[1]);
                    mma<DT>(st.o[k + 1], a0, a1, a2, a3, f[2], f[3]);
                }
            }
            __syncwarp();   // the staged values have been read
        }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        st.l[r] += __shfl_xor_sync(0xffffffffu, st.l[r], 1);
        st.l[r] += __shfl_xor_sync(0xffffffffu, st.l[r], 2);
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
        for (int x = 0; x < 4; ++x)
            if (tok[x >> 1] >= first[8 * k + 2 * cs + (x & 1)]) st.o[k][x] = NAN;
    __syncwarp();
}

template <int D, int DT>
__global__ void __launch_bounds__(kRowWarps * 32, kRowCtas)
    pool_rows_kernel(const __grid_constant__ AttnCall c, const __grid_constant__ AttnTab t)
{
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, tq = lane >> 2, cs = lane & 3;
    uint8_t *sm = smem + wid * RowsSmem<D>::PER_WARP;
    const long long w = (long long)blockIdx.x * kRowWarps + wid;
    if (w >= c.warps) return;
    const long long tot = t.off[t.nb];
    const long long lo = range_at(w, tot, c.warps), hi = range_at(w + 1, tot, c.warps);
    long long pos = lo;
#pragma unroll 1
    while (pos < hi) {
        const Seg sg = find_segment(t, c, pos);
        const int e = sg.e, ng = t.ng[e];
        const int items = ng + (t.r[e] + 31) / 32 + (t.nk[e] + 31) / 32;
        // Items whose start lies in the warp's range.
        auto first_item = [&](long long rel) {
            if (rel <= ng) return (int)rel;
            return min(items, ng + (int)((rel - ng + kRawWeight - 1) / kRawWeight));
        };
        const long long rb = min(sg.C, hi - sg.base);
        const int i0 = min(items, first_item(pos - sg.base)), i1 = rb == sg.C ? items : first_item(rb);
        State<D> st;
        run_items<D, DT>(c, t, sg, i0, max(i0, i1), sm, st);
        if (sg.base >= lo && rb == sg.C) {
            // The whole segment: normalise and store.
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = 16 * sg.rt + tq + 8 * r, tok = row / c.group;
                if (tok >= t.n[e]) continue;
                const float inv = st.l[r] == 0.0f ? 0.0f : 1.0f / st.l[r];
                uint16_t *o = c.out
                              + ((long long)(t.row0[e] + tok) * c.H_q + sg.h * c.group + row - tok * c.group) * D + 2 * cs;
#pragma unroll
                for (int k = 0; k < D / 8; ++k)
                    *(uint32_t *)(o + 8 * k) = pack2<DT>(st.o[k][2 * r] * inv, st.o[k][2 * r + 1] * inv);
            }
        } else {
            float *part = c.part + (2 * w + (sg.base >= lo ? 1 : 0)) * kPartFloats<D>;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = tq + 8 * r;
                if ((16 * sg.rt + row) / c.group >= t.n[e]) continue;
#pragma unroll
                for (int k = 0; k < D / 8; ++k)
                    *(float2 *)(part + row * D + 8 * k + 2 * cs) = make_float2(st.o[k][2 * r], st.o[k][2 * r + 1]);
                if (cs == 0) *(float2 *)(part + 16 * D + 2 * row) = make_float2(st.m[r], st.l[r]);
            }
        }
        pos = sg.base + rb;
    }
}

// Adds the partial results of the segment that starts in warp blockIdx.x's
// range and ends behind it (if there is one), in the order of its warps: one
// warp per row.
template <int D, int DT>
__global__ void __launch_bounds__(512) pool_join_kernel(const __grid_constant__ AttnCall c,
                                                        const __grid_constant__ AttnTab t)
{
    const long long w = blockIdx.x, tot = t.off[t.nb];
    const long long lo = range_at(w, tot, c.warps), hi = range_at(w + 1, tot, c.warps);
    if (hi >= tot || lo >= hi) return;
    const Seg sg = find_segment(t, c, hi - 1);
    if (sg.base < lo || sg.base + sg.C <= hi) return;
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, e = sg.e;
    const int row = 16 * sg.rt + wid, tok = row / c.group;
    if (tok >= t.n[e]) return;
    constexpr int E = D / 32;
    float m = -INFINITY, l = 0.0f, o[E];
#pragma unroll
    for (int k = 0; k < E; ++k) o[k] = 0.0f;
    for (long long x = w;; ++x) {
        const float *part = c.part + (2 * x + (x == w ? 1 : 0)) * kPartFloats<D>;
        const float2 ml = *(const float2 *)(part + 16 * D + 2 * wid);
        if (ml.y != 0.0f) {   // (a NaN sum counts)
            const float mn = fmaxf(m, ml.x);
            const float f = m == -INFINITY ? 0.0f : ex2(m - mn), g = ex2(ml.x - mn);
            l = l * f + ml.y * g;
#pragma unroll
            for (int k = 0; k < E; ++k) o[k] = o[k] * f + part[wid * D + lane * E + k] * g;
            m = mn;
        }
        if (range_at(x + 1, tot, c.warps) >= sg.base + sg.C) break;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint16_t *out = c.out + ((long long)(t.row0[e] + tok) * c.H_q + sg.h * c.group + row - tok * c.group) * D;
#pragma unroll
    for (int k = 0; k < E; k += 2) *(uint32_t *)(out + lane * E + k) = pack2<DT>(o[k] * inv, o[k + 1] * inv);
}

template <int D, int DT>
cudaError_t rows_t(AttnCall &c, AttnTab &t, cudaStream_t st)
{
    static PerDeviceOnce once;
    cudaError_t e = set_smem_once(once, pool_rows_kernel<D, DT>, RowsSmem<D>::BYTES);
    if (e != cudaSuccess) return e;
    pool_rows_kernel<D, DT><<<(unsigned)((c.warps + kRowWarps - 1) / kRowWarps), kRowWarps * 32, RowsSmem<D>::BYTES, st>>>(
        c, t);
    e = cudaGetLastError();
    if (e != cudaSuccess || c.warps == 1) return e;
    pool_join_kernel<D, DT><<<(unsigned)c.warps, 512, 0, st>>>(c, t);
    return cudaGetLastError();
}

long long split_warps(int sms) { return (long long)sms * kRowCtas * kRowWarps; }

}  // namespace

size_t pool_rows_scratch(int D, int sms)
{
    return (size_t)(2 * split_warps(sms)) * (D == 64 ? kPartFloats<64> : kPartFloats<128>);
}

// Fills the split (t.off, c.warps) and launches.
cudaError_t launch_pool_rows(AttnCall &c, AttnTab &t, int sms, cudaStream_t st)
{
    t.off[0] = 0;
    for (int e = 0; e < t.nb; ++e) {
        const long long C = t.ng[e] + (long long)((t.r[e] + 31) / 32 + (t.nk[e] + 31) / 32) * kRawWeight;
        const long long tiles = ((long long)t.n[e] * c.group + 15) / 16;
        t.off[e + 1] = t.off[e] + tiles * c.v.H * (C > 0 ? C : 1);
    }
    const long long tot = t.off[t.nb];
    if (tot == 0) return cudaSuccess;
    c.warps = split_warps(sms);
    if (c.warps > tot) c.warps = tot;
    if (tot > (1LL << 62) / (c.warps + 1)) return cudaErrorInvalidValue;
    if (c.v.D == 64) return c.v.dtype ? rows_t<64, 1>(c, t, st) : rows_t<64, 0>(c, t, st);
    return c.v.dtype ? rows_t<128, 1>(c, t, st) : rows_t<128, 0>(c, t, st);
}

}  // namespace kivi
