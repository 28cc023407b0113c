// Row tiles of few rows (single tokens, drafts): up to 16 rows (token, query
// head) that share one key/value head.  The cache is read once and nothing is
// reused, so a wave works alone on blocks of 32 keys, straight from memory to
// registers.  The matrix products are taken transposed,
//     S^T = K Q^T (16 keys x 16 rows, twice),   O^T = V^T P^T,
// because then a lane holds one row's scores in both: statistics stay in the
// lane but for two exchanges, and P^T leaves the first product in the very
// lanes and order that the second wants it in.  For that, row m of the first
// product's two tiles is key 8 (m / 4) + m % 4, and that + 4: lane group g then
// holds the scores of keys 8 g .. 8 g + 7 of its row, which are the 8 values
// along k that the second product's operand asks of it.  V is read by rows
// (16 bytes a lane, 256 bytes a row for 128-wide heads) and turned within the
// lane: 8 keys by 8 values with 32 byte permutes.
//
// Memory-bound where the keys are many: 64 requests of up to 16384 keys (2.19 GB, 32
// query and 8 key/value heads of 128) take 410 us, 5.34 TB/s; one over 131072 keys
// 104 to 108 us, 4.95 to 5.15 TB/s.  With heads of 128 every wave has 16 KB on its way
// all the time (8 with heads of 64): a block's k and v are asked for one round ahead
// (409 us against 416 without), its page ids two.  Heads of 256 have no registers for
// that: 64 requests of up to 8192 keys (2.2 GB) take 406 us all the same, 5.4 TB/s.
// Where the keys are few it is latency: one token over 4099 keys 15.6 us on the GPU.
//
// The weights are rounded to 16 bits for the product with v, as the matrix cores take
// them; for a float32 result they go as two pieces (17.9 us and 412 us of the above).
#pragma once

#include "paged_attn_device.h"

namespace gemv {
namespace {

constexpr int kFewRows = kAttnRows;
constexpr int kFewBlock = 32; // keys a wave takes at a time
// floats of a part: sums over v, maxima, weight sums
constexpr int few_part(int dim) { return kFewRows * (dim + 2); }

// The largest of a lane's row: lanes l, l ^ 16, l ^ 32 and l ^ 48 share it.
__device__ __forceinline__ float row_max(float v)
{
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}

__device__ __forceinline__ float row_sum(float v)
{
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

template <bool BF, int D, bool F32OUT, int PAGES> struct FewRows {
    static constexpr bool PAGE8 = PAGES != 0; // eight keys from a multiple of eight on lie in one page
    static constexpr int KS = D / 32;    // k steps of the first product
    static constexpr int VPL = D / 16;   // values of a v row in a lane
    static constexpr int VW = VPL / 2;   // the same in words
    static constexpr int NK = PAGE8 ? 1 : 2, NV = PAGE8 ? 1 : 8;

    const AttnArgs &a;
    const uint16_t *kbase, *vbase; // of the key/value head
    const int32_t *table;          // of the request
    int p_lo, p_hi, p_row;         // positions of the tile's rows; of this lane's (-1: no row)
    int lane, col, grp;
    u32x4 qf[KS];
    f32x4 o[VPL];
    float m, l, scale;
    Paging paging;

    __device__ FewRows(const AttnArgs &args) : a(args) {}

    __device__ __forceinline__ void begin(const Request &rq, int r, int head, int thread)
    {
        lane = thread & (kWave - 1);
        col = lane & 15;
        grp = lane >> 4;
        const int rows = rq.n * a.group, row = col;
        p_lo = rq.kv - rq.n;
        p_hi = rq.kv - 1;
        kbase = a.k + (int64_t)head * a.k_stride[2];
        vbase = a.v + (int64_t)head * a.v_stride[2];
        table = a.table + r * a.table_stride;
        paging = paging_of(a);
        scale = kept(a.scale_log2);
        p_row = -1;
#pragma unroll
        for (int s = 0; s < KS; ++s)
            qf[s] = u32x4{0, 0, 0, 0};
        if (row < rows) {
            const int i = div_by(a.per_group, row), g = row - i * a.group;
            p_row = rq.kv - rq.n + i;
            const uint16_t *src = a.q + (int64_t)(rq.q0 + i) * a.q_ts + (int64_t)(head * a.group + g) * a.q_hs + 8 * grp;
#pragma unroll
            for (int s = 0; s < KS; ++s)
                qf[s] = (*reinterpret_cast<const u32x4 *>(src + 32 * s) & a.q_keep) ^ a.q_flip;
        }
        m = kNegInf;
        l = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            o[i] = f32x4{0, 0, 0, 0};
    }

    // Page ids of a block's keys that this lane reads, as the table has them (they
    // are checked where they are used, so that their load is waited for there): of
    // k the keys krun and krun + 4, of v the eight from vrun on.
    struct Ids {
        int k[NK], v[NV];
    };
    // A block's k and v as this lane needs them; bit i of has: v's key vrun + i has a page.
    struct Data {
        u32x4 k[2][KS];
        uint32_t v[8][VW];
        uint32_t has;
    };

    __device__ __forceinline__ int krun(int j0) const { return j0 + 8 * (col >> 2) + (col & 3); }
    __device__ __forceinline__ int vrun(int j0) const { return j0 + 8 * grp; }

    __device__ __forceinline__ void load_ids(int j0, Ids &ids) const
    {
#pragma unroll
        for (int i = 0; i < NK; ++i)
            ids.k[i] = paging.raw(table, krun(j0) + 4 * i);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            ids.v[i] = paging.raw(table, vrun(j0) + i);
    }

    // Asks for a block's k and v.
    __device__ __forceinline__ void load(int j0, const Ids &ids, Data &x) const
    {
        const uint16_t *kp = kbase + 8 * grp, *vp = vbase + VPL * col;
        if constexpr (PAGE8) { // a run of eight lies in one page
            kp += paging.template offset<false>(paging.checked(ids.k[0]), krun(j0));
            vp += paging.template offset<true>(paging.checked(ids.v[0]), vrun(j0));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint16_t *src = PAGE8 ? kp + 4ull * i * paging.k1
                                        : kp + paging.template offset<false>(paging.checked(ids.k[PAGE8 ? 0 : i]), krun(j0) + 4 * i);
#pragma unroll
            for (int s = 0; s < KS; ++s)
                x.k[i][s] = *reinterpret_cast<const u32x4 *>(src + 32 * s);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint16_t *src = PAGE8 ? vp + (uint64_t)i * paging.v1
                                        : vp + paging.template offset<true>(paging.checked(ids.v[PAGE8 ? 0 : i]), vrun(j0) + i);
            if constexpr (VW == 2) {
                const u32x2 y = *reinterpret_cast<const u32x2 *>(src);
                x.v[i][0] = y[0];
                x.v[i][1] = y[1];
            } else {
#pragma unroll
                for (int w = 0; w < VW; w += 4) {
                    const u32x4 y = *reinterpret_cast<const u32x4 *>(src + 2 * w);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x.v[i][w + e] = y[e];
                }
            }
        }
        x.has = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x.has |= (uint32_t)(paging.checked(ids.v[PAGE8 ? 0 : i]) >= 0) << i;
        __builtin_amdgcn_sched_barrier(0); // all are asked for before anything waits for one
    }

    __device__ __forceinline__ void block(int j0, Data &x)
    {
        float p[8];
        {
            f32x4 s0 = {0, 0, 0, 0}, s1 = {0, 0, 0, 0};
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                s0 = mfma16<BF>(x.k[0][s], qf[s], s0);
                s1 = mfma16<BF>(x.k[1][s], qf[s], s1);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[i] = s0[i] * scale;
                p[4 + i] = s1[i] * scale;
            }
        }
        // every row of the tile sees every key of the block
        const bool whole = sees_all(a, p_lo, p_hi, j0, kFewBlock) && !__any(x.has != 0xff);
        if (!whole) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                p[i] = (x.has >> i & 1) && sees(a, p_row, vrun(j0) + i) ? p[i] : kNegInf;
        }
        float top = fmaxf(fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3])), fmaxf(fmaxf(p[4], p[5]), fmaxf(p[6], p[7])));
        top = fmaxf(m, row_max(top));
        if (__any(top > m)) {
            const float f = top == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(m - top);
            l *= f;
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                o[i] *= f;
            m = top;
        }
        const float base = m == kNegInf ? 0.0f : m;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            p[i] = __builtin_amdgcn_exp2f(BF ? p[i] - base : p[i] - base + kF16Lift);
            l += p[i];
        }
        bool special = false;
        if (!whole) {
            // keys past the last row's and keys without a page hold anything:
            // their v is taken as 0.  An infinity or NaN of a key that only some
            // rows see must not reach the others through 0 * v: it is taken out
            // here and added for the rows that see it below.
            uint32_t bad = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool keep = (x.has >> i & 1) && vrun(j0) + i <= p_hi;
#pragma unroll
                for (int w = 0; w < VW; ++w) {
                    x.v[i][w] = keep ? x.v[i][w] : 0;
                    bad |= not_finite<BF>(x.v[i][w]);
                }
            }
            special = __any(bad != 0);
            if (special) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int w = 0; w < VW; ++w) {
                        const uint32_t n = not_finite<BF>(x.v[i][w]);
                        x.v[i][w] &= ~((n >> 15) * 0xffffu);
                    }
            }
        }
        u32x4 pf, pl; // the weights in 16 bits; the second piece of them
        if constexpr (F32OUT) {
            float rest[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                rest[i] = p[i];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                pf[i] = split2<BF>(rest + 2 * i);
            pl = round8<BF>(rest);
        } else {
            pf = round8<BF>(p);
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            u32x4 vf;
#pragma unroll
            for (int w = 0; w < 4; ++w)
                vf[w] = __builtin_amdgcn_perm(x.v[2 * w + 1][i / 2], x.v[2 * w][i / 2], i & 1 ? 0x07060302u : 0x05040100u);
            o[i] = mfma16<BF>(vf, pf, o[i]);
            if constexpr (F32OUT)
                o[i] = mfma16<BF>(vf, pl, o[i]);
        }
        if (special)
            add_special(j0, p);
    }

    // Adds p v for the infinities and NaN of v in block j0, to the rows that see
    // their key.  Rare, so it reads v again, key by key.
    __device__ __forceinline__ void add_special(int j0, const float *p)
    {
#pragma unroll 1
        for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int j = j0 + 8 * g + i, id = paging.checked(paging.raw(table, j));
                const float w = __shfl(p[i], 16 * g + col);
                if (id < 0 || !sees(a, p_row, j))
                    continue;
                const uint16_t *src = vbase + paging.template offset<true>(id, j) + 4 * VPL * grp;
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int c = 0; c < VPL; ++c) {
                        const uint32_t x = src[e * VPL + c];
                        if (not_finite<BF>(x) & 0x8000u)
                            o[c][e] = fmaf(w, as_float<BF>(x), o[c][e]);
                    }
            }
    }
};

// A share of a row tile's keys.  lds0 to lds3: one a wave, of at least 16 (D + 4)
// floats each; they are free again on return.
template <bool BF, int D, bool F32OUT, int PAGES>
__device__ __forceinline__ void run_few(const AttnArgs &a, const Request &rq, int r, int head, const Share &sh,
                                        float *lds0, float *lds1, float *lds2, float *lds3)
{
    constexpr int VPL = D / 16, ROW = D + 4; // padded: the lanes of a group write 16 rows at once
    __shared__ float lds_m[kWaves * kFewRows], lds_l[kWaves * kFewRows];
    __shared__ int lds_last;
    const int thread = thread_here(), wave = uniform(thread / kWave);

    FewRows<BF, D, F32OUT, PAGES> t(a);
    t.begin(rq, r, head, thread);
    const Walk walk = walk_of<kFewBlock>(a, t.p_lo, t.p_hi);
    // shares begin at whole rounds of the waves
    const int b0 = sh.from(walk.count) & -kWaves;
    const int b1 = sh.b + sh.len == sh.nb ? walk.count : sh.to(walk.count) & -kWaves;
    const auto key = [&](int b) { return walk.block(b) * kFewBlock; };
    // A block's page ids are asked for two rounds ahead and its k and v one round
    // ahead (the widest heads have no registers for that).
    int b = b0 + wave;
    typename decltype(t)::Ids ids;
    if (b < b1)
        t.load_ids(key(b), ids);
    if constexpr (D == 256) {
        for (; b < b1; b += kWaves) {
            typename decltype(t)::Ids next;
            if (b + kWaves < b1)
                t.load_ids(key(b + kWaves), next);
            typename decltype(t)::Data x;
            t.load(key(b), ids, x);
            t.block(key(b), x);
            ids = next;
        }
    } else {
        typename decltype(t)::Data x, y;
        // asks for block b's k and v and the ids of the one after
        const auto ahead = [&](int b, auto &x) {
            if (b < b1) {
                const auto now = ids;
                if (b + kWaves < b1)
                    t.load_ids(key(b + kWaves), ids);
                t.load(key(b), now, x);
            }
        };
        ahead(b, x);
        while (b < b1) {
            ahead(b + kWaves, y);
            t.block(key(b), x);
            b += kWaves;
            if (b >= b1)
                break;
            ahead(b + kWaves, x);
            t.block(key(b), y);
            b += kWaves;
        }
    }

    // join the waves
    const float l = row_sum(t.l);
    if (t.grp == 0) {
        lds_m[wave * kFewRows + t.col] = t.m;
        lds_l[wave * kFewRows + t.col] = l;
    }
    __syncthreads();
    {
        float top = kNegInf;
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            top = fmaxf(top, lds_m[w * kFewRows + t.col]);
        const float f = t.m == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(t.m - top);
        float *buffer = wave < 2 ? (wave == 0 ? lds0 : lds1) : (wave == 2 ? lds2 : lds3);
        float *dst = buffer + t.col * ROW + 4 * VPL * t.grp;
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int c = 0; c < VPL; ++c)
                dst[e * VPL + c] = t.o[c][e] * f;
    }
    __syncthreads();
    const int rows = rq.n * a.group;
    int row = thread / 16;                 // 16 threads to a row
    const int d0 = (thread & 15) * VPL;
    float top = kNegInf, sum = 0.0f, acc[VPL];
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
        top = fmaxf(top, lds_m[w * kFewRows + row]);
#pragma unroll
    for (int c = 0; c < VPL; ++c)
        acc[c] = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const float mw = lds_m[w * kFewRows + row];
        sum += lds_l[w * kFewRows + row] * (mw == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(mw - top)); // keeps a NaN
#pragma unroll
        for (int c = 0; c < VPL; ++c)
            acc[c] += (w < 2 ? (w == 0 ? lds0 : lds1) : (w == 2 ? lds2 : lds3))[row * ROW + d0 + c];
    }
    bool write = row < rows;

    if (sh.np > 1) {
        if (write) {
            const Parts parts(a);
            const int mine = sh.part(sh.me);
#pragma unroll
            for (int c = 0; c < VPL; c += 4)
                parts.put4(mine + row * D + d0 + c, f32x4{acc[c], acc[c + 1], acc[c + 2], acc[c + 3]});
            if (d0 == 0) {
                parts.put(mine + kFewRows * D + row, top);
                parts.put(mine + kFewRows * D + kFewRows + row, sum);
            }
        }
        if (!last_part(a, sh, thread, &lds_last))
            return;
        // 16 threads to a row again; what rows the tile lacks gives the others
        // more threads, each set of them taking every sets-th part
        const int sets = kFewRows / rows, set = row / rows;
        row -= set * rows;
        top = kNegInf;
        sum = 0.0f;
#pragma unroll
        for (int c = 0; c < VPL; ++c)
            acc[c] = 0.0f;
        if (set < sets) {
            constexpr int kAhead = 4;
            const Parts parts(a);
            for (int i0 = set; i0 < sh.np; i0 += kAhead * sets) {
                float m[kAhead], s[kAhead];
                f32x4 x[kAhead][VPL / 4];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int i = i0 + u * sets;
                    const int at = sh.part(min(i, sh.np - 1));
                    m[u] = parts.get(at + kFewRows * D + row);
                    s[u] = parts.get(at + kFewRows * D + kFewRows + row);
#pragma unroll
                    for (int c = 0; c < VPL / 4; ++c)
                        x[u][c] = parts.get4(at + row * D + d0 + 4 * c);
                    if (i >= sh.np) {
                        m[u] = kNegInf;
                        s[u] = 0.0f;
#pragma unroll
                        for (int c = 0; c < VPL / 4; ++c)
                            x[u][c] = f32x4{0, 0, 0, 0};
                    }
                }
                float next = top;
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
                    next = fmaxf(next, m[u]);
                const float f0 = top == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(top - next);
                sum *= f0;
#pragma unroll
                for (int c = 0; c < VPL; ++c)
                    acc[c] *= f0;
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const float f = m[u] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(m[u] - next);
                    sum += s[u] * f;
#pragma unroll
                    for (int c = 0; c < VPL; ++c)
                        acc[c] += x[u][c / 4][c % 4] * f;
                }
                top = next;
            }
        }
        // join the sets: set 0 adds the others' in order.  They lie in lds0:
        // at most 16 rows of VPL 16 floats, and their maxima and sums.
        if (set < sets && set > 0) {
            float *dst = lds0 + (set * rows + row) * D + d0;
#pragma unroll
            for (int c = 0; c < VPL; c += 4)
                *reinterpret_cast<f32x4 *>(dst + c) = f32x4{acc[c], acc[c + 1], acc[c + 2], acc[c + 3]};
            if (d0 == 0) {
                lds_m[set * rows + row] = top;
                lds_l[set * rows + row] = sum;
            }
        }
        __syncthreads();
        write = set == 0;
        if (write) {
            for (int s = 1; s < sets; ++s) {
                const float m = lds_m[s * rows + row], next = fmaxf(top, m);
                const float f0 = top == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(top - next);
                const float f1 = m == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(m - next);
                sum = sum * f0 + lds_l[s * rows + row] * f1;
#pragma unroll
                for (int c = 0; c < VPL; ++c)
                    acc[c] = acc[c] * f0 + lds0[(s * rows + row) * D + d0 + c] * f1;
                top = next;
            }
        }
    }
    if (write) {
        const int i = div_by(a.per_group, row), g = row - i * a.group;
        const int64_t to = (int64_t)(rq.q0 + i) * a.o_ts + (int64_t)(head * a.group + g) * a.o_hs + d0;
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum; // no key seen: zeros
#pragma unroll
        for (int c = 0; c < VPL; c += 4)
            store4<BF, F32OUT>(a.out, to + c, f32x4{acc[c] * inv, acc[c + 1] * inv, acc[c + 2] * inv, acc[c + 3] * inv});
    }
    __syncthreads(); // the buffers are free for the next share
}

} // namespace
} // namespace gemv
