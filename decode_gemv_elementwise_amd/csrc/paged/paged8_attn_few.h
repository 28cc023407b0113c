// Row tiles of 16 rows (token, query head) that share one key/value head: single
// tokens, drafts.  The cache is read once and nothing is reused, so a wave works alone
// on rounds of 32 SUB keys, straight from memory to registers, and widens the codes to q's
// type there: e4m3 two at a time by one instruction that scales too, int8 through 32
// bits.  The products are taken transposed,
//     S^T = K Q^T (16 keys x 16 rows, twice),   O^T = V^T P^T,
// because then a lane holds one row's scores in both: statistics stay in the lane but
// for two exchanges, and P^T leaves the first product in the very lanes and order that
// the second wants it in.  For that, row m of the first product's two tiles is key
// 8 (m / 4) + m % 4, and that + 4.  A lane's 16 bytes of k are 16 neighbouring values:
// two steps of the product take them, and q is laid out alike.
//
// Memory-bound: 64 single tokens over up to 16384 keys of 8 heads of 128 (1.04 GB) take 209 us
// in int8, 205 in e4m3 and 197 where a head's rows of a page lie together, 5.0 to 5.3 TB/s;
// 294 us with two blocks ahead (which spilled), a product for every value of v and tiles of
// one head.  More blocks ahead, or three or four workgroups a unit, gave nothing.
// One token over 4099 keys takes 16.4 us, of which 8.5 are a call over one key (launch,
// lengths, table, q) and the rest blocks, parts and their join; one over 131072 64 to 72.
// Heads of 256 keep one block of k on its way and are bound by that: 269 us for 8192 keys,
// 3.9 TB/s.  A float32 result costs a second product: 64 single tokens 205 us beside 204.
// Query heads of a large group over one key/value head are several tiles, each reading the
// keys again: 64 single tokens of 64 over one, 16384 keys each, 130 us, 62 of 16 over one.
#pragma once

#include "paged8_attn_device.h"

namespace gemv {
namespace {

constexpr int few_part(int dim) { return kAttnRows * (dim + 2); } // floats: sums over v, maxima, weight sums

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

// RUNS: eight keys from a multiple of eight on lie in one page and share a scale.
template <int CODE, bool BF, int D, bool F32OUT, bool RUNS> struct FewRows {
    static constexpr int kRows = kAttnRows, kBlock = 32; // keys of one product
    static constexpr int KS = D / 32;  // k steps of the first product
    static constexpr int KL = D / 64;  // 16-byte loads of a key in a lane
    static constexpr int VPL = D / 16; // values of a v row in a lane
    static constexpr int VW = VPL / 2; // the same in words of 16 bits
    static constexpr int VL = VPL / 4; // and in words of codes
    static constexpr int NK = RUNS ? 1 : 2, NV = RUNS ? 1 : 8;

    const Attn8Args &a;
    Paging8 at;
    int p_lo, p_hi, p_row; // positions of the tile's rows; of this lane's (-1: no row)
    int col, grp;
    u32x4 qf[KS];
    f32x4 o[VPL];
    float m, l, scale;
    int window, sinks; // of the arguments, kept: read again at every block they would be waited for
    uint32_t special; // not 0: an infinity or NaN of v was taken out

    __device__ FewRows(const Attn8Args &args) : a(args) {}

    __device__ __forceinline__ void begin(const Request &rq, int r, int tile, int head, int thread)
    {
        const int lane = thread & (kWave - 1);
        col = lane & 15;
        grp = lane >> 4;
        const int rows = rq.n * a.group, row0 = tile * kRows, row = row0 + col, before = rq.kv - rq.n;
        p_lo = before + (int)div_by(a.per_group, row0);
        p_hi = before + (int)div_by(a.per_group, min(row0 + kRows, rows) - 1);
        at.begin(a, r, head);
        scale = kept(a.scale_log2);
        window = kept(a.window), sinks = kept(a.sinks);
        p_row = -1;
#pragma unroll
        for (int s = 0; s < KS; ++s)
            qf[s] = u32x4{0, 0, 0, 0};
        if (row < rows) {
            const int i = div_by(a.per_group, row), g = row - i * a.group;
            p_row = before + i;
            const uint16_t *src = a.q + (int64_t)(rq.q0 + i) * a.q_ts + (int64_t)(head * a.group + g) * a.q_hs + 16 * grp;
#pragma unroll
            for (int s = 0; s < KS; ++s)
                qf[s] = (*reinterpret_cast<const u32x4 *>(src + s / 2 * 64 + s % 2 * 8) & a.q_keep) ^ a.q_flip;
        }
        m = kNegInf;
        l = 0.0f;
        special = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            o[i] = f32x4{0, 0, 0, 0};
    }

    __device__ __forceinline__ bool sees(int j) const
    {
        return j <= p_row && (window == 0 || j > p_row - window || j < sinks);
    }
    // Every row of the tile sees every key of [j0, j0 + n).
    __device__ __forceinline__ bool sees_all(int j0, int n) const
    {
        return j0 + n - 1 <= p_lo && (window == 0 || j0 > p_hi - window || j0 + n <= sinks);
    }

    // Page ids of a block's keys that this lane reads, as the table has them (they are
    // checked where they are used, so that their load is waited for there): of k the keys
    // krun and krun + 4, of v the eight from vrun on.
    struct Ids {
        int k[NK], v[NV];
    };
    // A block's codes and scales as this lane needs them; bit i of has: v's key vrun + i has a page.
    struct Data {
        u32x4 k[2][KL];
        uint32_t v[8][VL];
        uint32_t has;
        uint8_t ks[NV], vs[NV];
        int vid[NV]; // checked pages of v's keys
    };

    __device__ __forceinline__ int krun(int j0) const { return j0 + 8 * (col >> 2) + (col & 3); }
    __device__ __forceinline__ int vrun(int j0) const { return j0 + 8 * grp; }

    __device__ __forceinline__ void load_ids(int j0, Ids &ids) const
    {
#pragma unroll
        for (int i = 0; i < NK; ++i)
            ids.k[i] = at.raw(krun(j0) + 4 * i);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            ids.v[i] = at.raw(vrun(j0) + i);
    }

    // Asks for a block's k and the scales of both.
    __device__ __forceinline__ void load_k(int j0, const Ids &ids, Data &x) const
    {
        int kid[NK];
#pragma unroll
        for (int i = 0; i < NK; ++i)
            kid[i] = at.checked(ids.k[i]);
        x.has = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            x.vid[i] = at.checked(ids.v[i]);
            x.ks[i] = *at.template scale<false>(x.vid[i], vrun(j0) + i);
            x.vs[i] = *at.template scale<true>(x.vid[i], vrun(j0) + i);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x.has |= (uint32_t)(x.vid[RUNS ? 0 : i] >= 0) << i;
        const uint8_t *kp = at.template codes<false>(kid[0], krun(j0)) + 16 * grp;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint8_t *src = i == 0 ? kp : RUNS ? kp + 4ull * at.k1
                                                    : at.template codes<false>(kid[NK - 1], krun(j0) + 4) + 16 * grp;
#pragma unroll
            for (int s = 0; s < KL; ++s)
                x.k[i][s] = *reinterpret_cast<const u32x4 *>(src + 64 * s);
        }
    }

    // Asks for its v.
    __device__ __forceinline__ void load_v(int j0, Data &x) const
    {
        const uint8_t *vp = at.template codes<true>(x.vid[0], vrun(j0)) + VPL * col;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint8_t *src = RUNS ? vp + (uint64_t)i * at.v1 : at.template codes<true>(x.vid[RUNS ? 0 : i], vrun(j0) + i) + VPL * col;
            if constexpr (VL == 1) {
                x.v[i][0] = *reinterpret_cast<const uint32_t *>(src);
            } else if constexpr (VL == 2) {
                const u32x2 y = *reinterpret_cast<const u32x2 *>(src);
                x.v[i][0] = y[0];
                x.v[i][1] = y[1];
            } else {
                const u32x4 y = *reinterpret_cast<const u32x4 *>(src);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x.v[i][e] = y[e];
            }
        }
        __builtin_amdgcn_sched_barrier(0); // all are asked for before anything waits for one
    }

    __device__ __forceinline__ void block(int j0, const Data &x)
    {
        float p[8];
        {
            f32x4 s0 = {0, 0, 0, 0}, s1 = {0, 0, 0, 0};
            const auto codes = [](u32x4 w, int s) {
                const u32x2 x = codes16<CODE, BF>(w[s % 2 * 2]), y = codes16<CODE, BF>(w[s % 2 * 2 + 1]);
                return u32x4{x[0], x[1], y[0], y[1]};
            };
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                s0 = mfma16<BF>(codes(x.k[0][s / 2], s), qf[s], s0);
                s1 = mfma16<BF>(codes(x.k[1][s / 2], s), qf[s], s1);
                __builtin_amdgcn_sched_barrier(0);
            }
            // a lane's scores are of the keys vrun, whose scales of k are asked for with v's
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[i] = s0[i] * scale_of(x.ks[RUNS ? 0 : i]) * scale; // the scales' product may not fit where theirs do
                p[4 + i] = s1[i] * scale_of(x.ks[RUNS ? 0 : 4 + i]) * scale;
            }
        }
        // every row of the tile sees every key of the block
        const bool whole = sees_all(j0, kBlock) && !__any(x.has != 0xff);
        uint32_t seen = 0xff; // this row sees the lane's i-th key
        if (!whole) {
            seen = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool see = (x.has >> i & 1) && sees(vrun(j0) + i);
                seen |= (uint32_t)see << i;
                p[i] = see ? p[i] : kNegInf;
            }
        }
        float top = fmaxf(fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3])), fmaxf(fmaxf(p[4], p[5]), fmaxf(p[6], p[7])));
        if (__any(top > m)) { // else it moves in no lane, nor in those that share its row
            top = fmaxf(m, row_max(top));
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
            // bf16 has the range to take v's scale on the weight, a power of two: the codes
            // need no product then.  Below 2^-126 it has fewer bits, down to none at 2^-134:
            // there a code of 448 makes a part of 2^-117 at most, where float32 sums of parts
            // end soon too.  Of a NaN scale only rows that see the key take it.
            if constexpr (BF)
                p[i] = seen >> i & 1 ? p[i] * scale_of(x.vs[RUNS ? 0 : i]) : 0.0f;
        }
        // The weights in 16 bits, as the product takes them: half a step each, beside which l has
        // them whole, adds about what the result's own rounding to 16 bits does (0.0018 of a bf16
        // result in all, 0.0017 with exact weights).  For a float32 result a second piece holds
        // the rest, and as much of each weight as l has.
        u32x4 pf, pl;
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
        // v word by word of codes: four values of each of the lane's eight keys at a time, and no
        // further ahead (left alone, the compiler widens all at once and has no registers for it)
        uint32_t bad = 0;
#pragma unroll
        for (int w = 0; w < VL; ++w) {
            uint32_t v[8][2];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const u32x2 y = BF ? codes16<CODE, BF>(x.v[i][w]) : widen4<CODE, BF>(x.v[i][w], Scale<CODE, BF>(x.vs[RUNS ? 0 : i]));
                v[i][0] = y[0];
                v[i][1] = y[1];
            }
            if (!whole) {
                // keys past the last row's and keys without a page hold anything: their v is
                // taken as 0.  A NaN (a block's scale of 255) or infinity (binary16) of a key
                // that only some rows see must not reach the others through 0 * v: it is taken
                // out here and added for the rows that see it at the share's end.
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const bool keep = (x.has >> i & 1) && vrun(j0) + i <= p_hi;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t y = keep ? v[i][e] : 0, n = not_finite<BF>(y);
                        v[i][e] = y & ~((n >> 15) * 0xffffu);
                        bad |= n;
                    }
                }
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                u32x4 vf;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    vf[e] = __builtin_amdgcn_perm(v[2 * e + 1][c / 2], v[2 * e][c / 2], c & 1 ? 0x07060302u : 0x05040100u);
                o[4 * w + c] = mfma16<BF>(vf, pf, o[4 * w + c]);
                if constexpr (F32OUT)
                    o[4 * w + c] = mfma16<BF>(vf, pl, o[4 * w + c]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        special |= bad;
    }

    // Adds the infinities and NaN of v of the keys [j0, j0 + n) to the rows that see their
    // key, whatever its weight: that makes no difference to them.  Rare, so it reads v
    // again, key by key.
    __device__ __forceinline__ void add_special(int j0, int n)
    {
#pragma unroll 1
        for (int j = j0; j < j0 + n; ++j) {
            const int id = at.checked(at.raw(j));
            if (id < 0 || !sees(j))
                continue;
            const uint8_t *src = at.template codes<true>(id, j) + 4 * VPL * grp;
            const Scale<CODE, BF> f(*at.template scale<true>(id, j));
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int w = 0; w < VL; ++w) {
                    const u32x2 x = widen4<CODE, BF>(reinterpret_cast<const uint32_t *>(src)[e * VL + w], f);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t one = c & 1 ? x[c / 2] >> 16 : x[c / 2] & 0xffffu;
                        o[4 * w + c][e] += not_finite<BF>(one) & 0x8000u ? as_float<BF>((uint16_t)one) : 0.0f;
                    }
                    asm volatile("" ::: "memory"); // one load at a time
                }
        }
    }
};

// One share of a tile of few rows.  A wave has the next block's k and v on their way; of
// the widest heads, for which there are no registers, its k, and asks for v at a block's
// start.  A tile may be of `spread` neighbouring heads (1, 2 or 4), each with its
// share of the four waves: where a token's heads lie together in memory the waves then
// read neighbouring rows at one time.
template <int CODE, bool BF, int D, bool F32OUT, bool RUNS> struct FewTile {
    typedef FewRows<CODE, BF, D, F32OUT, RUNS> Rows;
    static constexpr int kRows = Rows::kRows, kPart = few_part(D);
    static constexpr uint32_t kLeast = D == 64 ? 16 : 8, kEdge = kLeast;
    static constexpr int kBuffer = kRows * (D + 4); // floats: a wave's sums, padded so that the lanes of a group meet no bank

    // lds: kWaves buffers, free again on return.  head: the tile's first.
    static __device__ __forceinline__ void run(const Attn8Args &a, const Request &rq, int r, int tile, int head, int spread,
                                               const Share &sh, char *lds)
    {
        constexpr int VPL = D / 16, ROW = D + 4;
        __shared__ float lds_m[kWaves * kRows], lds_l[kWaves * kRows];
        __shared__ int lds_last;
        float *const buffers = reinterpret_cast<float *>(lds);
        const int thread = thread_here(), wave = uniform(thread / kWave);
        const int waves = kWaves / spread; // of a head

        Rows t(a);
        t.begin(rq, r, tile, head + wave / waves, thread);
        const Walk walk = walk_of<Rows::kBlock>(a, t.p_lo, t.p_hi);
        // shares begin at whole rounds of the waves
        const int b0 = sh.from(walk.count) & -waves;
        const int b1 = sh.b + sh.len == sh.nb ? walk.count : sh.to(walk.count) & -waves;
        const auto key = [&](int b) { return walk.block(b) * Rows::kBlock; };
        // A block's page ids are asked for two rounds ahead, its k and v one.
        constexpr bool kLate = D == 256;
        int b = b0 + (wave & (waves - 1));
        typename Rows::Ids ids;
        typename Rows::Data x, y;
        const auto ahead = [&](int b, typename Rows::Data &x) {
            if (b < b1) {
                const typename Rows::Ids now = ids;
                if (b + waves < b1)
                    t.load_ids(key(b + waves), ids);
                t.load_k(key(b), now, x);
                if constexpr (!kLate)
                    t.load_v(key(b), x);
            }
        };
        const auto round = [&](typename Rows::Data &x, typename Rows::Data &next) {
            if constexpr (kLate)
                t.load_v(key(b), x);
            ahead(b + waves, next);
            t.block(key(b), x);
            b += waves;
        };
        if (b < b1)
            t.load_ids(key(b), ids);
        ahead(b, x);
        while (b < b1) {
            round(x, y);
            if (b >= b1)
                break;
            round(y, x);
        }
        if (__any(t.special != 0))
            for (b = b0 + (wave & (waves - 1)); b < b1; b += waves)
                t.add_special(key(b), Rows::kBlock);

        // join the waves of a head
        const float l = row_sum(t.l);
        if (t.grp == 0) {
            lds_m[wave * kRows + t.col] = t.m;
            lds_l[wave * kRows + t.col] = l;
        }
        __syncthreads();
        {
            float top = kNegInf;
            for (int w = wave & -waves; w < (wave & -waves) + waves; ++w)
                top = fmaxf(top, lds_m[w * kRows + t.col]);
            const float f = t.m == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(t.m - top);
            float *dst = buffers + wave * kBuffer + t.col * ROW + 4 * VPL * t.grp;
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int c = 0; c < VPL; ++c)
                    dst[e * VPL + c] = t.o[c][e] * f;
        }
        __syncthreads();
        // From here on 16 threads to a row, VPL values each, and the rows of all heads one
        // after the other, 16 at a time.
        const int rows = min(rq.n * a.group - tile * kRows, kRows), all = rows * spread;
        const int mine = thread / 16, d0 = (thread & 15) * VPL;
        const Parts parts(a);
        const auto store = [&](int i, int row, float sum, const float *acc) {
            row += tile * kRows;
            const int token = div_by(a.per_group, row), g = row - token * a.group;
            const int64_t to = (int64_t)(rq.q0 + token) * a.o_ts + (int64_t)((head + i) * a.group + g) * a.o_hs + d0;
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum; // no key seen: zeros
#pragma unroll
            for (int c = 0; c < VPL; c += 4)
                store4<BF, F32OUT>(a.out, to + c, f32x4{acc[c] * inv, acc[c + 1] * inv, acc[c + 2] * inv, acc[c + 3] * inv});
        };
        for (int at = mine; at < all; at += kRows) {
            const int i = at / rows, row = at - i * rows, w0 = i * waves;
            float top = kNegInf, sum = 0.0f, acc[VPL];
#pragma unroll
            for (int c = 0; c < VPL; ++c)
                acc[c] = 0.0f;
            for (int w = w0; w < w0 + waves; ++w)
                top = fmaxf(top, lds_m[w * kRows + row]);
            for (int w = w0; w < w0 + waves; ++w) {
                const float mw = lds_m[w * kRows + row];
                sum += lds_l[w * kRows + row] * (mw == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(mw - top)); // keeps a NaN
#pragma unroll
                for (int c = 0; c < VPL; ++c)
                    acc[c] += buffers[w * kBuffer + row * ROW + d0 + c];
            }
            if (sh.np == 1) {
                store(i, row, sum, acc);
            } else {
                const int to = sh.part(sh.me) + i * kPart;
#pragma unroll
                for (int c = 0; c < VPL; c += 4)
                    parts.put4(to + row * D + d0 + c, f32x4{acc[c], acc[c + 1], acc[c + 2], acc[c + 3]});
                if (d0 == 0) {
                    parts.put(to + kRows * D + row, top);
                    parts.put(to + kRows * D + kRows + row, sum);
                }
            }
        }
        if (sh.np > 1 && last_part(a, sh, thread, &lds_last)) {
            // what rows the tile lacks gives the others more threads, each set of them taking
            // every sets-th part
            const int sets = max(1, kRows / all);
            for (int at0 = 0; at0 < all; at0 += kRows) {
                const int set = sets == 1 ? 0 : mine / all, at = sets == 1 ? at0 + mine : mine - set * all;
                const int i = at / rows, row = at - i * rows;
                const bool on = set < sets && at < all;
                float top = kNegInf, sum = 0.0f, acc[VPL];
#pragma unroll
                for (int c = 0; c < VPL; ++c)
                    acc[c] = 0.0f;
                if (on) {
                    constexpr int kAhead = D == 256 ? 4 : 8; // parts on their way at once
                    for (int i0 = set; i0 < sh.np; i0 += kAhead * sets) {
                        float m[kAhead], s[kAhead];
                        f32x4 x[kAhead][VPL / 4];
#pragma unroll
                        for (int u = 0; u < kAhead; ++u) {
                            const int p = i0 + u * sets, from = sh.part(min(p, sh.np - 1)) + i * kPart;
                            m[u] = parts.get(from + kRows * D + row);
                            s[u] = parts.get(from + kRows * D + kRows + row);
#pragma unroll
                            for (int c = 0; c < VPL / 4; ++c)
                                x[u][c] = parts.get4(from + row * D + d0 + 4 * c);
                            if (p >= sh.np) {
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
                // join the sets: set 0 adds the others' in order.  They lie in the first
                // buffer: at most 16 rows of VPL 16 floats, and their maxima and sums.
                if (on && set > 0) {
                    float *dst = buffers + (set * all + at) * D + d0;
#pragma unroll
                    for (int c = 0; c < VPL; c += 4)
                        *reinterpret_cast<f32x4 *>(dst + c) = f32x4{acc[c], acc[c + 1], acc[c + 2], acc[c + 3]};
                    if (d0 == 0) {
                        lds_m[set * all + at] = top;
                        lds_l[set * all + at] = sum;
                    }
                }
                __syncthreads();
                if (on && set == 0) {
                    for (int s = 1; s < sets; ++s) {
                        const float m = lds_m[s * all + at], next = fmaxf(top, m);
                        const float f0 = top == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(top - next);
                        const float f1 = m == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(m - next);
                        sum = sum * f0 + lds_l[s * all + at] * f1;
#pragma unroll
                        for (int c = 0; c < VPL; ++c)
                            acc[c] = acc[c] * f0 + buffers[(s * all + at) * D + d0 + c] * f1;
                        top = next;
                    }
                    store(i, row, sum, acc);
                }
            }
        }
        __syncthreads(); // the buffers are free for the next share
    }
};

template <int CODE, bool BF, int D, bool F32OUT, bool RUNS>
__global__ __launch_bounds__(kThreads, 2) void paged8_few_kernel(Attn8Args)
{
    typedef FewTile<CODE, BF, D, F32OUT, RUNS> Tile;
    __shared__ __align__(16) char lds[kWaves * Tile::kBuffer * sizeof(float)];
    run_plan<Tile>(lds);
}

} // namespace
} // namespace gemv
