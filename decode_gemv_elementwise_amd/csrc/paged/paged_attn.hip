// Attention of a request's new tokens over its paged cache (gemv_paged_attn).
//
// Mathematics: with s_j = scale q.k_j, the softmax is formed in one pass over
// the keys with the running maximum m and sum l of the rows, in powers of two
// (scale log2(e) folded into s): a block of keys with maximum b moves m to
// m' = max(m, b), scales l and the sums over v by 2^(m - m'), and adds
// 2^(s_j - m') v_j.  Parts of a row's keys join by the same rule.
//
// Few rows (single tokens, drafts): the cache is read once and nothing is
// reused, so a row tile is the 16 rows (token, query head) that share one
// key/value head, and a wave works alone on blocks of 32 keys, straight from
// memory to registers.  The matrix products are taken transposed,
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
// Splitting: the host does not know the lengths, so every workgroup works the
// plan out from them (a sum over the requests, then a prefix sum): blocks per
// unit of work such that all units together fill the card.  A row tile whose
// keys are split leaves its parts in the workspace; the workgroup that counts
// the last of them joins them in order, so the result does not depend on which
// came last.
#include "paged_device.h"

namespace gemv {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / kWave;
constexpr int kRows = kAttnRows;  // rows of a tile
constexpr int kBlock = 32;        // keys a wave takes at a time
constexpr int kGrid = 512;        // two workgroups on each of 256 compute units
constexpr int kMinBlocks = 8;     // blocks of a unit at least: two a wave
constexpr int kMaxSplit = 128;    // parts of a row tile at most
constexpr float kNegInf = -__builtin_inff();
// A weight 2^(s - m) of binary16 is carried 2^14 times its size (the sums l and
// over v alike, so it cancels): its smallest step, 2^-24, would otherwise lose
// the many small weights of a long row beside one large one.
constexpr float kF16Lift = 14.0f;

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

struct AttnArgs {
    const uint16_t *q, *k, *v;
    int64_t q_ts, q_hs, k_stride[3], v_stride[3], o_ts, o_hs;
    const int32_t *table, *query_start, *kv_len;
    int64_t table_stride;
    void *out;
    int32_t *counters;
    float *parts;
    int32_t width, requests, tokens, heads, group, num_pages, window, sinks, max_parts;
    int64_t reach; // keys that a table row can hold
    float scale_log2;
    FastDiv page, per_group;
};

__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }

template <bool BF> __device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c)
{
    if constexpr (BF)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
}

// Eight floats rounded to nearest into 16 bits, and what each lost.
template <bool BF> __device__ __forceinline__ u32x4 round8(const float *p, float *rest)
{
    if constexpr (BF) {
        bf16x8 r;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            r[i] = (__bf16)p[i];
            rest[i] = p[i] - (float)r[i];
        }
        return __builtin_bit_cast(u32x4, r);
    } else {
        f16x8 r;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            r[i] = (_Float16)p[i];
            rest[i] = p[i] - (float)r[i];
        }
        return __builtin_bit_cast(u32x4, r);
    }
}

template <bool BF> __device__ __forceinline__ float as_float(uint16_t x)
{
    if constexpr (BF)
        return __builtin_bit_cast(float, (uint32_t)x << 16);
    else
        return (float)__builtin_bit_cast(_Float16, x);
}

// Bits 15 and 31 are set where that half is an infinity or NaN: adding one to a
// full exponent carries into the sign's place, and the sign is masked off.
template <bool BF> __device__ __forceinline__ uint32_t not_finite(uint32_t x)
{
    constexpr uint32_t e = BF ? 0x7f807f80u : 0x7c007c00u, one = BF ? 0x00800080u : 0x04000400u;
    return ((x & e) + one) & 0x80008000u;
}

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

struct Request {
    int q0, n, kv;
};

__device__ __forceinline__ Request request_of(const AttnArgs &a, int r)
{
    const int q0 = min(max(a.query_start[r], 0), a.tokens), q1 = min(max(a.query_start[r + 1], q0), a.tokens);
    return Request{q0, q1 - q0, max(a.kv_len[r], 0)};
}

__device__ __forceinline__ int tiles_of(const AttnArgs &a, const Request &q)
{
    return (int)(((int64_t)q.n * a.group + kRows - 1) / kRows);
}

// The most blocks of keys that a row tile of the request visits.
__device__ __forceinline__ int blocks_most(const AttnArgs &a, const Request &q)
{
    const int all = (int)((min((int64_t)q.kv, a.reach) + kBlock - 1) / kBlock);
    if (a.window == 0)
        return all;
    const int64_t some = ((int64_t)a.sinks + kBlock - 1) / kBlock + ((int64_t)a.window + kRows + 2 * kBlock - 2) / kBlock;
    return (int)min((int64_t)all, some);
}

// The keys of one row tile: blocks [0, first) hold the first tokens that stay
// visible, then blocks from `skip` on.
struct Walk {
    int first, skip, count; // block i is key block (i < first ? i : i - first + skip)
};

__device__ __forceinline__ Walk walk_of(const AttnArgs &a, int p_lo, int p_hi)
{
    const int64_t end = min((int64_t)p_hi + 1, a.reach);
    if (end <= 0)
        return Walk{0, 0, 0};
    const int all = (int)((end + kBlock - 1) / kBlock);
    if (a.window == 0)
        return Walk{0, 0, all};
    const int first = (int)((min((int64_t)a.sinks, end) + kBlock - 1) / kBlock);
    const int64_t lo = max((int64_t)0, (int64_t)p_lo - a.window + 1);
    const int skip = max((int)min(lo / kBlock, (int64_t)all), first);
    return Walk{first, skip, first + max(0, all - skip)};
}

template <bool BF, int D, bool F32OUT, bool PAGE8> struct RowTile {
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
    float m, l;

    __device__ RowTile(const AttnArgs &args) : a(args) {}

    __device__ __forceinline__ bool sees(int j) const
    {
        return j <= p_row && (a.window == 0 || j > p_row - a.window || j < a.sinks);
    }

    // The page id of key j, -1 where there is none.
    __device__ __forceinline__ int id_of(int j) const
    {
        const uint32_t at = div_by(a.page, j);
        const int id = at < (uint32_t)a.width ? table[at] : -1;
        return (unsigned)id < (unsigned)a.num_pages ? id : -1;
    }

    // Element offset of key j in page id (a key without a page reads page 0,
    // and what is read is dropped).
    __device__ __forceinline__ int64_t offset(const int64_t *stride, int id, int j) const
    {
        const uint32_t in = j - div_by(a.page, j) * a.page.d;
        return (int64_t)max(id, 0) * stride[0] + (int64_t)in * stride[1];
    }

    __device__ __forceinline__ void begin(const Request &rq, int r, int tile, int head)
    {
        lane = threadIdx.x & (kWave - 1);
        col = lane & 15;
        grp = lane >> 4;
        const int rows = rq.n * a.group, row0 = tile * kRows;
        const int last = min(row0 + kRows, rows) - 1;
        p_lo = rq.kv - rq.n + (int)div_by(a.per_group, row0);
        p_hi = rq.kv - rq.n + (int)div_by(a.per_group, last);
        kbase = a.k + head * a.k_stride[2];
        vbase = a.v + head * a.v_stride[2];
        table = a.table + r * a.table_stride;
        const int row = row0 + col;
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
                qf[s] = *reinterpret_cast<const u32x4 *>(src + 32 * s);
        }
        m = kNegInf;
        l = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            o[i] = f32x4{0, 0, 0, 0};
    }

    // Page ids of a block's keys that this lane reads: of k the keys krun and
    // krun + 4, of v the eight from vrun on.
    __device__ __forceinline__ void ids_of(int j0, int *kid, int *vid) const
    {
        const int krun = j0 + 8 * (col >> 2) + (col & 3), vrun = j0 + 8 * grp;
#pragma unroll
        for (int i = 0; i < NK; ++i)
            kid[i] = id_of(krun + 4 * i);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            vid[i] = id_of(vrun + i);
    }

    __device__ __forceinline__ void block(int j0, const int *kid, const int *vid)
    {
        const int krun = j0 + 8 * (col >> 2) + (col & 3), vrun = j0 + 8 * grp;
        u32x4 kf[2][KS];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint16_t *src = kbase + offset(a.k_stride, kid[PAGE8 ? 0 : i], krun + 4 * i) + 8 * grp;
#pragma unroll
            for (int s = 0; s < KS; ++s)
                kf[i][s] = *reinterpret_cast<const u32x4 *>(src + 32 * s);
        }
        uint32_t vw[8][VW];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint16_t *src = vbase + offset(a.v_stride, vid[PAGE8 ? 0 : i], vrun + i) + VPL * col;
            if constexpr (VW == 2) {
                const u32x2 x = *reinterpret_cast<const u32x2 *>(src);
                vw[i][0] = x[0];
                vw[i][1] = x[1];
            } else {
#pragma unroll
                for (int w = 0; w < VW; w += 4) {
                    const u32x4 x = *reinterpret_cast<const u32x4 *>(src + 2 * w);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        vw[i][w + e] = x[e];
                }
            }
        }
        uint32_t has = 0; // bit i: v's key vrun + i has a page
#pragma unroll
        for (int i = 0; i < 8; ++i)
            has |= (uint32_t)(vid[PAGE8 ? 0 : i] >= 0) << i;

        float p[8];
        {
            f32x4 s0 = {0, 0, 0, 0}, s1 = {0, 0, 0, 0};
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                s0 = mfma16<BF>(kf[0][s], qf[s], s0);
                s1 = mfma16<BF>(kf[1][s], qf[s], s1);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[i] = s0[i] * a.scale_log2;
                p[4 + i] = s1[i] * a.scale_log2;
            }
        }
        // every row of the tile sees every key of the block
        const bool whole = j0 + kBlock - 1 <= p_lo &&
                           (a.window == 0 || j0 > p_hi - a.window || j0 + kBlock <= a.sinks) && !__any(has != 0xff);
        if (!whole) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                p[i] = (has >> i & 1) && sees(vrun + i) ? p[i] : kNegInf;
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
        const float base = m == kNegInf ? 0.0f : BF ? m : m - kF16Lift;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            p[i] = __builtin_amdgcn_exp2f(p[i] - base);
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
                const bool keep = (has >> i & 1) && vrun + i <= p_hi;
#pragma unroll
                for (int w = 0; w < VW; ++w) {
                    vw[i][w] = keep ? vw[i][w] : 0;
                    bad |= not_finite<BF>(vw[i][w]);
                }
            }
            special = __any(bad != 0);
            if (special) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int w = 0; w < VW; ++w) {
                        const uint32_t n = not_finite<BF>(vw[i][w]);
                        vw[i][w] &= ~((n >> 15) * 0xffffu);
                    }
            }
        }
        float rest[8];
        const u32x4 pf = round8<BF>(p, rest);
        u32x4 pl;
        if constexpr (F32OUT) {
            float none[8];
            pl = round8<BF>(rest, none);
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            u32x4 vf;
#pragma unroll
            for (int w = 0; w < 4; ++w)
                vf[w] = __builtin_amdgcn_perm(vw[2 * w + 1][i / 2], vw[2 * w][i / 2], i & 1 ? 0x07060302u : 0x05040100u);
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
                const int j = j0 + 8 * g + i, id = id_of(j);
                const float w = __shfl(p[i], 16 * g + col);
                if (id < 0 || !sees(j))
                    continue;
                const uint16_t *src = vbase + offset(a.v_stride, id, j) + 4 * VPL * grp;
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

// The unit of work: a row tile of a request's key/value head, and its share s
// of ns of the keys.  part: where the tile's parts begin (-1: not split).
template <bool BF, int D, bool F32OUT, bool PAGE8>
__device__ __forceinline__ void run_unit(const AttnArgs &a, const Request &rq, int r, int tile, int head, int s, int ns,
                                         int part, float *lds)
{
    constexpr int VPL = D / 16, ROW = D + 4; // padded: the lanes of a group write 16 rows at once
    float *lds_m = lds + kWaves * kRows * ROW, *lds_l = lds_m + kWaves * kRows;
    int *lds_last = reinterpret_cast<int *>(lds_l + kWaves * kRows);
    const int wave = uniform(threadIdx.x / kWave);

    RowTile<BF, D, F32OUT, PAGE8> t(a);
    t.begin(rq, r, tile, head);
    const Walk walk = walk_of(a, t.p_lo, t.p_hi);
    const int b0 = (int)((int64_t)walk.count * s / ns), b1 = (int)((int64_t)walk.count * (s + 1) / ns);
    auto key = [&](int b) { return (b < walk.first ? b : b - walk.first + walk.skip) * kBlock; };
    int kid[t.NK], vid[t.NV];
    if (b0 + wave < b1)
        t.ids_of(key(b0 + wave), kid, vid);
    for (int b = b0 + wave; b < b1; b += kWaves) {
        int nkid[t.NK], nvid[t.NV];
        if (b + kWaves < b1)
            t.ids_of(key(b + kWaves), nkid, nvid);
        t.block(key(b), kid, vid);
#pragma unroll
        for (int i = 0; i < t.NK; ++i)
            kid[i] = nkid[i];
#pragma unroll
        for (int i = 0; i < t.NV; ++i)
            vid[i] = nvid[i];
    }

    // join the waves
    const float l = row_sum(t.l);
    if (t.grp == 0) {
        lds_m[wave * kRows + t.col] = t.m;
        lds_l[wave * kRows + t.col] = l;
    }
    __syncthreads();
    {
        float top = kNegInf;
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            top = fmaxf(top, lds_m[w * kRows + t.col]);
        const float f = t.m == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(t.m - top);
        float *dst = lds + (wave * kRows + t.col) * ROW + 4 * VPL * t.grp;
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int c = 0; c < VPL; ++c)
                dst[e * VPL + c] = t.o[c][e] * f;
    }
    __syncthreads();
    const int row = threadIdx.x / 16, d0 = (threadIdx.x & 15) * VPL; // 16 threads to a row
    float top = kNegInf, sum = 0.0f, acc[VPL];
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
        top = fmaxf(top, lds_m[w * kRows + row]);
#pragma unroll
    for (int c = 0; c < VPL; ++c)
        acc[c] = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const float mw = lds_m[w * kRows + row];
        sum += mw == kNegInf ? 0.0f : lds_l[w * kRows + row] * __builtin_amdgcn_exp2f(mw - top);
#pragma unroll
        for (int c = 0; c < VPL; ++c)
            acc[c] += lds[(w * kRows + row) * ROW + d0 + c];
    }
    const int rows = rq.n * a.group, at = tile * kRows + row;
    bool write = at < rows;

    if (part >= 0) {
        constexpr int64_t size = attn_part_floats(D);
        float *mine = a.parts + (part + s) * size;
        if (write) {
#pragma unroll
            for (int c = 0; c < VPL; c += 4)
                *reinterpret_cast<f32x4 *>(mine + row * D + d0 + c) = f32x4{acc[c], acc[c + 1], acc[c + 2], acc[c + 3]};
            if (d0 == 0) {
                mine[kRows * D + row] = top;
                mine[kRows * D + kRows + row] = sum;
            }
        }
        // every wave's stores are in the L2 cache before the barrier; thread 0's
        // release then writes that cache back, and its acquire drops what this
        // unit's caches may hold of the other parts
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (threadIdx.x == 0) {
            const int before = __hip_atomic_fetch_add(a.counters + part, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
            *lds_last = before == ns - 1;
            if (before == ns - 1) // ready for the next call
                __hip_atomic_store(a.counters + part, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        __syncthreads();
        write = write && *lds_last;
        if (write) {
            top = kNegInf;
            sum = 0.0f;
            const float *all = a.parts + part * size;
            for (int i = 0; i < ns; ++i)
                top = fmaxf(top, all[i * size + kRows * D + row]);
#pragma unroll
            for (int c = 0; c < VPL; ++c)
                acc[c] = 0.0f;
            for (int i = 0; i < ns; ++i) {
                const float *x = all + i * size;
                const float mi = x[kRows * D + row], f = mi == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(mi - top);
                sum = fmaf(x[kRows * D + kRows + row], f, sum);
#pragma unroll
                for (int c = 0; c < VPL; ++c)
                    acc[c] = fmaf(x[row * D + d0 + c], f, acc[c]);
            }
        }
    }
    if (write) {
        const int i = div_by(a.per_group, at), g = at - i * a.group;
        const int64_t to = (int64_t)(rq.q0 + i) * a.o_ts + (int64_t)(head * a.group + g) * a.o_hs + d0;
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum; // no key seen: zeros
        if constexpr (F32OUT) {
#pragma unroll
            for (int c = 0; c < VPL; c += 4)
                *reinterpret_cast<f32x4 *>(static_cast<float *>(a.out) + to + c) =
                    f32x4{acc[c] * inv, acc[c + 1] * inv, acc[c + 2] * inv, acc[c + 3] * inv};
        } else {
            typedef typename std::conditional<BF, __bf16, _Float16>::type T;
            typedef T t4 __attribute__((ext_vector_type(4)));
#pragma unroll
            for (int c = 0; c < VPL; c += 4) {
                t4 x;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[e] = (T)(acc[c + e] * inv);
                *reinterpret_cast<t4 *>(static_cast<T *>(a.out) + to + c) = x;
            }
        }
    }
    __syncthreads(); // lds is free for the next unit
}

__device__ __forceinline__ float block_sum(float v, float *scratch)
{
#pragma unroll
    for (int d = 1; d < kWave; d *= 2)
        v += __shfl_xor(v, d);
    if ((threadIdx.x & (kWave - 1)) == 0)
        scratch[threadIdx.x / kWave] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
        s += scratch[w];
    __syncthreads();
    return s;
}

template <bool BF, int D, bool F32OUT, bool PAGE8>
__global__ __launch_bounds__(kThreads, 2) void paged_attn_kernel(AttnArgs a)
{
    __shared__ float lds[kWaves * kRows * (D + 4) + 2 * kWaves * kRows + 1];
    __shared__ uint32_t unit0[kThreads], part0[kThreads], scratch[2 * kWaves];

    // blocks per unit: all row tiles' blocks over the grid
    float work = 0.0f;
    for (int r = threadIdx.x; r < a.requests; r += kThreads) {
        const Request q = request_of(a, r);
        work += (float)tiles_of(a, q) * (float)blocks_most(a, q);
    }
    work = block_sum(work, reinterpret_cast<float *>(scratch)) * (float)a.heads;
    const int share = (int)fminf(fmaxf(ceilf(work / (float)kGrid), (float)kMinBlocks), 1e9f);

    auto sum = [](uint32_t x, uint32_t y) { return x + y; };
    uint32_t ubase = 0, pbase = 0;
    for (int r0 = 0; r0 < a.requests; r0 += kThreads) {
        const int r = r0 + threadIdx.x;
        uint32_t units = 0, parts = 0;
        if (r < a.requests) {
            const Request q = request_of(a, r);
            const int ns = min(max((blocks_most(a, q) + share - 1) / share, 1), kMaxSplit);
            units = (uint32_t)tiles_of(a, q) * a.heads * ns;
            parts = ns > 1 ? units : 0;
        }
        uint32_t utotal, ptotal;
        unit0[threadIdx.x] = block_prefix<kWaves>(units, scratch, &utotal, sum);
        part0[threadIdx.x] = block_prefix<kWaves>(parts, scratch + kWaves, &ptotal, sum);
        __syncthreads();
        const int n = min(kThreads, a.requests - r0);
        // this workgroup's units are those congruent to its index
        uint32_t u = (blockIdx.x + gridDim.x - ubase % gridDim.x) % gridDim.x;
        for (; u < utotal; u += gridDim.x) {
            int lo = 0, hi = n;
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (unit0[mid] <= u)
                    lo = mid;
                else
                    hi = mid;
            }
            const int req = uniform(r0 + lo);
            const Request q = request_of(a, req);
            int ns = min(max((blocks_most(a, q) + share - 1) / share, 1), kMaxSplit);
            const uint32_t in = uniform(u - unit0[lo]);
            const uint32_t head = in % a.heads, rest = in / a.heads, tile = rest / ns;
            int s = rest % ns, part = -1;
            if (ns > 1) {
                const uint32_t first = pbase + uniform(part0[lo]) + (tile * a.heads + head) * ns;
                if (first + ns <= (uint32_t)a.max_parts) {
                    part = first;
                } else { // no room for the parts: the first unit takes the whole tile
                    if (s > 0)
                        continue;
                    ns = 1;
                }
            }
            run_unit<BF, D, F32OUT, PAGE8>(a, q, req, tile, head, s, ns, part, lds);
        }
        ubase += utotal;
        pbase += ptotal;
        __syncthreads();
    }
}

template <bool BF, int D> const void *kernel_of(bool f32out, bool page8)
{
    if (f32out)
        return page8 ? reinterpret_cast<const void *>(&paged_attn_kernel<BF, D, true, true>)
                     : reinterpret_cast<const void *>(&paged_attn_kernel<BF, D, true, false>);
    return page8 ? reinterpret_cast<const void *>(&paged_attn_kernel<BF, D, false, true>)
                 : reinterpret_cast<const void *>(&paged_attn_kernel<BF, D, false, false>);
}

template <int D> const void *kernel_of(int type, bool f32out, bool page8)
{
    return type == GEMV_W_BF16 ? kernel_of<true, D>(f32out, page8) : kernel_of<false, D>(f32out, page8);
}

} // namespace
} // namespace gemv

extern "C" int gemv_paged_attn(const void *q, int64_t q_token_stride, int64_t q_head_stride,
                               const gemv_kv_cache *cache, const int32_t *block_table, int64_t table_width,
                               int64_t table_stride, const int32_t *query_start, const int32_t *kv_len,
                               int64_t requests, int64_t tokens, int64_t q_heads, float scale, int64_t window,
                               int64_t sinks, void *out, int out_type, int64_t out_token_stride,
                               int64_t out_head_stride, void *workspace, int64_t workspace_bytes, void *hip_stream)
{
    const int st = gemv::validate_attn(q, q_token_stride, q_head_stride, cache, block_table, table_width, table_stride,
                                       query_start, kv_len, requests, tokens, q_heads, scale, window, sinks, out,
                                       out_type, out_token_stride, out_head_stride, workspace, workspace_bytes);
    if (st != GEMV_OK)
        return st;
    if (tokens == 0)
        return gemv::finish_launch((int)hipSuccess);
    gemv::AttnArgs a{};
    a.q = static_cast<const uint16_t *>(q);
    a.k = static_cast<const uint16_t *>(cache->k);
    a.v = static_cast<const uint16_t *>(cache->v);
    a.q_ts = q_token_stride, a.q_hs = q_head_stride, a.o_ts = out_token_stride, a.o_hs = out_head_stride;
    for (int d = 0; d < 3; ++d)
        a.k_stride[d] = cache->k_stride[d], a.v_stride[d] = cache->v_stride[d];
    a.table = block_table, a.query_start = query_start, a.kv_len = kv_len, a.table_stride = table_stride;
    a.out = out;
    const int64_t room = (workspace_bytes - gemv::kAttnCounters * 4) / (gemv::attn_part_floats(cache->dim) * 4);
    a.counters = static_cast<int32_t *>(workspace);
    a.parts = reinterpret_cast<float *>(a.counters + gemv::kAttnCounters);
    a.max_parts = (int)(room < 0 ? 0 : room < gemv::kAttnParts ? room : gemv::kAttnParts);
    a.width = (int)table_width, a.requests = (int)requests, a.tokens = (int)tokens, a.heads = cache->heads;
    a.group = (int)(q_heads / cache->heads), a.num_pages = (int)cache->num_pages;
    a.window = (int)window, a.sinks = window > 0 ? (int)sinks : 0;
    a.reach = table_width * cache->page_size; // a block's last key stays below 2^31
    a.reach = a.reach < INT_MAX - 63 ? a.reach : INT_MAX - 63;
    a.scale_log2 = scale * 1.44269504088896340736f;
    a.page = gemv::fast_div(cache->page_size), a.per_group = gemv::fast_div(a.group);

    const bool f32out = out_type == GEMV_W_F32, page8 = cache->page_size % 8 == 0;
    const void *fn = cache->dim == 64    ? gemv::kernel_of<64>(cache->type, f32out, page8)
                     : cache->dim == 128 ? gemv::kernel_of<128>(cache->type, f32out, page8)
                                         : gemv::kernel_of<256>(cache->type, f32out, page8);
    // no more workgroups than units can be: row tiles times the splits that the
    // table's width allows
    const int64_t blocks = (a.reach + gemv::kBlock - 1) / gemv::kBlock;
    int64_t split = (blocks + gemv::kMinBlocks - 1) / gemv::kMinBlocks;
    split = split < gemv::kMaxSplit ? split : gemv::kMaxSplit;
    const int64_t tiles = (tokens * a.group + gemv::kRows - 1) / gemv::kRows + requests;
    const int64_t units = tiles * a.heads * split;
    const int grid = (int)(units < gemv::kGrid ? units : gemv::kGrid);
    void *args[] = {&a};
    const hipError_t e = hipLaunchKernel(fn, dim3((unsigned)grid), dim3(gemv::kThreads), args, 0,
                                         static_cast<hipStream_t>(hip_stream));
    return gemv::finish_launch((int)e);
}
