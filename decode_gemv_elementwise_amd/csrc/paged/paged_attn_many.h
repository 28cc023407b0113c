// Row tiles of many rows (chunks): 128 rows (token, query head) that share one
// key/value head, 32 to each of four waves, over blocks of 64 keys that the
// workgroup brings into LDS once for all of them.
//
// As with few rows the products are taken transposed, here 32 x 32 x 16:
//     S^T = K Q^T (32 keys x 32 rows, twice),   O^T = V^T P^T.
// A lane then holds 16 scores of one row per 32 keys, keys 8 (i / 4) + 4 h + i % 4
// for lane half h, so statistics stay in the lane but for one exchange with the
// lane 32 away.  The order of keys along the second product's k is free as long
// as both operands agree: P^T is taken as it lies, and V's operand is read from
// LDS in that order, turned on the way by the transposing 64-bit LDS read (4 keys
// by 16 values to 16 lanes).
//
// A wave forms a block's weights while the matrix core forms the next block's
// scores: exponentials and products then share the time instead of adding up.
//
// Memory to LDS goes without registers, 16 bytes a lane, ahead of the products:
// two buffers for k and two for v, one barrier a block.  A row of
// D values lies in one piece; which 16-byte chunk of it a lane fetches is
// permuted by the row, so that the products' reads meet no bank twice (k_turn,
// v_turn).
//
// Bound by the matrix cores and the exponentials beside them: 2048 new tokens over
// 8192 keys (240 GFLOP, 32 query and 8 key/value heads of 128) take 254 to 277 us
// from box to box, 870 to 947 TFLOP/s, and up to 300 where a profiler leaves gaps
// between the passes.  By the cycle counter read between a block's steps, of its
// 3600 cycles a wave (two share a SIMD) 2550 are products and weights, 900 the start
// of the next copies and 140 waits; the LDS counts no bank conflict.
//
// The running maximum only moves when a row's new one is more than kSlack above
// it: most blocks then skip the pass over the 32 x D sums.  A weight may then be up
// to 2^kSlack, and the largest, which would be 1, is rounded like the others: 7% more
// error of a bf16 chunk's results over 4099 keys.
//
// Weights go to the product with v in 16 bits, the type that the matrix cores take
// at their full rate: half a step of it (2^-8 of a bf16 weight at most, 2^-11 of a
// binary16 one) moves a result by about as much as its own rounding does (bf16 over
// 4099 keys, root mean square: 1.1e-4 from the exact result with both, 0.8e-4 with
// its own alone).  A float32 result takes two such pieces and twice the products:
// 467 us there.
#pragma once

#include "paged_attn_device.h"

namespace gemv {
namespace {

// The widest heads would need more registers than two waves on a SIMD have: there
// two waves share 32 rows, form the same scores and take half of the values each,
// over blocks of 32 keys.
constexpr int many_halves(int dim) { return dim == 256 ? 2 : 1; }
constexpr int many_rows(int dim) { return 32 * kWaves / many_halves(dim); } // rows of a tile
constexpr int many_block(int dim) { return dim == 256 ? 32 : 64; }          // keys of a block
// floats of a part: sums as the lanes hold them, m and l of each lane
constexpr int many_part(int dim) { return kWaves * (32 * (dim / many_halves(dim)) + 2 * kWave); }

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) void lds_void;
typedef const __attribute__((address_space(1))) void global_void;

// The largest over a lane and the lane 32 away, and the sum.
__device__ __forceinline__ float half_max(float v)
{
    const auto x = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v),
                                                    false, false);
    return fmaxf(__builtin_bit_cast(float, (uint32_t)x[0]), __builtin_bit_cast(float, (uint32_t)x[1]));
}

__device__ __forceinline__ float half_sum(float v)
{
    const auto x = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v),
                                                    false, false);
    return __builtin_bit_cast(float, (uint32_t)x[0]) + __builtin_bit_cast(float, (uint32_t)x[1]);
}

template <bool BF, int D, bool F32OUT, int PAGES> struct ManyRows {
    static constexpr int kBlock = many_block(D), KT = kBlock / 32; // keys of a block; tiles of 32 of them
    static constexpr int kRowBytes = 2 * D, kChunks = D / 8;      // 16-byte chunks of a row
    static constexpr int kRun = kWave / kChunks;                  // rows that one wave instruction brings
    static constexpr int kFetch = kBlock / (kRun * kWaves);   // such instructions of a wave per block
    static constexpr int kOwn = kBlock / kWaves;                  // rows, next to each other, that a wave brings
    static constexpr int KS = D / 16;                             // k steps of the first product
    static constexpr int kHalves = many_halves(D), DW = D / kHalves, DT = DW / 32; // values of a wave, tiles of them
    static constexpr int kAhead = 2, kVAhead = 2; // products between a read of LDS and its use
    // binary16's weights are lifted, which leaves one power of two to its largest
    static constexpr float kSlack = BF ? 8.0f : 1.0f;
    // m of this size has steps of 2^-16 (and 2^-17 below): what its rounding moves a weight by
    static constexpr float kFar = 128.0f;

    const AttnArgs &a;
    const char *kbase, *vbase; // of the key/value head
    const int32_t *table;      // of the request
    int p_lo, p_hi;            // positions of the tile's rows
    int w_lo, w_hi, p_row;     // of the wave's rows, of this lane's (-1: no row)
    bool live;                 // the wave has rows
    int thread, lane, wave, col, half;
    int values; // first of the wave's values
    uint32_t k_piece, v_piece; // byte of a row at which the lane's piece of the wave's first run lies
    Paging paging;
    float scale;
    u32x4 qf[KS];
    f32x16 o[DT];
    float m, l;

    __device__ ManyRows(const AttnArgs &args) : a(args) {}

    // Where a row's chunk c lies: at chunk c ^ turn.  k is read 16 rows at a time,
    // one chunk of each; v 4 rows at a time, 64 bytes of each.
    static __device__ __forceinline__ int k_turn(int row)
    {
        return (kRowBytes == 128 ? row >> 1 : row) & (kChunks < 16 ? kChunks - 1 : 15);
    }
    static __device__ __forceinline__ int v_turn(int row)
    {
        return kRowBytes == 128 ? (row & 2) << 1 : (row & 3) << 2;
    }

    __device__ __forceinline__ void begin(const Request &rq, int r, int tile, int head)
    {
        thread = thread_here();
        wave = uniform(thread / kWave);
        lane = thread & (kWave - 1);
        col = lane & 31;
        half = lane >> 5;
        values = wave % kHalves * DW;
        const int rows = rq.n * a.group, row0 = tile * many_rows(D), wrow = row0 + wave / kHalves * 32,
                  before = rq.kv - rq.n;
        p_lo = before + (int)div_by(a.per_group, row0);
        p_hi = before + (int)div_by(a.per_group, min(row0 + many_rows(D), rows) - 1);
        live = wrow < rows;
        w_lo = before + (int)div_by(a.per_group, min(wrow, rows - 1));
        w_hi = before + (int)div_by(a.per_group, min(wrow + 32, rows) - 1);
        kbase = reinterpret_cast<const char *>(a.k + (int64_t)head * a.k_stride[2]);
        vbase = reinterpret_cast<const char *>(a.v + (int64_t)head * a.v_stride[2]);
        table = a.table + r * a.table_stride;
        paging = paging_of(a);
        scale = kept(a.scale_log2);
        k_piece = 16 * (lane % kChunks ^ k_turn(wave * kOwn + lane / kChunks));
        v_piece = 16 * (lane % kChunks ^ v_turn(wave * kOwn + lane / kChunks));
        p_row = -1;
        const int row = wrow + col;
        const int i = div_by(a.per_group, min(row, rows - 1)), g = min(row, rows - 1) - i * a.group;
        if (row < rows)
            p_row = before + i;
        // lanes without a row take the last one's q: nothing of theirs is kept
        const uint16_t *src = a.q + (int64_t)(rq.q0 + i) * a.q_ts + (int64_t)(head * a.group + g) * a.q_hs + 8 * half;
#pragma unroll
        for (int s = 0; s < KS; ++s)
            qf[s] = (*reinterpret_cast<const u32x4 *>(src + 16 * s) & a.q_keep) ^ a.q_flip;
        m = kNegInf;
        l = 0.0f;
#pragma unroll
        for (int i = 0; i < DT; ++i)
            o[i] = f32x16{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
    }

    // Starts the copy of block j0 of k (or v) into LDS; ids: the page of each lane's key.
    template <bool V> __device__ __forceinline__ void fetch(int j0, int ids, char *to) const
    {
        const int own = wave * kOwn, r = lane / kChunks;
        const char *base = V ? vbase : kbase;
        const uint32_t piece = V ? v_piece : k_piece, step = 2 * (V ? paging.v1 : paging.k1);
        if constexpr (PAGES == 16) // a wave's rows lie in one page
            base += 2 * paging.template offset<V>(__builtin_amdgcn_readlane(ids, own), j0 + own);
#pragma unroll
        for (int f = 0; f < kFetch; ++f) {
            // the turns of rows own + r and f kRun have no bits in common: together they are the row's
            const uint32_t at = piece ^ (16 * (V ? v_turn(f * kRun) : k_turn(f * kRun)));
            const char *from;
            if constexpr (PAGES == 16) {
                from = base + (r * step + at);
                base += (uint64_t)kRun * step;
            } else {
                const int row = own + f * kRun + r;
                from = base + 2 * paging.template offset<V>(__shfl(ids, row), j0 + row) + at;
            }
            __builtin_amdgcn_global_load_lds((global_void *)from, (lds_void *)(to + (own + f * kRun) * kRowBytes), 16, 0, 0);
        }
    }

    // Makes a block of v safe to multiply by weights of 0: keys past the tile's
    // last row and keys without a page hold anything and are taken as 0, and an
    // infinity or NaN of a key that only some rows see is taken out (true if there
    // was one: add_special adds it for the rows that see it).
    __device__ __forceinline__ bool clean(int j0, uint64_t has, char *v, uint32_t *flags) const
    {
        uint32_t bad = 0;
        for (int at = thread; at < kBlock * kChunks; at += kThreads) {
            const int key = at / kChunks;
            u32x4 x = *reinterpret_cast<u32x4 *>(v + at * 16);
            const bool keep = (has >> key & 1) && j0 + key <= p_hi;
            uint32_t drop = keep ? 0 : 1;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                x[w] = keep ? x[w] : 0;
                const uint32_t n = not_finite<BF>(x[w]);
                x[w] &= ~((n >> 15) * 0xffffu);
                bad |= n;
                drop |= n;
            }
            if (drop)
                *reinterpret_cast<u32x4 *>(v + at * 16) = x;
        }
        return any_thread(thread, bad != 0, flags);
    }

    // Bit i: this lane's row sees key j0 + i.
    __device__ __forceinline__ uint64_t seen_of(int j0, uint64_t has) const
    {
        const auto below = [](int64_t n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1; };
        const int64_t p = (int64_t)p_row - j0;
        uint64_t seen = has & below(p + 1);
        if (a.window != 0)
            seen &= ~below(p - a.window + 1) | below((int64_t)a.sinks - j0);
        return seen;
    }

    // This lane's words of a block of k for the first product's n-th step, and of v
    // for the second's.
    struct KAt {
        const char *k;
        int row, turn;
        __device__ __forceinline__ KAt(const char *k, int ln)
            : k(k), row((ln & 31) * kRowBytes), turn(16 * ((ln >> 5) ^ k_turn(ln & 31)))
        {
        }
        __device__ __forceinline__ u32x4 operator()(int n) const // rows 32 apart have the same turn
        {
            return *reinterpret_cast<const u32x4 *>(k + (row + (turn ^ (32 * (n / KT)))) + n % KT * 32 * kRowBytes);
        }
    };
    struct VAt {
        const char *v;
        int row, turn;
        // 16 lanes bring 4 keys by 16 values
        __device__ __forceinline__ VAt(const char *v, int ln, int values) : v(v)
        {
            const int key = 4 * (ln >> 5) + ((ln & 15) >> 2), chunk = 2 * ((ln >> 4) & 1) + ((ln & 3) >> 1);
            row = key * kRowBytes + 2 * values + 8 * (ln & 1);
            turn = 16 * (chunk ^ v_turn(key));
        }
        __device__ __forceinline__ u32x4 operator()(int n) const // rows 8 apart have the same turn
        {
            const char *at = v + (row + (turn ^ (64 * (n % DT))));
            const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(at + 16 * (n / DT) * kRowBytes));
            const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(at + (16 * (n / DT) + 8) * kRowBytes));
            const u32x2 lo = __builtin_bit_cast(u32x2, x), hi = __builtin_bit_cast(u32x2, y);
            return u32x4{lo[0], lo[1], hi[0], hi[1]};
        }
    };

    // The lane as the compiler knows no other: places in LDS are formed where they
    // are used; all of them at once, for all buffers, would not leave registers enough.
    __device__ __forceinline__ int lane_here() const
    {
        int ln = lane;
        asm volatile("" : "+v"(ln));
        return ln;
    }

    // The scores of a block of keys, with `between(n)` after the n-th of its N
    // products: work of other registers that the matrix core does not wait for.
    // The order is kept as written: left alone, the compiler waits for each read.
    template <class F> __device__ __forceinline__ void scores(const char *k, f32x16 *s, F between) const
    {
        constexpr int N = KS * KT;
        const KAt at(k, lane_here());
#pragma unroll
        for (int t = 0; t < KT; ++t)
            s[t] = f32x16{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
        u32x4 f[kAhead];
#pragma unroll
        for (int n = 0; n < kAhead; ++n)
            f[n] = at(n);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            s[n % KT] = mfma32<BF>(f[n % kAhead], qf[n / KT], s[n % KT]);
            if (n + kAhead < N)
                f[n % kAhead] = at(n + kAhead);
            between(n);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // One block of keys whose scores are in s: their weights, formed while the
    // products of the next block (k there) run into `next`, then the sums over v.
    // part: some rows do not see some of its keys.
    __device__ __forceinline__ void block(int j0, uint64_t has, const char *k, const char *v, bool part, bool special,
                                          f32x16 *s, f32x16 *next)
    {
        if (part) {
            // by masks of all bits, not by comparisons: 32 of those would take 64 scalar registers
            const uint64_t seen = seen_of(j0, has) >> (4 * half);
#pragma unroll
            for (int t = 0; t < KT; ++t) {
                const int32_t word = (int32_t)(uint32_t)(seen >> (32 * t));
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const uint32_t see = __builtin_amdgcn_sbfe(word, 8 * (i / 4) + i % 4, 1);
                    const float x = s[t][i];
                    s[t][i] = __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, x) & see) | (0xff800000u & ~see));
                }
            }
        }
        float top = s[0][0];
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                top = fmaxf(top, s[t][i]);
        top = half_max(top) * scale;
        if (__any(top - m > kSlack)) { // by the difference: m + kSlack may round up a step
            const float to = fmaxf(m, top);
            const float f = to == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(m - to);
            l *= f;
#pragma unroll
            for (int d = 0; d < DT; ++d)
                o[d] *= f;
            m = to;
        }
        // A weight is 2^(by s - off): one fused step, whose s scale is exact where m is
        // s scale rounded.  From kFar on that difference shows, and from 2^24 it can
        // take a weight past binary16 or down to 0: there the scores are replaced by
        // s scale - m, both rounded alike, first (2048 new tokens over 8192 keys: 263 us
        // against 247).  With keys found one by one always: the branch would cost tiles
        // of few rows their registers (64 single tokens over up to 8192 keys, pages of
        // 5: 240 us against 226; 2048 over 8192 332 against 336).
        const float base = m == kNegInf ? 0.0f : m;
        float by = scale, off = BF ? base : base - kF16Lift;
        if (PAGES == 0 || __any(__builtin_fabsf(base) >= kFar)) {
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    s[t][i] = s[t][i] * scale - base;
            by = 1.0f;
            off = BF ? 0.0f : -kF16Lift;
        }
        u32x4 pf[2 * KT], pl[F32OUT ? 2 * KT : 1]; // the weights in pairs, and the second piece of them
        // the other workgroup's wave on this SIMD starts its copies meanwhile, at the lower
        // priority: 281 -> 274 us for 2048 new tokens over 8192 keys
        __builtin_amdgcn_s_setprio(1);
        scores(k, next, [&](int n) {
            constexpr int N = KS * KT, kPairs = 8 * KT;
#pragma unroll
            for (int e = n * kPairs / N; e < (n + 1) * kPairs / N; ++e) {
                float p[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    p[i] = __builtin_amdgcn_exp2f(fmaf(s[e / 8][2 * e % 16 + i], by, -off));
                    l += p[i];
                }
                if constexpr (F32OUT) {
                    pf[e / 4][e % 4] = split2<BF>(p);
                    pl[e / 4][e % 4] = round2<BF>(p);
                } else {
                    pf[e / 4][e % 4] = round2<BF>(p);
                }
            }
        });
        {
            constexpr int N = 2 * KT * DT;
            const VAt at(v, lane_here(), values);
            u32x4 f[kVAhead];
#pragma unroll
            for (int n = 0; n < kVAhead; ++n)
                f[n] = at(n);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int n = 0; n < N; ++n) {
                o[n % DT] = mfma32<BF>(f[n % kVAhead], pf[n / DT], o[n % DT]);
                if constexpr (F32OUT)
                    o[n % DT] = mfma32<BF>(f[n % kVAhead], pl[n / DT], o[n % DT]);
                if (n + kVAhead < N)
                    f[n % kVAhead] = at(n + kVAhead);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        __builtin_amdgcn_s_setprio(0);
        if (special)
            add_special(j0, has, pf);
    }

    // Adds p v for the infinities and NaN of v in block j0, to the rows that see
    // their key.  Rare, so it reads v again, key by key.
    __device__ __forceinline__ void add_special(int j0, uint64_t has, const u32x4 *pf)
    {
#pragma unroll 1
        for (int key = 0; key < kBlock; ++key) {
            if (!(has >> key & 1) || j0 + key > p_hi)
                continue;
            // weight e = 8 (key / 16) + ... of lane half (key / 4) % 2
            const int e = (key >> 5) * 16 + ((key >> 3) & 3) * 4 + (key & 3), from = (key >> 2) & 1;
            uint32_t pair = 0;
#pragma unroll
            for (int i = 0; i < 8 * KT; ++i)
                pair = e / 2 == i ? pf[i / 4][i % 4] : pair;
            const float w = as_float<BF>((uint16_t)(e & 1 ? pair >> 16 : pair));
            const float p = __shfl(w, 32 * from + col);
            if (!sees(a, p_row, j0 + key))
                continue;
            const char *src = vbase + 2 * paging.offset<true>(paging.checked(paging.raw(table, j0 + key)), j0 + key) + 2 * values + 8 * half;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const u32x2 x = *reinterpret_cast<const u32x2 *>(src + 2 * (32 * d + 8 * i));
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t one = e & 1 ? x[e / 2] >> 16 : x[e / 2] & 0xffffu;
                        const uint32_t odd = __builtin_amdgcn_sbfe(not_finite<BF>(one), 15, 1);
                        o[d][4 * i + e] = fmaf(p, as_float<BF>((uint16_t)(one & odd)), o[d][4 * i + e]);
                    }
                    asm volatile("" ::: "memory"); // one load at a time: registers are short here
                }
        }
    }
};

// A share of a row tile's keys.  k and v: two buffers each of a block's rows;
// they are free again on return.
template <bool BF, int D, bool F32OUT, int PAGES>
__device__ __forceinline__ void run_many(const AttnArgs &a, const Request &rq, int r, int tile, int head, const Share &sh,
                                         char *ka, char *va, char *kb, char *vb)
{
    constexpr int DT = D / many_halves(D) / 32, kBlock = many_block(D);
    constexpr uint64_t kAll = kBlock == 64 ? ~0ull : (1ull << kBlock % 64) - 1; // every key of a block has a page
    __shared__ int lds_last;
    __shared__ uint32_t flags[kWaves];
    ManyRows<BF, D, F32OUT, PAGES> t(a);
    t.begin(rq, r, tile, head);
    const Walk walk = walk_of<kBlock>(a, t.p_lo, t.p_hi);
    const int b0 = sh.from(walk.count), b1 = sh.to(walk.count);

    auto key = [&](int b) { return walk.block(b) * kBlock; };
    // Block b's scores are formed during block b - 1, so its k is copied two blocks
    // ahead and its v one.  id1: checked pages of block b + 1's keys (a lane's key
    // each), raw2: of block b + 2's as the table has them, so that their load is
    // waited for where they are used; has0, has1: which keys of b and b + 1 have one.
    const auto raw_at = [&](int b) { return b < b1 ? t.paging.raw(t.table, key(b) + t.lane) : -1; };
    int id1 = t.paging.checked(raw_at(b0)), raw2 = raw_at(b0 + 1);
    uint64_t has0 = __ballot(id1 >= 0), has1 = 0;
    f32x16 sa[t.KT], sb[t.KT];
    if (b0 < b1) {
        t.template fetch<false>(key(b0), id1, ka);
        t.template fetch<true>(key(b0), id1, va);
        id1 = t.paging.checked(raw2);
        has1 = __ballot(id1 >= 0);
        raw2 = raw_at(b0 + 2);
        if (b0 + 1 < b1)
            t.template fetch<false>(key(b0 + 1), id1, kb);
        __builtin_amdgcn_s_waitcnt(0x0f70); // vmcnt(0): this wave's rows are in LDS
        __syncthreads();
        t.scores(ka, sa, [](int) {});
    }
    // The buffers by name in two copies of the step: the compiler then knows that
    // reads of one need not wait for the copy into the other.  Past the last block
    // scores are formed of whatever lies in LDS, and dropped.
    const auto step = [&](int b, char *k, char *knext, char *v, char *vnext, f32x16 *s, f32x16 *next) {
        const int j0 = key(b);
        __builtin_amdgcn_s_waitcnt(0x0f70);
        __syncthreads(); // block b's v and b + 1's k are there; b's k and b - 1's v are done with
        const int id2 = t.paging.checked(raw2);
        if (b + 1 < b1)
            t.template fetch<true>(key(b + 1), id1, vnext);
        if (b + 2 < b1)
            t.template fetch<false>(key(b + 2), id2, k);
        raw2 = raw_at(b + 3);
        // one body for both kinds of block: in two, the sums would be copied between them
        const bool part = !sees_all(a, t.p_lo, t.p_hi, j0, kBlock) || (has0 & kAll) != kAll;
        const bool special = part && t.clean(j0, has0, v, flags);
        if (t.live)
            t.block(j0, has0, knext, v, part, special, s, next);
        has0 = has1;
        has1 = __ballot(id2 >= 0);
        id1 = id2;
    };
    for (int b = b0; b < b1; b += 2) {
        step(b, ka, kb, va, vb, sa, sb);
        if (b + 1 < b1)
            step(b + 1, kb, ka, vb, va, sb, sa);
    }

    if (sh.np > 1) {
        const Parts parts(a);
        const auto sums = [&](int i) { return sh.part(i) + t.wave * (1024 * DT) + 4 * t.lane; };
        const auto stats = [&](int i) { return sh.part(i) + kWaves * 1024 * DT + t.wave * (2 * kWave) + t.lane; };
        if (t.live) {
            const int to = sums(sh.me), st = stats(sh.me);
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    parts.put4(to + (d * 4 + e) * (4 * kWave),
                               f32x4{t.o[d][4 * e], t.o[d][4 * e + 1], t.o[d][4 * e + 2], t.o[d][4 * e + 3]});
            parts.put(st, t.m);
            parts.put(st + kWave, t.l);
        }
        if (!last_part(a, sh, t.thread, &lds_last))
            return;
        if (t.live) {
            t.m = kNegInf;
            t.l = 0.0f;
#pragma unroll
            for (int d = 0; d < DT; ++d)
                t.o[d] = f32x16{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
            for (int i0 = 0; i0 < sh.np; i0 += 2) { // two at a time: a round trip to memory each
                const int i1 = min(i0 + 1, sh.np - 1), from0 = sums(i0), from1 = sums(i1);
                f32x4 x[2][4 * DT];
                float m[2] = {parts.get(stats(i0)), parts.get(stats(i1))};
                float l[2] = {parts.get(stats(i0) + kWave), parts.get(stats(i1) + kWave)};
#pragma unroll
                for (int e = 0; e < 4 * DT; ++e) {
                    x[0][e] = parts.get4(from0 + e * (4 * kWave));
                    x[1][e] = parts.get4(from1 + e * (4 * kWave));
                }
                if (i1 == i0) { // counted once
                    m[1] = kNegInf;
                    l[1] = 0.0f;
#pragma unroll
                    for (int e = 0; e < 4 * DT; ++e)
                        x[1][e] = f32x4{0, 0, 0, 0};
                }
                const float next = fmaxf(t.m, fmaxf(m[0], m[1]));
                const float f = t.m == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(t.m - next);
                const float f0 = m[0] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(m[0] - next);
                const float f1 = m[1] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(m[1] - next);
                t.l = t.l * f + l[0] * f0 + l[1] * f1;
#pragma unroll
                for (int d = 0; d < DT; ++d)
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        t.o[d][e] = fmaf(x[1][4 * d + e / 4][e % 4], f1, fmaf(x[0][4 * d + e / 4][e % 4], f0, t.o[d][e] * f));
                t.m = next;
            }
        }
    }
    const float l = half_sum(t.l);
    const int row = tile * many_rows(D) + t.wave / many_halves(D) * 32 + t.col;
    if (row < rq.n * a.group) {
        const int i = div_by(a.per_group, row), g = row - i * a.group;
        const int64_t to = (int64_t)(rq.q0 + i) * a.o_ts + (int64_t)(head * a.group + g) * a.o_hs + t.values +
                           4 * t.half;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l; // no key seen: zeros
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                store4<BF, F32OUT>(a.out, to + 32 * d + 8 * e,
                                   f32x4{t.o[d][4 * e] * inv, t.o[d][4 * e + 1] * inv, t.o[d][4 * e + 2] * inv,
                                         t.o[d][4 * e + 3] * inv});
    }
    __syncthreads(); // the buffers are free for the next share
}

} // namespace
} // namespace gemv
