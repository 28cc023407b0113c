// Row tiles of many rows (chunks): 128 rows (token, query head) that share one
// key/value head, 32 to each of four waves, over blocks of 64 keys that the workgroup
// widens to q's type into LDS once for all of them.
//
// As with few rows the products are taken transposed, here 32 x 32 x 16:
//     S^T = K Q^T (32 keys x 32 rows, twice),   O^T = V^T P^T.
// A lane then holds 16 scores of one row per 32 keys, keys 8 (i / 4) + 4 h + i % 4 for
// lane half h, so statistics stay in the lane but for one exchange with the lane 32
// away.  The order of keys along the second product's k is free as long as both
// operands agree: P^T is taken as it lies, and V's operand is read from LDS in that
// order, turned on the way by the transposing 64-bit LDS read (4 keys by 16 values to
// 16 lanes).  A wave forms a block's weights while the matrix core forms the next
// block's scores.
//
// Codes come through registers, 16 bytes a lane: k's are asked for at a block's start
// and widened into LDS among its products with v, v's are asked for between its two
// products and widened at its end, in the same step or (kDeep) the next.  Two buffers for k
// and two for v, one barrier a block.  Which 16-byte chunk of a row lies where is permuted
// by the row, so that the products' reads meet no bank twice (k_turn, v_turn).
//
// The running maximum only moves when a row's new one is more than kSlack above it:
// most blocks then skip the pass over the 32 x D sums.  A weight may then be up to
// 2^kSlack, and the largest, which would be 1, is rounded like the others.
//
// 2048 tokens over 8192 keys, 32/8 heads of 128, take 266 to 277 us in e4m3 (868 to 902
// TFLOP/s) and 300 in int8, 312 with binary16; the 16-bit cache's kernel 268.  Neither the
// matrix cores (237 M of their cycles, 100 us of the time) nor the vector units (65 M
// instructions, 120 us) are full: they wait for one another.  Without widening v it would be
// 250: each tile widens all its codes itself.  Bank conflicts on the way into LDS cost 20 us
// before rows were turned, k's widening ahead of the products 27.  A float32 result takes 355
// (int8 380), for its second products; pages of 8 and 24, whose keys are found one by one,
// 273 and 270.  2048 tokens over themselves 65, 8192 791: the plan counts every tile
// of a request for its last one.
#pragma once

#include "paged8_attn_device.h"

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

// RUNS: 16 keys from a multiple of 16 on lie in one page, and a block of scales does not
// begin or end within them, or is a power of two below 16.
template <int CODE, bool BF, int D, bool F32OUT, bool RUNS> struct ManyRows {
    static constexpr int kBlock = many_block(D), KT = kBlock / 32; // keys of a block; tiles of 32 of them
    static constexpr int kRowBytes = 2 * D, kChunks = D / 8;      // 16-byte chunks of a row
    static constexpr int kOwn = kBlock / kWaves;                  // rows, next to each other, that a wave brings
    static constexpr int kPieces = D / 16, kRun = kWave / kPieces; // lanes of a row's codes; rows of one instruction
    static constexpr int kAsk = kOwn / kRun;                      // such instructions of a wave per block
    static_assert(kOwn % kRun == 0, "a wave's rows are whole instructions");
    static constexpr int KS = D / 16;                             // k steps of the first product
    static constexpr int kHalves = many_halves(D), DW = D / kHalves, DT = DW / 32; // values of a wave, tiles of them
    static constexpr int kAhead = 2, kVAhead = 2; // products between a read of LDS and its use
    // binary16's weights are lifted, which leaves one power of two to its largest
    static constexpr float kSlack = BF ? 8.0f : 1.0f;
    // m of this size has steps of 2^-16 (and 2^-17 below): what its rounding moves a weight by
    static constexpr float kFar = 128.0f;

    const Attn8Args &a;
    Paging8 at;
    int p_lo, p_hi;            // positions of the tile's rows
    int w_lo, w_hi, p_row;     // of the wave's rows, of this lane's (-1: no row)
    bool live;                 // the wave has rows
    int thread, lane, wave, col, half;
    int values; // first of the wave's values
    float scale;
    uint32_t scale_row[RUNS ? kAsk : 1]; // blocks of scales between the wave's first row and the lane's
    uint32_t special; // not 0: an infinity or NaN of v was taken out
    u32x4 qf[KS];
    f32x16 o[DT];
    float m, l;

    __device__ ManyRows(const Attn8Args &args) : a(args) {}

    // Where a row's chunk c lies: at place(c) ^ turn.  A lane writes chunks 2 i and 2 i + 1,
    // eight lanes next to each other all 2 i at a time: those fill the row's first half.
    // k is read 16 rows at a time, one chunk of each; v 4 rows at a time, 64 bytes of each.
    static __device__ __forceinline__ int place(int c) { return (c >> 1) + (c & 1) * (kChunks / 2); }
    static __device__ __forceinline__ int k_turn(int row)
    {
        return (kRowBytes == 128 ? row >> 1 : row) & (kChunks < 16 ? kChunks - 1 : 15);
    }
    static __device__ __forceinline__ int v_turn(int row) { return kRowBytes == 128 ? row & 2 : (row & 3) << 1; }

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
        at.begin(a, r, head);
        scale = kept(a.scale_log2);
        special = 0;
        if constexpr (RUNS) {
#pragma unroll
            for (int f = 0; f < kAsk; ++f)
                scale_row[f] = div_by(at.block, f * kRun + lane / kPieces);
        }
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

    // A lane's 16-byte pieces of a block of k (or v), and their rows' scales.
    struct Raw {
        u32x4 x[kAsk];
        uint8_t s[kAsk];
    };
    __device__ __forceinline__ int own_row(int f) const { return wave * kOwn + f * kRun + lane / kPieces; }

    // Asks for them; ids: the page of each lane's key.
    template <bool V> __device__ __forceinline__ void ask(int j0, int ids, Raw &raw) const
    {
        if constexpr (RUNS) { // a wave's rows lie in one page, whose place is the same for all lanes
            const int own = wave * kOwn, id = __builtin_amdgcn_readlane(ids, own);
            const uint8_t *base = at.template codes<V>(id, j0 + own), *scales = at.template scale<V>(id, j0 + own);
            const uint32_t step = V ? at.v1 : at.k1, sstep = V ? at.vs1 : at.ks1;
            const uint32_t off = lane / kPieces * step + 16 * (lane % kPieces);
#pragma unroll
            for (int f = 0; f < kAsk; ++f) {
                raw.x[f] = *reinterpret_cast<const u32x4 *>(base + (uint64_t)(f * kRun) * step + off);
                raw.s[f] = scales[scale_row[f] * sstep];
            }
            return;
        }
#pragma unroll
        for (int f = 0; f < kAsk; ++f) {
            const int row = own_row(f), id = __shfl(ids, row);
            raw.x[f] = *reinterpret_cast<const u32x4 *>(at.template codes<V>(id, j0 + row) + 16 * (lane % kPieces));
            raw.s[f] = *at.template scale<V>(id, j0 + row);
        }
    }

    // Widens them into LDS: one of 2 kAsk chunks, or all.
    template <bool V> __device__ __forceinline__ void put(const Raw &raw, char *to, int i) const
    {
        const int f = i / 2, row = own_row(f), chunk = lane % kPieces ^ (V ? v_turn(row) : k_turn(row));
        const Scale<CODE, BF> s(raw.s[f]);
        *reinterpret_cast<u32x4 *>(to + row * kRowBytes + 16 * (i % 2 ? chunk ^ kChunks / 2 : chunk)) =
            widen8<CODE, BF>(raw.x[f][i % 2 * 2], raw.x[f][i % 2 * 2 + 1], s);
    }
    template <bool V> __device__ __forceinline__ void put(const Raw &raw, char *to) const
    {
#pragma unroll
        for (int i = 0; i < 2 * kAsk; ++i)
            put<V>(raw, to, i);
    }

    // Makes a block of v safe to multiply by weights of 0: keys past the tile's
    // last row and keys without a page hold anything and are taken as 0, and an
    // infinity or NaN of a key that only some rows see is taken out (add_special adds
    // it at the share's end for the rows that see it).
    __device__ __forceinline__ void clean(int j0, uint64_t has, char *v)
    {
        for (int c = thread; c < kBlock * kChunks; c += kThreads) {
            const int key = c / kChunks;
            u32x4 x = *reinterpret_cast<u32x4 *>(v + c * 16);
            const bool keep = (has >> key & 1) && j0 + key <= p_hi;
            uint32_t drop = keep ? 0 : 1;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                x[w] = keep ? x[w] : 0;
                const uint32_t n = not_finite<BF>(x[w]);
                x[w] &= ~((n >> 15) * 0xffffu);
                special |= n;
                drop |= n;
            }
            if (drop)
                *reinterpret_cast<u32x4 *>(v + c * 16) = x;
        }
        __syncthreads();
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
            : k(k), row((ln & 31) * kRowBytes), turn(16 * (place(ln >> 5) ^ k_turn(ln & 31)))
        {
        }
        __device__ __forceinline__ u32x4 operator()(int n) const // rows 32 apart have the same turn
        {
            return *reinterpret_cast<const u32x4 *>(k + ((row + turn) ^ (16 * (n / KT))) + n % KT * 32 * kRowBytes);
        }
    };
    struct VAt {
        const char *v;
        int row, turn;
        // 16 lanes bring 4 keys by 16 values
        __device__ __forceinline__ VAt(const char *v, int ln, int values) : v(v)
        {
            const int key = 4 * (ln >> 5) + ((ln & 15) >> 2), chunk = 2 * ((ln >> 4) & 1) + ((ln & 3) >> 1);
            row = key * kRowBytes + 8 * (ln & 1);
            turn = 16 * ((place(chunk) + values / 16) ^ v_turn(key)); // 2 DT values / 16 at most: no bit of them meets
        }
        __device__ __forceinline__ u32x4 operator()(int n) const // rows 8 apart have the same turn
        {
            const char *at = v + ((row + turn) ^ (32 * (n % DT)));
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
    // part: some rows do not see some of its keys.  between: work to do after the scores;
    // among(i): that of 2 kAsk pieces, spread over the products with v.
    template <class F, class G>
    __device__ __forceinline__ void block(int j0, uint64_t has, const char *k, const char *v, bool part, f32x16 *s,
                                          f32x16 *next, F between, G among)
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
        // s scale - m, both rounded alike, first.
        const float base = m == kNegInf ? 0.0f : m;
        float by = scale, off = BF ? base : base - kF16Lift;
        if (__any(__builtin_fabsf(base) >= kFar)) {
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    s[t][i] = s[t][i] * scale - base;
            by = 1.0f;
            off = BF ? 0.0f : -kF16Lift;
        }
        // The weights in pairs, rounded to 16 bits as the product takes them, the largest too (of up to
        // 2^kSlack it is no power of two), while l has them whole: 0.0023 of a bf16 result in all,
        // 0.0017 with exact weights.  For a float32 result a second piece holds the rest.
        u32x4 pf[2 * KT], pl[F32OUT ? 2 * KT : 1];
        // the other workgroup's wave on this SIMD widens its codes meanwhile, at the lower priority
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
        between();
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
                constexpr int kEvery = N / (2 * kAsk);
                if (n % kEvery == kEvery / 2)
                    among(n / kEvery);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        __builtin_amdgcn_s_setprio(0);
    }

    // Adds the infinities and NaN of v of block j0 to the rows that see their key,
    // whatever its weight: that makes no difference to them.  Rare, so it reads v again,
    // key by key.
    __device__ __forceinline__ void add_special(int j0)
    {
#pragma unroll 1
        for (int j = j0; j < j0 + kBlock; ++j) {
            const int id = at.checked(at.raw(j));
            if (id < 0 || !sees(a, p_row, j))
                continue;
            const uint8_t *src = at.template codes<true>(id, j) + values + 4 * half;
            const Scale<CODE, BF> f(*at.template scale<true>(id, j));
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const u32x2 x = widen4<CODE, BF>(*reinterpret_cast<const uint32_t *>(src + 32 * d + 8 * i), f);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t one = e & 1 ? x[e / 2] >> 16 : x[e / 2] & 0xffffu;
                        o[d][4 * i + e] += not_finite<BF>(one) & 0x8000u ? as_float<BF>((uint16_t)one) : 0.0f;
                    }
                    asm volatile("" ::: "memory"); // one load at a time: registers are short here
                }
        }
    }
};

// One share of a tile of many rows.
template <int CODE, bool BF, int D, bool F32OUT, bool RUNS> struct ManyTile {
    typedef ManyRows<CODE, BF, D, F32OUT, RUNS> Rows;
    static constexpr int kRows = many_rows(D), kPart = many_part(D);
    static constexpr uint32_t kLeast = D == 64 ? 16 : 8, kEdge = 8;
    static constexpr int kBuffer = Rows::kBlock * Rows::kRowBytes;
    // Codes are on their way for a step more where there are registers: 2048 tokens over 8192
    // keys of heads of 64 189 to 181 us, 64 over 32768 63 to 57; of 256 166 to 162.  Heads of
    // 128 have none left (273 to 285).
    static constexpr int kDeep = D == 128 ? 0 : 1;

    // lds: two buffers for k and two for v, free again on return
    static __device__ __forceinline__ void run(const Attn8Args &a, const Request &rq, int r, int tile, int head, int,
                                               const Share &sh, char *lds)
    {
        constexpr int DT = Rows::DT, kBlock = Rows::kBlock;
        constexpr uint64_t kAll = kBlock == 64 ? ~0ull : (1ull << kBlock % 64) - 1; // every key of a block has a page
        __shared__ int lds_last;
        char *const ka = lds, *const va = lds + kBuffer, *const kb = lds + 2 * kBuffer, *const vb = lds + 3 * kBuffer;
        Rows t(a);
        t.begin(rq, r, tile, head);
        const Walk walk = walk_of<kBlock>(a, t.p_lo, t.p_hi);
        const int b0 = sh.from(walk.count), b1 = sh.to(walk.count);

        const auto key = [&](int b) { return walk.block(b) * kBlock; };
        // Block b's scores are formed during block b - 1, so its k is widened two blocks
        // ahead and its v one; both are asked for kDeep blocks before.  idm: checked pages of
        // block b + kDeep + 1's keys (a lane's key each), raw: of the next block's as the table
        // has them, so that their load is waited for where they are used; has: which keys of b
        // and the blocks after it have one.
        const auto raw_at = [&](int b) { return b < b1 ? t.at.raw(key(b) + t.lane) : -1; };
        const auto last = [&](int b) { return key(min(b, b1 - 1)); }; // past the last block its codes are widened again, and dropped
        uint64_t has[kDeep + 2];
        int idm = 0, raw = 0;
        f32x16 sa[Rows::KT], sb[Rows::KT];
        typename Rows::Raw x[kDeep + 1], y[kDeep + 1];
        if (b0 < b1) {
            int ids[kDeep + 2];
#pragma unroll
            for (int i = 0; i < kDeep + 2; ++i)
                ids[i] = raw_at(b0 + i);
            raw = raw_at(b0 + kDeep + 2);
#pragma unroll
            for (int i = 0; i < kDeep + 2; ++i) {
                ids[i] = t.at.checked(ids[i]);
                has[i] = __ballot(ids[i] >= 0);
            }
            typename Rows::Raw z, u;
            t.template ask<false>(key(b0), ids[0], z);
            t.template ask<true>(key(b0), ids[0], u);
            t.template put<false>(z, ka);
            t.template put<true>(u, va);
            t.template ask<false>(last(b0 + 1), ids[1], z);
            if constexpr (kDeep) {
                t.template ask<false>(last(b0 + 2), ids[kDeep + 1], x[0]);
                t.template ask<true>(last(b0 + 1), ids[1], y[0]);
            }
            t.template put<false>(z, kb);
            idm = ids[kDeep + 1];
            __syncthreads();
            t.scores(ka, sa, [](int) {});
        }
        // The buffers by name in two copies of the step: the compiler then knows that
        // reads of one need not wait for the writes of the other.  Past the last block
        // scores are formed of whatever lies in LDS, and dropped.
        const auto step = [&](int b, char *k, char *knext, char *v, char *vnext, f32x16 *s, f32x16 *next,
                              typename Rows::Raw &xnow, typename Rows::Raw &xnext, typename Rows::Raw &ynow,
                              typename Rows::Raw &ynext) {
            const int j0 = key(b);
            __syncthreads(); // block b's v and b + 1's k are there; b's k and b - 1's v are done with
            const int idl = t.at.checked(raw);
            t.template ask<false>(last(b + kDeep + 2), idl, xnext);
            raw = raw_at(b + kDeep + 3);
            const auto between = [&] {
                if constexpr (F32OUT) // both pieces of the weights leave no registers for k's codes among the products
                    t.template put<false>(xnow, k);
                t.template ask<true>(last(b + kDeep + 1), idm, ynext);
            };
            const auto among = [&](int i) {
                if constexpr (!F32OUT)
                    t.template put<false>(xnow, k, i);
            };
            // one body for both kinds of block: in two, the sums would be copied between them
            const bool part = !sees_all(a, t.p_lo, t.p_hi, j0, kBlock) || (has[0] & kAll) != kAll;
            if (part)
                t.clean(j0, has[0], v);
            if (t.live) {
                t.block(j0, has[0], knext, v, part, s, next, between, among);
            } else {
                between();
#pragma unroll
                for (int i = 0; i < 2 * Rows::kAsk; ++i)
                    among(i);
            }
            t.template put<true>(ynow, vnext);
#pragma unroll
            for (int i = 0; i < kDeep + 1; ++i)
                has[i] = has[i + 1];
            has[kDeep + 1] = __ballot(idl >= 0);
            idm = idl;
        };
        for (int b = b0; b < b1; b += 2) {
            step(b, ka, kb, va, vb, sa, sb, x[0], x[kDeep], y[0], y[kDeep]);
            if (b + 1 < b1)
                step(b + 1, kb, ka, vb, va, sb, sa, x[kDeep], x[0], y[kDeep], y[0]);
        }
        if (__syncthreads_or(t.special != 0))
            for (int b = b0; b < b1; ++b)
                t.add_special(key(b));

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
        const int row = tile * kRows + t.wave / many_halves(D) * 32 + t.col;
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
};

template <int CODE, bool BF, int D, bool F32OUT, bool RUNS>
__global__ __launch_bounds__(kThreads, 2) void paged8_many_kernel(Attn8Args)
{
    typedef ManyTile<CODE, BF, D, F32OUT, RUNS> Tile;
    __shared__ __align__(16) char lds[4 * Tile::kBuffer];
    run_plan<Tile>(lds);
}

} // namespace
} // namespace gemv
