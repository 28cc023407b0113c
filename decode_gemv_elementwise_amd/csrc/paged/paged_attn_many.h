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
// Memory to LDS goes without registers, 16 bytes a lane, one block ahead of the
// products: two buffers for k and two for v, one barrier a block.  A row of
// D values lies in one piece; which 16-byte chunk of it a lane fetches is
// permuted by the row, so that the products' reads meet no bank twice (k_turn,
// v_turn).
//
// The running maximum only moves when a row's new one is more than kSlack above
// it (weights up to 2^kSlack are as good as weights up to 1): most blocks then
// skip the pass over the 32 x D sums.
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

template <bool BF, int D, bool F32OUT, bool PAGE8> struct ManyRows {
    static constexpr int kBlock = many_block(D), KT = kBlock / 32; // keys of a block; tiles of 32 of them
    static constexpr int kRowBytes = 2 * D, kChunks = D / 8;      // 16-byte chunks of a row
    static constexpr int kRun = kWave / kChunks;                  // rows that one wave instruction brings
    static constexpr int kFetch = kBlock / (kRun * kWaves);   // such instructions of a wave per block
    static constexpr int KS = D / 16;                             // k steps of the first product
    static constexpr int kHalves = many_halves(D), DW = D / kHalves, DT = DW / 32; // values of a wave, tiles of them
    static constexpr int kAhead = 2; // products between a read of LDS and its use
    // binary16's weights are lifted, which leaves one power of two to its largest
    static constexpr float kSlack = BF ? 8.0f : 1.0f;

    const AttnArgs &a;
    const char *kbase, *vbase; // of the key/value head
    const int32_t *table;      // of the request
    int p_lo, p_hi;            // positions of the tile's rows
    int w_lo, w_hi, p_row;     // of the wave's rows, of this lane's (-1: no row)
    bool live;                 // the wave has rows
    int thread, lane, wave, col, half;
    int values; // first of the wave's values
    int64_t k_lane, v_lane; // byte offset of the lane's row within a run
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
        kbase = reinterpret_cast<const char *>(a.k + head * a.k_stride[2]);
        vbase = reinterpret_cast<const char *>(a.v + head * a.v_stride[2]);
        table = a.table + r * a.table_stride;
        k_lane = 2 * (lane / kChunks) * a.k_stride[1];
        v_lane = 2 * (lane / kChunks) * a.v_stride[1];
        asm volatile("" : "+v"(k_lane), "+v"(v_lane)); // kept as they are: the rest of an address is the wave's
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

    // Starts the copy of block j0 into LDS; ids: the page of each lane's key.
    __device__ __forceinline__ void fetch(int j0, int ids, char *k, char *v) const
    {
        const int r = lane / kChunks, phys = lane % kChunks;
#pragma unroll
        for (int f = 0; f < kFetch; ++f) {
            const int row0 = (f * kWaves + wave) * kRun, row = row0 + r;
            const int kc = 16 * (phys ^ k_turn(row)), vc = 16 * (phys ^ v_turn(row));
            const char *kp, *vp;
            if constexpr (PAGE8) { // a run lies in one page
                const int id = __builtin_amdgcn_readlane(ids, row0);
                kp = kbase + 2 * key_offset(a, a.k_stride, id, j0 + row0) + k_lane;
                vp = vbase + 2 * key_offset(a, a.v_stride, id, j0 + row0) + v_lane;
            } else {
                const int id = __shfl(ids, row);
                kp = kbase + 2 * key_offset(a, a.k_stride, id, j0 + row);
                vp = vbase + 2 * key_offset(a, a.v_stride, id, j0 + row);
            }
            __builtin_amdgcn_global_load_lds((global_void *)(kp + kc), (lds_void *)(k + row0 * kRowBytes), 16, 0, 0);
            __builtin_amdgcn_global_load_lds((global_void *)(vp + vc), (lds_void *)(v + row0 * kRowBytes), 16, 0, 0);
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

    // One block of keys; part: some rows do not see some of its keys.
    template <bool PART> __device__ __forceinline__ void block(int j0, uint64_t has, const char *k, const char *v, bool special)
    {
        // places in LDS are formed here each time: all of them at once, for both
        // buffers, would not leave registers enough
        int ln = lane;
        asm volatile("" : "+v"(ln));
        f32x16 s[KT];
        {
            const int row = (ln & 31) * kRowBytes;
            const int turn = 16 * ((ln >> 5) ^ k_turn(ln & 31));
#pragma unroll
            for (int t = 0; t < KT; ++t)
                s[t] = f32x16{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
            // rows 32 apart have the same turn
            const auto read = [&](int n) {
                return *reinterpret_cast<const u32x4 *>(k + (row + n % KT * 32 * kRowBytes + (turn ^ (32 * (n / KT)))));
            };
            u32x4 f[kAhead];
#pragma unroll
            for (int n = 0; n < kAhead; ++n)
                f[n] = read(n);
            // the order is kept: left alone, the compiler waits for each read in turn
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int n = 0; n < KS * KT; ++n) {
                s[n % KT] = mfma32<BF>(f[n % kAhead], qf[n / KT], s[n % KT]);
                if (n + kAhead < KS * KT)
                    f[n % kAhead] = read(n + kAhead);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if constexpr (PART) {
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
        top = half_max(top) * a.scale_log2;
        if (__any(top > m + kSlack)) {
            const float to = fmaxf(m, top);
            const float f = to == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(m - to);
            l *= f;
#pragma unroll
            for (int d = 0; d < DT; ++d)
                o[d] *= f;
            m = to;
        }
        const float base = m == kNegInf ? 0.0f : BF ? m : m - kF16Lift;
        u32x4 pf[2 * KT], pl[F32OUT ? 2 * KT : 1];
#pragma unroll
        for (int t = 0; t < 2 * KT; ++t) {
            float p[8], rest[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                p[i] = __builtin_amdgcn_exp2f(fmaf(s[t / 2][8 * (t & 1) + i], a.scale_log2, -base));
                l += p[i];
            }
            pf[t] = round8<BF>(p, rest);
            if constexpr (F32OUT) {
                float none[8];
                pl[t] = round8<BF>(rest, none);
            }
        }
        {
            // 16 lanes bring 4 keys by 16 values
            const int key = 4 * (ln >> 5) + ((ln & 15) >> 2), chunk = 2 * ((ln >> 4) & 1) + ((ln & 3) >> 1);
            const int row = key * kRowBytes + 2 * values + 8 * (ln & 1);
            const int turn = 16 * (chunk ^ v_turn(key));
            const auto read = [&](int n) { // rows 8 apart have the same turn
                const int at = row + 16 * (n / DT) * kRowBytes + (turn ^ (64 * (n % DT)));
                const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(v + at));
                const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(v + (at + 8 * kRowBytes)));
                const u32x2 lo = __builtin_bit_cast(u32x2, x), hi = __builtin_bit_cast(u32x2, y);
                return u32x4{lo[0], lo[1], hi[0], hi[1]};
            };
            u32x4 f[kAhead];
#pragma unroll
            for (int n = 0; n < kAhead; ++n)
                f[n] = read(n);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int n = 0; n < 2 * KT * DT; ++n) {
                o[n % DT] = mfma32<BF>(f[n % kAhead], pf[n / DT], o[n % DT]);
                if constexpr (F32OUT)
                    o[n % DT] = mfma32<BF>(f[n % kAhead], pl[n / DT], o[n % DT]);
                if (n + kAhead < 2 * KT * DT)
                    f[n % kAhead] = read(n + kAhead);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if constexpr (PART)
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
            const char *src = vbase + 2 * key_offset(a, a.v_stride, id_of(a, table, j0 + key), j0 + key) + 2 * values + 8 * half;
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
template <bool BF, int D, bool F32OUT, bool PAGE8>
__device__ __forceinline__ void run_many(const AttnArgs &a, const Request &rq, int r, int tile, int head, const Share &sh,
                                         char *ka, char *va, char *kb, char *vb)
{
    constexpr int DT = D / many_halves(D) / 32, kBlock = many_block(D);
    constexpr uint64_t kAll = kBlock == 64 ? ~0ull : (1ull << kBlock % 64) - 1; // every key of a block has a page
    __shared__ int lds_last;
    __shared__ uint32_t flags[kWaves];
    ManyRows<BF, D, F32OUT, PAGE8> t(a);
    t.begin(rq, r, tile, head);
    const Walk walk = walk_of<kBlock>(a, t.p_lo, t.p_hi);
    const int b0 = sh.from(walk.count), b1 = sh.to(walk.count);

    auto key = [&](int b) { return walk.block(b) * kBlock; };
    // ids of the block after next, and which keys of this and the next have a page
    // (an id is checked where it is used, so that its load is waited for there)
    const auto id_at = [&](int b) { return raw_id(a, t.table, key(b) + t.lane); };
    int ids = b0 < b1 ? checked_id(a, id_at(b0)) : -1;
    uint64_t has = 0, has_next = __ballot(ids >= 0);
    if (b0 < b1)
        t.fetch(key(b0), ids, ka, va);
    if (b0 + 1 < b1)
        ids = id_at(b0 + 1);
    // The buffers by name in two copies of the step: the compiler then knows that
    // reads of one need not wait for the copy into the other.
    const auto step = [&](int b, char *k, char *v, char *knext, char *vnext) {
        const int j0 = key(b);
        has = has_next;
        __builtin_amdgcn_s_waitcnt(0x0f70); // vmcnt(0): this wave's rows of the block are in LDS
        __syncthreads();                    // everyone's are, and everyone is done with the other buffers
        if (b + 1 < b1) {
            ids = checked_id(a, ids);
            has_next = __ballot(ids >= 0);
            t.fetch(key(b + 1), ids, knext, vnext);
            if (b + 2 < b1)
                ids = id_at(b + 2);
        }
        if (!sees_all(a, t.p_lo, t.p_hi, j0, kBlock) || (has & kAll) != kAll) {
            const bool special = t.clean(j0, has, v, flags);
            if (t.live && j0 <= t.w_hi)
                t.template block<true>(j0, has, k, v, special);
        } else if (t.live) {
            t.template block<false>(j0, has, k, v, false);
        }
    };
    for (int b = b0; b < b1; b += 2) {
        step(b, ka, va, kb, vb);
        if (b + 1 < b1)
            step(b + 1, kb, vb, ka, va);
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
