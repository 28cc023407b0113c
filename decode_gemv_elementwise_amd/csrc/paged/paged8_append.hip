// Rotary positions and the quantising write into a paged cache of 8-bit codes
// (gemv_paged8_append).
//
// Tokens of one call in one block of a page share its scale, so they form a run, and a
// run's head is written as one: a wave holds it whole, a lane 16 values of a token (for
// halves 8 and their 8 partners), turned by angles that it forms once for all its heads.
// Largest size, scale and codes then come from registers: k and v are read once and
// written once, and waves do not wait for one another.  A workgroup finds the runs that
// begin within its few tokens from the slots alone and deals their heads out to its
// waves.  A single token is one sixteenth of a wave's values or so: there a wave takes
// several heads at once.  Blocks of more tokens than a wave holds are taken by four,
// which exchange the largest size through LDS.  q goes by workgroups of its own, one a
// token, whose threads share the angles through LDS.
//
// A size is compared by its bits: of floats from 0 up they are ordered like whole
// numbers, infinities and NaN above all others.
//
// Memory-bound where the tokens are many: 8192 of 32 + 2 x 8 heads of 128, bf16 to e4m3 in
// blocks of 16, take 40 to 42 us, 4.4 to 4.6 TB/s of the 185 MB that they are: 134 at first,
// 47 once a wave held a run's head whole, 40 once a die's stretches were neighbours (in blocks
// of 64 80 and 38).  Latency-bound where they are few: 8 tokens 6.9 us, for slots, then what
// the block holds, then its codes follow one another.  Where a single token makes its block's
// scale grow, the lanes of its head (8 of 128 values) rescale the block, a read and a write
// after the other: 8 tokens into blocks of 16, 32, 64 and 128 take 15, 25, 52 and 96 us in int8 and
// 13, 23, 46 and 87 in e4m3 where every block grows.
#include "paged8_device.h"
#include "rotary.h"

namespace gemv {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / kWave;
constexpr int64_t kMostGroups = 1 << 29; // workgroups of either part, where larger shares can see to it

struct Append8Args {
    const void *src[3]; // q, k, v
    int64_t src_stride[3];
    const int32_t *positions, *axis, *slots;
    const float *inv_freq;
    void *q_out;
    uint8_t *codes[2], *scales[2]; // k, v
    int64_t c_stride[2][3], s_stride[2][3];
    int32_t tokens, axes, q_heads, heads, dim, half; // half = rot / 2
    int32_t num_slots;
    int32_t pairs, e4m3, bf;     // pairing by neighbours; the codes; q_out's type
    FastDiv page, block;
    FastDiv items;               // lanes that a token's head takes
    FastDiv q_items;             // items of 16 values that a token's q has
    FastDiv q_shares, kv_shares; // workgroups that share one token's q, one stretch's k and v
    int32_t stretch;             // tokens in which a workgroup looks for runs
    int32_t die_stretches;       // stretches of a die
    int32_t q_share, kv_share;   // items of q, rows of k and v of a workgroup
    int32_t q_tokens;            // tokens of a q workgroup
    int32_t kv_groups, groups;   // workgroups for k and v, and all
};

// Sixteen values of a row, eight from lo on and eight from hi on, as they lie in memory.
template <class S> struct Raw16 {
    u32x4 x[sizeof(S)];
    __device__ __forceinline__ void load(const S *row, int lo, int hi)
    {
        constexpr int N = sizeof(S) / 2;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            x[i] = reinterpret_cast<const u32x4 *>(row + lo)[i];
            x[N + i] = reinterpret_cast<const u32x4 *>(row + hi)[i];
        }
    }
    __device__ __forceinline__ void widen(float *v) const
    {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if constexpr (sizeof(S) == 4) {
                const uint32_t w = x[i / 4][i % 4];
                v[i] = __builtin_bit_cast(float, w);
            } else {
                const uint16_t w = (uint16_t)(x[i / 8][i % 8 / 2] >> (16 * (i % 2)));
                v[i] = (float)__builtin_bit_cast(S, w);
            }
        }
    }
};

// Where a lane's sixteen values lie in a row of q or k.  Pair 8 item + e is values
// (2 e, 2 e + 1) of them, or (e, 8 + e) for halves.
struct Place {
    int lo, hi;
};
template <bool PAIRS> __device__ __forceinline__ Place place_of(const Append8Args &a, int item)
{
    if (PAIRS)
        return Place{16 * item, 16 * item + 8};
    if (8 * item < a.half)
        return Place{8 * item, a.half + 8 * item};
    const int lo = 2 * a.half + 16 * (item - a.half / 8);
    return Place{lo, lo + 8};
}

__device__ __forceinline__ float2 turn_at(const Append8Args &a, int t, int pair)
{
    const int ax = a.axis ? a.axis[pair] : 0;
    return (unsigned)ax < (unsigned)a.axes ? turn_close(a.positions[(int64_t)ax * a.tokens + t], a.inv_freq[pair])
                                           : float2{1.0f, 0.0f};
}

// The turns of a lane's eight pairs; pairs past rot are not turned.
__device__ __forceinline__ void turns_of(const Append8Args &a, int t, int item, float2 *turn)
{
#pragma unroll
    for (int e = 0; e < 8; ++e)
        turn[e] = 8 * item + e < a.half ? turn_at(a, t, 8 * item + e) : float2{1.0f, 0.0f};
}

__device__ __forceinline__ void turn_pair(float &x, float &y, float2 cs)
{
    const float nx = fmaf(x, cs.x, -(y * cs.y)), ny = fmaf(y, cs.x, x * cs.y);
    x = nx;
    y = ny;
}

// Turns a lane's values.  What is not turned stays as it is, infinities among it.
template <bool PAIRS> __device__ __forceinline__ void turn16(const Append8Args &a, int item, const float2 *turn, float *x)
{
    if constexpr (PAIRS) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (8 * item + e < a.half)
                turn_pair(x[2 * e], x[2 * e + 1], turn[e]);
    } else if (8 * item < a.half) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            turn_pair(x[e], x[8 + e], turn[e]);
    }
}

__device__ __forceinline__ void store16(const Append8Args &a, uint16_t *row, Place p, const float *x)
{
    u32x4 lo, hi;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        lo[i] = a.bf ? pack2<true>(x[2 * i], x[2 * i + 1]) : pack2<false>(x[2 * i], x[2 * i + 1]);
        hi[i] = a.bf ? pack2<true>(x[8 + 2 * i], x[9 + 2 * i]) : pack2<false>(x[8 + 2 * i], x[9 + 2 * i]);
    }
    *reinterpret_cast<u32x4 *>(row + p.lo) = lo;
    *reinterpret_cast<u32x4 *>(row + p.hi) = hi;
}

// Four values times 2^(127 - b) as codes.  Within the codes' range, so an e4m3 needs no
// limit, and a whole number is the low byte of its sum with 1.5 2^23, rounded to even.
__device__ __forceinline__ uint32_t codes4(bool e4m3, const float *x, float inv)
{
    if (e4m3) {
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * inv, x[1] * inv, 0, false);
        return __builtin_amdgcn_cvt_pk_fp8_f32(x[2] * inv, x[3] * inv, lo, true);
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __builtin_bit_cast(uint32_t, fmaf(x[i], inv, 12582912.0f));
    const uint32_t lo = __builtin_amdgcn_perm(w[1], w[0], 0x0c0c0400u), hi = __builtin_amdgcn_perm(w[3], w[2], 0x04000c0cu);
    return lo | hi;
}

// The largest over a wave.
__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
    v = max(v, dpp<0x111, 0xf>(v));
    v = max(v, dpp<0x112, 0xf>(v));
    v = max(v, dpp<0x114, 0xf>(v));
    v = max(v, dpp<0x118, 0xf>(v));
    v = max(v, dpp<0x142, 0xa>(v));
    v = max(v, dpp<0x143, 0xc>(v));
    return __builtin_amdgcn_readlane(v, kWave - 1);
}

// The scale's byte for a largest size (its bits).  127 is 1.984375 2^6, 448 is 1.75 2^8.
__device__ __forceinline__ int byte_of(bool e4m3, uint32_t bits)
{
    if (bits >= 0x7f800000u)
        return 255;
    const int e = bits >> 23, m = bits & 0x7fffffu;
    return max(1, e4m3 ? e - 8 + (m > 0x600000) : e - 6 + (m > 0x7e0000));
}

// 2^(127 - b); a block that is NaN needs no codes.  2^-127, for the largest scale, is below
// the normal numbers: half the least of them.
__device__ __forceinline__ float inverse_of(int b)
{
    return b == 255 ? 0.0f : __builtin_bit_cast(float, max((uint32_t)(254 - b) << 23, 0x00400000u));
}

// Tokens [first, first + n) of one block.
struct Run {
    int first, n, block;
    int slot;      // the first token's
    bool begun;    // the block's first place is among theirs
    bool straight; // their places follow one another
};

__device__ __forceinline__ int slot_at(const Append8Args &a, uint32_t t) { return t < (uint32_t)a.tokens ? a.slots[t] : -1; }

// A slot's block; -1 where it is none.
__device__ __forceinline__ int block_of(const Append8Args &a, int slot)
{
    return slot >= 0 && slot < a.num_slots ? (int)div_by(a.block, slot) : -1;
}

// Adds the run's next tokens, at most a wave's: lane i's slot is that of token `at` + i.
// True where the run may go on behind them.
__device__ __forceinline__ bool extend(const Append8Args &a, Run &r, uint32_t at, int slot, int lane)
{
    const int from = (int)((uint32_t)r.first + r.n - at); // lane of the next token
    const uint64_t other = __ballot(block_of(a, slot) != r.block) & (~0ull << from);
    const int to = other ? __builtin_ctzll(other) : kWave;
    const bool mine = lane >= from && lane < to;
    r.begun = r.begun || __any(mine && slot == r.block * (int)a.block.d);
    r.straight = r.straight && !__any(mine && (uint32_t)slot - r.slot != at + lane - r.first);
    r.n += to - from;
    return to == kWave;
}

// Whether one of the run's tokens has place p of the block.
__device__ __forceinline__ bool has_place(const Append8Args &a, const Run &r, int p)
{
    const int slot = r.block * (int)a.block.d + p;
    if (r.straight)
        return slot >= r.slot && slot - r.slot < r.n;
    for (int i = 0; i < r.n; ++i)
        if (a.slots[r.first + i] == slot)
            return true;
    return false;
}

// A head's codes and scale of a block.
struct Target {
    uint8_t *codes;
    uint8_t *scale;
    int64_t place; // stride of places
};
__device__ __forceinline__ Target target_of(const Append8Args &a, int block, int v, int head)
{
    const uint32_t first = (uint32_t)block * a.block.d, id = div_by(a.page, first), in = first - id * a.page.d;
    const int64_t *c = a.c_stride[v], *s = a.s_stride[v];
    return Target{a.codes[v] + id * c[0] + in * c[1] + head * c[2],
                  a.scales[v] + id * s[0] + div_by(a.block, in) * s[1] + head * s[2], c[1]};
}

// What a block holds beside the run (taken(p): place p is one of its tokens'), from scale
// byte `old` to the larger b, by `threads` threads of which this is the i-th.  16 codes at
// a time.
template <class F>
__device__ __forceinline__ void rescale(const Append8Args &a, F taken, const Target &to, int old, int b, int i, int threads)
{
    const int pieces = a.dim / 16;
    const float f = __builtin_bit_cast(float, (uint32_t)max(127 + old - b, 0) << 23); // a step so small leaves 0 either way
    for (int at = i; at < (int)a.block.d * pieces; at += threads) {
        const int p = at / pieces;
        if (taken(p))
            continue;
        u32x4 *const w = reinterpret_cast<u32x4 *>(to.codes + p * to.place + 16 * (at - p * pieces));
        u32x4 x = *w;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const f32x4 y = a.e4m3 ? floats4<GEMV_KV_E4M3>(x[e]) : floats4<GEMV_KV_INT8>(x[e]);
            const float z[4] = {y[0], y[1], y[2], y[3]};
            x[e] = codes4(a.e4m3, z, f);
        }
        *w = x;
    }
}

// A grid's x counts its threads in 32 bits, so past 2^16 workgroups y goes on.
constexpr int64_t kGroupsX = 65536;
__device__ __forceinline__ int group_here() { return blockIdx.y * kGroupsX + blockIdx.x; }

// The workgroups of k and v: stretches of tokens times shares of the 2 heads rows.
// one(run, share): the work on a run.
template <class F> __device__ __forceinline__ void each_run(const Append8Args &a, int group, F one)
{
    const int lane = threadIdx.x & (kWave - 1);
    // Workgroups go to the 8 dies in turn, and of a chunk's stretches one in so many begins a
    // run: a die takes neighbouring ones, so that no die gets all of those.
    const int turn = group / 8, at = div_by(a.kv_shares, turn), share = turn - at * a.kv_shares.d;
    const uint32_t t0 = ((uint32_t)(group % 8) * a.die_stretches + at) * a.stretch;
    if (t0 >= (uint32_t)a.tokens)
        return;
    // lane i: does a run begin at token t0 + i; a stretch is shorter than a wave
    const int slot = slot_at(a, t0 + lane), before = slot_at(a, t0 + lane - 1), mine = block_of(a, slot);
    uint64_t begins = __ballot(lane < a.stretch && mine >= 0 && mine != block_of(a, before));
    while (begins) {
        const int i = __builtin_ctzll(begins);
        begins &= begins - 1;
        Run r{(int)(t0 + i), 0, (int)__builtin_amdgcn_readlane(mine, i), (int)__builtin_amdgcn_readlane(slot, i), false, true};
        bool more = extend(a, r, t0, slot, lane);
        while (more) {
            const uint32_t next = (uint32_t)r.first + r.n;
            more = extend(a, r, next, slot_at(a, next + lane), lane);
        }
        one(r, share);
    }
}

// q of a few tokens, an item of 16 values a thread; the turns are formed while the first
// items are on their way.
template <class S, bool PAIRS> __device__ __forceinline__ void turn_q(const Append8Args &a, int group, float2 *turns)
{
    const int at = div_by(a.q_shares, group), share = group - at * a.q_shares.d;
    const uint32_t t0 = (uint32_t)at * a.q_tokens;
    const int tokens = (int)min((uint32_t)a.q_tokens, (uint32_t)a.tokens - t0), per = min(a.q_share, (int)a.q_items.d - share * a.q_share);
    bool formed = false;
    for (int i = threadIdx.x;; i += kThreads) {
        const bool live = i < tokens * per;
        Raw16<S> raw;
        int sub = 0, head = 0, item = 0;
        Place p{};
        if (live) {
            sub = a.q_tokens == 1 ? 0 : i / per;
            const int in = share * a.q_share + i - sub * per;
            head = div_by(a.items, in);
            item = in - head * a.items.d;
            p = place_of<PAIRS>(a, item);
            raw.load(static_cast<const S *>(a.src[0]) + (int64_t)(t0 + sub) * a.src_stride[0] + head * a.dim, p.lo, p.hi);
        }
        if (!formed) {
            for (int e = threadIdx.x; e < tokens * a.half; e += kThreads) {
                const int k = a.q_tokens == 1 ? 0 : e / a.half;
                turns[e] = turn_at(a, t0 + k, e - k * a.half);
            }
            __syncthreads();
            formed = true;
        }
        if (!live)
            return;
        float x[16];
        raw.widen(x);
        float2 turn[8];
        if (8 * item < a.half) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                turn[e] = turns[sub * a.half + min(8 * item + e, a.half - 1)];
            turn16<PAIRS>(a, item, turn, x);
        }
        store16(a, static_cast<uint16_t *>(a.q_out) + ((int64_t)(t0 + sub) * a.q_heads + head) * a.dim, p, x);
    }
}

// A barrier for what lies in LDS: __syncthreads would wait for every store to memory on
// its way, some us a head.
__device__ __forceinline__ void meet()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

__device__ __forceinline__ uint32_t largest_of(const float *x, uint32_t top)
{
#pragma unroll
    for (int e = 0; e < 16; ++e)
        top = max(top, __builtin_bit_cast(uint32_t, x[e]) & 0x7fffffffu);
    return top;
}

__device__ __forceinline__ void put16(const Append8Args &a, uint8_t *out, Place p, const float *x, float inv)
{
    *reinterpret_cast<u32x2 *>(out + p.lo) = u32x2{codes4(a.e4m3, x, inv), codes4(a.e4m3, x + 4, inv)};
    *reinterpret_cast<u32x2 *>(out + p.hi) = u32x2{codes4(a.e4m3, x + 8, inv), codes4(a.e4m3, x + 12, inv)};
}

// One token: a wave takes as many rows as it has lanes for.  items is a power of two.
template <class S, bool PAIRS>
__device__ __forceinline__ void write_token(const Append8Args &a, const Run &r, int row, int end, int item)
{
    const bool live = row < end;
    const int v = live && row >= a.heads, head = v ? row - a.heads : row;
    const Place p = v ? Place{16 * item, 16 * item + 8} : place_of<PAIRS>(a, item);
    Raw16<S> raw;
    Target to{};
    int old = 0;
    float2 turn[8];
    if (live) {
        raw.load(static_cast<const S *>(v ? a.src[2] : a.src[1]) + (int64_t)r.first * (v ? a.src_stride[2] : a.src_stride[1]) + head * a.dim,
                 p.lo, p.hi);
        to = target_of(a, r.block, v, head);
        if (!r.begun)
            old = *to.scale;
    }
    turns_of(a, r.first, item, turn);
    float x[16];
    uint32_t top = 0;
    if (live) {
        raw.widen(x);
        if (!v)
            turn16<PAIRS>(a, item, turn, x);
        top = largest_of(x, 0);
    }
    for (int d = 1; d < (int)a.items.d; d *= 2)
        top = max(top, (uint32_t)__shfl_xor((int)top, d));
    if (!live)
        return;
    const int b = r.begun ? byte_of(a.e4m3, top) : max(byte_of(a.e4m3, top), old);
    if (!r.begun && b > old && b < 255)
        rescale(a, [&](int p) { return has_place(a, r, p); }, to, old, b, item, a.items.d);
    if (item == 0)
        *to.scale = (uint8_t)b;
    put16(a, to.codes + (r.slot - r.block * (int)a.block.d) * to.place, p, x, inverse_of(b));
}

// The wide path: 16-byte vectors of whole rows.  PP: tokens that a lane holds values of, so
// that four waves hold a whole block's.  A run of more tokens than that (two of one slot
// are in it) is taken in parts.
template <class S, bool PAIRS, int PP>
__global__ __launch_bounds__(kThreads) void paged8_append_kernel(Append8Args a)
{
    extern __shared__ float2 turns[];
    const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    if (group_here() >= a.groups)
        return;
    if (group_here() >= a.kv_groups) {
        turn_q<S, PAIRS>(a, group_here() - a.kv_groups, turns);
        return;
    }
    const int sub = div_by(a.items, lane), item = lane - sub * a.items.d;
    const int per = kWave / (int)a.items.d; // tokens of a wave at a time
    const Place kq = place_of<PAIRS>(a, item), plain{16 * item, 16 * item + 8};
    __shared__ uint32_t largest[2][kWaves];
    int turned = 0; // which half of `largest`
    int dealt = 0; // rows, or pieces of single tokens' rows, given out so far
    each_run(a, group_here(), [&](const Run &r, int share) {
        const int row0 = share * a.kv_share, end = min(row0 + a.kv_share, 2 * a.heads);
        if (r.n == 1 && (a.items.d & (a.items.d - 1)) == 0) {
            const int pieces = (end - row0 + per - 1) / per;
            for (int i = (wave - dealt) & (kWaves - 1); i < pieces; i += kWaves)
                write_token<S, PAIRS>(a, r, row0 + i * per + sub, end, item);
            dealt += pieces;
            return;
        }
        const int most = kWaves * PP * per;
        for (int left = r.n; left > 0; left -= most) {
            const int from = r.first + (r.n - left), n = min(left, most);
            // waves that hold a head together, a team; their teams take heads in turn
            const int waves = n <= PP * per ? 1 : n <= 2 * PP * per ? 2 : kWaves, teams = kWaves / waves;
            const int team = wave / waves, me = wave & (waves - 1);
            const bool begun = r.begun && from == r.first;
            const Run part{from, n, r.block, r.slot, begun, r.straight && n == r.n};
            uint32_t t[PP];
            int place[PP];
            bool live[PP];
#pragma unroll
            for (int i = 0; i < PP; ++i) {
                const int off = (i * waves + me) * per + sub;
                t[i] = (uint32_t)from + off;
                live[i] = sub < per && off < n;
                place[i] = live[i] ? a.slots[t[i]] - r.block * (int)a.block.d : 0;
            }
            float2 turn[PP][8];
            Raw16<S> raw[PP];
            const auto load = [&](int row) {
                const int v = row >= a.heads, head = v ? row - a.heads : row;
                const Place p = v ? plain : kq;
                const S *src = static_cast<const S *>(v ? a.src[2] : a.src[1]) + head * a.dim;
                const int64_t stride = v ? a.src_stride[2] : a.src_stride[1];
#pragma unroll
                for (int i = 0; i < PP; ++i)
                    if (live[i])
                        raw[i].load(src + (int64_t)t[i] * stride, p.lo, p.hi);
            };
            int row = row0 + ((team - dealt) & (teams - 1));
            dealt += end - row0;
            if (row < end)
                load(row);
#pragma unroll
            for (int i = 0; i < PP; ++i)
                if (row < a.heads && live[i]) // a first row of v: so are the others
                    turns_of(a, t[i], item, turn[i]);
            // teams of several waves go through as many rounds each: they meet in every one
            for (int rounds = (end - row0 + teams - 1) / teams; waves == 1 ? row < end : rounds > 0; row += teams, --rounds) {
                const bool on = row < end;
                const int v = row >= a.heads, head = v ? row - a.heads : row;
                const Place p = v ? plain : kq;
                const Target to = target_of(a, r.block, v, on ? head : 0);
                int old = 0;
                if (!begun)
                    old = *to.scale;
                float x[PP][16];
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < PP; ++i)
                    if (live[i]) {
                        raw[i].widen(x[i]);
                        if (!v)
                            turn16<PAIRS>(a, item, turn[i], x[i]);
                        top = largest_of(x[i], top);
                    }
                if (row + teams < end)
                    load(row + teams); // on its way while this one is written
                top = wave_max(top);
                if (waves > 1) {
                    if (lane == 0)
                        largest[turned][wave] = top;
                    asm volatile("" ::"v"(old)); // read by all before one of them writes the new one
                    meet();
                    for (int w = 0; w < waves; ++w)
                        top = max(top, largest[turned][team * waves + w]);
                    turned ^= 1; // the next head's go where none reads any more
                    if (!on)
                        continue;
                }
                const int b = begun ? byte_of(a.e4m3, top) : max(byte_of(a.e4m3, top), old);
                if (!begun && b > old && b < 255)
                    rescale(a, [&](int p) { return has_place(a, part, p); }, to, old, b, me * kWave + lane, waves * kWave);
                const float inv = inverse_of(b);
                if (me == 0 && lane == 0)
                    *to.scale = (uint8_t)b;
#pragma unroll
                for (int i = 0; i < PP; ++i)
                    if (live[i])
                        put16(a, to.codes + place[i] * to.place, p, x[i], inv);
            }
            if (left > most)
                __syncthreads(); // the further part's reads of this one's writes
        }
    });
}

// Any alignment, any even rot, any block: a thread takes one value at a time, twice, and
// forms its angle each time.  The 8192 tokens take 223 us off 16-byte alignment; in blocks
// larger than four waves hold one workgroup takes a run's rows one after the other: blocks
// of 256 at 128 wide 2.4 ms, of 128 at 256 wide (16 + 2 x 4 heads) 1.9 ms, against 65 us in
// blocks of 128 and 82 us in blocks of 64.
template <class S> __global__ __launch_bounds__(kThreads) void paged8_append_generic_kernel(Append8Args a)
{
    const auto value = [&](int which, int t, int head, int e) {
        const S *row = static_cast<const S *>(a.src[which]) + (int64_t)t * a.src_stride[which] + head * a.dim;
        if (which == 2 || e >= 2 * a.half)
            return (float)row[e];
        const int pair = a.pairs ? e / 2 : e < a.half ? e : e - a.half;
        const int lo = a.pairs ? 2 * pair : pair, hi = a.pairs ? lo + 1 : lo + a.half;
        float x = (float)row[lo], y = (float)row[hi];
        turn_pair(x, y, turn_at(a, t, pair));
        return e == lo ? x : y;
    };
    if (group_here() >= a.groups)
        return;
    if (group_here() >= a.kv_groups) { // q: a workgroup for a share of a token's values
        const int group = group_here() - a.kv_groups, t = div_by(a.q_shares, group), share = group - t * a.q_shares.d;
        const int e0 = share * a.q_share * 16, e1 = min(e0 + a.q_share * 16, a.q_heads * a.dim);
        uint16_t *out = static_cast<uint16_t *>(a.q_out) + (int64_t)t * a.q_heads * a.dim;
        for (int i = e0 + threadIdx.x; i < e1; i += kThreads) {
            const int h = i / a.dim;
            const float x = value(0, t, h, i - h * a.dim);
            out[i] = (uint16_t)(a.bf ? pack2<true>(x, 0.0f) : pack2<false>(x, 0.0f));
        }
        return;
    }
    __shared__ uint32_t largest[kWaves];
    __shared__ uint32_t taken[GEMV_PAGED_MAX_PAGE / 32]; // a bit for each place: a block may have too many to look for
    each_run(a, group_here(), [&](Run r, int share) {
        if (!r.straight) {
            for (int i = threadIdx.x; i < ((int)a.block.d + 31) / 32; i += kThreads)
                taken[i] = 0;
            __syncthreads();
            for (int i = threadIdx.x; i < r.n; i += kThreads) {
                const int p = a.slots[r.first + i] - r.block * (int)a.block.d;
                atomicOr(&taken[p / 32], 1u << (p % 32));
            }
            __syncthreads();
        }
        const auto has = [&](int p) { return r.straight ? has_place(a, r, p) : (taken[p / 32] >> (p % 32) & 1) != 0; };
        const int last = min((share + 1) * a.kv_share, 2 * a.heads);
        for (int row = share * a.kv_share; row < last; ++row) {
            const int v = row >= a.heads, head = v ? row - a.heads : row;
            const Target to = target_of(a, r.block, v, head);
            const int old = *to.scale;
            uint32_t top = 0;
            for (int64_t i = threadIdx.x; i < (int64_t)r.n * a.dim; i += kThreads) {
                const int at = (int)(i / a.dim);
                top = max(top, __builtin_bit_cast(uint32_t, value(1 + v, r.first + at, head, (int)(i - (int64_t)at * a.dim))) & 0x7fffffffu);
            }
            top = wave_max(top);
            if ((threadIdx.x & (kWave - 1)) == 0)
                largest[threadIdx.x / kWave] = top;
            __syncthreads(); // and the scale is read by all
            for (int w = 0; w < kWaves; ++w)
                top = max(top, largest[w]);
            const int b = r.begun ? byte_of(a.e4m3, top) : max(byte_of(a.e4m3, top), old);
            if (!r.begun && b > old && b < 255)
                rescale(a, has, to, old, b, threadIdx.x, kThreads);
            const float inv = inverse_of(b);
            if (threadIdx.x == 0)
                *to.scale = (uint8_t)b;
            for (int64_t i = threadIdx.x; i < (int64_t)r.n * a.dim; i += kThreads) {
                const int at = (int)(i / a.dim), e = (int)(i - (int64_t)at * a.dim);
                const float x[4] = {value(1 + v, r.first + at, head, e), 0.0f, 0.0f, 0.0f};
                to.codes[(a.slots[r.first + at] - r.block * (int)a.block.d) * to.place + e] = (uint8_t)codes4(a.e4m3, x, inv);
            }
            __syncthreads(); // `largest` is free, and what this run wrote is there for the next
        }
    });
}

// passes: tokens that a lane of one wave would hold of a whole block, 0 for what the wide path does not take.
template <class S, bool PAIRS> const void *kernel_of(int passes)
{
    return passes <= 4   ? reinterpret_cast<const void *>(&paged8_append_kernel<S, PAIRS, 1>)
           : passes <= 8 ? reinterpret_cast<const void *>(&paged8_append_kernel<S, PAIRS, 2>)
                         : reinterpret_cast<const void *>(&paged8_append_kernel<S, PAIRS, 4>);
}

template <class S> const void *kernel_of(bool pairs, int passes)
{
    return passes == 0 ? reinterpret_cast<const void *>(&paged8_append_generic_kernel<S>)
           : pairs     ? kernel_of<S, true>(passes)
                       : kernel_of<S, false>(passes);
}

} // namespace
} // namespace gemv

extern "C" int gemv_paged8_append(const void *q, const void *k, const void *v, int src_type, int64_t tokens,
                                  int64_t q_heads, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                  const int32_t *positions, int64_t axes, const int32_t *axis, const float *inv_freq,
                                  int64_t rot, int style, const int32_t *slots, void *q_out, int q_out_type,
                                  const gemv_kv_cache8 *cache, void *hip_stream)
{
    const int st = gemv::validate_append8(q, k, v, src_type, tokens, q_heads, q_stride, k_stride, v_stride, positions,
                                          axes, axis, inv_freq, rot, style, slots, q_out, q_out_type, cache);
    if (st != GEMV_OK)
        return st;
    if (tokens == 0)
        return gemv::finish_launch((int)hipSuccess);
    gemv::Append8Args a{};
    a.src[0] = q, a.src[1] = k, a.src[2] = v;
    a.src_stride[0] = q_stride, a.src_stride[1] = k_stride, a.src_stride[2] = v_stride;
    a.positions = positions, a.axis = axis, a.slots = slots, a.inv_freq = inv_freq, a.q_out = q_out;
    a.codes[0] = static_cast<uint8_t *>(cache->k), a.codes[1] = static_cast<uint8_t *>(cache->v);
    a.scales[0] = cache->k_scale, a.scales[1] = cache->v_scale;
    for (int d = 0; d < 3; ++d) {
        a.c_stride[0][d] = cache->k_stride[d], a.c_stride[1][d] = cache->v_stride[d];
        a.s_stride[0][d] = cache->ks_stride[d], a.s_stride[1][d] = cache->vs_stride[d];
    }
    a.tokens = (int)tokens, a.axes = (int)axes, a.q_heads = (int)q_heads, a.heads = cache->heads, a.dim = cache->dim;
    a.half = (int)(rot / 2), a.pairs = style == GEMV_ROPE_PAIRS;
    a.num_slots = (int)(cache->num_pages * cache->page_size);
    a.e4m3 = cache->code == GEMV_KV_E4M3, a.bf = q_out_type == GEMV_W_BF16;
    a.page = gemv::fast_div(cache->page_size), a.block = gemv::fast_div(cache->block);

    // wide: 16-byte vectors of whole rows.  The cache and q_out always allow them
    // (checked strides and alignment); the rows of q, k and v and rot may not.
    const int64_t size = src_type == GEMV_W_F32 ? 4 : 2;
    bool wide = rot % (a.pairs ? 8 : 16) == 0;
    for (int i = 0; i < 3; ++i)
        wide = wide && reinterpret_cast<uintptr_t>(a.src[i]) % 16 == 0 && a.src_stride[i] * size % 16 == 0;
    const int items = cache->dim / 16, per = gemv::kWave / items; // lanes of a token's head, tokens of a wave at a time
    a.items = gemv::fast_div(items);
    int64_t passes = (cache->block + per - 1) / per; // tokens that a lane of one wave would hold of a whole block
    if (!wide || passes > 16)
        passes = 0;

    // Some thousand workgroups for k and v, each for four rows (one a wave) of a stretch of
    // tokens: of a chunk few begin a run, and more rows would be taken one after the other
    // (8192 tokens, blocks of 64: 33 us with 4 rows, 40 with 8; 512 tokens 10 and 15).  Where
    // the tokens are many and a wave or two hold a block's, eight: fewer workgroups form the
    // same angles, and single tokens' rows fill a wave (8192 tokens in blocks of 16 40 us,
    // 44 with 4 rows; 4096 single tokens 25 and 34; 1024 tokens of one chunk 18 and 14).
    const int64_t rows = 2 * (int64_t)a.heads;
    int64_t kv_share = tokens >= 1024 && passes <= 2 ? 8 : 4;
    int64_t stretch = tokens * ((rows + kv_share - 1) / kv_share) / 1024;
    stretch = stretch < 1 ? 1 : stretch < 32 ? stretch : 32;
    const int64_t per_die = ((tokens + stretch - 1) / stretch + 7) / 8, stretches = 8 * per_die;
    a.die_stretches = (int)per_die;
    int64_t kv_shares = (rows + kv_share - 1) / kv_share;
    while (stretches * kv_shares > gemv::kMostGroups && kv_share < rows) {
        kv_share *= 2;
        kv_shares = (rows + kv_share - 1) / kv_share;
    }
    a.stretch = (int)stretch, a.kv_share = (int)kv_share;
    const int64_t kv_groups = stretches * kv_shares;
    // q: an item a thread; of heads so few that a token has fewer items, several tokens
    const int64_t q_items = q_heads * items;
    int64_t q_tokens = passes ? gemv::kThreads / q_items : 1;
    const int64_t room = 1024 / (a.half > 0 ? a.half : 1); // turns that lie in LDS
    q_tokens = q_tokens < room ? q_tokens : room;
    q_tokens = q_tokens < 1 ? 1 : q_tokens;
    const int64_t q_groups = (tokens + q_tokens - 1) / q_tokens;
    int64_t q_share = tokens < 512 ? gemv::kThreads : 4 * gemv::kThreads;
    q_share = q_share < q_items ? q_share : q_items;
    while (q_groups * ((q_items + q_share - 1) / q_share) > gemv::kMostGroups && q_share < q_items)
        q_share *= 2;
    // below 2^31: of at most 2^30 tokens up to 2^30 for q (one a token), and 2^29 for k and v
    const int64_t q_shares = (q_items + q_share - 1) / q_share, groups = kv_groups + q_groups * q_shares;
    a.q_share = (int)q_share, a.q_tokens = (int)q_tokens, a.q_items = gemv::fast_div(q_items);
    a.q_shares = gemv::fast_div(q_shares), a.kv_shares = gemv::fast_div(kv_shares);
    a.kv_groups = (int)kv_groups, a.groups = (int)groups;
    const void *fn = src_type == GEMV_W_F32   ? gemv::kernel_of<float>(a.pairs, (int)passes)
                     : src_type == GEMV_W_F16 ? gemv::kernel_of<_Float16>(a.pairs, (int)passes)
                                              : gemv::kernel_of<__bf16>(a.pairs, (int)passes);
    void *args[] = {&a};
    const int64_t x = groups < gemv::kGroupsX ? groups : gemv::kGroupsX;
    const hipError_t e = hipLaunchKernel(fn, dim3((unsigned)x, (unsigned)((groups + x - 1) / x)), dim3(gemv::kThreads), args,
                                         (size_t)q_tokens * a.half * sizeof(float2), static_cast<hipStream_t>(hip_stream));
    return gemv::finish_launch((int)e);
}
