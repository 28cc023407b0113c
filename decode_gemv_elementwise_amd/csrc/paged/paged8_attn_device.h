// What the two kernels of gemv_paged8_attn share beyond paged_attn_device.h:
// arguments, where a key and its scale lie, and the plan.
//
// Mathematics and plan are those of gemv_paged_attn (one pass over the keys with the
// running maximum and sum; the blocks of all row tiles in one line that the
// workgroups share equally), over values that a code and a scale stand for.  Here the
// two kinds of row tile are kernels of their own, and the host chooses by the mean
// count of rows: together in one kernel they leave each other too few registers for
// the codes on their way.
#pragma once

#include "paged8_device.h"
#include "paged_attn_device.h"

namespace gemv {
namespace {

constexpr uint32_t kMostCost = INT_MAX;
constexpr int kCostBlock = 32; // keys of a block, as the plan counts
constexpr uint32_t kSpreadFrom = 64; // such blocks of a workgroup, from which on tiles are of several heads

struct Attn8Args : AttnArgs { // k and v are bytes
    const uint8_t *k_scale, *v_scale;
    uint32_t ks_stride[3], vs_stride[3]; // page, block in page, head; below 2^31
    FastDiv block;
    int32_t spread; // a tile of few rows may be of 2^spread heads, a divisor of all: 1, 2 or 4
};

// The kernel's arguments, read again from here on.
__device__ __forceinline__ const Attn8Args &arguments()
{
    auto p = (const __attribute__((address_space(4))) Attn8Args *)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *(const Attn8Args *)p;
}

// What finds a key of one head and its scale in the cache.
struct Paging8 {
    FastDiv page, block;
    uint32_t width, pages, k0, k1, v0, v1, ks0, ks1, vs0, vs1;
    const uint8_t *k, *v, *k_scale, *v_scale; // of the key/value head
    const int32_t *table;                     // of the request

    __device__ __forceinline__ void begin(const Attn8Args &a, int r, int head)
    {
        page = FastDiv{kept(a.page.mul), kept(a.page.shift), kept(a.page.d)};
        block = FastDiv{kept(a.block.mul), kept(a.block.shift), kept(a.block.d)};
        width = kept((uint32_t)a.width), pages = kept((uint32_t)a.num_pages);
        k0 = kept(a.k_stride[0]), k1 = kept(a.k_stride[1]), v0 = kept(a.v_stride[0]), v1 = kept(a.v_stride[1]);
        ks0 = kept(a.ks_stride[0]), ks1 = kept(a.ks_stride[1]), vs0 = kept(a.vs_stride[0]), vs1 = kept(a.vs_stride[1]);
        k = reinterpret_cast<const uint8_t *>(a.k) + (int64_t)head * a.k_stride[2];
        v = reinterpret_cast<const uint8_t *>(a.v) + (int64_t)head * a.v_stride[2];
        k_scale = a.k_scale + (int64_t)head * a.ks_stride[2];
        v_scale = a.v_scale + (int64_t)head * a.vs_stride[2];
        table = a.table + r * a.table_stride;
    }
    // The page id of key j as the table has it, -1 past the table's end.
    __device__ __forceinline__ int raw(int j) const
    {
        const uint32_t at = div_by(page, j);
        return at < width ? table[at] : -1;
    }
    // -1 for what is no page.
    __device__ __forceinline__ int checked(int id) const { return (uint32_t)id < pages ? id : -1; }
    // Key j's codes in page id, and its scale's byte (a key without a page reads page
    // 0, and what is read is dropped).
    template <bool V> __device__ __forceinline__ const uint8_t *codes(int id, int j) const
    {
        const uint32_t in = j - div_by(page, j) * page.d;
        return (V ? v : k) + ((uint64_t)(uint32_t)max(id, 0) * (V ? v0 : k0) + (uint64_t)in * (V ? v1 : k1));
    }
    template <bool V> __device__ __forceinline__ const uint8_t *scale(int id, int j) const
    {
        const uint32_t in = j - div_by(page, j) * page.d;
        return (V ? v_scale : k_scale) +
               ((uint64_t)(uint32_t)max(id, 0) * (V ? vs0 : ks0) + (uint64_t)div_by(block, in) * (V ? vs1 : ks1));
    }
};

// The plan, for row tiles of ROWS rows: TILE::run does one share of a tile's keys.
// The blocks of 32 keys of all tiles form one line (request, head, tile, block), from
// a prefix sum over the requests, and workgroup w takes the w-th equal share of it,
// whatever tiles that cuts; an end of a share within TILE::kEdge of a tile's edge moves
// there.  A tile counts a.tile_cost on top for starting on it.  A tile whose keys are cut
// leaves its parts in the workspace, and the workgroup that counts the last of them
// joins them in order, so the result does not depend on which came last.
template <class TILE> __device__ __forceinline__ void run_plan(char *lds)
{
    const Attn8Args &a = arguments();
    __shared__ uint32_t before[kThreads], scratch[kWaves];
    __shared__ Request requests[kThreads];
    const auto sum = [](uint32_t x, uint32_t y) { return min(x + y, kMostCost); };
    const auto tiles_of = [&](const Request &q) { // rows are below 2^31, as all rows together
        return ((uint32_t)q.n * a.group + TILE::kRows - 1) / TILE::kRows;
    };
    // the blocks of 32 keys that one tile visits at most, in units of 2^unit_log2 blocks
    const auto cost_of = [&](const Request &q) {
        uint32_t keys = (uint32_t)min((int64_t)q.kv, a.reach);
        if (a.window != 0) {
            const uint32_t some = (uint32_t)a.window + min(q.n, TILE::kRows) + 4 * kCostBlock; // below 2^32
            keys = min(keys, min((uint32_t)a.sinks, keys) + min(some, keys));
        }
        return ((keys + kCostBlock - 1) / kCostBlock >> a.unit_log2) + a.tile_cost;
    };
    const auto costs = [&](const Request &q) {
        return (uint32_t)min((uint64_t)tiles_of(q) * a.heads * cost_of(q), (uint64_t)kMostCost);
    };
    const bool once = a.requests <= kThreads;
    uint32_t total = 0;
    if (!once) {
        uint32_t cost = 0;
        for (int r = threadIdx.x; r < a.requests; r += kThreads)
            cost = sum(cost, costs(request_of(a, r)));
        block_prefix<kWaves>(threadIdx.x, cost, scratch, &total, sum);
        total = uniform(total);
        __syncthreads();
    }

    int spread = 0, stride = TILE::kPart; // floats from one part's place to the next
    // this workgroup's share [x, x1): every group has `each` places, the first `more` one in addition
    uint32_t base = 0, x = 0, x1 = 0, each = 0, more = 0, edge = 0;
    // Neighbouring shares go to one of the 8 dies, which share an L2 cache; and where a
    // compute unit holds two workgroups the second half of a die's shares goes backwards:
    // later tiles of a chunk see more keys, so a unit gets a long and a short one.
    uint32_t w = blockIdx.x;
    if (gridDim.x % 16 == 0 && gridDim.x >= (uint32_t)kAttnGroups) {
        const uint32_t per = gridDim.x / 8, i = w / 8;
        w = w % 8 * per + (i < per / 2 ? i : per + per / 2 - 1 - i);
    }
    for (int r0 = 0; r0 < a.requests; r0 += kThreads) {
        const int thread = thread_here(), r = r0 + thread;
        Request q{0, 0, 0};
        if (r < a.requests)
            q = request_of(a, r);
        uint32_t here;
        before[thread] = block_prefix<kWaves>(thread, costs(q), scratch, &here, sum);
        requests[thread] = q;
        here = uniform(here);
        __syncthreads();
        if (r0 == 0) {
            if (once)
                total = here;
            if (total == kMostCost)
                return;
            if (total >= gridDim.x * kSpreadFrom) {
                spread = a.spread;
                stride <<= spread;
                total >>= spread; // nothing is lost: every tile was counted once for each head
            }
            const uint32_t groups = uniform(min(gridDim.x, (total + TILE::kLeast - 1) / TILE::kLeast));
            if (w >= groups)
                return;
            each = uniform(total / groups);
            more = total - each * groups;
            x = w * each + min(w, more);
            x1 = x + each + (w < more);
            // a tile is cut only if the parts have room: two for each workgroup, below 2^28 floats in all
            edge = a.part_room < 2 * (int64_t)groups * stride ? kMostCost / 2 : TILE::kEdge;
        }
        here >>= spread;
        while (x < x1 && x < base + here) {
            int lo = 0, hi = min(kThreads, a.requests - r0);
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (before[mid] >> spread <= x - base)
                    lo = mid;
                else
                    hi = mid;
            }
            lo = uniform(lo);
            const Request q = {(int)uniform(requests[lo].q0), (int)uniform(requests[lo].n), (int)uniform(requests[lo].kv)};
            const uint32_t y = x - base - (uniform(before[lo]) >> spread), nb = uniform(cost_of(q)), tiles = uniform(tiles_of(q));
            const uint32_t unit = uniform(y / nb), start = x - (y - unit * nb); // of the tile
            // both ends of the share, as places of this tile; one near an edge of it moves there
            const auto moved = [&](uint32_t b) {
                return b >= nb ? nb : b < edge && b <= nb - b ? 0 : nb - b < edge && nb - b < b ? nb : b;
            };
            const uint32_t b0 = moved(x - start), b1 = moved(x1 - start);
            x = start + nb;
            if (b0 >= b1)
                continue;
            Share sh{(int)b0, (int)(b1 - b0), (int)nb, 1, 0, 0, stride};
            if (sh.len < (int)nb) {
                const auto group_of = [&](uint32_t place) {
                    const uint32_t longer = more * (each + 1);
                    return uniform(place < longer ? place / (each + 1) : more + (place - longer) / each);
                };
                sh.first = group_of(start + edge - 1);
                sh.np = group_of(start + nb - edge) - sh.first + 1;
                sh.me = w - sh.first;
            }
            const int head = uniform(unit / tiles), tile = unit - head * tiles;
            TILE::run(arguments(), q, r0 + lo, tile, head << spread, 1 << spread, sh, lds);
        }
        if (x >= x1)
            return;
        base += here;
        __syncthreads();
    }
}

} // namespace
} // namespace gemv
