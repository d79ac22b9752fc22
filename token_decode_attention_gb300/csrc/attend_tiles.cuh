// attend_tiles.cuh -- how the key tiles of all items are shared by the CTAs of
// attend_tiles_kernel.cuh, for it and for the kernels that merge what it leaves.
//
// The items of a key/value head, one head after the other, are laid end to end in units of
// key tiles; an item adds kItemExtra units ahead of its tiles, about what beginning it costs.
// The whole is cut into equal ranges, one per CTA, whatever the mix of long and short
// items.  The part of an item that a CTA holds is a piece of it.  A CTA has at
// most one piece of an item that an earlier CTA began (slot 2c) and one that it began and
// a later CTA goes on with (slot 2c + 1).
#pragma once

#include "attend_rows.cuh"
#include "streamk.h"

namespace dattn {
namespace attend {

constexpr int kItemExtra = 1;

__device__ __forceinline__ int key_tiles(int n, int keys) { return max(1, (n + keys - 1) / keys); }

struct Shares {
    long long total;  // units of a key/value head
    long long all;    // of all of them
    int items, ctas;
    int uniform;      // shared positions: units of every item, or 0
};

__device__ __forceinline__ Shares shares_of(const AttendArgs &a, const TileArgs &t, int dp) {
    Shares s;
    if (t.plan != nullptr) {
        s.total = t.plan->total;
        s.items = t.plan->items;
        s.ctas = t.plan->ctas;
        s.uniform = 0;
    } else {
        s.uniform = key_tiles(a.shared, tile_keys(dp)) + kItemExtra;
        s.items = static_cast<int>((static_cast<long long>(a.B) * a.group + tile_rows(dp) - 1) / tile_rows(dp));
        s.total = static_cast<long long>(s.items) * s.uniform;
        s.ctas = t.ctas;
    }
    s.all = s.total * a.Hk;
    return s;
}

__device__ __forceinline__ long long units_before(const TileArgs &t, const Shares &s, int item) {
    return s.uniform ? static_cast<long long>(item) * s.uniform : t.before[item];
}

// The item that holds unit x of a key/value head, found by a whole warp: 32 items are
// looked at in a round, so that a round trip to memory leaves a 32nd of them.
__device__ __forceinline__ int item_at(const TileArgs &t, const Shares &s, long long x) {
    if (s.uniform) return static_cast<int>(x / s.uniform);
    const int lane = threadIdx.x & 31;
    int lo = 0, n = s.items;
    while (n > 1) {
        const int step = (n + 31) / 32, i = lo + lane * step;
        const unsigned below = __ballot_sync(0xffffffffu, lane * step < n && t.before[i] <= x);
        const int last = 31 - __clz(below);  // lane 0's begins at or before x
        lo += last * step;
        n = min(step, n - last * step);
    }
    return lo;
}

__device__ __forceinline__ TileItem item_of(const AttendArgs &a, const TileArgs &t, const Shares &s, int rows,
                                            int item) {
    if (!s.uniform) {
        const int4 *at = reinterpret_cast<const int4 *>(t.items + item);
        const int4 x = at[0], y = at[1];
        return TileItem{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    }
    const int row = item * rows, token = fast_div(row, t.div_group);
    return TileItem{0, token, row - token * a.group, min(rows, a.B * a.group - row), 0, 0, 0, a.shared};
}

// A CTA's walk over its pieces: tiles [j0, j1) of `item`, key/value head kvh.
struct Walk {
    long long x, x1;
    long long at, end;  // units of the item, of its key/value head
    int kvh, item;
    int j0, j1;
    bool begins, ends;

    __device__ __forceinline__ void start(const TileArgs &t, const Shares &s, int cta) {
        x = range_begin(cta, s.all, s.ctas);
        x1 = range_begin(cta + 1, s.all, s.ctas);
        if (x >= x1) return;
        kvh = static_cast<int>(x / s.total);
        item = item_at(t, s, x - kvh * s.total);
        at = units_before(t, s, item);
        end = units_before(t, s, item + 1);
    }
    __device__ __forceinline__ bool next(const TileArgs &t, const Shares &s) {
        while (x < x1) {
            const long long rel = x - kvh * s.total;
            if (rel >= end) {
                if (++item == s.items) {
                    item = 0;
                    ++kvh;
                }
                at = item == 0 ? 0 : end;
                end = units_before(t, s, item + 1);
                continue;
            }
            const long long from = rel - at, take = min(x1 - x, end - rel);
            x += take;
            j0 = max(0, static_cast<int>(from) - kItemExtra);
            j1 = static_cast<int>(from + take) - kItemExtra;
            if (j1 <= j0) continue;  // none of the item's own tiles
            begins = j0 == 0;
            ends = from + take == end - at;
            return true;
        }
        return false;
    }
};

// The CTAs that hold tiles of an item at units [at, end) of key/value head kvh.
__device__ __forceinline__ int2 holders(const Shares &s, int kvh, long long at, long long end) {
    const long long base = kvh * s.total;
    return make_int2(static_cast<int>(range_owner(base + at + kItemExtra, s.all, s.ctas)),
                     static_cast<int>(range_owner(base + end - 1, s.all, s.ctas)));
}

}  // namespace attend
}  // namespace dattn
