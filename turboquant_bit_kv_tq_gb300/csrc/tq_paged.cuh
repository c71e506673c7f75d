// Work units and workspace of decode attention over the 8-bit and 4-bit caches.
#pragma once

#include "tq_device.cuh"

namespace tq {

// Decode grids: kPagedWarps warps per block, at most kPagedCtas blocks per SM and
// kPagedMaxSms SMs; the workspace holds two partial sums for each block.
constexpr int kPagedWarps = 4, kPagedCtas = 3, kPagedMaxSms = 160;
constexpr int kPagedSlots = 2 * kPagedCtas * kPagedMaxSms;
// Places a unit takes beside its pages where pages are dealt out, at most: its start
// and its sums take a block about as long as 8 (d = 128) to 16 (d = 256) pages.  With
// 0, 4, 8, 16, 24, 32: 8 x up to 32768 tokens, d = 256: 81, 73, 68, 60, 59, 58 us;
// 64 x up to 2000, d = 128: 56, 48, 37, 35, 34, 35 us.  At 4 bits, where a page takes less
// time: 16 x 8192, d = 128, with 0, 12, 24, 32, 48: 42.9, 42.3, 40.8, 39.8, 40.2 us.
__host__ __device__ constexpr int paged_unit_cost(int bits) { return bits == 8 ? 24 : 32; }

// Query heads of one KV head that one work unit serves (nhg units per KV head
// share its pages through L2 when G > 16), in n-tiles of 8 heads.
struct PagedGeom {
    int group, nhg, hp, nt;
};
template <class Config>
PagedGeom paged_geom(const Config& c) {
    PagedGeom g;
    g.group = c.num_q_heads / c.num_kv_heads;
    g.nhg = (g.group + 15) / 16;
    g.hp = (g.group + g.nhg - 1) / g.nhg;
    g.nt = g.hp > 8 ? 2 : 1;
    return g;
}

struct PagedWorkspace {
    // err: the error word; cnt: one counter per (sequence, KV head, head group);
    // gcnt: one per slot; part: [kPagedSlots][d/16][nt][32][4] fp32 sums in
    // fragment order; meta: [kPagedSlots][8 nt] {r, x, l, -}
    size_t err, cnt, gcnt, zeroed, part, meta, total;
};
template <class Config>
PagedWorkspace paged_workspace(const Config& c) {
    const PagedGeom g = paged_geom(c);
    PagedWorkspace w;
    w.err = 0;
    w.cnt = 16;
    w.gcnt = w.cnt + (size_t)c.max_batch * c.num_kv_heads * g.nhg * 4;
    w.zeroed = w.gcnt + (size_t)kPagedSlots * 4;
    size_t off = (w.zeroed + 255) & ~(size_t)255;
    w.part = off;
    off += (size_t)kPagedSlots * 8 * g.nt * c.head_dim * 4;
    w.meta = off;
    off += (size_t)kPagedSlots * 8 * g.nt * 16;
    w.total = off;
    return w;
}

}  // namespace tq
