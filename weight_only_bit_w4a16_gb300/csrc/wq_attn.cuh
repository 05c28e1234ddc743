// wq_attn.cuh -- attention over a shared prefix: the arguments and the plan
// that its kernels share.
//
// The work of a call is a line of blocks of BK keys.  A unit is one head of
// keys with ROWS of its query rows (row = query token * group + head of the
// group): first the prefix's units (all tokens' rows), then each sequence's
// own.  Where sequences have many rows each, a unit's blocks are the prefix's
// and then the sequence's own instead ("concat").  The line is cut into equal runs, one for each CTA, whatever the
// lengths are: a CTA computes a piece (softmax maximum, sum and weighted
// values) of each unit that its run touches, and the pieces of a row are
// joined by combine_kernel.  Piece number = run number + unit number, which
// grows along the line, so pieces need no table.
//
// Lengths are on the device, so every CTA makes the plan for itself: sums over
// the sequences, held in shared memory.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "wq_internal.h"
#include "wq_tc.cuh"

namespace wq {
namespace attn {

struct Args {
    wq_attention t;
    int group;        // query heads of a key head
    int prefix;       // the kernel's line has the prefix's units
    int own;          // ... the sequences' own
    int concat;       // each sequence's units take the prefix's blocks first (own, not prefix)
    int runs;         // CTAs
    int min_run;      // blocks of a run at least
    int box;          // rows of a TMA box: a power of two that divides the page size
    int stages;       // of the ring (tiles_kernel)
    int max_pieces;   // room in the workspace
    float scale_log2; // scale * log2 e
    float* part_o;    // (pieces, ROWS, DP): sums of weights * values
    float2* part_ml;  // (pieces, ROWS): maximum (in powers of 2) and sum of weights
    int* plan;        // see publish_plan
};

constexpr int kMaxSeq = 1024;
// shared memory of the plan's sums
__host__ __device__ constexpr size_t plan_smem(int sequences) { return ((size_t)sequences + 1) * 8 + 16; }

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

// a sequence's query tokens and keys, whatever the arrays hold
struct Seq {
    int t0, n, len;
};

__device__ __forceinline__ int seq_start(const wq_attention& t, int b) {
    return t.q_start ? clampi(t.q_start[b], 0, t.tokens) : b * (t.tokens / t.sequences);
}

__device__ __forceinline__ Seq seq_at(const wq_attention& t, int b) {
    Seq s;
    s.t0 = seq_start(t, b);
    const int t1 = seq_start(t, b + 1);
    s.n = t1 > s.t0 ? t1 - s.t0 : 0;
    s.len = clampi(t.seq_lens[b], 0, t.table_pages * t.cache.page_size);
    return s;
}

__device__ __forceinline__ int divide(int a, int b) { return (int)((unsigned)a / (unsigned)b); }
__host__ __device__ __forceinline__ int ceil_div(int a, int b) { return (int)(((unsigned)a + (unsigned)b - 1) / (unsigned)b); }

// keys that the row tile `rt` of a sequence can see: those of its last row
__device__ __forceinline__ int tile_keys(const Seq& s, int group, int rows, int rt) {
    const int query = group == 1 ? (rt + 1) * rows - 1 : divide((rt + 1) * rows - 1, group);
    const int q = query < s.n ? query : s.n - 1;
    const int keys = s.len - s.n + q + 1;
    return keys < 0 ? 0 : keys;
}

// blocks of that tile
template <int ROWS, int BK>
__device__ __forceinline__ int tile_blocks(const Args& a, const Seq& s, int rt) {
    return (a.concat ? ceil_div(a.t.prefix_len, BK) : 0) + ceil_div(tile_keys(s, a.group, ROWS, rt), BK);
}

// Sums over the sequences before b, for one key head: blocks and row tiles.
// (The launcher refuses calls whose line could pass 31 bits.)
struct Plan {
    int2* sums;          // sequences + 1, in shared memory: blocks, tiles
    int tokens;          // query tokens of all sequences
    int prefix_blocks;   // of one unit
    int prefix_tiles;
    int prefix_line;     // blocks of all prefix units
    int line;            // all blocks
    int run;             // blocks of a run
    int2 scratch[32];
};

// Made by all threads of the CTA (NT of them, a multiple of 32), its sums at
// `sums` (plan_smem bytes, 8-byte aligned); ends with a barrier.
template <int NT, int ROWS, int BK>
__device__ __forceinline__ void make_plan(Plan& p, const Args& a, void* sums) {
    const wq_attention& t = a.t;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int B = a.own ? t.sequences : 0;
    const int tokens = t.q_start ? clampi(t.q_start[t.sequences], 0, t.tokens) : t.tokens;
    int2* const sum = static_cast<int2*>(sums);
    // this thread's sequences
    const int per = (B + NT - 1) / NT, b0 = tid * per, b1 = b0 + per < B ? b0 + per : B;
    int2 mine = make_int2(0, 0);
    for (int b = b0; b < b1; ++b) {
        const Seq s = seq_at(t, b);
        const int rt = ceil_div(s.n * a.group, ROWS);
        int w = 0;
        for (int i = 0; i < rt; ++i) w += tile_blocks<ROWS, BK>(a, s, i);
        mine.x += w;
        mine.y += rt;
        sum[b + 1] = make_int2(w, rt);
    }
    // sums over the threads before this one
    int2 s = mine;
    if (B > 1) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int ux = __shfl_up_sync(0xffffffffu, s.x, o), uy = __shfl_up_sync(0xffffffffu, s.y, o);
            if (lane >= o) {
                s.x += ux;
                s.y += uy;
            }
        }
    }
    if (lane == (B > 1 ? 31 : 0)) p.scratch[warp] = s;
    __syncthreads();
    int2 all = make_int2(0, 0), before = make_int2(s.x - mine.x, s.y - mine.y);
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        const int2 v = p.scratch[w];
        if (w < warp) {
            before.x += v.x;
            before.y += v.y;
        }
        all.x += v.x;
        all.y += v.y;
    }
    for (int b = b0; b < b1; ++b) {
        const int2 v = sum[b + 1];
        before.x += v.x;
        before.y += v.y;
        sum[b + 1] = before;
    }
    if (tid == 0) {
        sum[0] = make_int2(0, 0);
        p.sums = sum;
        p.tokens = tokens;
        p.prefix_tiles = a.prefix ? ceil_div(tokens * a.group, ROWS) : 0;
        p.prefix_blocks = a.prefix ? ceil_div(t.prefix_len, BK) : 0;
        p.prefix_line = p.prefix_blocks * p.prefix_tiles * t.kv_heads;
        p.line = p.prefix_line + all.x * t.kv_heads;
        const int run = ceil_div(p.line, a.runs);
        p.run = run < a.min_run ? a.min_run : run;
    }
    __syncthreads();
}

// For combine_kernel: run length, prefix tiles, blocks and line, then the sums.
constexpr int kPlanHead = 4;
constexpr size_t kPlanBytes = sizeof(int) * (kPlanHead + 2 * (kMaxSeq + 1));

template <int NT>
__device__ __forceinline__ void publish_plan(const Plan& p, const Args& a) {
    const int B = a.own ? a.t.sequences : 0;
    if (threadIdx.x == 0)
        *reinterpret_cast<int4*>(a.plan) = make_int4(p.run, p.prefix_tiles, p.prefix_blocks, p.prefix_line);
    for (int b = threadIdx.x; b <= B; b += NT) *reinterpret_cast<int2*>(a.plan + kPlanHead + 2 * b) = p.sums[b];
}

// Where a block of the line lies.
struct Unit {
    int seq;            // sequence, -1: prefix
    int head, tile;     // key head, row tile
    int unit;           // number along the line
    int first;          // the unit's first block on the line
    int blocks;         // of the unit
    int t0, n, len;     // tokens and keys (prefix: all tokens, prefix_len)
};

template <int ROWS, int BK>
__device__ __forceinline__ Unit unit_of(const Plan& p, const Args& a, int x) {
    const wq_attention& t = a.t;
    Unit u;
    if (x < p.prefix_line) {
        u.seq = -1;
        u.unit = divide(x, p.prefix_blocks);
        u.head = p.prefix_tiles == 1 ? u.unit : divide(u.unit, p.prefix_tiles);
        u.tile = u.unit - u.head * p.prefix_tiles;
        u.first = u.unit * p.prefix_blocks;
        u.blocks = p.prefix_blocks;
        u.t0 = 0;
        u.n = p.tokens;
        u.len = t.prefix_len;
        return u;
    }
    const int y = x - p.prefix_line;
    // the last sequence whose blocks begin at or before y
    int lo = 0, hi = t.sequences - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.sums[mid].x * t.kv_heads <= y) lo = mid;
        else hi = mid - 1;
    }
    const Seq s = seq_at(t, lo);
    const int2 c0 = p.sums[lo], c1 = p.sums[lo + 1];
    const int w = c1.x - c0.x, z = y - c0.x * t.kv_heads, tiles = c1.y - c0.y;
    u.seq = lo;
    u.head = divide(z, w);
    int r = z - u.head * w, first = x - r, tile = 0, n = 0;
    for (;; ++tile) {
        n = tile_blocks<ROWS, BK>(a, s, tile);
        if (r < n || tile + 1 >= tiles) break;
        r -= n;
        first += n;
    }
    u.tile = tile;
    u.unit = (p.prefix_tiles + c0.y) * t.kv_heads + u.head * tiles + tile;
    u.first = first;
    u.blocks = n;
    u.t0 = s.t0;
    u.n = s.n;
    u.len = s.len;
    return u;
}

// The page that holds key `key` (of a sequence or the prefix); -1 past the
// table, which a bulk copy reads as zeros.
__device__ __forceinline__ int page_of(const wq_attention& t, int seq, int key) {
    const int i = divide(key, t.cache.page_size);
    if (seq < 0) return i < t.prefix_table_pages ? t.prefix_pages[i] : -1;
    return i < t.table_pages ? t.tables[seq * t.table_stride + i] : -1;
}

}  // namespace attn
}  // namespace wq
