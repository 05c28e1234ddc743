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
    long long* plan;  // see Plan::publish
};

constexpr int kMaxSeq = 1024;
// shared memory of the plan's sums
__host__ __device__ constexpr size_t plan_smem(int sequences) { return ((size_t)sequences + 1) * 12 + 16; }

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

// keys that the row tile `rt` of a sequence can see: those of its last row
__device__ __forceinline__ int tile_keys(const Seq& s, int group, int rows, int rt) {
    const long long last = (long long)(rt + 1) * rows - 1;
    const long long query = last / group;
    const int q = query < s.n ? (int)query : s.n - 1;
    const int keys = s.len - s.n + q + 1;
    return keys < 0 ? 0 : keys;
}

__device__ __forceinline__ int row_tiles(int n, int group, int rows) {
    return (int)(((long long)n * group + rows - 1) / rows);
}

// blocks of that tile
template <int ROWS, int BK>
__device__ __forceinline__ int tile_blocks(const Args& a, const Seq& s, int rt) {
    return (a.concat ? (a.t.prefix_len + BK - 1) / BK : 0) + (tile_keys(s, a.group, ROWS, rt) + BK - 1) / BK;
}

// Sums over the sequences before b, for one key head: blocks and row tiles.
struct Plan {
    long long* blocks;         // sequences + 1, in shared memory
    int* tiles;
    long long prefix_blocks;   // of one unit
    int prefix_tiles;
    long long prefix_line;     // blocks of all prefix units
    long long line;            // all blocks
    long long run;             // blocks of a run
    long long scratch[32];
};

// Made by all threads of the CTA (NT of them, a multiple of 32), its sums at
// `sums` (plan_smem bytes, 8-byte aligned); ends with a barrier.
template <int NT, int ROWS, int BK>
__device__ void make_plan(Plan& p, const Args& a, void* sums) {
    const wq_attention& t = a.t;
    if (threadIdx.x == 0) {
        p.blocks = static_cast<long long*>(sums);
        p.tiles = reinterpret_cast<int*>(p.blocks + t.sequences + 1);
    }
    __syncthreads();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int B = a.own ? t.sequences : 0;
    const int per = (B + NT - 1) / NT;
    // this thread's sequences
    long long blocks = 0;
    int tiles = 0;
    const int b0 = tid * per, b1 = b0 + per < B ? b0 + per : B;
    for (int b = b0; b < b1; ++b) {
        const Seq s = seq_at(t, b);
        const int rt = row_tiles(s.n, a.group, ROWS);
        long long w = 0;
        for (int i = 0; i < rt; ++i) w += tile_blocks<ROWS, BK>(a, s, i);
        p.blocks[b + 1] = w;
        p.tiles[b + 1] = rt;
        blocks += w;
        tiles += rt;
    }
    // exclusive sums over the threads
    long long sb = blocks;
    int st = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long ub = __shfl_up_sync(0xffffffffu, sb, o);
        const int ut = __shfl_up_sync(0xffffffffu, st, o);
        if (lane >= o) {
            sb += ub;
            st += ut;
        }
    }
    if (lane == 31) {
        p.scratch[warp] = sb;
        p.scratch[16 + warp] = st;
    }
    __syncthreads();
    long long ab = sb - blocks;
    int at = st - tiles;
    for (int w = 0; w < warp; ++w) {
        ab += p.scratch[w];
        at += (int)p.scratch[16 + w];
    }
    for (int b = b0; b < b1; ++b) {
        ab += p.blocks[b + 1];
        at += p.tiles[b + 1];
        p.blocks[b + 1] = ab;
        p.tiles[b + 1] = at;
    }
    if (tid == 0) {
        p.blocks[0] = 0;
        p.tiles[0] = 0;
    }
    __syncthreads();
    if (tid == 0) {
        const int rows = a.prefix ? (t.q_start ? clampi(t.q_start[t.sequences], 0, t.tokens) : t.tokens) : 0;
        p.prefix_tiles = row_tiles(rows, a.group, ROWS);
        p.prefix_blocks = a.prefix ? ((long long)t.prefix_len + BK - 1) / BK : 0;
        p.prefix_line = p.prefix_blocks * p.prefix_tiles * t.kv_heads;
        p.line = p.prefix_line + p.blocks[B] * t.kv_heads;
        const long long run = (p.line + a.runs - 1) / a.runs;
        p.run = run < a.min_run ? a.min_run : run;
    }
    __syncthreads();
}

// For combine_kernel: run length, prefix tiles and blocks, then the sums.
constexpr int kPlanHead = 4;
constexpr size_t kPlanBytes = sizeof(long long) * (kPlanHead + 2 * (kMaxSeq + 1));

template <int NT>
__device__ void publish_plan(const Plan& p, const Args& a) {
    const int B = a.own ? a.t.sequences : 0;
    if (threadIdx.x == 0) {
        a.plan[0] = p.run;
        a.plan[1] = p.prefix_tiles;
        a.plan[2] = p.prefix_blocks;
        a.plan[3] = p.prefix_line;
    }
    for (int b = threadIdx.x; b <= B; b += NT) {
        a.plan[kPlanHead + 2 * b] = p.blocks[b];
        a.plan[kPlanHead + 2 * b + 1] = p.tiles[b];
    }
}

// Where a block of the line lies.
struct Unit {
    int seq;            // sequence, -1: prefix
    int head, tile;     // key head, row tile
    int unit;           // number along the line
    long long first;    // the unit's first block on the line
    int blocks;         // of the unit
    int t0, n, len;     // tokens and keys (prefix: all tokens, prefix_len)
};

template <int ROWS, int BK>
__device__ __forceinline__ Unit unit_of(const Plan& p, const Args& a, long long x) {
    const wq_attention& t = a.t;
    Unit u;
    if (x < p.prefix_line) {
        u.seq = -1;
        u.unit = (int)(x / p.prefix_blocks);
        u.head = u.unit / p.prefix_tiles;
        u.tile = u.unit - u.head * p.prefix_tiles;
        u.first = u.unit * p.prefix_blocks;
        u.blocks = (int)p.prefix_blocks;
        u.t0 = 0;
        u.n = t.q_start ? clampi(t.q_start[t.sequences], 0, t.tokens) : t.tokens;
        u.len = t.prefix_len;
        return u;
    }
    const long long y = x - p.prefix_line;
    // the last sequence whose blocks begin at or before y
    int lo = 0, hi = t.sequences - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.blocks[mid] * t.kv_heads <= y) lo = mid;
        else hi = mid - 1;
    }
    const Seq s = seq_at(t, lo);
    const long long w = p.blocks[lo + 1] - p.blocks[lo];
    const long long z = y - p.blocks[lo] * t.kv_heads;
    const int tiles = p.tiles[lo + 1] - p.tiles[lo];
    u.seq = lo;
    u.head = (int)(z / w);
    long long r = z - u.head * w, first = p.prefix_line + p.blocks[lo] * t.kv_heads + u.head * w;
    int tile = 0, n = 0;
    for (;; ++tile) {
        n = tile_blocks<ROWS, BK>(a, s, tile);
        if (r < n || tile + 1 >= tiles) break;
        r -= n;
        first += n;
    }
    u.tile = tile;
    u.unit = p.prefix_tiles * t.kv_heads + p.tiles[lo] * t.kv_heads + u.head * tiles + tile;
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
    const int i = key / t.cache.page_size;
    if (seq < 0) return i < t.prefix_table_pages ? t.prefix_pages[i] : -1;
    return i < t.table_pages ? t.tables[seq * t.table_stride + i] : -1;
}

}  // namespace attn
}  // namespace wq
