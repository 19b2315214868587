// Experts in FP8 with block scales: for pair p of a token (row a of A) and expert e
//
//   D[p][n] = sum_b sa[a][b] sw[e][b][n / 128] sum_{k in block b} A[a][k] W[e][k][n]
//
// with blocks of 128 along K, E4M3 codes on the MFMA of 8-bit types in its unscaled form
// (its own scales are powers of two), one 16 x 16 x 128 product per block, each product
// scaled in fp32 and added to the fp32 sum, one rounding to bf16.  Inside
// a block the instruction cuts the products of 8 neighbouring K to 13 bits below the
// largest one's power of two before it adds them (measured on gfx950, the unscaled
// 16 x 16 x 32 form too): 2^-18.6 of the block's sum of absolute values rms, 1/50 of
// what the bf16 rounding of the result takes.
//
// The rows of an expert are cut into m-tiles (expert, first sorted row, rows).
// Routing: up to kF8InlineP pairs, each workgroup finds its m-tile from the ids or
// the offsets by itself; above, a counting sort by expert and the tile list come
// first: one workgroup up to kF8Chunk pairs, else histograms of chunks in one launch,
// and a second in which each chunk's workgroup sums the histograms for itself and
// places its pairs (32760 pairs: 14 us; with launches of their own for the scan and the
// ranks 17).  Rows of an expert come in any order: a row's sums do not depend on its
// place.
#include "hq_device.hpp"
#include "hq_layer.h"

#include <type_traits>
#include <utility>

namespace hq {

namespace {

constexpr int kF8InlineP = 64;   // one pair per lane of a wave
constexpr int kF8Chunk = 4096;   // pairs of one routing workgroup
constexpr int kF8TileRows = 256; // rows of a large m-tile, at most
constexpr int kF8LeastRows = 96; // (three subtiles of a wave: the fewest that the pipeline of loads is built for)
constexpr int kF8Rows = 32;      // rows that the weight stream takes at a time
// Which experts the weight stream takes: those of up to kF8Rows rows where experts have
// up to kF8Mean rows in the mean, else none.  Two launches of which each has a part of the
// experts end one after the other, so what suits the mean runs it all.  32 experts of
// 4096 x 7168, stream / tiles (us): mean 4 147 / 172, 8 149 / 171, 16 159 / 171, and with
// the stream for up to 16 rows against tiles alone: mean 24 191 / 173, 32 186 / 175; 256
// experts of 7168 x 2048: mean 8 611 / 624, 16 662 / 642, 31 703 / 668.
constexpr int64_t kF8Mean = 16;
constexpr int kF8Sa = 64;        // K blocks of activation scales in LDS at a time (weight stream)

size_t al16(size_t b) { return (b + 15) / 16 * 16; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// An m-tile: `rows` sorted rows from `first`.  In the list of the larger ones: all rows of
// the expert, and the number of the tile among the expert's.
struct Tile {
    int expert, first, rows, number;
};

struct F8Layout {  // byte offsets into the workspace
    size_t hist, sorted, tiles[2], ntiles, bytes;
    int stream, tile_rows;  // as in F8Lists
    int64_t max_tiles[2];  // bounds of the lists of the weight stream's m-tiles and of the others
};
struct F8Lists {
    int stream;     // experts of up to so many rows are for the weight stream (0: none)
    int tile_rows;  // of a larger m-tile, at most
    Tile* tiles[2];
    int* ntiles;  // [2]
    int max_tiles[2];
};

// Rows of the large m-tiles: as few as leave all tiles, by the experts' mean, one for each CU.
// (96 rows or 256, us: 1000 rows on 2 experts of 2048 x 7168 51, 85; 512 on one of 4096 x 4096 32,
// 54; 4096 on one of 1024 x 2048 24, 37; but 3460 on 2 of 4096 x 640, where 96 make 576 tiles, 30, 23.)
int f8_rows_of_tiles(int64_t P, int64_t held, int64_t N) {
    int rows = kF8LeastRows;
    while (P > 0 && rows < kF8TileRows && held * ceil_div(P, held * rows) * ceil_div(N, 256) > 256) rows += 32;
    return rows;
}

F8Layout f8_layout(int64_t T, int top_k, int E, int64_t N) {
    const int64_t P = T * top_k, C = ceil_div(P, kF8Chunk);
    F8Layout L{};
    const int64_t held = E < P ? E : P;  // experts that can have a row
    L.stream = P <= kF8InlineP || P <= kF8Mean * held ? kF8Rows : 0;
    L.max_tiles[0] = L.stream ? held : 0;
    const int64_t many = P / (L.stream + 1);  // experts that can have more rows
    L.tile_rows = f8_rows_of_tiles(P, held, N);
    L.max_tiles[1] = P / L.tile_rows + (E < many ? E : many);
    // room for the lists whichever way is taken: more tokens never need less
    const int64_t most[2] = {held, P / kF8LeastRows + held};
    size_t o = 0;
    L.hist = o;
    o += C > 1 ? al16((size_t)C * E * 4) : 0;
    L.sorted = o;
    o += al16((size_t)P * 4);
    for (int i = 0; i < 2; ++i) {
        L.tiles[i] = o;
        o += al16((size_t)most[i] * sizeof(Tile));
    }
    L.ntiles = o;
    o += 16;
    L.bytes = o;
    return L;
}

// ---------------------------------------------------------------------------
// routing
// ---------------------------------------------------------------------------

// Exclusive scan of three values per thread over 1024 threads (tmp: 48 ints).
__device__ void scan3_1024(int (&v)[3], int* tmp) {
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    int incl[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        incl[i] = v[i];
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int o = __shfl_up(incl[i], off);
            if (lane >= off) incl[i] += o;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 3; ++i)
        if (lane == 63) tmp[16 * i + wave] = incl[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        int before = 0;
        for (int w = 0; w < wave; ++w) before += tmp[16 * i + w];
        v[i] = before + incl[i] - v[i];
    }
}

// How many m-tiles an expert of c rows has in a list, and how many rows each (the last
// may have fewer): the tiles of a large expert are as even as 32 rows allow.
__device__ __forceinline__ int f8_tiles(int c, int list, const F8Lists& l) {
    return c == 0 || (c <= l.stream) != (list == 0) ? 0 : list == 0 ? 1 : (c + l.tile_rows - 1) / l.tile_rows;
}
__device__ __forceinline__ int f8_tile_rows(int c, int most) {
    const int n = (c + most - 1) / most;
    return ((c + 31) / 32 + n - 1) / n * 32;
}

// Where the experts' rows begin (in start), and the tile lists (where `list`), from the
// counts of at most 4096 experts, 4 per thread; `given`: start holds it already.
__device__ void offsets_and_tiles(const int (&cnt)[4], int (&start)[4], bool given, bool list, int E, const F8Lists& lists, int* tmp) {
    const int t = threadIdx.x;
    int v[3] = {};  // rows, tiles of either list
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        v[0] += cnt[k];
        v[1] += f8_tiles(cnt[k], 0, lists);
        v[2] += f8_tiles(cnt[k], 1, lists);
    }
    const int mine[2] = {v[1], v[2]};
    scan3_1024(v, tmp);
    if (list && t == 1023) {
        lists.ntiles[0] = min(v[1] + mine[0], lists.max_tiles[0]);
        lists.ntiles[1] = min(v[2] + mine[1], lists.max_tiles[1]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int e = 4 * t + k;
        if (e < E) {
            if (!given) start[k] = v[0];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int n = f8_tiles(cnt[k], i, lists);
                for (int q = 0; list && q < n && v[1 + i] + q < lists.max_tiles[i]; ++q)
                    lists.tiles[i][v[1 + i] + q] = Tile{e, start[k], cnt[k], q};
                v[1 + i] += n;
            }
        }
        v[0] += cnt[k];
    }
}

constexpr int kF8Each = kF8Chunk / 1024;  // pairs of a thread

// The ids of this thread's pairs (-1: none, or outside), and (where `count`) their counts in cnt[0..4095].
__device__ __forceinline__ void f8_count(const int* ids, int64_t P, int E, bool count, int* cnt, int (&id)[kF8Each]) {
    const int t = threadIdx.x;
    const int64_t p0 = (int64_t)blockIdx.x * kF8Chunk + t;
#pragma unroll
    for (int i = 0; i < kF8Each; ++i) {
        const int v = p0 + i * 1024 < P ? ids[p0 + i * 1024] : -1;
        id[i] = v >= 0 && v < E ? v : -1;
    }
    if (!count) return;
    for (int e = t; e < 4096; e += 1024) cnt[e] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kF8Each; ++i)
        if (id[i] >= 0) atomicAdd(&cnt[id[i]], 1);
    __syncthreads();
}

// Several chunks: the counts of each, ...
__global__ __launch_bounds__(1024) void f8_hist_kernel(const int* __restrict__ ids, int64_t P, int E, int* __restrict__ hist) {
    __shared__ int cnt[4096];
    int id[kF8Each];
    f8_count(ids, P, E, true, cnt, id);
    for (int e = threadIdx.x; e < E; e += 1024) hist[(int64_t)blockIdx.x * E + e] = cnt[e];
}
// ... and the places of its pairs, behind the experts before theirs and the chunks before its own.  One
// chunk (hist NULL): all in one launch.  The tile lists come from the first workgroup.  Each workgroup reads
// every chunk's histogram, which grows with the square of the chunks (256 experts, us: 8 chunks 9, 64 44, 256
// 158, 1024 1150; at 256, a million pairs, the product takes some 100 times that).
__global__ __launch_bounds__(1024) void f8_place_kernel(const int* __restrict__ ids, int64_t P, int E, const int* __restrict__ hist, int* __restrict__ sorted,
                                                        F8Lists lists) {
    __shared__ int cnt[4096];
    __shared__ int tmp[48];
    const int t = threadIdx.x;
    int id[kF8Each];
    f8_count(ids, P, E, !hist, cnt, id);
    int all[4] = {}, before[4] = {}, start[4] = {};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int e = 4 * t + k;
        if (!hist) all[k] = cnt[e];
        else if (e < E)
            for (int c = 0; c < (int)gridDim.x; ++c) {
                const int n = hist[(int64_t)c * E + e];
                all[k] += n;
                before[k] += c < (int)blockIdx.x ? n : 0;
            }
    }
    offsets_and_tiles(all, start, false, blockIdx.x == 0, E, lists, tmp);  // (barriers inside: cnt is read)
#pragma unroll
    for (int k = 0; k < 4; ++k) cnt[4 * t + k] = start[k] + before[k];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kF8Each; ++i)
        if (id[i] >= 0) sorted[atomicAdd(&cnt[id[i]], 1)] = (int)((int64_t)blockIdx.x * kF8Chunk + i * 1024 + t);
}
// Grouped: the lists alone, from the offsets given.
__global__ __launch_bounds__(1024) void f8_list_kernel(const int* __restrict__ given, int64_t P, int E, F8Lists lists) {
    __shared__ int tmp[48];
    int c[4] = {}, first[4] = {};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int e = 4 * (int)threadIdx.x + k;
        if (e >= E) continue;
        // clamped: malformed offsets never address rows outside A or D
        first[k] = min(max(given[e], 0), (int)P);
        c[k] = min(max(given[e + 1], first[k]), (int)P) - first[k];
    }
    offsets_and_tiles(c, first, true, true, E, lists, tmp);
}

// ---------------------------------------------------------------------------
// the products
// ---------------------------------------------------------------------------

struct F8Params {
    const uint8_t* A;
    const float* sa;
    const uint8_t* W;
    const float* S;
    uint16_t* D;
    int64_t w_estride, s_estride;  // bytes, floats
    int K, N, nb, ncb;             // nb: blocks of 128 along K; ncb: along N
    uint32_t strips;               // padded N / 16
    int64_t a_rows;
    int top_k;
    const Tile* tiles;
    const int* ntiles;
    int max_tiles;      // entries of `tiles`
    int tile_rows;      // as in F8Lists
    const int* sorted;  // Indexed: pair of each sorted row
    // at most kF8InlineP pairs: the tile from the ids (Indexed) or offsets (Grouped)
    const int *ids, *offsets;
    int P, E;
};

constexpr uint32_t kNone = 0x80000000u;  // past every weight and scale resource: reads zeros (of A: some byte, or zeros)
constexpr int kF8SaRow = kF8Sa + 1;      // (one word more: the rows' scales of a block lie on different banks)

// s_waitcnt vmcnt(N), the other counters left alone (gfx9 encoding).
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
    static_assert(N >= 0 && N < 64, "vmcnt is a 6-bit counter");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}
// Workgroup barriers for direct loads to LDS: a wave has waited for its own by then, and
// __syncthreads() would wait for every load in flight.  lds_sync: for LDS writes too.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}
__device__ __forceinline__ void lds_sync() {
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    lds_barrier();
}

union F8Frag {
    v4u q[2];
    v8i v;
};

// One product of a block: 16 columns of weights as the MFMA's rows, 16 rows of A as its
// columns.  So a lane's results belong to ONE row of A (column lane & 15 of the result):
// the row's scale is one value per lane, and its four results are neighbouring columns
// of D (4 (lane >> 4) .. + 3).
__device__ __forceinline__ v4f f8_product(const F8Frag& w, const F8Frag& a) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w.v, a.v, v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);  // (no scales: the unscaled form)
}
// Columns n .. n + 3 of row `row` of D (-1: none).
__device__ __forceinline__ void f8_store(const F8Params& p, int row, int n, const v4f& v) {
    if (row < 0) return;
    uint16_t* d = p.D + (int64_t)row * p.N + n;
    if (p.N % 4 == 0) {  // (then n + 3 < N wherever n < N, and the address is a multiple of 8)
        if (n < p.N)
            *(uint2*)d = make_uint2((uint32_t)f32_to_bf16_bits(v[0]) | ((uint32_t)f32_to_bf16_bits(v[1]) << 16),
                                    (uint32_t)f32_to_bf16_bits(v[2]) | ((uint32_t)f32_to_bf16_bits(v[3]) << 16));
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (n + r < p.N) d[r] = f32_to_bf16_bits(v[r]);
    }
}

// The products of one m-tile (MT x 16 rows) with 128 columns: four waves of two strips
// (16 columns) each.  Every wave streams its weights from HBM to registers, PF blocks
// ahead: a lane's 32 bytes of a block are its MFMA operand as packed.  The rows' codes
// come the same way: they are few, and the other waves' and workgroups' reads of them
// hit the caches.  No barrier in the stream; scales of the rows sit in LDS.
template <int MT>
__device__ __forceinline__ void f8_stream(const F8Params& p, const Tile& tile, int cb, const int* rowA, const int* rowD, float* sal) {
    constexpr int NT = 2, PF = 4;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, quad = lane >> 4;
    const int nb = p.nb;
    const rsrc_t rW = make_rsrc(p.W + (int64_t)tile.expert * p.w_estride, (uint32_t)p.w_estride);
    const rsrc_t rA = make_rsrc(p.A, (uint32_t)(p.a_rows * p.K));
    const rsrc_t rS = make_rsrc(p.S + (int64_t)tile.expert * p.s_estride, (uint32_t)(p.s_estride * 4));
    uint32_t boff[NT], aoff[MT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const uint32_t strip = (uint32_t)(cb * 8 + wave * NT + j);
        boff[j] = strip < p.strips ? strip * (uint32_t)nb * 2048u + (uint32_t)lane * 16u : kNone;
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) aoff[i] = (uint32_t)rowA[i * 16 + col] * (uint32_t)p.K + (uint32_t)quad * 16u;

    F8Frag b[PF][NT], a[PF][MT];
    auto load = [&](int s, int blk) {
        const bool ok = blk < nb;  // (past K: nothing is fetched)
        const uint32_t at = ok ? (uint32_t)blk : 0u;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) b[s][j].q[h] = buf16<true>(rW, ok ? boff[j] : kNone, at * 2048u + h * 1024u);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) a[s][i].q[h] = buf16(rA, ok ? aoff[i] : kNone, at * 128u + h * 64u);
    };
    v4f acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < PF; ++s) load(s, s);

    for (int b0 = 0; b0 < nb; b0 += kF8Sa) {
        const int n = min(nb - b0, kF8Sa);
        // scales of the rows; lane l keeps the weight scale of block b0 + l
        __syncthreads();
        for (int i = tid; i < MT * 16 * kF8Sa; i += 256) {
            const int r = i / kF8Sa, s = i % kF8Sa;
            if (s < n) sal[r * kF8SaRow + s] = p.sa[(int64_t)rowA[r] * nb + b0 + s];
        }
        const float sw_lane = __uint_as_float(buf4(rS, lane < n ? (uint32_t)((b0 + lane) * p.ncb + cb) * 4u : kNone, 0u));
        __syncthreads();
        for (int s0 = 0; s0 < n; s0 += PF) {
#pragma unroll
            for (int s = 0; s < PF; ++s) {
                if (s0 + s < n) {  // (blocks past K add nothing)
                    const float sw = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(sw_lane), s0 + s));
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        const float sc = sal[(i * 16 + col) * kF8SaRow + s0 + s] * sw;
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            const v4f part = f8_product(b[s][j], a[s][i]);
#pragma unroll
                            for (int r = 0; r < 4; ++r) acc[i][j][r] += part[r] * sc;
                        }
                    }
                }
                load(s, b0 + s0 + s + PF);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i) f8_store(p, rowD[i * 16 + col], (cb * 8 + wave * NT + j) * 16 + quad * 4, acc[i][j]);
}

__global__ __launch_bounds__(256) void f8_stream_kernel(F8Params p) {
    __shared__ int rowA[kF8InlineP], rowD[kF8InlineP];
    __shared__ __attribute__((aligned(16))) float sal[kF8SaRow * kF8Rows];
    __shared__ int owner[kF8InlineP];
    const int tid = threadIdx.x, lane = tid & 63;
    const int cb = blockIdx.x % (unsigned)p.ncb, mt = blockIdx.x / (unsigned)p.ncb;  // column block, m-tile
    Tile tile;
    if (p.ids || p.offsets) {
        // pair (or sorted row) `lane` and its expert; tile t is the t-th expert in order of
        // its first pair
        if (p.offsets) {
            if (tid < kF8InlineP) owner[tid] = -1;
            __syncthreads();
            for (int e = tid; e < p.E; e += 256) {
                const int lo = min(max(p.offsets[e], 0), p.P), hi = min(max(p.offsets[e + 1], lo), p.P);
                for (int i = lo; i < hi; ++i) owner[i] = e;  // (overlapping ranges: one owner)
            }
            __syncthreads();
        }
        int id = -1;
        if (lane < p.P) id = p.ids ? p.ids[lane] : owner[lane];
        if (id < 0 || id >= p.E) id = -1;
        int before = 0;
        for (int j = 0; j < p.P; ++j) {
            const int v = __builtin_amdgcn_readlane(id, j);
            before += v == id && j < lane ? 1 : 0;
        }
        const uint64_t leads = __ballot(id >= 0 && before == 0);
        if (mt >= __popcll(leads)) return;
        const int t = __popcll(leads & ((1ull << lane) - 1ull));
        const uint64_t mine = __ballot(id >= 0 && before == 0 && t == mt);
        const int e = __builtin_amdgcn_readlane(id, __builtin_ctzll(mine));
        const uint64_t rows = __ballot(id == e);
        tile = Tile{e, 0, (int)__popcll(rows), 0};
        if (tid < kF8InlineP) {
            rowD[lane] = -1;
            rowA[lane] = p.ids ? __builtin_ctzll(rows) / p.top_k : __builtin_ctzll(rows);
            if (id == e) {
                rowD[before] = lane;
                rowA[before] = p.ids ? lane / p.top_k : lane;
            }
        }
    } else {
        if (mt >= *p.ntiles) return;
        tile = p.tiles[mt];
        if (tid < kF8Rows) {
            const int pos = tile.first + min(tid, tile.rows - 1);
            const int pair = p.sorted ? p.sorted[pos] : pos;
            rowA[tid] = p.sorted ? pair / p.top_k : pos;
            rowD[tid] = tid < tile.rows ? pair : -1;
        }
    }
    tile.expert = __builtin_amdgcn_readfirstlane(tile.expert);
    tile.rows = __builtin_amdgcn_readfirstlane(tile.rows);
    __syncthreads();
    // (more than kF8Rows only where the pairs are so few that no list was made)
    for (int r = 0; r < tile.rows; r += kF8Rows) {
        if (tile.rows - r <= 16) f8_stream<1>(p, tile, cb, rowA + r, rowD + r, sal);
        else f8_stream<2>(p, tile, cb, rowA + r, rowD + r, sal);
    }
}

// ---- m-tiles of more rows: 256 x 256 of D on eight waves ----
//
// Wave (wm, wn) has the 16-row subtiles 2 i + wm (i < MT) and the columns 64 wn .. + 63.
// Codes of rows and weights both go to LDS by direct loads: a CU takes 51 bytes a clock
// from L2 that way, into registers 39 (measured), and LDS gives 214; with the weights
// loaded to registers by each of the two waves that need them the tile ran at half the
// rate.  Two stages of 64 KB fill the LDS, and are filled again piece by piece as they
// come free, so that every piece has one and a half blocks' time to land:
//   P(s), before the last subtile of block s - 1: the weights and the first rows of block
//        s have landed, block s - 1 is read to its end; A2(s + 1) is asked for
//   M(s), before subtile H - 1 of block s: its later rows (A2) have landed, its weights
//        are in registers and its first rows (A1) read; A1(s + 2) and B(s + 2) are asked for
// The rows' scales come four blocks at a time through registers, the weights' wait in a
// lane each.
// m-tiles of an expert that run side by side (32 experts of 4096 x 7168, 32760 / 16384 rows, us: one 985 / 530,
// four 928 / 521, six 938 / 510, sixteen 957 / 516)
constexpr int kF8Group = 6;
constexpr int kF8Half = 128 * 128;  // bytes of A1 or A2 of a stage: 128 rows of a block

// The row of A of local row r (past the tile's last: that one), and its row of D (past it: -1).
__device__ __forceinline__ int f8_row(const F8Params& p, const Tile& tile, int r, int* d) {
    const int pos = tile.first + min(r, tile.rows - 1), pair = p.sorted ? p.sorted[pos] : pos;
    if (d) *d = r < tile.rows ? pair : -1;
    return p.sorted ? pair / p.top_k : pos;
}

struct F8Stage {
    char *a1[2], *a2[2], *b[2];
    float* sa;
};

template <class F, int... I>
__device__ __forceinline__ void each_of(F& f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}

template <int MT>
__device__ __forceinline__ void f8_tile(const F8Params& p, const Tile& tile, int tn, int* rowD, const F8Stage& st) {
    constexpr int NT = 4, H = MT >= 6 ? 4 : 2;                       // strips of a wave; subtiles of A1
    constexpr int L1 = H / 2, L2 = (MT - H + 1) / 2, LB = 4;         // loads of a block: 64 rows each, 8 KB each
    constexpr int kSa = kF8TileRows * 4;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 2, wn = wave & 3, col = lane & 15, quad = lane >> 4;
    const int nb = p.nb, cb = tn * 2 + (wn >> 1);
    const rsrc_t rW = make_rsrc(p.W + (int64_t)tile.expert * p.w_estride, (uint32_t)p.w_estride);
    const rsrc_t rA = make_rsrc(p.A, (uint32_t)(p.a_rows * p.K));
    const rsrc_t rS = make_rsrc(p.S + (int64_t)tile.expert * p.s_estride, (uint32_t)(p.s_estride * 4));
    const rsrc_t rSA = make_rsrc(p.sa, (uint32_t)(p.a_rows * nb * 4));
    // wave w loads the strips 2 w and 2 w + 1 (past the last: that one, for columns that are not stored)
    const uint32_t strip_bytes = (uint32_t)nb * 2048u, boff = (uint32_t)lane * 16u;
    const uint32_t strip[2] = {min((uint32_t)(tn * 16 + wave * 2), p.strips - 1u) * strip_bytes, min((uint32_t)(tn * 16 + wave * 2 + 1), p.strips - 1u) * strip_bytes};
#pragma unroll
    for (int n = 0; n < LB; ++n)  // (block 0's weights: they need no row)
        dma16(rW, (lds_char*)st.b[0] + wave * 4096 + n * 1024, boff, strip[n >> 1] + (n & 1) * 1024u);
    // 16-byte slot i * 512 + tid of A1 and A2 together: row slot / 8, and of it the unit
    // slot % 8 ^ (row >> 1 & 7), which spreads the reads of 16 rows over the banks
    uint32_t aoff[L1 + L2];
#pragma unroll
    for (int i = 0; i < L1 + L2; ++i) {
        const int row = i * 64 + (tid >> 3), unit = (tid & 7) ^ ((row >> 1) & 7);
        aoff[i] = (uint32_t)f8_row(p, tile, row, nullptr) * (uint32_t)p.K + (uint32_t)unit * 16u;
    }
    uint32_t saoff = 0;
    if (tid < kF8TileRows) saoff = (uint32_t)f8_row(p, tile, tid, rowD + tid) * (uint32_t)nb * 4u;
    // load n of the L1 + LB that M asks for (weights first), or of P's L2; past K the last
    // block again, not used
    auto load_m = [&](int blk, int s, int n) {
        const int at = min(blk, nb - 1);
        if (n < LB)
            dma16(rW, (lds_char*)st.b[s] + wave * 4096 + n * 1024, boff, strip[n >> 1] + (uint32_t)at * 2048u + (n & 1) * 1024u);
        else
            dma16(rA, (lds_char*)st.a1[s] + wave * 1024 + (n - LB) * 8192, aoff[n - LB], (uint32_t)at * 128u);
    };
    auto load_p = [&](int blk, int s, int n) {
        dma16(rA, (lds_char*)st.a2[s] + wave * 1024 + n * 8192, aoff[L1 + n], (uint32_t)min(blk, nb - 1) * 128u);
    };
    float acc[MT][NT][4] = {};
    v4u sa_next = buf16(rSA, saoff, 0u);
    float sw_lane = 0.f, sw = 0.f;
    // this lane's operand of a subtile: units quad and 4 + quad of its row
    const int f0 = (wm * 16 + col) * 128 + ((quad ^ ((col >> 1) & 7)) * 16), f1 = f0 ^ 64;
    F8Frag a[2], b[NT];
    float sa[2], sc = 0.f;
    v4f part[4] = {};
    auto read_a = [&](auto s, auto ic, int to) {  // subtile i of block s
        constexpr int S = decltype(s)::value, i = decltype(ic)::value;
        const char* A = i < H ? st.a1[S & 1] + i * 4096 : st.a2[S & 1] + (i - H) * 4096;
        a[to].q[0] = *(const v4u*)(A + f0);
        a[to].q[1] = *(const v4u*)(A + f1);
    };
    auto read_b = [&](auto s, int j) {
        const char* B = st.b[decltype(s)::value & 1] + (wn * NT + j) * 2048 + lane * 16;
        b[j].q[0] = *(const v4u*)B;
        b[j].q[1] = *(const v4u*)(B + 1024);
    };
    // Block s: product k = 4 i + j, and the fp32 sum of the product before the last, so that
    // no sum waits for its product (the last two of a block are summed in the next one).
    auto block = [&](int s, const float* sal, const float* sal_next, float* sa_to, auto cur) {
        constexpr int S = decltype(cur)::value;
        using Next = std::integral_constant<int, S + 1>;
        auto subtile = [&](auto ic) {
            constexpr int i = decltype(ic)::value;
            // (an odd MT swaps the two operand sets from block to block)
            constexpr int now = (MT & 1) ? (i + S) & 1 : i & 1;
            if constexpr (i == H - 1) {  // M(s)
                wait_vmcnt<L1 + L2 + LB>();
                lds_sync();
                if constexpr (S == 0) sa_next = buf16(rSA, saoff, (uint32_t)min(s + 4, nb - 1) * 4u);
            }
            if constexpr (i == MT - 1) {  // P(s + 1)
                wait_vmcnt<L1 + L2 + LB>();
                if constexpr (S == 3)
                    if (tid < kF8TileRows) *(v4u*)(sa_to + tid * 4) = sa_next;
                lds_sync();
                read_a(Next{}, std::integral_constant<int, 0>{}, now ^ 1);
                sa[now ^ 1] = S < 3 ? sal[S + 1] : sal_next[0];
            } else {
                read_a(cur, std::integral_constant<int, i + 1>{}, now ^ 1);
                sa[now ^ 1] = sal[(i + 1) * 128 + S];
            }
            if constexpr (i == 0) sw = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(sw_lane), s & 63));
            const float before = sc;
            sc = sa[now] * sw;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                // product (i, j); sum of (i, j - 2), or of the subtile before
                float(&sum)[4] = j >= 2 ? acc[i][j - 2] : acc[i > 0 ? i - 1 : MT - 1][j + NT - 2];
                part[j & 3] = f8_product(b[j], a[now]);
                if constexpr (i == MT - 1) read_b(Next{}, j);
                // the loads that the last barrier allows, a few with each product
                const int since = i == MT - 1 ? j : (i - (H - 1)) * NT + j;
                if constexpr (i == MT - 1) {
                    if (since < L2) load_p(s + 2, S & 1, since);
                } else if constexpr (i >= H - 1) {
                    constexpr int each = (L1 + LB + (MT - H) * NT - 1) / ((MT - H) * NT);
#pragma unroll
                    for (int n = since * each; n < since * each + each; ++n)
                        if (n < L1 + LB) load_m(s + 2, S & 1, n);
                }
                const float c = j >= 2 ? sc : before;
#pragma unroll
                for (int r = 0; r < 4; ++r) sum[r] += part[(j + 2) & 3][r] * c;
                // the sum is wanted now: without this the products of several blocks are put
                // off behind the loads that follow, and their operands do not fit the registers
                asm volatile("" : "+v"(sum[0]), "+v"(sum[1]), "+v"(sum[2]), "+v"(sum[3]));
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        each_of(subtile, std::make_integer_sequence<int, MT>{});
    };
    using S0 = std::integral_constant<int, 0>;
    using S1 = std::integral_constant<int, 1>;
    using S2 = std::integral_constant<int, 2>;
    using S3 = std::integral_constant<int, 3>;
#pragma unroll
    for (int n = LB; n < L1 + LB; ++n) load_m(0, 0, n);
#pragma unroll
    for (int n = 0; n < L2; ++n) load_p(0, 0, n);
#pragma unroll
    for (int n = 0; n < L1 + LB; ++n) load_m(1, 1, n);
    if (tid < kF8TileRows) *(v4u*)(st.sa + tid * 4) = sa_next;
    wait_vmcnt<L1 + L2 + LB>();  // P(0)
    lds_sync();
#pragma unroll
    for (int n = 0; n < L2; ++n) load_p(1, 1, n);
    const float* sal = st.sa + (wm * 16 + col) * 4;
    read_a(S0{}, S0{}, 0);
    sa[0] = sal[0];
#pragma unroll
    for (int j = 0; j < NT; ++j) read_b(S0{}, j);
    // four blocks a turn, without branches between them (across one the compiler moves the
    // products behind the loads that follow), then the last one to three
    int s = 0;
    auto scales = [&](float*& to, const float*& here, const float*& next) {
        const int now = (s >> 2) & 1;  // which of the two buffers
        here = sal + now * kSa;
        next = sal + (now ^ 1) * kSa;
        to = st.sa + (now ^ 1) * kSa;
        if ((s & 63) == 0) {
            sw_lane = __uint_as_float(buf4(rS, s + lane < nb ? (uint32_t)((s + lane) * p.ncb + cb) * 4u : kNone, 0u));
            asm volatile("" : "+v"(sw_lane));  // (waited for here, not at each use)
        }
    };
    float* to;
    const float *here, *next;
    for (; s + 4 <= nb; s += 4) {
        scales(to, here, next);
        block(s, here, next, to, S0{});
        block(s + 1, here, next, to, S1{});
        block(s + 2, here, next, to, S2{});
        block(s + 3, here, next, to, S3{});
    }
    if (s < nb) {
        scales(to, here, next);
        block(s, here, next, to, S0{});
        if (s + 1 < nb) block(s + 1, here, next, to, S1{});
        if (s + 2 < nb) block(s + 2, here, next, to, S2{});
    }
#pragma unroll
    for (int j = NT - 2; j < NT; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[MT - 1][j][r] += part[j & 3][r] * sc;
    wait_vmcnt<0>();  // no direct load is in flight any more
    if (p.N % 8 == 0) {
        // through LDS, a subtile at a time and each wave for itself: a lane holds 4 columns of
        // a row, and 8 lanes store the wave's 128 bytes of it in 16 each (stored from where
        // they are, 32 bytes of a row at a time, D took 58 us of 897)
        lds_sync();  // every wave is done with the stages
        char* mine = st.b[0] + wave * 2304;
        const int r8 = lane >> 3, n = tn * 256 + wn * 64 + (lane & 7) * 8;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
                *(uint2*)(mine + col * 144 + j * 32 + quad * 8) =
                    make_uint2((uint32_t)f32_to_bf16_bits(acc[i][j][0]) | ((uint32_t)f32_to_bf16_bits(acc[i][j][1]) << 16),
                               (uint32_t)f32_to_bf16_bits(acc[i][j][2]) | ((uint32_t)f32_to_bf16_bits(acc[i][j][3]) << 16));
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const v4u v = *(const v4u*)(mine + (h * 8 + r8) * 144 + (lane & 7) * 16);
                const int row = rowD[(2 * i + wm) * 16 + h * 8 + r8];
                if (row >= 0 && n < p.N) *(v4u*)(p.D + (int64_t)row * p.N + n) = v;
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
    } else {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int row = rowD[(2 * i + wm) * 16 + col];
#pragma unroll
            for (int j = 0; j < NT; ++j)
                f8_store(p, row, tn * 256 + wn * 64 + j * 16 + quad * 4, v4f{acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]});
        }
    }
}

__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void f8_tile_kernel(F8Params p) {
    // (an array for each piece: the compiler then knows that a direct load into one does not
    // touch what is read from another)
    __shared__ __attribute__((aligned(1024))) char a10[kF8Half], a11[kF8Half], a20[kF8Half], a21[kF8Half], b0[2 * kF8Half], b1[2 * kF8Half];
    __shared__ __attribute__((aligned(16))) float sas[2 * kF8TileRows * 4];
    __shared__ int rowD[kF8TileRows];
    const F8Stage st{{a10, a11}, {a20, a21}, {b0, b1}, sas};
    // Workgroups go round the 8 XCDs: neighbouring tiles to one of them.  Some 32 run on an
    // XCD at a time, and what they read in common comes into its L2 once: so up to kF8Group
    // m-tiles of one expert run side by side, for one 256 columns after the other
    // (256 workgroups at a time, 32 for each XCD: which tile is whose does not wait for how many there are)
    const int tiles_n = (p.N + 255) / 256;
    const int id = (blockIdx.x & ~255) + (blockIdx.x & 7) * 32 + ((blockIdx.x >> 3) & 31);
    if (id / tiles_n >= p.max_tiles) return;
    const int ntiles = p.ntiles[1];
    Tile tile = p.tiles[id / tiles_n];  // a tile of the same group
    if (id / tiles_n >= ntiles) return;
    tile.expert = __builtin_amdgcn_readfirstlane(tile.expert);
    const int count = __builtin_amdgcn_readfirstlane(tile.rows), step = f8_tile_rows(count, p.tile_rows), number = __builtin_amdgcn_readfirstlane(tile.number);
    const int group = number / kF8Group * kF8Group, n = min(kF8Group, (count + p.tile_rows - 1) / p.tile_rows - group);
    const int in_group = id - (id / tiles_n - (number - group)) * tiles_n, tn = in_group / n, m = group + in_group % n;
    tile.first += m * step;
    tile.rows = min(step, count - m * step);
    switch ((tile.rows + 31) / 32) {
        case 1:
        case 2:
        case 3: return f8_tile<3>(p, tile, tn, rowD, st);
        case 4: return f8_tile<4>(p, tile, tn, rowD, st);
        case 5: return f8_tile<5>(p, tile, tn, rowD, st);
        case 6: return f8_tile<6>(p, tile, tn, rowD, st);
        case 7: return f8_tile<7>(p, tile, tn, rowD, st);
        default: return f8_tile<8>(p, tile, tn, rowD, st);
    }
}

}  // namespace

size_t moe_f8_workspace(int64_t T, int top_k, int E) {
    return f8_layout(T, top_k, E, 1).bytes;
}

hipError_t moe_f8_launch(const MoeF8Args& a) {
    const int64_t P = a.T * a.top_k;
    const F8Layout L = f8_layout(a.T, a.top_k, a.E, a.N);
    char* ws = (char*)a.ws;
    F8Params p{};
    p.A = (const uint8_t*)a.A;
    p.sa = a.sa;
    p.W = (const uint8_t*)a.w;
    p.S = (const float*)a.s;
    p.D = (uint16_t*)a.D;
    p.K = (int)a.K;
    p.N = (int)a.N;
    p.nb = (int)(a.K / 128);
    p.ncb = (int)ceil_div(a.N, 128);
    p.strips = (uint32_t)ceil_div(a.N, 16);
    p.w_estride = (int64_t)p.strips * 16 * a.K;
    p.s_estride = (int64_t)p.nb * p.ncb;
    p.a_rows = a.indexed ? a.T : P;
    p.top_k = a.top_k;
    p.P = (int)P;
    p.E = a.E;
    hipError_t e = hipSuccess;
    if (P <= kF8InlineP) {
        p.ids = a.indexed ? a.ids : nullptr;
        p.offsets = a.indexed ? nullptr : a.offsets;
        hipLaunchKernelGGL(f8_stream_kernel, dim3((unsigned)(L.max_tiles[0] * p.ncb)), dim3(256), 0, a.stream, p);
        return hipGetLastError();
    }
    int* sorted = (int*)(ws + L.sorted);
    F8Lists lists{};
    lists.stream = L.stream;
    lists.tile_rows = p.tile_rows = L.tile_rows;
    for (int i = 0; i < 2; ++i) {
        lists.tiles[i] = (Tile*)(ws + L.tiles[i]);
        lists.max_tiles[i] = (int)L.max_tiles[i];
    }
    lists.ntiles = (int*)(ws + L.ntiles);
    if (a.indexed) {
        const unsigned C = (unsigned)ceil_div(P, kF8Chunk);
        int* hist = C > 1 ? (int*)(ws + L.hist) : nullptr;
        if (hist) {
            hipLaunchKernelGGL(f8_hist_kernel, dim3(C), dim3(1024), 0, a.stream, a.ids, P, a.E, hist);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
        hipLaunchKernelGGL(f8_place_kernel, dim3(C), dim3(1024), 0, a.stream, a.ids, P, a.E, (const int*)hist, sorted, lists);
    } else {
        hipLaunchKernelGGL(f8_list_kernel, dim3(1), dim3(1024), 0, a.stream, a.offsets, P, a.E, lists);
    }
    if ((e = hipGetLastError()) != hipSuccess) return e;
    p.ntiles = lists.ntiles;
    p.sorted = a.indexed ? sorted : nullptr;
    if (L.max_tiles[1] > 0) {
        p.tiles = lists.tiles[1];
        p.max_tiles = lists.max_tiles[1];
        hipLaunchKernelGGL(f8_tile_kernel, dim3((unsigned)(ceil_div(L.max_tiles[1] * ceil_div(a.N, 256), 256) * 256)), dim3(512), 0, a.stream, p);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (L.max_tiles[0] == 0) return hipSuccess;
    p.tiles = lists.tiles[0];
    hipLaunchKernelGGL(f8_stream_kernel, dim3((unsigned)(L.max_tiles[0] * p.ncb)), dim3(256), 0, a.stream, p);
    return hipGetLastError();
}

}  // namespace hq
