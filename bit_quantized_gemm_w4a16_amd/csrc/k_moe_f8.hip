// Experts in FP8 with block scales: for pair p of a token (row a of A) and expert e
//
//   D[p][n] = sum_b sa[a][b] sw[e][b][n / 128] sum_{k in block b} A[a][k] W[e][k][n]
//
// with blocks of 128 along K, E4M3 codes on the scaled MFMA (unit scales: the
// instruction's own scales are powers of two), one 16 x 16 x 128 product per block,
// each product scaled in fp32 and added to the fp32 sum, one rounding to bf16.  Inside
// a block the instruction cuts the products of 8 neighbouring K to 13 bits below the
// largest one's power of two before it adds them (measured on gfx950, the unscaled
// 16 x 16 x 32 form too): 2^-18.6 of the block's sum of absolute values rms, 1/50 of
// what the bf16 rounding of the result takes.
//
// The rows of an expert are cut into m-tiles (expert, first sorted row, rows).
// Routing: up to kF8InlineP pairs, each workgroup finds its m-tile from the ids or
// the offsets by itself; above, a counting sort by expert and the tile list come
// first (one workgroup up to kF8Chunk pairs, else histograms of chunks, a scan and
// the placing).  Rows of an expert come in any order: a row's sums do not depend on
// its place.
#include "hq_device.hpp"
#include "hq_layer.h"

namespace hq {

namespace {

constexpr int kF8InlineP = 64;   // one pair per lane of a wave
constexpr int kF8Chunk = 8192;   // pairs of one routing workgroup
constexpr int kF8Rows = 64;      // rows of an m-tile
constexpr int kF8Sa = 64;        // K blocks of activation scales in LDS at a time

size_t al16(size_t b) { return (b + 15) / 16 * 16; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Tile {
    int expert, first, rows;
};

struct F8Layout {  // byte offsets into the workspace
    size_t hist, rank, offsets, sorted, tiles, ntiles, bytes;
    int64_t max_tiles;
};

F8Layout f8_layout(int64_t T, int top_k, int E) {
    const int64_t P = T * top_k, C = ceil_div(P, kF8Chunk);
    F8Layout L{};
    // an expert with c rows has ceil(c / kF8Rows) tiles
    L.max_tiles = P / kF8Rows + (E < P ? E : P);
    size_t o = 0;
    L.hist = o;
    o += C > 1 ? al16((size_t)C * E * 4) : 0;
    L.rank = o;
    o += C > 1 ? al16((size_t)P * 4) : 0;
    L.offsets = o;
    o += al16((size_t)(E + 1) * 4);
    L.sorted = o;
    o += al16((size_t)P * 4);
    L.tiles = o;
    o += al16((size_t)L.max_tiles * sizeof(Tile));
    L.ntiles = o;
    o += 16;
    L.bytes = o;
    return L;
}

// ---------------------------------------------------------------------------
// routing
// ---------------------------------------------------------------------------

// Exclusive scan of two values per thread over 1024 threads (tmp: 32 ints).
__device__ void scan2_1024(int& a, int& b, int* tmp) {
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    int ia = a, ib = b;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int oa = __shfl_up(ia, off), ob = __shfl_up(ib, off);
        if (lane >= off) {
            ia += oa;
            ib += ob;
        }
    }
    __syncthreads();
    if (lane == 63) {
        tmp[wave] = ia;
        tmp[16 + wave] = ib;
    }
    __syncthreads();
    int ba = 0, bb = 0;
    for (int w = 0; w < wave; ++w) {
        ba += tmp[w];
        bb += tmp[16 + w];
    }
    a = ba + ia - a;
    b = bb + ib - b;
}

// Offsets (written to off[0..E], global or LDS) and the tile list from counts of at
// most 4096 experts, 4 per thread.
__device__ void offsets_and_tiles(const int (&cnt)[4], const int (&first_of)[4], bool given, int E, int* off, Tile* tiles, int* ntiles,
                                  int max_tiles, int* tmp) {
    const int t = threadIdx.x;
    int rows = 0, nt = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        rows += cnt[k];
        nt += (cnt[k] + kF8Rows - 1) / kF8Rows;
    }
    const int my_nt = nt;
    scan2_1024(rows, nt, tmp);
    if (t == 1023) *ntiles = min(nt + my_nt, max_tiles);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int e = 4 * t + k;
        if (e < E) {
            const int start = given ? first_of[k] : rows;
            if (off) off[e] = start;
            for (int r = 0; r < cnt[k]; r += kF8Rows, ++nt)
                if (nt < max_tiles) tiles[nt] = Tile{e, start + r, min(kF8Rows, cnt[k] - r)};
        }
        rows += cnt[k];
    }
}

// The whole routing of at most kF8Chunk pairs (Indexed).
__global__ __launch_bounds__(1024) void f8_route_kernel(const int* __restrict__ ids, int P, int E, int* __restrict__ sorted, Tile* __restrict__ tiles,
                                                        int* __restrict__ ntiles, int max_tiles) {
    __shared__ int cnt[4096];
    __shared__ int tmp[32];
    const int t = threadIdx.x;
    for (int e = t; e < 4096; e += 1024) cnt[e] = 0;
    __syncthreads();
    int id[kF8Chunk / 1024], rank[kF8Chunk / 1024];
#pragma unroll
    for (int i = 0; i < kF8Chunk / 1024; ++i) {
        const int p = i * 1024 + t;
        const int v = p < P ? ids[p] : -1;
        id[i] = v >= 0 && v < E ? v : -1;
    }
#pragma unroll
    for (int i = 0; i < kF8Chunk / 1024; ++i) rank[i] = id[i] >= 0 ? atomicAdd(&cnt[id[i]], 1) : 0;
    __syncthreads();
    int c[4], none[4] = {};
#pragma unroll
    for (int k = 0; k < 4; ++k) c[k] = cnt[4 * t + k];
    __syncthreads();
    offsets_and_tiles(c, none, false, E, cnt, tiles, ntiles, max_tiles, tmp);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kF8Chunk / 1024; ++i)
        if (id[i] >= 0) sorted[cnt[id[i]] + rank[i]] = i * 1024 + t;
}

// Several chunks: counts and ranks of each chunk, ...
__global__ __launch_bounds__(1024) void f8_hist_kernel(const int* __restrict__ ids, int64_t P, int E, int* __restrict__ hist, int* __restrict__ rank) {
    __shared__ int cnt[4096];
    const int t = threadIdx.x;
    for (int e = t; e < E; e += 1024) cnt[e] = 0;
    __syncthreads();
    for (int i = t; i < kF8Chunk; i += 1024) {
        const int64_t p = (int64_t)blockIdx.x * kF8Chunk + i;
        const int v = p < P ? ids[p] : -1;
        if (v >= 0 && v < E) rank[p] = atomicAdd(&cnt[v], 1);
    }
    __syncthreads();
    for (int e = t; e < E; e += 1024) hist[(int64_t)blockIdx.x * E + e] = cnt[e];
}
// ... the scan over chunks and experts with the tile list (or the list alone, from given offsets), ...
__global__ __launch_bounds__(1024) void f8_scan_kernel(int* __restrict__ hist, int C, const int* __restrict__ given, int64_t P, int E,
                                                       int* __restrict__ off, Tile* __restrict__ tiles, int* __restrict__ ntiles, int max_tiles) {
    __shared__ int tmp[32];
    const int t = threadIdx.x;
    int c[4], first[4] = {};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int e = 4 * t + k;
        c[k] = 0;
        if (e >= E) continue;
        if (given) {  // clamped: malformed offsets never address rows outside A or D
            first[k] = min(max(given[e], 0), (int)P);
            c[k] = min(max(given[e + 1], first[k]), (int)P) - first[k];
        } else {
            for (int i = 0; i < C; ++i) {
                const int n = hist[(int64_t)i * E + e];
                hist[(int64_t)i * E + e] = c[k];
                c[k] += n;
            }
        }
    }
    offsets_and_tiles(c, first, given != nullptr, E, given ? nullptr : off, tiles, ntiles, max_tiles, tmp);
}
// ... and the placing.
__global__ __launch_bounds__(256) void f8_place_kernel(const int* __restrict__ ids, int64_t P, int E, const int* __restrict__ hist,
                                                       const int* __restrict__ off, const int* __restrict__ rank, int* __restrict__ sorted) {
    const int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (p >= P) return;
    const int v = ids[p];
    if (v >= 0 && v < E) sorted[off[v] + hist[p / kF8Chunk * E + v] + rank[p]] = (int)p;
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
    const int* sorted;  // Indexed: pair of each sorted row
    // at most kF8InlineP pairs: the tile from the ids (Indexed) or offsets (Grouped)
    const int *ids, *offsets;
    int P, E;
};

union F8Frag {
    v4u q[2];
    v8i v;
};

// The products of one m-tile (MT x 16 rows) with 128 columns: four waves of two strips
// (16 columns) each.  Every wave streams its weights from HBM to registers, PF blocks
// ahead: a lane's 32 bytes of a block are its MFMA operand as packed.  The rows' codes
// come the same way: they are few, and the other waves' and workgroups' reads of them
// hit the caches.  No barrier in the stream; scales of the rows sit in LDS.
template <int MT>
__device__ __forceinline__ void f8_stream(const F8Params& p, const Tile& tile, int cb, const int* rowA, const int* rowD, float* sal) {
    constexpr int NT = 2, PF = MT == 4 ? 2 : 4;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, quad = lane >> 4;
    const int nb = p.nb;
    const rsrc_t rW = make_rsrc(p.W + (int64_t)tile.expert * p.w_estride, (uint32_t)p.w_estride);
    const rsrc_t rA = make_rsrc(p.A, (uint32_t)(p.a_rows * p.K));
    const rsrc_t rS = make_rsrc(p.S + (int64_t)tile.expert * p.s_estride, (uint32_t)(p.s_estride * 4));
    constexpr uint32_t kNone = 0x80000000u;  // past every weight and scale resource: reads zeros
    constexpr uint32_t kPast = 0x7F000000u;  // a block past K: zeros, or bytes that are not used
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
        const bool ok = blk < nb;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) b[s][j].q[h] = buf16<true>(rW, boff[j], ok ? (uint32_t)blk * 2048u + h * 1024u : kPast);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) a[s][i].q[h] = buf16(rA, aoff[i], ok ? (uint32_t)blk * 128u + h * 64u : kPast);
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
        // scales of the rows, [block][row]; lane l keeps the weight scale of block b0 + l
        __syncthreads();
        for (int i = tid; i < MT * 16 * kF8Sa; i += 256) {
            const int r = i / kF8Sa, s = i % kF8Sa;
            if (s < n) sal[s * (MT * 16) + r] = p.sa[(int64_t)rowA[r] * nb + b0 + s];
        }
        const float sw_lane = __uint_as_float(buf4(rS, lane < n ? (uint32_t)((b0 + lane) * p.ncb + cb) * 4u : kNone, 0u));
        __syncthreads();
        for (int s0 = 0; s0 < n; s0 += PF) {
#pragma unroll
            for (int s = 0; s < PF; ++s) {
                // blocks past K: their scales are not read, and nothing is added
                const bool live = s0 + s < n;
                const float sw = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(sw_lane), (s0 + s) & 63));
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    v4f sc = *(const v4f*)(sal + (live ? s0 + s : 0) * (MT * 16) + i * 16 + quad * 4);
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const v4f part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a[s][i].v, b[s][j].v, v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0x7F, 0, 0x7F);
                        if (live) {
#pragma unroll
                            for (int r = 0; r < 4; ++r) acc[i][j][r] += part[r] * (sc[r] * sw);
                        }
                    }
                }
                load(s, b0 + s0 + s + PF);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int n = (cb * 8 + wave * NT + j) * 16 + col;
        if (n >= p.N) continue;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = rowD[i * 16 + quad * 4 + r];
                if (row >= 0) p.D[(int64_t)row * p.N + n] = f32_to_bf16_bits(acc[i][j][r]);
            }
    }
}

__global__ __launch_bounds__(256) void f8_stream_kernel(F8Params p) {
    __shared__ int rowA[kF8Rows], rowD[kF8Rows];
    __shared__ __attribute__((aligned(16))) float sal[kF8Sa * kF8Rows];
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
        tile = Tile{e, 0, (int)__popcll(rows)};
        if (tid < kF8Rows) {
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
    if (tile.rows <= 16) f8_stream<1>(p, tile, cb, rowA, rowD, sal);
    else if (tile.rows <= 32) f8_stream<2>(p, tile, cb, rowA, rowD, sal);
    else f8_stream<4>(p, tile, cb, rowA, rowD, sal);
}

}  // namespace

size_t moe_f8_workspace(int64_t T, int top_k, int E) {
    return f8_layout(T, top_k, E).bytes;
}

hipError_t moe_f8_launch(const MoeF8Args& a) {
    const int64_t P = a.T * a.top_k;
    const F8Layout L = f8_layout(a.T, a.top_k, a.E);
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
    int64_t tiles = L.max_tiles;
    hipError_t e = hipSuccess;
    if (P <= kF8InlineP) {
        p.ids = a.indexed ? a.ids : nullptr;
        p.offsets = a.indexed ? nullptr : a.offsets;
        tiles = a.E < P ? a.E : P;
    } else {
        int* off = (int*)(ws + L.offsets);
        int* sorted = (int*)(ws + L.sorted);
        Tile* list = (Tile*)(ws + L.tiles);
        int* ntiles = (int*)(ws + L.ntiles);
        const int C = (int)ceil_div(P, kF8Chunk);
        if (!a.indexed) {
            hipLaunchKernelGGL(f8_scan_kernel, dim3(1), dim3(1024), 0, a.stream, (int*)nullptr, 0, a.offsets, P, a.E, (int*)nullptr, list, ntiles, (int)L.max_tiles);
        } else if (C == 1) {
            hipLaunchKernelGGL(f8_route_kernel, dim3(1), dim3(1024), 0, a.stream, a.ids, (int)P, a.E, sorted, list, ntiles, (int)L.max_tiles);
        } else {
            int *hist = (int*)(ws + L.hist), *rank = (int*)(ws + L.rank);
            hipLaunchKernelGGL(f8_hist_kernel, dim3((unsigned)C), dim3(1024), 0, a.stream, a.ids, P, a.E, hist, rank);
            if ((e = hipGetLastError()) != hipSuccess) return e;
            hipLaunchKernelGGL(f8_scan_kernel, dim3(1), dim3(1024), 0, a.stream, hist, C, (const int*)nullptr, P, a.E, off, list, ntiles, (int)L.max_tiles);
            if ((e = hipGetLastError()) != hipSuccess) return e;
            hipLaunchKernelGGL(f8_place_kernel, dim3((unsigned)ceil_div(P, 256)), dim3(256), 0, a.stream, a.ids, P, a.E, (const int*)hist, (const int*)off,
                               (const int*)rank, sorted);
        }
        if ((e = hipGetLastError()) != hipSuccess) return e;
        p.tiles = list;
        p.ntiles = ntiles;
        p.sorted = a.indexed ? sorted : nullptr;
    }
    hipLaunchKernelGGL(f8_stream_kernel, dim3((unsigned)(tiles * p.ncb)), dim3(256), 0, a.stream, p);
    return hipGetLastError();
}

}  // namespace hq
