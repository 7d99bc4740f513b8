// dllm_embed: the packed box's token ids to scaled embedding rows; dllm_embed_grad: the table's
// gradient.
//
// [BlockServe] = page "BlockServe: 块粒度连续批处理实现高吞吐扩散大语言模型服务" §II-E 逻辑位置对齐:
// the box is a dense left-padded tensor, which the forward embeds; padding contributes nothing.
//
//   out[n] = scale * table[ids[n]];     grad_table[v] (+)= scale * sum over tokens n of v of grad_out[n].
//
// Lookup (gfx950): a gather bound by HBM writes (and reads of the distinct rows).  A wave takes one token
// and 2048 of its columns (kLookVecs vectors of 8 elements per lane, all in flight together); narrow
// tables put several tokens side by side in a wave.  128 x 1280 tokens of width 4096, bf16 (0.33 GB of rows
// read, 1.34 GB written) take 305 us = 5.5 TB/s; 1, 2, 3, 8 vectors per lane take 424, 322, 314, 323, four tokens
// per thread 389, non-temporal row reads 378 (hot rows live in the caches), plain stores 366.
//
// Gradient: the tokens are sorted by id (stable, so a row's terms are summed in token order and the
// bits never depend on timing; no float atomics), then every run of equal ids is summed once and
// written once.
//   1. Sort: least-significant-digit radix sort of (id, position), kDigit bits a pass, as few passes as
//      the vocabulary's bits need.  A pass counts digits per tile, then moves the items; a wave finds
//      an item's rank among equal digits by one ballot per digit bit.  One tile: all passes in one
//      launch.  The sort keeps few compute units busy, so each of its launches also writes zeros to as
//      much of the table as hides it; what a large table has left, a launch of its own clears faster.
//      Rows that do occur are written again in step 2.  (Looking up which rows occur and clearing the
//      others beside the sums instead took 317 us for 1.25 GB of bf16 table and 64 x 544 tokens.)
//   2. Sum: one wave per piece of kPiece sorted tokens and 512 columns.  It loads kAhead tokens at a time
//      whatever run they belong to (most runs are a token or two), adds them in order, and writes a
//      row where a run ends.  A piece sums the runs that start in it, following the last one past its
//      end, so runs up to kPiece tokens are never split.  A longer run (the mask token of a training
//      box can hold half of all tokens) leaves one partial sum per piece it covers.
//   3. Join: the partial sums of each long run, in order.
// 64 x 544 tokens of width 4096 into 152066 bf16 rows take 285 us, of which the zeros (1.25 GB) 202 with the sort
// behind a quarter of them, the sums 75 (0.32 GB, while the last-level cache still drains zeros; 75 for 0.41 GB when
// accumulating), the join 8.  Two batches of 1600 tokens of width 1000 take 49 us, bound by six dependent launches.
#include <algorithm>
#include <type_traits>

#include "elem_common.h"

namespace {

using namespace dllm;

constexpr int kVec = 8;                        // elements per vector
constexpr int kLookWaves = 2;                  // waves per workgroup of the lookup
constexpr int kLookVecs = 4;                   // vectors per lane

// A lane's 8 columns: c .. c+7, or (SPLIT) c .. c+3 and c+half .. c+half+3.  8 neighbours are 16 bytes of bf16; of
// fp32 they are two stores that each cover half of every 32 bytes, where two groups of 4 are two dense ones: 292 us
// against 446 for 163840 rows of 2048 looked up from bf16 into fp32, 339 against 406 from fp32.  (The gradient's
// sums gain nothing from it: they are bound elsewhere, and bf16 loads of 8 bytes cost its small case 10 us of 48.)
template <bool BF16>
struct Group {
    typedef uint32_t vec __attribute__((ext_vector_type(BF16 ? 2 : 4)));
    typedef vec any __attribute__((aligned(BF16 ? 2 : 4)));
};
// 4 columns as stored (0 past D), the row's ragged end element by element.
template <bool BF16>
__device__ __forceinline__ typename Group<BF16>::vec load_group(const char *row, int c, int D) {
    typedef typename Group<BF16>::any any;
    if (c + 4 <= D) return *(const any *)(row + (int64_t)c * (BF16 ? 2 : 4));
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        w[e] = c + e >= D ? 0u : BF16 ? (uint32_t)((const uint16_t *)row)[c + e] : ((const uint32_t *)row)[c + e];
    typename Group<BF16>::vec r;
    if constexpr (BF16) r = {w[0] | w[1] << 16, w[2] | w[3] << 16};
    else r = {w[0], w[1], w[2], w[3]};
    return r;
}
template <bool BF16>
struct Raw {
    u32x4 a[BF16 ? 1 : 2];
};
template <bool BF16, bool SPLIT>
__device__ __forceinline__ Raw<BF16> load_raw(const char *row, int c, int half, int D) {
    typedef typename Row<BF16>::vec vec;
    Raw<BF16> r;
    if constexpr (SPLIT) {
        const auto lo = load_group<BF16>(row, c, D), hi = load_group<BF16>(row, c + half, D);
        if constexpr (BF16) {
            r.a[0] = u32x4{lo.x, lo.y, hi.x, hi.y};
        } else {
            r.a[0] = lo;
            r.a[1] = hi;
        }
    } else if (c + 8 <= D) {
        const vec *at = (const vec *)(row + (int64_t)c * (BF16 ? 2 : 4));
        r.a[0] = at[0];
        if (!BF16) r.a[BF16 ? 0 : 1] = at[1];
    } else {
        uint32_t w[kVec];
#pragma unroll
        for (int e = 0; e < kVec; ++e)
            w[e] = c + e >= D ? 0u : BF16 ? (uint32_t)((const uint16_t *)row)[c + e] : ((const uint32_t *)row)[c + e];
        if (BF16) {
            r.a[0] = u32x4{w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16};
        } else {
            r.a[0] = u32x4{w[0], w[1], w[2], w[3]};
            r.a[BF16 ? 0 : 1] = u32x4{w[4], w[5], w[6], w[7]};
        }
    }
    return r;
}
template <bool BF16>
__device__ __forceinline__ void widen(const Raw<BF16> &r, float (&x)[kVec]) {
    unpack<BF16>(r.a[0], x);
    if (!BF16) unpack<BF16>(r.a[BF16 ? 0 : 1], x + 4);
}
template <bool BF16>
__device__ __forceinline__ void store_group(char *row, int c, int D, const float *x) {
    typedef typename Group<BF16>::any any;
    if (c + 4 <= D) {
        typename Group<BF16>::vec v;
        if constexpr (BF16) v = {pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
        else v = {__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
        __builtin_nontemporal_store(v, (any *)(row + (int64_t)c * (BF16 ? 2 : 4)));
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (c + e < D) {
            if (BF16) ((uint16_t *)row)[c + e] = (uint16_t)pack_bf16(x[e], 0.0f);
            else ((float *)row)[c + e] = x[e];
        }
    }
}
template <bool BF16, bool SPLIT>
__device__ __forceinline__ void store8(char *row, int c, int half, int D, const float (&x)[kVec]) {
    typedef typename Row<BF16>::vec vec;
    if (!SPLIT && c + 8 <= D) {
        vec *at = (vec *)(row + (int64_t)c * (BF16 ? 2 : 4));
        if (BF16) {
            const u32x4 a = {pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
            __builtin_nontemporal_store(a, at);
        } else {
            const u32x4 a = {__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
            const u32x4 b = {__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7])};
            __builtin_nontemporal_store(a, at);
            __builtin_nontemporal_store(b, at + 1);
        }
        return;
    }
    if (SPLIT) {
        store_group<BF16>(row, c, D, x);
        store_group<BF16>(row, c + half, D, x + 4);
        return;
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
        if (c + e < D) {
            if (BF16) ((uint16_t *)row)[c + e] = (uint16_t)pack_bf16(x[e], 0.0f);
            else ((float *)row)[c + e] = x[e];
        }
    }
}

struct EmbedParams {
    const char *table;
    int64_t table_stride_b;
    char *out;
    int64_t out_stride_b;
    const int32_t *ids;
    const uint8_t *valid;
    int32_t n, n_vocab, D;
    int32_t lanes_log2, segs;                  // lanes per token (a power of two); waves per token when that is 64
    float scale;
    int32_t *status;
};

// WIDE: a whole wave per token, so the token and its id are wave-uniform (scalar loads).
template <bool TB, bool OB, bool WIDE>
__global__ __launch_bounds__(64 * kLookWaves) void embed_kernel(EmbedParams P) {
    fetch_args(P.table, P.table_stride_b, P.out, P.out_stride_b, P.ids, P.valid, P.n, P.n_vocab, P.D, P.scale);
    constexpr bool SPLIT = !OB;
    const uint32_t unit = blockIdx.x * kLookWaves + uni(threadIdx.x >> 6);
    const int lane = lane_id(), step = WIDE ? 64 : 1 << P.lanes_log2;
    const int half = SPLIT ? step * 4 : 4;
    uint32_t t;
    int c0 = 0, lv = lane;                     // first column of the wave's part of the token; lane within it
    if (WIDE) {
        t = unit / P.segs;
        c0 = (unit - t * P.segs) * (64 * kLookVecs * kVec);
    } else {
        t = (unit << (6 - P.lanes_log2)) + (lane >> P.lanes_log2);
        lv = lane & (step - 1);
    }
    if (t >= (uint32_t)P.n) return;
    int id = P.ids[t];                         // the row to read, -1 for zeros
    if (P.valid != nullptr && P.valid[t] == 0) id = -1;
    else if (id < 0 || id >= P.n_vocab) {
        id = -1;
        set_status(P.status, DLLM_ERR_ARG);
    }
    const char *row = P.table + id * P.table_stride_b;
    char *out = P.out + t * P.out_stride_b;
    c0 += lv * (SPLIT ? 4 : kVec);
    Raw<TB> raw[kLookVecs];
#pragma unroll
    for (int i = 0; i < kLookVecs; ++i) {
        const int c = c0 + i * step * kVec;
        if (id >= 0 && c < P.D) raw[i] = load_raw<TB, SPLIT>(row, c, half, P.D);
    }
#pragma unroll
    for (int i = 0; i < kLookVecs; ++i) {
        const int c = c0 + i * step * kVec;
        if (c >= P.D) continue;
        float x[kVec];
        widen<TB>(raw[i], x);
#pragma unroll
        for (int e = 0; e < kVec; ++e) x[e] = id >= 0 ? x[e] * P.scale : 0.0f;
        store8<OB, SPLIT>(out, c, half, P.D, x);
    }
}

// ---- zeros ---------------------------------------------------------------------------------------
struct Table {
    char *p;
    int64_t stride_b;
    int32_t n_vocab, D;
    int32_t fill, fill_log2;                   // 16-byte vectors of a row (a ragged one too), also as a power of two not below it
};

// Rows a workgroup of `threads` clears: its threads lie along one row, or several narrow ones, one store
// each for rows up to 16 bytes a thread.  What counts is that the stores in flight form a dense front in
// the table.  One 16-byte store per thread in workgroups of 256 with 35 KB of LDS each, which holds four of them on
// a compute unit, clears 1.22 GB in 191 us = 6.4 TB/s (best 6.85), without that LDS in 202 = 6.0, and 0.91 GB behind
// the sort in 142 us = 6.4 (6.0 without); 1024 threads write 6.0, two stores per thread 5.9.  Non-temporal, so the
// zeros leave the last-level cache to the sums.
constexpr int rows_at_once(int threads, int fill_log2) { return (1 << fill_log2) < threads ? threads >> fill_log2 : 1; }

template <bool TB, int THREADS>
__device__ __forceinline__ void fill_rows(const Table &T, int first, int end) {
    typedef typename Row<TB>::vec vec;
    constexpr int E = TB ? 8 : 4;
    const bool narrow = (1 << T.fill_log2) < THREADS;
    const int v0 = narrow ? threadIdx.x & ((1 << T.fill_log2) - 1) : threadIdx.x;
    const int r = first + (narrow ? threadIdx.x >> T.fill_log2 : 0);
    if (r >= end) return;
    char *row = T.p + r * T.stride_b;
    const u32x4 z = {0, 0, 0, 0};
    for (int v = v0; v < T.fill; v += THREADS) {
        if ((v + 1) * E <= T.D) {
            __builtin_nontemporal_store(z, (vec *)row + v);
        } else {
            for (int d = v * E; d < T.D; ++d) {
                if (TB) ((uint16_t *)row)[d] = 0;
                else ((float *)row)[d] = 0.0f;
            }
        }
    }
}

// ---- sort ----------------------------------------------------------------------------------------
constexpr int kDigit = 9;
constexpr int kBins = 1 << kDigit;
constexpr int kSortThreads = 1024;
constexpr int kZeroThreads = 256;              // of the launch that only clears
constexpr int kMinTile = 4096;                 // a multiple of 64 items per wave
constexpr int kMaxTiles = 256;                 // a moving workgroup adds up the counts of the tiles before its own

struct SortParams {
    const int32_t *ids;                        // first pass: the ids themselves
    const uint8_t *valid;
    const uint64_t *in;                        // later passes: id << 32 | position
    uint64_t *out;
    int32_t *hist;                             // [tiles][kBins]
    int32_t *n_long;                           // cleared by the first launch
    int32_t n, n_vocab, tile, tiles, shift, bits;
    int32_t fill_first, fill_end;              // table rows to clear beside the sort
    Table table;
    int32_t *status;
};

// Tokens that add nothing sort behind every id, as n_vocab.
__device__ __forceinline__ uint64_t first_item(const SortParams &P, int i, bool report) {
    int id = P.ids[i];
    if (P.valid != nullptr && P.valid[i] == 0) id = P.n_vocab;
    else if (id < 0 || id >= P.n_vocab) {
        id = P.n_vocab;
        if (report) set_status(P.status, DLLM_ERR_ARG);
    }
    return (uint64_t)(uint32_t)id << 32 | (uint32_t)i;
}
template <bool FIRST>
__device__ __forceinline__ uint64_t sort_item(const SortParams &P, int i, bool report) {
    if (FIRST) return first_item(P, i, report);
    return P.in[i];
}
__device__ __forceinline__ int digit_of(uint64_t item, int shift) { return (int)((item >> 32) >> shift) & (kBins - 1); }

// The filling workgroups of a launch follow its `sorting` ones.
template <bool TB, int T>
__device__ __forceinline__ bool fills(const SortParams &P, int sorting) {
    if ((int)blockIdx.x < sorting) return false;
    const int first = P.fill_first + ((int)blockIdx.x - sorting) * rows_at_once(T, P.table.fill_log2);
    fill_rows<TB, T>(P.table, first, P.fill_end);
    return true;
}

template <bool FIRST, bool TB>
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortParams P) {
    constexpr int T = kSortThreads;
    __shared__ int s_count[kBins];
    if (fills<TB, T>(P, P.tiles)) return;
    const int tid = threadIdx.x, tile = blockIdx.x;
    if (FIRST && tile == 0 && tid == 0) *P.n_long = 0;
    for (int b = tid; b < kBins; b += T) s_count[b] = 0;
    __syncthreads();
    const int i0 = tile * P.tile, end = min(P.n, i0 + P.tile);
    for (int i = i0 + tid; i < end; i += T) atomicAdd(&s_count[digit_of(sort_item<FIRST>(P, i, true), P.shift)], 1);
    __syncthreads();
    for (int b = tid; b < kBins; b += T) P.hist[tile * kBins + b] = s_count[b];
}

// Zeros alone: the rows that the launches of the sort leave.
template <bool TB>
__global__ __launch_bounds__(kZeroThreads) void embed_zero_kernel(SortParams P) {
    fills<TB, kZeroThreads>(P, 0);
}

// Lanes of the wave that hold the same digit (only lanes with `on` count).
__device__ __forceinline__ uint64_t same_digit(int d, bool on) {
    uint64_t m = __ballot(on);
#pragma unroll
    for (int b = 0; b < kDigit; ++b) {
        const uint64_t set = __ballot((d >> b) & 1);
        m &= (d >> b) & 1 ? set : ~set;
    }
    return m;
}

// The counts of a workgroup's waves, and from them where each wave's next item of each digit goes.
struct Places {
    static constexpr int kWaves = kSortThreads / 64;
    int at[kWaves][kBins];
    int sum[kBins / 64];

    __device__ __forceinline__ void clear() {
        for (int b = threadIdx.x; b < kWaves * kBins; b += kSortThreads) (&at[0][0])[b] = 0;
    }
    // Each of the first kBins threads owns a digit: `total` of it in all tiles, `before` in earlier ones.
    // An item goes behind those of smaller digits, of earlier tiles and of earlier waves.
    __device__ __forceinline__ void place(int before, int total) {
        const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
        int incl = 0;
        if (tid < kBins) {
            incl = wave_incl_scan(total);
            if (lane == 63) sum[wave] = incl;
        }
        __syncthreads();
        if (tid < kBins) {
            int to = incl - total + before;
            for (int w = 0; w < wave; ++w) to += sum[w];
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const int c = at[w][tid];
                at[w][tid] = to;
                to += c;
            }
        }
        __syncthreads();
    }
    // The place of this lane's item, the wave's lanes in order.
    __device__ __forceinline__ int take(int d, bool on) {
        int *own = at[threadIdx.x >> 6];
        const uint64_t peers = same_digit(d, on);
        const int rank = __popcll(peers & ((1ull << lane_id()) - 1));
        int first = 0;
        if (on) first = __atomic_load_n(&own[d], __ATOMIC_RELAXED);
        // every lane has read its digit's place before the first lane of that digit moves it on
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (on && rank == 0) __atomic_store_n(&own[d], first + __popcll(peers), __ATOMIC_RELAXED);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        return first + rank;
    }
};

// Moves a tile's items; wave w moves consecutive ones, after those of waves < w.
template <bool FIRST, bool TB>
__global__ __launch_bounds__(kSortThreads) void sort_move_kernel(SortParams P) {
    __shared__ Places s;
    if (fills<TB, kSortThreads>(P, P.tiles)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, mine = blockIdx.x;
    s.clear();
    int before = 0, total = 0;
    if (tid < kBins) {
#pragma unroll 8
        for (int t = 0; t < P.tiles; ++t) {
            const int c = P.hist[t * kBins + tid];
            before += t < mine ? c : 0;
            total += c;
        }
    }
    __syncthreads();
    const int share = P.tile / Places::kWaves, w0 = mine * P.tile + wave * share;
    for (int i = w0 + lane; i < w0 + share; i += 64)
        if (i < P.n) atomicAdd(&s.at[wave][digit_of(sort_item<FIRST>(P, i, false), P.shift)], 1);
    __syncthreads();
    s.place(before, total);
    for (int i = w0 + lane; i - lane < w0 + share; i += 64) {
        const bool on = i < P.n;
        const uint64_t item = on ? sort_item<FIRST>(P, i, false) : 0;
        const int to = s.take(digit_of(item, P.shift), on);
        if (on) P.out[to] = item;
    }
}

// One tile: every pass in one workgroup, the items in LDS between the passes.
template <bool TB>
__global__ __launch_bounds__(kSortThreads) void sort_one_kernel(SortParams P) {
    constexpr int kHeld = kMinTile / kSortThreads;   // items per thread
    __shared__ Places s;
    __shared__ uint64_t s_item[kMinTile];
    if (fills<TB, kSortThreads>(P, 1)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int share = P.tile / Places::kWaves, w0 = wave * share;
    if (tid == 0) *P.n_long = 0;
    uint64_t item[kHeld];
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {
        const int i = w0 + h * 64 + lane;
        item[h] = 0;
        if (h * 64 < share && i < P.n) item[h] = first_item(P, i, true);
    }
    for (int shift = 0; shift < P.bits; shift += kDigit) {
        s.clear();
        __syncthreads();
        if (shift > 0) {
#pragma unroll
            for (int h = 0; h < kHeld; ++h)
                if (h * 64 < share) item[h] = s_item[w0 + h * 64 + lane];
        }
#pragma unroll
        for (int h = 0; h < kHeld; ++h)
            if (h * 64 < share && w0 + h * 64 + lane < P.n) atomicAdd(&s.at[wave][digit_of(item[h], shift)], 1);
        __syncthreads();
        int total = 0;
        if (tid < kBins) {
#pragma unroll
            for (int w = 0; w < Places::kWaves; ++w) total += s.at[w][tid];
        }
        s.place(0, total);
        const bool last = shift + kDigit >= P.bits;
#pragma unroll
        for (int h = 0; h < kHeld; ++h) {
            if (h * 64 >= share) continue;
            const bool on = w0 + h * 64 + lane < P.n;
            const int to = s.take(digit_of(item[h], shift), on);
            if (on) {
                if (last) P.out[to] = item[h];
                else s_item[to] = item[h];
            }
        }
        __syncthreads();
    }
}

// ---- sum and join ---------------------------------------------------------------------------------
// Sorted tokens per piece: many where there is work for every compute unit, few where a wave's own chain of
// loads is what takes the time: two batches of 1600 tokens of width 1000 take 51, 48, 46 us with 16, 12, 8; two of
// 8192 of width 2048 take 116, 114, 123, and 147 with 64.
constexpr int kPiece = 64, kSmallPiece = 12;
constexpr int kSumThreads = 256;
constexpr int kSumWaves = kSumThreads / 64;
constexpr int kSumCols = 64 * kVec;            // columns per wave
// Tokens whose loads are in flight together; with the table's old rows beside them, half as many.
constexpr int kAhead = 8, kAheadOld = 4;      // 2 to 16 make no difference at 64 x 544 tokens (HBM-bound)

struct SumParams {
    const char *grad;
    int64_t grad_stride_b;
    Table table;
    const uint64_t *sorted;
    float *part;                               // [pieces][2][D]: the run entering from before, the run leaving
    int32_t *n_long, *long_piece;              // pieces in which a long run starts
    int32_t n, pieces, colblocks, accumulate;
    float scale;
};

__device__ __forceinline__ int key_of(uint64_t item) { return (int)(item >> 32); }

// table row = (old +) scale * sum, rounded once.
template <bool TB>
__device__ __forceinline__ void write_row(const SumParams &P, int id, int c, const float (&a)[kVec], const float (&old)[kVec]) {
    float o[kVec];
#pragma unroll
    for (int e = 0; e < kVec; ++e) o[e] = fmaf(P.scale, a[e], old[e]);
    store8<TB, false>(P.table.p + id * P.table.stride_b, c, 4, P.table.D, o);
}

// The window of three pieces around piece [N, 2N): ids, positions, run starts as bits (a position whose id
// differs from the one before; the window's first counts) and counts of tokens with an id.
template <int N>                               // up to 21 tokens: the window in one register, lanes 0 .. 3N-1
struct Window {
    int k, p;
    __device__ __forceinline__ void load(const uint64_t *sorted, int64_t first, int n, uint64_t none) {
        const int64_t i = first - N + lane_id();
        const uint64_t w = i >= 0 && i < n && lane_id() < 3 * N ? sorted[i] : none;
        k = (int)(w >> 32), p = (int)(uint32_t)w;
    }
    __device__ __forceinline__ void starts(uint64_t &s0, uint64_t &s1, uint64_t &s2) const {
        constexpr uint64_t kPart = (1ull << N) - 1;
        const int below = up_one(k);
        const uint64_t s = __ballot(lane_id() == 0 || k != below);
        s0 = s & kPart, s1 = (s >> N) & kPart, s2 = (s >> (2 * N)) & kPart;
    }
    __device__ __forceinline__ void counts(int none, int &c1, int &c2) const {
        constexpr uint64_t kPart = (1ull << N) - 1;
        const uint64_t on = __ballot(k != none);
        c1 = __popcll((on >> N) & kPart), c2 = __popcll((on >> (2 * N)) & kPart);
    }
    __device__ __forceinline__ int key(int t) const { return __builtin_amdgcn_readlane(k, t); }
    __device__ __forceinline__ int pos(int t) const { return __builtin_amdgcn_readlane(p, t); }
};
template <>
struct Window<64> {
    int k0, k1, k2, p1, p2;
    __device__ __forceinline__ void load(const uint64_t *sorted, int64_t first, int n, uint64_t none) {
        const int64_t i = first + lane_id();
        const uint64_t w0 = i >= 64 ? sorted[i - 64] : none, w1 = i < n ? sorted[i] : none,
                       w2 = i + 64 < n ? sorted[i + 64] : none;
        k0 = (int)(w0 >> 32), k1 = (int)(w1 >> 32), k2 = (int)(w2 >> 32), p1 = (int)(uint32_t)w1, p2 = (int)(uint32_t)w2;
    }
    __device__ __forceinline__ void starts(uint64_t &s0, uint64_t &s1, uint64_t &s2) const {
        const int lane = lane_id(), b0 = up_one(k0), b1 = up_one(k1), b2 = up_one(k2);
        s0 = __ballot(lane == 0 || k0 != b0);
        s1 = __ballot(k1 != (lane == 0 ? __builtin_amdgcn_readlane(k0, 63) : b1));
        s2 = __ballot(k2 != (lane == 0 ? __builtin_amdgcn_readlane(k1, 63) : b2));
    }
    __device__ __forceinline__ void counts(int none, int &c1, int &c2) const {
        c1 = __popcll(__ballot(k1 != none));
        c2 = __popcll(__ballot(k2 != none));
    }
    __device__ __forceinline__ int key(int t) const {
        return t < 128 ? __builtin_amdgcn_readlane(k1, t - 64) : __builtin_amdgcn_readlane(k2, t - 128);
    }
    __device__ __forceinline__ int pos(int t) const {
        return t < 128 ? __builtin_amdgcn_readlane(p1, t - 64) : __builtin_amdgcn_readlane(p2, t - 128);
    }
};
// One wave: piece `piece`, columns colblock*512 ...
template <bool GB, bool TB, int N, bool OLD>
__device__ void sum_piece(const SumParams &P, int piece, int colblock) {
    constexpr int kStep = OLD ? kAheadOld : kAhead;
    const int D = P.table.D, none = P.table.n_vocab;               // `none`: tokens that add nothing, last
    Window<N> w;
    w.load(P.sorted, (int64_t)piece * N, P.n, (uint64_t)none << 32);
    uint64_t s0, s1, s2;
    int c1, c2;
    w.starts(s0, s1, s2);
    w.counts(none, c1, c2);
    if (c1 == 0) return;
    // first start at or after window position i >= N (3N: none in the window)
    auto next_start = [&](int i) {
        if (i < 2 * N) {
            const uint64_t m = s1 & (~0ull << (i - N));
            if (m != 0) return N + (int)__builtin_ctzll(m);
            i = 2 * N;
        }
        const uint64_t m = i < 3 * N ? s2 & (~0ull << (i - 2 * N)) : 0ull;
        return m != 0 ? 2 * N + (int)__builtin_ctzll(m) : 3 * N;
    };
    int begin = N, end;
    // the run that enters from the piece before: its part here if it is long, nothing otherwise
    int head_end = 0;                          // > 0: tokens [N, head_end) go to partial sum 0
    if (!(s1 & 1)) {
        const int lo = 63 - (int)__builtin_clzll(s0), hi = next_start(N + 1);
        if (hi - lo > N) head_end = min(hi, 2 * N);
        else begin = hi;
    }
    // the last run that starts here: to its end, or to the piece's end and into partial sum 1 if it is long
    int tail = 3 * N;                          // < 3N: where a long run starts
    if (c1 < N) {
        end = N + c1;
    } else if (s1 != 0) {
        const int last = N + 63 - (int)__builtin_clzll(s1), hi = next_start(last + 1);
        end = min(hi, 2 * N + c2);
        if (hi - last > N) {
            tail = last;
            end = 2 * N;
        }
    } else {
        end = 2 * N;                           // one long run covers the piece
    }
    if (begin >= end) return;
    if (tail < 3 * N && colblock == 0 && lane_id() == 0) P.long_piece[atomicAdd(P.n_long, 1)] = piece;

    // lanes past the last column keep running (their registers are read across the wave) on its vector
    const int own = colblock * kSumCols + lane_id() * kVec;
    const bool live = own < D;
    const int c = min(own, (D - 1) / kVec * kVec);
    auto ends_run = [&](int t) { return t + 1 == end || next_start(t + 1) == t + 1; };
    auto to_row = [&](int t) { return t + 1 != head_end && t < tail; };
    float a[kVec];
#pragma unroll
    for (int e = 0; e < kVec; ++e) a[e] = 0.0f;
    for (int t0 = begin; t0 < end; t0 += kStep) {
        Raw<GB> raw[kStep];
        Raw<TB> old[kStep];
#pragma unroll
        for (int u = 0; u < kStep; ++u) {
            const int t = t0 + u;
            if (t < end) {
                raw[u] = load_raw<GB, false>(P.grad + w.pos(t) * P.grad_stride_b, c, 4, D);
                if (OLD && ends_run(t) && to_row(t)) old[u] = load_raw<TB, false>(P.table.p + w.key(t) * P.table.stride_b, c, 4, D);
            }
        }
#pragma unroll
        for (int u = 0; u < kStep; ++u) {
            const int t = t0 + u;
            if (t >= end) break;
            float x[kVec];
            widen<GB>(raw[u], x);
#pragma unroll
            for (int e = 0; e < kVec; ++e) a[e] += x[e];
            if (!ends_run(t)) continue;
            if (to_row(t)) {
                float o[kVec];
#pragma unroll
                for (int e = 0; e < kVec; ++e) o[e] = 0.0f;
                if (OLD) widen<TB>(old[u], o);
                const int id = w.key(t);
                if (live) write_row<TB>(P, id, c, a, o);
            } else {
                float *part = P.part + ((int64_t)piece * 2 + (t + 1 == head_end ? 0 : 1)) * D;
#pragma unroll
                for (int e = 0; e < kVec; ++e)
                    if (live && c + e < D) part[c + e] = a[e];
            }
#pragma unroll
            for (int e = 0; e < kVec; ++e) a[e] = 0.0f;
        }
    }
}

template <bool GB, bool TB, int N, bool OLD>
__global__ __launch_bounds__(kSumThreads) void embed_sum_kernel(SumParams P) {
    const int unit = (int)blockIdx.x * kSumWaves + uni(threadIdx.x >> 6);
    if (unit < P.pieces * P.colblocks) sum_piece<GB, TB, N, OLD>(P, uni(unit / P.colblocks), uni(unit % P.colblocks));
}

// The partial sums of each long run: 16 threads side by side on 4 columns each, 16 slices of pieces.
constexpr int kJoinCols = 64, kJoinSlices = 16;

constexpr int kJoinRuns = 16;                  // long runs side by side

template <bool TB, int N>
__global__ __launch_bounds__(256) void embed_join_kernel(SumParams P) {
    __shared__ float s_sum[kJoinSlices][kJoinCols];
    __shared__ int s_more[4];
    const int tid = threadIdx.x, slice = tid >> 4, c = (tid & 15) * 4, D = P.table.D;
    const int col = blockIdx.x * kJoinCols + c;
    const int n_long = *P.n_long;
    for (int l = blockIdx.y; l < n_long; l += gridDim.y) {
        const int p0 = P.long_piece[l];
        const int key = key_of(P.sorted[(int64_t)p0 * N + N - 1]);
        // the pieces after p0 that start with the run's id, 256 at a time
        int count = 1;
        while (true) {
            const int64_t i = ((int64_t)p0 + count + tid) * N;
            const uint64_t in = __ballot(i < P.n && key_of(P.sorted[i]) == key);
            if ((tid & 63) == 0) s_more[tid >> 6] = __popcll(in);
            __syncthreads();
            const int more = s_more[0] + s_more[1] + s_more[2] + s_more[3];
            __syncthreads();
            count += more;
            if (more < 256) break;
        }
        const int per = (count + kJoinSlices - 1) / kJoinSlices;
        float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
        for (int p = slice * per; p < min((slice + 1) * per, count); ++p) {
            const float *part = P.part + ((int64_t)(p0 + p) * 2 + (p == 0 ? 1 : 0)) * D + col;
            if (col + 4 <= D) {
                const u32x4 x = *(const Row<false>::vec *)part;
#pragma unroll
                for (int e = 0; e < 4; ++e) a[e] += __uint_as_float(x[e]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (col + e < D) a[e] += part[e];
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s_sum[slice][c + e] = a[e];
        __syncthreads();
        if (tid < kJoinCols / kVec) {
            const int c8 = blockIdx.x * kJoinCols + tid * kVec;
            float t[kVec];
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                t[e] = 0.0f;
                for (int s = 0; s < kJoinSlices; ++s) t[e] += s_sum[s][tid * kVec + e];
            }
            if (c8 < D) {
                float o[kVec];
#pragma unroll
                for (int e = 0; e < kVec; ++e) o[e] = 0.0f;
                if (P.accumulate) widen<TB>(load_raw<TB, false>(P.table.p + key * P.table.stride_b, c8, 4, D), o);
                write_row<TB>(P, key, c8, t, o);
            }
        }
        __syncthreads();
    }
}

// ---- host -----------------------------------------------------------------------------------------
constexpr int64_t kSmallUnits = 2048;
// Bytes of zeros that a launch of the sort hides: one of several, and a single one by its tokens.  Its 1024
// threads write 6.0 TB/s, the zeros' own launch 6.4 (and what the last-level cache takes in of a smaller table), at
// 2.5 us for the launch: 52 MiB left over gain nothing, 97 a microsecond.  All beside the sort against this rule: 518 MB and 160 tokens 102 us and 85, 4096 tokens 104
// and 94; 623 MB and 8192 tokens 137 and 128; 131 MB and 160 tokens 32.1 and 31.0.  Of several launches, each
// hiding 32, 64, 96, 128 MiB takes 131, 127, 129, 134 us there, and 297, 287, 285, 288 for 1.25 GB and 34816 tokens.
constexpr int64_t kBesideLaunch = 80 << 20, kBesideOne = 24 << 20, kBesideToken = 24 << 10;
constexpr int64_t kApart = 80 << 20;           // zeros beyond those that are worth a launch of their own
constexpr size_t kZeroFront = 35 << 10;        // LDS that holds four of its workgroups on a compute unit; 518 MB: 85 us, 90 without

struct GradSpace {
    size_t a, b, hist, n_long, long_piece, part, bytes;
    int tile, tiles, piece, pieces;
};
GradSpace grad_space(int64_t n, int64_t D) {
    GradSpace w{};
    // whole rounds of 64 items for each wave of the wider sort
    w.tile = (int)std::max<int64_t>(kSortThreads, std::min<int64_t>(kMinTile, (n + kSortThreads - 1) / kSortThreads * kSortThreads));
    while ((n + w.tile - 1) / w.tile > kMaxTiles) w.tile *= 2;
    w.tiles = (int)((n + w.tile - 1) / w.tile);
    // Fewer than kSmallUnits waves at kPiece tokens leave compute units idle while each wave works through
    // its tokens: shorter pieces then (a limit of 512 costs 16384 tokens of width 1024 10 us, one of 8192
    // costs 163840 of width 64 20 us).
    const int64_t units = (n + kPiece - 1) / kPiece * ((D + kSumCols - 1) / kSumCols);
    w.piece = units < kSmallUnits ? kSmallPiece : kPiece;
    w.pieces = (int)((n + w.piece - 1) / w.piece);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) & ~(size_t)255;
        return here;
    };
    w.a = take((size_t)n * 8);
    w.b = take((size_t)n * 8);
    w.hist = take((size_t)kBins * w.tiles * 4);
    w.n_long = take(4);
    w.long_piece = take((size_t)w.pieces * 4);
    w.part = take((size_t)w.pieces * 2 * (size_t)D * 4);
    w.bytes = at;
    return w;
}

// What serves any box of up to n tokens.  A layout's size grows with its tokens but where their pieces get longer
// and where a sort tile doubles (fewer counts), so those before each fall count too.
size_t space_up_to(int64_t n, int64_t D) {
    size_t bytes = grad_space(n, D).bytes;
    const int64_t short_pieces = (kSmallUnits - 1) / ((D + kSumCols - 1) / kSumCols) * kPiece;
    if (n > short_pieces) bytes = std::max(bytes, grad_space(short_pieces, D).bytes);
    for (int64_t full = (int64_t)kMaxTiles * kMinTile; full < n; full *= 2) bytes = std::max(bytes, grad_space(full, D).bytes);
    return bytes;
}

bool sizes_ok(int32_t n_tokens, int32_t n_vocab, int32_t D) {
    return n_tokens >= 0 && n_tokens <= DLLM_MAX_TOKENS && n_vocab >= 1 && n_vocab <= DLLM_MAX_VOCAB && D >= 1 && D <= DLLM_MAX_WIDTH;
}
dllm_status check_sizes(const char *who, int32_t n_tokens, int32_t n_vocab, int32_t D, int32_t dt_a, int32_t dt_b,
                        int64_t stride_a, int64_t stride_b) {
    if ((dt_a != DLLM_FP32 && dt_a != DLLM_BF16) || (dt_b != DLLM_FP32 && dt_b != DLLM_BF16))
        return fail(DLLM_ERR_DTYPE, "%s: unknown dtype %d or %d", who, (int)dt_a, (int)dt_b);
    if (n_tokens < 0) return fail(DLLM_ERR_ARG, "%s: n_tokens < 0", who);
    if (!sizes_ok(n_tokens, n_vocab, D))
        return fail(DLLM_ERR_SHAPE, "%s: n_tokens=%d, n_vocab=%d, D=%d outside the limits", who, n_tokens, n_vocab, D);
    if (stride_a < D || stride_b < D)
        return fail(DLLM_ERR_ARG, "%s: strides %lld, %lld smaller than D=%d", who, (long long)stride_a, (long long)stride_b, D);
    return DLLM_OK;
}
int vectors_of(int32_t D) { return (D + kVec - 1) / kVec; }
// log2 of the smallest power of two not below n
int log2_up(int n) {
    int l = 0;
    while ((1 << l) < n) ++l;
    return l;
}
bool misaligned(const void *p, int32_t dtype) { return ((uintptr_t)p & (dtype == DLLM_BF16 ? 1 : 3)) != 0; }
bool overlap(const void *a, size_t na, const void *b, size_t nb) {
    return (uintptr_t)a < (uintptr_t)b + nb && (uintptr_t)b < (uintptr_t)a + na;
}

}  // namespace

extern "C" dllm_status dllm_embed(void *stream, const void *table, int32_t table_dtype, int64_t table_stride,
                                  int32_t n_vocab, int32_t D, const int32_t *ids, const uint8_t *valid, int32_t n_tokens,
                                  float scale, void *out, int32_t out_dtype, int64_t out_stride, int32_t *status) {
    const char *who = "dllm_embed";
    dllm_status rc = check_sizes(who, n_tokens, n_vocab, D, table_dtype, out_dtype, table_stride, out_stride);
    if (rc != DLLM_OK || n_tokens == 0) return rc;
    if (!table || !ids || !out || !status) return fail(DLLM_ERR_ARG, "%s: null required pointer", who);
    if (misaligned(table, table_dtype) || misaligned(out, out_dtype))
        return fail(DLLM_ERR_ARG, "%s: table or out not aligned to its type", who);
    EmbedParams P{};
    const int ts = table_dtype == DLLM_BF16 ? 2 : 4, os = out_dtype == DLLM_BF16 ? 2 : 4;
    const size_t tb = ((size_t)(n_vocab - 1) * table_stride + D) * ts, ob = ((size_t)(n_tokens - 1) * out_stride + D) * os;
    if (overlap(out, ob, table, tb) || overlap(out, ob, ids, (size_t)n_tokens * 4) || (valid && overlap(out, ob, valid, n_tokens)))
        return fail(DLLM_ERR_ARG, "%s: out overlaps an input", who);
    P.table = (const char *)table;
    P.table_stride_b = table_stride * ts;
    P.out = (char *)out;
    P.out_stride_b = out_stride * os;
    P.ids = ids; P.valid = valid;
    P.n = n_tokens; P.n_vocab = n_vocab; P.D = D;
    P.scale = scale;
    P.status = status;
    const int nv = vectors_of(D);
    P.lanes_log2 = std::min(log2_up(nv), 6);
    P.segs = (nv + 64 * kLookVecs - 1) / (64 * kLookVecs);
    const bool wide = P.lanes_log2 == 6;
    const int per = 64 >> P.lanes_log2;
    const int64_t units = wide ? (int64_t)n_tokens * P.segs : ((int64_t)n_tokens + per - 1) / per;
    const int64_t blocks = (units + kLookWaves - 1) / kLookWaves;
    if (!launchable(blocks, 64 * kLookWaves)) return fail(DLLM_ERR_SHAPE, "%s: n_tokens * D too large", who);
    const hipStream_t st = (hipStream_t)stream;
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(64 * kLookWaves), 0, st, P); };
    if (table_dtype == DLLM_BF16) {
        if (out_dtype == DLLM_BF16) wide ? go(embed_kernel<true, true, true>) : go(embed_kernel<true, true, false>);
        else wide ? go(embed_kernel<true, false, true>) : go(embed_kernel<true, false, false>);
    } else {
        if (out_dtype == DLLM_BF16) wide ? go(embed_kernel<false, true, true>) : go(embed_kernel<false, true, false>);
        else wide ? go(embed_kernel<false, false, true>) : go(embed_kernel<false, false, false>);
    }
    return check_hip(hipGetLastError(), "dllm_embed launch");
}

extern "C" size_t dllm_embed_grad_workspace_bytes(int32_t n_tokens, int32_t n_vocab, int32_t D) {
    if (!sizes_ok(n_tokens, n_vocab, D)) return 0;
    return space_up_to(n_tokens, D);
}

extern "C" dllm_status dllm_embed_grad(void *stream, const void *grad_out, int32_t grad_dtype, int64_t grad_stride,
                                       const int32_t *ids, const uint8_t *valid, int32_t n_tokens, float scale,
                                       int32_t n_vocab, int32_t D, void *grad_table, int32_t table_dtype,
                                       int64_t table_stride, int32_t accumulate, void *workspace, size_t workspace_bytes,
                                       int32_t *status) {
    const char *who = "dllm_embed_grad";
    dllm_status rc = check_sizes(who, n_tokens, n_vocab, D, grad_dtype, table_dtype, grad_stride, table_stride);
    if (rc != DLLM_OK || (n_tokens == 0 && accumulate)) return rc;
    if (!grad_table || !status || (n_tokens > 0 && (!grad_out || !ids)))
        return fail(DLLM_ERR_ARG, "%s: null required pointer", who);
    if (misaligned(grad_out, grad_dtype) || misaligned(grad_table, table_dtype))
        return fail(DLLM_ERR_ARG, "%s: grad_out or grad_table not aligned to its type", who);
    const int gs = grad_dtype == DLLM_BF16 ? 2 : 4, ts = table_dtype == DLLM_BF16 ? 2 : 4;
    const GradSpace w = grad_space(n_tokens, D);
    if (w.bytes > 0 && !workspace) return fail(DLLM_ERR_ARG, "%s: null workspace", who);
    if (workspace_bytes < w.bytes)
        return fail(DLLM_ERR_ARG, "%s: workspace %zu bytes < %zu needed", who, workspace_bytes, w.bytes);
    if (((uintptr_t)workspace & 255) != 0) return fail(DLLM_ERR_ARG, "%s: workspace not 256-byte aligned", who);
    const size_t tbytes = ((size_t)(n_vocab - 1) * table_stride + D) * ts;
    const size_t gbytes = n_tokens ? ((size_t)(n_tokens - 1) * grad_stride + D) * gs : 0;
    if (overlap(grad_table, tbytes, grad_out, gbytes) || overlap(grad_table, tbytes, ids, (size_t)n_tokens * 4) ||
        (valid && overlap(grad_table, tbytes, valid, n_tokens)) || overlap(grad_table, tbytes, workspace, w.bytes) ||
        overlap(workspace, w.bytes, grad_out, gbytes) || overlap(workspace, w.bytes, ids, (size_t)n_tokens * 4) ||
        (valid && overlap(workspace, w.bytes, valid, n_tokens)))
        return fail(DLLM_ERR_ARG, "%s: grad_table or workspace overlaps another buffer", who);
    char *ws = (char *)workspace;
    const hipStream_t st = (hipStream_t)stream;

    const int fill = (D * ts + 15) / 16;
    const Table table = {(char *)grad_table, table_stride * ts, n_vocab, D, fill, log2_up(fill)};
    const bool tb = table_dtype == DLLM_BF16, gb = grad_dtype == DLLM_BF16, old = accumulate != 0;
    SortParams S{};
    S.ids = ids; S.valid = valid;
    S.hist = (int32_t *)(ws + w.hist);
    S.n_long = (int32_t *)(ws + w.n_long);
    S.n = n_tokens; S.n_vocab = n_vocab; S.tile = w.tile; S.tiles = w.tiles;
    S.table = table;
    S.status = status;
    uint64_t *from = (uint64_t *)(ws + w.a), *to = (uint64_t *)(ws + w.b);
    S.bits = 1;                                // ids 0 .. n_vocab, n_vocab itself standing for no id
    while (n_vocab >> S.bits) ++S.bits;
    const int passes = (S.bits + kDigit - 1) / kDigit;
    // Each launch of the sort clears an even share of the table's rows, or of those that it hides.
    const bool one = w.tiles <= 1;
    const int launches = one ? 1 : 2 * passes;
    const int64_t zeros = old ? 0 : (int64_t)n_vocab * D * ts;
    const int64_t beside = one ? kBesideOne + n_tokens * kBesideToken : launches * kBesideLaunch;
    const bool apart = zeros >= beside + kApart;
    const int sort_rows = old ? 0 : apart ? (int)(n_vocab * beside / zeros) : n_vocab;
    auto launch = [&](auto kernel, int threads, int sorting, int rows_end, size_t front) {
        const int at_once = rows_at_once(threads, table.fill_log2);
        S.fill_first = S.fill_end;
        S.fill_end = rows_end;
        const int blocks = sorting + (S.fill_end - S.fill_first + at_once - 1) / at_once;
        hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3((unsigned)threads), front, st, S);
    };
    int launched = 0;
    auto sort_step = [&](auto kernel, int sorting) {
        launch(kernel, kSortThreads, sorting, (int)((int64_t)sort_rows * ++launched / launches), 0);
    };
    auto sort = [&](auto bf16) {
        constexpr bool B = decltype(bf16)::value;
        if (one) {
            S.out = to;
            sort_step(sort_one_kernel<B>, 1);
            std::swap(from, to);
        }
        for (int pass = 0; pass < passes && !one; ++pass) {
            S.shift = pass * kDigit;
            S.in = from;
            S.out = to;
            if (pass == 0) {
                sort_step(sort_count_kernel<true, B>, w.tiles);
                sort_step(sort_move_kernel<true, B>, w.tiles);
            } else {
                sort_step(sort_count_kernel<false, B>, w.tiles);
                sort_step(sort_move_kernel<false, B>, w.tiles);
            }
            std::swap(from, to);
        }
        if (apart) launch(embed_zero_kernel<B>, kZeroThreads, 0, n_vocab, kZeroFront);
    };
    tb ? sort(std::true_type()) : sort(std::false_type());
    rc = check_hip(hipGetLastError(), "dllm_embed_grad sort launch");
    if (rc != DLLM_OK || n_tokens == 0) return rc;

    SumParams Q{};
    Q.grad = (const char *)grad_out;
    Q.grad_stride_b = grad_stride * gs;
    Q.table = table;
    Q.sorted = from;
    Q.part = (float *)(ws + w.part);
    Q.n_long = S.n_long;
    Q.long_piece = (int32_t *)(ws + w.long_piece);
    Q.n = n_tokens;
    Q.pieces = w.pieces;
    Q.colblocks = (D + kSumCols - 1) / kSumCols;
    Q.accumulate = old;
    Q.scale = scale;
    const int blocks = (int)(((int64_t)Q.pieces * Q.colblocks + kSumWaves - 1) / kSumWaves);
    auto sum = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(kSumThreads), 0, st, Q); };
    auto sum_of = [&](auto piece, auto with_old) {
        constexpr int N = decltype(piece)::value;
        constexpr bool O = decltype(with_old)::value;
        if (gb) tb ? sum(embed_sum_kernel<true, true, N, O>) : sum(embed_sum_kernel<true, false, N, O>);
        else tb ? sum(embed_sum_kernel<false, true, N, O>) : sum(embed_sum_kernel<false, false, N, O>);
    };
    typedef std::integral_constant<int, kPiece> Long;
    typedef std::integral_constant<int, kSmallPiece> Short;
    const bool small = w.piece == kSmallPiece;
    if (old) small ? sum_of(Short(), std::true_type()) : sum_of(Long(), std::true_type());
    else small ? sum_of(Short(), std::false_type()) : sum_of(Long(), std::false_type());
    rc = check_hip(hipGetLastError(), "dllm_embed_grad sum launch");
    if (rc != DLLM_OK || n_tokens <= w.piece) return rc;     // no run longer than a piece
    const dim3 jg((unsigned)((D + kJoinCols - 1) / kJoinCols), kJoinRuns);
    auto join = [&](auto kernel) { hipLaunchKernelGGL(kernel, jg, dim3(256), 0, st, Q); };
    if (small) tb ? join(embed_join_kernel<true, kSmallPiece>) : join(embed_join_kernel<false, kSmallPiece>);
    else tb ? join(embed_join_kernel<true, kPiece>) : join(embed_join_kernel<false, kPiece>);
    return check_hip(hipGetLastError(), "dllm_embed_grad join launch");
}
