// dllm_embed: the packed box's token ids to scaled embedding rows; dllm_embed_grad: the table's
// gradient.
//
// [BlockServe] = page "BlockServe: 块粒度连续批处理实现高吞吐扩散大语言模型服务" §II-E 逻辑位置对齐:
// the box is a dense left-padded tensor, which the forward embeds; padding contributes nothing.
//
//   out[n] = scale * table[ids[n]];     grad_table[v] (+)= scale * sum over tokens n of v of grad_out[n].
//
// Lookup (gfx950): a gather bound by HBM writes (and reads of the distinct rows).  The lanes of a
// workgroup lie along the width, 8 elements each; the ids of kTokens tokens per thread load first,
// then all their rows, then all stores.
//
// Gradient: the tokens are sorted by id (stable, so a row's terms are summed in token order and the
// bits never depend on timing; no float atomics), then every run of equal ids is summed once and
// written once.
//   1. Sort: least-significant-digit radix sort of (id, position), kDigit bits a pass, as few passes as
//      the vocabulary's bits need.  A pass counts digits per tile, then moves the items; a wave finds
//      an item's rank among equal digits by one ballot per digit bit.  One tile: all passes in one
//      launch.  The sort keeps few compute units busy for some microseconds a launch, so each of its
//      launches also writes zeros to a share of the table (kFillBytes).
//   2. Sum: one wave per piece of kPiece sorted tokens and 512 columns.  It loads kAhead tokens at a time
//      whatever run they belong to (most runs are a token or two), adds them in order, and writes a
//      row where a run ends.  A piece sums the runs that start in it, following the last one past its
//      end, so runs up to kPiece tokens are never split.  A longer run (the mask token of a training
//      box can hold half of all tokens) leaves one partial sum per piece it covers.  Other workgroups of
//      the same launch write the remaining zeros, of ids that do not occur.
//   3. Join: the partial sums of each long run, in order.
#include <algorithm>

#include "elem_common.h"

namespace {

using namespace dllm;

constexpr int kVec = 8;                        // elements per thread
constexpr int kEmbedThreads = 256;
constexpr int kTokens = 4;                     // tokens per thread, their loads in flight together

// Elements [v*8, v*8 + 8) of a row of D: as stored, to keep several in flight, and widened.  Only a row's
// ragged end is read element by element.
template <bool BF16>
struct Raw {
    u32x4 a[BF16 ? 1 : 2];
};
template <bool BF16>
__device__ __forceinline__ Raw<BF16> load_raw(const char *row, int v, int D) {
    typedef typename Row<BF16>::vec vec;
    Raw<BF16> r;
    if ((v + 1) * kVec <= D) {
        if (BF16) {
            r.a[0] = ((const vec *)row)[v];
        } else {
            r.a[0] = ((const vec *)row)[2 * v];
            r.a[BF16 ? 0 : 1] = ((const vec *)row)[2 * v + 1];
        }
    } else {
        uint32_t w[kVec];
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            const int d = v * kVec + e;
            w[e] = d >= D ? 0u : BF16 ? (uint32_t)((const uint16_t *)row)[d] : ((const uint32_t *)row)[d];
        }
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
__device__ __forceinline__ void store8(char *row, int v, int D, const float (&x)[kVec]) {
    typedef typename Row<BF16>::vec vec;
    if ((v + 1) * kVec <= D) {
        if (BF16) {
            const u32x4 a = {pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
            __builtin_nontemporal_store(a, (vec *)row + v);
        } else {
            const u32x4 a = {__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
            const u32x4 b = {__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7])};
            __builtin_nontemporal_store(a, (vec *)row + 2 * v);
            __builtin_nontemporal_store(b, (vec *)row + 2 * v + 1);
        }
    } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            const int d = v * kVec + e;
            if (d < D) {
                if (BF16) ((uint16_t *)row)[d] = (uint16_t)pack_bf16(x[e], 0.0f);
                else ((float *)row)[d] = x[e];
            }
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
    int32_t n, n_vocab, D, lanes_log2;         // a token's lanes: a power of two
    float scale;
    int32_t *status;
};

template <bool TB, bool OB>
__global__ __launch_bounds__(kEmbedThreads) void embed_kernel(EmbedParams P) {
    fetch_args(P.table, P.table_stride_b, P.out, P.out_stride_b, P.ids, P.valid, P.n, P.n_vocab, P.D, P.scale);
    const int sub = threadIdx.x >> P.lanes_log2, lv = threadIdx.x & ((1 << P.lanes_log2) - 1);
    const int per = kEmbedThreads >> P.lanes_log2;
    const int nv = (P.D + kVec - 1) / kVec;
    int id[kTokens];                           // the row to read, -1 for zeros
    int tok[kTokens];
#pragma unroll
    for (int u = 0; u < kTokens; ++u) {
        const int64_t t = ((int64_t)blockIdx.x * kTokens + u) * per + sub;
        tok[u] = t < P.n ? (int)t : -1;
        id[u] = -1;
        if (tok[u] >= 0) {
            id[u] = P.ids[t];
            if (P.valid != nullptr && P.valid[t] == 0) id[u] = -1;
            else if (id[u] < 0 || id[u] >= P.n_vocab) {
                id[u] = -1;
                if (lv == 0) set_status(P.status, DLLM_ERR_ARG);
            }
        }
    }
    for (int v = lv; v < nv; v += 1 << P.lanes_log2) {
        Raw<TB> raw[kTokens];
#pragma unroll
        for (int u = 0; u < kTokens; ++u)
            if (id[u] >= 0) raw[u] = load_raw<TB>(P.table + id[u] * P.table_stride_b, v, P.D);
#pragma unroll
        for (int u = 0; u < kTokens; ++u) {
            if (tok[u] < 0) continue;
            float x[kVec];
            widen<TB>(raw[u], x);
#pragma unroll
            for (int e = 0; e < kVec; ++e) x[e] = id[u] >= 0 ? x[e] * P.scale : 0.0f;
            store8<OB>(P.out + tok[u] * P.out_stride_b, v, P.D, x);
        }
    }
}

// ---- zeros ---------------------------------------------------------------------------------------
constexpr int kFillRows = 64;                  // table rows a filling workgroup looks at
// Bytes of zeros each launch of the sort writes beside it: what the card writes in about 6 us, as long
// as such a launch takes.
constexpr int64_t kFillBytes = 40 << 20;

struct Table {
    char *p;
    int64_t stride_b;
    int32_t n_vocab, D, lanes_log2;            // a row's lanes: a power of two
};

// Rows v0 .. v0 + kFillRows - 1 whose bit is set in `rows`, by a workgroup of THREADS.
template <bool TB, int THREADS>
__device__ __forceinline__ void fill_rows(const Table &T, int v0, uint64_t rows) {
    const int nv = (T.D + kVec - 1) / kVec, lv = threadIdx.x & ((1 << T.lanes_log2) - 1);
    const float z[kVec] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    for (int r = threadIdx.x >> T.lanes_log2; r < kFillRows; r += THREADS >> T.lanes_log2) {
        if (!((rows >> r) & 1)) continue;
        char *row = T.p + (int64_t)(v0 + r) * T.stride_b;
        for (int v = lv; v < nv; v += 1 << T.lanes_log2) store8<TB>(row, v, T.D, z);
    }
}

// ---- sort ----------------------------------------------------------------------------------------
constexpr int kDigit = 9;
constexpr int kBins = 1 << kDigit;
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kMinTile = 4096;                 // a multiple of kSortThreads
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
__device__ __forceinline__ uint64_t sort_item(const SortParams &P, const uint64_t *in, int i, bool report) {
    if (FIRST) return first_item(P, i, report);
    return in[i];
}
__device__ __forceinline__ int digit_of(uint64_t item, int shift) { return (int)((item >> 32) >> shift) & (kBins - 1); }

// The filling workgroups of a sort launch follow its `sorting` ones.
template <bool TB>
__device__ __forceinline__ bool fills(const SortParams &P, int sorting) {
    if ((int)blockIdx.x < sorting) return false;
    const int v0 = P.fill_first + ((int)blockIdx.x - sorting) * kFillRows, n = min(kFillRows, P.fill_end - v0);
    fill_rows<TB, kSortThreads>(P.table, v0, n >= 64 ? ~0ull : (1ull << n) - 1);
    return true;
}

template <bool FIRST, bool TB>
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortParams P) {
    __shared__ int s_count[kBins];
    if (fills<TB>(P, P.tiles)) return;
    const int tid = threadIdx.x, tile = blockIdx.x;
    if (FIRST && tile == 0 && tid == 0) *P.n_long = 0;
    if (tid < kBins) s_count[tid] = 0;
    __syncthreads();
    const int i0 = tile * P.tile, end = min(P.n, i0 + P.tile);
    for (int i = i0 + tid; i < end; i += kSortThreads) atomicAdd(&s_count[digit_of(sort_item<FIRST>(P, P.in, i, true), P.shift)], 1);
    __syncthreads();
    if (tid < kBins) P.hist[tile * kBins + tid] = s_count[tid];
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

// Moves items [i0, i0 + tile) of one pass: `before` is the number of items of digit threadIdx.x in
// earlier tiles, `total` in all tiles.  Wave w moves consecutive items, after those of waves < w.
template <bool FIRST>
__device__ __forceinline__ void move_tile(const SortParams &P, const uint64_t *in, uint64_t *out, int i0, int tile, int shift,
                                          int before, int total, int (&s_at)[kSortWaves][kBins],
                                          int (&s_wave)[kBins / 64]) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int b = tid; b < kSortWaves * kBins; b += kSortThreads) (&s_at[0][0])[b] = 0;
    __syncthreads();
    const int share = tile / kSortWaves, w0 = i0 + wave * share;
    for (int i = w0 + lane; i < w0 + share; i += 64)
        if (i < P.n) atomicAdd(&s_at[wave][digit_of(sort_item<FIRST>(P, in, i, false), shift)], 1);
    // where each digit starts in the output: the totals of the digits below it
    int incl = 0;
    if (tid < kBins) {
        incl = wave_incl_scan(total);
        if (lane == 63) s_wave[wave] = incl;
    }
    __syncthreads();
    if (tid < kBins) {
        int at = incl - total + before;
        for (int w = 0; w < wave; ++w) at += s_wave[w];
        for (int w = 0; w < kSortWaves; ++w) {
            const int c = s_at[w][tid];
            s_at[w][tid] = at;
            at += c;
        }
    }
    __syncthreads();
    for (int i = w0 + lane; i - lane < w0 + share; i += 64) {
        const bool on = i < P.n;
        const uint64_t item = on ? sort_item<FIRST>(P, in, i, false) : 0;
        const int d = digit_of(item, shift);
        const uint64_t peers = same_digit(d, on);
        const int rank = __popcll(peers & ((1ull << lane) - 1));
        int at = 0;
        if (on) {
            at = __atomic_load_n(&s_at[wave][d], __ATOMIC_RELAXED);
            out[at + rank] = item;
        }
        // every lane has read its digit's place before the first lane of that digit moves it on
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (on && rank == 0) __atomic_store_n(&s_at[wave][d], at + __popcll(peers), __ATOMIC_RELAXED);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

template <bool FIRST, bool TB>
__global__ __launch_bounds__(kSortThreads) void sort_move_kernel(SortParams P) {
    __shared__ int s_at[kSortWaves][kBins];
    __shared__ int s_wave[kBins / 64];
    if (fills<TB>(P, P.tiles)) return;
    const int tid = threadIdx.x, mine = blockIdx.x;
    int before = 0, total = 0;
    if (tid < kBins) {
#pragma unroll 8
        for (int t = 0; t < P.tiles; ++t) {
            const int c = P.hist[t * kBins + tid];
            before += t < mine ? c : 0;
            total += c;
        }
    }
    move_tile<FIRST>(P, P.in, P.out, mine * P.tile, P.tile, P.shift, before, total, s_at, s_wave);
}

// One tile: every pass in one workgroup.  The items go through global memory between the passes.
template <bool TB>
__global__ __launch_bounds__(kSortThreads) void sort_one_kernel(SortParams P) {
    __shared__ int s_at[kSortWaves][kBins];
    __shared__ int s_wave[kBins / 64];
    __shared__ int s_count[kBins];
    if (fills<TB>(P, 1)) return;
    const int tid = threadIdx.x;
    if (tid == 0) *P.n_long = 0;
    const uint64_t *in = P.in;
    uint64_t *out = P.out;
    for (int shift = 0; shift < P.bits; shift += kDigit) {
        if (tid < kBins) s_count[tid] = 0;
        __syncthreads();
        for (int i = tid; i < P.n; i += kSortThreads) {
            const uint64_t item = shift == 0 ? first_item(P, i, true) : in[i];
            atomicAdd(&s_count[digit_of(item, shift)], 1);
        }
        __syncthreads();
        const int total = tid < kBins ? s_count[tid] : 0;
        if (shift == 0) move_tile<true>(P, in, out, 0, P.tile, shift, 0, total, s_at, s_wave);
        else move_tile<false>(P, in, out, 0, P.tile, shift, 0, total, s_at, s_wave);
        __syncthreads();
        uint64_t *t = (uint64_t *)in;
        in = out;
        out = t;
    }
}

// ---- sum and join ---------------------------------------------------------------------------------
constexpr int kPiece = 64;
constexpr int kSumThreads = 256;
constexpr int kSumWaves = kSumThreads / 64;
constexpr int kSumCols = 64 * kVec;            // columns per wave
constexpr int kAhead = 8;                      // tokens whose loads are in flight together

struct SumParams {
    const char *grad;
    int64_t grad_stride_b;
    Table table;
    const uint64_t *sorted;
    float *part;                               // [pieces][2][D]: the run entering from before, the run leaving
    int32_t *n_long, *long_piece;              // pieces in which a long run starts
    int32_t n, pieces, colblocks, accumulate, sum_blocks, fill_first;
    float scale;
};

__device__ __forceinline__ int key_of(uint64_t item) { return (int)(item >> 32); }

// table row = (old +) scale * sum, rounded once.
template <bool TB>
__device__ __forceinline__ void write_row(const SumParams &P, int id, int v, const float (&a)[kVec]) {
    char *row = P.table.p + id * P.table.stride_b;
    float o[kVec];
#pragma unroll
    for (int e = 0; e < kVec; ++e) o[e] = 0.0f;
    if (P.accumulate) widen<TB>(load_raw<TB>(row, v, P.table.D), o);
#pragma unroll
    for (int e = 0; e < kVec; ++e) o[e] = fmaf(P.scale, a[e], o[e]);
    store8<TB>(row, v, P.table.D, o);
}

// One wave: piece `piece`, columns colblock*512 ...  Positions in the window of three pieces around it:
// [64, 128) is the piece itself.
template <bool GB, bool TB>
__device__ void sum_piece(const SumParams &P, int piece, int colblock) {
    const int lane = lane_id(), D = P.table.D;
    const int64_t i0 = (int64_t)piece * kPiece + lane;
    const uint64_t none = (uint64_t)P.table.n_vocab << 32;         // a token that adds nothing
    const uint64_t w0 = i0 >= kPiece ? P.sorted[i0 - kPiece] : none;
    const uint64_t w1 = i0 < P.n ? P.sorted[i0] : none;
    const uint64_t w2 = i0 + kPiece < P.n ? P.sorted[i0 + kPiece] : none;
    const int k0 = key_of(w0), k1 = key_of(w1), k2 = key_of(w2), p1 = (int)(uint32_t)w1, p2 = (int)(uint32_t)w2;
    // run starts as bits; ids stop at the first token that adds nothing
    auto starts = [&](int k, int previous) {
        const int below = up_one(k);           // before the choice: every lane takes part
        return __ballot(k != (lane == 0 ? previous : below));
    };
    const uint64_t s0 = starts(k0, -1), s1 = starts(k1, __builtin_amdgcn_readlane(k0, 63)),
                   s2 = starts(k2, __builtin_amdgcn_readlane(k1, 63));
    const int ids1 = __popcll(__ballot(k1 != P.table.n_vocab)), ids2 = __popcll(__ballot(k2 != P.table.n_vocab));
    if (ids1 == 0) return;
    // first start at or after window position i >= 64 (192: none in the window)
    auto next_start = [&](int i) {
        if (i < 128) {
            const uint64_t m = s1 & (~0ull << (i - 64));
            if (m != 0) return 64 + (int)__builtin_ctzll(m);
            i = 128;
        }
        const uint64_t m = i < 192 ? s2 & (~0ull << (i - 128)) : 0ull;
        return m != 0 ? 128 + (int)__builtin_ctzll(m) : 192;
    };
    int begin = 64, end;
    // the run that enters from the piece before: its part here if it is long, nothing otherwise
    int head_end = 0;                          // > 0: tokens [64, head_end) go to partial sum 0
    if (!(s1 & 1)) {
        const int lo = s0 != 0 ? 63 - (int)__builtin_clzll(s0) : 0, hi = next_start(65);
        if (hi - lo > kPiece) head_end = min(hi, 128);
        else begin = hi;
    }
    // the last run that starts here: to its end, or to the piece's end and into partial sum 1 if it is long
    int tail = 192;                            // < 192: where a long run starts
    if (ids1 < 64) {
        end = 64 + ids1;
    } else if (s1 != 0) {
        const int last = 127 - (int)__builtin_clzll(s1), hi = next_start(last + 1);
        end = min(hi, 128 + ids2);
        if (hi - last > kPiece) {
            tail = last;
            end = 128;
        }
    } else {
        end = 128;                             // one run covers the piece: head_end is set, or nothing starts here
    }
    if (begin >= end) return;
    if (tail < 192 && colblock == 0 && lane == 0) P.long_piece[atomicAdd(P.n_long, 1)] = piece;

    // lanes past the last column keep running (their registers are read across the wave) on its vector
    const int nv = (D + kVec - 1) / kVec, own = colblock * 64 + lane, v = min(own, nv - 1);
    const bool live = own < nv;
    float a[kVec];
#pragma unroll
    for (int e = 0; e < kVec; ++e) a[e] = 0.0f;
    for (int t0 = begin; t0 < end; t0 += kAhead) {
        Raw<GB> raw[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int t = t0 + u;
            if (t < end) {
                const int pos = t < 128 ? __builtin_amdgcn_readlane(p1, t - 64) : __builtin_amdgcn_readlane(p2, t - 128);
                raw[u] = load_raw<GB>(P.grad + pos * P.grad_stride_b, v, D);
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int t = t0 + u;
            if (t >= end) break;
            float x[kVec];
            widen<GB>(raw[u], x);
#pragma unroll
            for (int e = 0; e < kVec; ++e) a[e] += x[e];
            if (t + 1 < end && next_start(t + 1) != t + 1) continue;
            if (t + 1 == head_end || (t >= tail && t + 1 == end)) {
                float *part = P.part + ((int64_t)piece * 2 + (t + 1 == head_end ? 0 : 1)) * D;
#pragma unroll
                for (int e = 0; e < kVec; ++e)
                    if (live && v * kVec + e < D) part[v * kVec + e] = a[e];
            } else {
                const int id = t < 128 ? __builtin_amdgcn_readlane(k1, t - 64) : __builtin_amdgcn_readlane(k2, t - 128);
                if (live) write_row<TB>(P, id, v, a);
            }
#pragma unroll
            for (int e = 0; e < kVec; ++e) a[e] = 0.0f;
        }
    }
}

// First sorted position whose id is at least `key`.
__device__ __forceinline__ int first_at_least(const uint64_t *sorted, int n, int key) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = lo + (hi - lo) / 2;
        if (key_of(sorted[mid]) < key) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

template <bool GB, bool TB>
__global__ __launch_bounds__(kSumThreads) void embed_sum_kernel(SumParams P) {
    if ((int)blockIdx.x < P.sum_blocks) {
        const int unit = (int)blockIdx.x * kSumWaves + uni(threadIdx.x >> 6);
        if (unit < P.pieces * P.colblocks) sum_piece<GB, TB>(P, uni(unit / P.colblocks), uni(unit % P.colblocks));
        return;
    }
    // zeros for ids without a token
    __shared__ uint64_t s_absent;
    const int v0 = P.fill_first + ((int)blockIdx.x - P.sum_blocks) * kFillRows, tid = threadIdx.x;
    if (tid < kFillRows) {
        const int id = v0 + tid;
        bool absent = id < P.table.n_vocab;
        if (absent) {
            const int at = first_at_least(P.sorted, P.n, id);
            absent = at >= P.n || key_of(P.sorted[at]) != id;
        }
        const uint64_t b = __ballot(absent);
        if (tid == 0) s_absent = b;
    }
    __syncthreads();
    fill_rows<TB, kSumThreads>(P.table, v0, s_absent);
}

// The partial sums of each long run: 16 threads side by side on 4 columns each, 16 slices of pieces.
constexpr int kJoinCols = 64, kJoinSlices = 16;

constexpr int kJoinRuns = 16;                  // long runs side by side

template <bool TB>
__global__ __launch_bounds__(256) void embed_join_kernel(SumParams P) {
    __shared__ float s_sum[kJoinSlices][kJoinCols];
    __shared__ int s_more[4];
    const int tid = threadIdx.x, slice = tid >> 4, c = (tid & 15) * 4, D = P.table.D;
    const int col = blockIdx.x * kJoinCols + c;
    const int n_long = *P.n_long;
    for (int l = blockIdx.y; l < n_long; l += gridDim.y) {
        const int p0 = P.long_piece[l];
        const int key = key_of(P.sorted[(int64_t)p0 * kPiece + kPiece - 1]);
        // the pieces after p0 that start with the run's id, 256 at a time
        int count = 1;
        while (true) {
            const int64_t i = ((int64_t)p0 + count + tid) * kPiece;
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
            const float *part = P.part + ((int64_t)(p0 + p) * 2 + (p == 0 ? 1 : 0)) * D;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col + e < D) a[e] += part[col + e];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s_sum[slice][c + e] = a[e];
        __syncthreads();
        if (tid < kJoinCols / kVec) {
            const int v = blockIdx.x * (kJoinCols / kVec) + tid;
            float t[kVec];
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                t[e] = 0.0f;
                for (int s = 0; s < kJoinSlices; ++s) t[e] += s_sum[s][tid * kVec + e];
            }
            if (v * kVec < D) write_row<TB>(P, key, v, t);
        }
        __syncthreads();
    }
}

// ---- host -----------------------------------------------------------------------------------------
struct GradSpace {
    size_t a, b, hist, n_long, long_piece, part, bytes;
    int tile, tiles, pieces;
};
GradSpace grad_space(int64_t n, int64_t D) {
    GradSpace w{};
    w.tile = (int)std::min<int64_t>(kMinTile, (n + kSortThreads - 1) / kSortThreads * kSortThreads);
    if (w.tile == 0) w.tile = kSortThreads;
    while ((n + w.tile - 1) / w.tile > kMaxTiles) w.tile *= 2;
    w.tiles = (int)((n + w.tile - 1) / w.tile);
    w.pieces = (int)((n + kPiece - 1) / kPiece);
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
// log2 of the lanes that share a row of D: as many as its 8-element vectors, in a workgroup of 256.
int lanes_of(int32_t D) {
    const int nv = (D + kVec - 1) / kVec;
    int l = 0;
    while ((1 << l) < nv && (1 << l) < kEmbedThreads) ++l;
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
    P.lanes_log2 = lanes_of(D);
    const int64_t per = (int64_t)(kEmbedThreads >> P.lanes_log2) * kTokens;
    const dim3 grid((unsigned)((n_tokens + per - 1) / per)), block(kEmbedThreads);
    const hipStream_t st = (hipStream_t)stream;
    if (table_dtype == DLLM_BF16) {
        if (out_dtype == DLLM_BF16) hipLaunchKernelGGL((embed_kernel<true, true>), grid, block, 0, st, P);
        else hipLaunchKernelGGL((embed_kernel<true, false>), grid, block, 0, st, P);
    } else {
        if (out_dtype == DLLM_BF16) hipLaunchKernelGGL((embed_kernel<false, true>), grid, block, 0, st, P);
        else hipLaunchKernelGGL((embed_kernel<false, false>), grid, block, 0, st, P);
    }
    return check_hip(hipGetLastError(), "dllm_embed launch");
}

extern "C" size_t dllm_embed_grad_workspace_bytes(int32_t n_tokens, int32_t n_vocab, int32_t D) {
    if (!sizes_ok(n_tokens, n_vocab, D)) return 0;
    return grad_space(n_tokens, D).bytes;
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
    const size_t gb = n_tokens ? ((size_t)(n_tokens - 1) * grad_stride + D) * gs : 0;
    if (overlap(grad_table, tbytes, grad_out, gb) || overlap(grad_table, tbytes, ids, (size_t)n_tokens * 4) ||
        (valid && overlap(grad_table, tbytes, valid, n_tokens)) || overlap(grad_table, tbytes, workspace, w.bytes) ||
        overlap(workspace, w.bytes, grad_out, gb) || overlap(workspace, w.bytes, ids, (size_t)n_tokens * 4) ||
        (valid && overlap(workspace, w.bytes, valid, n_tokens)))
        return fail(DLLM_ERR_ARG, "%s: grad_table or workspace overlaps another buffer", who);
    char *ws = (char *)workspace;
    const hipStream_t st = (hipStream_t)stream;

    const Table table = {(char *)grad_table, table_stride * ts, n_vocab, D, lanes_of(D)};
    const bool tb = table_dtype == DLLM_BF16;
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
    int filled = 0;
    if (n_tokens > 0) {
        // rows each sort launch clears, in whole filling workgroups
        const int64_t row_bytes = (int64_t)D * ts, quota = accumulate ? 0 : (kFillBytes / row_bytes + kFillRows - 1) / kFillRows * kFillRows;
        auto launch = [&](auto kernel, int sorting) {
            S.fill_first = filled;
            S.fill_end = filled = (int)std::min<int64_t>(n_vocab, filled + quota);
            const int blocks = sorting + (S.fill_end - S.fill_first + kFillRows - 1) / kFillRows;
            hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(kSortThreads), 0, st, S);
        };
        if (w.tiles == 1) {
            S.in = from;
            S.out = to;
            tb ? launch(sort_one_kernel<true>, 1) : launch(sort_one_kernel<false>, 1);
            if (passes & 1) std::swap(from, to);
        } else {
            for (int pass = 0; pass < passes; ++pass) {
                S.shift = pass * kDigit;
                S.in = from;
                S.out = to;
                if (pass == 0) {
                    tb ? launch(sort_count_kernel<true, true>, w.tiles) : launch(sort_count_kernel<true, false>, w.tiles);
                    tb ? launch(sort_move_kernel<true, true>, w.tiles) : launch(sort_move_kernel<true, false>, w.tiles);
                } else {
                    tb ? launch(sort_count_kernel<false, true>, w.tiles) : launch(sort_count_kernel<false, false>, w.tiles);
                    tb ? launch(sort_move_kernel<false, true>, w.tiles) : launch(sort_move_kernel<false, false>, w.tiles);
                }
                std::swap(from, to);
            }
        }
        rc = check_hip(hipGetLastError(), "dllm_embed_grad sort launch");
        if (rc != DLLM_OK) return rc;
    }

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
    Q.accumulate = accumulate != 0;
    Q.sum_blocks = (int)(((int64_t)Q.pieces * Q.colblocks + kSumWaves - 1) / kSumWaves);
    Q.fill_first = filled;
    Q.scale = scale;
    const int blocks = Q.sum_blocks + (accumulate ? 0 : (n_vocab - filled + kFillRows - 1) / kFillRows);
    if (blocks == 0) return DLLM_OK;
    auto sum = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(kSumThreads), 0, st, Q); };
    if (grad_dtype == DLLM_BF16) tb ? sum(embed_sum_kernel<true, true>) : sum(embed_sum_kernel<true, false>);
    else tb ? sum(embed_sum_kernel<false, true>) : sum(embed_sum_kernel<false, false>);
    rc = check_hip(hipGetLastError(), "dllm_embed_grad sum launch");
    if (rc != DLLM_OK || n_tokens <= kPiece) return rc;      // no run longer than a piece
    const dim3 jg((unsigned)((D + kJoinCols - 1) / kJoinCols), kJoinRuns);
    if (tb) hipLaunchKernelGGL(embed_join_kernel<true>, jg, dim3(256), 0, st, Q);
    else hipLaunchKernelGGL(embed_join_kernel<false>, jg, dim3(256), 0, st, Q);
    return check_hip(hipGetLastError(), "dllm_embed_grad join launch");
}
