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
//      the vocabulary's bits need.  Each pass counts digits per tile, scans the counts, and moves the
//      items; a wave finds an item's rank among equal digits by one ballot per digit bit.
//   2. Sum: pieces of kPiece sorted tokens.  A piece sums the runs that start in it, following the last
//      one past its end, so runs up to kPiece tokens are never split.  A longer run (the mask token
//      of a training box can hold half of all tokens) leaves one partial sum per piece it covers.
//      Other workgroups of the same launch write the zeros of ids that do not occur.
//   3. Join: the partial sums of each long run, in order.
#include "elem_common.h"

namespace {

using namespace dllm;

constexpr int kVec = 8;                        // elements per thread
constexpr int kEmbedThreads = 256;
constexpr int kTokens = 4;                     // tokens per thread, their loads in flight together

// Elements [v*8, v*8 + 8) of a row of D.
template <bool BF16>
__device__ __forceinline__ void load8(const char *row, int v, int D, float (&x)[kVec]) {
    typedef typename Row<BF16>::vec vec;
    if ((v + 1) * kVec <= D) {
        if (BF16) {
            const u32x4 a = ((const vec *)row)[v];
            unpack<true>(a, x);
        } else {
            const u32x4 a = ((const vec *)row)[2 * v], b = ((const vec *)row)[2 * v + 1];
            unpack<false>(a, x);
            unpack<false>(b, x + 4);
        }
    } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            const int d = v * kVec + e;
            x[e] = d >= D ? 0.0f : BF16 ? __uint_as_float((uint32_t)((const uint16_t *)row)[d] << 16) : ((const float *)row)[d];
        }
    }
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
        float x[kTokens][kVec];
#pragma unroll
        for (int u = 0; u < kTokens; ++u) {
            if (id[u] >= 0) {
                load8<TB>(P.table + id[u] * P.table_stride_b, v, P.D, x[u]);
            } else {
#pragma unroll
                for (int e = 0; e < kVec; ++e) x[u][e] = 0.0f;
            }
        }
#pragma unroll
        for (int u = 0; u < kTokens; ++u) {
            if (tok[u] < 0) continue;
#pragma unroll
            for (int e = 0; e < kVec; ++e) x[u][e] = id[u] >= 0 ? x[u][e] * P.scale : 0.0f;
            store8<OB>(P.out + tok[u] * P.out_stride_b, v, P.D, x[u]);
        }
    }
}

// ---- sort ----------------------------------------------------------------------------------------
constexpr int kDigit = 9;
constexpr int kBins = 1 << kDigit;
constexpr int kSortThreads = 256;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSortTile = 4096;
constexpr int kWaveItems = kSortTile / kSortWaves;   // consecutive items a wave moves

struct SortParams {
    const int32_t *ids;                        // first pass: the ids themselves
    const uint8_t *valid;
    const uint64_t *in;                        // later passes: id << 32 | position
    uint64_t *out;
    int32_t *hist;                             // [kBins * tiles]: counts, then positions
    int32_t *total;                            // [kBins]
    int32_t *n_long;                           // cleared by the first pass
    int32_t n, n_vocab, tiles, shift;
    int32_t *status;
};

// Tokens that add nothing sort behind every id, as n_vocab.
template <bool FIRST>
__device__ __forceinline__ uint64_t sort_item(const SortParams &P, int i, bool report) {
    if (!FIRST) return P.in[i];
    int id = P.ids[i];
    if (P.valid != nullptr && P.valid[i] == 0) id = P.n_vocab;
    else if (id < 0 || id >= P.n_vocab) {
        id = P.n_vocab;
        if (report) set_status(P.status, DLLM_ERR_ARG);
    }
    return (uint64_t)(uint32_t)id << 32 | (uint32_t)i;
}
__device__ __forceinline__ int digit_of(uint64_t item, int shift) { return (int)((item >> 32) >> shift) & (kBins - 1); }

template <bool FIRST>
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortParams P) {
    __shared__ int s_count[kBins];
    const int tid = threadIdx.x, tile = blockIdx.x;
    if (FIRST && tile == 0 && tid == 0) *P.n_long = 0;
    for (int b = tid; b < kBins; b += kSortThreads) s_count[b] = 0;
    __syncthreads();
    const int end = (int)min((int64_t)P.n, ((int64_t)tile + 1) * kSortTile);
    for (int i = tile * kSortTile + tid; i < end; i += kSortThreads)
        atomicAdd(&s_count[digit_of(sort_item<FIRST>(P, i, true), P.shift)], 1);
    __syncthreads();
    for (int b = tid; b < kBins; b += kSortThreads) P.hist[(int64_t)b * P.tiles + tile] = s_count[b];
}

// One workgroup per digit: exclusive positions over the tiles, and the digit's total.
__global__ __launch_bounds__(kSortThreads) void sort_scan_kernel(SortParams P) {
    __shared__ int s_wave[kSortWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int32_t *h = P.hist + (int64_t)blockIdx.x * P.tiles;
    int run = 0;
    for (int t0 = 0; t0 < P.tiles; t0 += kSortThreads) {
        const int t = t0 + tid;
        const int c = t < P.tiles ? h[t] : 0;
        const int incl = wave_incl_scan(c);
        if (lane == 63) s_wave[wave] = incl;
        __syncthreads();
        int before = run, all = 0;
        for (int w = 0; w < kSortWaves; ++w) {
            before += w < wave ? s_wave[w] : 0;
            all += s_wave[w];
        }
        if (t < P.tiles) h[t] = before + incl - c;
        run += all;
        __syncthreads();
    }
    if (tid == 0) P.total[blockIdx.x] = run;
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

template <bool FIRST>
__global__ __launch_bounds__(kSortThreads) void sort_move_kernel(SortParams P) {
    __shared__ int s_at[kSortWaves][kBins];    // counts of a wave's items, then where its next item goes
    __shared__ int s_wave[kSortWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, tile = blockIdx.x;
    for (int b = tid; b < kSortWaves * kBins; b += kSortThreads) (&s_at[0][0])[b] = 0;
    __syncthreads();
    const int i0 = tile * kSortTile + wave * kWaveItems;
    for (int i = i0 + lane; i < i0 + kWaveItems; i += 64)
        if (i < P.n) atomicAdd(&s_at[wave][digit_of(sort_item<FIRST>(P, i, false), P.shift)], 1);
    // where each digit starts in the output: two digits per thread, scanned
    const int c0 = P.total[2 * tid], c1 = P.total[2 * tid + 1];
    const int incl = wave_incl_scan(c0 + c1);
    if (lane == 63) s_wave[wave] = incl;
    __syncthreads();
    int start = incl - c0 - c1;
    for (int w = 0; w < wave; ++w) start += s_wave[w];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int b = 2 * tid + h;
        int at = (h ? start + c0 : start) + P.hist[(int64_t)b * P.tiles + tile];
        for (int w = 0; w < kSortWaves; ++w) {
            const int c = s_at[w][b];
            s_at[w][b] = at;
            at += c;
        }
    }
    __syncthreads();
    for (int i = i0 + lane; i - lane < i0 + kWaveItems; i += 64) {
        const bool on = i < P.n;
        const uint64_t item = on ? sort_item<FIRST>(P, i, false) : 0;
        const int d = digit_of(item, P.shift);
        const uint64_t peers = same_digit(d, on);
        const int rank = __popcll(peers & ((1ull << lane) - 1));
        if (on) {
            const int at = __atomic_load_n(&s_at[wave][d], __ATOMIC_RELAXED);
            P.out[at + rank] = item;
        }
        __builtin_amdgcn_wave_barrier();       // every lane has read before one of them writes
        if (on && rank == 0) __atomic_store_n(&s_at[wave][d], __atomic_load_n(&s_at[wave][d], __ATOMIC_RELAXED) + __popcll(peers), __ATOMIC_RELAXED);
        __builtin_amdgcn_wave_barrier();
    }
}

// ---- sum and join ---------------------------------------------------------------------------------
constexpr int kPiece = 64;
constexpr int kSumThreads = 256;
constexpr int kSumCols = kSumThreads * kVec;   // columns per workgroup
constexpr int kAhead = 8;                      // tokens whose loads are in flight together
constexpr int kZeroRows = 64;                  // table rows a zeroing workgroup looks at

struct SumParams {
    const char *grad;
    int64_t grad_stride_b;
    char *table;
    int64_t table_stride_b;
    const uint64_t *sorted;
    float *part;                               // [pieces][2][D]: the run entering from before, the run leaving
    int32_t *n_long, *long_piece;              // pieces in which a long run starts
    int32_t n, n_vocab, D, pieces, colblocks, accumulate;
    float scale;
};

__device__ __forceinline__ int key_of(uint64_t item) { return (int)(item >> 32); }

// table row (+)= scale * sum, rounded once.
template <bool TB>
__device__ __forceinline__ void write_row(const SumParams &P, int id, int v, float (&a)[kVec]) {
    char *row = P.table + id * P.table_stride_b;
    float o[kVec];
#pragma unroll
    for (int e = 0; e < kVec; ++e) o[e] = 0.0f;
    if (P.accumulate) load8<TB>(row, v, P.D, o);
#pragma unroll
    for (int e = 0; e < kVec; ++e) o[e] = fmaf(P.scale, a[e], o[e]);
    store8<TB>(row, v, P.D, o);
}

template <bool GB, bool TB>
__device__ void sum_piece(const SumParams &P, int piece, int colblock) {
    // ids and positions of this piece, with the ids of the pieces on either side (-1 outside)
    __shared__ int s_key[3 * kPiece];
    __shared__ int s_pos[2 * kPiece];
    const int tid = threadIdx.x;
    const int64_t i0 = (int64_t)piece * kPiece;
    if (tid < 3 * kPiece) {
        const int64_t i = i0 - kPiece + tid;
        uint64_t item = (uint64_t)(uint32_t)-1 << 32;
        if (i >= 0 && i < P.n) item = P.sorted[i];
        const int key = key_of(item);
        s_key[tid] = key == P.n_vocab ? -1 : key;
        if (tid >= kPiece) s_pos[tid - kPiece] = (int)(uint32_t)item;
    }
    __syncthreads();
    const int v = colblock * kSumThreads + tid, nv = (P.D + kVec - 1) / kVec;
    const bool live = v < nv;
    // runs in window coordinates: [kPiece, 2*kPiece) is this piece
    int i = kPiece;
    while (i < 2 * kPiece) {
        const int key = uni(s_key[i]);
        if (key < 0) break;                    // only tokens that add nothing follow
        const bool entering = i == kPiece && uni(s_key[i - 1]) == key;
        // first and last position of the run within the window
        int lo = i, hi = i + 1;
        while (lo > 0 && uni(s_key[lo - 1]) == key) --lo;
        while (hi < 3 * kPiece && uni(s_key[hi]) == key) ++hi;
        const bool is_long = hi - lo > kPiece;
        int end = hi;
        if (is_long) end = min(hi, 2 * kPiece);      // this piece's part of it
        if (!entering || is_long) {
            float a[kVec];
#pragma unroll
            for (int e = 0; e < kVec; ++e) a[e] = 0.0f;
            if (live) {
                for (int t = i; t < end; t += kAhead) {
                    float x[kAhead][kVec];
#pragma unroll
                    for (int u = 0; u < kAhead; ++u) {
                        if (t + u < end)
                            load8<GB>(P.grad + uni(s_pos[t + u - kPiece]) * P.grad_stride_b, v, P.D, x[u]);
                    }
#pragma unroll
                    for (int u = 0; u < kAhead; ++u) {
                        if (t + u < end) {
#pragma unroll
                            for (int e = 0; e < kVec; ++e) a[e] += x[u][e];
                        }
                    }
                }
                if (!is_long) {
                    write_row<TB>(P, key, v, a);
                } else {
                    float *part = P.part + ((int64_t)piece * 2 + (entering ? 0 : 1)) * P.D;
#pragma unroll
                    for (int e = 0; e < kVec; ++e)
                        if (v * kVec + e < P.D) part[v * kVec + e] = a[e];
                }
            }
            if (is_long && !entering && colblock == 0 && tid == 0) P.long_piece[atomicAdd(P.n_long, 1)] = piece;
        }
        i = hi;
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
    const int sums = P.pieces * P.colblocks;
    if ((int)blockIdx.x < sums) {
        sum_piece<GB, TB>(P, blockIdx.x / P.colblocks, blockIdx.x % P.colblocks);
        return;
    }
    // zeros for ids without a token
    __shared__ uint64_t s_absent;
    const int v0 = (blockIdx.x - sums) * kZeroRows, tid = threadIdx.x;
    if (tid < kZeroRows) {
        const int id = v0 + tid;
        bool absent = id < P.n_vocab;
        if (absent) {
            const int at = first_at_least(P.sorted, P.n, id);
            absent = at >= P.n || key_of(P.sorted[at]) != id;
        }
        const uint64_t b = __ballot(absent);
        if (tid == 0) s_absent = b;
    }
    __syncthreads();
    const uint64_t absent = s_absent;
    const int nv = (P.D + kVec - 1) / kVec;
    const float z[kVec] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    for (int r = 0; r < kZeroRows; ++r) {
        if (!((absent >> r) & 1)) continue;
        char *row = P.table + (int64_t)(v0 + r) * P.table_stride_b;
        for (int v = tid; v < nv; v += kSumThreads) store8<TB>(row, v, P.D, z);
    }
}

// The partial sums of each long run: 16 threads side by side on 4 columns each, 16 slices of pieces.
constexpr int kJoinCols = 64, kJoinSlices = 16;

template <bool TB>
__global__ __launch_bounds__(256) void embed_join_kernel(SumParams P) {
    __shared__ float s_sum[kJoinSlices][kJoinCols];
    const int tid = threadIdx.x, slice = tid >> 4, c = (tid & 15) * 4;
    const int col = blockIdx.x * kJoinCols + c;
    const int n_long = *P.n_long;
    for (int l = blockIdx.y; l < n_long; l += gridDim.y) {
        const int p0 = P.long_piece[l];
        const int key = key_of(P.sorted[(int64_t)p0 * kPiece + kPiece - 1]);
        const int p1 = (first_at_least(P.sorted, P.n, key + 1) - 1) / kPiece;   // the run's last piece
        const int count = p1 - p0 + 1, per = (count + kJoinSlices - 1) / kJoinSlices;
        float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int p = p0 + slice * per; p < min(p0 + (slice + 1) * per, p1 + 1); ++p) {
            const float *part = P.part + ((int64_t)p * 2 + (p == p0 ? 1 : 0)) * P.D;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col + e < P.D) a[e] += part[col + e];
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
            if (v * kVec < P.D) write_row<TB>(P, key, v, t);
        }
        __syncthreads();
    }
}

// ---- host -----------------------------------------------------------------------------------------
struct GradSpace {
    size_t a, b, hist, total, n_long, long_piece, part, bytes;
    int tiles, pieces;
};
GradSpace grad_space(int64_t n, int64_t D) {
    GradSpace w{};
    w.tiles = (int)((n + kSortTile - 1) / kSortTile);
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
    w.total = take((size_t)kBins * 4);
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
    const int nv = (D + kVec - 1) / kVec;
    while ((1 << P.lanes_log2) < nv && (1 << P.lanes_log2) < kEmbedThreads) ++P.lanes_log2;
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
    const size_t tb = ((size_t)(n_vocab - 1) * table_stride + D) * ts;
    const size_t gb = n_tokens ? ((size_t)(n_tokens - 1) * grad_stride + D) * gs : 0;
    if (overlap(grad_table, tb, grad_out, gb) || overlap(grad_table, tb, ids, (size_t)n_tokens * 4) ||
        (valid && overlap(grad_table, tb, valid, n_tokens)) || overlap(grad_table, tb, workspace, w.bytes) ||
        overlap(workspace, w.bytes, grad_out, gb) || overlap(workspace, w.bytes, ids, (size_t)n_tokens * 4) ||
        (valid && overlap(workspace, w.bytes, valid, n_tokens)))
        return fail(DLLM_ERR_ARG, "%s: grad_table or workspace overlaps another buffer", who);
    char *ws = (char *)workspace;
    const hipStream_t st = (hipStream_t)stream;

    SortParams S{};
    S.ids = ids; S.valid = valid;
    S.hist = (int32_t *)(ws + w.hist);
    S.total = (int32_t *)(ws + w.total);
    S.n_long = (int32_t *)(ws + w.n_long);
    S.n = n_tokens; S.n_vocab = n_vocab; S.tiles = w.tiles;
    S.status = status;
    uint64_t *from = (uint64_t *)(ws + w.a), *to = (uint64_t *)(ws + w.b);
    int bits = 1;                              // ids 0 .. n_vocab, n_vocab itself standing for no id
    while (n_vocab >> bits) ++bits;
    if (n_tokens > 0) {
        for (int shift = 0; shift < bits; shift += kDigit) {
            S.shift = shift;
            S.in = from;
            S.out = to;
            if (shift == 0) {
                hipLaunchKernelGGL(sort_count_kernel<true>, dim3(w.tiles), dim3(kSortThreads), 0, st, S);
                hipLaunchKernelGGL(sort_scan_kernel, dim3(kBins), dim3(kSortThreads), 0, st, S);
                hipLaunchKernelGGL(sort_move_kernel<true>, dim3(w.tiles), dim3(kSortThreads), 0, st, S);
            } else {
                hipLaunchKernelGGL(sort_count_kernel<false>, dim3(w.tiles), dim3(kSortThreads), 0, st, S);
                hipLaunchKernelGGL(sort_scan_kernel, dim3(kBins), dim3(kSortThreads), 0, st, S);
                hipLaunchKernelGGL(sort_move_kernel<false>, dim3(w.tiles), dim3(kSortThreads), 0, st, S);
            }
            rc = check_hip(hipGetLastError(), "dllm_embed_grad sort launch");
            if (rc != DLLM_OK) return rc;
            uint64_t *t = from;
            from = to;
            to = t;
        }
    }

    SumParams Q{};
    Q.grad = (const char *)grad_out;
    Q.grad_stride_b = grad_stride * gs;
    Q.table = (char *)grad_table;
    Q.table_stride_b = table_stride * ts;
    Q.sorted = from;
    Q.part = (float *)(ws + w.part);
    Q.n_long = S.n_long;
    Q.long_piece = (int32_t *)(ws + w.long_piece);
    Q.n = n_tokens; Q.n_vocab = n_vocab; Q.D = D;
    Q.pieces = w.pieces;
    Q.colblocks = (D + kSumCols - 1) / kSumCols;
    Q.accumulate = accumulate != 0;
    Q.scale = scale;
    const int64_t blocks = (int64_t)Q.pieces * Q.colblocks + (accumulate ? 0 : (n_vocab + kZeroRows - 1) / kZeroRows);
    if (blocks >= (int64_t)1 << 31) return fail(DLLM_ERR_SHAPE, "%s: n_tokens * D too large", who);
    auto sum = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(kSumThreads), 0, st, Q); };
    if (grad_dtype == DLLM_BF16) table_dtype == DLLM_BF16 ? sum(embed_sum_kernel<true, true>) : sum(embed_sum_kernel<true, false>);
    else table_dtype == DLLM_BF16 ? sum(embed_sum_kernel<false, true>) : sum(embed_sum_kernel<false, false>);
    rc = check_hip(hipGetLastError(), "dllm_embed_grad sum launch");
    if (rc != DLLM_OK || n_tokens <= kPiece) return rc;      // no run longer than a piece
    const dim3 jg((unsigned)((D + kJoinCols - 1) / kJoinCols), 4);
    if (table_dtype == DLLM_BF16) hipLaunchKernelGGL(embed_join_kernel<true>, jg, dim3(256), 0, st, Q);
    else hipLaunchKernelGGL(embed_join_kernel<false>, jg, dim3(256), 0, st, Q);
    return check_hip(hipGetLastError(), "dllm_embed_grad join launch");
}
