// dllm_logprobs: log probabilities of given tokens at selected slots, with the distribution's entropy
// and its top alternatives; dllm_logprobs_grad: their gradient with respect to the logits.
//
// What is computed ([DiLaServe] = page "DiLaServe: High SLO Attainment Serving for Diffusion Language
// Models" §三 3.1: the softmax distribution over a masked slot's vocabulary logits, of which the step
// keeps the largest probability only).  With x the V logits of a slot, m = max x and
// S = sum exp(x - m):
//   log p_v = x_v - m - log S;   entropy = log S - (1/S) sum exp(x - m) (x - m);
//   alternatives = the k largest x, the lowest column first among equals.
//
// How (gfx950).  A streaming reduction over the selected slots' rows, bound by HBM, on the scoring
// kernel's work split: rows are cut into chunks of 64*kVPL 16-byte vectors, a workgroup has an even
// share of all selected slots' chunks, and its waves take chunks one at a time from an LDS counter.
//   - One pass gives max, sum and the entropy's weighted sum T = sum e * y in base 2, with
//     y = (x - m) log2 e and e = 2^y: the entropy costs a max and an FMA per element beside the
//     unpack, max3, FMA, v_exp and add of the sum.  All terms of T have one sign, so the entropy
//     has no cancellation.
//   - S is held as r = S - 1, what it has beside the largest term, through chunks, lanes and log(1 + r): a token of
//     probability near 1 has log probability -r, of which 1 + r would keep the bits above 2^-24 only.  A
//     chunk's r is S - 1 where S >= 1.25; below, the lane that has the maximum hands its values to the wave, which
//     adds all but that one (0.2 to 0.4 us of 24 for 192 confident slots; 16384 slots 815 us for 814; 1024
//     slots all of whose chunks are like that 61.8 us for 59.6).
//   - y is one FMA, x*log2e - m*log2e.  The product m*log2e is rounded once per chunk; its residual
//     (exact, by an FMA) is taken out of the sums by a factor 2^-residual, so large offsets of the logits
//     cost no accuracy.  Chunks whose maximum lies beyond kNearMax subtract first instead.
//   - Alternatives: while a chunk is in registers each lane's largest element is known anyway; it is
//     kept (2 or 4 bytes per 128-byte lane share).  The k-th largest of those maxima cannot exceed the
//     k-th largest element, so the k best lie in the few lane shares whose maximum reaches it.
//   - A second kernel joins the chunk records in a fixed order, so the sums' bits do not depend on
//     timing, and looks up the given token's logit.  For the alternatives it bounds the k-th best
//     from below (the k-th largest of 64 group maxima, by ballots), reads again only the lane shares
//     that reach the bound (about 25 of 2432 for k = 20 and V = 152064), and puts each of their
//     elements above the bound into its place by counting the ones before it.
//     Keeping sorted lists in the streaming kernel instead took 2.3 times as long.
#include <algorithm>
#include <type_traits>

#include "elem_common.h"

namespace {

using namespace dllm;

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2eShort = 1.3349758e-8f;   // (log2 e - kLog2e) / kLog2e
constexpr float kFarBelow = -300.0f;           // base-2 exponent whose power is 0 in fp32 (2^-149 is the least)
constexpr float kNearMax = 65536.0f;           // |m| up to which rounding m * log2e moves y by less than 2^-8
constexpr float kPeaked = 1.25f;               // sum of powers of a chunk below which its largest element is set apart
constexpr int kNoKey = (int)0x80000000;        // below the key of every number

struct LogprobParams {
    const char *logits;
    int64_t pos_stride_b, row_stride_b;        // strides in bytes
    int32_t rows, L, V, NV, NC, k;
    const uint8_t *mask, *exclude;             // selected: mask != 0 and (exclude NULL or exclude == 0)
    const int32_t *tokens;
    int64_t token_stride;
    float *logprob, *entropy;
    float2 *stats;
    int32_t *top_ids;
    float *top_lp;
    float4 *partials;                          // [rows*L*NC] {max, sum, weighted sum, -}
    char *lane_max;                            // [rows*L*NC*64] each lane's largest element, in the logits' type
    int32_t *status;
};

// Integer order of floats: larger value, larger key; -0 and +0 share one, NaN has that of -inf.  A lane's
// largest value passes over NaN, so one of its elements has that value's key or a larger one, whatever they are.
__device__ __forceinline__ int order_key(float x) {
    const int b = __float_as_int(x != x ? -INFINITY : x + 0.0f);
    return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float key_value(int key) { return __int_as_float(key ^ ((key >> 31) & 0x7FFFFFFF)); }

// Selected slots among the 16 that start at s0, as bits.
__device__ __forceinline__ uint32_t selected16(const LogprobParams &P, int s0, int S) {
    uint32_t b = mask_bits16(P.mask, s0, S);
    if (P.exclude != nullptr) b &= ~mask_bits16(P.exclude, s0, S);
    return b;
}

// The kVPL loads of a chunk for this lane, whose first nf vectors are whole.  A row's ragged last
// vector, and every one past it, is read as the row's last E elements (a vector that lies in the row);
// widen() drops what belongs to other vectors.  Rows shorter than a vector are read there by element.
template <bool BF16>
__device__ __forceinline__ void issue_chunk(u32x4 (&raw)[kVPL], const char *row, int vb, int nf, int V) {
    typedef typename Row<BF16>::vec vec;
    constexpr int E = Fmt<BF16>::E;
    const int lane = lane_id();
    if (nf == kCH) {
        const vec *base = (const vec *)row + vb;
#pragma unroll
        for (int k = 0; k < kVPL; ++k) raw[k] = __builtin_nontemporal_load(base + k * 64 + lane);
    } else if (V >= E) {
#pragma unroll
        for (int k = 0; k < kVPL; ++k) {
            const uint32_t at = (uint32_t)min((vb + k * 64 + lane) * E, V - E) * (16 / E);
            raw[k] = __builtin_nontemporal_load((const vec *)(row + at));
        }
        asm volatile("; short chunk");         // keeps these loads apart: merged, both would hold 16 address registers
    }
}
// The chunk's values, in an order of their own within a lane; -inf where there is no element.
template <bool BF16>
__device__ __forceinline__ void widen(const u32x4 (&raw)[kVPL], float (&x)[kVPL][Fmt<BF16>::E], const char *row, int nf,
                                      int V) {
    constexpr int E = Fmt<BF16>::E;
#pragma unroll
    for (int k = 0; k < kVPL; ++k) unpack<BF16>(raw[k], x[k]);
    if (nf < kCH) {
        const int lane = lane_id(), ragged = V % E;
        if (V < E) load_vec_elems<BF16>(row, 0, V, x[0]);
#pragma unroll
        for (int k = 0; k < kVPL; ++k) {
            const int v = k * 64 + lane;
            const int first = v < nf || (V < E && v == 0) ? 0 : v == nf ? E - ragged : E;   // elements before it are not this vector's
#pragma unroll
            for (int e = 0; e < E; ++e) x[k][e] = e < first ? -INFINITY : x[k][e];
        }
    }
}

// ---- the k best, one per lane in order ----------------------------------------------------------
struct Best {
    int key, col;                              // this lane's entry
    int cut;                                   // key of entry k-1: what an element has to beat
};

// Insert after `at` entries: the entries from there move up a lane.
__device__ __forceinline__ void insert_at(Best &b, int at, int key, int col, int k) {
    const int lane = lane_id();
    const int mk = up_one(b.key), mc = up_one(b.col);
    b.key = lane < at ? b.key : lane == at ? key : mk;
    b.col = lane < at ? b.col : lane == at ? col : mc;
    b.cut = __builtin_amdgcn_readlane(b.key, k - 1);
}

// A lower bound of the k-th largest of the 64 lanes' keys (exact in its upper 16 bits), minus one: the
// floor that elements have to exceed.
__device__ __forceinline__ int kth_floor(int key, int k) {
    const uint32_t u = (uint32_t)key ^ 0x80000000u;
    uint32_t t = 0;
#pragma unroll 1
    for (int bit = 31; bit >= 16; --bit) {
        const uint32_t trial = t | (1u << bit);
        if (__popcll(__ballot(u >= trial)) >= k) t = trial;
    }
    return t == 0 ? kNoKey : (int)(t ^ 0x80000000u) - 1;
}

// Number the selected slots in slot order (16 per thread and tile) and list in s_id those of this
// workgroup, numbers q_lo .. q_hi that range(M, q_lo, q_hi) gives for M selected slots; false if it gives
// none.  The caller's next barrier makes the list visible.
template <typename Range>
__device__ __forceinline__ bool list_slots(const LogprobParams &P, int *s_id, int (&s_tmp)[2][kWaves], Range range) {
    const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
    const int S = P.rows * P.L, ntiles = (S + kTile - 1) / kTile;
    const uint32_t mb0 = selected16(P, tid * 16, S);
    fetch_args(P.logits, P.row_stride_b, P.pos_stride_b, P.partials, P.lane_max, P.V, P.NC);
    int more_cnt = 0;
    for (int t = 1; t < ntiles; ++t) more_cnt += __popc(selected16(P, t * kTile + tid * 16, S));
    // slots selected before this thread's 16 in its tile, and in the whole tile
    auto place = [&](uint32_t mb, int *tmp, int &before, int &total) {
        const int c = __popc(mb);
        const int incl = wave_incl_scan(c);
        if (lane == 63) tmp[wave] = incl;
        __syncthreads();
        before = incl - c;
        total = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const int v = tmp[w];
            before += w < wave ? v : 0;
            total += v;
        }
    };
    int before, base;
    place(mb0, s_tmp[0], before, base);
    int M = base;
    if (ntiles > 1) M += block_sum(more_cnt, s_tmp[1]);
    int q_lo, q_hi;
    if (!range(uni(M), q_lo, q_hi)) return false;      // uniform over the workgroup
    auto list = [&](uint32_t mb, int q, int s0) {
        for (; mb != 0 && q <= q_hi; ++q) {
            if (q >= q_lo) s_id[q - q_lo] = s0 + __builtin_ctz(mb);
            mb &= mb - 1;
        }
    };
    list(mb0, before, tid * 16);
    for (int t = 1; t < ntiles && base <= q_hi; ++t) {
        const uint32_t mb = selected16(P, t * kTile + tid * 16, S);
        int total;
        __syncthreads();                       // the previous user of s_tmp[1] is done
        place(mb, s_tmp[1], before, total);
        list(mb, base + before, t * kTile + tid * 16);
        base += total;
    }
    return true;
}
__device__ __forceinline__ const char *slot_row(const LogprobParams &P, int slot) {
    const int r = slot / P.L, j = slot - r * P.L;
    return P.logits + (int64_t)r * P.row_stride_b + (int64_t)j * P.pos_stride_b;
}

// A chunk's record {max, sum - 1, weighted sum} from its values, which it may overwrite; lm: this lane's
// largest value; spread: 64 values of LDS of this wave's own.  The sum's largest term is 1: without it the sum of
// the others keeps its own bits, which is all there is to a token of probability near 1.
template <int E, bool ENT>
__device__ __forceinline__ float4 chunk_record(float (&x)[kVPL][E], float &lm, float *spread) {
    lm = x[0][0];
#pragma unroll
    for (int kk = 0; kk < kVPL; ++kk) {
#pragma unroll
        for (int e = 0; e < E; ++e) lm = fmaxf(lm, x[kk][e]);
    }
    const float m = red_max_bc(lm);
    float near = m;                            // what the FMA takes off
    if (!(fabsf(m) <= kNearMax)) {             // far from 0, or no finite logit: subtract first
        near = 0.0f;
        if (m != -INFINITY) {
#pragma unroll
            for (int kk = 0; kk < kVPL; ++kk) {
#pragma unroll
                for (int e = 0; e < E; ++e) x[kk][e] -= m;
            }
        }
    }
    const float nml = -near * kLog2e;
    float s4[4] = {0.0f, 0.0f, 0.0f, 0.0f}, w4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int kk = 0; kk < kVPL; ++kk) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float y = fmaf(x[kk][e], kLog2e, nml);
            const float p = __builtin_amdgcn_exp2f(y);
            s4[e % 4] += p;
            if (ENT) w4[e % 4] = fmaf(p, fmaxf(y, kFarBelow), w4[e % 4]);
        }
    }
    const float r = fmaf(near, kLog2e, nml);   // what rounding nml added to every y
    const float back = __builtin_amdgcn_exp2f(-r);
    float s = (s4[0] + s4[1]) + (s4[2] + s4[3]), w = (w4[0] + w4[1]) + (w4[2] + w4[3]);
    const float sum = red_sum_bc(s), s1 = sum * back;
    if (s1 > 0.0f && s1 < kPeaked) {           // one element outweighs all others: add those alone
        const int owner = (int)__builtin_ctzll(__ballot(lm == m));
        const int lane = lane_id();
        if (lane == owner) {
#pragma unroll
            for (int kk = 0; kk < kVPL; ++kk) {
#pragma unroll
                for (int e = 0; e < E; ++e) spread[kk * E + e] = x[kk][e];
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const float v = lane < kVPL * E ? spread[lane] : -INFINITY;    // lane i: the owner's i-th element
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();       // read before the wave's next such chunk writes
        const int largest = (int)__builtin_ctzll(__ballot(v == near));
        const float y = fmaf(v, kLog2e, nml);
        const float p = lane == largest ? 0.0f : __builtin_amdgcn_exp2f(y);
        s = (lane == owner ? 0.0f : s) + p;
        const float others = red_sum_bc(s);
        if (ENT) w = fmaf(-r, others, red_sum_bc((lane == owner ? 0.0f : w) + p * fmaxf(y, kFarBelow))) * back;
        return make_float4(m, others * back, w, 0.0f);
    }
    // s1 - 1 is exact below 2 and off by no more than s1 itself beyond
    if (ENT) w = fmaf(-r, sum, red_sum_bc(w)) * back;
    return make_float4(m, s1 - 1.0f, w, 0.0f);
}

// Kernel 1: one record per chunk of every selected slot, and its lanes' maxima.  Bound by HBM: 1005 slots of
// 152064 bf16 (305.6 MB) take 52.5 us = 5.8 TB/s, 16384 (4.98 GB) 795 us = 6.3 TB/s; a plain read of as much
// reaches 6.4 and 7.0.  Few slots are bound by the prologue and the latency of a few chunks (192: 15.9 us, one: 5.3).
template <bool BF16, bool ENT, bool TOP>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(4))) void logprob_chunks_kernel(LogprobParams P) {
    extern __shared__ int s_id[];              // [win] selected slots of this workgroup's window
    __shared__ int s_tmp[2][kWaves];
    __shared__ int s_next;
    __shared__ float s_spread[kWaves][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = uni(tid >> 6);
    const int NC = P.NC;
    int t0 = 0, t1 = 0, q_lo = 0;              // chunk t is chunk t % NC of selected slot t / NC
    if (!list_slots(P, s_id, s_tmp, [&](int M, int &lo, int &hi) {
            const int I = M * NC, G = gridDim.x, g = blockIdx.x;
            const int per = I / G, rem = I - per * G;
            t0 = g * per + min(g, rem), t1 = t0 + per + (g < rem ? 1 : 0);
            if (t0 >= t1) return false;
            lo = q_lo = t0 / NC, hi = (t1 - 1) / NC;
            return true;
        }))
        return;
    if (tid == 0) s_next = t0 + kWaves;
    __syncthreads();

    // Wave w starts with chunk t0 + w, then takes the next untaken one.
    int t = t0 + wave;
    if (t >= t1) return;                       // no barrier follows
    constexpr int E = Fmt<BF16>::E;
    const int V = P.V, full = V / E;           // whole vectors of a row
    auto whole = [&](int c) { return min(max(full - c * kCH, 0), kCH); };
    // lane i holds the wave's i-th pending record: a store between loads would hold every later load
    // back until it completed, so records leave 64 at a time
    float4 pend = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    int pend_at = 0, npend = 0;
    int q = uni(t / NC), c = t - q * NC;
    int slot = uni(s_id[q - q_lo]);
    const char *row = slot_row(P, slot);
    u32x4 raw[kVPL];
    issue_chunk<BF16>(raw, row, c * kCH, whole(c), V);
    while (true) {
        int tn = 0;
        if (lane == 0) tn = atomicAdd(&s_next, 1);
        tn = uni(tn);
        float x[kVPL][E];
        widen<BF16>(raw, x, row, whole(c), V);
        const int at = slot * NC + c;
        const bool more = tn < t1;
        const int qn = more ? uni(tn / NC) : -1, cn = tn - qn * NC;
        if (more) {
            if (qn != q) {
                slot = uni(s_id[qn - q_lo]);
                row = slot_row(P, slot);
            }
            issue_chunk<BF16>(raw, row, cn * kCH, whole(cn), V);
        }
        float lm;
        const float4 rec = chunk_record<E, ENT>(x, lm, s_spread[wave]);
        if (TOP) {
            char *to = P.lane_max + (int64_t)at * (64 * (16 / E));
            if (BF16) ((uint16_t *)to)[lane] = (uint16_t)(__float_as_uint(lm) >> 16);
            else ((float *)to)[lane] = lm;
        }
        if (lane == npend) {
            pend = rec;
            pend_at = at;
        }
        if (++npend == 64 || !more) {
            if (lane < npend) P.partials[pend_at] = pend;
            npend = 0;
        }
        if (!more) break;
        q = qn;
        c = cn;
    }
}

// Kernel 2, without alternatives: one wave per slot.  Bound by latency (token, then its logit, beside the
// records) and, with many slots, by log(1 + r): 12.8 us for 16384 (10.2 with log S).
constexpr int kJoinWaves = 4;

struct Softmax {
    float m, ls;                               // max, log sum
    float h;                                   // entropy
};

// One wave: a slot's chunk records, each lane its own in order (the first one, record lane_id(), already
// loaded), then the lanes by a fixed tree.  A row without a finite logit has a sum of 0: its log is
// -inf, and -inf - -inf is the NaN reported.  A NaN logit makes its chunk's sum NaN, and every sum that takes
// it in, at weight 0 too.
__device__ __forceinline__ Softmax join_records(const float4 *rec, int NC, float4 p) {
    float m = -INFINITY, t = -1.0f, w = 0.0f;  // the sum of powers is 1 + t
    for (int c = lane_id(); c < NC; c += 64) {
        if (c >= 64) p = rec[c];
        const float mm = fmaxf(m, p.x);
        if (mm == -INFINITY) {                 // sums of 0, or NaN: the maximum passes over NaN
            t += 1.0f + p.y;
            w += p.z;
            continue;
        }
        const float da = fmaxf((m - mm) * kLog2e, kFarBelow), db = fmaxf((p.x - mm) * kLog2e, kFarBelow);
        const float ea = __builtin_amdgcn_exp2f(da), eb = __builtin_amdgcn_exp2f(db);
        w = ea * fmaf(da, 1.0f + t, w) + eb * fmaf(db, 1.0f + p.y, p.z);
        t = p.x > m ? fmaf(ea, 1.0f + t, p.y) : fmaf(eb, 1.0f + p.y, t);
        m = mm;
    }
    const float mw = red_max_bc(m);
    const float d = mw == -INFINITY ? 0.0f : fmaxf((m - mw) * kLog2e, kFarBelow);
    const float sc = __builtin_amdgcn_exp2f(d);
    w = red_sum_bc(sc * fmaf(d, 1.0f + t, w));
    const int owner = (int)__builtin_ctzll(__ballot(m == mw));
    t = red_sum_bc(lane_id() == owner ? t : sc * (1.0f + t));
    // Powers of 2^(log2e as a float) are powers of a base a little below e; with kLog2eShort of itself more in the
    // exponents, log S moves by that much of the mean of x - m.  (The entropy moves by as much of the variance
    // only.  A call without entropy has no such mean, its w is 0, and keeps log S as it is: high by 0.22 of 2^-24 of
    // the mean |x - m|.)  A NaN compares false and stays.
    const float ls = log1pf(t), u = kLn2 * (w / (1.0f + t)), h = ls - u;
    return {mw, fmaf(kLog2eShort, u, ls), h <= 0.0f ? 0.0f : h};
}
// The given token's column; -1 for none, or one out of range.
__device__ __forceinline__ int given_token(const LogprobParams &P, int slot) {
    if (P.tokens == nullptr) return -1;
    const int r = slot / P.L, j = slot - r * P.L;
    const int t = P.tokens[(int64_t)r * P.token_stride + j];
    return t >= 0 && t < P.V ? t : -1;
}
template <bool BF16>
__device__ __forceinline__ float logit_at(const char *row, int col) {
    return BF16 ? __uint_as_float((uint32_t)((const uint16_t *)row)[col] << 16) : ((const float *)row)[col];
}
__device__ __forceinline__ bool selected(const LogprobParams &P, int slot) {
    return P.mask[slot] != 0 && (P.exclude == nullptr || P.exclude[slot] == 0);
}
__device__ __forceinline__ void write_slot(const LogprobParams &P, int slot, const Softmax &f, int tok, float x) {
    if (P.logprob != nullptr) {
        if (tok < 0) {
            set_status(P.status, DLLM_ERR_ARG);
            ((uint32_t *)P.logprob)[slot] = 0x7FC00000u;
        } else {
            P.logprob[slot] = (x - f.m) - f.ls;
        }
    }
    if (P.entropy != nullptr) P.entropy[slot] = f.h;
    if (P.stats != nullptr) P.stats[slot] = make_float2(f.m, f.ls);
}

template <bool BF16>
__global__ __launch_bounds__(64 * kJoinWaves) void logprob_join_kernel(LogprobParams P) {
    const int slot = uni(blockIdx.x * kJoinWaves + (threadIdx.x >> 6));
    if (slot >= P.rows * P.L) return;
    fetch_args(P.mask, P.exclude, P.partials, P.tokens, P.token_stride, P.logits, P.NC);
    // all three loads go out together, for a slot that is not selected too
    const float4 *rec = P.partials + (int64_t)slot * P.NC;
    const float4 first = rec[min(lane_id(), P.NC - 1)];
    const int tok = given_token(P, slot);
    if (!selected(P, slot)) return;
    const float x = tok >= 0 ? logit_at<BF16>(slot_row(P, slot), tok) : 0.0f;
    const Softmax f = join_records(rec, P.NC, first);
    if (lane_id() == 0) write_slot(P, slot, f, tok, x);
}

// ---- alternatives of one slot, by a workgroup of WAVES ---------------------------------------------
constexpr int kTopChunks = 10;                 // chunks per wave whose maxima stay in registers
constexpr int kTopShares = 256;                // lane shares, and elements, the quick way has room for

template <int WAVES>
struct TopShared {
    int group[WAVES][64];
    int share[kTopShares];
    int2 elem[kTopShares];
    int n[2];                                  // shares, elements
    float m, ls;
};

// key_of(c): the key of this lane's largest element of chunk c; softmax(): the slot's softmax, asked of the
// last wave only, late.
template <bool BF16, int WAVES, typename KeyOf, typename SoftmaxOf>
__device__ __forceinline__ void top_of_slot(const LogprobParams &P, TopShared<WAVES> &sh, int slot, const char *row, KeyOf key_of,
                                            SoftmaxOf softmax) {
    typedef typename Row<BF16>::vec vec;
    constexpr int E = Fmt<BF16>::E, kSpan = kTopChunks * WAVES;
    const int tid = threadIdx.x, lane = lane_id(), wave = uni(tid >> 6), NC = P.NC, V = P.V, k = P.k;
    if (tid < 2) sh.n[tid] = 0;
    // Wave w holds chunks w, w + WAVES, ...  Lane l's maxima form group l; the k-th largest of the 64 group
    // maxima is a lower bound of the k-th largest element.
    int key[kTopChunks];
    auto load_keys = [&](int c0) {
#pragma unroll
        for (int i = 0; i < kTopChunks; ++i) {
            const int c = c0 + i * WAVES + wave;
            key[i] = c < NC ? key_of(c) : kNoKey;
        }
    };
    int group = kNoKey;
    for (int c0 = 0; c0 < NC; c0 += kSpan) {
        load_keys(c0);
#pragma unroll
        for (int i = 0; i < kTopChunks; ++i) group = max(group, key[i]);
    }
    sh.group[wave][lane] = group;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WAVES; ++w) group = max(group, sh.group[w][lane]);
    const int floor = kth_floor(group, k);

    // Room for `mine` entries of this thread in a shared list: one atomic per wave.
    auto room = [&](int mine, int *count) {
        const int incl = wave_incl_scan(mine);
        int at = 0;
        if (lane == 63) at = incl > 0 ? atomicAdd(count, incl) : 0;
        return __builtin_amdgcn_readlane(at, 63) + incl - mine;
    };
    // The lane shares (chunk, lane) above the bound.
    for (int c0 = 0; c0 < NC; c0 += kSpan) {
        if (NC > kSpan) load_keys(c0);
        int mine = 0;
#pragma unroll
        for (int i = 0; i < kTopChunks; ++i) mine += key[i] > floor;
        int at = room(mine, &sh.n[0]);
        if (__ballot(mine > 0) != 0) {
#pragma unroll
            for (int i = 0; i < kTopChunks; ++i) {
                if (key[i] > floor) {
                    if (at < kTopShares) sh.share[at] = (c0 + i * WAVES + wave) * 64 + lane;
                    ++at;
                }
            }
        }
    }
    __syncthreads();
    const int shares = sh.n[0];
    auto load_share = [&](int share, int kk, float (&x)[E], int &col) {
        const int v = (share >> 6) * kCH + kk * 64 + (share & 63);
        col = v * E;
        if (col + E <= V) {
            const u32x4 raw = ((const vec *)row)[v];
            unpack<BF16>(raw, x);
        } else {
            load_vec_elems<BF16>(row, min(v, P.NV), V, x);
        }
    };
    // Their elements above the bound: at least k, with few more unless many logits are equal.
    if (shares <= kTopShares) {
        for (int i0 = wave * 64; i0 < shares * kVPL; i0 += 64 * WAVES) {
            const int i = i0 + lane;
            float x[E];
            int col = V, mine = 0;
            if (i < shares * kVPL) load_share(sh.share[i / kVPL], i % kVPL, x, col);
            int ek[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                ek[e] = col + e < V ? order_key(x[e]) : kNoKey;
                mine += ek[e] > floor;
            }
            int at = room(mine, &sh.n[1]);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (ek[e] > floor) {
                    if (at < kTopShares) sh.elem[at] = make_int2(ek[e], col + e);
                    ++at;
                }
            }
        }
    }
    if (wave == WAVES - 1) {
        const Softmax f = softmax();
        if (lane == 0) {
            sh.m = f.m;
            sh.ls = f.ls;
        }
    }
    __syncthreads();
    const int elems = sh.n[1];
    const float m = sh.m, ls = sh.ls;
    if (shares <= kTopShares && elems <= kTopShares) {
        // an element's place is the number of elements before it in the full order
        if (tid < elems) {
            const int2 own = sh.elem[tid];
            int place = 0;
#pragma unroll 4
            for (int i = 0; i < elems; ++i) {
                const int2 o = sh.elem[i];
                place += o.x > own.x || (o.x == own.x && o.y < own.y);
            }
            if (place < k) {
                P.top_ids[(int64_t)slot * k + place] = own.y;
                P.top_lp[(int64_t)slot * k + place] = (key_value(own.x) - m) - ls;
            }
        }
    } else if (wave == 0) {
        // Many logits equal to the k-th: one wave inserts share after share into a list sorted across its
        // lanes.  Columns of a chunk lie above every column of the chunks before it, so once the list is
        // full a share has to exceed its last entry, and the first chunks settle it.
        Best b = {kNoKey, 0x7FFFFFFF, kNoKey};
        int cut_col = 0x7FFFFFFF;
        for (int c = 0; c < NC; ++c) {
            const bool on = key_of(c) > max(floor, b.cut);
            if (__ballot(on) == 0) continue;
#pragma unroll 1
            for (int kk = 0; kk < kVPL; ++kk) {
                float x[E];
                int col = V;
                if (on) load_share(c * 64 + lane, kk, x, col);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int ek = col + e < V ? order_key(x[e]) : kNoKey;
                    uint64_t in = __ballot(ek > floor && (ek > b.cut || (ek == b.cut && col + e < cut_col)));
                    while (in != 0) {
                        const int l = __builtin_ctzll(in);
                        const int nk = __builtin_amdgcn_readlane(ek, l), nc = __builtin_amdgcn_readlane(col + e, l);
                        insert_at(b, __popcll(__ballot(b.key > nk || (b.key == nk && b.col < nc))), nk, nc, k);
                        cut_col = __builtin_amdgcn_readlane(b.col, k - 1);
                        in &= in - 1;
                        in &= __ballot(ek > b.cut || (ek == b.cut && col + e < cut_col));
                    }
                }
            }
        }
        if (lane < k) {
            P.top_ids[(int64_t)slot * k + lane] = b.col;
            P.top_lp[(int64_t)slot * k + lane] = (key_value(b.key) - m) - ls;
        }
    }
}

// Kernel 2, with alternatives: one workgroup per slot.  Bound by latency (mask, maxima, shares, each a round trip
// behind the other, and three barriers): 6.5 us for one slot, 15.8 us for 1005 with k = 20, where 4 waves per slot
// are better than 2 (19) and 8 (17).
template <bool BF16>
__global__ __launch_bounds__(64 * kJoinWaves) void logprob_top_kernel(LogprobParams P) {
    __shared__ TopShared<kJoinWaves> sh;
    const int lane = lane_id(), slot = blockIdx.x, NC = P.NC;
    fetch_args(P.mask, P.exclude, P.partials, P.lane_max, P.tokens, P.token_stride, P.logits, P.NC, P.V, P.k);
    const int tok = given_token(P, slot);
    if (!selected(P, slot)) return;
    const char *row = slot_row(P, slot);
    const float4 *rec = P.partials + (int64_t)slot * NC;
    // the last wave also joins the records: its loads go out now, their use waits for a quiet moment
    float4 first = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float xt = 0.0f;
    if (uni(threadIdx.x >> 6) == kJoinWaves - 1) {
        first = rec[min(lane, NC - 1)];
        if (tok >= 0) xt = logit_at<BF16>(row, tok);
    }
    const char *lm = P.lane_max + (int64_t)slot * NC * (64 * (BF16 ? 2 : 4));
    top_of_slot<BF16>(
        P, sh, slot, row,
        [&](int c) {
            const int64_t at = (int64_t)c * 64 + lane;
            return order_key(BF16 ? __uint_as_float((uint32_t)((const uint16_t *)lm)[at] << 16) : ((const float *)lm)[at]);
        },
        [&]() {
            const Softmax f = join_records(rec, NC, first);
            if (lane == 0) write_slot(P, slot, f, tok, xt);
            return f;
        });
}

// ---- one kernel -----------------------------------------------------------------------------------
// For few short rows: a workgroup per slot.  Its waves take the slot's chunks in turn, keep records and lane
// maxima in LDS, and finish the slot there (the same arithmetic in the same order: the same bits), which
// saves the second launch and the mask scan.  Bound by latency: 231 slots of 20011 fp32 with k = 20 take 11.3 us.
constexpr int kShortRow = 16;                  // chunks of a row at most

template <bool BF16, bool ENT, bool TOP>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(4))) void logprob_rows_kernel(LogprobParams P) {
    __shared__ float4 s_rec[kShortRow];
    __shared__ float s_spread[kWaves][64];
    __shared__ int s_key[TOP ? kShortRow : 1][64];
    __shared__ TopShared<kWaves> sh;
    const int lane = lane_id(), wave = uni(threadIdx.x >> 6), slot = blockIdx.x;
    fetch_args(P.mask, P.exclude, P.tokens, P.token_stride, P.logits, P.row_stride_b, P.pos_stride_b, P.NC, P.V, P.k);
    const int tok = given_token(P, slot);
    if (!selected(P, slot)) return;
    const int NC = P.NC, V = P.V;
    constexpr int E = Fmt<BF16>::E;
    const int full = V / E;                    // whole vectors of the row
    auto whole = [&](int c) { return min(max(full - c * kCH, 0), kCH); };
    const char *row = slot_row(P, slot);
    const bool joins = wave == kWaves - 1;
    float xt = 0.0f;
    if (joins && tok >= 0) xt = logit_at<BF16>(row, tok);
    u32x4 raw[kVPL];
    if (wave < NC) issue_chunk<BF16>(raw, row, wave * kCH, whole(wave), V);
    for (int c = wave; c < NC; c += kWaves) {
        float x[kVPL][E];
        widen<BF16>(raw, x, row, whole(c), V);
        if (c + kWaves < NC) issue_chunk<BF16>(raw, row, (c + kWaves) * kCH, whole(c + kWaves), V);
        float lm;
        const float4 rec = chunk_record<E, ENT>(x, lm, s_spread[wave]);
        if (lane == 0) s_rec[c] = rec;
        if (TOP) s_key[c][lane] = order_key(lm);
    }
    __syncthreads();
    auto softmax = [&]() {
        const Softmax f = join_records(s_rec, NC, s_rec[min(lane, NC - 1)]);
        if (lane == 0) write_slot(P, slot, f, tok, xt);
        return f;
    };
    if (TOP) top_of_slot<BF16>(P, sh, slot, row, [&](int c) { return s_key[c][lane]; }, softmax);
    else if (joins) softmax();
}

// ---- gradient -------------------------------------------------------------------------------------
// d/dx_v of gl * logprob + gh * entropy = gl (v == token) - p_v (gl + gh (log p_v + entropy)), with
// p_v = exp(x_v - m - log S) from the forward's statistics: one read of the selected slots' logits
// and one write of every slot's gradient (zeros where a slot is not selected).  Elementwise, bound
// by HBM; per element an unpack, a subtraction, an FMA, a max, v_exp, an FMA and two multiplications (with entropy
// also an FMA) and half a pack.  A thread reads its vectors before it writes them, so the gradient
// may replace the logits in place.  1005 of 2048 slots of 152064 bf16 (0.31 GB read, 0.62 GB written) take 159 us =
// 5.85 TB/s, 512 of 126464 fp32 with entropy 88 us = 5.9 TB/s.
struct GradParams {
    const char *logits;
    int64_t pos_stride_b, row_stride_b;
    char *grad;
    int64_t gpos_stride_b, grow_stride_b;
    int32_t L, V, NV, nseg;
    const uint8_t *mask, *exclude;
    const int32_t *tokens;
    int64_t token_stride;
    const float2 *stats;
    const float *gl, *entropy, *gh;
    int32_t *status;
};
constexpr int kGradThreads = 256;
constexpr int kGradVecs = 2;                   // vectors per thread: 158 us on 64 x 32 x 152064 bf16; 1: 197, 3: 161, 4: 168

template <bool BF16, bool ENT>
__global__ __launch_bounds__(kGradThreads) void logprob_grad_kernel(GradParams P) {
    typedef typename Row<BF16>::vec vec;
    constexpr int E = Fmt<BF16>::E;
    fetch_args(P.logits, P.grad, P.mask, P.exclude, P.tokens, P.stats, P.gl, P.V, P.NV);
    const int slot = blockIdx.x / P.nseg, seg = blockIdx.x - slot * P.nseg;
    const int r = slot / P.L, j = slot - r * P.L, V = P.V;
    char *out = P.grad + (int64_t)r * P.grow_stride_b + (int64_t)j * P.gpos_stride_b;
    const int v0 = seg * kGradThreads * kGradVecs + threadIdx.x;
    const int full = V / E;
    const bool on = P.mask[slot] != 0 && (P.exclude == nullptr || P.exclude[slot] == 0);
    if (!on) {
        const u32x4 z = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < kGradVecs; ++i) {
            const int v = v0 + i * kGradThreads;
            if (v < full) {
                __builtin_nontemporal_store(z, (vec *)out + v);
            } else if (v < P.NV) {
                for (int e = v * E; e < V; ++e) {
                    if (BF16) ((uint16_t *)out)[e] = 0;
                    else ((float *)out)[e] = 0.0f;
                }
            }
        }
        return;
    }
    const char *row = P.logits + (int64_t)r * P.row_stride_b + (int64_t)j * P.pos_stride_b;
    u32x4 raw[kGradVecs];
#pragma unroll
    for (int i = 0; i < kGradVecs; ++i) {
        const int v = v0 + i * kGradThreads;
        if (v < full) raw[i] = __builtin_nontemporal_load((const vec *)row + v);
    }
    int tok = -1;
    float gl = 0.0f;
    if (P.tokens != nullptr) {
        tok = P.tokens[(int64_t)r * P.token_stride + j];
        gl = P.gl[slot];
        if (tok < 0 || tok >= V) {             // no such token: no logprob gradient
            tok = -1;
            gl = 0.0f;
            if (seg == 0 && threadIdx.x == 0) set_status(P.status, DLLM_ERR_ARG);
        }
    }
    const float2 st = P.stats[slot];
    // log2 p = (x - m - log S) log2 e = y + rest + kLog2eShort y, with y in floats and `rest` what rounding nls left, so
    // p = 2^y (c0 + c1 y).
    const float nls = -st.y * kLog2e;
    const float c0 = fmaf(kLn2, fmaf(-st.y, kLog2e, -nls), 1.0f), c1 = kLn2 * kLog2eShort;
    float a = -gl, b = 0.0f;                   // the gradient is p (a + b log2 p)
    if (ENT) {
        const float gh = P.gh[slot];
        a = -fmaf(gh, P.entropy[slot], gl);
        b = -gh * kLn2;
    }
#pragma unroll
    for (int i = 0; i < kGradVecs; ++i) {
        const int v = v0 + i * kGradThreads;
        if (v >= P.NV) continue;
        float x[E], g[E];
        if (v < full) unpack<BF16>(raw[i], x);
        else load_vec_elems<BF16>(row, v, V, x);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float y = fmaf(x[e] - st.x, kLog2e, nls), yf = fmaxf(y, kFarBelow);   // finite beside a power of 0
            const float p = __builtin_amdgcn_exp2f(y) * fmaf(yf, c1, c0);
            g[e] = p * (ENT ? fmaf(yf, b, a) : a);
        }
        if (tok >= 0 && tok / E == v) {
#pragma unroll
            for (int e = 0; e < E; ++e) g[e] += tok - v * E == e ? gl : 0.0f;
        }
        if (v < full) {
            u32x4 o;
            if (BF16) {
                o = u32x4{pack_bf16(g[0], g[1]), pack_bf16(g[2], g[3]), pack_bf16(g[E - 4], g[E - 3]), pack_bf16(g[E - 2], g[E - 1])};
            } else {
                o = u32x4{__float_as_uint(g[0]), __float_as_uint(g[1]), __float_as_uint(g[2]), __float_as_uint(g[3])};
            }
            __builtin_nontemporal_store(o, (vec *)out + v);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (v * E + e < V) {
                    if (BF16) ((uint16_t *)out)[v * E + e] = (uint16_t)pack_bf16(g[e], 0.0f);
                    else ((float *)out)[v * E + e] = g[e];
                }
            }
        }
    }
}

// ---- host -----------------------------------------------------------------------------------------
// One kernel or two: a workgroup per slot while all of them are resident at once and the rows are short.
// 231 slots of 20011 fp32: 12.7 us against 16.4; 128 of 1024: 8.2 against 10.3; but 16384 of 20011 337
// against 337, 4096 of 1024 43 against 24, one of 126464 bf16 16 against 12 (the workgroup's compute unit is
// then the limit).
bool one_kernel(int64_t S, int64_t NC, int64_t cus) { return S <= 2 * cus && NC <= kShortRow; }

constexpr int kChunksKernel = 0, kRowsKernel = 1;
template <int K, bool BF16, bool ENT, bool TOP>
constexpr auto kernel_of() {
    if constexpr (K == kRowsKernel) return logprob_rows_kernel<BF16, ENT, TOP>;
    else return logprob_chunks_kernel<BF16, ENT, TOP>;
}

// Records and lane maxima (with alternatives only) of a workspace, each part 256-byte aligned.
bool workspace_of(int32_t rows, int32_t L, int32_t V, int32_t k, int32_t dtype, int &NV, int &NC, size_t &records,
                  size_t &total) {
    if (k < 0 || k > DLLM_MAX_TOP || !shape_of(rows, L, V, dtype, NV, NC, records)) return false;
    const size_t maxima = (size_t)rows * (size_t)L * (size_t)NC * 64 * (dtype == DLLM_BF16 ? 2 : 4);
    total = records + (k > 0 ? (maxima + 255) & ~(size_t)255 : 0);
    return true;
}

// Argument checks the two entry points share.
dllm_status check_box(const char *who, const void *logits, int32_t dtype, int64_t pos_stride, int64_t row_stride,
                      int32_t rows, int32_t L, int32_t V, const uint8_t *mask, const int32_t *tokens,
                      int64_t token_stride, const int32_t *status) {
    if (dtype != DLLM_FP32 && dtype != DLLM_BF16) return fail(DLLM_ERR_DTYPE, "%s: unknown dtype %d", who, (int)dtype);
    if (rows < 0) return fail(DLLM_ERR_ARG, "%s: rows < 0", who);
    if (L < 1 || L > DLLM_MAX_L) return fail(DLLM_ERR_SHAPE, "%s: L=%d outside [1, %d]", who, L, DLLM_MAX_L);
    if (V < 1) return fail(DLLM_ERR_ARG, "%s: V < 1", who);
    if (V > 1 << 30) return fail(DLLM_ERR_SHAPE, "%s: V=%d > 2^30", who, V);   // columns plus a chunk stay in 32 bits
    if (rows > DLLM_MAX_ROWS || (int64_t)rows * L > DLLM_MAX_POSITIONS)
        return fail(DLLM_ERR_SHAPE, "%s: rows=%d, L=%d exceed the limits", who, rows, L);
    const int64_t nv = ((int64_t)V + (dtype == DLLM_BF16 ? 7 : 3)) / (dtype == DLLM_BF16 ? 8 : 4);
    if ((int64_t)rows * L * ((nv + kCH - 1) / kCH) >= (int64_t)1 << 31)
        return fail(DLLM_ERR_SHAPE, "%s: rows*L*chunks too large", who);
    if (pos_stride < V || row_stride < (int64_t)L * pos_stride)
        return fail(DLLM_ERR_ARG, "%s: strides too small (pos %lld, row %lld)", who, (long long)pos_stride,
                    (long long)row_stride);
    if (tokens && token_stride < L)
        return fail(DLLM_ERR_ARG, "%s: token stride %lld < L", who, (long long)token_stride);
    if (rows > 0 && (!logits || !mask || !status)) return fail(DLLM_ERR_ARG, "%s: null required pointer", who);
    if (((uintptr_t)logits & (dtype == DLLM_BF16 ? 1 : 3)) != 0)
        return fail(DLLM_ERR_ARG, "%s: logits not aligned to their type", who);
    return DLLM_OK;
}

}  // namespace

extern "C" size_t dllm_logprobs_workspace_bytes(int32_t rows, int32_t L, int32_t V, int32_t k, int32_t dtype) {
    int NV, NC;
    size_t records, total;
    return workspace_of(rows, L, V, k, dtype, NV, NC, records, total) ? total : 0;
}

extern "C" dllm_status dllm_logprobs(void *stream, const void *logits, int32_t dtype, int64_t pos_stride,
                                     int64_t row_stride, int32_t rows, int32_t L, int32_t V, const uint8_t *mask,
                                     const uint8_t *exclude, const int32_t *tokens, int64_t token_stride, int32_t k,
                                     float *logprob, float *entropy, float *stats, int32_t *top_ids,
                                     float *top_logprobs, void *workspace, size_t workspace_bytes, int32_t *status) {
    const char *who = "dllm_logprobs";
    dllm_status rc = check_box(who, logits, dtype, pos_stride, row_stride, rows, L, V, mask, tokens, token_stride, status);
    if (rc != DLLM_OK) return rc;
    if (k < 0 || k > DLLM_MAX_TOP || k > V)
        return fail(DLLM_ERR_ARG, "%s: k=%d outside [0, min(%d, V)]", who, k, DLLM_MAX_TOP);
    if (rows == 0) return DLLM_OK;
    if ((tokens == nullptr) != (logprob == nullptr))
        return fail(DLLM_ERR_ARG, "%s: tokens and logprob must be both given or both NULL", who);
    if (k > 0 && (!top_ids || !top_logprobs)) return fail(DLLM_ERR_ARG, "%s: k=%d without top_ids and top_logprobs", who, k);
    if (!logprob && !entropy && !stats && k == 0) return fail(DLLM_ERR_ARG, "%s: nothing to compute", who);
    if (((uintptr_t)stats & 7) != 0) return fail(DLLM_ERR_ARG, "%s: stats not 8-byte aligned", who);
    LogprobParams P{};
    size_t records, need;
    workspace_of(rows, L, V, k, dtype, P.NV, P.NC, records, need);
    if (!workspace) return fail(DLLM_ERR_ARG, "%s: null workspace", who);
    if (workspace_bytes < need) return fail(DLLM_ERR_ARG, "%s: workspace %zu bytes < %zu needed", who, workspace_bytes, need);
    if (((uintptr_t)workspace & 15) != 0) return fail(DLLM_ERR_ARG, "%s: workspace not 16-byte aligned", who);
    const int es = dtype == DLLM_BF16 ? 2 : 4;
    P.logits = (const char *)logits;
    P.pos_stride_b = pos_stride * es;
    P.row_stride_b = row_stride * es;
    P.rows = rows; P.L = L; P.V = V; P.k = k;
    P.mask = mask; P.exclude = exclude;
    P.tokens = tokens; P.token_stride = token_stride;
    P.logprob = logprob; P.entropy = entropy; P.stats = (float2 *)stats;
    P.top_ids = top_ids; P.top_lp = top_logprobs;
    P.partials = (float4 *)workspace;
    P.lane_max = (char *)workspace + records;
    P.status = status;

    const hipStream_t st = (hipStream_t)stream;
    const int64_t S = (int64_t)rows * L, cus = cu_count(), boxed = S * P.NC;
    const bool bf = dtype == DLLM_BF16, ent = entropy != nullptr, top = k > 0;
    auto pick = [&](auto go, auto kind) {
        constexpr int K = decltype(kind)::value;
        if (bf) {
            if (top) ent ? go(kernel_of<K, true, true, true>()) : go(kernel_of<K, true, false, true>());
            else ent ? go(kernel_of<K, true, true, false>()) : go(kernel_of<K, true, false, false>());
        } else {
            if (top) ent ? go(kernel_of<K, false, true, true>()) : go(kernel_of<K, false, false, true>());
            else ent ? go(kernel_of<K, false, true, false>()) : go(kernel_of<K, false, false, false>());
        }
    };
    if (one_kernel(S, P.NC, cus)) {
        pick([&](auto kernel) { hipLaunchKernelGGL(kernel, dim3((unsigned)S), dim3(kThreads), 0, st, P); },
             std::integral_constant<int, kRowsKernel>());
        return check_hip(hipGetLastError(), "dllm_logprobs launch");
    }
    // One workgroup per compute unit, whatever the box: the host does not know how many slots are selected, and
    // against two and four per unit this gains 1 to 3.5 us up to 1500 selected slots of 152064 (23.8, 24.6,
    // 26.0 us for 192; 70, 73, 75 for 1005) and loses at most 2 % beyond (16384: 809, 813, 806).  More only
    // where the list of a workgroup's slots would exceed 2048 entries.
    int64_t grid = cus;
    grid = std::max(grid, (S + 2047) / 2048);
    grid = std::min(grid, (boxed + kWaves - 1) / kWaves);
    const int64_t per = (boxed + grid - 1) / grid;
    const size_t lds = (size_t)((per + P.NC - 1) / P.NC + 2) * sizeof(int);
    pick([&](auto kernel) { hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(kThreads), lds, st, P); },
         std::integral_constant<int, kChunksKernel>());
    rc = check_hip(hipGetLastError(), "dllm_logprobs chunks launch");
    if (rc != DLLM_OK) return rc;
    if (top) {
        if (bf) hipLaunchKernelGGL(logprob_top_kernel<true>, dim3((unsigned)S), dim3(64 * kJoinWaves), 0, st, P);
        else hipLaunchKernelGGL(logprob_top_kernel<false>, dim3((unsigned)S), dim3(64 * kJoinWaves), 0, st, P);
        return check_hip(hipGetLastError(), "dllm_logprobs alternatives launch");
    }
    const dim3 jg((unsigned)((S + kJoinWaves - 1) / kJoinWaves)), jb(64 * kJoinWaves);
    if (bf) hipLaunchKernelGGL(logprob_join_kernel<true>, jg, jb, 0, st, P);
    else hipLaunchKernelGGL(logprob_join_kernel<false>, jg, jb, 0, st, P);
    return check_hip(hipGetLastError(), "dllm_logprobs join launch");
}

extern "C" dllm_status dllm_logprobs_grad(void *stream, const void *logits, int32_t dtype, int64_t pos_stride,
                                          int64_t row_stride, int32_t rows, int32_t L, int32_t V, const uint8_t *mask,
                                          const uint8_t *exclude, const int32_t *tokens, int64_t token_stride,
                                          const float *stats, const float *grad_logprob, const float *entropy,
                                          const float *grad_entropy, void *grad_logits, int64_t grad_pos_stride,
                                          int64_t grad_row_stride, int32_t *status) {
    const char *who = "dllm_logprobs_grad";
    dllm_status rc = check_box(who, logits, dtype, pos_stride, row_stride, rows, L, V, mask, tokens, token_stride, status);
    if (rc != DLLM_OK) return rc;
    if (grad_pos_stride < V || grad_row_stride < (int64_t)L * grad_pos_stride)
        return fail(DLLM_ERR_ARG, "%s: gradient strides too small (pos %lld, row %lld)", who, (long long)grad_pos_stride,
                    (long long)grad_row_stride);
    if (rows == 0) return DLLM_OK;
    if (!stats || !grad_logits) return fail(DLLM_ERR_ARG, "%s: null required pointer", who);
    if ((tokens == nullptr) != (grad_logprob == nullptr))
        return fail(DLLM_ERR_ARG, "%s: tokens and grad_logprob must be both given or both NULL", who);
    if (grad_entropy && !entropy) return fail(DLLM_ERR_ARG, "%s: grad_entropy without the forward's entropy", who);
    if (!grad_logprob && !grad_entropy) return fail(DLLM_ERR_ARG, "%s: no gradient given", who);
    if (((uintptr_t)stats & 7) != 0) return fail(DLLM_ERR_ARG, "%s: stats not 8-byte aligned", who);
    const int es = dtype == DLLM_BF16 ? 2 : 4;
    if (((uintptr_t)grad_logits & (es - 1)) != 0) return fail(DLLM_ERR_ARG, "%s: grad_logits not aligned to their type", who);
    const uintptr_t a = (uintptr_t)logits, b = (uintptr_t)grad_logits;
    const uintptr_t an = (((uintptr_t)(rows - 1) * row_stride) + (uintptr_t)(L - 1) * pos_stride + V) * es;
    const uintptr_t bn = (((uintptr_t)(rows - 1) * grad_row_stride) + (uintptr_t)(L - 1) * grad_pos_stride + V) * es;
    if (a < b + bn && b < a + an && !(a == b && pos_stride == grad_pos_stride && row_stride == grad_row_stride))
        return fail(DLLM_ERR_ARG, "%s: grad_logits overlaps logits without being it", who);
    GradParams P{};
    P.logits = (const char *)logits;
    P.pos_stride_b = pos_stride * es;
    P.row_stride_b = row_stride * es;
    P.grad = (char *)grad_logits;
    P.gpos_stride_b = grad_pos_stride * es;
    P.grow_stride_b = grad_row_stride * es;
    P.L = L; P.V = V;
    P.NV = (int)(((int64_t)V + 16 / es - 1) / (16 / es));
    P.nseg = (P.NV + kGradThreads * kGradVecs - 1) / (kGradThreads * kGradVecs);
    P.mask = mask; P.exclude = exclude;
    P.tokens = tokens; P.token_stride = token_stride;
    P.stats = (const float2 *)stats;
    P.gl = grad_logprob; P.entropy = entropy; P.gh = grad_entropy;
    P.status = status;
    const int64_t blocks = (int64_t)rows * L * P.nseg;
    if (!launchable(blocks, kGradThreads)) return fail(DLLM_ERR_SHAPE, "%s: rows*L*V too large", who);
    const dim3 grid((unsigned)blocks), block(kGradThreads);
    const hipStream_t st = (hipStream_t)stream;
    if (dtype == DLLM_BF16) {
        if (grad_entropy) hipLaunchKernelGGL((logprob_grad_kernel<true, true>), grid, block, 0, st, P);
        else hipLaunchKernelGGL((logprob_grad_kernel<true, false>), grid, block, 0, st, P);
    } else {
        if (grad_entropy) hipLaunchKernelGGL((logprob_grad_kernel<false, true>), grid, block, 0, st, P);
        else hipLaunchKernelGGL((logprob_grad_kernel<false, false>), grid, block, 0, st, P);
    }
    return check_hip(hipGetLastError(), "dllm_logprobs_grad launch");
}
