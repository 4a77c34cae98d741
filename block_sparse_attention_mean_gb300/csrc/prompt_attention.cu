// prompt_attention.cu -- attention over packed sequences, causal or not, with grouped heads (bsa_prompt_attention).
//
// 4 d multiplications and additions per visible (query, key) pair and head bound it: the tensor cores' rate, at which a
// 128 x 128 block of one head takes 2 x 512 cycles of an SM (d = 128) and its 16384 exponentials about 550.
//
//   * A tile is 128 rows of S = Q K^T: floor(128 / g) tokens of a sequence with the g query heads of one key head, loaded
//     by one TMA box, so that grouped heads share each K and V block that is fetched. One persistent CTA per SM.
//   * Two groups of four softmax warps, a thread per row, take a tile's steps in turn: a step's chain (load S, 128
//     exponentials and sums, store P) is twice as long as its products take on the tensor cores. Of the other four
//     warps one issues the Q K^T, up to three steps ahead (three S / P buffers in TMEM), one the P V; one hands out the
//     items and loads Q and K, and one loads V.
//   * Online softmax in log2, P in bf16 over S in TMEM: the running maximum of a row is raised only when a step's sum
//     passes 2^8 (the step is then done again and O rescaled). The groups share it: a step is computed with the
//     maximum as last seen; before its P is stored, each row looks at what the step before settled on (shared memory, with
//     the step's number) and the warp does the step again if that raised it. Each group sums its own steps; the one of the
//     last step adds them up. The sums are fp32. P is rounded to bf16, each weight by at most half a step (2^-8 of it), and
//     O is divided by the sum of the weights before that: summing the rounded ones too cost a third of the step's
//     instructions on the slowest path (1640 against 1020 cycles for a step's exponentials) for an error that is the same
//     but in rows of one large weight, where it doubles that of O's own rounding.
//   * Items are (sequence, key head, tile); each CTA looks at the lengths itself, or, of many sequences, a launch of one
//     CTA before does. With many items, CTAs take them from a counter: longest sequences first, a sequence's heads one
//     after another, so that K and V of the one or two in use stay in L2 (32768 tokens, 16 heads of 128: five heads in
//     use cost a quarter of the rate, two heads a sixth), and of each head the longest items first. The last heads, two
//     rounds of items of all CTAs, go together, longest items first, so that the work ends with short ones. Where that
//     would leave CTAs idle (few items, or one far above a CTA's average), all steps in a row are cut evenly over the
//     CTAs instead, and a last launch joins the parts of an item that a cut runs through, in order.
//   * What bounds it: no unit by itself. Of a 128 x 128 step's 1550 cycles (8192 causal tokens, 16 heads of 128, the tiles'
//     ends among them) the tensor cores work 66%; the path from shared memory to them, 64 KB of Q and K and 32 KB of V, is
//     taken 49% (768 cycles, as counted), beside 64 KB of K and V that come in. If both shared 128 bytes a cycle they
//     would take 1250 cycles; the counters do not show that. The rest is the chain of a step and the ends of tiles.
//     32768 causal tokens, 16 heads of 128: 2.58 to 2.62 ms in a few calls after a pause (1710 to 1680 TFLOP/s, 89% of the
//     library's rate), 2.75 to 3.1 ms in long loops of calls (1600 to 1430: the power cap); 8192: 198 us (1390). Six packed
//     sequences of 513 to 4224 tokens, 24 heads over 8: 274 to 295 us (1220 to 1140). 16384 tokens, 16 heads of 64: 490 us
//     (1120), 1070 cycles a step, of which 512 are products.
//   * 0 * NaN: a masked weight of zero still multiplies V. In steps where a mask ends, the softmax warps look through V before
//     they hand P over, a quarter of the rows each: rows behind the sequence are zeroed in shared memory, and other
//     values that are not finite too; these are then added in the epilogue to the rows that see them. Steps that every row
//     sees whole are not looked at.
//   * Every wait is bounded (BSA_ERR_TIMEOUT in the workspace, clean exit).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <math_constants.h>

#include "cache_internal.h"
#include "ptx.cuh"

namespace bsa {
namespace {

constexpr int kTileM = 128;
constexpr int kStep = 128;  // keys of a step
constexpr int kSoftmaxWarps = 8;
constexpr int kLoadWarp = 8, kQkWarp = 9, kPvWarp = 10, kValueWarp = 11;
constexpr int kRing = 4;  // items in flight
constexpr int kThreads = 12 * 32;
// registers a thread after the split: 256 * 184 + 128 * 136 = 384 * 168, what the block is launched with
constexpr int kSoftmaxRegs = 184, kOtherRegs = 136;
constexpr float kRescaleSum = 256.0f;
constexpr uint32_t kDbgStall = 1u;  // of bsa_debug_config
constexpr unsigned long long kDrainNs = 1000000000ull;  // copies and products in flight are waited for this long

constexpr int kMaxSlots = 320;       // partial results (a tile each): two per CTA
constexpr int kMaxCutItems = 65536;  // items (of all key heads) up to which the steps are cut evenly
constexpr int kCutSteps = 8;          // what a cut has to save, in steps
constexpr int kShortKeys = kCutSteps * kStep;  // no item longer than that: the steps are never cut
// At most so many sequences and tiles: each CTA's loading warp makes the plan for itself, a lane a sequence, while the
// others set up. (A launch of its own took 6 to 11 us; two launches of the call are left, one without long sequences.
// Four sequences of 12 to 128 tokens, 24 heads of 64: 8 us on the device, 15 us with a plan's launch.)
constexpr int kWarpPlan = 32, kWarpItems = 4096;
constexpr int kPlanThreads = 1024;
constexpr int kSmallPlan = 256, kSmallItems = 2048;  // sequences and items that a plan holds in shared memory

// A part of an item (or all of it) where the steps are cut evenly
struct __align__(16) Entry {
    int b, t0, kh;  // sequence, first token, key head
    int lo, hi;     // steps of 128 keys
    int slot;       // of its partial result, or -1: it is whole
    int pad[2];
};
// An item in parts, in the record of the CTA c0 whose last one is the first of them (the others are the first of the CTAs
// after it). parts 0: none.
struct __align__(16) Split {
    int q0, tokens, kh, c0, parts;  // first query (packed) and how many there are of the tile
    int pad[3];
};
__host__ __device__ constexpr int slot_of(int c0, int part) { return part == 0 ? 2 * c0 + 1 : 2 * (c0 + part); }

struct PlanHeader {  // in the workspace, behind the tickets
    uint32_t next, n_items;
    int cut;  // CTAs that the steps are cut over; 0: items come from the counter
    int pad;
};

struct Seqs {
    const int32_t *cu_q, *cu_k;
    int Tq, Tk, B, Hk, g, tpt, causal;
};

struct Seq {
    int q0, n_q, k0, n_k;
};

// Sequence b, or one without queries where it is malformed (reported)
__device__ __forceinline__ Seq seq_of(const Seqs &s, int b, uint32_t *err)
{
    Seq r;
    r.q0 = __ldg(s.cu_q + b);
    r.k0 = __ldg(s.cu_k + b);
    const int q1 = __ldg(s.cu_q + b + 1), k1 = __ldg(s.cu_k + b + 1);
    r.n_q = q1 - r.q0;
    r.n_k = k1 - r.k0;
    if (r.q0 < 0 || q1 < r.q0 || q1 > s.Tq || r.k0 < 0 || k1 < r.k0 || k1 > s.Tk) {
        raise_error(err, BSA_ERR_INVALID_ARG);
        r = Seq{0, 0, 0, 0};
    }
    return r;
}

// keys that query t of the sequence sees
__device__ __forceinline__ int visible(int causal, int n_q, int n_k, int t)
{
    return causal ? max(0, min(n_k, t + 1 + n_k - n_q)) : n_k;
}
// steps of 128 keys of tokens [t0, t0 + n) (those of them that exist)
__device__ __forceinline__ int steps_of(int causal, int n_q, int n_k, int t0, int n)
{
    if (t0 >= n_q) return 0;
    return (visible(causal, n_q, n_k, min(t0 + n, n_q) - 1) + kStep - 1) / kStep;
}
__device__ __forceinline__ int item_steps(const Seqs &s, const Seq &q, int t0)
{
    return steps_of(s.causal, q.n_q, q.n_k, t0, s.tpt);
}

// ---------------------------------------------------------------- plan

struct PlanArgs {
    Seqs s;
    int ctas;
    long long max_items;
    PlanHeader *hdr;
    int32_t *rank;         // [B] sequences, longest first
    int32_t *item0;        // [B + 1] items of the ranks before
    long long *step0;      // [B] steps of all heads of the ranks before
    int32_t *item_step0;   // [items] steps of the items before in the sequence (only where the steps are cut)
    int32_t *first;        // [CTAs + 1] first entry of a CTA
    Entry *entries;
    Split *splits;
    uint32_t *err;
};

// CTAs that the steps are cut over, or 0: with items from a counter no CTA works much longer than the average. That one
// would have whole rounds of items where all are as long, else about its share and what is left of an item at the
// end. Cutting costs about eight steps (partial results, the join), and spreads the CTAs over all heads, whose K and V then
// share L2: it has to gain an eighth of the share besides.
__device__ __forceinline__ int cut_over(long long n_items, long long steps, int longest, int ctas)
{
    const long long share = max(1ll, (steps + ctas - 1) / ctas), rounds = (n_items + ctas - 1) / ctas;
    const long long uncut = steps == n_items * longest || rounds == 1 ? rounds * longest
                                                                      : max(static_cast<long long>(longest), share + longest / 8);
    if (n_items > kMaxCutItems || 2 * ctas > kMaxSlots || uncut <= share + share / 8 + kCutSteps) return 0;
    return static_cast<int>(max(1ll, min(static_cast<long long>(ctas), steps)));
}
// The record of an item of which CTA c has the first part; `end`: the steps up to its last one
__device__ __forceinline__ Split split_of(const Seqs &s, const Seq &q, int t0, int kh, int c, long long end, long long total, int ctas)
{
    const int last = static_cast<int>((end * ctas + total - 1) / total) - 1;  // CTA of its last step
    return Split{q.q0 + t0, min(s.tpt, q.n_q - t0), kh, c, last - c + 1, {0, 0, 0}};
}

// Item `rest` of a sequence of n tiles: the last `mixed` heads tile by tile, the others head by head; last tiles first
__device__ __forceinline__ void item_of(int rest, int n, int Hk, int ctas, int tpt, int &kh, int &t0)
{
    const int mixed = min(Hk, (2 * ctas + n - 1) / n), in_order = (Hk - mixed) * n, tail = rest - in_order;
    kh = tail < 0 ? rest / n : Hk - mixed + tail % mixed;
    t0 = (n - 1 - (tail < 0 ? rest % n : tail / mixed)) * tpt;
}

// Exclusive prefix over the block's threads, and the total
__device__ __forceinline__ long long block_prefix(long long v, long long &total, long long *warp_sums)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        long long w = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xFFFFFFFFu, w, o);
            if (lane >= o) w += y;
        }
        warp_sums[lane] = w;
    }
    __syncthreads();
    total = warp_sums[31];
    const long long excl = x - v + (warp > 0 ? warp_sums[warp - 1] : 0);
    __syncthreads();
    return excl;
}

// The steps [from, to) of all items in a row, as entries of CTA c; their number, and written where `out` is given. Items
// without steps belong to the CTA that they lie in front of, or to the last one.
__device__ int walk_cut(const PlanArgs &a, int c, int ctas, long long from, long long to, long long total, Entry *out)
{
    const Seqs &s = a.s;
    // the rank and head where the range begins: the first rank at `from`, else the one that `from` is inside of
    int lo = 0, hi = s.B;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.step0[mid] >= from) hi = mid;
        else lo = mid + 1;
    }
    int r = lo, kh = 0, i = 0;
    long long at = from;  // steps in front of item i of head kh of rank r
    int skip = 0;         // steps of it that belong to the CTA before
    if (r == s.B || a.step0[r] > from) {
        --r;
        const long long head = ((r + 1 < s.B ? a.step0[r + 1] : total) - a.step0[r]) / s.Hk;  // > 0: `from` is inside
        kh = static_cast<int>((from - a.step0[r]) / head);
        const int off = static_cast<int>((from - a.step0[r]) % head);
        const int base = a.item0[r], n = a.item0[r + 1] - base;
        int l = 0, h = n;
        while (l < h) {
            const int mid = (l + h) >> 1;
            if (a.item_step0[base + mid] >= off) h = mid;
            else l = mid + 1;
        }
        i = l;
        if (i == n || a.item_step0[base + i] > off) {
            --i;
            skip = off - a.item_step0[base + i];
            at = from - skip;
        }
    }
    int count = 0;
    for (; r < s.B; ++r, kh = 0) {
        const int b = a.rank[r];
        const Seq q = seq_of(s, b, a.err);
        const int n = a.item0[r + 1] - a.item0[r];
        for (; n > 0 && kh < s.Hk; ++kh, i = 0)
            for (; i < n; ++i) {
                if (at >= to && c + 1 < ctas) return count;
                const int steps = item_steps(s, q, i * s.tpt);
                const long long end = at + steps;
                const bool more = end > to;  // it goes on in the next CTA
                if (out) {
                    Entry e{};
                    e.b = b;
                    e.t0 = i * s.tpt;
                    e.kh = kh;
                    e.lo = skip;
                    e.hi = more ? static_cast<int>(to - at) : steps;
                    e.slot = skip > 0 ? 2 * c : more ? 2 * c + 1 : -1;
                    out[count] = e;
                    if (skip == 0 && more) a.splits[c] = split_of(s, q, e.t0, kh, c, end, total, ctas);
                }
                ++count;
                if (more) return count;
                skip = 0;
                at = end;
            }
        i = 0;
    }
    return count;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs a)
{
    grid_launch_dependents();
    __shared__ long long warp_sums[32];
    __shared__ int bucket[kPlanThreads];
    __shared__ int longest;
    // small plans are made in shared memory (the attention reads rank and item0 in the workspace)
    __shared__ int s_rank[kSmallPlan], s_item0[kSmallPlan + 1], s_item_step0[kSmallItems];
    __shared__ long long s_step0[kSmallPlan];
    PlanArgs pl = a;
    if (a.s.B <= kSmallPlan) pl.rank = s_rank, pl.item0 = s_item0, pl.step0 = s_step0;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Seqs &s = a.s;
    bucket[tid] = 0;
    if (tid == 0) longest = 0;
    __syncthreads();
    // sequences by their last item's steps, longest first (counting sort; 1023 steps and more count as equal)
    auto key = [&](const Seq &q) -> int {
        if (q.n_q == 0) return kPlanThreads - 1;
        const int n = (visible(s.causal, q.n_q, q.n_k, q.n_q - 1) + kStep - 1) / kStep;
        return kPlanThreads - 1 - min(n, kPlanThreads - 1);
    };
    for (int b = tid; b < s.B; b += kPlanThreads) atomicAdd(&bucket[key(seq_of(s, b, a.err))], 1);
    __syncthreads();
    long long total;
    const int start = static_cast<int>(block_prefix(bucket[tid], total, warp_sums));
    bucket[tid] = start;
    __syncthreads();
    // placed warp by warp, in the sequences' order where the key is the same: where the steps are cut, it decides which
    // keys are summed together
    for (int b0 = 0; b0 < s.B; b0 += 32) {
        if (((b0 >> 5) & 31) == warp) {
            const int b = b0 + lane, k = b < s.B ? key(seq_of(s, b, a.err)) : -1;
            const unsigned same = __match_any_sync(0xFFFFFFFFu, k);
            if (k >= 0) pl.rank[bucket[k] + __popc(same & ((1u << lane) - 1u))] = b;
            __syncwarp();
            if (k >= 0 && (same >> lane) == 1u) bucket[k] += __popc(same);  // the last of them
        }
        __syncthreads();
    }
    // items and steps of each, and the longest item
    int most = 0;
    for (int r = warp; r < s.B; r += 32) {
        const Seq q = seq_of(s, pl.rank[r], a.err);
        const int items = (q.n_q + s.tpt - 1) / s.tpt;
        long long sum = 0;
        for (int i = lane; i < items; i += 32) {
            const int n = item_steps(s, q, i * s.tpt);
            sum += n;
            most = max(most, n);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if (lane == 0) {
            pl.item0[r] = items;
            pl.step0[r] = sum * s.Hk;
        }
    }
    atomicMax(&longest, most);
    __syncthreads();
    // exclusive sums over the ranks
    const int run = (s.B + kPlanThreads - 1) / kPlanThreads;
    const int lo = min(s.B, tid * run), hi = min(s.B, lo + run);
    long long items = 0, steps = 0, all_items, all_steps;
    for (int r = lo; r < hi; ++r) items += pl.item0[r], steps += pl.step0[r];
    items = block_prefix(items, all_items, warp_sums);
    steps = block_prefix(steps, all_steps, warp_sums);
    for (int r = lo; r < hi; ++r) {
        const int n = pl.item0[r];
        const long long m = pl.step0[r];
        pl.item0[r] = static_cast<int>(items);
        pl.step0[r] = steps;
        items += n;
        steps += m;
    }
    const bool sound = all_items <= a.max_items;  // else sequences overlap: more tokens than there are
    if (!sound) raise_error(a.err, BSA_ERR_INVALID_ARG);
    const int ctas = sound ? cut_over(all_items * s.Hk, all_steps, longest, a.ctas) : 0;
    if (pl.rank != a.rank)
        for (int r = lo; r < hi; ++r) a.rank[r] = pl.rank[r], a.item0[r] = pl.item0[r];
    if (all_items <= kSmallItems) pl.item_step0 = s_item_step0;
    if (tid == 0) {
        a.item0[s.B] = pl.item0[s.B] = sound ? static_cast<int>(all_items) : 0;
        a.hdr->next = 0u;
        a.hdr->n_items = sound ? static_cast<uint32_t>(all_items) * static_cast<uint32_t>(s.Hk) : 0u;
        a.hdr->cut = ctas;
    }
    if (!ctas) return;
    if (tid < ctas) a.splits[tid].parts = 0;
    __syncthreads();
    for (int r = warp; r < s.B; r += 32) {
        const Seq q = seq_of(s, pl.rank[r], a.err);
        const int base = pl.item0[r], n = pl.item0[r + 1] - base;
        int before = 0;
        for (int i0 = 0; i0 < n; i0 += 32) {
            const int i = i0 + lane;
            const int m = i < n ? item_steps(s, q, i * s.tpt) : 0;
            int incl = m;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
                if (lane >= o) incl += y;
            }
            if (i < n) pl.item_step0[base + i] = before + incl - m;
            before += __shfl_sync(0xFFFFFFFFu, incl, 31);
        }
    }
    __syncthreads();
    const long long from = tid < ctas ? tid * all_steps / ctas : 0, to = tid < ctas ? (tid + 1) * all_steps / ctas : 0;
    const int mine = tid < ctas ? walk_cut(pl, tid, ctas, from, to, all_steps, nullptr) : 0;
    const int at = static_cast<int>(block_prefix(mine, total, warp_sums));
    if (tid <= ctas) a.first[tid] = at;
    if (tid < ctas) walk_cut(pl, tid, ctas, from, to, all_steps, a.entries + at);
}

// ---------------------------------------------------------------- the attention

struct Params {
    Seqs s;
    float scale_log2;
    PackedView o, v;
    float *lse;
    long long max_items;
    PlanHeader *hdr;
    const int32_t *rank, *item0, *first;
    const Entry *entries;
    Split *splits;
    uint32_t *counter;  // without a plan: the next item, and CTAs that are done (both zero between calls)
    float *part_o;       // [slot][128][D]
    float2 *part_stats;  // [slot][128] (max in log2, sum)
    uint32_t *err;
    unsigned long long wait_limit_ns;
    int stall;  // load and multiply nothing: the first waits run out
};

struct Item {
    int b, t0, n_q, n_k, q0, k0, kh, lo, hi, slot;
};

template <int D>
struct Cfg {
    static constexpr int QS = D == 128 ? 2 : 3, NK = D == 128 ? 2 : 4, NV = D == 128 ? 2 : 4, NSB = 3;  // Q, K, V slots; S / P buffers
    static constexpr int kQBytes = kTileM * D * 2, kKVBytes = kStep * D * 2;
    static constexpr int kSlab = 128 * 128;  // bytes of 64 columns of 128 rows
    static constexpr int Q_OFF = 0, K_OFF = QS * kQBytes, V_OFF = K_OFF + NK * kKVBytes, BAR_OFF = V_OFF + NV * kKVBytes;
    static constexpr int B_QFULL = 0, B_QEMPTY = B_QFULL + QS, B_KFULL = B_QEMPTY + QS, B_KEMPTY = B_KFULL + NK,
                         B_VFULL = B_KEMPTY + NK, B_VEMPTY = B_VFULL + NV, B_SFULL = B_VEMPTY + NV,
                         B_PFULL = B_SFULL + NSB, B_PVDONE = B_PFULL + NSB, B_OEMPTY = B_PVDONE + NSB, B_TFULL = B_OEMPTY + 1,
                         B_TEMPTY = B_TFULL + kRing, B_SUMS = B_TEMPTY + kRing, B_DRAIN = B_SUMS + 8, NBAR = B_DRAIN + 2;
    static constexpr int MISC_OFF = (BAR_OFF + NBAR * 8 + 15) / 16 * 16;
    static constexpr int kItemWords = 12;
    static constexpr int MISC_WORDS = 2 + kRing + kRing * kItemWords;  // TMEM base, abort flag, V flags of the items, the items
    static constexpr int ROWS_OFF = (MISC_OFF + 4 * MISC_WORDS + 15) / 16 * 16;  // settled maxima [128][2], sums [2][128]
    static constexpr int SMEM = ROWS_OFF + 4 * (128 * 2 + 2 * 128);
    static constexpr int SMEM_ALLOC = SMEM + 1024;
    static constexpr uint32_t IDESC_QK = idesc_bf16_f32(kTileM, kStep, 0, 0);
    static constexpr uint32_t IDESC_PV = idesc_bf16_f32(kTileM, D, 0, 1);
    static constexpr int T_O = NSB * kStep;  // TMEM columns: the S / P buffers, then O
};

// ---- bounded waits, inlined: a kernel that moves registers between its warps calls no functions
struct Ctl {
    volatile uint32_t *abort_flag;
    uint32_t *err;
    unsigned long long limit;
};

// Waits for a barrier's phase with all lanes of a warp. False (the abort flag raised, and BSA_ERR_TIMEOUT) after `limit`
// ns, or when another warp gave up.
__device__ __forceinline__ bool warp_wait_all(uint32_t bar, uint32_t parity, const Ctl &c)
{
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) {
        const uint64_t t0 = globaltimer_ns();
        while (!(ok = mbar_try_wait_sleep(bar, parity, 50000u))) {
            if (*c.abort_flag) break;
            if (globaltimer_ns() - t0 > c.limit) {
                *c.abort_flag = 1u;
                raise_error(c.err, BSA_ERR_TIMEOUT);
                break;
            }
        }
    }
    return __all_sync(0xFFFFFFFFu, ok ? 1 : 0) != 0;
}

// For copies and products in flight on the way out: whatever the abort flag says
__device__ __forceinline__ void wait_bar_drain(uint32_t bar, uint32_t parity)
{
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait_sleep(bar, parity, 50000u))
        if (globaltimer_ns() - t0 > kDrainNs) return;
}

template <int N>
__device__ __forceinline__ void regs_up()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// The next item from the ring; false at the end or when a wait gave up
template <class C>
__device__ __forceinline__ bool fetch(uint32_t sbase, const volatile int *items, const Ctl &ctl, int lane, int &count, Item &it)
{
    const int slot = count % kRing;
    if (!warp_wait_all(sbase + C::BAR_OFF + 8u * (C::B_TFULL + slot), (count / kRing) & 1, ctl)) return false;
    const volatile int *w = items + slot * C::kItemWords;
    it.b = w[0], it.t0 = w[1], it.n_q = w[2], it.n_k = w[3], it.q0 = w[4], it.k0 = w[5], it.kh = w[6], it.lo = w[7], it.hi = w[8],
    it.slot = w[9];
    ++count;
    return it.b >= 0;
}
// ... and the slot may be written again
template <class C>
__device__ __forceinline__ void done_with(uint32_t sbase, int lane, int count)
{
    __syncwarp();
    if (lane == 0) mbar_arrive(sbase + C::BAR_OFF + 8u * (C::B_TEMPTY + (count - 1) % kRing));
}

// The plan of a warp for itself: lane r has the r-th longest sequence
struct WarpPlan {
    int b, items, n_q, n_k;     // the lane's sequence
    int item_end;               // items of the ranks up to the lane's
    long long step0, head;      // steps of all heads of the ranks before, steps of one head of this one
    uint32_t n_items;
    int cut;
    // where the steps are cut: this CTA's range, and where it is in it
    long long total, at, to;
    int r, kh, i, skip;

    __device__ __forceinline__ void make(const Params &p, int lane)
    {
        const Seqs &s = p.s;
        Seq q{0, 0, 0, 0};
        if (lane < s.B) q = seq_of(s, lane, p.err);
        const int key = q.n_q > 0 ? visible(s.causal, q.n_q, q.n_k, q.n_q - 1) : -1;
        int rank = 0, from = lane;  // lanes without a sequence come last, in order
        for (int j = 0; j < s.B; ++j) {
            const int other = __shfl_sync(0xFFFFFFFFu, key, j);
            rank += other > key || (other == key && j < lane);
        }
        for (int j = 0; j < s.B; ++j)
            if (__shfl_sync(0xFFFFFFFFu, rank, j) == lane && lane < s.B) from = j;
        b = from;
        n_q = __shfl_sync(0xFFFFFFFFu, q.n_q, from);
        n_k = __shfl_sync(0xFFFFFFFFu, q.n_k, from);
        items = (n_q + s.tpt - 1) / s.tpt;
        item_end = items;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, item_end, o);
            if (lane >= o) item_end += y;
        }
        const int all = __shfl_sync(0xFFFFFFFFu, item_end, 31);
        const bool sound = all <= p.max_items;  // else sequences overlap
        if (!sound) raise_error(p.err, BSA_ERR_INVALID_ARG);
        n_items = sound ? static_cast<uint32_t>(all) * static_cast<uint32_t>(s.Hk) : 0u;
        cut = 0;
        head = 0;
        if (s.Tk > kShortKeys && sound) {
            int longest = 0;
            for (int j = 0; j < s.B; ++j) {
                const int nq = __shfl_sync(0xFFFFFFFFu, n_q, j), nk = __shfl_sync(0xFFFFFFFFu, n_k, j), n = __shfl_sync(0xFFFFFFFFu, items, j);
                long long wide = 0;
                for (int t = lane; t < n; t += 32) {
                    const int m = steps_of(s.causal, nq, nk, t * s.tpt, s.tpt);
                    wide += m;
                    longest = max(longest, m);
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) wide += __shfl_xor_sync(0xFFFFFFFFu, wide, o);
                if (lane == j) head = wide;
            }
            longest = __reduce_max_sync(0xFFFFFFFFu, longest);
            long long end = head * s.Hk;
            step0 = end;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xFFFFFFFFu, end, o);
                if (lane >= o) end += y;
            }
            step0 = end - step0;
            total = __shfl_sync(0xFFFFFFFFu, end, 31);
            cut = cut_over(n_items, total, longest, gridDim.x);
        }
        if (blockIdx.x == 0 && lane == 0) p.hdr->cut = cut;  // for the join
        if (cut) begin_parts(p, lane);
    }

    // item `id` where they come from the counter
    __device__ __forceinline__ void item(const Params &p, int id, Item &it) const
    {
        const int of = id / p.s.Hk, j = __popc(__ballot_sync(0xFFFFFFFFu, item_end <= of));  // the first that ends behind it
        const int n = __shfl_sync(0xFFFFFFFFu, items, j), base = __shfl_sync(0xFFFFFFFFu, item_end, j) - n;
        it.b = __shfl_sync(0xFFFFFFFFu, b, j);
        it.lo = 0;
        item_of(id - base * p.s.Hk, n, p.s.Hk, gridDim.x, p.s.tpt, it.kh, it.t0);
    }

    // this CTA's range of the steps, and the item that it begins in (as walk_cut)
    __device__ __forceinline__ void begin_parts(const Params &p, int lane)
    {
        const Seqs &s = p.s;
        const int c = blockIdx.x;
        r = s.B;
        if (c >= cut) return;
        if (lane == 0) p.splits[c].parts = 0;
        const long long from = c * total / cut;
        to = (c + 1) * total / cut;
        at = from;
        kh = i = skip = 0;
        r = __popc(__ballot_sync(0xFFFFFFFFu, lane < s.B && step0 < from));  // the first rank at or behind `from`
        const long long next = __shfl_sync(0xFFFFFFFFu, step0, min(r, 31));
        if (r < s.B && next == from) return;
        --r;
        const long long off = from - __shfl_sync(0xFFFFFFFFu, step0, r), one = __shfl_sync(0xFFFFFFFFu, head, r);
        const int nq = __shfl_sync(0xFFFFFFFFu, n_q, r), nk = __shfl_sync(0xFFFFFFFFu, n_k, r), n = __shfl_sync(0xFFFFFFFFu, items, r);
        kh = static_cast<int>(off / one);
        const long long in = off - kh * one;  // steps of this head in front of `from`
        long long before = 0;
        i = n;
        for (int t0 = 0; t0 < n; t0 += 32) {
            const int m = t0 + lane < n ? steps_of(s.causal, nq, nk, (t0 + lane) * s.tpt, s.tpt) : 0;
            long long incl = m;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
                if (lane >= o) incl += y;
            }
            const unsigned reached = __ballot_sync(0xFFFFFFFFu, t0 + lane < n && before + incl - m >= in);
            if (reached) {
                i = t0 + __ffs(reached) - 1;
                before += __shfl_sync(0xFFFFFFFFu, incl - m, __ffs(reached) - 1);
                break;
            }
            before += __shfl_sync(0xFFFFFFFFu, incl, 31);
        }
        if (i == n || before > in) {  // `from` is inside the one before
            --i;
            before -= steps_of(s.causal, nq, nk, i * s.tpt, s.tpt);
            skip = static_cast<int>(in - before);
            at = from - skip;
        }
    }

    // the next part or item of this CTA, or it.b = -1
    __device__ __forceinline__ void next_part(const Params &p, int lane, Item &it)
    {
        const Seqs &s = p.s;
        const int c = blockIdx.x;
        for (;;) {
            if (r >= s.B) return;
            const int n = __shfl_sync(0xFFFFFFFFu, items, r);
            if (i < n) break;
            i = 0;
            if (n == 0 || ++kh >= s.Hk) kh = 0, ++r;
        }
        if (at >= to && c + 1 < cut) {
            r = s.B;
            return;
        }
        it.b = __shfl_sync(0xFFFFFFFFu, b, r);
        it.kh = kh;
        it.t0 = i * s.tpt;
        const Seq q = seq_of(s, it.b, p.err);
        const int steps = item_steps(s, q, it.t0);
        const long long end = at + steps;
        const bool more = end > to;
        it.lo = skip;
        it.hi = more ? static_cast<int>(to - at) : steps;
        it.slot = skip > 0 ? 2 * c : more ? 2 * c + 1 : -1;
        if (skip == 0 && more && lane == 0) p.splits[c] = split_of(s, q, it.t0, kh, c, end, total, cut);
        skip = 0;
        at = end;
        ++i;
        if (more) r = s.B;
    }
};

// first step of the item in which some row of the tile does not see all keys
__device__ __forceinline__ int first_masked(const Params &p, const Item &it)
{
    return max(it.lo, visible(p.s.causal, it.n_q, it.n_k, it.t0) / kStep);
}

// Adds what is not finite among the rows [j_lo, j_hi) of V to a row of D results (fp32 or bf16) in global memory
template <int D>
__device__ __forceinline__ void add_not_finite(const char *v, int64_t stride, int j_lo, int j_hi, char *row, bool fp32)
{
    for (int j = j_lo; j < j_hi; ++j)
        for (int c = 0; c < D; ++c) {
            const float x = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(v + j * stride)[c]);
            if ((__float_as_uint(x) & 0x7F800000u) != 0x7F800000u) continue;
            float *f = reinterpret_cast<float *>(row) + c;
            __nv_bfloat16 *h = reinterpret_cast<__nv_bfloat16 *>(row) + c;
            if (fp32) *f += x;
            else *h = __float2bfloat16(__bfloat162float(*h) + x);
        }
}

// 32 lanes x 16 columns of TMEM, as tmem_ld32
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                   "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr));
}

template <int D, class C>
__device__ __forceinline__ void softmax_role(const Params &p, uint32_t sbase, uint32_t tmem, uint32_t settled_at,
                                             volatile float *row_sums, uint8_t *queries, uint8_t *values, const volatile int *items,
                                             volatile uint32_t *vflags, const Ctl &ctl, int warp, int lane)
{
    auto bar = [&](int idx) -> uint32_t { return sbase + C::BAR_OFF + 8u * idx; };
    constexpr int NC = kStep / 32;
    const int group = warp >> 2, w4 = warp & 3;
    const int trow = w4 * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(w4 * 32) << 16;
    const uint32_t tO = tmem + lanes + C::T_O;
    const int rt = trow / p.s.g, rh = trow % p.s.g;  // token and head of the row within the tile
    int G = 0, count = 0, pairs = 0, e = 0;  // steps and items so far, items of three steps and more, of any steps
    bool lead = group == 0;  // has a tile's first step
    Item it;
    while (fetch<C>(sbase, items, ctl, lane, count, it)) {
        const int n = it.hi - it.lo, from = first_masked(p, it);
        const int tok = it.t0 + rt;
        const bool real = rt < p.s.tpt && tok < it.n_q;
        // Rows without a query hold anything and go nowhere: they are never masked (a warp with one would mask every step:
        // six packed sequences of three heads to a key head 327 us, 286 us so), their scores count as zero and so does
        // their maximum.
        const int nvis = real ? visible(p.s.causal, it.n_q, it.n_k, tok) : INT_MAX;
        const float scale = real ? p.scale_log2 : 0.0f;
        float m_run = -CUDART_INF_F;
        uint64_t acc[2] = {0ull, 0ull};
        float m_other = -CUDART_INF_F;  // the maximum that the other group's sums are relative to
        auto rescale_sums = [&](float alpha) {
            const uint64_t a2 = f2_pack(alpha, alpha);
#pragma unroll
            for (int k = 0; k < 2; ++k) acc[k] = f2_fma(acc[k], a2, 0ull);
        };
        // The group that writes the tile before out is late: the other one has the first two steps, then they take turns.
        // (With the results' way out, below: six packed sequences 287 us with steps in strict turn, 275 us so.)
        for (int i = lead ? 0 : 2; i < n; i += lead && i == 0 ? 1 : 2) {
            const int g = G + i, b = g % C::NSB;
            const uint32_t tS = tmem + lanes + b * kStep;
            if (!warp_wait_all(bar(C::B_SFULL + b), (g / C::NSB) & 1, ctl)) return;
            tc_fence_after();
            const int nv = nvis - (it.lo + i) * kStep;  // columns that the row sees
            if (__any_sync(0xFFFFFFFFu, nv < kStep)) {
                // a mask ends in this step: S is masked in place, so that the loop below (the code that counts) is short
#pragma unroll 1
                for (int c = 0; c < NC; ++c) {
                    uint32_t sv[32];
                    tmem_ld32(tS + c * 32, sv);
                    tmem_wait_ld();
                    reg_fence32(sv);
#pragma unroll
                    for (int t = 0; t < 32; ++t)
                        if (c * 32 + t >= nv) sv[t] = 0xFF800000u;
                    tmem_st32(tS + c * 32, sv);
                }
                tmem_wait_st();
            }
            auto step_max = [&]() -> float {
                float mx[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll 1
                for (int c = 0; c < NC; ++c) {
                    uint32_t sv[32];
                    tmem_ld32(tS + c * 32, sv);
                    tmem_wait_ld();
                    reg_fence32(sv);
#pragma unroll
                    for (int t = 0; t < 32; t += 8)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mx[k] = fmax3(mx[k], __uint_as_float(sv[t + 2 * k]), __uint_as_float(sv[t + 2 * k + 1]));
                }
                return fmax3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * p.scale_log2;
            };
            const uint64_t c2x = f2_pack(scale, scale);
            uint64_t sacc[2];
            uint32_t pk[NC][16];  // P, stored over S when the step's maximum is settled
            auto exps = [&](float m) {
                const float base = m == -CUDART_INF_F ? 0.0f : m;  // a row that has seen no key yet: every weight 0
                const uint64_t nm2 = f2_pack(-base, -base);
                sacc[0] = sacc[1] = 0ull;
                uint32_t sv[2][16];  // 16 columns at a time: with 32 the registers did not suffice
                tmem_ld16(tS, sv[0]);
#pragma unroll
                for (int c = 0; c < 2 * NC; ++c) {
                    tmem_wait_ld();
                    reg_fence(sv[c & 1]);
                    if (c + 1 < 2 * NC) tmem_ld16(tS + (c + 1) * 16, sv[(c + 1) & 1]);
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        float x0, x1;
                        f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[c & 1][2 * q]), __uint_as_float(sv[c & 1][2 * q + 1])), c2x, nm2),
                                  x0, x1);
                        const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
                        sacc[q & 1] = f2_add(sacc[q & 1], f2_pack(p0, p1));
                        pk[c >> 1][(c & 1) * 8 + q] = pack_bf16x2(p0, p1);
                    }
                }
            };
            // What the step before settled on for this row. Each step writes (maximum, its number plus one) in one access:
            // the number says whose it is. False where the other group's warp gave up.
            auto wait_settled = [&](float &m) -> bool {
                uint32_t tag;
                uint64_t t0 = 0ull;
                for (;;) {
                    asm volatile("ld.volatile.shared.v2.b32 {%0, %1}, [%2];" : "=f"(m), "=r"(tag) : "r"(settled_at + trow * 8) : "memory");
                    if (__all_sync(0xFFFFFFFFu, tag == static_cast<uint32_t>(g))) return true;
                    if (t0 == 0ull) t0 = globaltimer_ns();
                    else if (__any_sync(0xFFFFFFFFu, *ctl.abort_flag != 0u || globaltimer_ns() - t0 > ctl.limit)) break;
                }
                if (lane == 0 && !*ctl.abort_flag) {
                    *ctl.abort_flag = 1u;
                    raise_error(ctl.err, BSA_ERR_TIMEOUT);
                }
                return false;
            };
            auto settle = [&](float m) {
                asm volatile("st.volatile.shared.v2.b32 [%0], {%1, %2};" ::"r"(settled_at + trow * 8), "f"(m), "r"(g + 1) : "memory");
            };
            bool settled = false;  // the step before is known
            if (i == 0) {  // a new tile: its first step's maximum, known before the exponentials are
                m_run = step_max();
                if (!real) m_run = 0.0f;
                float before;
                if (!wait_settled(before)) return;
                settle(m_run);
            } else if (i <= 2) {  // the group's second or first step
                if (!wait_settled(m_run)) return;
                m_other = m_run;
                settled = true;
            }
            bool raised = false;
            for (;;) {
                exps(m_run);
                if (i == 0) break;
                if (!settled) {
                    float m_now;
                    if (!wait_settled(m_now)) return;
                    settled = true;
                    m_other = m_now;
                    if (__any_sync(0xFFFFFFFFu, m_now != m_run)) {
                        rescale_sums(m_now != m_run ? ex2_approx(m_run - m_now) : 1.0f);
                        m_run = m_now;
                        continue;
                    }
                }
                if (raised) break;
                // a step sum of at most 2^8 bounds every weight: only a larger one raises the maximum (NaN stays NaN either way);
                // and, of a row that has seen nothing but scores of -inf, any: its weights may all vanish beside the base of zero
                float s0, s1;
                f2_unpack(f2_add(sacc[0], sacc[1]), s0, s1);
                const bool raise = s0 + s1 > (m_run == -CUDART_INF_F ? -1.0f : kRescaleSum);
                if (!__any_sync(0xFFFFFFFFu, raise)) break;
                raised = true;  // the whole warp: TMEM accesses are the warp's
                const float m_all = step_max();
                const float m_step = raise ? fmaxf(m_run, m_all) : m_run;
                const float alpha = m_step != m_run ? ex2_approx(m_run - m_step) : 1.0f;
                m_run = m_step;
                rescale_sums(alpha);
                if (!warp_wait_all(bar(C::B_PVDONE + (g - 1) % C::NSB), ((g - 1) / C::NSB) & 1, ctl)) return;
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t ov[32];
                    tmem_ld32(tO + c * 32, ov);
                    tmem_wait_ld();
                    reg_fence32(ov);
#pragma unroll
                    for (int q = 0; q < 32; ++q) ov[q] = __float_as_uint(__uint_as_float(ov[q]) * alpha);
                    tmem_st32(tO + c * 32, ov);
                }
            }
            if (i > 0) settle(m_run);
            if (it.lo + i >= from) {
                // V: this warp's rows of the block
                const int s = g % C::NV;
                if (!warp_wait_all(bar(C::B_VFULL + s), (g / C::NV) & 1, ctl)) return;
                const int rows = it.n_k - (it.lo + i) * kStep - w4 * 32;  // of the 32 that are the sequence's
                uint32_t big = 0u;  // largest magnitude of either half
#pragma unroll 1
                for (int c = 0; c < D / 64; ++c) {
                    uint4 *slab = reinterpret_cast<uint4 *>(values + s * C::kKVBytes + c * C::kSlab + w4 * 32 * 128);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int at = k * 32 + lane;  // 16 bytes of row at / 8
                        if ((at >> 3) >= rows) slab[at] = make_uint4(0u, 0u, 0u, 0u);
                        const uint4 w = slab[at];
                        big = __vmaxu2(big, __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                                                     __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu)));
                    }
                }
                if (__any_sync(0xFFFFFFFFu, (big & 0xFFFFu) >= 0x7F80u || (big >> 16) >= 0x7F80u)) {
#pragma unroll 1
                    for (int c = 0; c < D / 64; ++c) {
                        uint16_t *slab = reinterpret_cast<uint16_t *>(values + s * C::kKVBytes + c * C::kSlab + w4 * 32 * 128);
#pragma unroll 1
                        for (int k = lane; k < 32 * 64; k += 32)
                            if ((slab[k] & 0x7F80u) == 0x7F80u) slab[k] = 0;
                    }
                    if (lane == 0) {
                        vflags[(count - 1) % kRing] = 1u;
                        __threadfence_block();
                    }
                }
                fence_proxy_async_smem();
            }
#pragma unroll
            for (int c = 0; c < NC; ++c) tmem_st16(tS + c * 16, pk[c]);
#pragma unroll
            for (int k = 0; k < 2; ++k) acc[k] = f2_add(acc[k], sacc[k]);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::B_PFULL + b));
        }
        float e0, e1;
        f2_unpack(f2_add(acc[0], acc[1]), e0, e1);
        float l = e0 + e1;
        // The group of the last step finishes the tile; the other one, which has steps where there are three or more, leaves
        // its sums. Two buffers with a barrier each, used in turn: it may be one such tile ahead, not two, since both have
        // steps in each and every step waits until the one before is settled. (With one barrier it could be two phases
        // ahead of a wait, which then never ends.)
        const bool finishes = n > 0 ? lead == (n == 1 || n % 2 == 0) : group == 0;
        volatile float *sum = row_sums + (pairs & 1) * 128 + trow;
        if (n >= 3 && !finishes) {
            *sum = l;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::B_SUMS + (pairs & 1) * 4 + w4));
        }
        if (finishes) {
            if (n >= 3) {
                if (!warp_wait_all(bar(C::B_SUMS + (pairs & 1) * 4 + w4), (pairs >> 1) & 1, ctl)) return;
                // its sums are relative to the maximum after the last step but one
                l += (m_other == m_run ? 1.0f : ex2_approx(m_other - m_run)) * *sum;
            }
            const bool part = it.slot >= 0;
            const int head = it.kh * p.s.g + rh;
            // Rows go out through the tile's Q, which nothing reads any more: 16 bytes a lane in, a row's 128 bytes by eight
            // lanes out. (Each lane 16 bytes of a row of its own, half a sector: an epilogue took 8000 to 11000 cycles.)
            // A quarter of a warp has the rows lane / 8, + 4, ... of the warp's; addresses are 0 for rows that do not exist.
            const unsigned long long own =
                part ? reinterpret_cast<unsigned long long>(p.part_o + (static_cast<size_t>(it.slot) * kTileM + trow) * D)
                     : real ? reinterpret_cast<unsigned long long>(p.o.p + static_cast<int64_t>(it.q0 + tok) * p.o.token + head * p.o.head)
                            : 0ull;
            uint8_t *const stage = queries + (e % C::QS) * C::kQBytes + w4 * 32 * 128;
            auto put = [&](const uint32_t (&v)[D / 2], int at) {  // this row's bytes [at, at + 2 D)
#pragma unroll
                for (int x = 0; x < D / 8; ++x)
                    *reinterpret_cast<uint4 *>(stage + (x >> 3) * C::kSlab + lane * 128 + ((x ^ lane) & 7) * 16) =
                        make_uint4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int r = k * 4 + (lane >> 3);
                    char *to = reinterpret_cast<char *>(__shfl_sync(0xFFFFFFFFu, own, r));
#pragma unroll
                    for (int x = 0; x < D / 64; ++x) {
                        const uint4 w = *reinterpret_cast<const uint4 *>(stage + x * C::kSlab + r * 128 + ((lane ^ r) & 7) * 16);
                        if (to) *reinterpret_cast<uint4 *>(to + at + x * 128 + (lane & 7) * 16) = w;
                    }
                }
                __syncwarp();
            };
            bool dirty = false;
            if (n > 0) {
                const int t = G + n - 1;
                if (!warp_wait_all(bar(C::B_PVDONE + t % C::NSB), (t / C::NSB) & 1, ctl)) return;
                tc_fence_after();
                dirty = vflags[(count - 1) % kRing] != 0u;
            }
            auto o_is_read = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::B_OEMPTY));
            };
            if (n == 0) {
                const uint4 none = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int x = 0; x < D / 8; ++x)
                    if (real) *reinterpret_cast<uint4 *>(reinterpret_cast<char *>(own) + x * 16) = none;
            } else if (part) {
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    uint32_t o[D / 2];
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t ov[16];
                        tmem_ld16(tO + half * (D / 2) + c * 16, ov);
                        tmem_wait_ld();
                        reg_fence(ov);
#pragma unroll
                        for (int q = 0; q < 16; ++q) o[c * 16 + q] = ov[q];
                    }
                    if (half == 1) o_is_read();
                    put(o, half * D * 2);
                }
            } else {
                // all of O first: the next tile's first product waits for it, and these warps are missed by the next tile's
                // steps (32768 tokens: 2666 us with loads and stores in turn, 2571 us so)
                const float inv = l != 0.0f ? 1.0f / l : 0.0f;
                uint32_t o[D / 2], ov[2][16];
                tmem_ld16(tO, ov[0]);
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                    tmem_wait_ld();
                    reg_fence(ov[c & 1]);
                    if (c + 1 < D / 16) tmem_ld16(tO + (c + 1) * 16, ov[(c + 1) & 1]);
                    else o_is_read();
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        o[c * 8 + q] = pack_bf16x2(__uint_as_float(ov[c & 1][2 * q]) * inv, __uint_as_float(ov[c & 1][2 * q + 1]) * inv);
                }
                put(o, 0);
            }
            if (n > 0) {  // the slot is the next Q's but one
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::B_QEMPTY + e % C::QS));
            }
            if (__any_sync(0xFFFFFFFFu, dirty && real)) __threadfence_block();  // the row is read back
            if (dirty && real) {
                add_not_finite<D>(p.v.p + static_cast<int64_t>(it.k0) * p.v.token + it.kh * p.v.head, p.v.token, from * kStep,
                                  min(nvis, it.hi * kStep), reinterpret_cast<char *>(own), part);
            }
            if (part) p.part_stats[static_cast<size_t>(it.slot) * kTileM + trow] = make_float2(m_run, l);
            else if (real && p.lse)
                p.lse[static_cast<int64_t>(head) * p.s.Tq + it.q0 + tok] = (m_run + log2f(l)) * 0.69314718055994530942f;
        }
        if (n >= 3) ++pairs;
        if (n > 0) lead = !finishes;
        if (n > 0) ++e;
        G += n;
        done_with<C>(sbase, lane, count);
    }
}

// PLANNED: after plan_kernel; else the loading warps plan for themselves
template <int D, bool PLANNED>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const Params p)
{
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    auto bar = [&](int idx) -> uint32_t { return sbase + C::BAR_OFF + 8u * idx; };
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + C::MISC_OFF);
    volatile uint32_t *vflags = misc + 2;
    volatile int *items = reinterpret_cast<volatile int *>(misc + 2 + kRing);
    volatile float *row_sums = reinterpret_cast<volatile float *>(smem + C::ROWS_OFF + 128 * 8);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::QS; ++s) {
            mbar_init(bar(C::B_QFULL + s), 1);
            mbar_init(bar(C::B_QEMPTY + s), 4);  // the warps that finish a tile
        }
        for (int s = 0; s < C::NK; ++s) {
            mbar_init(bar(C::B_KFULL + s), 1);
            mbar_init(bar(C::B_KEMPTY + s), 1);
        }
        for (int s = 0; s < C::NV; ++s) {
            mbar_init(bar(C::B_VFULL + s), 1);
            mbar_init(bar(C::B_VEMPTY + s), 1);
        }
        for (int b = 0; b < C::NSB; ++b) {
            mbar_init(bar(C::B_SFULL + b), 1);
            mbar_init(bar(C::B_PFULL + b), 4);
            mbar_init(bar(C::B_PVDONE + b), 1);
        }
        mbar_init(bar(C::B_OEMPTY), 4);
        for (int x = 0; x < kRing; ++x) {
            mbar_init(bar(C::B_TFULL + x), 1);
            mbar_init(bar(C::B_TEMPTY + x), kSoftmaxWarps + 3);  // softmax, Q K^T, P V, V
        }
        mbar_init(bar(C::B_DRAIN), 1);
        mbar_init(bar(C::B_DRAIN + 1), 1);
        for (int w = 0; w < 8; ++w) mbar_init(bar(C::B_SUMS + w), 1);
        misc[1] = 0u;
        fence_mbar_init();
    }
    // no step has settled on anything: step 0 looks for the number 0
    if (threadIdx.x < 256) reinterpret_cast<uint32_t *>(smem + C::ROWS_OFF)[threadIdx.x] = 0u;
    if (warp == kPvWarp) {
        tmem_alloc(smem_u32(misc), 512);
        tmem_relinquish();
    }
    if (warp == kLoadWarp && lane == 0) {
        tma_prefetch_map(&tmQ);
        tma_prefetch_map(&tmK);
        tma_prefetch_map(&tmV);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_dependency_wait();  // the plan's results are read from here on
    const uint32_t tmem = misc[0];
    const Ctl ctl{reinterpret_cast<volatile uint32_t *>(misc + 1), p.err, p.wait_limit_ns};

    if (warp < kSoftmaxWarps) {
        regs_up<kSoftmaxRegs>();
        softmax_role<D, C>(p, sbase, tmem, sbase + C::ROWS_OFF, row_sums,
                           smem + C::Q_OFF, smem + C::V_OFF, items, vflags, ctl, warp, lane);
    } else {
        regs_down<kOtherRegs>();
        if (warp == kLoadWarp) {
            // ------------------------------------------------------------ items, Q, K
            // The item after the one at hand is fetched while its first steps run.
            uint32_t n_items;
            int cut = 0, due = 0, due_end = 0;  // where the steps are cut: this CTA's entries
            WarpPlan plan;
            if constexpr (PLANNED) {  // (past L1: the plan was written while this kernel was on its way)
                n_items = __ldcg(&p.hdr->n_items);
                cut = __ldcg(&p.hdr->cut);
                if (static_cast<int>(blockIdx.x) < cut) due = __ldcg(p.first + blockIdx.x), due_end = __ldcg(p.first + blockIdx.x + 1);
            } else {
                plan.make(p, lane);
                n_items = plan.n_items;
                cut = plan.cut;
            }
            int count = 0, G = 0, e = 0;
            auto hand_out = [&](Item &it) -> bool {
                it.b = -1;
                it.slot = -1;
                if (cut && !PLANNED) {
                    plan.next_part(p, lane, it);
                } else if (cut) {
                    if (due < due_end) {
                        const int4 *en = reinterpret_cast<const int4 *>(p.entries + due++);
                        const int4 x = __ldcg(en), y = __ldcg(en + 1);
                        it.b = x.x, it.t0 = x.y, it.kh = x.z, it.lo = x.w, it.hi = y.x, it.slot = y.y;
                    }
                } else if constexpr (!PLANNED) {
                    uint32_t id = blockIdx.x;  // the first is the CTA's own
                    if (count > 0) {
                        if (lane == 0) id = gridDim.x + atomicAdd(p.counter, 1u);
                        id = __shfl_sync(0xFFFFFFFFu, id, 0);
                    }
                    if (id < n_items) plan.item(p, static_cast<int>(id), it);
                } else {
                    uint32_t id = 0u;
                    if (lane == 0) id = atomicAdd(&p.hdr->next, 1u);
                    id = __shfl_sync(0xFFFFFFFFu, id, 0);
                    if (id < n_items) {
                        // the rank: the last r with item0[r] <= id / Hk, 32 places looked at together
                        const int item = static_cast<int>(id / static_cast<uint32_t>(p.s.Hk));
                        int r = 0;
                        for (int n = p.s.B; n > 1;) {
                            const int step = (n + 31) / 32, k = r + lane * step;
                            const bool below = lane * step < n && __ldcg(p.item0 + k) <= item;
                            const int last = 31 - __clz(__ballot_sync(0xFFFFFFFFu, below));
                            r += last * step;
                            n = min(step, n - last * step);
                        }
                        const int base = __ldcg(p.item0 + r), n = __ldcg(p.item0 + r + 1) - base;
                        it.b = __ldcg(p.rank + r);
                        it.lo = 0;
                        item_of(static_cast<int>(id) - base * p.s.Hk, n, p.s.Hk, gridDim.x, p.s.tpt, it.kh, it.t0);
                    }
                }
                if (it.b >= 0) {
                    const Seq q = seq_of(p.s, it.b, p.err);
                    it.n_q = q.n_q, it.n_k = q.n_k, it.q0 = q.q0, it.k0 = q.k0;
                    if (!cut) it.hi = item_steps(p.s, q, it.t0);
                }
                const int slot = count % kRing;
                if (count >= kRing && !warp_wait_all(bar(C::B_TEMPTY + slot), ((count / kRing) - 1) & 1, ctl)) return false;
                if (lane == 0) {
                    volatile int *w = items + slot * C::kItemWords;
                    w[0] = it.b, w[1] = it.t0, w[2] = it.n_q, w[3] = it.n_k, w[4] = it.q0, w[5] = it.k0, w[6] = it.kh, w[7] = it.lo,
                    w[8] = it.hi, w[9] = it.slot;
                    vflags[slot] = 0u;
                    mbar_arrive(bar(C::B_TFULL + slot));
                }
                __syncwarp();
                ++count;
                return true;
            };
            Item it{}, next{};
            bool ok = hand_out(it);
            while (ok && it.b >= 0) {
                bool fetched = false;
                if (it.hi > it.lo && !p.stall) {
                    const int qs = e % C::QS;
                    if (e >= C::QS && !warp_wait_all(bar(C::B_QEMPTY + qs), ((e / C::QS) - 1) & 1, ctl)) break;
                    if (elect_one()) {
                        mbar_arrive_expect_tx(bar(C::B_QFULL + qs), static_cast<uint32_t>(p.s.g * p.s.tpt * D * 2));
#pragma unroll
                        for (int c = 0; c < D / 64; ++c)
                            tma_load_3d(sbase + C::Q_OFF + qs * C::kQBytes + c * C::kSlab, &tmQ, c * 64, it.kh * p.s.g, it.q0 + it.t0,
                                        bar(C::B_QFULL + qs));
                    }
                    __syncwarp();
                    ++e;
                    for (int i = it.lo; i < it.hi; ++i, ++G) {
                        const int s = G % C::NK;
                        if (G >= C::NK && !warp_wait_all(bar(C::B_KEMPTY + s), ((G / C::NK) - 1) & 1, ctl)) {
                            ok = false;
                            break;
                        }
                        if (elect_one()) {
                            mbar_arrive_expect_tx(bar(C::B_KFULL + s), C::kKVBytes);
#pragma unroll
                            for (int c = 0; c < D / 64; ++c)
                                tma_load_3d(sbase + C::K_OFF + s * C::kKVBytes + c * C::kSlab, &tmK, c * 64, it.k0 + i * kStep, it.kh,
                                            bar(C::B_KFULL + s));
                        }
                        __syncwarp();
                        if (!fetched && (i == it.lo + 1 || i + 1 == it.hi)) {
                            fetched = true;
                            if (!hand_out(next)) {
                                ++G;  // its copy is in flight
                                ok = false;
                                break;
                            }
                        }
                    }
                }
                if (ok && !fetched) ok = hand_out(next);
                it = next;
            }
            if (!PLANNED && !cut && lane == 0 && atomicAdd(p.counter + 1, 1u) == gridDim.x - 1)
                p.counter[0] = p.counter[1] = 0u;  // the last CTA; for the next call
            // after an abort: no copy of this warp is in flight when the CTA ends
            if (lane == 0 && *ctl.abort_flag) {
                for (int q = max(0, e - C::QS); q < e; ++q) wait_bar_drain(bar(C::B_QFULL + q % C::QS), (q / C::QS) & 1);
                for (int g = max(0, G - C::NK); g < G; ++g) wait_bar_drain(bar(C::B_KFULL + g % C::NK), (g / C::NK) & 1);
            }
            __syncwarp();
        } else if (warp == kValueWarp) {
            // ------------------------------------------------------------ V
            int count = 0, G = 0;
            bool ok = !p.stall;
            Item it;
            while (ok && fetch<C>(sbase, items, ctl, lane, count, it)) {
                done_with<C>(sbase, lane, count);
                for (int i = it.lo; i < it.hi; ++i, ++G) {
                    const int s = G % C::NV;
                    if (G >= C::NV && !warp_wait_all(bar(C::B_VEMPTY + s), ((G / C::NV) - 1) & 1, ctl)) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) {
                        mbar_arrive_expect_tx(bar(C::B_VFULL + s), C::kKVBytes);
#pragma unroll
                        for (int c = 0; c < D / 64; ++c)
                            tma_load_3d(sbase + C::V_OFF + s * C::kKVBytes + c * C::kSlab, &tmV, c * 64, it.k0 + i * kStep, it.kh,
                                        bar(C::B_VFULL + s));
                    }
                    __syncwarp();
                }
            }
            if (lane == 0 && *ctl.abort_flag)
                for (int g = max(0, G - C::NV); g < G; ++g) wait_bar_drain(bar(C::B_VFULL + g % C::NV), (g / C::NV) & 1);
            __syncwarp();
        } else if (warp == kQkWarp) {
            // ------------------------------------------------------------ S = Q K^T
            const uint64_t qdesc0 = sdesc_sw128(sbase + C::Q_OFF, 16, 1024), kdesc0 = sdesc_sw128(sbase + C::K_OFF, 16, 1024);
            int count = 0, G = 0, e = 0;
            bool ok = true;
            Item it;
            while (ok && !p.stall && fetch<C>(sbase, items, ctl, lane, count, it)) {
                const int n = it.hi - it.lo;
                done_with<C>(sbase, lane, count);
                if (n == 0) continue;
                const int qs = e % C::QS;
                if (!warp_wait_all(bar(C::B_QFULL + qs), (e / C::QS) & 1, ctl)) break;
                const uint64_t qd = qdesc0 + static_cast<uint64_t>(qs * (C::kQBytes >> 4));
                for (int i = 0; i < n; ++i, ++G) {
                    const int s = G % C::NK, b = G % C::NSB;
                    if (!warp_wait_all(bar(C::B_KFULL + s), (G / C::NK) & 1, ctl) ||
                        (G >= C::NSB && !warp_wait_all(bar(C::B_PVDONE + b), ((G / C::NSB) - 1) & 1, ctl))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t kd = kdesc0 + static_cast<uint64_t>(s * (C::kKVBytes >> 4));
                    __syncwarp();
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint64_t off = static_cast<uint64_t>(((kk >> 2) * C::kSlab + (kk & 3) * 32) >> 4);
                            mma_ss(tmem + b * kStep, qd + off, kd + off, C::IDESC_QK, kk > 0 ? 1u : 0u);
                        }
                        tc_commit(bar(C::B_SFULL + b));
                        tc_commit(bar(C::B_KEMPTY + s));
                    }
                    __syncwarp();
                }
                ++e;
            }
            // all products of the elected lane have completed before TMEM is freed
            __syncwarp();
            if (elect_one()) {
                tc_commit(bar(C::B_DRAIN));
                wait_bar_drain(bar(C::B_DRAIN), 0);
            }
            __syncwarp();
        } else {
            // ------------------------------------------------------------ O += P V
            const uint64_t vdesc0 = sdesc_sw128(sbase + C::V_OFF, C::kSlab, 1024);
            int count = 0, G = 0, e = 0;
            bool ok = true;
            Item it;
            while (ok && !p.stall && fetch<C>(sbase, items, ctl, lane, count, it)) {
                const int n = it.hi - it.lo;
                done_with<C>(sbase, lane, count);
                for (int i = 0; i < n; ++i, ++G) {
                    const int s = G % C::NV, b = G % C::NSB;
                    // the first product of a tile overwrites O: the tile before has been read
                    if (!warp_wait_all(bar(C::B_VFULL + s), (G / C::NV) & 1, ctl) ||
                        (i == 0 && e >= 1 && !warp_wait_all(bar(C::B_OEMPTY), (e - 1) & 1, ctl)) ||
                        !warp_wait_all(bar(C::B_PFULL + b), (G / C::NSB) & 1, ctl)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t vd = vdesc0 + static_cast<uint64_t>(s * (C::kKVBytes >> 4));
                    __syncwarp();
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < kStep / 16; ++kk)
                            mma_ts(tmem + C::T_O, tmem + b * kStep + kk * 8, vd + static_cast<uint64_t>(kk * (16 * 128 >> 4)),
                                   C::IDESC_PV, i == 0 && kk == 0 ? 0u : 1u);
                        tc_commit(bar(C::B_PVDONE + b));
                        tc_commit(bar(C::B_VEMPTY + s));
                    }
                    __syncwarp();
                }
                if (n > 0) ++e;
            }
            __syncwarp();
            if (elect_one()) {
                tc_commit(bar(C::B_DRAIN + 1));
                wait_bar_drain(bar(C::B_DRAIN + 1), 0);
            }
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kPvWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- joining the parts

struct JoinArgs {
    Seqs s;
    PackedView o;
    float *lse;
    const PlanHeader *hdr;
    const Split *splits;
    const float *part_o;
    const float2 *part_stats;
};

// A warp per row, or, where there are no more rows than CTAs, a CTA: its warps take a share of the
// parts each, as the loads' latency is all there is then (16 queries over 31,760 keys in parts of
// 38 CTAs: 35 -> 24.5 us for the call).  O = sum w_k O_k / sum w_k l_k, LSE = ln2 (M + log2 sum w_k l_k), w_k = 2^(m_k - M)
template <int D>
__global__ void __launch_bounds__(256) join_kernel(const JoinArgs a)
{
    constexpr int V = D / 32;  // channels of a lane
    grid_dependency_wait();
    __shared__ float share[8][32][V + 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // the CTAs' records that hold an item in parts, as bits
    const int ctas = __ldcg(&a.hdr->cut);
    unsigned held[kMaxSlots / 2 / 32];
    int rows = 0;
#pragma unroll
    for (int w = 0; w < kMaxSlots / 2 / 32; ++w) {
        const int c = w * 32 + lane;
        held[w] = __ballot_sync(0xFFFFFFFFu, c < ctas && __ldcg(&a.splits[c].parts) > 0);
        rows += __popc(held[w]) * kTileM;
    }
    const bool wide = rows <= static_cast<int>(gridDim.x);
    const int stride = static_cast<int>(gridDim.x) * (wide ? 1 : 8);
    for (int i = wide ? blockIdx.x : blockIdx.x * 8 + warp; i < rows; i += stride) {
        const int trow = i % kTileM;
        int nth = i / kTileM, c = 0;
#pragma unroll
        for (int w = 0; w < kMaxSlots / 2 / 32; ++w) {
            // the lane whose bit is the nth of this word, where the word has so many
            const unsigned bit = 1u << lane;
            const unsigned here = __ballot_sync(0xFFFFFFFFu, (held[w] & bit) && __popc(held[w] & (bit - 1)) == nth);
            if (here) c = w * 32 + __ffs(here) - 1;
            nth -= __popc(held[w]);
        }
        const int4 *record = reinterpret_cast<const int4 *>(a.splits + c);
        const int4 sp = __ldcg(record);  // q0, tokens, kh, c0
        const int parts = __ldcg(record + 1).x;
        const int rt = trow / a.s.g, rh = trow % a.s.g;
        if (rt >= sp.y) continue;
        auto row_of = [&](int part) { return static_cast<size_t>(slot_of(sp.w, part)) * kTileM + trow; };
        float M = -CUDART_INF_F, L = 0.0f, out[V];
#pragma unroll
        for (int c = 0; c < V; ++c) out[c] = 0.0f;
        const int each = wide ? (parts + 7) / 8 : parts, begin = wide ? warp * each : 0;
        const int end = min(begin + each, parts);
        for (int k0 = begin; k0 < end; k0 += 32) {
            // 32 parts' statistics at a time, a lane each; then their rows, 16 loads in flight
            float2 st = make_float2(-CUDART_INF_F, 0.0f);
            if (k0 + lane < end) st = __ldcg(a.part_stats + row_of(k0 + lane));
            float m = st.x;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            m = fmaxf(m, M);
            const float old = m == M ? 1.0f : ex2_approx(M - m), w = st.x == m ? 1.0f : ex2_approx(st.x - m);
            M = m;
            float l = k0 + lane < end ? w * st.y : 0.0f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
            L = L * old + l;
#pragma unroll
            for (int c = 0; c < V; ++c) out[c] *= old;
            const int n = min(32, end - k0);
            for (int j0 = 0; j0 < n; j0 += 16) {
                float v[16][V];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float *src = a.part_o + row_of(k0 + min(j0 + j, n - 1)) * D + lane * V;
                    if constexpr (V == 4) {
                        const float4 x = __ldcg(reinterpret_cast<const float4 *>(src));
                        v[j][0] = x.x, v[j][1] = x.y, v[j][2] = x.z, v[j][3] = x.w;
                    } else {
                        const float2 x = __ldcg(reinterpret_cast<const float2 *>(src));
                        v[j][0] = x.x, v[j][1] = x.y;
                    }
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float wj = __shfl_sync(0xFFFFFFFFu, w, min(j0 + j, 31));
                    if (j0 + j >= n) break;
#pragma unroll
                    for (int c = 0; c < V; ++c) out[c] = fmaf(wj, v[j][c], out[c]);
                }
            }
        }
        if (wide) {
            share[warp][lane][0] = M, share[warp][lane][1] = L;
#pragma unroll
            for (int c = 0; c < V; ++c) share[warp][lane][2 + c] = out[c];
            __syncthreads();
            if (warp != 0) return;  // a CTA has one row
            for (int k = 0; k < 8; ++k) M = fmaxf(M, share[k][lane][0]);
            L = 0.0f;
#pragma unroll
            for (int c = 0; c < V; ++c) out[c] = 0.0f;
            for (int k = 0; k < 8; ++k) {
                const float m = share[k][lane][0], w = m == M ? 1.0f : ex2_approx(m - M);
                L += w * share[k][lane][1];
#pragma unroll
                for (int c = 0; c < V; ++c) out[c] = fmaf(w, share[k][lane][2 + c], out[c]);
            }
        }
        const float inv = L != 0.0f ? 1.0f / L : 0.0f;
        const int head = sp.z * a.s.g + rh;
        char *dst = a.o.p + static_cast<int64_t>(sp.x + rt) * a.o.token + head * a.o.head + lane * V * 2;
        if constexpr (V == 4)
            *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(out[0] * inv, out[1] * inv), pack_bf16x2(out[2] * inv, out[3] * inv));
        else
            *reinterpret_cast<uint32_t *>(dst) = pack_bf16x2(out[0] * inv, out[1] * inv);
        if (lane == 0 && a.lse)
            a.lse[static_cast<int64_t>(head) * a.s.Tq + sp.x + rt] = (M + log2f(L)) * 0.69314718055994530942f;
    }
}

// ---------------------------------------------------------------- host

struct Layout {
    size_t hdr, rank, item0, step0, item_step0, first, entries, splits, stats, part, total;
    int64_t max_items;
};

int tokens_per_tile(int H, int Hk) { return kTileM / (H / Hk); }

Layout layout_of(int T, int B, int H, int Hk, int d)
{
    Layout l;
    l.max_items = T / tokens_per_tile(H, Hk) + static_cast<int64_t>(B);
    const int64_t cut_items = l.max_items * Hk < kMaxCutItems ? l.max_items * Hk : kMaxCutItems;
    const int64_t max_entries = cut_items + kMaxSlots;  // an item has an entry in each CTA that it is part of: one more per cut
    size_t at = kCacheScratch;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at = align_up(at + bytes, 256);
        return here;
    };
    l.hdr = take(sizeof(PlanHeader));
    l.rank = take(sizeof(int32_t) * static_cast<size_t>(B));
    l.item0 = take(sizeof(int32_t) * (static_cast<size_t>(B) + 1));
    l.step0 = take(sizeof(long long) * static_cast<size_t>(B));
    l.item_step0 = take(sizeof(int32_t) * static_cast<size_t>(cut_items));
    l.first = take(sizeof(int32_t) * (kMaxSlots / 2 + 1));
    l.entries = take(sizeof(Entry) * static_cast<size_t>(max_entries));
    l.splits = take(sizeof(Split) * (kMaxSlots / 2));
    l.stats = take(sizeof(float2) * kTileM * kMaxSlots);
    l.part = take(sizeof(float) * kTileM * static_cast<size_t>(d) * kMaxSlots);
    l.total = at - kCacheScratch;
    return l;
}

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled find_encode_tiled()
{
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
        return nullptr;
    return reinterpret_cast<EncodeTiled>(fn);
}

// {channel, head, token} of Q, or {channel, token, head} of K and V: 64 channels x n1 x n2 boxes, 128-byte swizzle
bool make_map(CUtensorMap *m, const PackedView &t, int d, uint64_t n1, int64_t s1, uint64_t n2, int64_t s2, uint32_t box1, uint32_t box2)
{
    static const EncodeTiled fn = find_encode_tiled();
    if (!fn) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), n1, n2};
    const cuuint64_t strides[2] = {n1 > 1 ? static_cast<cuuint64_t>(s1) : static_cast<cuuint64_t>(d) * 2,
                                   n2 > 1 ? static_cast<cuuint64_t>(s2) : static_cast<cuuint64_t>(d) * 2};
    const cuuint32_t box[3] = {64u, box1, box2}, es[3] = {1u, 1u, 1u};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, t.p, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool PLANNED>
bsa_status launch(const PromptArgs &a, cudaStream_t st)
{
    using C = Cfg<D>;
    static_assert(C::SMEM_ALLOC <= 227 * 1024, "shared memory");
    static_assert(C::T_O + D <= 512, "TMEM columns");
    int sms = 0;
    const bsa_status s = current_sm_count(&sms);
    if (s != BSA_OK) return s;
    auto kern = prompt_kernel<D, PLANNED>;
    static std::atomic<uint64_t> ready{0};
    if (!allow_shared_memory(kern, C::SMEM_ALLOC, ready)) return BSA_ERR_CUDA;
    // setmaxnreg hands out what the block was launched with: with fewer registers the split would wait for ever
    static const bool split_fits = [&] {
        cudaFuncAttributes f;
        return cudaFuncGetAttributes(&f, kern) == cudaSuccess &&
               f.numRegs * kThreads >= kSoftmaxWarps * 32 * kSoftmaxRegs + (kThreads - kSoftmaxWarps * 32) * kOtherRegs;
    }();
    if (!split_fits) return BSA_ERR_UNSUPPORTED;
    const Layout l = layout_of(a.Tq, a.B, a.H, a.Hk, a.d);
    const int g = a.H / a.Hk, tpt = tokens_per_tile(a.H, a.Hk);
    CUtensorMap mq, mk, mv;
    // without keys no step is loaded: any tensor does in their place
    const bool keys = a.Tk > 0;
    if (!make_map(&mq, a.q, D, a.H, a.q.head, a.Tq, a.q.token, g, tpt) ||
        !make_map(&mk, keys ? a.k : a.q, D, keys ? a.Tk : 1, a.k.token, keys ? a.Hk : 1, a.k.head, kStep, 1) ||
        !make_map(&mv, keys ? a.v : a.q, D, keys ? a.Tk : 1, a.v.token, keys ? a.Hk : 1, a.v.head, kStep, 1))
        return BSA_ERR_CUDA;
    const Seqs seqs{a.cu_q, a.cu_k, a.Tq, a.Tk, a.B, a.Hk, g, tpt, a.causal != 0};
    uint32_t *err = reinterpret_cast<uint32_t *>(a.ws);
    PlanHeader *hdr = reinterpret_cast<PlanHeader *>(a.ws + l.hdr);
    PlanArgs pa;
    pa.s = seqs;
    pa.ctas = sms;
    pa.max_items = l.max_items;
    pa.hdr = hdr;
    pa.rank = reinterpret_cast<int32_t *>(a.ws + l.rank);
    pa.item0 = reinterpret_cast<int32_t *>(a.ws + l.item0);
    pa.step0 = reinterpret_cast<long long *>(a.ws + l.step0);
    pa.item_step0 = reinterpret_cast<int32_t *>(a.ws + l.item_step0);
    pa.first = reinterpret_cast<int32_t *>(a.ws + l.first);
    pa.entries = reinterpret_cast<Entry *>(a.ws + l.entries);
    pa.splits = reinterpret_cast<Split *>(a.ws + l.splits);
    pa.err = err;
    Params p;
    p.s = seqs;
    p.scale_log2 = a.scale * 1.44269504088896340736f;
    p.o = a.o;
    p.v = a.v;
    p.lse = a.lse;
    p.max_items = l.max_items;
    p.hdr = hdr;
    p.rank = pa.rank;
    p.item0 = pa.item0;
    p.first = pa.first;
    p.entries = pa.entries;
    p.splits = pa.splits;
    p.counter = reinterpret_cast<uint32_t *>(a.ws + kCacheCounter);
    p.part_o = reinterpret_cast<float *>(a.ws + l.part);
    p.part_stats = reinterpret_cast<float2 *>(a.ws + l.stats);
    p.err = err;
    p.wait_limit_ns = a.wait_limit_ns;
    p.stall = (a.dbg_flags & kDbgStall) != 0u;
    if constexpr (PLANNED) {
        plan_kernel<<<1, kPlanThreads, 0, st>>>(pa);
        if (cudaGetLastError() != cudaSuccess) return BSA_ERR_CUDA;
        if (!pdl_launch(kern, dim3(static_cast<unsigned>(sms)), kThreads, C::SMEM_ALLOC, st, mq, mk, mv, p)) return BSA_ERR_CUDA;
    } else {
        // all SMs where steps may be cut, else no more than there can be items
        const int64_t items = l.max_items * a.Hk;
        const int ctas = a.Tk > kShortKeys || items > sms ? sms : static_cast<int>(items);
        kern<<<static_cast<unsigned>(ctas), kThreads, C::SMEM_ALLOC, st>>>(mq, mk, mv, p);
        if (cudaGetLastError() != cudaSuccess) return BSA_ERR_CUDA;
    }
    if (a.Tk <= kShortKeys) return BSA_OK;  // nothing is cut
    const JoinArgs ja{seqs, a.o, a.lse, hdr, pa.splits, p.part_o, p.part_stats};
    if (!pdl_launch(join_kernel<D>, dim3(static_cast<unsigned>(4 * sms)), 256, 0, st, ja)) return BSA_ERR_CUDA;
    return BSA_OK;
}

}  // namespace

size_t prompt_workspace(int T, int B, int H, int Hk, int d) { return layout_of(T, B, H, Hk, d).total; }

bsa_status launch_prompt_attention(const PromptArgs &a, cudaStream_t st)
{
    const bool planned = a.B > kWarpPlan || layout_of(a.Tq, a.B, a.H, a.Hk, a.d).max_items > kWarpItems;
    if (a.d == 128) return planned ? launch<128, true>(a, st) : launch<128, false>(a, st);
    return planned ? launch<64, true>(a, st) : launch<64, false>(a, st);
}

}  // namespace bsa
