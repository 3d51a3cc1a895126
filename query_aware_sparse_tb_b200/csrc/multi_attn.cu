// Attention of several new tokens per sequence over the KV cache: packed
// prompts (or chunks of prompts) with a causal mask, and trees of drafted
// tokens with an ancestor mask.  One kernel serves both: the masks differ in
// the last few tiles only.
//
// For token i of sequence b (n new tokens, length T counting them, so token i
// sits at cache row T - n + i) and query head h of KV head g = h / G:
//
//   out = sum_t p_t v_t / sum_t p_t,   p_t = 2^(c q.k_t - m),  c = scale * log2(e)
//
// over t <= T - n + i (prompt), or t < T - n and the drafted rows whose bit is
// set (tree).  m is a running reference, not the exact maximum: it is raised
// only when a logit exceeds it by more than 32 (log2 units), so the accumulator
// is rescaled rarely; p stays below 2^32 and the sums, held in fp32, are exact
// up to fp32 rounding either way.
//
// Work item: 256 rows of one KV head, a row being (token, head of the group),
// so the G heads of a group share every K and V tile.  A CTA has two slots of
// 128 rows, each with its own softmax warpgroup (thread = row), S/P and O
// accumulators in tensor memory.  While one slot's softmax runs, the tensor
// cores work for the other.  An item of at most 128 rows instead gives both
// slots the same rows and every other K/V tile (the slots' states are merged
// at the end), so short items keep both warpgroups busy too.
//
// Warps: 0-3 softmax of slot 0, 4-7 softmax of slot 1, 8 issues the products,
// 9 loads (TMA), 10 schedules, 11 looks over the V tiles that are masked for
// some rows.  These four need few registers; the softmax warps take the rest
// (a softmax thread holds a whole row of a tile, 128 logits).  Tensor memory:
// S0 | S1 | O0 | O1, 128 columns each; the weights P (bf16) overwrite the first
// half of their S columns (at 64 head dims they have columns of their own) and
// are read from there as the A operand of the second product.
//
// The grid is one CTA per SM, each working through a list of segments (an item
// or a part of its K/V tiles) that warp 10 describes to the other warps one
// segment ahead, so the next segment's loads and first products overlap the
// end of the current one.  Two ways to deal the work out, chosen on the host:
//   - many items: a counter, longest items of each sequence first;
//   - few items over long contexts: all tiles of all items in one line, cut
//     into equal shares.  A CTA's share may begin and end inside an item; such
//     parts leave their rows' unnormalised state in the workspace and a second
//     kernel joins them.
//
// What bounds it, on a B200 (32 query heads, 8 KV heads, 128 head dims):
//   - long prompts: the tensor cores and the power they draw.  A tile of 256
//     rows x 128 keys is 2,048 cycles of products and takes about 3,100, the
//     rest being the latency of the chain S, softmax, PV within a slot; 32K
//     tokens run 6.7 ms from a cold GPU (1,310 TFLOP/s) and 7.6 to 7.7 ms once
//     the power cap holds the clock near 1.55 GHz (1,145 TFLOP/s; a plain bf16
//     matrix product does 1,400 there).
//   - 64 head dims: the waits between softmax and products.  The products are
//     half as long, the exponentials as many; the exponential unit is 70 % busy
//     and the tensor cores 35 %: 730 TFLOP/s for ragged prompts of 0.5K to 5K.
//   - trees and single tokens over long contexts: HBM first.  26 drafted tokens
//     over 64K rows (269 MB, 41 us at the copy rate) take 59 to 60 us back to
//     back.  Without the join it is 6 less; the rest is the start of the work,
//     its ragged end and the writing of 10 MB of states.
#include <cuda.h>
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "multi.h"

namespace tb {
namespace {

constexpr int kSlotRows = 128;              // rows of a slot = MMA M = TMEM lanes
constexpr int kItemRows = 2 * kSlotRows;
constexpr int kTile = 128;                  // K/V rows per tile
constexpr int kThreads = 384;
// Registers a thread: 168 at launch (384 threads fill the file); the third
// warpgroup gives most of its share to the two softmax warpgroups
// (2 * 128 * 216 + 128 * 72 = 384 * 168).
constexpr int kRegsSoftmax = 216, kRegsOther = 72;
static_assert(256 * kRegsSoftmax + 128 * kRegsOther <= kThreads * 168, "register split");
constexpr uint32_t kTmemCols = 512;
// How far (log2 units) a logit may exceed the reference m before m is raised.
// A raise rescales the sums in tensor memory, about 1,000 cycles a tile, and
// with a few large keys in the context some row of 32 wants one in most of the
// first tiles.  Weights up to 2^32 lose nothing, bf16 and fp32 having the same
// exponents; the sums (weights x 2^22 rows x |v|) stay finite to |v| of 2^72.
// At 8 an 8K prompt with 1% of its keys scaled by 4 took 540 us, at 32 505.
constexpr float kLazy = 32.0f;
constexpr uint32_t kFullMask = 0xffffffffu;

// Masked tiles of an item: its new tokens' rows (1024 at most for a tree, 256
// for a prompt) and a ragged end on either side.  A list entry is the tile and
// a bit for each of its 128 rows; entry 0 holds the count.
constexpr int kMaxMasked = 10, kBadBytes = 4 + 20 * kMaxMasked;

template <int D>
struct Lay {
    static constexpr int kAtoms = D / 64;
    static constexpr int kOperand = 128 * D * 2;  // bytes of a 128-row operand (Q slot, K or V tile)
    // Tensor memory columns of slot s: S at 128 s.  At 64 head dims the sums
    // leave room for P beside S, so the next S can be worked out while the
    // softmax of the current one runs; at 128 P overwrites its S.
    static constexpr bool kSepP = D == 64;
    static constexpr uint32_t kO = 256, kOStep = D, kP = kSepP ? 384 : 0, kPStep = kSepP ? 64 : 128;
    // K and V tiles share one ring: 160 KB in flight covers the latency of HBM
    static constexpr int kStages = D == 128 ? 5 : 10;
    static constexpr int kRing = 2 * kOperand;
    static constexpr int kBar = kRing + kStages * kOperand;
    static constexpr int kNumBars = 2 * kStages + 38;
    static constexpr int kMisc = kBar + kNumBars * 8;       // TMEM base, abort flag
    static constexpr int kSeg = (kMisc + 8 + 15) / 16 * 16; // two segment descriptions
    static constexpr int kBad = kSeg + 2 * 64;              // two lists of V rows taken out of the product
    static constexpr int kState = kBad + 2 * kBadBytes;     // the slots' m and l [2 slots][2][128]
    static constexpr int kBytes = kState + 2048;
    static_assert(kBar % 8 == 0, "mbarrier alignment");
    static_assert(kBytes <= 227 * 1024, "shared memory");
};

// A bounded mbarrier wait that also gives up as soon as another role of the
// CTA has given up.  The thread sleeps in the barrier between checks.
__device__ __forceinline__ bool wait_role(uint32_t bar, uint32_t parity, volatile int *abort_flag, uint32_t *flags) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    for (;;) {
        if (mbar_try_wait_sleep(bar, parity, 20000u)) return true;
        if (*abort_flag) return false;
        if (clock64() - t0 > kWaitBudgetCycles) {
            raise_flag(flags, TB_FLAG_TIMEOUT);
            *abort_flag = 1;
            return false;
        }
    }
}

// One lane of the calling (converged) warp.  Unlike a test of the lane number
// it tells the compiler that the branch is taken by one thread of a uniform
// warp, so operands of the instructions inside stay in uniform registers: with
// `lane == 0` eight products took about 850 cycles to issue, with this less
// than they take to run (8 x 64).
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(r));
    return r != 0;
}

// wait_role by a whole warp: one answer for all lanes.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int *abort_flag, uint32_t *flags) {
    return __all_sync(kFullMask, wait_role(bar, parity, abort_flag, flags));
}

// What a row's c and m are multiplied by for its weights 2^(s c - m): 1, and from
// |m| = 2^30 on the power of two that brings m below that.  m is a rounded
// product s_ref c and the fused s c - m keeps its rounding error as a common
// factor of the row's weights: no error, but 2^64 for |m| at 2^30, and past
// 2^31 the weights of whole rows were 0 or infinite.  Scaled, the factor stays
// within 2^32, and no weight that counts changes: logits that differ do so by
// 2^5 or more as scaled, by a multiple of that in truth, so all but the ones
// equal to the largest have weights below 2^-32 either way.  (To take s_ref off
// each logit first is 64 to 128 instructions more beside the path of the raise:
// a tree over 64K 59.0 -> 60.5 to 61.7 us; with the factor 59.3.)
__device__ __forceinline__ float row_factor(float m) {
    const int e = (__float_as_int(m) >> 23) & 0xff;
    return m == -INFINITY ? 1.f : __int_as_float((127 - max(0, e - (127 + 29))) << 23);
}

// bits 0 .. n-1 set (n clamped to [0, 32])
__device__ __forceinline__ uint32_t bits_below(int n) {
    return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Pairs of fp32 in a 64-bit register: one instruction works on both.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// The largest of three; NaN if one of them is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// two fp32 -> packed bf16 (round to nearest even), `lo` in the low half
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];\n" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// The two products' tcgen05.mma, issued by one thread.  Of a shared-memory
// descriptor only the low word varies (start address; the leading byte offset
// is the same for every operand here), so the callers step 32-bit words.
// D(tmem) (+)= A(smem) * B(smem)^T, both K-major.
__device__ __forceinline__ void umma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %3};\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
        : "memory");
}
// D(tmem) (+)= A(tmem) * B(smem), B MN-major.
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
        : "memory");
}

#define TB_O4(v, o) "=r"(v[o]), "=r"(v[o + 1]), "=r"(v[o + 2]), "=r"(v[o + 3])
#define TB_IO4(v, o) "+r"(v[o]), "+r"(v[o + 1]), "+r"(v[o + 2]), "+r"(v[o + 3])
#define TB_I4(v, o) "r"(v[o]), "r"(v[o + 1]), "r"(v[o + 2]), "r"(v[o + 3])

// 32 consecutive TMEM columns of this thread's lane; the values are there
// after tmem_wait32 on the same array.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        : TB_O4(v, 0), TB_O4(v, 4), TB_O4(v, 8), TB_O4(v, 12), TB_O4(v, 16), TB_O4(v, 20), TB_O4(v, 24), TB_O4(v, 28)
        : "r"(taddr));
}
// Wait for this thread's TMEM loads; naming the array keeps its uses below.
__device__ __forceinline__ void tmem_wait32(uint32_t (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;\n"
                 : TB_IO4(v, 0), TB_IO4(v, 4), TB_IO4(v, 8), TB_IO4(v, 12), TB_IO4(v, 16), TB_IO4(v, 20),
                   TB_IO4(v, 24), TB_IO4(v, 28)
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};\n" ::TB_I4(v, 0),
        TB_I4(v, 4), TB_I4(v, 8), TB_I4(v, 12), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

struct Params {
    const int32_t *q_begin, *ctx_len;
    const uint32_t *mask;   // nullptr: causal
    const uint16_t *Q, *K, *V;  // (read here only for rows that are not finite; else by TMA)
    uint16_t *out;
    float *part;            // shares: two states per CTA; nullptr: the counter deals whole items out
    int32_t *joins;         // shares: what to join, 8 words an entry (first CTA or -1, CTAs, token, head, rows)
    uint32_t *flags, *counter;  // counter[0]: next item, counter[1]: CTAs that ask no more
    int batch, Hq, Hkv, cap, n_tokens, max_new, mask_words;
    int g_shift;            // G = 1 << g_shift heads per group
    int item_bound;         // items of a KV head, at most
    int ctas;               // CTAs of multi_attn_kernel
    float c;                // scale * log2(e)
};

// A segment as warp 10 describes it to the others.
template <int N>
struct Const {
    static constexpr int value = N;
};
enum SegField {
    kEnd,        // 1: no further segment
    kPair,       // slots: 1 = two row blocks over the same tiles, 0 = one row block, every other tile
    kRowBase,    // first cache row of the (sequence, KV head)
    kTok,        // packed index of the item's first token
    kHead,       // first query head of the group
    kNTok,       // tokens of the item
    kLen,        // T
    kBase,       // T - n, the first new token's cache row
    kTok0,       // the item's first token within the sequence
    kDraftEnd,   // end of the drafted rows the mask covers
    kFirst,      // first K/V tile
    kTiles,      // tiles
    kTiles0,     // tiles of slot 0
    kTiles1,     // tiles of slot 1
    kMaskLo,     // tiles that reach past this cache row hold rows that some token does not see
    kPart,       // state to write, -1: the result itself
    kSegFields
};
static_assert(kSegFields * 4 <= 64, "segment description");

// The new tokens of one sequence (n clamped to max_new for the items).
struct Seq {
    int b, begin, n, kept, T;
};
__device__ __forceinline__ Seq load_seq(const Params &p, int b) {
    Seq q{b, 0, 0, 0, 1};
    if (b < p.batch) {
        const SeqSpan sp = seq_span(p.q_begin, b, p.n_tokens);
        q.begin = sp.begin;
        q.n = sp.n;
        q.kept = min(sp.n, p.max_new);
        q.T = clamp_ctx(p.ctx_len[b], p.cap, nullptr, false);
    }
    return q;
}
__device__ __forceinline__ Seq shfl_seq(const Seq &q, int lane) {
    return {__shfl_sync(kFullMask, q.b, lane), __shfl_sync(kFullMask, q.begin, lane),
            __shfl_sync(kFullMask, q.n, lane), __shfl_sync(kFullMask, q.kept, lane),
            __shfl_sync(kFullMask, q.T, lane)};
}
__device__ __forceinline__ int items_of(const Params &p, int kept) {
    const int tpi = kItemRows >> p.g_shift;
    return (kept + tpi - 1) / tpi;
}
// K/V tiles that the sequence's tokens up to `last` attend to.
__device__ __forceinline__ int tiles_upto(const Params &p, const Seq &q, int last) {
    const int rows = p.mask ? q.T : min(q.T, q.T - q.n + last + 1);
    return max(0, (rows + kTile - 1) / kTile);
}
__device__ __forceinline__ int item_tiles(const Params &p, const Seq &q, int item) {
    const int tpi = kItemRows >> p.g_shift;
    return tiles_upto(p, q, min((item + 1) * tpi, q.kept) - 1);
}
// Inclusive sum over the lanes' sequences (one sequence: that of lane 0).
template <typename T>
__device__ __forceinline__ T warp_prefix(const Params &p, T v, int lane) {
    if (p.batch == 1) return __shfl_sync(kFullMask, v, 0);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T u = __shfl_up_sync(kFullMask, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// Sequence and number within it of item `tau`, counted over the sequences in
// packing order, 32 sequences at a time by all lanes of a warp.  A CTA's items
// come from the last to the first, so the search goes on from where it was.
struct ItemSearch {
    int b0 = 0, before = 0;  // the 32 sequences looked at last, items before them
    __device__ __forceinline__ bool find(const Params &p, int tau, int lane, Seq &q, int &item) {
        for (bool back = false; b0 < p.batch;) {
            const Seq mine = load_seq(p, b0 + lane);
            const int items = items_of(p, mine.kept), incl = warp_prefix(p, items, lane);
            const int all = __shfl_sync(kFullMask, incl, 31);
            if (back) before -= all;
            if (tau < before) {
                b0 -= 32;
                back = true;
                continue;
            }
            const uint32_t hit = __ballot_sync(kFullMask, tau < before + incl);
            if (hit) {
                const int l = __ffs(hit) - 1;
                q = shfl_seq(mine, l);
                item = tau - before - (l > 0 ? __shfl_sync(kFullMask, incl, l > 0 ? l - 1 : 0) : 0);
                return true;
            }
            if (b0 + 32 >= p.batch) return false;  // behind the last item
            before += all;
            b0 += 32;
            back = false;
        }
        return false;
    }
};

// Shares: the tiles of all items in one line (sequences in packing order, its
// items in order, KV heads inside an item), each as long as it takes.  A tile
// of 256 rows takes 3,100 cycles; one of 128 rows takes 1,900, or what its
// bytes take from HBM (2,600) where no other item reads them: 7 to 5.
// An item's first tile counts one more, for its start and its epilogue.
__device__ __forceinline__ int tile_units(const Params &p, const Seq &q, int item) {
    const bool pair = min(kItemRows >> p.g_shift, q.kept - item * (kItemRows >> p.g_shift)) > (kSlotRows >> p.g_shift);
    return pair ? 7 : 5;
}
// (32 bits hold the line: the host deals longer ones out by the counter.)
__device__ __forceinline__ uint32_t item_units(int tiles, int unit) { return tiles > 0 ? (uint32_t)(tiles + 1) * unit : 0u; }
// The first tile that begins at or behind unit x of an item.
__device__ __forceinline__ int tile_behind(uint32_t x, uint32_t unit) {
    return x == 0 ? 0 : max(1, (int)((x + unit - 1) / unit) - 1);
}
// One sequence's part of the line.
__device__ __forceinline__ uint32_t seq_units(const Params &p, const Seq &q) {
    const int items = items_of(p, q.kept);
    if (items == 0) return 0;
    const int base = q.T - q.n, last = items - 1;
    uint32_t t = item_units(item_tiles(p, q, last), tile_units(p, q, last));
    if (last > 0) {  // the full items
        const int unit = tile_units(p, q, 0);
        if (p.mask) {
            t += last * item_units(tiles_upto(p, q, 0), unit);
        } else if (base < 0) {
            for (int i = 0; i < last; ++i) t += item_units(item_tiles(p, q, i), unit);
        } else {
            // sum of ceil((base + i tpi) / 128) over i = 1 .. last: every `k`
            // items (k = 128 / tpi) the tiles grow by `d`
            const int tpi = kItemRows >> p.g_shift, k = max(1, kTile / tpi), d = max(1, tpi / kTile);
            const int blocks = last / k;
            int tiles = 0;
            for (int r = 1; r <= k; ++r) {  // i = r, r + k, ..: `count` of them
                const int count = blocks + (r <= last % k);
                tiles += count * ((base + r * tpi + kTile - 1) / kTile) + d * (count * (count - 1) / 2);
            }
            t += (uint32_t)(tiles + last) * unit;
        }
    }
    return t * p.Hkv;
}
// The line in `ctas` shares that differ by one unit at most.
struct Shares {
    uint32_t total, each;
    int rest, ctas;
    __device__ __forceinline__ Shares(uint32_t units, int grid) : total(units) {
        // no share is below 4 tiles: short contexts keep to fewer CTAs
        ctas = max(1, min(grid, (int)(units >> 5)));
        each = units / ctas;
        rest = (int)(units - each * ctas);
    }
    __device__ __forceinline__ uint32_t begin(int c) const { return c >= ctas ? total : each * c + min(c, rest); }
    __device__ __forceinline__ int holding(uint32_t u) const {  // the share with unit u
        const uint32_t big = (each + 1) * rest;
        return (int)(u < big ? u / (each + 1) : rest + (u - big) / each);
    }
};

// Rows of an item's slots behind its last token hold queries of other
// sequences or of nobody.  Where they are a quarter or more, warp 11 clears
// them before the products use them: products with zeros draw less power, and
// power is what bounds the clock (16 ragged trees: 415 -> 391 us; the look at
// the queries costs about 0.4 us an item: 16 trees over 16K, items of 64 tokens,
// 33 of them live: 286 us without, 272 with; 48 live: 291, 285; 60 live: 300, 297).
__device__ __forceinline__ bool many_dead(int live, int rows) { return 4 * (rows - live) >= rows; }

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
multi_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const Params p) {
    using L = Lay<D>;
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sb = smem_addr(sm);
    if (sb & 1023u) {  // the operands' layout needs it; no room is left to align here
        if (threadIdx.x == 0) raise_flag(p.flags, TB_FLAG_TIMEOUT);
        return;
    }
    volatile int *misc = reinterpret_cast<volatile int *>(sm + L::kMisc);
    volatile int *abort_flag = misc + 1;
    auto bar = [&](int i) -> uint32_t { return sb + L::kBar + 8u * (uint32_t)i; };
    auto full = [&](int s) { return bar(s); };
    auto empty = [&](int s) { return bar(L::kStages + s); };
    constexpr int kB = 2 * L::kStages;
    const uint32_t q_full = bar(kB), q_empty = bar(kB + 1), loaded = bar(kB + 2), drain = bar(kB + 3);
    const uint32_t o_free = bar(kB + 4);
    auto seg_full = [&](int i) { return bar(kB + 5 + i); };
    auto seg_empty = [&](int i) { return bar(kB + 7 + i); };
    const uint32_t state_full = bar(kB + 9), state_empty = bar(kB + 10);
    auto s_full = [&](int s) { return bar(kB + 11 + s); };
    auto p_full = [&](int s, int half) { return bar(kB + 13 + 2 * s + half); };  // keys 0..63, 64..127
    auto o_done = [&](int s) { return bar(kB + 17 + s); };
    auto s_read = [&](int s) { return bar(kB + 19 + s); };
    auto v_loading = [&](int m) { return bar(kB + 21 + (m & 7)); };
    const uint32_t q_raw = bar(kB + 37);
    auto v_clean = [&](int m) { return bar(kB + 29 + (m & 7)); };
    auto seg = [&](int i) { return reinterpret_cast<volatile int *>(sm + L::kSeg + i * 64); };

    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(kFullMask, tid >> 5, 0);
    if (tid == 0) {
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        mbar_init(q_full, 1);
        mbar_init(q_raw, 1);
        mbar_init(q_empty, 1);
        mbar_init(drain, 1);
        mbar_init(loaded, 1);
        mbar_init(o_free, 8);
        mbar_init(state_full, 8);
        mbar_init(state_empty, 8);
        for (int s = 0; s < 2; ++s) {
            mbar_init(seg_full(s), 1);
            mbar_init(seg_empty(s), 11);
            mbar_init(s_full(s), 1);
            mbar_init(s_read(s), 4);
            mbar_init(p_full(s, 0), 4);
            mbar_init(p_full(s, 1), 4);
            mbar_init(o_done(s), 1);
        }
        for (int m = 0; m < 8; ++m) {
            mbar_init(v_loading(m), 1);
            mbar_init(v_clean(m), 1);
        }
        misc[1] = 0;
        fence_mbar_init();
    }
    if (warp == 9 && lane == 0) {
        prefetch_tensormap(&tmQ);
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    if (warp == 8) {
        tmem_alloc(sb + L::kMisc, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // (up to here nothing in global memory was touched)
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t tmem = (uint32_t)misc[0];
    const int tps = kSlotRows >> p.g_shift;  // tokens per slot

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegsOther));
        if (warp == 10) {
            // ======================================================== schedule
            int k = 0;  // segments described so far
            bool ok = true;
            // what only the device sees: reported once per sequence
            auto report = [&](const Seq &q) {
                const int t = p.ctx_len[q.b];
                if (lane == 0 && (t < 1 || t > p.cap || q.n > q.T || q.n > p.max_new)) raise_flag(p.flags, TB_FLAG_CTX_RANGE);
            };
            // an item whose tokens see no cache row at all (more new tokens than rows)
            auto zero_item = [&](const Seq &q, int item, int g) {
                const int tok0 = item * 2 * tps, ntok = min(2 * tps, q.kept - tok0), per = (D / 8) << p.g_shift;
                for (int i = lane; i < ntok * per; i += 32)
                    reinterpret_cast<uint4 *>(p.out + ((size_t)(q.begin + tok0 + i / per) * p.Hq + (g << p.g_shift)) * D)[i % per] =
                        make_uint4(0, 0, 0, 0);
            };
            // tiles [first, last), at least one, of item `item` of sequence q for KV head g
            auto emit = [&](const Seq &q, int item, int g, int first, int last, int part) {
                if (k >= 2) ok = wait_warp(seg_empty(k & 1), ((k >> 1) + 1) & 1, abort_flag, p.flags);
                if (!ok) return;
                if (lane == 0) {
                    const int tok0 = item * 2 * tps, ntok = min(2 * tps, q.kept - tok0), nt = last - first;
                    const bool pair = ntok > tps;
                    volatile int *f = seg(k & 1);
                    f[kEnd] = 0;
                    f[kPair] = pair;
                    f[kRowBase] = (int)(((size_t)q.b * p.Hkv + g) * (size_t)p.cap);  // < 2^31 (checked on the host)
                    f[kTok] = q.begin + tok0;
                    f[kHead] = g << p.g_shift;
                    f[kNTok] = ntok;
                    f[kLen] = q.T;
                    f[kBase] = q.T - q.n;
                    f[kTok0] = tok0;
                    f[kDraftEnd] = q.T - q.n + q.kept;
                    f[kFirst] = first;
                    f[kTiles] = nt;
                    // in pairs slot 0's rows, the earlier tokens, may end a tile or two before slot 1's
                    f[kTiles0] = pair ? max(0, min(last, tiles_upto(p, q, tok0 + tps - 1)) - first) : (nt + 1) / 2;
                    f[kTiles1] = pair ? nt : nt / 2;
                    f[kMaskLo] = p.mask ? q.T - q.n : q.T - q.n + tok0 + 1;
                    f[kPart] = part;
                    // no V row taken out yet: seg_full hands that to every
                    // role, those that no tile orders behind warp 11 too
                    *reinterpret_cast<volatile int *>(sm + L::kBad + (k & 1) * kBadBytes) = 0;
                    mbar_arrive(seg_full(k & 1));
                }
                __syncwarp();
                ++k;
            };
            if (p.part == nullptr) {
                // from the last item to the first: a sequence's last tokens have the most tiles
                bool first_item = true;
                ItemSearch search;
                while (ok) {
                    // the next item is taken when the current one's last tiles
                    // are on their way: early enough to overlap, and no CTA
                    // holds a second long item while others run dry
                    if (k > 0) ok = wait_warp(loaded, (k - 1) & 1, abort_flag, p.flags);
                    if (!ok) break;
                    int next = blockIdx.x;  // the first item needs no counter
                    if (!first_item) {
                        if (lane == 0) next = (int)(gridDim.x + atomicAdd(p.counter, 1u));
                        next = __shfl_sync(kFullMask, next, 0);
                    }
                    first_item = false;
                    if (next >= p.item_bound * p.Hkv) break;
                    Seq q;
                    int item;
                    if (!search.find(p, p.item_bound - 1 - next / p.Hkv, lane, q, item)) continue;
                    const int g = next % p.Hkv, tiles = item_tiles(p, q, item);
                    if (item == 0 && g == 0) report(q);
                    if (tiles > 0)
                        emit(q, item, g, 0, tiles, -1);
                    else
                        zero_item(q, item, g);
                }
                // the last CTA to ask leaves the counter as it was found
                if (lane == 0 && atom_add_acq_rel_gpu(p.counter + 1, 1u) == gridDim.x - 1) {
                    p.counter[0] = 0u;
                    p.counter[1] = 0u;
                }
            } else {
                const int cta = blockIdx.x;
                const Seq seq0 = load_seq(p, lane);  // of the first 32 sequences
                const uint32_t units0 = warp_prefix(p, seq_units(p, seq0), lane);
                const int items0 = warp_prefix(p, items_of(p, seq0.kept), lane);
                uint32_t total = __shfl_sync(kFullMask, units0, 31);
                int total_items = __shfl_sync(kFullMask, items0, 31);
                for (int b0 = 32; b0 < p.batch; b0 += 32) {
                    const Seq mine = load_seq(p, b0 + lane);
                    total += __shfl_sync(kFullMask, warp_prefix(p, seq_units(p, mine), lane), 31);
                    total_items += __shfl_sync(kFullMask, warp_prefix(p, items_of(p, mine.kept), lane), 31);
                }
                total_items *= p.Hkv;
                const Shares sh(total, gridDim.x);
                uint32_t w = sh.begin(cta);
                const uint32_t w1 = sh.begin(cta + 1);
                // an entry for every item, or where there are more items than
                // CTAs, for every CTA (one item at most ends in it that began earlier)
                const bool by_item = p.item_bound * p.Hkv <= (int)gridDim.x;
                // (a q_begin that does not rise may give more items than the host's
                // bound: what is behind the list is not written)
                auto join = [&](int entry, int from, int tok, int head, int rows) {
                    if (entry >= (int)gridDim.x) return;
                    if (lane == 0) *reinterpret_cast<int4 *>(p.joins + 8 * entry) = make_int4(from, cta - from + 1, tok, head);
                    if (lane == 0) p.joins[8 * entry + 4] = rows;
                };
                bool joined = false;
                // the sequence that holds unit w: `at` is where its part of the line begins
                uint32_t at = 0;
                int b = p.batch, items_before = 0;
                Seq q;
                for (int b0 = 0; w < w1 && b0 < p.batch; b0 += 32) {
                    const Seq mine = b0 == 0 ? seq0 : load_seq(p, b0 + lane);
                    const uint32_t incl = b0 == 0 ? units0 : warp_prefix(p, seq_units(p, mine), lane);
                    const int before = b0 == 0 ? items0 : warp_prefix(p, items_of(p, mine.kept), lane);
                    const uint32_t hit = __ballot_sync(kFullMask, w < at + incl);
                    if (hit) {
                        const int l = __ffs(hit) - 1;
                        b = b0 + l;
                        q = shfl_seq(mine, l);
                        if (l > 0) at += __shfl_sync(kFullMask, incl, l - 1);
                        if (l > 0) items_before += __shfl_sync(kFullMask, before, l - 1);
                        break;
                    }
                    at += __shfl_sync(kFullMask, incl, 31);
                    items_before += __shfl_sync(kFullMask, before, 31);
                }
                while (ok && w < w1 && b < p.batch) {
                    const int items = items_of(p, q.kept);
                    for (int i = 0; i < items && ok && w < w1; ++i) {
                        const int tiles = item_tiles(p, q, i), unit = tile_units(p, q, i);
                        const uint32_t len = item_units(tiles, unit);
                        if (w >= at + len * p.Hkv) {
                            at += len * p.Hkv;
                            continue;
                        }
                        for (int g = 0; g < p.Hkv && ok && w < w1; ++g, at += len) {
                            if (w >= at + len) continue;
                            // the tiles that begin in this share
                            const int first = tile_behind(w - at, unit);
                            const int last = min(tiles, tile_behind(w1 - at, unit));
                            w = min(at + len, w1);
                            if (first >= last) continue;
                            // states: 2 c for an item begun in an earlier share, 2 c + 1 for one that goes on in the next
                            emit(q, i, g, first, last, first == 0 && last == tiles ? -1 : 2 * cta + (first == 0));
                            if (last == tiles && (first > 0 || by_item)) {  // ends here
                                const int tok0 = i * 2 * tps;
                                join(by_item ? (items_before + i) * p.Hkv + g : cta, first > 0 ? sh.holding(at) : -1,
                                     q.begin + tok0, g << p.g_shift, min(2 * tps, q.kept - tok0) << p.g_shift);
                                joined = true;
                            }
                        }
                    }
                    items_before += items;
                    if (++b < p.batch) q = load_seq(p, b);
                }
                if (cta == 0) {  // the lengths' report, and items without a tile, which are in nobody's share
                    int before = 0;
                    for (int b0 = 0; b0 < p.batch; b0 += 32) {
                        bool odd = false;
                        const Seq mine = load_seq(p, b0 + lane);
                        const int upto = before + warp_prefix(p, items_of(p, mine.kept), lane);
                        before = __shfl_sync(kFullMask, upto, 31);
                        if (b0 + lane < p.batch) {
                            const Seq q = mine;
                            const int t = q.n > 0 ? p.ctx_len[q.b] : 1;  // (an idle sequence's length is not looked at)
                            odd = t < 1 || t > p.cap || (q.n > 0 && q.n > q.T) || q.n > p.max_new;
                        }
                        for (uint32_t hits = __ballot_sync(kFullMask, odd); hits; hits &= hits - 1) {
                            const int l = __ffs(hits) - 1, items = __shfl_sync(kFullMask, items_of(p, mine.kept), l);
                            const int at_item = __shfl_sync(kFullMask, upto, l) - items;
                            const Seq q = shfl_seq(mine, l);
                            report(q);
                            for (int i = 0; i < items && item_tiles(p, q, i) == 0; ++i)
                                for (int g = 0; g < p.Hkv; ++g) {
                                    zero_item(q, i, g);
                                    if (by_item) join((at_item + i) * p.Hkv + g, -1, 0, 0, 0);
                                }
                        }
                    }
                }
                // entries nobody else writes: this CTA's, or those behind the last item
                if (by_item ? cta >= total_items && cta < p.item_bound * p.Hkv : !joined) join(cta, -1, 0, 0, 0);
            }
            if (ok && k >= 2) ok = wait_warp(seg_empty(k & 1), ((k >> 1) + 1) & 1, abort_flag, p.flags);
            if (ok && lane == 0) {
                seg(k & 1)[kEnd] = 1;
                mbar_arrive(seg_full(k & 1));
            }
            __syncwarp();
        } else if (warp == 9) {
            // ======================================================== loads
            // Ring order = the order in which the products use the tiles: K0
            // V0 K1 V1 .. in pairs, K0 K1 V0 K2 V1 .. for every other tile, and
            // one more K ahead where the next S does not wait for P.
            int stage = 0, issued = 0, masked = 0, queries = 0, k = 0;
            uint32_t parity = 1;  // of a stage's previous release (passes at once in the first round)
            bool ok = true;
            for (;; ++k) {
                ok = wait_warp(seg_full(k & 1), (k >> 1) & 1, abort_flag, p.flags);
                if (!ok) break;
                volatile const int *f = seg(k & 1);
                if (f[kEnd]) break;
                const bool pair = f[kPair];
                const int nt = f[kTiles], row0 = f[kRowBase] + f[kFirst] * kTile;
                const int mask_lo = f[kMaskLo] - f[kFirst] * kTile;  // within the segment's rows
                if (k > 0) ok = wait_warp(q_empty, (k - 1) & 1, abort_flag, p.flags);
                if (!ok) break;
                if (lane == 0) {
                    const int qn = pair ? 2 : 1, tok = f[kTok], head = f[kHead];
                    const uint32_t qb = many_dead(f[kNTok] << p.g_shift, qn * kSlotRows) ? q_raw : q_full;
                    mbar_arrive_expect_tx(qb, (uint32_t)(qn * L::kOperand));
                    for (int s = 0; s < qn; ++s)
#pragma unroll
                        for (int a = 0; a < L::kAtoms; ++a)
                            tma_load_3d(sb + s * L::kOperand + a * 16384, &tmQ, qb, a * 64, head, tok + s * tps);
                }
                ++queries;
                auto load = [&](bool is_k, int tile) {
                    if (!ok) return;
                    ok = wait_warp(empty(stage), parity, abort_flag, p.flags);
                    if (!ok) return;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(full(stage), L::kOperand);
#pragma unroll
                        for (int a = 0; a < L::kAtoms; ++a)
                            tma_load_2d(sb + L::kRing + stage * L::kOperand + a * 16384, is_k ? &tmK : &tmV, full(stage),
                                        a * 64, row0 + tile * kTile);
                    }
                    ++issued;
                    if (++stage == L::kStages) {
                        stage = 0;
                        parity ^= 1u;
                    }
                };
                // K tiles run `ahead` tiles before V
                const int ahead = (pair ? 0 : 1) + (L::kSepP ? 1 : 0);
                for (int t = 0; t <= ahead && t < nt; ++t) load(true, t);
                for (int t = 0; t < nt && ok; ++t) {
                    load(false, t);
                    if (ok && (t + 1) * kTile > mask_lo) {
                        if (lane == 0) mbar_arrive(v_loading(masked));
                        ++masked;
                    }
                    if (t + ahead + 1 < nt) load(true, t + ahead + 1);
                }
                if (!ok) break;
                if (lane == 0) {
                    mbar_arrive(loaded);
                    mbar_arrive(seg_empty(k & 1));
                }
                __syncwarp();
            }
            // leave only when every copy has landed
            if (queries > 0) mbar_wait_bounded(q_full, (queries - 1) & 1, p.flags);
            for (int i = max(0, issued - L::kStages); i < issued; ++i)
                mbar_wait_bounded(full(i % L::kStages), (i / L::kStages) & 1, p.flags);
        } else if (warp == 11) {
            // ======================================================== masked tiles
            // V tiles with rows that not every token of the item sees, before
            // the product with P uses them: a weight of 0 for such a row does
            // not keep a NaN or an infinity in it out of the sums.  Rows at and
            // past the length, which may hold anything, are cleared; so are
            // rows with a value that is not finite, and listed: the epilogue
            // adds those to the tokens that see them.
            int masked = 0, ring = 0, raws = 0;
            bool ok = true;
            for (int k = 0; ok; ++k) {
                ok = wait_warp(seg_full(k & 1), (k >> 1) & 1, abort_flag, p.flags);
                if (!ok) break;
                volatile const int *f = seg(k & 1);
                if (f[kEnd]) break;
                const int nt = f[kTiles], ahead = (f[kPair] ? 0 : 1) + (L::kSepP ? 1 : 0);
                const int row0 = f[kFirst] * kTile, mask_lo = f[kMaskLo] - row0, len = f[kLen] - row0;
                volatile int *bad = reinterpret_cast<volatile int *>(sm + L::kBad + (k & 1) * kBadBytes);
                const int live = f[kNTok] << p.g_shift, rows = f[kPair] ? kItemRows : kSlotRows;
                if (many_dead(live, rows)) {
                    ok = wait_warp(q_raw, raws & 1, abort_flag, p.flags);
                    if (!ok) break;
                    ++raws;
                    for (int r = live; r < rows; r += 4)
                        for (int a = 0; a < L::kAtoms; ++a) {
                            const int rr = r + (lane >> 3);
                            if (rr < rows)
                                *reinterpret_cast<uint4 *>(sm + (rr >> 7) * L::kOperand + a * 16384 + (rr & 127) * 128 + (lane & 7) * 16) =
                                    make_uint4(0, 0, 0, 0);
                        }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(q_full);
                }
                int n_bad = 0;
                for (int t = max(0, mask_lo / kTile); t < nt && ok; ++t) {
                    if ((t + 1) * kTile <= mask_lo) continue;
                    // once the load is issued the barrier is in this tile's phase
                    ok = wait_warp(v_loading(masked), (masked >> 3) & 1, abort_flag, p.flags);
                    const int item = ring + min(nt, t + ahead + 1) + t;
                    if (ok) ok = wait_warp(full(item % L::kStages), (item / L::kStages) & 1, abort_flag, p.flags);
                    if (!ok) break;
                    uint8_t *v = sm + L::kRing + (item % L::kStages) * L::kOperand;
                    const int r0 = max(0, mask_lo - t * kTile), r1 = max(r0, min(kTile, len - t * kTile));
                    bool wrote = r1 < kTile;
#pragma unroll
                    for (int a = 0; a < L::kAtoms; ++a)
                        for (int o = r1 * 128 + lane * 16; o < kTile * 128; o += 512)
                            *reinterpret_cast<uint4 *>(v + a * 16384 + o) = make_uint4(0, 0, 0, 0);
                    uint32_t top = 0u;  // the largest magnitudes, as pairs of 16-bit integers
#pragma unroll
                    for (int a = 0; a < L::kAtoms; ++a)
#pragma unroll 4
                        for (int o = r0 * 128 + lane * 16; o < r1 * 128; o += 512) {
                            const uint4 x = *reinterpret_cast<const uint4 *>(v + a * 16384 + o);
                            top = __vmaxu2(top, __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                                                         __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu)));
                        }
                    if (__any_sync(kFullMask, (top & 0xffffu) >= 0x7f80u || (top >> 16) >= 0x7f80u)) {
                        // which rows: lane by lane
                        if (lane == 0 && n_bad < kMaxMasked) bad[1 + 5 * n_bad] = row0 + t * kTile;
                        for (int q = 0; q < 4; ++q) {
                            const int r = q * 32 + lane;
                            bool odd = false;
                            if (r >= r0 && r < r1)
                                for (int a = 0; a < L::kAtoms; ++a)
                                    for (int o = 0; o < 128; o += 4) {
                                        const uint32_t x = *reinterpret_cast<const uint32_t *>(v + a * 16384 + r * 128 + o);
                                        odd |= (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
                                    }
                            if (odd)
                                for (int a = 0; a < L::kAtoms; ++a)
                                    for (int o = 0; o < 128; o += 16)
                                        *reinterpret_cast<uint4 *>(v + a * 16384 + r * 128 + o) = make_uint4(0, 0, 0, 0);
                            const uint32_t w = __ballot_sync(kFullMask, odd);
                            if (lane == 0 && n_bad < kMaxMasked) bad[2 + 5 * n_bad + q] = (int)w;
                        }
                        n_bad = min(n_bad + 1, kMaxMasked);
                        // (a pair's first slot may read the list meanwhile: the
                        // entry before its count)
                        __threadfence_block();
                        if (lane == 0) bad[0] = n_bad;
                        wrote = true;
                    }
                    if (wrote) fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(v_clean(masked));
                    ++masked;
                }
                ring += 2 * nt;
                if (lane == 0) mbar_arrive(seg_empty(k & 1));
                __syncwarp();
            }
        } else if (warp == 8) {
            // ======================================================== products
            // One thread issues all of them.  Per slot the order is S(0), then
            // PV(j) S(j+1): S(j+1) overwrites the columns of P(j), which PV(j)
            // has read by then (the products of one thread run in order).  PV
            // is issued in two halves of 64 keys, so that its first half runs
            // while the softmax works out the second half of the weights.
            if (elect_one()) {
                constexpr uint32_t id_s = idesc_bf16_f32(128, kTile);
                constexpr uint32_t id_o = idesc_bf16_f32(128, D) | (1u << 16);  // B (V) MN-major
                constexpr uint32_t kStep = L::kOperand >> 4;
                const uint64_t kd = sw128_kmajor_desc(sb), vd = sw128_mnmajor_desc(sb + L::kRing, 16384);
                const uint32_t q_lo = (uint32_t)kd, hi = (uint32_t)(kd >> 32);
                const uint32_t k_lo = q_lo + (L::kRing >> 4), v_lo = (uint32_t)vd;
                int k_stage = 0, v_stage = 0, next = 0;
                uint32_t next_parity = 0;
                int masked = 0;
                uint32_t done = 0, read = 0;  // bit s = parity of slot s's tiles so far (P used, S read)
                bool ok = true;
                auto acquire = [&](int &st) {
                    st = next;
                    if (ok) ok = wait_role(full(next), next_parity, abort_flag, p.flags);
                    if (++next == L::kStages) {
                        next = 0;
                        next_parity ^= 1u;
                    }
                };
                for (int k = 0; ok; ++k) {
                    ok = wait_role(seg_full(k & 1), (k >> 1) & 1, abort_flag, p.flags);
                    if (!ok) break;
                    volatile const int *f = seg(k & 1);
                    if (f[kEnd]) break;
                    const bool pair = f[kPair];
                    const int nt = f[kTiles], nt0 = f[kTiles0], nt1 = f[kTiles1];
                    const int mask_lo = f[kMaskLo] - f[kFirst] * kTile;
                    ok = wait_role(q_full, k & 1, abort_flag, p.flags);
                    // round j: slot 0's and slot 1's step, each the PV of its
                    // tile j and the S of its tile j + 1.  In pairs both use
                    // K/V tile j, else tiles 2j and 2j + 1.  The S overwrites
                    // the columns of P (PV has read them by then: the products
                    // of one thread run in order); where P has columns of its
                    // own it goes first, once the softmax has read the last.
                    const int rounds = pair ? nt : (nt + 1) >> 1;
                    auto next_s = [&](auto slot_c, int j) {
                        constexpr int slot = decltype(slot_c)::value;
                        // (in pairs slot 1 has every tile, so it also releases them)
                        const bool uses = pair ? j + 1 < nt : 2 * (j + 1) + slot < nt;
                        if (!ok || !uses) return;
                        if (!pair || slot == 0) acquire(k_stage);
                        if (j + 1 < (slot ? nt1 : nt0)) {
                            if (L::kSepP && j >= 0 && ok) {
                                ok = wait_role(s_read(slot), (read >> slot) & 1u, abort_flag, p.flags);
                                read ^= 1u << slot;
                            }
                            if (!ok) return;
                            tc_fence_after();
                            const uint32_t q = q_lo + (pair ? slot : 0) * kStep, kl = k_lo + k_stage * kStep;
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                const uint32_t o = (uint32_t)((kk >> 2) * 1024 + (kk & 3) * 2);
                                umma_ss(tmem + slot * 128, q + o, kl + o, hi, id_s, kk > 0);
                            }
                            umma_commit(s_full(slot));
                        }
                        if (!ok) return;
                        if (!pair || slot == 1) umma_commit(empty(k_stage));
                        // the segment's last S: the queries are free
                        if (pair ? slot == 1 && j + 2 == nt : 2 * (j + 1) + slot + 1 == nt) umma_commit(q_empty);
                    };
                    auto pv = [&](auto slot_c, int j) {
                        constexpr int slot = decltype(slot_c)::value;
                        const int tile = pair ? j : 2 * j + slot;
                        if (!ok || tile >= nt) return;
                        if (!pair || slot == 0) {
                            acquire(v_stage);
                            if ((tile + 1) * kTile > mask_lo) {  // looked over by warp 11
                                if (ok) ok = wait_role(v_clean(masked), (masked >> 3) & 1, abort_flag, p.flags);
                                ++masked;
                            }
                            // the previous segment's sums have been read
                            if (slot == 0 && j == 0 && k > 0 && ok) ok = wait_role(o_free, (k - 1) & 1, abort_flag, p.flags);
                        }
                        if (j < (slot ? nt1 : nt0)) {
                            const uint32_t v = v_lo + v_stage * kStep;
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                if (ok) ok = wait_role(p_full(slot, half), (done >> slot) & 1u, abort_flag, p.flags);
                                if (!ok) return;
                                tc_fence_after();
#pragma unroll
                                for (int kk = half * 4; kk < half * 4 + 4; ++kk)
                                    umma_ts(tmem + L::kO + slot * L::kOStep, tmem + L::kP + slot * L::kPStep + kk * 8,
                                            v + kk * 128, hi, id_o, (j | kk) ? 1u : 0u);
                            }
                            umma_commit(o_done(slot));
                            done ^= 1u << slot;
                        }
                        if (ok && (!pair || slot == 1)) umma_commit(empty(v_stage));
                    };
                    using Slot0 = Const<0>;
                    using Slot1 = Const<1>;
                    next_s(Slot0{}, -1);
                    next_s(Slot1{}, -1);
#pragma unroll 1
                    for (int j = 0; j < rounds && ok; ++j) {
                        if (L::kSepP) next_s(Slot0{}, j);
                        pv(Slot0{}, j);
                        if (!L::kSepP) next_s(Slot0{}, j);
                        if (L::kSepP) next_s(Slot1{}, j);
                        pv(Slot1{}, j);
                        if (!L::kSepP) next_s(Slot1{}, j);
                    }
                    if (!ok) break;
                    if (L::kSepP && ok) {
                        // each slot's last S was read too: keep the barriers' phases in step
                        for (int slot = 0; slot < 2; ++slot)
                            if ((slot ? nt1 : nt0) > 0) read ^= 1u << slot;
                    }
                    if (!ok) break;
                    mbar_arrive(seg_empty(k & 1));
                }
                umma_commit(drain);  // no product is in flight when the CTA ends
                mbar_wait_bounded(drain, 0, p.flags);
            }
            __syncwarp();
        }
    } else {
        // ============================================================ softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kRegsSoftmax));
        const int slot = warp >> 2;
        const int row = tid & 127;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lane_base + slot * 128, to = tmem + lane_base + L::kO;
        const uint32_t tp = tmem + lane_base + L::kP + slot * L::kPStep;
        uint32_t count = 0, merges = 0;  // tiles of this slot so far; merged segments so far
        uint32_t other_count = 0;        // tiles of the other slot so far
        bool ok = true;
        for (int k = 0; ok; ++k) {
            ok = wait_warp(seg_full(k & 1), (k >> 1) & 1, abort_flag, p.flags);
            if (!ok) break;
            volatile const int *f = seg(k & 1);
            if (f[kEnd]) break;
            const bool pair = f[kPair];
            const int t_step = pair ? 1 : 2, n_mine = slot ? f[kTiles1] : f[kTiles0];
            const int p_step = t_step * kTile;
            int p0 = (f[kFirst] + (pair ? 0 : slot)) * kTile;  // the tile's first cache row
            int n_loop = n_mine;
            // the row sees every cache row below all_end, and of the drafted
            // rows from all_end to draft_end those with a bit in mrow
            const uint32_t *mrow = nullptr;
            int all_end = 0, draft_end = 0, masked_from;
            {
                const int ti = (pair ? slot * tps : 0) + (row >> p.g_shift);  // token of the item
                const int base = f[kBase];
                if (ti < f[kNTok]) {
                    all_end = p.mask ? base : base + f[kTok0] + ti + 1;
                    draft_end = f[kDraftEnd];
                    if (p.mask) mrow = p.mask + (size_t)(f[kTok] + ti) * p.mask_words;
                }
                // tiles that reach past this cache row hold rows that some row of this slot does not see
                masked_from = p.mask ? base : base + f[kTok0] + (pair ? slot * tps : 0) + 1;
            }
            float m = -INFINITY, l = 0.f;
            float rf = 1.f;  // row_factor(m)
            // a warp whose 32 rows all lie behind the item's last token only
            // keeps the barriers going: its rows' weights and sums are whatever
            // the columns hold, and nobody reads them
            if ((pair ? slot * tps : 0) + (((warp & 3) * 32) >> p.g_shift) >= f[kNTok]) {
                for (int j = 0; j < n_mine; ++j, ++count) {
                    ok = wait_warp(s_full(slot), count & 1, abort_flag, p.flags);
                    // (as below: not a tile ahead of the slot's other warps)
                    if (ok && L::kSepP && j > 0) ok = wait_warp(o_done(slot), (count - 1) & 1, abort_flag, p.flags);
                    if (!ok) break;
                    if (lane == 0) {
                        if (L::kSepP) mbar_arrive(s_read(slot));
                        mbar_arrive(p_full(slot, 0));
                        mbar_arrive(p_full(slot, 1));
                    }
                    __syncwarp();
                }
                n_loop = 0;
            }

            // which of the 32 cache rows from r on this row attends to
            auto allowed = [&](int r) -> uint32_t {
                uint32_t d = bits_below(all_end - r);
                if (mrow) {
                    const int j0 = r - all_end;  // drafted token at r
                    uint32_t x = 0u;
                    if (j0 >= 0) {
                        const int w = j0 >> 5, sh = j0 & 31;
                        if (w < p.mask_words) x = __ldg(mrow + w) >> sh;
                        if (sh && w + 1 < p.mask_words) x |= __ldg(mrow + w + 1) << (32 - sh);
                    } else if (j0 > -32) {
                        x = __ldg(mrow) << -j0;
                    }
                    d |= x & bits_below(draft_end - r);
                }
                return d;
            };

            for (int j = 0; j < n_loop; ++j, p0 += p_step, ++count) {
                const bool masked = p0 + kTile > masked_from;
                uint32_t see[4];
                if (masked) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) see[q] = allowed(p0 + q * 32);
                }
                ok = wait_warp(s_full(slot), count & 1, abort_flag, p.flags);
                if (!ok) break;
                tc_fence_after();
                uint32_t s[4][32];
#pragma unroll
                for (int q = 0; q < 4; ++q) tmem_ld32(ts + q * 32, s[q]);
#pragma unroll
                for (int q = 0; q < 4; ++q) tmem_wait32(s[q]);
                if (L::kSepP) {  // the next S may overwrite this one
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(s_read(slot));
                }
                if (masked) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!((see[q] >> i) & 1u)) s[q][i] = 0xff800000u;  // -inf
                }
                float mx[4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    mx[q] = max3_nan(__uint_as_float(s[q][0]), __uint_as_float(s[q][1]), __uint_as_float(s[q][2]));
#pragma unroll
                for (int i = 3; i < 31; i += 2)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        mx[q] = max3_nan(mx[q], __uint_as_float(s[q][i]), __uint_as_float(s[q][i + 1]));
#pragma unroll
                for (int q = 0; q < 4; ++q) mx[q] = max3_nan(mx[q], __uint_as_float(s[q][31]), mx[q]);
                float top = max3_nan(mx[0], mx[1], max3_nan(mx[2], mx[3], mx[3])) * p.c;
                // a NaN or +inf logit makes the row's softmax NaN: so becomes m, and l with it
                if (!(top < INFINITY)) top = NAN;
                const bool raise = !(top <= m + kLazy);  // also the first logit of a row (m = -inf)
                if (L::kSepP && j > 0) {  // the previous P has been read
                    ok = wait_warp(o_done(slot), (count - 1) & 1, abort_flag, p.flags);
                    if (!ok) break;
                    tc_fence_after();
                }
                if (__any_sync(kFullMask, raise)) {
                    const float m_new = raise ? top : m;
                    const float fac = m_new == m ? 1.f : ex2(m - m_new);  // (-inf stays -inf while nothing is seen)
                    if (j > 0) {
                        if (!L::kSepP) ok = wait_warp(o_done(slot), (count - 1) & 1, abort_flag, p.flags);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int q = 0; q < D / 16; ++q) {  // rare: kept small, the logits fill the registers
                            float o[16];
                            uint32_t w[16];
                            tmem_ld16(to + slot * L::kOStep + q * 16, o);
#pragma unroll
                            for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(o[i] * fac);
                            tmem_st16(to + slot * L::kOStep + q * 16, w);
                        }
                    }
                    l *= fac;
                    m = m_new;
                    rf = row_factor(m);
                }
                const float mm = m == -INFINITY ? 0.f : m * rf;  // a row that has seen nothing: 2^(-inf - 0) = 0
                const uint64_t c2 = pack2(p.c * rf, p.c * rf), nm2 = pack2(-mm, -mm);
                uint64_t sum2[2] = {0ull, 0ull};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const uint64_t x2 =
                            fma2(pack2(__uint_as_float(s[q][2 * i]), __uint_as_float(s[q][2 * i + 1])), c2, nm2);
                        // (a quarter of the exponentials by a polynomial on
                        // the FMA pipe, beside the unit's 16 a cycle, made no
                        // difference under the power cap: 510 against 512 us
                        // for an 8K prompt of 128 head dims; not measured at 64)
                        float e0, e1;
                        unpack2(x2, e0, e1);
                        e0 = ex2(e0);
                        e1 = ex2(e1);
                        sum2[i & 1] = add2(sum2[i & 1], pack2(e0, e1));
                        // rounded to bf16 for the second product: at most 2^-8
                        // relative per weight, as the rounding of the result.
                        // Together they are off by 0.0023 (2-norm), the result
                        // alone by 0.0017; a product with the remainders too
                        // would be half as much tensor work again, which is
                        // what bounds the prompts
                        w[i] = pack_bf16(e0, e1);
                    }
                    tmem_st16(tp + q * 16, w);
                    if (q & 1) {  // half of the weights are in place
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(p_full(slot, q >> 1));
                    }
                }
                float u0, u1;
                unpack2(add2(sum2[0], sum2[1]), u0, u1);
                l += u0 + u1;
            }
            if (!ok) break;

            // ---- epilogue: in pairs each slot its own rows; else both slots
            // the same rows, each half of the head dims of the merged sums
            const int n_other = slot ? f[kTiles0] : f[kTiles1];
            if (n_mine > 0) ok = wait_warp(o_done(slot), (count - 1) & 1, abort_flag, p.flags);
            if (!ok) break;
            float f0 = 1.f, f1 = 0.f;  // this slot's and the other's factor
            if (!pair) {
                volatile float *st = reinterpret_cast<volatile float *>(sm + L::kState);
                if (merges > 0) ok = wait_warp(state_empty, (merges - 1) & 1, abort_flag, p.flags);
                if (!ok) break;
                st[slot * 256 + row] = m;
                st[slot * 256 + 128 + row] = l;
                __syncwarp();
                if (lane == 0) mbar_arrive(state_full);
                ok = wait_warp(state_full, merges & 1, abort_flag, p.flags);
                if (ok && n_other > 0)
                    ok = wait_warp(o_done(slot ^ 1), (other_count + n_other - 1) & 1, abort_flag, p.flags);
                if (!ok) break;
                ++merges;
                const float m1 = st[(slot ^ 1) * 256 + row], l1 = st[(slot ^ 1) * 256 + 128 + row];
                __syncwarp();
                if (lane == 0) mbar_arrive(state_empty);
                // (a NaN m makes its factor NaN; both slots do the same arithmetic on (slot 0, slot 1))
                const float mn = fmaxf(m, m1);
                f0 = m == -INFINITY ? 0.f : ex2(m - mn);
                f1 = m1 == -INFINITY ? 0.f : ex2(m1 - mn);
                l = slot ? fmaf(l1, f1, l * f0) : fmaf(l, f0, l1 * f1);
                m = mn;
            }
            other_count += n_other;
            tc_fence_after();
            const int part_slot = f[kPart];
            const bool empty_row = m == -INFINITY && l == 0.f;  // attended to nothing: 0 (a NaN sum stays NaN)
            if (part_slot < 0) {
                const float inv = empty_row ? 0.f : 1.f / l;
                f0 *= inv;
                f1 *= inv;
            }
            const int ti = (pair ? slot * tps : 0) + (row >> p.g_shift);
            const bool store = ti < f[kNTok];
            const int h = f[kHead] + (row & ((1 << p.g_shift) - 1));
            uint16_t *dst = p.out + ((size_t)(f[kTok] + ti) * p.Hq + h) * D;
            float *part = p.part + (size_t)max(part_slot, 0) * ((D + 2) * kItemRows) + (pair ? slot : 0) * kSlotRows + row;
            volatile const int *bad = reinterpret_cast<volatile const int *>(sm + L::kBad + (k & 1) * kBadBytes);
            // (the tiles this slot used are in the list: their products waited
            // for warp 11; further ones may come in, for rows it does not see)
            const int n_bad = n_mine > 0 || !pair ? bad[0] : 0;
            if (n_bad > 0) __threadfence_block();
            const int q0 = pair ? 0 : slot * (D / 32), q1 = pair ? D / 16 : q0 + D / 32;  // groups of 16 head dims
#pragma unroll 1
            for (int q = q0; q < q1; ++q) {
                float o[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = 0.f;
                if (n_mine > 0) tmem_ld16(to + slot * L::kOStep + q * 16, o);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] *= f0;
                if (!pair && n_other > 0) {
                    float o1[16];
                    tmem_ld16(to + (slot ^ 1) * L::kOStep + q * 16, o1);
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = fmaf(o1[i], f1, o[i]);
                }
                if (q + 1 == q1) {  // the sums have been read: the next segment may overwrite them
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(o_free);
                }
                if (empty_row) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = 0.f;
                }
                // V rows that warp 11 took out (none, as a rule): p v for those this row sees
#pragma unroll 1
                for (int e = 0; e < n_bad; ++e) {
                    const int r0 = bad[1 + 5 * e];
#pragma unroll 1
                    for (int j = 0; j < kTile; ++j) {
                        if (!((bad[2 + 5 * e + (j >> 5)] >> (j & 31)) & 1) || !(allowed(r0 + j) & 1u)) continue;
                        const size_t kv = ((size_t)f[kRowBase] + r0 + j) * D;
                        const uint16_t *qr = p.Q + (dst - p.out);
                        float x = 0.f;
#pragma unroll 1
                        for (int i = 0; i < D; ++i)
                            x = fmaf(__uint_as_float((uint32_t)qr[i] << 16), __uint_as_float((uint32_t)p.K[kv + i] << 16), x);
                        rf = row_factor(m);
                        x = ex2(fmaf(x, p.c * rf, -m * rf)) * (part_slot < 0 ? 1.f / l : 1.f);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            o[i] = fmaf(x, __uint_as_float((uint32_t)p.V[kv + q * 16 + i] << 16), o[i]);
                    }
                }
                if (part_slot < 0) {
                    if (store) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint4 w;
                            w.x = pack_bf16(o[8 * i + 0], o[8 * i + 1]);
                            w.y = pack_bf16(o[8 * i + 2], o[8 * i + 3]);
                            w.z = pack_bf16(o[8 * i + 4], o[8 * i + 5]);
                            w.w = pack_bf16(o[8 * i + 6], o[8 * i + 7]);
                            *reinterpret_cast<uint4 *>(dst + q * 16 + i * 8) = w;
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) part[(size_t)(q * 16 + i) * kItemRows] = o[i];
                }
            }
            if (part_slot >= 0 && (pair || slot == 0)) {
                part[(size_t)D * kItemRows] = m;
                part[(size_t)(D + 1) * kItemRows] = l;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(seg_empty(k & 1));
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Joins the states of an item that was shared out:
//   out = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s.
// blockIdx.x is the entry, y a block of 32 rows (lane = row, so the states are
// read 128 bytes at a time), z a block of 32 head dims, 8 per warp.  Latency is
// all there is to it: the loads of 8 states are in flight at once, and where an
// item has many states (few items over a long context) SG = 4 groups of 4
// warps take every fourth state each (a 64K tree's 19 states in one round
// trip instead of three).
template <int D, int SG>
__global__ void __launch_bounds__(128 * SG)
multi_join_kernel(const Params p) {
    __shared__ float tile[SG][32][33], ml[SG][2][32];
    const int tid = threadIdx.x, lane = tid & 31, dg = (tid >> 5) & 3, sg = tid >> 7;
    griddep_wait();
    griddep_launch_dependents();
    const int4 e = *reinterpret_cast<const int4 *>(p.joins + 8 * blockIdx.x);
    const int rows = p.joins[8 * blockIdx.x + 4];
    // CTAs from .. from + n - 1: state 2 c + 1 of the first, 2 c of the others
    const int from = e.x, n = e.y, tok = e.z, head = e.w;
    if (from < 0 || (int)blockIdx.y * 32 >= rows) return;
    // (entries of a call whose waits ran out may be anything: stay in the arrays)
    if (n < 1 || from + n > p.ctas || rows > kItemRows || tok < 0 || tok + (rows >> p.g_shift) > p.n_tokens ||
        head < 0 || head + (1 << p.g_shift) > p.Hq)
        return;
    constexpr size_t kRec = (size_t)(D + 2) * kItemRows;
    const int d0 = blockIdx.z * 32 + dg * 8;
    const float *base = p.part + blockIdx.y * 32 + lane;
    float M = -INFINITY, l = 0.f, acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    constexpr int kBatch = 8;
    for (int s0 = sg; s0 < n; s0 += SG * kBatch) {
        float ms[kBatch], ls[kBatch], v[kBatch][8];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int s = s0 + SG * u;
            ms[u] = -INFINITY;
            ls[u] = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] = 0.f;
            if (s < n) {
                const float *r = base + (size_t)(2 * (from + s) + (s == 0)) * kRec;
                ms[u] = r[(size_t)D * kItemRows];
                ls[u] = r[(size_t)(D + 1) * kItemRows];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[u][i] = r[(size_t)(d0 + i) * kItemRows];
            }
        }
        float mn = M;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) mn = fmaxf(mn, ms[u]);
        const float f = M == -INFINITY ? 0.f : ex2(M - mn);
        l *= f;
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] *= f;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const float fu = ms[u] == -INFINITY ? 0.f : ex2(ms[u] - mn);  // NaN stays NaN
            l = fmaf(ls[u], fu, l);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = fmaf(v[u][i], fu, acc[i]);
        }
        M = mn;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) tile[sg][lane][dg * 8 + i] = acc[i];
    if (dg == 0) {
        ml[sg][0][lane] = M;
        ml[sg][1][lane] = l;
    }
    __syncthreads();
    if (tid >= 128) return;
    const int r = tid >> 2, c8 = (tid & 3) * 8, rr = blockIdx.y * 32 + r;
    if (rr >= rows) return;
    float mn = -INFINITY, f[SG], sum = 0.f;
#pragma unroll
    for (int g = 0; g < SG; ++g) mn = fmaxf(mn, ml[g][0][r]);
#pragma unroll
    for (int g = 0; g < SG; ++g) {
        f[g] = ml[g][0][r] == -INFINITY ? 0.f : ex2(ml[g][0][r] - mn);
        sum = fmaf(ml[g][1][r], f[g], sum);
    }
    const float inv = mn == -INFINITY && sum == 0.f ? 0.f : 1.f / sum;  // (attended to nothing: 0)
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float x = 0.f;
#pragma unroll
        for (int g = 0; g < SG; ++g) x = fmaf(tile[g][r][c8 + i], f[g], x);
        o[i] = x * inv;
    }
    const uint4 w = make_uint4(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7]));
    const size_t at = (size_t)(tok + (rr >> p.g_shift)) * p.Hq + head + (rr & ((1 << p.g_shift) - 1));
    *reinterpret_cast<uint4 *>(p.out + at * D + blockIdx.z * 32 + c8) = w;
}

// ---------------------------------------------------------------- host side

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeTiledFn>(f);
    }();
    return fn;
}

// bf16 tensor of `rank` dimensions (innermost first, packed), 128-byte
// swizzled boxes, zero fill outside.
bool make_map(CUtensorMap *m, const void *base, int rank, const cuuint64_t *dims, const cuuint32_t *box) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t strides[2] = {dims[0] * 2, dims[0] * dims[1] * 2};
    cuuint32_t es[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void *>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int log2_int(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

// Items of one KV head: every sequence's tokens in groups of 256 / G.
long long item_bound(const tb_dims &d, int32_t n_tokens, int32_t max_new) {
    const int tpi = kItemRows / (d.n_q_heads / d.n_kv_heads);
    const long long a = (long long)n_tokens / tpi + d.batch, b = (long long)d.batch * ((max_new + tpi - 1) / tpi);
    return a < b ? a : b;
}

// Deal whole items out by the counter, or equal shares of all tiles?  In tiles
// of the longest context the cache holds (the lengths are the device's): whole
// items take the average load and, at the end, about half of the smallest item
// that may come last; at least one whole item.  Shares are even but write and
// join states, about 16 tiles' time
// (992 items of 25 to 64 tiles: 371 us in shares, 358 by the counter; 16 items of
// 514 tiles: 141 against 838).  Where the cache is much larger than what it
// holds the rule takes short sequences for long ones: 16 prompts of 1 to 300
// tokens 11.6 us in a cache of 512 rows, by the counter, and 22.4 in one of
// 64K, in shares; five of 500 to 5,000 tokens 347 us (8K rows) and 362 (64K).
bool use_shares(const tb_dims &d, int32_t max_new, bool tree, long long items) {
    const double ctas = num_sms(), n = (double)items * d.n_kv_heads;
    const double longest = (d.ctx_cap + kTile - 1) / kTile;
    const double shortest = tree ? longest : fmax(1.0, (double)(d.ctx_cap - max_new) / kTile);
    const double average = 0.5 * (longest + shortest);
    if (n * (longest + 1.0) * 7.0 >= 2147483648.0) return false;  // (positions on the line are 32 bits)
    const double whole = fmax(longest, n * average / ctas + 0.5 * shortest);
    return n * average / ctas + 16.0 < whole;
}

template <int D>
cudaError_t launch_d(const tb_dims &d, const uint16_t *Q, const uint16_t *K, const uint16_t *V, Params &p,
                     cudaStream_t st) {
    using L = Lay<D>;
    const cuuint32_t G = 1u << p.g_shift;
    CUtensorMap mQ, mK, mV;
    const cuuint64_t qd[3] = {D, (cuuint64_t)d.n_q_heads, (cuuint64_t)p.n_tokens};
    const cuuint32_t qb[3] = {64, G, kSlotRows / G};
    const cuuint64_t kd[2] = {D, (cuuint64_t)d.batch * d.n_kv_heads * d.ctx_cap};
    const cuuint32_t kb[2] = {64, kTile};
    if (!make_map(&mQ, Q, 3, qd, qb) || !make_map(&mK, K, 2, kd, kb) || !make_map(&mV, V, 2, kd, kb))
        return cudaErrorInvalidValue;
    static std::atomic<int> smem_set[kMaxDevices];
    cudaError_t e = ensure_dynamic_smem((const void *)multi_attn_kernel<D>, L::kBytes, smem_set);
    if (e != cudaSuccess) return e;
    const long long items = (long long)p.item_bound * p.Hkv, sms = num_sms();
    const unsigned ctas = (unsigned)(p.part || items > sms ? sms : items);
    p.ctas = (int)ctas;
    e = launch_pdl(multi_attn_kernel<D>, dim3(ctas), dim3(kThreads), L::kBytes, st, mQ, mK, mV, p);
    if (e != cudaSuccess || !p.part) return e;
    const dim3 grid(items < sms ? (unsigned)items : ctas, kItemRows / 32, D / 32);
    // about sms / items states an item: above 6, 4 groups of warps read them
    // (trees over 32K, both kernels: 8 items 39.4 us with one group, 36.1 with
    // four; 16 items 58.8, 59.0; 32 items 98, 104)
    if (sms > 6 * items) return launch_pdl(multi_join_kernel<D, 4>, grid, dim3(512), 0, st, p);
    return launch_pdl(multi_join_kernel<D, 1>, grid, dim3(128), 0, st, p);
}

}  // namespace

// Workspace: flag word, counter (at 64), a word for each (sequence, KV head) that
// is left alone, the CTAs' join entries, their states.  The words are the decode
// attention's tickets, which have to be zero between calls: a program that
// verifies a tree and then decodes may use one workspace for both.
size_t joins_at(const tb_dims &d) { return kWsHeaderBytes + align_up((size_t)d.batch * d.n_kv_heads * 4, 256); }
size_t states_at(const tb_dims &d) { return joins_at(d) + align_up((size_t)num_sms() * 32, 256); }

size_t multi_attn_ws_bytes(const tb_dims &d, int32_t n_tokens, int32_t max_new, bool tree) {
    if (!use_shares(d, max_new, tree, item_bound(d, n_tokens, max_new))) return kWsHeaderBytes;
    return states_at(d) + (size_t)num_sms() * 2 * (d.head_dim + 2) * kItemRows * sizeof(float);
}

cudaError_t launch_multi_attn(const tb_dims &d, const uint16_t *Q, const uint16_t *K, const uint16_t *V,
                              const int32_t *q_begin, int32_t n_tokens, int32_t max_new, const int32_t *ctx_len,
                              const uint32_t *mask, float scale, uint16_t *out, void *ws, cudaStream_t st) {
    Params p{};
    uint8_t *w = static_cast<uint8_t *>(ws);
    p.q_begin = q_begin;
    p.ctx_len = ctx_len;
    p.mask = mask;
    p.Q = Q;
    p.K = K;
    p.V = V;
    p.out = out;
    p.flags = reinterpret_cast<uint32_t *>(w);
    p.counter = reinterpret_cast<uint32_t *>(w + 64);
    p.batch = d.batch;
    p.Hq = d.n_q_heads;
    p.Hkv = d.n_kv_heads;
    p.cap = d.ctx_cap;
    p.n_tokens = n_tokens;
    p.max_new = max_new;
    p.mask_words = (max_new + 31) / 32;
    p.g_shift = log2_int(d.n_q_heads / d.n_kv_heads);
    p.item_bound = (int)item_bound(d, n_tokens, max_new);
    if (use_shares(d, max_new, mask != nullptr, p.item_bound)) {
        p.joins = reinterpret_cast<int32_t *>(w + joins_at(d));
        p.part = reinterpret_cast<float *>(w + states_at(d));
    }
    p.c = scale * 1.4426950408889634f;
    return d.head_dim == 128 ? launch_d<128>(d, Q, K, V, p, st) : launch_d<64>(d, Q, K, V, p, st);
}

}  // namespace tb
