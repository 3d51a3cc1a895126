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
// only when a logit exceeds it by more than 8 (log2 units), so the accumulator
// is rescaled rarely; p stays below 2^8 and the sums, held in fp32, are exact
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
// 9 loads (TMA); 10 and 11 only complete the warpgroup whose registers the
// softmax warps take over (a softmax thread holds a whole row of a tile, 128
// logits).  Tensor memory: S0 | S1 | O0 | O1, 128 columns each; the
// weights P (bf16) overwrite the first half of their S columns and are read
// from there as the A operand of the second product.
//
// Few items over a long context are split along it (gridDim covers
// splits x items); each CTA then writes its rows' unnormalised state and a
// second kernel joins them.
#include <cuda.h>

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
// (2 * 128 * 224 + 128 * 56 = 384 * 168).
constexpr int kRegsSoftmax = 216, kRegsOther = 72;
static_assert(256 * kRegsSoftmax + 128 * kRegsOther <= kThreads * 168, "register split");
constexpr int kMaxSplits = 32;
constexpr uint32_t kTmemCols = 512;
constexpr float kLazy = 8.0f;               // log2 units
constexpr uint32_t kBarMerge = 1;           // named barrier of the 256 softmax threads
constexpr int kPolyOf8 = 2;                 // of 8 pairs of weights, those worked out on the FMA pipe
constexpr uint32_t kFullMask = 0xffffffffu;

template <int D>
struct Lay {
    static constexpr int kAtoms = D / 64;
    static constexpr int kOperand = 128 * D * 2;  // bytes of a 128-row operand (Q slot, K or V tile)
    // K and V tiles share one ring: 160 KB in flight covers the latency of HBM
    static constexpr int kStages = D == 128 ? 5 : 10;
    static constexpr int kRing = 2 * kOperand;
    static constexpr int kBar = kRing + kStages * kOperand;
    static constexpr int kNumBars = 2 * kStages + 3 + 8;
    static constexpr int kMisc = kBar + kNumBars * 8;
    static constexpr int kBytes = kMisc + 64 + 1024;  // + alignment slack
    static_assert(kBar % 8 == 0, "mbarrier alignment");
    static_assert(kBytes <= 227 * 1024, "shared memory");
};

// A bounded mbarrier wait that also gives up as soon as another role of the
// CTA has given up.  The thread sleeps in the barrier between checks.
__device__ __forceinline__ bool wait_role(uint32_t bar, uint32_t parity, volatile int *abort_flag, uint32_t *flags) {
    if (mbar_try_wait_sleep(bar, parity, 20000u)) return true;
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
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// 2^x for a pair on the FMA pipe: x = n + f with n the nearest integer, 2^f by
// a cubic with the smallest largest relative error on [-1/2, 1/2] (1.02e-4,
// fitted for this kernel; 2^0 = 1 exactly; the weights' rounding to bf16 is up
// to 40 times that), n added to the exponent.  x is
// held at -127 or above, where the result is exactly 0.
__device__ __forceinline__ void ex2_poly2(uint64_t x2, float &e0, float &e1) {
    float a, b;
    unpack2(x2, a, b);
    const uint64_t x = pack2(fmaxf(a, -127.f), fmaxf(b, -127.f));
    constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer in the low bits
    const uint64_t t = add2(x, pack2(kMagic, kMagic));
    const uint64_t n = add2(t, pack2(-kMagic, -kMagic));
    const uint64_t f = sub2(x, n);
    uint64_t r = fma2(f, pack2(0.05500893294811249f, 0.05500893294811249f),
                      pack2(0.24221095442771912f, 0.24221095442771912f));
    r = fma2(r, f, pack2(0.6932829022407532f, 0.6932829022407532f));
    r = fma2(r, f, pack2(1.f, 1.f));
    float t0, t1, r0, r1;
    unpack2(t, t0, t1);
    unpack2(r, r0, r1);
    e0 = __uint_as_float(__float_as_uint(r0) + (__float_as_uint(t0) << 23));
    e1 = __uint_as_float(__float_as_uint(r1) + (__float_as_uint(t1) << 23));
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
    uint16_t *out;
    float *part;            // split states, nullptr when splits == 1
    uint32_t *flags;
    int batch, Hq, Hkv, cap, n_tokens, max_new, mask_words;
    int g_shift;            // G = 1 << g_shift heads per group
    int item_bound, splits;
    float c;                // scale * log2(e)
};

// One work item: up to 256 rows (tokens tok0 .. tok0 + ntok of sequence b).
struct Item {
    int b, begin, n, T;  // the sequence: first packed token, new tokens, length
    int tok0, ntok;      // tokens of this item (index within the sequence)
    int index;           // among all items of a KV head
    bool any;
};

// Item `tau` counted over the sequences in packing order.  Every lane of the
// calling warp takes part; sequences with more than max_new tokens keep
// max_new (the rest is reported and left out).
__device__ __forceinline__ Item find_item(const Params &p, int tau, int lane) {
    const int tpi_shift = 8 - p.g_shift;  // tokens per item: 256 / G
    Item it{};
    int before = 0;
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
        int n = 0;
        if (b0 + lane < p.batch) n = min(seq_span(p.q_begin, b0 + lane, p.n_tokens).n, p.max_new);
        const int items = (n + (1 << tpi_shift) - 1) >> tpi_shift;
        int incl = items;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kFullMask, incl, o);
            if (lane >= o) incl += v;
        }
        const uint32_t hit = __ballot_sync(kFullMask, tau < before + incl);
        if (hit) {
            const int l = __ffs(hit) - 1;
            const int first = before + __shfl_sync(kFullMask, incl - items, l);
            it.b = b0 + l;
            const SeqSpan sp = seq_span(p.q_begin, it.b, p.n_tokens);
            it.begin = sp.begin;
            it.n = sp.n;
            it.tok0 = (tau - first) << tpi_shift;
            it.ntok = min(1 << tpi_shift, min(sp.n, p.max_new) - it.tok0);
            it.index = tau;
            it.any = true;
            return it;
        }
        before += __shfl_sync(kFullMask, incl, 31);
    }
    return it;
}

// K/V tiles that tokens up to `last` of the item's sequence attend to.
__device__ __forceinline__ int tiles_upto(const Params &p, const Item &it, int last) {
    const int rows = p.mask ? it.T : min(it.T, it.T - it.n + last + 1);
    return max(0, (rows + kTile - 1) / kTile);
}

// Tiles of split s of an item with `tiles` tiles: [first, last).
__device__ __forceinline__ void split_range(int tiles, int splits, int s, int &first, int &last) {
    const int per = (tiles + splits - 1) / splits;
    first = min(s * per, tiles);
    last = min(first + per, tiles);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
multi_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const Params p) {
    using L = Lay<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_addr(sm);
    volatile int *misc = reinterpret_cast<volatile int *>(sm + L::kMisc);  // TMEM base, abort flag, item
    volatile int *abort_flag = misc + 1;
    auto bar = [&](int i) -> uint32_t { return sb + L::kBar + 8u * (uint32_t)i; };
    auto full = [&](int s) { return bar(s); };
    auto empty = [&](int s) { return bar(L::kStages + s); };
    const uint32_t q_full = bar(2 * L::kStages), drain = bar(2 * L::kStages + 1), tail_done = bar(2 * L::kStages + 2);
    auto s_full = [&](int s) { return bar(2 * L::kStages + 3 + s); };
    auto p_full = [&](int s, int half) { return bar(2 * L::kStages + 5 + 2 * s + half); };  // keys 0..63, 64..127
    auto o_done = [&](int s) { return bar(2 * L::kStages + 9 + s); };

    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(kFullMask, tid >> 5, 0);
    griddep_wait();
    griddep_launch_dependents();

    // grid: items from the last to the first (a sequence's last tokens have
    // the most tiles, so the long items start first), KV heads and splits inside
    const int per_item = p.Hkv * p.splits;
    const int tau = p.item_bound - 1 - (int)(blockIdx.x / per_item);
    const int rem = (int)(blockIdx.x % per_item);
    const int g = rem / p.splits, split = rem % p.splits;
    Item it = find_item(p, tau, lane);
    if (!it.any) return;
    const bool report = tid == 0 && g == 0 && split == 0;
    it.T = clamp_ctx(p.ctx_len[it.b], p.cap, p.flags, report);
    if (report && (it.n > it.T || it.n > p.max_new)) raise_flag(p.flags, TB_FLAG_CTX_RANGE);

    // Two ways to use the slots: `pair`: rows 0..127 and 128..255 over the
    // same tiles; else both slots hold rows 0..127 and take every other tile.
    const int tps = kSlotRows >> p.g_shift;  // tokens per slot
    const bool pair = it.ntok > tps;
    const int tiles_item = tiles_upto(p, it, it.tok0 + it.ntok - 1);
    int t_first, t_last;
    split_range(tiles_item, p.splits, split, t_first, t_last);
    if (p.splits > 1 && t_first >= t_last) return;  // the join skips empty splits
    // tiles of the whole CTA and of slot 0 (in pairs its rows, the earlier
    // tokens, may end a tile or two before slot 1's)
    const int nt = t_last - t_first;
    const int nt0 = pair ? max(0, min(t_last, tiles_upto(p, it, it.tok0 + tps - 1)) - t_first) : (nt + 1) / 2;
    const int nt1 = pair ? nt : nt / 2;
    // rows of the CTA's last tile that lie below the length, if not all do (else 0)
    const int tail_rows = nt > 0 && t_last * kTile > it.T ? it.T - (t_last - 1) * kTile : 0;

    if (tid == 0) {
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        mbar_init(q_full, 1);
        mbar_init(drain, 1);
        mbar_init(tail_done, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(s_full(s), 1);
            mbar_init(p_full(s, 0), 4);
            mbar_init(p_full(s, 1), 4);
            mbar_init(o_done(s), 1);
        }
        misc[1] = 0;
        misc[2] = it.begin + it.tok0;  // what only the epilogue needs: kept out of the loop's registers
        misc[3] = it.ntok;
        misc[4] = it.index;
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(sb + L::kMisc, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)misc[0];
    const int row_base = (int)(((size_t)it.b * p.Hkv + g) * (size_t)p.cap);  // < 2^31 (checked on the host)

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegsOther));
        if (warp == 9) {
        // ============================================================ loads
        // Ring order = the order in which the products use the tiles: in
        // pairs K0 V0 K1 V1 ..; else K0 K1 V0 K2 V1 .. V(n-2) V(n-1).
        int n_issued = 0;
        if (lane == 0) {
            prefetch_tensormap(&tmQ);
            prefetch_tensormap(&tmK);
            prefetch_tensormap(&tmV);
            const int qn = pair ? 2 : 1;
            mbar_arrive_expect_tx(q_full, (uint32_t)(qn * L::kOperand));
            for (int s = 0; s < qn; ++s)
#pragma unroll
                for (int a = 0; a < L::kAtoms; ++a)
                    tma_load_3d(sb + s * L::kOperand + a * 16384, &tmQ, q_full, a * 64, g << p.g_shift,
                                it.begin + it.tok0 + s * tps);
            int i = 0;
            bool ok = true;
            auto load = [&](const CUtensorMap *map, int tile) {
                const int s = i % L::kStages;
                if (i >= L::kStages) ok = ok && wait_role(empty(s), ((i / L::kStages) + 1) & 1, abort_flag, p.flags);
                if (!ok) return;
                mbar_arrive_expect_tx(full(s), L::kOperand);
#pragma unroll
                for (int a = 0; a < L::kAtoms; ++a)
                    tma_load_2d(sb + L::kRing + s * L::kOperand + a * 16384, map, full(s), a * 64,
                                row_base + (t_first + tile) * kTile);
                ++i;
            };
            if (pair) {
                for (int t = 0; t < nt && ok; ++t) {
                    load(&tmK, t);
                    if (ok) load(&tmV, t);
                }
            } else {
                if (nt > 0) load(&tmK, 0);
                if (nt > 1) load(&tmK, 1);
                for (int t = 0; t < nt && ok; ++t) {
                    load(&tmV, t);
                    if (ok && t + 2 < nt) load(&tmK, t + 2);
                }
            }
            mbar_wait_bounded(q_full, 0, p.flags);
            n_issued = i;
        }
        n_issued = __shfl_sync(kFullMask, n_issued, 0);
        // leave only when every copy has landed
        for (int k = max(0, n_issued - L::kStages); k < n_issued; ++k)
            mbar_wait_bounded(full(k % L::kStages), (k / L::kStages) & 1, p.flags);
        if (tail_rows > 0) {
            // the last V tile (the ring's last item) reaches past the length:
            // cache rows there may hold anything, NaN included, and 0 * NaN
            // must not reach the sums
            uint8_t *v = sm + L::kRing + ((2 * nt - 1) % L::kStages) * L::kOperand;
            if (n_issued == 2 * nt) {
#pragma unroll
                for (int a = 0; a < L::kAtoms; ++a)
                    for (int o = tail_rows * 128 + lane * 16; o < kTile * 128; o += 512)
                        *reinterpret_cast<uint4 *>(v + a * 16384 + o) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(tail_done);
        }
        }
        if (warp == 8) {
        // ============================================================ products
        // One thread issues all of them.  Per slot the order is S(0), then
        // PV(j) S(j+1): S(j+1) overwrites the columns of P(j), which PV(j)
        // has read by then (the products of one thread run in order).  PV is
        // issued in two halves of 64 keys, so that its first half runs while
        // the softmax works out the second half of the weights.
        if (elect_one()) {
            constexpr uint32_t id_s = idesc_bf16_f32(128, kTile);
            constexpr uint32_t id_o = idesc_bf16_f32(128, D) | (1u << 16);  // B (V) MN-major
            constexpr uint32_t kStep = L::kOperand >> 4;
            const uint64_t kd = sw128_kmajor_desc(sb), vd = sw128_mnmajor_desc(sb + L::kRing, 16384);
            const uint32_t q_lo = (uint32_t)kd, hi = (uint32_t)(kd >> 32);
            const uint32_t k_lo = q_lo + (L::kRing >> 4), v_lo = (uint32_t)vd;
            int k_stage = 0, v_stage = 0, next = 0;
            uint32_t next_parity = 0;
            bool ok = wait_role(q_full, 0, abort_flag, p.flags);
            auto acquire = [&](int &stage) {
                stage = next;
                if (ok) ok = wait_role(full(next), next_parity, abort_flag, p.flags);
                if (++next == L::kStages) {
                    next = 0;
                    next_parity ^= 1u;
                }
            };
            auto issue_s = [&](int slot) {
                tc_fence_after();
                const uint32_t q = q_lo + (pair ? slot : 0) * kStep, k = k_lo + k_stage * kStep;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t o = (uint32_t)((kk >> 2) * 1024 + (kk & 3) * 2);
                    umma_ss(tmem + slot * 128, q + o, k + o, hi, id_s, kk > 0);
                }
                umma_commit(s_full(slot));
            };
            auto issue_pv = [&](int slot, int j) {
                const uint32_t v = v_lo + v_stage * kStep;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (ok) ok = wait_role(p_full(slot, half), j & 1, abort_flag, p.flags);
                    if (!ok) return;
                    tc_fence_after();
#pragma unroll
                    for (int kk = half * 4; kk < half * 4 + 4; ++kk)
                        umma_ts(tmem + 256 + slot * 128, tmem + slot * 128 + kk * 8, v + kk * 128, hi, id_o,
                                (j | kk) ? 1u : 0u);
                }
                umma_commit(o_done(slot));
            };
            // step i belongs to slot i & 1; in pairs steps 2t and 2t + 1 use
            // tile t, else step i uses tile i.  Each round: the step's PV,
            // then the same slot's next S.
            const int steps = pair ? 2 * nt : nt;
#pragma unroll 1
            for (int i = -2; i < steps && ok; ++i) {
                const int slot = i & 1, j = i >> 1, n_slot = slot ? nt1 : nt0;
                const bool first = !pair || slot == 0, last = !pair || slot == 1;
                if (i >= 0) {
                    if (first) {
                        acquire(v_stage);
                        if (tail_rows > 0 && (pair ? j : i) + 1 == nt && ok)
                            ok = wait_role(tail_done, 0, abort_flag, p.flags);
                    }
                    if (j < n_slot) issue_pv(slot, j);
                    if (!ok) break;
                    if (last) umma_commit(empty(v_stage));
                }
                if (i + 2 < steps) {
                    if (first) acquire(k_stage);
                    if (!ok) break;
                    if (j + 1 < n_slot) issue_s(slot);
                    if (last) umma_commit(empty(k_stage));
                }
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
        const uint32_t ts = tmem + lane_base + slot * 128, to = tmem + lane_base + 256 + slot * 128;
        // this thread's row: token (within the sequence) and its last visible row
        const int tok = it.tok0 + ((pair ? slot : 0) * tps) + (row >> p.g_shift);
        const bool live = tok < it.tok0 + it.ntok;
        const int base = it.T - it.n;  // first row of the new tokens
        // the row sees every cache row below all_end, and of the drafted rows
        // from all_end to draft_end those with a bit in mrow
        const uint32_t *mrow = p.mask && live ? p.mask + (size_t)(it.begin + tok) * p.mask_words : nullptr;
        const int all_end = !live ? 0 : p.mask ? base : base + tok + 1;
        const int draft_end = base + min(it.n, p.max_new);
        const int n_mine = slot ? nt1 : nt0;
        // tiles from `masked_from` on hold rows that some row of this slot does not see
        const int masked_from = p.mask ? max(base, 0) / kTile
                                       : max(0, base + it.tok0 + (pair ? slot : 0) * tps + 1) / kTile;
        float m = -INFINITY, l = 0.f;
        bool ok = true;

        // which of the 32 cache rows from p0 on this row attends to
        auto allowed = [&](int p0) -> uint32_t {
            uint32_t d = bits_below(all_end - p0);
            if (mrow) {
                const int j0 = p0 - all_end;  // drafted token at p0
                uint32_t x = 0u;
                if (j0 >= 0) {
                    const int w = j0 >> 5, sh = j0 & 31;
                    if (w < p.mask_words) x = __ldg(mrow + w) >> sh;
                    if (sh && w + 1 < p.mask_words) x |= __ldg(mrow + w + 1) << (32 - sh);
                } else if (j0 > -32) {
                    x = __ldg(mrow) << -j0;
                }
                d |= x & bits_below(draft_end - p0);
            }
            return d;
        };

        for (int j = 0; j < n_mine; ++j) {
            const int tile = t_first + (pair ? j : 2 * j + slot);
            const bool masked = tile >= masked_from;
            uint32_t see[4];
            if (masked) {
#pragma unroll
                for (int q = 0; q < 4; ++q) see[q] = allowed(tile * kTile + q * 32);
            }
            ok = wait_warp(s_full(slot), j & 1, abort_flag, p.flags);
            if (!ok) break;
            tc_fence_after();
            uint32_t s[4][32];
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_ld32(ts + q * 32, s[q]);
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_wait32(s[q]);
            if (masked) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (!((see[q] >> k) & 1u)) s[q][k] = 0xff800000u;  // -inf
            }
            float mx[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) mx[q] = max3_nan(__uint_as_float(s[q][0]), __uint_as_float(s[q][1]), __uint_as_float(s[q][2]));
#pragma unroll
            for (int k = 3; k < 31; k += 2)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    mx[q] = max3_nan(mx[q], __uint_as_float(s[q][k]), __uint_as_float(s[q][k + 1]));
#pragma unroll
            for (int q = 0; q < 4; ++q) mx[q] = max3_nan(mx[q], __uint_as_float(s[q][31]), mx[q]);
            float top = max3_nan(mx[0], mx[1], max3_nan(mx[2], mx[3], mx[3])) * p.c;
            // a NaN or +inf logit makes the row's softmax NaN: so becomes m, and l with it
            if (!(top < INFINITY)) top = NAN;
            const bool raise = !(top <= m + kLazy);  // also the first logit of a row (m = -inf)
            if (__any_sync(kFullMask, raise)) {
                const float m_new = raise ? top : m;
                const float f = m_new == m ? 1.f : ex2(m - m_new);  // (-inf stays -inf while nothing is seen)
                if (j > 0) {
                    ok = wait_warp(o_done(slot), (j - 1) & 1, abort_flag, p.flags);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int q = 0; q < D / 16; ++q) {  // rare: kept small, the logits fill the registers
                        float o[16];
                        uint32_t w[16];
                        tmem_ld16(to + q * 16, o);
#pragma unroll
                        for (int k = 0; k < 16; ++k) w[k] = __float_as_uint(o[k] * f);
                        tmem_st16(to + q * 16, w);
                    }
                }
                l *= f;
                m = m_new;
            }
            const float mm = m == -INFINITY ? 0.f : m;  // a row that has seen nothing: 2^(-inf - 0) = 0
            const uint64_t c2 = pack2(p.c, p.c), nm2 = pack2(-mm, -mm);
            uint64_t sum2[2] = {0ull, 0ull};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t w[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const uint64_t x2 = fma2(pack2(__uint_as_float(s[q][2 * k]), __uint_as_float(s[q][2 * k + 1])), c2, nm2);
                    float e0, e1;
                    if ((k & 7) < kPolyOf8) {
                        ex2_poly2(x2, e0, e1);
                    } else {
                        unpack2(x2, e0, e1);
                        e0 = ex2(e0);
                        e1 = ex2(e1);
                    }
                    sum2[k & 1] = add2(sum2[k & 1], pack2(e0, e1));
                    // rounded to bf16 for the second product: 2^-9 relative per
                    // weight, below the rounding of the bf16 result
                    w[k] = pack_bf16(e0, e1);
                }
                tmem_st16(ts + q * 16, w);
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

        // ---- epilogue
        if (ok && n_mine > 0) ok = wait_warp(o_done(slot), (n_mine - 1) & 1, abort_flag, p.flags);
        if (!pair && ok) {  // both slots' products are done before the ring's memory is reused
            const int other = slot ? nt0 : nt1;
            if (other > 0) ok = wait_warp(o_done(slot ^ 1), (other - 1) & 1, abort_flag, p.flags);
        }
        tc_fence_after();
        float *xch = reinterpret_cast<float *>(sm + L::kRing);  // [D + 2][128]: slot 1's state
        if (!pair && nt1 > 0) {
            if (slot == 1) {
                if (ok) {
#pragma unroll 1
                    for (int q = 0; q < D / 32; ++q) {
                        uint32_t o[32];
                        tmem_ld32(to + q * 32, o);
                        tmem_wait32(o);
#pragma unroll
                        for (int k = 0; k < 32; ++k) xch[(q * 32 + k) * 128 + row] = __uint_as_float(o[k]);
                    }
                    xch[D * 128 + row] = m;
                    xch[(D + 1) * 128 + row] = l;
                }
            }
            bar_named(kBarMerge, 256);
        }
        if (ok && (pair || slot == 0)) {
            float f0 = 1.f, f1 = 0.f;
            const bool two = !pair && nt1 > 0;
            if (two) {
                const float m1 = xch[D * 128 + row], l1 = xch[(D + 1) * 128 + row];
                const float mn = fmaxf(m, m1);
                f0 = m == -INFINITY ? 0.f : ex2(m - mn);
                f1 = m1 == -INFINITY ? 0.f : ex2(m1 - mn);
                l = l * f0 + l1 * f1;
                m = mn;
            }
            const bool empty_row = !(l > 0.f) && !(l != l);  // attended to nothing: 0 (a NaN sum stays NaN)
            if (p.splits == 1) {
                const float inv = empty_row ? 0.f : 1.f / l;
                f0 *= inv;
                f1 *= inv;
            }
            const int h = (g << p.g_shift) + (row & ((1 << p.g_shift) - 1));
            const int ti = (pair ? slot * tps : 0) + (row >> p.g_shift);  // token of the item
            const bool store = ti < misc[3];
            uint16_t *dst = p.out + ((size_t)(misc[2] + ti) * p.Hq + h) * D;
            float *part = p.part ? p.part + (((size_t)misc[4] * p.Hkv + g) * p.splits + split) * ((D + 2) * kItemRows) +
                                       (pair ? slot : 0) * kSlotRows + row
                                 : nullptr;
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
                uint32_t o[32];
                if (n_mine > 0) {
                    tmem_ld32(to + q * 32, o);
                    tmem_wait32(o);
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = 0u;
                }
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    float v = __uint_as_float(o[k]) * f0;
                    if (two) v = fmaf(xch[(q * 32 + k) * 128 + row], f1, v);
                    o[k] = empty_row ? 0u : __float_as_uint(v);
                }
                if (p.splits == 1) {
                    if (store) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint4 w;
                            w.x = pack_bf16(__uint_as_float(o[8 * k + 0]), __uint_as_float(o[8 * k + 1]));
                            w.y = pack_bf16(__uint_as_float(o[8 * k + 2]), __uint_as_float(o[8 * k + 3]));
                            w.z = pack_bf16(__uint_as_float(o[8 * k + 4]), __uint_as_float(o[8 * k + 5]));
                            w.w = pack_bf16(__uint_as_float(o[8 * k + 6]), __uint_as_float(o[8 * k + 7]));
                            *reinterpret_cast<uint4 *>(dst + q * 32 + k * 8) = w;
                        }
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) part[(size_t)(q * 32 + k) * kItemRows] = __uint_as_float(o[k]);
                }
            }
            if (p.splits > 1) {
                part[(size_t)D * kItemRows] = m;
                part[(size_t)(D + 1) * kItemRows] = l;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Joins the splits' states: out = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s.
// One CTA: 32 rows of one item; warp w takes the head dims congruent to w
// (lane = row, so the states are read 128 bytes at a time), then the tile is
// turned in shared memory and stored row by row.
template <int D>
__global__ void __launch_bounds__(256)
multi_join_kernel(const Params p) {
    __shared__ float tile[32][D + 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    griddep_wait();
    griddep_launch_dependents();
    Item it = find_item(p, (int)blockIdx.x, lane);
    if (!it.any) return;
    const int g = blockIdx.y, row = blockIdx.z * 32 + lane;
    const int rows = it.ntok << p.g_shift;
    if ((int)blockIdx.z * 32 >= rows) return;
    it.T = clamp_ctx(p.ctx_len[it.b], p.cap, nullptr, false);
    const int tiles = tiles_upto(p, it, it.tok0 + it.ntok - 1);
    const int per = (tiles + p.splits - 1) / p.splits;
    const int used = per > 0 ? (tiles + per - 1) / per : 0;  // splits that had a tile
    constexpr size_t kRec = (size_t)(D + 2) * kItemRows;
    const float *part = p.part + ((size_t)it.index * p.Hkv + g) * p.splits * kRec + row;
    float M = -INFINITY;
    for (int s = 0; s < used; ++s) M = fmaxf(M, part[s * kRec + (size_t)D * kItemRows]);
    float acc[D / 8], l = 0.f;
#pragma unroll
    for (int k = 0; k < D / 8; ++k) acc[k] = 0.f;
    for (int s = 0; s < used; ++s) {
        const float *ps = part + s * kRec;
        const float ms = ps[(size_t)D * kItemRows];
        const float f = ms == -INFINITY ? 0.f : ex2(ms - M);
        l = fmaf(ps[(size_t)(D + 1) * kItemRows], f, l);
#pragma unroll
        for (int k = 0; k < D / 8; ++k) acc[k] = fmaf(ps[(size_t)(k * 8 + warp) * kItemRows], f, acc[k]);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int k = 0; k < D / 8; ++k) tile[lane][k * 8 + warp] = acc[k] * inv;
    __syncthreads();
    for (int e = tid; e < 32 * (D / 8); e += 256) {
        const int r = e / (D / 8), c8 = e % (D / 8), rr = blockIdx.z * 32 + r;
        if (rr >= rows) break;
        const float *t = &tile[r][c8 * 8];
        uint4 w = make_uint4(pack_bf16(t[0], t[1]), pack_bf16(t[2], t[3]), pack_bf16(t[4], t[5]), pack_bf16(t[6], t[7]));
        const int tok = it.begin + it.tok0 + (rr >> p.g_shift);
        const int h = (g << p.g_shift) + (rr & ((1 << p.g_shift) - 1));
        *reinterpret_cast<uint4 *>(p.out + ((size_t)tok * p.Hq + h) * D + c8 * 8) = w;
    }
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

// Splits along the context: as many as fill the SMs in whole waves, counted
// in tiles of the longest possible item, each split paying a few tiles' time
// for its set-up, state and join.
int pick_splits(const tb_dims &d, long long items) {
    const long long ctas = items * d.n_kv_heads, sms = num_sms();
    const long long tiles = (d.ctx_cap + kTile - 1) / kTile;
    long long best = 0;
    int best_s = 1;
    for (int s = 1; s <= kMaxSplits && s <= tiles; ++s) {
        const long long waves = (ctas * s + sms - 1) / sms;
        const long long cost = waves * ((tiles + s - 1) / s + (s > 1 ? 8 : 2));
        if (s == 1 || cost < best) {
            best = cost;
            best_s = s;
        }
        if (ctas * s > 4 * sms) break;
    }
    return best_s;
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
    const dim3 grid((unsigned)((long long)p.item_bound * p.Hkv * p.splits));
    e = launch_pdl(multi_attn_kernel<D>, grid, dim3(kThreads), L::kBytes, st, mQ, mK, mV, p);
    if (e != cudaSuccess || p.splits == 1) return e;
    return launch_pdl(multi_join_kernel<D>, dim3((unsigned)p.item_bound, (unsigned)p.Hkv, kItemRows / 32), dim3(256), 0,
                      st, p);
}

}  // namespace

size_t multi_attn_ws_bytes(const tb_dims &d, int32_t n_tokens, int32_t max_new) {
    const long long items = item_bound(d, n_tokens, max_new);
    const int s = pick_splits(d, items);
    if (s == 1) return kWsHeaderBytes;
    return kWsHeaderBytes + (size_t)items * d.n_kv_heads * s * (d.head_dim + 2) * kItemRows * sizeof(float);
}

cudaError_t launch_multi_attn(const tb_dims &d, const uint16_t *Q, const uint16_t *K, const uint16_t *V,
                              const int32_t *q_begin, int32_t n_tokens, int32_t max_new, const int32_t *ctx_len,
                              const uint32_t *mask, float scale, uint16_t *out, void *ws, cudaStream_t st) {
    Params p{};
    p.q_begin = q_begin;
    p.ctx_len = ctx_len;
    p.mask = mask;
    p.out = out;
    p.flags = static_cast<uint32_t *>(ws);
    p.batch = d.batch;
    p.Hq = d.n_q_heads;
    p.Hkv = d.n_kv_heads;
    p.cap = d.ctx_cap;
    p.n_tokens = n_tokens;
    p.max_new = max_new;
    p.mask_words = (max_new + 31) / 32;
    p.g_shift = log2_int(d.n_q_heads / d.n_kv_heads);
    p.item_bound = (int)item_bound(d, n_tokens, max_new);
    p.splits = pick_splits(d, p.item_bound);
    p.part = p.splits > 1 ? reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + kWsHeaderBytes) : nullptr;
    p.c = scale * 1.4426950408889634f;
    return d.head_dim == 128 ? launch_d<128>(d, Q, K, V, p, st) : launch_d<64>(d, Q, K, V, p, st);
}

}  // namespace tb
