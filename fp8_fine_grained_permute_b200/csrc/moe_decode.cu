// moe_decode.cu -- the whole expert layer for a few tokens in one kernel.
//
// The layer as the chain of routing, permute + 1x128 quantize, gated
// up-projection + 1x128 quantize, down-projection and combine computes it
// (DeepSeek-V3 summary sec. 2.1, 2.2), for T <= 64 tokens:
//     ids, a = top-k of sigmoid(logits) + bias;  w = a / sum a
//     [G; U](p) = Wup[e] xq(t),  h(p) = quant(silu(G) U),  out(t) = sum_j w_j Wdn[e_j] h(t, j)
// A few tokens read every weight of the experts they meet once and do next to no
// arithmetic on it, so the time is that of 3 I C bytes an expert met over the HBM
// rate, and what a kernel can lose is latency: launches, half-empty waves of tiles,
// and pauses of the weight stream.  Hence
//   * one cooperative launch, one CTA an SM.  The work of each of the two
//     projections is a sequence of equal steps of 32 KB of weights, and every CTA
//     takes an equal contiguous share of it, wherever that begins or ends
//     (stream-K), so all SMs stream to the end for any number of experts.
//   * weights are operand A of the tensor core (128 weight rows = M), tokens are
//     operand B (N = 16 or 32 columns), so a token costs 128 bytes a step next to
//     the weights' 32 KB instead of padding to a 128-row tile.  TMA brings the
//     weights as they lie (E4M3, 128-byte swizzle) and the MMA reads them in
//     shared memory: no thread touches a weight.
//   * the weight producer runs ahead over the border between the projections: the
//     ring is full of down-projection weights while the CTAs meet at the barrier.
//
// Step of the up-projection: one K block of a gate block and the matching up block
// (2 x 128 x 128 bytes) for one group of at most N tokens of one expert.  Step of
// the down-projection: two K blocks of 128 output columns.  A unit is what ends in
// one result: (group, 128 columns of h), then 128 columns of out over all experts.
// A unit cut between CTAs is joined from fp32 partials in the caller's workspace,
// always in CTA order, so results do not vary between runs.  A unit of h is joined
// by its first CTA: the others meet it at the beginning of their shares, so their
// parts are there long before the first one's, the end of its share.  For out,
// whose partials hold all T tokens, every CTA that has a part joins its share of
// the T x 128 sums.
//
// x is quantized once, a tile a half-warp over all CTAs (the bits of
// fg8_quantize_act), while the routing is worked out; the meeting that this takes
// hides behind the first weights' way.
//
// Warps: 0 TMA producer, 1 MMA issuer, 4..7 promotion (thread = one weight row:
// acc[token] += partial * (activation scale * block scale), fp32), 8..11 fill
// operand B (codes of x or h) and the scale products.
//
// On a B200 (and the share of the measured copy rate that the weights alone make):
//   256 experts x 7168 x 2048, top 8: 1 token 69 us (0.79), 8 tokens 367 us (0.9 and
//   more, by the experts met), 64 tokens 1136 us (0.98); 64 experts x 2048 x 768, top
//   6: 1 token 17.3 us (0.25), 37 tokens 73 us (0.64).  The stream runs at HBM speed (a
//   step's 32 KB an SM take 0.68 us, its MMAs 0.6).  What is around it, of 17.3 us at 64
//   experts and 1 token: 2.5 until the lists stand (7 for 37 tokens), 3 more to the first
//   product (x's codes from all CTAs, the first weights), 2 for the joins of h, 1.5 for
//   the meeting, 1.5 to the first product after it, 1.5 for the joins of out, 1.8 for
//   the launch and the end; the two streams take 1.75 each.  Measured on the way there: x
//   quantized by every CTA for itself, flags and fences in the joins, unrolled code
//   (39 us for this case: instructions that run once are fetched cold).
// N = 16 for T <= 16: with N = 32 (a stage less, half of every product unused) the
// same cases take 19.8 us, 75.0 us (256 experts, 1 token) and 369 us (8 tokens)
// against 18.0, 68.2 and 359.  The router's registers an expert are cut to E: all
// 1024 slots in every call cost 74.7 against 68.2 us at 256 experts, 256 slots 18.5
// against 18.0 us at 64.
//
// Every wait is bounded (FG8_ERR_TIMEOUT in *status; the roles wind down and TMEM
// is released).  A meeting with more arrivals than CTAs is one with another call on
// the same workspace: the call ends there in the same way (FG8_ERR_WORKSPACE_SHARED).
#include <cuda.h>
#include <cuda_bf16.h>

#include <type_traits>

#include "fg8_columns.cuh"
#include "fg8_route.cuh"
#include "fg8_tcgen05.cuh"
#include "fg8_tma.cuh"

namespace {

using namespace fg8::tma;
using namespace fg8::tc;

constexpr int kThreads = 384;
constexpr int kMaxT = 64;
constexpr int kMaxE = 1024;
constexpr int kMaxCtas = 160;
constexpr unsigned kFull = 0xffffffffu;
constexpr uint32_t kABytes = 2 * 128 * 128;          // a step's weights
constexpr int kTmemBufs = 4;
constexpr int kFillWarps = 4;

// Contiguous shares of `total` equal steps: the first `rem` CTAs have q + 1, the
// others up to `ctas` q.  No more CTAs take part than there are steps, so that
// every CTA from a unit's first to its last has a part of it.
struct Share {
    int total, ctas, q, rem;
    FG8_DEV int begin(int c) const { return c >= ctas ? total : c * q + min(c, rem); }
    FG8_DEV int owner(int step) const {
        const int big = rem * (q + 1);
        return step < big ? step / (q + 1) : rem + (step - big) / q;
    }
};
FG8_DEV Share make_share(int total, int all) {
    Share s;
    s.total = total;
    s.ctas = min(total, all);
    s.q = total / max(1, s.ctas);
    s.rem = total - s.q * s.ctas;
    return s;
}

// Where a CTA's share of a projection begins and ends, and what steps are there:
// up-projection: unit a (group c, h block d), K block b; down-projection: output
// block a, inside it group c, pair of K blocks d.
struct Cursor {
    int step, a, b, c, d;
};
struct Plan {
    int G;
    Share up, dn;
    Cursor cur[4];   // up begin, up end, down begin, down end
};

// Variants: N tokens a group.  N = 16 when T <= 16 (an expert then rarely has
// more tokens and the ring is a stage deeper), else 32.
template <int N>
struct Cfg {
    static constexpr int kStages = N == 16 ? 5 : 4;
    static constexpr uint32_t kBBytes = 2 * N * 128;             // two K blocks of B (the first alone in the up-projection)
    static constexpr uint32_t kStage = kABytes + kBBytes;
    static constexpr int kTokens = N == 16 ? 16 : kMaxT;
    static constexpr int kPairs = kTokens * fg8::kRouteMaxK;
    static constexpr int kAccRows = kTokens > 2 * N ? kTokens : 2 * N;   // a group's gate and up, or the tokens' sums
    // factor slots: written for step n while steps up to n - kStages - kTmemBufs
    // have been promoted (their stage and partial buffer were free again)
    static constexpr int kSlots = kStages + kTmemBufs;
    static constexpr uint32_t kTmemCols = kTmemBufs * 2 * N;     // 128 or 256
    static constexpr uint32_t kOffAcc = kStages * kStage;        // float [kAccRows][128]
    static constexpr uint32_t kOffFactors = kOffAcc + kAccRows * 512;
    static constexpr uint32_t kOffRed = kOffFactors + kSlots * 2 * N * 4;   // float [2][4][N]
    static constexpr uint32_t kOffBars = kOffRed + 2 * 4 * N * 4;
    static constexpr int kNumBars = 2 * kStages + 2 * kTmemBufs + 4;    // full, empty, tfull, tempty, drain, group, x, h
    static constexpr uint32_t kOffMisc = kOffBars + 8 * kNumBars;           // tmem slot, abort, call number, -, filled[4]
    static constexpr uint32_t kOffPlan = kOffMisc + 32;
    static constexpr uint32_t kOffGroups = kOffPlan + 128;        // uint32 [kPairs]: n | first << 6 | expert << 16
    static constexpr uint32_t kOffList = kOffGroups + 4 * kPairs;   // uint32 [kPairs]: pair | token << 16, experts ascending
    static constexpr uint32_t kOffW = kOffList + 4 * kPairs;     // float [kPairs]: gate weight of a pair
    static constexpr uint32_t kOffAff = kOffW + 4 * kPairs;      // float [kPairs]
    static constexpr uint32_t kOffIds = kOffAff + 4 * kPairs;      // int32 [kPairs]
    static constexpr uint32_t kOffMet = kOffIds + 4 * kPairs;    // uint16 [kPairs]: experts met, by first pair
    static constexpr uint32_t kOffCnt = kOffMet + 2 * kPairs;    // int32 [kMaxE]: pairs, then first place in the list
    static constexpr uint32_t kSmem = kOffCnt + 4 * kMaxE + 1024;   // + alignment slack
    static_assert(kSmem <= 232448, "shared memory per CTA");
    static_assert(kStage % 1024 == 0, "swizzle atoms");
    static_assert(sizeof(Plan) <= 128, "plan");
    static_assert(kFillWarps == 4, "filled[4], step mod 4");
};

// workspace: a head of counters and the partials of cut units, both at fixed places
// and never used for anything else, then the codes and scales of x and h.  A word
// of a partial is {call tag, fp32 value} in 64 bits, so that a reader sees from the
// word itself that it is this call's: no flag, no fence and no second trip.  Tags
// come round every 2^30 calls; every kClearCalls calls a CTA clears its words, so
// that none is older than that.
constexpr uint32_t kClearCalls = 1u << 29;
constexpr size_t kHeadBytes = 4096;
struct Head {
    // arrivals are counted over all calls, so nothing is cleared between them
    uint32_t x_done, h_done;         // CTAs that have written their codes of x, of h
    uint32_t calls[kMaxCtas];        // calls that the CTA has finished
};
static_assert(sizeof(Head) <= kHeadBytes, "counter head");
constexpr int kPartWords = 128 * 64;   // a group's gate and up (2 x 32 x 128), or 64 tokens x 128 columns

struct Args {
    const uint16_t* x;
    const float* logits;
    const float* bias;
    int32_t* ids;
    float* affinity;
    const float* sw_up;      // [E][2 I / 128][C / 128]
    const float* sw_dn;      // [E][C / 128][I / 128]
    int T, k, E, C, I;
    uint32_t k_magic;        // ceil(2^32 / k), 0 for k = 1: pair / k by multiplication
    int normalize, out_f32;
    void* out;
    Head* head;
    uint8_t* xq;             // [T][C]
    float* sx;               // [T][C / 128]
    uint8_t* hq;             // [T k][I]
    float* sh;               // [T k][I / 128]
    uint64_t* part;          // [2 CTAs][kPartWords]
    int32_t* status;
};

FG8_DEV float silu_mul(float g, float u) { return __fdividef(g, 1.0f + __expf(-g)) * u; }

// 2 N consecutive TMEM columns of this thread's lane
FG8_DEV void tmem_ld(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,"
        "%28,%29,%30,%31}, [%32];\n"
        "tcgen05.wait::ld.sync.aligned;\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
          "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
          "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}

// mbar_wait with what follows a failed first try out of line: every wait of this
// kernel is code that some CTA meets cold
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag, int32_t* status) {
    return mbar_wait(bar, parity, abort_flag, status);
}
FG8_DEV bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag, int32_t* status) {
    return mbar_try_wait(bar, parity) || wait_slow(bar, parity, abort_flag, status);
}

__device__ __noinline__ void stop_call(int32_t code, volatile int* abort_flag, int32_t* status) {
    fg8::set_status(status, code);
    *abort_flag = 1;
}

// After an abort, with every role done: no copy may reach this CTA's shared memory
// once the CTA is gone.  The last `stages` issued steps lie each on its own stage,
// the phases before them are complete; where the fill warp of a step (step mod 4)
// gave up before it, its arrival is made up for, so that a stage's phase completes
// with the bytes.  Bounded, as everything.
__device__ __noinline__ void land_copies(uint32_t bar0, int stages, int issued, const int32_t* filled) {
#pragma unroll 1
    for (int m = max(0, issued - stages); m < issued; ++m) {
        const uint32_t bar = bar0 + 8u * (m % stages), parity = (uint32_t)(m / stages) & 1u;
        if (m >= filled[m & 3]) mbar_arrive(bar);
        const uint64_t t0 = fg8::globaltimer_ns();
        while (!mbar_try_wait(bar, parity) && fg8::globaltimer_ns() - t0 < 100000000ull) {
        }
    }
}

FG8_DEV void red_release_gpu(uint32_t* p, uint32_t v) {
    asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// partial words
FG8_DEV void put_word(uint64_t* p, uint32_t tag, float v) {
    asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p), "l"((uint64_t)tag << 32 | __float_as_uint(v)) : "memory");
}
FG8_DEV uint64_t get_word(const uint64_t* p) {
    uint64_t v;
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}
FG8_DEV void get_words2(const uint64_t* p, uint64_t& a, uint64_t& b) {   // each of the two as a whole
    asm volatile("ld.relaxed.gpu.global.v2.u64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "l"(p) : "memory");
}
// (0 and 3 in the low bits: no tag, so a cleared word is nobody's)
FG8_DEV uint32_t tag_of(uint32_t call, uint32_t down) { return 4u * call + 1u + down; }
__device__ __noinline__ void clear_words(uint64_t* p, int n) {   // by the promotion warps
#pragma unroll 1
    for (int i = threadIdx.x & 127; i < n; i += 128) p[i] = 0;
}
FG8_DEV bool tagged(uint64_t w, uint32_t tag) { return (uint32_t)(w >> 32) == tag; }
FG8_DEV float value_of(uint64_t w) { return __uint_as_float((uint32_t)w); }
// Between two tries at words that are not all there: false to give up (bounded:
// raises the abort flag and reports FG8_ERR_TIMEOUT).
__device__ __noinline__ bool try_again(uint64_t& t0, volatile int* abort_flag, int32_t* status) {
    const uint64_t now = fg8::globaltimer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > fg8::kWaitLimitNs) stop_call(FG8_ERR_TIMEOUT, abort_flag, status);
    return !*abort_flag;
}

// E4M3 codes of 8 bf16 values over their tile's scale: the quotient as product,
// residual and correction.  For every pair of a bf16 magnitude and a tile maximum
// it is the IEEE quotient, with reciprocals up to 2 units
// off (all of them in tests/test_corrected_quotient.py), and it takes a tenth of
// the division's instructions: code size is latency here.  Scales below kCorrectedMin
// take the division.  The order of the terms keeps the sign of a zero.
FG8_DEV uint2 quant8_corrected(const uint4& v, float s) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t c[4];
    if (s >= fg8::kCorrectedMin) {
        const float r = fg8::inv_scale(s);
        const float2 nr = make_float2(-r, -r), s2 = make_float2(s, s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 nx = make_float2(-fg8::bf16_lo(w[i]), -fg8::bf16_hi(w[i]));
            const float2 z0 = __fmul2_rn(nx, nr);
            const float2 z = __ffma2_rn(__ffma2_rn(z0, s2, nx), nr, z0);
            c[i] = fg8::cvt_e4m3x2(z.x, z.y);
        }
    } else {
#pragma unroll 1
        for (int i = 0; i < 4; ++i)
            c[i] = fg8::cvt_e4m3x2(__fdiv_rn(fg8::bf16_lo(w[i]), s), __fdiv_rn(fg8::bf16_hi(w[i]), s));
    }
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// One fp32 value over its tile's scale, likewise (to 2^-45 before the rounding).
FG8_DEV uint32_t code_of(float x, float s) {
    float z;
    if (s >= fg8::kCorrectedMin) {
        const float r = fg8::inv_scale(s);
        const float z0 = __fmul_rn(x, r);
        z = __fmaf_rn(__fmaf_rn(z0, s, -x), -r, z0);
    } else {
        z = __fdiv_rn(x, s);
    }
    return fg8::cvt_e4m3x2(z, 0.f) & 0xFFu;
}

// fg8::route_token's choice with warp reductions on keys that order like the
// scores (0: taken, or no expert); lane j < k ends with the j-th chosen expert
// and its affinity.
template <int PER_LANE>
FG8_DEV void route_token_keys(const float (&lu)[PER_LANE], const float (&lb)[PER_LANE], int E, int k, int lane,
                              int32_t& id, float& affinity) {
    uint32_t key[PER_LANE];
#pragma unroll
    for (int i = 0; i < PER_LANE; ++i) {
        const uint32_t b = __float_as_uint(__fadd_rn(fg8::route_sigmoid(lu[i]), lb[i]));
        key[i] = lane + 32 * i < E ? (b & 0x80000000u ? ~b : b | 0x80000000u) : 0u;
    }
    id = 0;
#pragma unroll 1
    for (int j = 0; j < k; ++j) {
        uint32_t best = key[0];
#pragma unroll
        for (int i = 1; i < PER_LANE; ++i) best = max(best, key[i]);
        const uint32_t top = __reduce_max_sync(kFull, best);
        int e = INT_MAX;   // lowest expert with it
#pragma unroll
        for (int i = PER_LANE - 1; i >= 0; --i)
            if (key[i] == top) e = lane + 32 * i;
        e = __reduce_min_sync(kFull, e);
#pragma unroll
        for (int i = 0; i < PER_LANE; ++i)
            if (lane + 32 * i == e) key[i] = 0u;
        if (lane == j) id = e;
    }
    float u = 0.f;
#pragma unroll
    for (int i = 0; i < PER_LANE; ++i) {
        const float v = __shfl_sync(kFull, lu[i], id & 31);
        if (id >> 5 == i) u = v;
    }
    affinity = fg8::route_sigmoid(u);
}

// The tokens t = warp, warp + kThreads / 32, ... of a CTA, a warp each, the next
// token's logits ahead.
template <int PER_LANE>
FG8_DEV void route_tokens(const Args& a, int warp, int lane, int32_t* s_ids, float* s_aff, bool write) {
    float lu[PER_LANE], lb[PER_LANE], nu[PER_LANE];
    auto load = [&](int t) {
#pragma unroll
        for (int i = 0; i < PER_LANE; ++i)
            nu[i] = t < a.T && lane + 32 * i < a.E ? __ldg(a.logits + (int64_t)t * a.E + lane + 32 * i) : 0.f;
    };
    load(warp);
#pragma unroll
    for (int i = 0; i < PER_LANE; ++i) lb[i] = lane + 32 * i < a.E ? __ldg(a.bias + lane + 32 * i) : 0.f;
#pragma unroll 1
    for (int t = warp; t < a.T; t += kThreads / 32) {
#pragma unroll
        for (int i = 0; i < PER_LANE; ++i) lu[i] = nu[i];
        load(t + kThreads / 32);
        int32_t id;
        float s;
        route_token_keys<PER_LANE>(lu, lb, a.E, a.k, lane, id, s);
        if (lane < a.k) {
            s_ids[t * a.k + lane] = id;
            s_aff[t * a.k + lane] = s;
            if (write) {
                a.ids[t * a.k + lane] = id;
                a.affinity[t * a.k + lane] = s;
            }
        }
    }
}

template <int N>
__global__ void __launch_bounds__(kThreads, 1)
moe_decode(const __grid_constant__ CUtensorMap tm_up, const __grid_constant__ CUtensorMap tm_dn, const Args a) {
    using K = Cfg<N>;
    constexpr int S = K::kStages;
    extern __shared__ uint8_t smem_raw[];
    // (an offset keeps the pointer a shared-memory one for the compiler)
    uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar0 = sbase + K::kOffBars;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (S + s); };
    auto tfull_bar = [&](int b) { return bar0 + 8u * (2 * S + b); };
    auto tempty_bar = [&](int b) { return bar0 + 8u * (2 * S + kTmemBufs + b); };
    const uint32_t drain_bar = bar0 + 8u * (2 * S + 2 * kTmemBufs);
    const uint32_t group_bar = drain_bar + 8u, x_bar = drain_bar + 16u, h_bar = drain_bar + 24u;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + K::kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + K::kOffMisc + 4);
    volatile uint32_t* s_call = reinterpret_cast<volatile uint32_t*>(smem + K::kOffMisc + 8);
    int32_t* s_filled = reinterpret_cast<int32_t*>(smem + K::kOffMisc + 16);   // a fill warp's first step not filled
    uint32_t* s_groups = reinterpret_cast<uint32_t*>(smem + K::kOffGroups);
    uint32_t* s_list = reinterpret_cast<uint32_t*>(smem + K::kOffList);
    float* s_w = reinterpret_cast<float*>(smem + K::kOffW);
    float* s_aff = reinterpret_cast<float*>(smem + K::kOffAff);
    int32_t* s_ids = reinterpret_cast<int32_t*>(smem + K::kOffIds);
    int32_t* s_cnt = reinterpret_cast<int32_t*>(smem + K::kOffCnt);
    uint16_t* s_met = reinterpret_cast<uint16_t*>(smem + K::kOffMet);
    Plan& plan = *reinterpret_cast<Plan*>(smem + K::kOffPlan);
    float* s_factors = reinterpret_cast<float*>(smem + K::kOffFactors);
    float* s_acc = reinterpret_cast<float*>(smem + K::kOffAcc);
    float* s_red = reinterpret_cast<float*>(smem + K::kOffRed);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = blockIdx.x, ctas = gridDim.x;
    const int CB = a.C / 128, IB = a.I / 128, IB2 = (IB + 1) / 2;
    const int R = a.T * a.k;

    // ------------------------------------------------------------ set-up and routing
    // every CTA routes every token: cheaper than a second grid barrier
    if (tid == 64) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), 2);      // weight producer (with the bytes), fill warp
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < kTmemBufs; ++b) {
            mbar_init(tfull_bar(b), 1);
            mbar_init(tempty_bar(b), 4);
        }
        mbar_init(drain_bar, 1);
        mbar_init(group_bar, 4);
        mbar_init(x_bar, 1);
        mbar_init(h_bar, 1);
        *abort_flag = 0;
        *s_call = a.head->calls[cta] + 1u;
        fence_barrier_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(K::kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 96) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_up)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_dn)) : "memory");
    }
    if (warp >= 4) {
        // tile i of x goes to CTA i mod ctas, half a warp a tile
        const int hl = lane & 15;
#pragma unroll 1
        for (int i = cta + ctas * (2 * (warp - 4) + (lane >> 4)), n = a.T * CB; i - ctas * (lane >> 4) < n; i += 16 * ctas) {
            // (uniform over the warp: the second half may be past the end)
            const bool in = i < n;
            const int64_t at = (int64_t)i * 128 + 8 * hl;   // tile i = token i / CB, block i % CB: contiguous in x
            const uint4 v = in ? __ldg(reinterpret_cast<const uint4*>(a.x + at)) : make_uint4(0u, 0u, 0u, 0u);
            float m = fg8::amax8(v);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
            const float sc = fg8::tile_scale_fast(m);
            const uint2 q = quant8_corrected(v, sc);
            if (in) {
                *reinterpret_cast<uint2*>(a.xq + at) = q;
                if (hl == 0) a.sx[i] = sc;
            }
        }
    }
    if (a.logits) {
        // warp 0 has no other set-up: with one token it starts on it at once
        if (a.E <= 64) route_tokens<2>(a, warp, lane, s_ids, s_aff, cta == 0);
        else if (a.E <= 256) route_tokens<8>(a, warp, lane, s_ids, s_aff, cta == 0);
        else route_tokens<32>(a, warp, lane, s_ids, s_aff, cta == 0);
    } else {
        for (int p = tid; p < R; p += kThreads) {
            int32_t id = a.ids[p];
            if (id < 0 || id >= a.E) {
                fg8::set_status(a.status, FG8_ERR_BAD_EXPERT_ID);
                id = -1;
            }
            s_ids[p] = id;
            s_aff[p] = a.affinity[p];
        }
    }
    for (int e = tid; e < a.E; e += kThreads) s_cnt[e] = 0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    if (tid == kThreads - 1) red_release_gpu(&a.head->x_done, 1u);
    auto token_of = [&](int p) { return a.k_magic ? (int)__umulhi((uint32_t)p, a.k_magic) : p; };
    // Lists of pairs by expert, experts in the order of their first pairs.  Every
    // CTA has to get the same lists (they index the partials that CTAs join), so
    // one warp makes them; the code is kept short, as what runs once costs its
    // instruction fetches.
    if (warp == 0) {
        int met = 0;
#pragma unroll 1
        for (int p0 = 0; p0 < R; p0 += 32) {
            const int p = p0 + lane, id = p < R ? s_ids[p] : -1;
            const unsigned same = __match_any_sync(kFull, id), below = (1u << lane) - 1u;
            const int before = id >= 0 ? s_cnt[id] : 0, rank = __popc(same & below);
            const bool lead = id >= 0 && rank == 0;
            const unsigned fresh = __ballot_sync(kFull, lead && before == 0);
            if (id >= 0) s_ids[p] = id | ((before + rank) << 10);
            if (lead) s_cnt[id] = before + __popc(same);
            if (lead && before == 0) s_met[met + __popc(fresh & below)] = (uint16_t)id;
            met += __popc(fresh);
            __syncwarp();
        }
        int base = 0;   // pairs (low half) and groups (high half) so far
#pragma unroll 1
        for (int x0 = 0; x0 < met; x0 += 32) {
            const int id = x0 + lane < met ? s_met[x0 + lane] : -1;
            const int c = id >= 0 ? s_cnt[id] : 0, mine = c | ((c + N - 1) / N << 16);
            int incl = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(kFull, incl, o);
                if (lane >= o) incl += y;
            }
            const int at = base + incl - mine;
            if (id >= 0) {
                const int first = at & 0xFFFF;
                s_cnt[id] = first;
#pragma unroll 1
                for (int i = 0; i < c; i += N)
                    s_groups[(at >> 16) + i / N] =
                        (uint32_t)min(N, c - i) | ((uint32_t)(first + i) << 6) | ((uint32_t)id << 16);
            }
            base += __shfl_sync(kFull, incl, 31);
        }
        // the CTA's shares: lane l < 4 works out plan.cur[l]
        const int G = base >> 16;
        const bool down = lane & 2;
        const Share sh = make_share(down ? CB * G * IB2 : G * IB * CB, ctas);
        const int unit = down ? G * IB2 : CB, inner = down ? IB2 : IB;
        Cursor c;
        c.step = sh.begin(cta + (lane & 1));
        c.a = c.step / max(1, unit);
        c.b = c.step - c.a * unit;
        const int x = down ? c.b : c.a;
        c.c = x / inner;
        c.d = x - c.c * inner;
        if (lane < 4) plan.cur[lane] = c;
        if (lane == 0) {
            plan.G = G;
            plan.up = sh;
        }
        if (lane == 2) plan.dn = sh;
        __syncwarp();
        asm volatile("bar.arrive 2, %0;" ::"n"(kThreads) : "memory");   // the producer needs no more than that
    } else {
        asm volatile("bar.sync 2, %0;" ::"n"(kThreads) : "memory");
        // a pair's place in the list, and its gate weight as fg8_unpermute_combine
#pragma unroll 1
        for (int p = tid - 32; p < R; p += kThreads - 32) {
            const int v = s_ids[p], t = token_of(p);
            if (v < 0) continue;
            s_list[s_cnt[v & 1023] + (v >> 10)] = (uint32_t)p | ((uint32_t)t << 16);
            float w = s_aff[p];
            if (a.normalize) {
                float sum = 0.f;
#pragma unroll 1
                for (int j = t * a.k; j < (t + 1) * a.k; ++j)
                    if (s_ids[j] >= 0) sum = __fadd_rn(sum, s_aff[j]);
                w = sum != 0.f ? __fdiv_rn(w, sum) : 0.f;
            }
            s_w[p] = w;
        }
        asm volatile("bar.sync 3, %0;" ::"n"(kThreads - 32) : "memory");
    }

    const int G = plan.G;
    const Cursor cu = plan.cur[0], cd = plan.cur[2];
    const int u0 = cu.step, u1 = plan.cur[1].step;
    const int d0 = cd.step, d1 = plan.cur[3].step;
    const int unit_dn = G * IB2;    // steps of an output block
    const int n_up = u1 - u0, n_all = n_up + (d1 - d0);
    auto group_n = [&](uint32_t g) { return (int)(g & 63u); };
    auto group_first = [&](uint32_t g) { return (int)((g >> 6) & 1023u); };
    auto group_e = [&](uint32_t g) { return (int)(g >> 16); };

    bool ok = true;
    int issued = 0;   // steps whose copies the producer has started
    if (warp == 0) {
        if (lane == 0) {
            // -------------------------------------------- weight producer
            uint32_t stage = 0, phase = 0;
            auto take = [&]() { return wait_bar(empty_bar(stage), phase ^ 1u, abort_flag, a.status); };
            auto next = [&]() {
                ++issued;
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
            };
            if (u0 < u1) {
                int cb = cu.b, g = cu.c, ib = cu.d;
#pragma unroll 1
                for (int s = u0; s < u1; ++s) {
                    if (!(ok = take())) break;
                    const uint32_t dst = sbase + stage * K::kStage;
                    const int row = group_e(s_groups[g]) * 2 * a.I + 128 * ib;
                    mbar_arrive_expect_tx(full_bar(stage), kABytes);
                    tma_load_2d(&tm_up, dst, full_bar(stage), 128 * cb, row);
                    tma_load_2d(&tm_up, dst + kABytes / 2, full_bar(stage), 128 * cb, row + a.I);
                    next();
                    if (++cb == CB) {
                        cb = 0;
                        if (++ib == IB) ib = 0, ++g;
                    }
                }
            }
            if (ok && d0 < d1) {
                int cb = cd.a, g = cd.c, k2 = cd.d;
#pragma unroll 1
                for (int s = d0; s < d1; ++s) {
                    if (!(ok = take())) break;
                    const uint32_t dst = sbase + stage * K::kStage;
                    const int row = group_e(s_groups[g]) * a.C + 128 * cb;
                    const bool two = 2 * k2 + 1 < IB;
                    mbar_arrive_expect_tx(full_bar(stage), two ? kABytes : kABytes / 2);
                    tma_load_2d(&tm_dn, dst, full_bar(stage), 256 * k2, row);
                    if (two) tma_load_2d(&tm_dn, dst + kABytes / 2, full_bar(stage), 256 * k2 + 128, row);
                    next();
                    if (++k2 == IB2) {
                        k2 = 0;
                        if (++g == G) g = 0, ++cb;
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // -------------------------------------------- MMA issuer
            constexpr uint32_t kIdesc = idesc_e4m3(128, N);
            uint32_t stage = 0, phase = 0, buf = 0, bphase = 0;
            int k2 = cd.d;
#pragma unroll 1
            for (int n = 0; n < n_all; ++n) {
                if (!wait_bar(tempty_bar(buf), bphase ^ 1u, abort_flag, a.status) ||
                    !wait_bar(full_bar(stage), phase, abort_flag, a.status))
                    break;
                tc_fence_after();
                const uint32_t sA = sbase + stage * K::kStage, sB = sA + kABytes;
                const uint32_t d = tmem_base + buf * 2 * N;
                const bool is_up = n < n_up;
                const bool two = is_up || 2 * k2 + 1 < IB;
                const uint32_t sB2 = is_up ? sB : sB + N * 128;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_e4m3(d, smem_desc(sA + 32 * kk), smem_desc(sB + 32 * kk), kIdesc, kk > 0 ? 1u : 0u);
                if (two) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_e4m3(d + N, smem_desc(sA + kABytes / 2 + 32 * kk), smem_desc(sB2 + 32 * kk), kIdesc,
                                 kk > 0 ? 1u : 0u);
                }
                mma_commit(empty_bar(stage));
                mma_commit(tfull_bar(buf));
                if (!is_up && ++k2 == IB2) k2 = 0;
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
                if (++buf == kTmemBufs) {
                    buf = 0;
                    bphase ^= 1u;
                }
            }
            // all MMAs issued by this thread are complete once drain_bar flips
            mma_commit(drain_bar);
            const uint64_t t0 = fg8::globaltimer_ns();
            while (!mbar_try_wait(drain_bar, 0) && fg8::globaltimer_ns() - t0 < 100000000ull) {
            }
        }
    } else if (warp >= 8) {
        // ------------------------------------------------ operand B
        // fill warp w takes the steps n = w, w + 4, ...: the first use of a stage
        // that is not yet free is at most one phase ahead (4 <= stages).  That is all
        // a wait by parity can tell apart, and it holds because one thread issues all
        // MMAs: stages are released in the order of the steps, so the release of n - 4's
        // stage, which this warp has waited for, comes after that of every stage before
        // (tests/test_moe_decode_ring.py)
        const int fw = warp - 8;
        const int sub = lane >> 3, ch = lane & 7;   // a row's 128 codes: 8 lanes
        uint32_t stage = fw, phase = 0;
        int slot = fw, n = fw;
        auto next = [&]() {
            n += kFillWarps;
            if ((stage += kFillWarps) >= S) {
                stage -= S;
                phase ^= 1u;
            }
            if ((slot += kFillWarps) >= K::kSlots) slot -= K::kSlots;
        };
        // all CTAs have written what this one reads next: the fill warp that comes
        // first watches, the others wait for it here
        auto wait_all = [&](const uint32_t* arrivals, uint32_t bar, int watch) {
            if (fw == watch && lane == 0) {
                const uint32_t all = *s_call * (uint32_t)ctas;
                const uint64_t t0 = fg8::globaltimer_ns();
                int32_t over;
                while ((over = (int32_t)(fg8::ld_acquire_gpu(arrivals) - all)) < 0 && !*abort_flag) {
                    if (fg8::globaltimer_ns() - t0 > fg8::kWaitLimitNs) stop_call(FG8_ERR_TIMEOUT, abort_flag, a.status);
                }
                // another call arrives here too: what was waited for may not be there
                if (over > 0) stop_call(FG8_ERR_WORKSPACE_SHARED, abort_flag, a.status);
                mbar_arrive(bar);
            }
            __syncwarp();
            return wait_bar(bar, 0, abort_flag, a.status) && !*abort_flag;
        };
        // rows of 128 codes, row j at base + stride * index(j): all loads, then,
        // once the stage is free, all stores
        auto load_rows = [&](uint4 (&v)[N / 4], const uint8_t* base, int stride, const uint32_t* list, int shift, int cnt) {
#pragma unroll
            for (int i = 0; i < N / 4; ++i)
                if (4 * i < cnt) {   // warp-uniform
                    const int j = min(4 * i + sub, cnt - 1);
                    v[i] = __ldcg(reinterpret_cast<const uint4*>(base + (int64_t)((list[j] >> shift) & 0xFFFFu) * stride + 16 * ch));
                }
        };
        auto store_rows = [&](const uint4 (&v)[N / 4], uint8_t* B, int cnt) {
#pragma unroll
            for (int i = 0; i < N / 4; ++i)
                if (4 * i < cnt) {
                    const int j = 4 * i + sub;   // rows past cnt, < N, repeat the last: their columns are not used
                    *reinterpret_cast<uint4*>(B + j * 128 + ((ch ^ (j & 7)) << 4)) = v[i];
                }
        };
        // this lane's factors: index 32 i + lane is token index % N of the first
        // (gate / first block) or second (up / second block) product
        constexpr int F = 2 * N / 32;
        auto publish = [&](const float (&fac)[F]) {
            float* f = s_factors + slot * 2 * N;
#pragma unroll
            for (int i = 0; i < F; ++i) f[32 * i + lane] = fac[i];
            fence_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(full_bar(stage));
        };
        if (n < n_up) {
            int cb = cu.b + n, g = cu.c, ib = cu.d;
            // block scales of a step, loaded a step ahead (they come from HBM)
            float sw[F];
            auto advance = [&]() {
#pragma unroll 1
                for (; cb >= CB; cb -= CB)
                    if (++ib == IB) ib = 0, ++g;
#pragma unroll
                for (int i = 0; i < F; ++i)
                    sw[i] = __ldg(a.sw_up + ((int64_t)group_e(s_groups[g]) * 2 * IB + ib + (32 * i + lane) / N * IB) * CB + cb);
            };
            advance();
            ok = wait_all(&a.head->x_done, x_bar, 0);
#pragma unroll 1
            while (ok && n < n_up) {
                const uint32_t gr = s_groups[g];
                const int cnt = group_n(gr);
                const uint32_t* list = s_list + group_first(gr);
                uint4 v[N / 4];
                load_rows(v, a.xq + 128 * cb, a.C, list, 16, cnt);
                float fac[F];
#pragma unroll
                for (int i = 0; i < F; ++i)
                    fac[i] = __ldcg(a.sx + (int64_t)(list[min((32 * i + lane) % N, cnt - 1)] >> 16) * CB + cb) * sw[i];
                if (n + kFillWarps < n_up) {
                    cb += kFillWarps;
                    advance();
                }
                if (!(ok = wait_bar(empty_bar(stage), phase ^ 1u, abort_flag, a.status))) break;
                store_rows(v, smem + stage * K::kStage + kABytes, cnt);
                publish(fac);
                next();
            }
        }
        if (ok && n < n_all) {
            int cb = cd.a, g = cd.c, k2 = cd.d + n - n_up;
            float sw[F];
            auto advance = [&]() {
#pragma unroll 1
                for (; k2 >= IB2; k2 -= IB2)
                    if (++g == G) g = 0, ++cb;
#pragma unroll
                for (int i = 0; i < F; ++i)
                    sw[i] = __ldg(a.sw_dn + ((int64_t)group_e(s_groups[g]) * CB + cb) * IB +
                                  min(2 * k2 + (32 * i + lane) / N, IB - 1));
            };
            advance();
            ok = wait_all(&a.head->h_done, h_bar, n_up % kFillWarps);
#pragma unroll 1
            while (ok && n < n_all) {
                const uint32_t gr = s_groups[g];
                const int cnt = group_n(gr);
                const uint32_t* list = s_list + group_first(gr);
                const bool two = 2 * k2 + 1 < IB;
                uint4 v[N / 4], w[N / 4];
                load_rows(v, a.hq + 256 * k2, a.I, list, 0, cnt);
                if (two) load_rows(w, a.hq + 256 * k2 + 128, a.I, list, 0, cnt);
                float fac[F];
#pragma unroll
                for (int i = 0; i < F; ++i) {
                    const int idx = 32 * i + lane, p = list[min(idx % N, cnt - 1)] & 0xFFFFu;
                    fac[i] = __ldcg(a.sh + (int64_t)p * IB + min(2 * k2 + idx / N, IB - 1)) * sw[i] * s_w[p];
                }
                if (n + kFillWarps < n_all) {
                    k2 += kFillWarps;
                    advance();
                }
                if (!(ok = wait_bar(empty_bar(stage), phase ^ 1u, abort_flag, a.status))) break;
                uint8_t* B = smem + stage * K::kStage + kABytes;
                store_rows(v, B, cnt);
                if (two) store_rows(w, B + N * 128, cnt);
                publish(fac);
                next();
            }
        }
        if (lane == 0) s_filled[fw] = n;
    } else if (warp >= 4) {
        // ------------------------------------------------ promotion
        const int quarter = warp & 3;
        const int row = 32 * quarter + lane;     // weight row of the tile
        const uint32_t lane_base = tmem_base + ((uint32_t)(32 * quarter) << 16);
        uint32_t buf = 0, bphase = 0, gphase = 0, joint = 0;
        int slot = 0;
        // barrier of the four promotion warps (bounded: false after an abort)
        auto meet = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(group_bar);
            const bool r = wait_bar(group_bar, gphase, abort_flag, a.status);
            gphase ^= 1u;
            return __all_sync(kFull, r) != 0;
        };
        float acc[2 * N];
        // acc[i] += partial[i] * factor[i] for one step's 2 N columns (the first
        // half only where the step has one K block)
        auto promote = [&](bool two) {
            if (!__all_sync(kFull, wait_bar(tfull_bar(buf), bphase, abort_flag, a.status))) return false;
            tc_fence_after();
            const float4* f4 = reinterpret_cast<const float4*>(s_factors + slot * 2 * N);
#pragma unroll
            for (int h = 0; h < 2 * N / 32; ++h) {
                uint32_t p[32];
                tmem_ld(lane_base + buf * 2 * N + 32 * h, p);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const int i = 32 * h + 4 * q;
                    if (i >= N && !two) continue;
                    const float4 f = f4[8 * h + q];
                    acc[i] = fmaf(__uint_as_float(p[4 * q]), f.x, acc[i]);
                    acc[i + 1] = fmaf(__uint_as_float(p[4 * q + 1]), f.y, acc[i + 1]);
                    acc[i + 2] = fmaf(__uint_as_float(p[4 * q + 2]), f.z, acc[i + 2]);
                    acc[i + 3] = fmaf(__uint_as_float(p[4 * q + 3]), f.w, acc[i + 3]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty_bar(buf));
            if (++buf == kTmemBufs) {
                buf = 0;
                bphase ^= 1u;
            }
            if (++slot == K::kSlots) slot = 0;
            return true;
        };
        // where CTA c keeps its partial of a unit that begins at step `begin`
        auto part_of = [&](int c, const Share& sh, int begin) {
            return a.part + (int64_t)(2 * c + (begin > sh.begin(c) ? 1 : 0)) * kPartWords;
        };

        const uint32_t tag_up = tag_of(*s_call, 0u), tag_dn = tag_of(*s_call, 1u);
        float* my_acc = s_acc + row;   // this thread's column, its alone
        auto clear = [&]() {
#pragma unroll
            for (int i = 0; i < 2 * N; ++i) acc[i] = 0.f;
        };
        if (*s_call % kClearCalls == 0) {
            clear_words(a.part + (int64_t)2 * cta * kPartWords, 2 * kPartWords);
            ok = meet();
        }
        // ---- up-projection
        if (ok && u0 < u1) {
            const Share up = plan.up;
            int u = cu.a, cb = cu.b;
            clear();
#pragma unroll 1
            for (int s = u0; s < u1; ++s) {
                if (!(ok = promote(true))) break;
                if (++cb < CB && s + 1 < u1) continue;
                // this CTA's part of unit u is done
                const int g = u / IB, ib = u - g * IB;
                const uint32_t gr = s_groups[g];
                const int cnt = group_n(gr);
                const uint32_t* list = s_list + group_first(gr);
                const int ub = u * CB, ue = ub + CB;
                if (ub < u0) {
                    // begun by an earlier CTA, which joins it
                    uint64_t* my = part_of(cta, up, ub) + row;
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        if (j < cnt) {
                            put_word(my + j * 128, tag_up, acc[j]);
                            put_word(my + (N + j) * 128, tag_up, acc[N + j]);
                        }
                } else {
#pragma unroll
                    for (int i = 0; i < 2 * N; ++i) my_acc[i * 128] = acc[i];
                    if (ue > u1) {   // the later CTAs' parts
                        const int c1 = up.owner(ue - 1);
#pragma unroll 1
                        for (int c = cta + 1; c <= c1; ++c) {
                            const uint64_t* pp = part_of(c, up, ub) + row;
#pragma unroll 1
                            for (int j0 = 0; j0 < cnt; j0 += 4) {
                                uint64_t w[8], t0 = 0;
                                bool all;
                                do {
                                    all = true;
#pragma unroll
                                    for (int i = 0; i < 8; ++i) {   // a token past the last: the last again
                                        w[i] = get_word(pp + ((i & 1) * N + min(j0 + i / 2, cnt - 1)) * 128);
                                        all &= tagged(w[i], tag_up);
                                    }
                                } while (!all && try_again(t0, abort_flag, a.status));
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    if (j0 + i / 2 < cnt) my_acc[((i & 1) * N + j0 + i / 2) * 128] += value_of(w[i]);
                            }
                        }
                    }
                    // h = silu(gate) up for this row's column of every token, one
                    // 1x128 tile a token over the 128 threads
                    float* red = s_red + (joint & 1u) * 4 * N;
#pragma unroll 2
                    for (int j = 0; j < cnt; ++j) {
                        const float h = silu_mul(my_acc[j * 128], my_acc[(N + j) * 128]);
                        my_acc[j * 128] = h;
                        const uint32_t m = __reduce_max_sync(kFull, __float_as_uint(fabsf(h)));
                        if (lane == 0) red[quarter * N + j] = __uint_as_float(m);
                    }
                    if (!(ok = meet())) break;
#pragma unroll 2
                    for (int j = 0; j < cnt; ++j) {
                        const float m = fmaxf(fmaxf(red[j], red[N + j]), fmaxf(red[2 * N + j], red[3 * N + j]));
                        const float sc = fg8::tile_scale_fast(m);
                        const int p = list[j] & 0xFFFFu;
                        a.hq[(int64_t)p * a.I + 128 * ib + row] = (uint8_t)code_of(my_acc[j * 128], sc);
                        if (row == 0) a.sh[(int64_t)p * IB + ib] = sc;
                    }
                }
                ++joint;
                cb = 0;
                ++u;
                clear();
            }
        }
        // ---- grid barrier: this CTA's h is written
        if (ok && (ok = meet()) && warp == 4 && lane == 0) {
            a.head->calls[cta] = *s_call;
            red_release_gpu(&a.head->h_done, 1u);
        }
        // ---- down-projection
        auto store_out = [&](int t, int c, float v) {
            if (a.out_f32) static_cast<float*>(a.out)[(int64_t)t * a.C + c] = v;
            else static_cast<uint16_t*>(a.out)[(int64_t)t * a.C + c] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
        };
        if (ok && d0 < d1) {
            const Share dn = plan.dn;
            int cb = cd.a, g = cd.c, k2 = cd.d;
#pragma unroll 1
            for (int t = 0; t < a.T; ++t) my_acc[t * 128] = 0.f;
            clear();
#pragma unroll 1
            for (int s = d0; s < d1; ++s) {
                if (!(ok = promote(2 * k2 + 1 < IB))) break;
                const bool cut = s + 1 == d1;
                if (++k2 < IB2 && !cut) continue;
                k2 = 0;
                // the group's (or this CTA's last) columns into their tokens' sums
                const uint32_t gr = s_groups[g];
                const int cnt = group_n(gr);
                const uint32_t* list = s_list + group_first(gr);
#pragma unroll
                for (int j = 0; j < N; ++j)
                    if (j < cnt) my_acc[(list[j] >> 16) * 128] += acc[j] + acc[N + j];
                clear();
                if (++g < G && !cut) continue;
                g = 0;
                // this CTA's part of output block cb is done
                const int ub = cb * unit_dn, ue = ub + unit_dn;
                if (ub >= d0 && ue <= d1) {
#pragma unroll 1
                    for (int t = 0; t < a.T; ++t) store_out(t, 128 * cb + row, my_acc[t * 128]);
                } else {
                    uint64_t* my = part_of(cta, dn, ub) + row;
#pragma unroll 4
                    for (int t = 0; t < a.T; ++t) put_word(my + t * 128, tag_dn, my_acc[t * 128]);
                }
#pragma unroll 1
                for (int t = 0; t < a.T; ++t) my_acc[t * 128] = 0.f;
                ++cb;
            }
            // cut blocks (at most the first and the last of this CTA's): each of their
            // CTAs joins its share of the T x 128 sums, four columns a thread
            const int cb0 = cd.a, cb1 = plan.cur[3].b ? plan.cur[3].a : plan.cur[3].a - 1;
#pragma unroll 1
            for (int c = cb0; ok && c <= cb1; c += max(1, cb1 - cb0)) {
                const int ub = c * unit_dn, ue = ub + unit_dn;
                if (ub >= d0 && ue <= d1) continue;
                const int c0 = dn.owner(ub), c1 = dn.owner(ue - 1), n = c1 - c0 + 1;
                const int quads = 32 * a.T, q1 = quads * (cta - c0 + 1) / n;
#pragma unroll 1
                for (int q = quads * (cta - c0) / n + row; q < q1; q += 128) {
                    float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
                    for (int w0 = c0; w0 <= c1; w0 += 6) {
                        uint64_t w[6][4], t0 = 0;
                        bool all;
                        do {
                            all = true;
#pragma unroll
                            for (int k = 0; k < 6; ++k) {   // a CTA past the last: the last again
                                const uint64_t* pp = part_of(min(w0 + k, c1), dn, ub) + 4 * q;
                                get_words2(pp, w[k][0], w[k][1]);
                                get_words2(pp + 2, w[k][2], w[k][3]);
                            }
#pragma unroll
                            for (int k = 0; k < 24; ++k) all &= tagged(w[k / 4][k & 3], tag_dn);
                        } while (!all && try_again(t0, abort_flag, a.status));
#pragma unroll
                        for (int k = 0; k < 6; ++k) {
                            if (w0 + k > c1) break;
#pragma unroll
                            for (int i = 0; i < 4; ++i) v[i] += value_of(w[k][i]);
                        }
                    }
                    const int t = q >> 5, col = 128 * c + 4 * (q & 31);
                    store_out(t, col, v[0]);
                    store_out(t, col + 1, v[1]);
                    store_out(t, col + 2, v[2]);
                    store_out(t, col + 3, v[3]);
                }
            }
        }
        // no pair has an expert: the output is zero
        if (G == 0)
            for (int c = cta; c < CB; c += ctas)
                for (int t = 0; t < a.T; ++t) store_out(t, 128 * c + row, 0.f);
    }

    tc_fence_before();
    __syncthreads();
    if (tid == 0 && *abort_flag) land_copies(bar0, S, issued, s_filled);
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(K::kTmemCols)
                     : "memory");
    }
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

struct Layout {
    size_t part, xq, sx, hq, sh, total;
};
Layout layout(int64_t T, int k, int64_t C, int64_t I) {
    Layout l;
    const int64_t R = T * k;
    l.part = kHeadBytes;
    l.xq = l.part + sizeof(uint64_t) * 2 * kMaxCtas * kPartWords;
    l.sx = l.xq + round256((size_t)(T * C));
    l.hq = l.sx + round256((size_t)(T * (C / 128) * 4));
    l.sh = l.hq + round256((size_t)(R * I));
    l.total = l.sh + round256((size_t)(R * (I / 128) * 4));
    return l;
}
static_assert(kPartWords >= 2 * 32 * 128 && kPartWords >= kMaxT * 128, "a part fits its slot");
static_assert(FG8_MOE_DECODE_HEAD == kHeadBytes + sizeof(uint64_t) * 2 * kMaxCtas * kPartWords, "what the caller zeroes");

template <int N>
fg8_status launch(const CUtensorMap& up, const CUtensorMap& dn, Args& a, cudaStream_t st) {
    auto kern = moe_decode<N>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<N>::kSmem) != cudaSuccess)
        return FG8_ERR_CUDA;
    int grid = fg8h::num_sms();
    if (grid > kMaxCtas) grid = kMaxCtas;
    void* args[] = {const_cast<CUtensorMap*>(&up), const_cast<CUtensorMap*>(&dn), &a};
    if (cudaLaunchCooperativeKernel((const void*)kern, dim3((unsigned)grid), dim3(kThreads), args, Cfg<N>::kSmem,
                                    st) != cudaSuccess) {
        cudaGetLastError();
        return FG8_ERR_CUDA;
    }
    return FG8_OK;
}

}  // namespace

extern "C" size_t fg8_moe_decode_workspace(int64_t T, int k, int64_t C, int64_t I) {
    if (T < 1 || T > kMaxT || k < 1 || k > fg8::kRouteMaxK || C < 128 || I < 128) return 0;
    return layout(T, k, C, I).total;
}

extern "C" fg8_status fg8_moe_decode(const uint16_t* x, int64_t T, int C, const float* logits, const float* bias,
                                     int32_t* topk_ids, float* affinity, int k, int E, const uint8_t* wq_up,
                                     const float* sw_up, int I, const uint8_t* wq_dn, const float* sw_dn,
                                     int normalize, int out_dtype, void* out, void* workspace, size_t ws_bytes,
                                     int32_t* dev_status, fg8_stream_t stream) {
    if (T < 0 || C < 128 || C % 128 || I < 128 || I % 128 || E < 1 || k < 1 || k > E ||
        (normalize != 0 && normalize != 1))
        return FG8_ERR_INVALID_ARG;
    if (out_dtype != FG8_OUT_BF16 && out_dtype != FG8_OUT_F32) return FG8_ERR_INVALID_ARG;
    if (T > kMaxT || k > fg8::kRouteMaxK || E > kMaxE) return FG8_ERR_UNSUPPORTED;
    if ((int64_t)E * 2 * I > INT32_MAX || (int64_t)E * C > INT32_MAX) return FG8_ERR_UNSUPPORTED;
    if ((T * k) * (int64_t)(I / 128) * (C / 128) > INT32_MAX) return FG8_ERR_UNSUPPORTED;   // steps
    if (T == 0) return FG8_OK;
    if (!x || !topk_ids || !affinity || !wq_up || !sw_up || !wq_dn || !sw_dn || !out || !workspace ||
        (logits && !bias))
        return FG8_ERR_INVALID_ARG;
    if (!fg8h::aligned16(x) || !fg8h::aligned16(wq_up) || !fg8h::aligned16(wq_dn) || !fg8h::aligned16(out) ||
        !fg8h::aligned16(workspace) ||
        ((reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(bias) |
          reinterpret_cast<uintptr_t>(topk_ids) | reinterpret_cast<uintptr_t>(affinity) |
          reinterpret_cast<uintptr_t>(sw_up) | reinterpret_cast<uintptr_t>(sw_dn)) & 3))
        return FG8_ERR_INVALID_ARG;
    const Layout l = layout(T, k, C, I);
    if (ws_bytes < l.total) return FG8_ERR_INVALID_ARG;
    CUtensorMap up, dn;
    if (!fg8h::make_tensor_map_2d(&up, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, wq_up, (uint64_t)E * 2 * I, (uint64_t)C, 128,
                                  128, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !fg8h::make_tensor_map_2d(&dn, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, wq_dn, (uint64_t)E * C, (uint64_t)I, 128,
                                  128, CU_TENSOR_MAP_SWIZZLE_128B))
        return FG8_ERR_CUDA;
    Args a;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.x = x; a.logits = logits; a.bias = bias; a.ids = topk_ids; a.affinity = affinity;
    a.sw_up = sw_up; a.sw_dn = sw_dn;
    a.T = (int)T; a.k = k; a.E = E; a.C = C; a.I = I;
    a.k_magic = k == 1 ? 0u : (uint32_t)(((1ull << 32) + k - 1) / k);
    a.normalize = normalize; a.out_f32 = out_dtype == FG8_OUT_F32; a.out = out;
    a.head = reinterpret_cast<Head*>(ws);
    a.xq = ws + l.xq;
    a.sx = reinterpret_cast<float*>(ws + l.sx);
    a.hq = ws + l.hq;
    a.sh = reinterpret_cast<float*>(ws + l.sh);
    a.part = reinterpret_cast<uint64_t*>(ws + l.part);
    a.status = dev_status;
    return T <= 16 ? launch<16>(up, dn, a, (cudaStream_t)stream) : launch<32>(up, dn, a, (cudaStream_t)stream);
}
