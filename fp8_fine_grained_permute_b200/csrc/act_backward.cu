// act_backward.cu -- the gated activation's backward from 8-bit checkpoints.
//
// The up-projection's forward saved gate and up as E4M3 codes in 1x128 tiles
// (fg8_grouped_gemm_swiglu_quant_save).  With g, u their values, dh the bf16
// gradient of the activation's output as the down-projection's dgrad of the
// unweighted output gradient gives it, and w the row's gate weight:
//     sig = 1 / (1 + exp(-g)),  h = g sig u,  d = w dh
//     dU = d g sig,   dG = d u sig (1 + g (1 - sig))
//     gate_dot[block][row] = sum over the 128-column block of dh h  (dL/dw in parts)
// and the three matrices that the GEMMs of the backward take leave in 8 bits:
// [dG dU] by rows (dgrad's A), [dG dU] down the token axis per expert (the up
// weight gradient's A) and w h down the token axis (the down weight gradient's).
//
// What it has to move is 2 + 2 bytes in and 2 + 2 + 1 bytes out an element, where
// the chain of separate passes (bf16 gradients and activations written, then read
// by each quantizer) moves 25.  Everything of a 128 x 128 block is formed once in
// registers and leaves twice:
//   * CTA = 512 threads, one persistent worker per SM; the (tile, column block)
//     items are cut into contiguous ranges, one a CTA.  TMA brings an item's
//     32 + 16 + 16 KB into one of two stages while the item before is worked on.
//   * thread = 4 columns x 8 rows (a warp reads whole 128-byte code rows); dG and
//     w silu(g) of these 32 elements stay in 64 registers between the pass that
//     finds the maxima and the one that forms the codes.
//   * a row's maximum is one warp reduction, and its codes are one 128-byte store
//     a warp; the column maxima of the 16 warps meet in shared memory.
//   * the column codes (8 tokens of a column a thread) are turned around through
//     shared memory, 8-byte pieces XOR-swizzled by column, and leave as 128-byte
//     lines of the token axis.
// On a B200: 430 us for 65536 rows x 2048 in 256 experts (1.24 GB: 2.9 TB/s, 45 %
// of the measured copy rate), 24 us for 1998 rows x 768 in 64.  The instructions
// bound it: when it took 426 us, 383 were left with every store taken out and 374
// with the special functions out as well; 55 instructions an element at 57 % of the
// issue slots, the conversion, maximum and byte-permute pipe busiest.  Measured and
// not kept (each against 426): two CTAs an SM, each with 64 of a tile's rows and the
// column maxima exchanged over a cluster pair (490 us); the row maxima, reciprocals
// and doubled factors through shared memory in place of shuffles and moves (fewer
// instructions, but 436 to 487 us); stores put off into the next item (slower); the
// last factor of dG as (1 + g) - g sig, which is 4 us faster and wrong from 2^24 on.
#include <type_traits>

#include "fg8_columns.cuh"
#include "fg8_tma.cuh"

namespace {

using namespace fg8::tma;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 128 / kWarps;          // rows of a thread: 8
constexpr unsigned kFull = 0xffffffffu;
static_assert(kRows == 8, "eight tokens make a thread's 8-byte column piece");

// shared memory map (from a 128-byte aligned base)
constexpr uint32_t kDhBytes = 128 * 256, kCodeBytes = 128 * 128;
constexpr uint32_t kStage = kDhBytes + 2 * kCodeBytes;             // 64 KB
constexpr uint32_t kOffTrans = 2 * kStage;                         // [3][128 columns][128 tokens]
constexpr uint32_t kOffColMax = kOffTrans + 3 * kCodeBytes;        // float [16][3][128]
constexpr uint32_t kOffColInv = kOffColMax + 4 * kWarps * 384;     // float [3][128]
constexpr uint32_t kOffScales = kOffColInv + 4 * 384;              // float4 [2][128]: gate scale, up scale, weight
constexpr uint32_t kOffBars = kOffScales + 2 * 16 * 128;            // 2 mbarriers, abort flag
constexpr uint32_t kOffPref = kOffBars + 32;                       // int32 [kColsMaxE + 1]
constexpr uint32_t kOffWarp = kOffPref + 4 * (fg8::kColsMaxE + 4); // int32 [36]
constexpr uint32_t kSmemBytes = kOffWarp + 4 * 36;
static_assert(kSmemBytes <= 232448, "shared memory per CTA");

struct Args {
    const float* sgu;         // [2 I / 128][R]
    const float* row_w;       // [R] or NULL
    const int32_t* offsets;
    int64_t R, P;
    int E, I;
    uint8_t* dq;              // [R][2 I]
    float* sd;                // [2 I / 128][R]
    uint8_t* dqT;             // [2 I][P]
    float* sdT;               // [P / 128][2 I]
    uint8_t* hqT;             // [I][P]
    float* shT;               // [P / 128][I]
    float* gate_dot;          // [I / 128][R] or NULL
    int32_t* offsets_out;
    int32_t* status;
};

FG8_DEV float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
FG8_DEV float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// max(|a|, |b|, |c|), one instruction on sm_100
FG8_DEV float max3_abs(float a, float b, float c) {
    float d;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// codes of v times r (or, exactly, v over the scale r: for subnormal scales),
// the first in bits 7..0
template <bool kExact>
FG8_DEV uint32_t code2(float2 v, float2 r) {
    const float2 z = kExact ? make_float2(__fdiv_rn(v.x, r.x), __fdiv_rn(v.y, r.y)) : __fmul2_rn(v, r);
    return fg8::cvt_e4m3x2(z.x, z.y);
}
// the same for two tokens of a column; `inv` is the reciprocal, or a subnormal
// scale negated
template <bool kExact>
FG8_DEV uint32_t code_pair(float x, float y, float inv) {
    if (kExact && inv < 0.f) return fg8::cvt_e4m3x2(__fdiv_rn(x, -inv), __fdiv_rn(y, -inv));
    return fg8::cvt_e4m3x2(x * inv, y * inv);
}
// Let copies already issued land before the CTA winds down: those of item n, whose
// wait ran out, and of the one after it, if the CTA has one (bounded).
__device__ __noinline__ void land_copies(uint32_t bars, int n, int items) {
    auto landed = [&](int m) { return m >= items || mbar_try_wait(bars + 8u * (m & 1), (m >> 1) & 1); };
    const uint64_t t0 = fg8::globaltimer_ns();
    while (!(landed(n) && landed(n + 1)) && fg8::globaltimer_ns() - t0 < 100000000ull) {
    }
}
FG8_DEV float2 splat(float x) { return make_float2(x, x); }

__global__ void __launch_bounds__(kThreads, 1)
act_backward(const __grid_constant__ CUtensorMap tm_dh, const __grid_constant__ CUtensorMap tm_gu,
             const Args a) {
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    float* s_colmax = reinterpret_cast<float*>(smem + kOffColMax);
    float* s_colinv = reinterpret_cast<float*>(smem + kOffColInv);
    float* s_scales = reinterpret_cast<float*>(smem + kOffScales);
    int32_t* s_pref = reinterpret_cast<int32_t*>(smem + kOffPref);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffBars + 16);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ncb = a.I / 128;
    auto full_bar = [&](int st) { return sbase + kOffBars + 8u * st; };

    if (tid == 0) {
        mbar_init(full_bar(0), 1);
        mbar_init(full_bar(1), 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    fg8::tile_prefix(a.offsets, a.E, s_pref, reinterpret_cast<int32_t*>(smem + kOffWarp));
    if (blockIdx.x == 0)
        for (int e = tid; e <= a.E; e += kThreads) a.offsets_out[e] = 128 * s_pref[e];

    const int tiles = (int)min((int64_t)s_pref[a.E], a.P / 128);
    const int64_t items = (int64_t)tiles * ncb;
    const int owned = min(a.offsets[a.E], (int)a.R);   // rows from here on belong to no expert
    const int i0 = (int)(items * blockIdx.x / gridDim.x), i1 = (int)(items * (blockIdx.x + 1) / gridDim.x);
    if (i0 >= i1) return;

    auto tile_of = [&](int tile) { return fg8::find_tile(tile, s_pref, a.offsets, a.E, (int)a.R); };
    auto issue = [&](int cb, int row0, int st) {   // one thread
        const uint32_t dst = sbase + st * kStage;
        mbar_arrive_expect_tx(full_bar(st), kStage);
        tma_load_2d(&tm_dh, dst, full_bar(st), 128 * cb, row0);
        tma_load_2d(&tm_gu, dst + kDhBytes, full_bar(st), 128 * cb, row0);
        tma_load_2d(&tm_gu, dst + kDhBytes + kCodeBytes, full_bar(st), a.I + 128 * cb, row0);
    };
    // one of an item's 3 x 128 row factors a thread, 0 for the rows of others;
    // asynchronous, so that nothing waits for it in the pass it is issued in
    auto load_factor = [&](int cb, const fg8::RowTile& t, int st) {
        const int which = tid >> 7, r = tid & 127;
        if (which > 2) return;
        float* dst = s_scales + 512 * st + 4 * r + which;
        if (which == 2 && a.row_w == nullptr) {
            *dst = r < t.n_in ? 1.0f : 0.f;
            return;
        }
        const float* src = which == 2 ? a.row_w : a.sgu + (int64_t)((which ? ncb : 0) + cb) * a.R;
        const uint32_t bytes = r < t.n_in ? 4u : 0u;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)),
                     "l"(src + (bytes ? t.row0 + r : 0)), "r"(bytes)
                     : "memory");
    };
    auto factors_landed = [] { asm volatile("cp.async.wait_all;" ::: "memory"); };

    fg8::RowTile cur = tile_of(i0 / ncb);
    int cb = i0 % ncb;
    if (tid == 0) {
        issue(cb, cur.row0, 0);
        if (i0 + 1 < i1) {
            if (cb + 1 < ncb) issue(cb + 1, cur.row0, 1);
            else issue(0, tile_of(cur.tile + 1).row0, 1);
        }
    }
    load_factor(cb, cur, 0);
    factors_landed();
    __syncthreads();

    for (int it = i0; it < i1; ++it) {
        const int n = it - i0, st = n & 1;
        if (it + 1 < i1) {
            if (cb + 1 < ncb) load_factor(cb + 1, cur, st ^ 1);
            else load_factor(0, tile_of(cur.tile + 1), st ^ 1);
        }
        const float4* fac = reinterpret_cast<const float4*>(s_scales + 512 * st);
        const uint8_t* sdh = smem + st * kStage + 8 * lane;
        const uint32_t a_g = sbase + st * kStage + kDhBytes + 4 * lane;   // gate codes; up codes kCodeBytes further on
        const int r0 = kRows * warp;
        const bool ok = mbar_wait(full_bar(st), (n >> 1) & 1, abort_flag, a.status);

        // rows that no expert owns may hold anything: zeros in their place.  (Rows of a
        // tile that belong to the next expert have factors of 0: what is finite there
        // is 0, the maxima drop the NaN that is left of the rest, its codes are masked.)
        if (cur.n_in < 128 && cur.row0 + 128 > owned) {
            const int first = max(cur.n_in, owned - cur.row0);
            uint8_t* stage = smem + st * kStage;
            for (int i = tid; i < (128 - first) * 32; i += kThreads) {
                const int r = first + (i >> 5), l = i & 31;
                *reinterpret_cast<uint2*>(stage + r * 256 + 8 * l) = make_uint2(0u, 0u);
                *reinterpret_cast<uint32_t*>(stage + kDhBytes + r * 128 + 4 * l) = 0u;
                *reinterpret_cast<uint32_t*>(stage + kDhBytes + kCodeBytes + r * 128 + 4 * l) = 0u;
            }
            fence_async_shared();   // before the stage's next TMA load
            __syncthreads();
        }

        // ---- first pass over 8 rows x 4 columns, column pairs in packed
        // arithmetic.  dG and S = w silu(g) stay in registers; dU = dh S and
        // w h = u S are formed again in the second pass from the staged inputs
        // (all three would not leave the compiler the registers it needs).
        float2 dG[kRows][2], S[kRows][2];
        float row_max = 0.f;   // lane i < 16: of row i & 7 of dG (i < 8) or dU
        {
            float dot[kRows];
            float4 mG = make_float4(0.f, 0.f, 0.f, 0.f), mU = mG, mH = mG;
            auto fold = [](float4& m, const float2 (&a)[2], const float2 (&b)[2]) {
                m.x = max3_abs(m.x, a[0].x, b[0].x);
                m.y = max3_abs(m.y, a[0].y, b[0].y);
                m.z = max3_abs(m.z, a[1].x, b[1].x);
                m.w = max3_abs(m.w, a[1].y, b[1].y);
            };
#pragma unroll
            for (int i = 0; i < kRows; i += 2) {
                float2 dU[2][2], H[2][2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = r0 + i + h;
                    const uint2 dw = *reinterpret_cast<const uint2*>(sdh + r * 256);
                    const float4 f4 = fac[r];
                    const float2 fg = splat(f4.x), fu = splat(f4.y), w = splat(f4.z);
                    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const float2 g = __fmul2_rn(fg8::e4m3x2_at(a_g + r * 128 + 2 * p), fg);
                        const float2 u = __fmul2_rn(fg8::e4m3x2_at(a_g + kCodeBytes + r * 128 + 2 * p), fu);
                        const uint32_t db = p ? dw.y : dw.x;
                        const float2 dh = make_float2(fg8::bf16_lo(db), fg8::bf16_hi(db));
                        // exp overflows to infinity for very negative gates: sig is 0 then
                        const float2 t = __fmul2_rn(g, splat(-1.4426950408889634f));
                        const float2 q = __fadd2_rn(make_float2(ex2(t.x), ex2(t.y)), splat(1.0f));
                        const float2 sig = make_float2(rcp(q.x), rcp(q.y));
                        const float2 silu = __fmul2_rn(g, sig);
                        sum = __ffma2_rn(dh, __fmul2_rn(silu, u), sum);
                        const float2 sw = __fmul2_rn(silu, w);
                        dU[h][p] = __fmul2_rn(dh, sw);
                        H[h][p] = __fmul2_rn(u, sw);
                        // 1 + g (1 - sig), in that order: g + 1 - g sig would lose the 1 for
                        // gates beyond 2^24, where sig is 1 and the difference g - g
                        const float2 f = __ffma2_rn(g, __ffma2_rn(sig, splat(-1.0f), splat(1.0f)), splat(1.0f));
                        dG[i + h][p] = __fmul2_rn(__fmul2_rn(__fmul2_rn(dh, w), __fmul2_rn(u, sig)), f);
                        S[i + h][p] = sw;
                    }
                    dot[i + h] = sum.x + sum.y;
                    const float2 (&vG)[2] = dG[i + h];
                    const float2 (&vU)[2] = dU[h];
                    const uint32_t xg = __reduce_max_sync(
                        kFull, __float_as_uint(max3_abs(max3_abs(vG[0].x, vG[0].y, vG[1].x), vG[1].y, 0.f)));
                    const uint32_t xu = __reduce_max_sync(
                        kFull, __float_as_uint(max3_abs(max3_abs(vU[0].x, vU[0].y, vU[1].x), vU[1].y, 0.f)));
                    if (lane == i + h) row_max = __uint_as_float(xg);
                    if (lane == kRows + i + h) row_max = __uint_as_float(xu);
                }
                fold(mG, dG[i], dG[i + 1]);
                fold(mU, dU[0], dU[1]);
                fold(mH, H[0], H[1]);
            }
            float4* cm = reinterpret_cast<float4*>(s_colmax + warp * 384) + lane;
            cm[0] = mG;
            cm[32] = mU;
            cm[64] = mH;
            // the rows' dots: 8 values over 32 lanes, halved at each exchange
            if (a.gate_dot) {
                float v4[4], v2[2], v1;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float keep = lane & 16 ? dot[4 + i] : dot[i], give = lane & 16 ? dot[i] : dot[4 + i];
                    v4[i] = keep + __shfl_xor_sync(kFull, give, 16);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float keep = lane & 8 ? v4[2 + i] : v4[i], give = lane & 8 ? v4[i] : v4[2 + i];
                    v2[i] = keep + __shfl_xor_sync(kFull, give, 8);
                }
                {
                    const float keep = lane & 4 ? v2[1] : v2[0], give = lane & 4 ? v2[0] : v2[1];
                    v1 = keep + __shfl_xor_sync(kFull, give, 4);
                }
                v1 += __shfl_xor_sync(kFull, v1, 2);
                v1 += __shfl_xor_sync(kFull, v1, 1);
                const int r = r0 + ((lane >> 4) & 1) * 4 + ((lane >> 3) & 1) * 2 + ((lane >> 2) & 1);
                if ((lane & 3) == 0 && r < cur.n_in) a.gate_dot[(int64_t)cb * a.R + cur.row0 + r] = v1;
            }
        }
        // row scales, a lane each
        const float row_s = fg8::tile_scale_fast(row_max), row_inv = fg8::inv_scale(row_s);
        {
            const int my_row = r0 + (lane & 7);
            if (lane < 16 && my_row < cur.n_in)
                a.sd[(int64_t)((lane >> 3) * ncb + cb) * a.R + cur.row0 + my_row] = row_s;
        }
        // all warps' maxima are there
        if (!__syncthreads_and(ok)) {
            factors_landed();
            if (tid == 0) land_copies(full_bar(0), n, i1 - i0);
            return;
        }
        // ---- column scales
        if (tid < 384) {
            float m = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; w += 2)
                m = max3_abs(m, s_colmax[w * 384 + tid], s_colmax[(w + 1) * 384 + tid]);
            const float s = fg8::tile_scale_fast(m);
            // a subnormal scale is handed on negated: its codes take the division
            s_colinv[tid] = fg8::scale_subnormal(s) ? -s : fg8::inv_scale(s);
            const int which = tid >> 7, c = 128 * cb + (tid & 127);
            const int64_t pt = cur.tile;
            if (which < 2) a.sdT[pt * (2 * (int64_t)a.I) + which * (int64_t)a.I + c] = s;
            else a.shT[pt * (int64_t)a.I + c] = s;
        }
        __syncthreads();

        // ---- second pass: codes by rows (a 128-byte line a warp and row) and by
        // columns (8 tokens of a column a thread, in pairs of tokens)
        {
            const float4* ci = reinterpret_cast<const float4*>(s_colinv) + lane;
            bool divide = fg8::scale_subnormal(row_s);
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                const float4 v = ci[32 * k];
                divide |= fminf(fminf(v.x, v.y), fminf(v.z, v.w)) < 0.f;
            }
            divide = __any_sync(kFull, divide);
            const int rows = cur.n_in - r0;
            uint8_t* out = a.dq + (int64_t)(cur.row0 + r0) * (2 * a.I) + 128 * cb + 4 * lane;
            uint2 code[3][4];   // [dG, dU, w h][column]: 8 tokens
            auto four = [&](int i, auto exact) {   // rows i .. i + 3, one matrix after the other (registers)
                constexpr bool kExact = decltype(exact)::value;
                auto by_rows = [&](const float2 (&v)[4][2], int src, int at) {
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const float2 r = splat(__shfl_sync(kFull, kExact ? row_s : row_inv, src + i + h));
                        const uint32_t w = __byte_perm(code2<kExact>(v[h][0], r), code2<kExact>(v[h][1], r), 0x5410);
                        if (i + h < rows) *reinterpret_cast<uint32_t*>(out + (i + h) * (2 * a.I) + at) = w;
                    }
                };
                auto by_columns = [&](const float2 (&v)[4][2], int k) {
                    const float4 inv = ci[32 * k];
                    const uint32_t q[4] = {
                        __byte_perm(code_pair<kExact>(v[0][0].x, v[1][0].x, inv.x), code_pair<kExact>(v[2][0].x, v[3][0].x, inv.x), 0x5410),
                        __byte_perm(code_pair<kExact>(v[0][0].y, v[1][0].y, inv.y), code_pair<kExact>(v[2][0].y, v[3][0].y, inv.y), 0x5410),
                        __byte_perm(code_pair<kExact>(v[0][1].x, v[1][1].x, inv.z), code_pair<kExact>(v[2][1].x, v[3][1].x, inv.z), 0x5410),
                        __byte_perm(code_pair<kExact>(v[0][1].y, v[1][1].y, inv.w), code_pair<kExact>(v[2][1].y, v[3][1].y, inv.w), 0x5410)};
#pragma unroll
                    for (int c = 0; c < 4; ++c) (i ? code[k][c].y : code[k][c].x) = q[c];
                };
                float2 v[4][2];
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    v[h][0] = dG[i + h][0];
                    v[h][1] = dG[i + h][1];
                }
                by_rows(v, 0, 0);
                by_columns(v, 0);
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const uint2 dw = *reinterpret_cast<const uint2*>(sdh + (r0 + i + h) * 256);
                    v[h][0] = __fmul2_rn(make_float2(fg8::bf16_lo(dw.x), fg8::bf16_hi(dw.x)), S[i + h][0]);
                    v[h][1] = __fmul2_rn(make_float2(fg8::bf16_lo(dw.y), fg8::bf16_hi(dw.y)), S[i + h][1]);
                }
                by_rows(v, kRows, a.I);
                by_columns(v, 1);
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const uint32_t a_u = a_g + kCodeBytes + (r0 + i + h) * 128;
                    const float2 fu = splat(fac[r0 + i + h].y);
                    v[h][0] = __fmul2_rn(__fmul2_rn(fg8::e4m3x2_at(a_u), fu), S[i + h][0]);
                    v[h][1] = __fmul2_rn(__fmul2_rn(fg8::e4m3x2_at(a_u + 2), fu), S[i + h][1]);
                }
                by_columns(v, 2);
            };
            if (!divide) {
                four(0, std::false_type());
                four(4, std::false_type());
            } else {
                four(0, std::true_type());
                four(4, std::true_type());
            }
            if (rows < kRows) {   // padding tokens: code 0 (not the code of -0)
                const int k0 = max(0, min(4, rows)), k1 = max(0, min(4, rows - 4));
                const uint32_t m0 = k0 == 4 ? 0xFFFFFFFFu : (1u << (8 * k0)) - 1u;
                const uint32_t m1 = k1 == 4 ? 0xFFFFFFFFu : (1u << (8 * k1)) - 1u;
#pragma unroll
                for (int k = 0; k < 3; ++k)
#pragma unroll
                    for (int c = 0; c < 4; ++c) code[k][c] = make_uint2(code[k][c].x & m0, code[k][c].y & m1);
            }
            uint8_t* base = smem + kOffTrans + 4 * lane * 128 + 8 * (warp ^ (lane & 15));
#pragma unroll
            for (int k = 0; k < 3; ++k)
#pragma unroll
                for (int c = 0; c < 4; ++c) *reinterpret_cast<uint2*>(base + k * kCodeBytes + c * 128) = code[k][c];
        }
        factors_landed();
        __syncthreads();   // the turned codes are there, and the stage has been read
        if (tid == 0 && it + 2 < i1) {
            const int up = (cb + 2) / ncb;   // tiles further on
            issue(cb + 2 - up * ncb, up ? tile_of(cur.tile + up).row0 : cur.row0, st);
        }
        {
            // 16 bytes of a column a thread: columns tid / 8 and 64 further on
            const int c0 = tid >> 3, p = tid & 7, f = (c0 >> 2) & 15;   // (col >> 2) & 15 is the same for both
            const uint8_t* src = smem + kOffTrans + c0 * 128 + 16 * (p ^ (f >> 1));
            uint8_t* dst[3];
            dst[0] = a.dqT + (int64_t)(128 * cb + c0) * a.P + 128 * (int64_t)cur.tile + 16 * p;
            dst[1] = dst[0] + (int64_t)a.I * a.P;
            dst[2] = a.hqT + (dst[0] - a.dqT);
            const int64_t half = 64 * a.P;
#pragma unroll
            for (int k = 0; k < 3; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint4 v = *reinterpret_cast<const uint4*>(src + k * kCodeBytes + h * 64 * 128);
                    if (f & 1) v = make_uint4(v.z, v.w, v.x, v.y);
                    *reinterpret_cast<uint4*>(dst[k] + h * half) = v;
                }
        }
        if (++cb == ncb) {
            cb = 0;
            if (it + 1 < i1) cur = tile_of(cur.tile + 1);
        }
    }
}

}  // namespace

extern "C" fg8_status fg8_swiglu_backward_quant(const uint16_t* dh, const uint8_t* guq, const float* sgu,
                                                const float* row_w, const int32_t* offsets, int64_t R,
                                                int I, int E, uint8_t* dq, float* sd, uint8_t* dqT,
                                                float* sdT, uint8_t* hqT, float* shT, float* gate_dot,
                                                int32_t* offsets_out, int32_t* dev_status,
                                                fg8_stream_t stream) {
    if (R < 0 || I < 128 || I % 128 || E < 1) return FG8_ERR_INVALID_ARG;
    if (!offsets || !offsets_out) return FG8_ERR_INVALID_ARG;
    if (E > fg8::kColsMaxE || R > INT32_MAX || I > INT32_MAX / 32) return FG8_ERR_UNSUPPORTED;
    if (R == 0)
        return cudaMemsetAsync(offsets_out, 0, sizeof(int32_t) * ((size_t)E + 1), (cudaStream_t)stream) ==
                       cudaSuccess ? FG8_OK : FG8_ERR_CUDA;
    if (!dh || !guq || !sgu || !dq || !sd || !dqT || !sdT || !hqT || !shT) return FG8_ERR_INVALID_ARG;
    if (!fg8h::aligned16(dh) || !fg8h::aligned16(guq) || !fg8h::aligned16(dq) || !fg8h::aligned16(dqT) ||
        !fg8h::aligned16(hqT))
        return FG8_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(sgu) | reinterpret_cast<uintptr_t>(row_w) |
         reinterpret_cast<uintptr_t>(offsets) | reinterpret_cast<uintptr_t>(sd) |
         reinterpret_cast<uintptr_t>(sdT) | reinterpret_cast<uintptr_t>(shT) |
         reinterpret_cast<uintptr_t>(gate_dot) | reinterpret_cast<uintptr_t>(offsets_out)) & 3)
        return FG8_ERR_INVALID_ARG;
    CUtensorMap m_dh, m_gu;
    if (!fg8h::make_tensor_map_2d(&m_dh, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, dh, (uint64_t)R, (uint64_t)I,
                                  128, 128, CU_TENSOR_MAP_SWIZZLE_NONE) ||
        !fg8h::make_tensor_map_2d(&m_gu, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, guq, (uint64_t)R,
                                  2 * (uint64_t)I, 128, 128, CU_TENSOR_MAP_SWIZZLE_NONE))
        return FG8_ERR_CUDA;
    if (cudaFuncSetAttribute(act_backward, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes) !=
        cudaSuccess)
        return FG8_ERR_CUDA;
    Args a;
    a.sgu = sgu; a.row_w = row_w; a.offsets = offsets;
    a.R = R; a.P = fg8_colwise_capacity(R, E);
    a.E = E; a.I = I;
    a.dq = dq; a.sd = sd; a.dqT = dqT; a.sdT = sdT; a.hqT = hqT; a.shT = shT;
    a.gate_dot = gate_dot; a.offsets_out = offsets_out; a.status = dev_status;
    const int64_t most = (R / 128 + E) * (int64_t)(I / 128);
    if (most > INT32_MAX) return FG8_ERR_UNSUPPORTED;
    int64_t grid = fg8h::num_sms();
    if (grid > most) grid = most;
    act_backward<<<(unsigned)grid, kThreads, kSmemBytes, (cudaStream_t)stream>>>(m_dh, m_gu, a);
    return fg8h::launch_status();
}
