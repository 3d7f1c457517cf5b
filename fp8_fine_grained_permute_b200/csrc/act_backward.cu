// act_backward.cu -- the gated activation's backward from 8-bit checkpoints.
//
// The up-projection's forward saved gate and up as E4M3 codes in 1x128 tiles
// (fg8_grouped_gemm_swiglu_quant_save).  With g, u their values, dh the bf16
// gradient of the activation's output as the down-projection's dgrad of the
// unweighted output gradient gives it, and w the row's gate weight:
//     sig = 1 / (1 + exp(-g)),  h = g sig u,  d = w dh
//     dU = d g sig,   dG = d u sig (1 + g - g sig)
//     gate_dot[block][row] = sum over the 128-column block of dh h  (dL/dw in parts)
// and the three matrices that the GEMMs of the backward take leave in 8 bits:
// [dG dU] by rows (dgrad's A), [dG dU] down the token axis per expert (the up
// weight gradient's A) and w h down the token axis (the down weight gradient's).
//
// Bound by HBM: 2 + 2 bytes in and 2 + 2 + 1 bytes out an element, where the
// chain of separate passes (bf16 gradients and activations written, then read by
// each quantizer) moves 25.  Everything of a 128 x 128 block is formed once in
// registers and leaves twice:
//   * CTA = 512 threads, one persistent worker per SM; the (tile, column block)
//     items are cut into contiguous ranges, one a CTA.  TMA brings an item's
//     32 + 16 + 16 KB into one of two stages while the item before is worked on.
//   * thread = 4 columns x 8 rows (a warp reads whole 128-byte code rows), dG, dU
//     and w h of these 32 elements in 96 registers.
//   * a row's maximum is one warp reduction, and its codes are one 128-byte store
//     a warp; the column maxima of the 16 warps meet in shared memory.
//   * the column codes (8 tokens of a column a thread) are turned around through
//     shared memory, 8-byte pieces XOR-swizzled by column, and leave as 128-byte
//     lines of the token axis.
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
constexpr uint32_t kOffScales = kOffColInv + 4 * 384;              // float [2][3][128]
constexpr uint32_t kOffBars = kOffScales + 2 * 4 * 384;            // 2 mbarriers, abort flag
constexpr uint32_t kOffPref = kOffBars + 32;                       // int32 [kColsMaxE + 1]
constexpr uint32_t kOffWarp = kOffPref + 4 * (fg8::kColsMaxE + 4); // int32 [36]
constexpr uint32_t kSmemBytes = kOffWarp + 4 * 36 + 128;           // + alignment slack
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

// code pair of (x, y) / s: with the reciprocal, or the division for a subnormal scale
FG8_DEV uint32_t code2(float x, float y, float inv) {
    return fg8::cvt_e4m3x2(fg8::mul_f32x2(fg8::pack_f32x2(x, y), fg8::pack_f32x2(inv, inv)));
}
FG8_DEV uint32_t code1_exact(float x, float s) { return fg8::cvt_e4m3x2(__fdiv_rn(x, s), 0.f) & 0xFFu; }

__global__ void __launch_bounds__(kThreads, 1)
act_backward(const __grid_constant__ CUtensorMap tm_dh, const __grid_constant__ CUtensorMap tm_gu,
             const Args a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~static_cast<uintptr_t>(127));
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

    const int64_t tiles = min((int64_t)s_pref[a.E], a.P / 128);
    const int64_t items = tiles * ncb;
    const int64_t i0 = items * blockIdx.x / gridDim.x, i1 = items * (blockIdx.x + 1) / gridDim.x;
    if (i0 >= i1) return;

    auto tile_of = [&](int64_t it) {
        return fg8::find_tile((int)(it / ncb), s_pref, a.offsets, a.E, a.R);
    };
    auto issue = [&](int64_t it, const fg8::RowTile& t, int st) {   // one thread
        const int cb = (int)(it % ncb), y = (int)max((int64_t)0, min(t.row0, a.R - 1));
        const uint32_t dst = sbase + st * kStage;
        mbar_arrive_expect_tx(full_bar(st), kStage);
        tma_load_2d(&tm_dh, dst, full_bar(st), 128 * cb, y);
        tma_load_2d(&tm_gu, dst + kDhBytes, full_bar(st), 128 * cb, y);
        tma_load_2d(&tm_gu, dst + kDhBytes + kCodeBytes, full_bar(st), a.I + 128 * cb, y);
    };
    // this thread's one of an item's 3 x 128 row factors: gate scale, up scale, weight
    auto load_factor = [&](int64_t it, const fg8::RowTile& t) {
        const int which = tid >> 7, r = tid & 127;
        if (which > 2 || r >= t.n_in) return 0.f;
        const int64_t row = t.row0 + r;
        if (which == 2) return a.row_w ? __ldg(a.row_w + row) : 1.0f;
        return __ldg(a.sgu + (int64_t)((which ? ncb : 0) + (int)(it % ncb)) * a.R + row);
    };

    fg8::RowTile cur = tile_of(i0);
    if (tid == 0) {
        issue(i0, cur, 0);
        if (i0 + 1 < i1) issue(i0 + 1, tile_of(i0 + 1), 1);
    }
    if (tid < 384) s_scales[tid] = load_factor(i0, cur);
    __syncthreads();

    bool ok = true;
    for (int64_t it = i0; it < i1; ++it) {
        const int n = (int)(it - i0), st = n & 1;
        const int cb = (int)(it % ncb);
        fg8::RowTile nxt = cur;
        float next_factor = 0.f;
        if (it + 1 < i1) {
            if ((it + 1) % ncb == 0) nxt = tile_of(it + 1);
            next_factor = load_factor(it + 1, nxt);
        }
        const float* fac = s_scales + 384 * st;
        const uint8_t* sdh = smem + st * kStage + 8 * lane;
        const uint8_t* sg = smem + st * kStage + kDhBytes + 4 * lane;
        const int r0 = kRows * warp;
        ok = mbar_wait(full_bar(st), (n >> 1) & 1, abort_flag, a.status);

        // ---- values of 8 rows x 4 columns
        float dG[kRows][4], dU[kRows][4], H[kRows][4];
        float dot[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = r0 + i;
            dot[i] = 0.f;
            if (r < cur.n_in) {   // warp-uniform; padding rows take no part
                const uint32_t gw = *reinterpret_cast<const uint32_t*>(sg + r * 128);
                const uint32_t uw = *reinterpret_cast<const uint32_t*>(sg + kCodeBytes + r * 128);
                const uint2 dw = *reinterpret_cast<const uint2*>(sdh + r * 256);
                const float fg = fac[r], fu = fac[128 + r], w = fac[256 + r];
                const float2 g2[2] = {fg8::e4m3x2_f32(gw & 0xFFFFu), fg8::e4m3x2_f32(gw >> 16)};
                const float2 u2[2] = {fg8::e4m3x2_f32(uw & 0xFFFFu), fg8::e4m3x2_f32(uw >> 16)};
                const float gc[4] = {g2[0].x, g2[0].y, g2[1].x, g2[1].y};
                const float uc[4] = {u2[0].x, u2[0].y, u2[1].x, u2[1].y};
                const float dc[4] = {fg8::bf16_lo(dw.x), fg8::bf16_hi(dw.x), fg8::bf16_lo(dw.y),
                                     fg8::bf16_hi(dw.y)};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float g = gc[c] * fg, u = uc[c] * fu;
                    // exp2's argument is clamped so that 1 + e stays finite (and
                    // its reciprocal above the flushed range): sig >= 2^-125
                    const float sig = rcp(1.0f + ex2(fminf(g * -1.4426950408889634f, 125.0f)));
                    const float silu = g * sig, h = silu * u;
                    dot[i] = fmaf(dc[c], h, dot[i]);
                    const float d = dc[c] * w;
                    dU[i][c] = d * silu;
                    dG[i][c] = d * u * sig * (1.0f + fmaf(-g, sig, g));
                    H[i][c] = h * w;
                }
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c) dG[i][c] = dU[i][c] = H[i][c] = 0.f;
            }
        }
        // ---- column maxima of this warp's rows
        {
            float m[3][4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                m[0][c] = m[1][c] = m[2][c] = 0.f;
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    m[0][c] = fmaxf(m[0][c], fabsf(dG[i][c]));
                    m[1][c] = fmaxf(m[1][c], fabsf(dU[i][c]));
                    m[2][c] = fmaxf(m[2][c], fabsf(H[i][c]));
                }
            }
#pragma unroll
            for (int k = 0; k < 3; ++k)
                *reinterpret_cast<float4*>(s_colmax + warp * 384 + k * 128 + 4 * lane) =
                    make_float4(m[k][0], m[k][1], m[k][2], m[k][3]);
        }
        // all warps' maxima are there, and the stage has been read
        if (!__syncthreads_and(ok)) {
            ok = false;
            break;
        }
        if (tid == 0 && it + 2 < i1) issue(it + 2, (it + 2) / ncb == it / ncb ? cur : tile_of(it + 2), st);

        // ---- by rows: lane i < 16 owns the scale of row i & 7 of dG (i < 8) or dU
        {
            float mine = 0.f;
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const float mg = fmaxf(fmaxf(fabsf(dG[i][0]), fabsf(dG[i][1])), fmaxf(fabsf(dG[i][2]), fabsf(dG[i][3])));
                const float mu = fmaxf(fmaxf(fabsf(dU[i][0]), fabsf(dU[i][1])), fmaxf(fabsf(dU[i][2]), fabsf(dU[i][3])));
                const uint32_t xg = __reduce_max_sync(kFull, __float_as_uint(mg));
                const uint32_t xu = __reduce_max_sync(kFull, __float_as_uint(mu));
                if (lane == i) mine = __uint_as_float(xg);
                if (lane == kRows + i) mine = __uint_as_float(xu);
            }
            const float s = fg8::tile_scale_fast(mine);
            const float inv = fg8::inv_scale(s);
            const int my_row = r0 + (lane & 7);
            if (lane < 16 && my_row < cur.n_in)
                a.sd[(int64_t)((lane >> 3) * ncb + cb) * a.R + cur.row0 + my_row] = s;
            const bool sub = __any_sync(kFull, lane < 16 && fg8::scale_subnormal(s));
            uint8_t* out = a.dq + (cur.row0 + r0) * (2 * (int64_t)a.I) + 128 * cb + 4 * lane;
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const float ig = __shfl_sync(kFull, inv, i), iu = __shfl_sync(kFull, inv, kRows + i);
                uint32_t cg = code2(dG[i][0], dG[i][1], ig) | (code2(dG[i][2], dG[i][3], ig) << 16);
                uint32_t cu = code2(dU[i][0], dU[i][1], iu) | (code2(dU[i][2], dU[i][3], iu) << 16);
                if (sub) {
                    const float sg_ = __shfl_sync(kFull, s, i), su_ = __shfl_sync(kFull, s, kRows + i);
                    cg = cu = 0u;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        cg |= code1_exact(dG[i][c], sg_) << (8 * c);
                        cu |= code1_exact(dU[i][c], su_) << (8 * c);
                    }
                }
                if (r0 + i < cur.n_in) {
                    uint8_t* o = out + (int64_t)i * (2 * (int64_t)a.I);
                    *reinterpret_cast<uint32_t*>(o) = cg;
                    *reinterpret_cast<uint32_t*>(o + a.I) = cu;
                }
            }
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
        // ---- column scales
        if (tid < 384) {
            float m = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_colmax[w * 384 + tid]);
            const float s = fg8::tile_scale_fast(m);
            // a subnormal scale is handed on negated: its codes take the division
            s_colinv[tid] = fg8::scale_subnormal(s) ? -s : fg8::inv_scale(s);
            const int which = tid >> 7, c = 128 * cb + (tid & 127);
            const int64_t pt = cur.pcol / 128;
            if (which < 2) a.sdT[pt * (2 * (int64_t)a.I) + which * (int64_t)a.I + c] = s;
            else a.shT[pt * (int64_t)a.I + c] = s;
        }
        __syncthreads();

        // ---- by columns: 8 tokens of 4 columns of the three matrices
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const float4 i4 = *reinterpret_cast<const float4*>(s_colinv + 128 * k + 4 * lane);
            const float inv[4] = {i4.x, i4.y, i4.z, i4.w};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float v[kRows];
#pragma unroll
                for (int i = 0; i < kRows; ++i) v[i] = k == 0 ? dG[i][c] : k == 1 ? dU[i][c] : H[i][c];
                uint2 q;
                if (inv[c] < 0.f) {
                    q = make_uint2(0u, 0u);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        q.x |= code1_exact(v[i], -inv[c]) << (8 * i);
                        q.y |= code1_exact(v[4 + i], -inv[c]) << (8 * i);
                    }
                } else {
                    q.x = code2(v[0], v[1], inv[c]) | (code2(v[2], v[3], inv[c]) << 16);
                    q.y = code2(v[4], v[5], inv[c]) | (code2(v[6], v[7], inv[c]) << 16);
                }
                *reinterpret_cast<uint2*>(smem + kOffTrans + k * kCodeBytes + (4 * lane + c) * 128 +
                                          8 * (warp ^ (lane & 15))) = q;
            }
        }
        if (tid < 384 && it + 1 < i1) s_scales[384 * (st ^ 1) + tid] = next_factor;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 3 * 128 * 8 / kThreads; ++j) {
            const int u = tid + kThreads * j, k = u >> 10, col = (u >> 3) & 127, p = u & 7;
            const int f = (col >> 2) & 15;
            uint4 v = *reinterpret_cast<const uint4*>(smem + kOffTrans + k * kCodeBytes + col * 128 +
                                                      16 * (p ^ (f >> 1)));
            if (f & 1) v = make_uint4(v.z, v.w, v.x, v.y);
            const int64_t c = 128 * cb + col;
            uint8_t* o = k < 2 ? a.dqT + (k * (int64_t)a.I + c) * a.P : a.hqT + c * a.P;
            *reinterpret_cast<uint4*>(o + cur.pcol + 16 * p) = v;
        }
        cur = nxt;
    }
    if (!ok && tid == 0) {   // let copies already issued land before the CTA winds down
        const uint64_t t0 = fg8::globaltimer_ns();
        while (!(mbar_try_wait(full_bar(0), 0) && mbar_try_wait(full_bar(1), 0)) &&
               fg8::globaltimer_ns() - t0 < 100000000ull) {
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
    if (E > fg8::kColsMaxE || R > INT32_MAX || I > INT32_MAX / 2) return FG8_ERR_UNSUPPORTED;
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
    int64_t grid = fg8h::num_sms();
    if (grid > most) grid = most;
    act_backward<<<(unsigned)grid, kThreads, kSmemBytes, (cudaStream_t)stream>>>(m_dh, m_gu, a);
    return fg8h::launch_status();
}
