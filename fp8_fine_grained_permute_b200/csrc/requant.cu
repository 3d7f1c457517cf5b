// requant.cu -- column-wise (token-axis) operand from rows saved in 8 bits.
//
// An activation checkpoint keeps a token's row as E4M3 codes with one scale per
// 1x128 tile (2 bytes a value less than fp32, half of bf16).  The weight
// gradient contracts over tokens and so needs 1x128 tiles along the token axis:
//     x = fp32(code * s),  sT = fp32(amax / 448) over 128 tokens of one expert,
//     q = E4M3(fp32(x / sT))
// -- fg8_quantize_act's column-wise mode on values read from the checkpoint,
// with its row gather, tiles, padding and outputs.
//
// Bytes in and out are 1 an element each (gathered rows come mostly from L2), so
// the instructions an element decide: conversions run at 32 a cycle and SM
// against 128 for FMAs.  An element takes one half of a two-wide conversion each
// way and the quotient as product, residual, correction in packed fp32 (three
// half instructions; two conversions of a bracket, as the 16-bit quantizers
// form, would double the conversions).  With r = fp32(1 / sT) correctly rounded,
// z0 = x r is off by 2^-23 at most, and z = z0 - (z0 sT - x) r is the quotient
// to 2^-45 before its own rounding to fp32.  (In that order, on -x and -r, the
// sign of a zero survives: z0 + (x - z0 sT) r turns -0 into +0.)
//
// CTA = 256 threads on one 128-token tile of an expert and a group of its
// 128-column blocks; cp.async gathers the next block's 16 KB while this one is
// converted.  Thread = 4 columns x 16 tokens: a warp reads whole 128-byte rows,
// the 8 warps' column maxima meet in shared memory, and the codes are turned
// around there too (16-byte pieces, XOR-swizzled by column) to leave as
// 128-byte lines.
#include "fg8_columns.cuh"
#include "fg8_tma.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 128 / kWarps;                  // tokens of a thread: 16
constexpr uint32_t kTile = 128 * 128;                // one block's codes
constexpr uint32_t kOffTrans = 2 * kTile;            // [128 columns][128 tokens]
constexpr uint32_t kOffMax = kOffTrans + kTile;      // float [8][128]
constexpr uint32_t kOffCol = kOffMax + 4 * kWarps * 128;   // float2 [128]: scale, reciprocal
constexpr uint32_t kOffScale = kOffCol + 8 * 128;    // float [2][128]: row scales
constexpr uint32_t kOffPref = kOffScale + 2 * 4 * 128;
constexpr uint32_t kOffWarp = kOffPref + 4 * (fg8::kColsMaxE + 4);
constexpr uint32_t kOffRows = kOffWarp + 4 * 36;     // int32 [128]
constexpr uint32_t kSmemBytes = kOffRows + 4 * 128;
constexpr int kColGroups = 4;                        // column groups per tile (grid.y)

struct Args {
    const uint8_t* xq;        // [T][K]
    const float* sx;          // [K / 128][T]
    const int32_t* row_token; // [R] or NULL
    const int32_t* offsets;
    int64_t T, R, K, P;
    int E;
    uint8_t* xqT;             // [K][P]
    float* saT;               // [P / 128][K]
    int32_t* offsets_out;
    int32_t* status;
};

FG8_DEV uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

__global__ void __launch_bounds__(kThreads, 2) requant_columns(const Args a) {
    extern __shared__ __align__(128) uint8_t smem[];
    float* s_max = reinterpret_cast<float*>(smem + kOffMax);
    float2* s_col = reinterpret_cast<float2*>(smem + kOffCol);
    float* s_scale = reinterpret_cast<float*>(smem + kOffScale);
    int32_t* s_pref = reinterpret_cast<int32_t*>(smem + kOffPref);
    int32_t* s_rows = reinterpret_cast<int32_t*>(smem + kOffRows);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    fg8::tile_prefix(a.offsets, a.E, s_pref, reinterpret_cast<int32_t*>(smem + kOffWarp));
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int e = tid; e <= a.E; e += kThreads) a.offsets_out[e] = 128 * s_pref[e];
    const int tile = blockIdx.x;
    if (tile >= s_pref[a.E] || 128 * (int64_t)tile + 128 > a.P) return;
    const fg8::RowTile t = fg8::find_tile(tile, s_pref, a.offsets, a.E, (int)a.R);
    if (tid < 128) {
        int32_t src = -1;
        if (tid < t.n_in) {
            const int64_t v = a.row_token ? (int64_t)a.row_token[t.row0 + tid] : (int64_t)t.row0 + tid;
            if (v >= 0 && v < a.T) src = (int32_t)v;
            else fg8::set_status(a.status, FG8_ERR_INVALID_ARG);
        }
        s_rows[tid] = src;
    }
    __syncthreads();
    const int ncb = (int)(a.K / 128);
    const int cb0 = (int)((int64_t)ncb * blockIdx.y / gridDim.y), cb1 = (int)((int64_t)ncb * (blockIdx.y + 1) / gridDim.y);
    if (cb0 >= cb1) return;

    const int32_t my_src = s_rows[tid & 127];
    auto issue = [&](int cb, int st) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int u = tid + kThreads * j, r = u >> 3, ch = u & 7;
            const int32_t src = s_rows[r];
            const uint8_t* p = a.xq + (src >= 0 ? (int64_t)src * a.K + 128 * cb + 16 * ch : 0);
            const uint32_t n = src >= 0 ? 16u : 0u;   // rows of padding: zeros
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                             fg8::tma::smem_u32(smem + st * kTile + 16 * u)),
                         "l"(p), "r"(n)
                         : "memory");
        }
        if (tid < 128) {
            const uint32_t n = my_src >= 0 ? 4u : 0u;
            const float* p = a.sx + (my_src >= 0 ? (int64_t)cb * a.T + my_src : 0);
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(
                             fg8::tma::smem_u32(s_scale + 128 * st + tid)),
                         "l"(p), "r"(n)
                         : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    issue(cb0, 0);
    for (int cb = cb0; cb < cb1; ++cb) {
        const int st = (cb - cb0) & 1;
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();   // this block is there; the other stage and the transposed codes have been read
        if (cb + 1 < cb1) issue(cb + 1, st ^ 1);

        // 16 tokens x 4 columns, negated
        uint64_t x[kRows][2];
        float m[4] = {0.f, 0.f, 0.f, 0.f};
        const uint8_t* src = smem + st * kTile + (kRows * warp) * 128 + 4 * lane;
        const float* sc = s_scale + 128 * st + kRows * warp;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(src + 128 * i);
            const float s = -sc[i];
            const float2 v0 = fg8::e4m3x2_f32(w & 0xFFFFu), v1 = fg8::e4m3x2_f32(w >> 16);
            const float2 p0 = __fmul2_rn(v0, make_float2(s, s)), p1 = __fmul2_rn(v1, make_float2(s, s));
            x[i][0] = fg8::pack_f32x2(p0.x, p0.y);
            x[i][1] = fg8::pack_f32x2(p1.x, p1.y);
            m[0] = fmaxf(m[0], fabsf(p0.x));
            m[1] = fmaxf(m[1], fabsf(p0.y));
            m[2] = fmaxf(m[2], fabsf(p1.x));
            m[3] = fmaxf(m[3], fabsf(p1.y));
        }
        *reinterpret_cast<float4*>(s_max + 128 * warp + 4 * lane) = make_float4(m[0], m[1], m[2], m[3]);
        __syncthreads();
        if (tid < 128) {
            float mm = s_max[tid];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) mm = fmaxf(mm, s_max[128 * w + tid]);
            const float s = fg8::tile_scale_fast(mm);
            // reciprocal 0: the quotient's residual would leave the normal range
            // (scales below 2^-100), these codes take the division
            s_col[tid] = make_float2(s, s >= 0x1p-100f ? __frcp_rn(s) : 0.f);
            a.saT[(int64_t)tile * a.K + 128 * cb + tid] = s;
        }
        __syncthreads();
        float sT[4], r[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float2 v = s_col[4 * lane + c];
            sT[c] = v.x;
            r[c] = v.y;
        }
        uint32_t code[kRows / 4][4];   // [token group][column]: 4 tokens a word
        const bool tiny = r[0] == 0.f || r[1] == 0.f || r[2] == 0.f || r[3] == 0.f;
        if (!tiny) {
            const uint64_t rr[2] = {fg8::pack_f32x2(-r[0], -r[1]), fg8::pack_f32x2(-r[2], -r[3])};
            const uint64_t ss[2] = {fg8::pack_f32x2(sT[0], sT[1]), fg8::pack_f32x2(sT[2], sT[3])};
#pragma unroll
            for (int g = 0; g < kRows / 4; ++g) {
                uint32_t w[4];   // token i's four codes, columns in bytes
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t h[2];
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const uint64_t xv = x[4 * g + i][p];
                        const uint64_t z0 = fg8::mul_f32x2(xv, rr[p]);
                        h[p] = fg8::cvt_e4m3x2(fma_f32x2(fma_f32x2(z0, ss[p], xv), rr[p], z0));
                    }
                    w[i] = h[0] | (h[1] << 16);
                }
                // 4 x 4 bytes turned: column words of 4 tokens
                const uint32_t a0 = __byte_perm(w[0], w[1], 0x5140), a1 = __byte_perm(w[2], w[3], 0x5140);
                const uint32_t b0 = __byte_perm(w[0], w[1], 0x7362), b1 = __byte_perm(w[2], w[3], 0x7362);
                code[g][0] = __byte_perm(a0, a1, 0x5410);
                code[g][1] = __byte_perm(a0, a1, 0x7632);
                code[g][2] = __byte_perm(b0, b1, 0x5410);
                code[g][3] = __byte_perm(b0, b1, 0x7632);
            }
        } else {
#pragma unroll
            for (int g = 0; g < kRows / 4; ++g) {
#pragma unroll
                for (int c = 0; c < 4; ++c) code[g][c] = 0u;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float v[4];
                    asm("mov.b64 {%0, %1}, %2;" : "=f"(v[0]), "=f"(v[1]) : "l"(x[4 * g + i][0]));
                    asm("mov.b64 {%0, %1}, %2;" : "=f"(v[2]), "=f"(v[3]) : "l"(x[4 * g + i][1]));
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        code[g][c] |= (fg8::cvt_e4m3x2(__fdiv_rn(-v[c], sT[c]), 0.f) & 0xFFu) << (8 * i);
                }
            }
        }
        // 16 tokens of a column: piece `warp` of its 128 bytes, at warp ^ (lane & 7)
#pragma unroll
        for (int c = 0; c < 4; ++c)
            *reinterpret_cast<uint4*>(smem + kOffTrans + (4 * lane + c) * 128 + 16 * (warp ^ (lane & 7))) =
                make_uint4(code[0][c], code[1][c], code[2][c], code[3][c]);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int u = tid + kThreads * j, col = u >> 3, p = u & 7;
            const uint4 v = *reinterpret_cast<const uint4*>(smem + kOffTrans + col * 128 +
                                                            16 * (p ^ ((col >> 2) & 7)));
            *reinterpret_cast<uint4*>(a.xqT + (int64_t)(128 * cb + col) * a.P + 128 * (int64_t)tile + 16 * p) = v;
        }
    }
}

}  // namespace

extern "C" fg8_status fg8_requantize_colwise(const uint8_t* xq, const float* sx, int64_t T, int64_t K,
                                             const int32_t* row_token, const int32_t* offsets, int64_t R,
                                             int E, uint8_t* xqT, float* saT, int32_t* offsets_out,
                                             int32_t* dev_status, fg8_stream_t stream) {
    if (T < 0 || R < 0 || K < 128 || K % 128 || E < 1) return FG8_ERR_INVALID_ARG;
    if (!offsets || !offsets_out) return FG8_ERR_INVALID_ARG;
    if (row_token == nullptr && R != T) return FG8_ERR_INVALID_ARG;
    if (E > fg8::kColsMaxE || R > INT32_MAX || T > INT32_MAX || K / 128 > INT32_MAX)
        return FG8_ERR_UNSUPPORTED;
    if (R == 0)
        return cudaMemsetAsync(offsets_out, 0, sizeof(int32_t) * ((size_t)E + 1), (cudaStream_t)stream) ==
                       cudaSuccess ? FG8_OK : FG8_ERR_CUDA;
    if (T == 0 || !xq || !sx || !xqT || !saT) return FG8_ERR_INVALID_ARG;
    if (!fg8h::aligned16(xq) || !fg8h::aligned16(xqT)) return FG8_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(sx) | reinterpret_cast<uintptr_t>(row_token) |
         reinterpret_cast<uintptr_t>(offsets) | reinterpret_cast<uintptr_t>(saT) |
         reinterpret_cast<uintptr_t>(offsets_out)) & 3)
        return FG8_ERR_INVALID_ARG;
    Args a;
    a.xq = xq; a.sx = sx; a.row_token = row_token; a.offsets = offsets;
    a.T = T; a.R = R; a.K = K; a.P = fg8_colwise_capacity(R, E);
    a.E = E; a.xqT = xqT; a.saT = saT; a.offsets_out = offsets_out; a.status = dev_status;
    if (cudaFuncSetAttribute(requant_columns, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes) !=
        cudaSuccess)
        return FG8_ERR_CUDA;
    const dim3 grid((unsigned)(R / 128 + E), (unsigned)kColGroups);
    requant_columns<<<grid, kThreads, kSmemBytes, (cudaStream_t)stream>>>(a);
    return fg8h::launch_status();
}
