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
// the instructions an element decide: conversions to E4M3 run at 32 a cycle and SM
// against 128 for FMAs.  An element takes one half of a two-wide conversion each
// way and the quotient as product, residual, correction in packed fp32 (three
// half instructions; two conversions of a bracket, as the 16-bit quantizers
// form, would double the conversions).  It gives the division's codes: see
// fg8::Corrected.  (Here on -x and -r: z0 - (z0 sT - x) r keeps the sign of a zero,
// z0 + (x - z0 sT) r turns -0 into +0; turning the codes' sign bits instead, as the
// saving GEMM does, took 288 us.)
//
// CTA = 256 threads, two a SM, with a contiguous range of (128-token tile, 128
// columns) items each; cp.async gathers three items ahead (two: 280 us, four: 281).
// A warp owns 16 columns of all 128 tokens, a thread 4 columns x 16 tokens: the
// column maxima are 16 values in a thread and three shuffles, a thread's codes of a
// column are 16 consecutive bytes, and the 8 lanes of a column write its whole
// 128-byte line -- no exchange through shared memory and one barrier an item.
//
// On a B200: 271 us for 8192 token rows x 7168 to 65536 rows of 256 experts (0.55 GB
// at least, 85 us at the copy rate; 0.64 GB with the padding), 13 us for 333 x 2048
// to 1998 rows of 64.  Of 280 us before the fourth stage the arithmetic alone took 257,
// gathers and stores alone 234 (gathers 66, stores 151: 128-byte lines of as many
// columns as an item has).  No pipe is saturated (counters of a 16384-row call: 55 % of
// the issue slots, ALU 42 %, FMA 35 %, LSU 26 %): 16 warps an SM wait for their own
// chains of load, conversion, maximum, shuffles, reciprocal and quotient and for the
// barrier of each item.
// Columns turned around through shared memory took 346 us; threads of 8 tokens, 32
// warps an SM at 64 registers, 336 us; two passes over the staged codes with more CTAs
// an SM were no faster.
#include "fg8_columns.cuh"
#include "fg8_tma.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kRows = 16;                            // tokens of a thread
constexpr int kCtasPerSm = 2;
constexpr int kStages = 4;
constexpr uint32_t kTile = 128 * 128;                // an item's codes
constexpr uint32_t kScalePitch = 20;                 // floats from 16 rows' scales to the next 16: conflict-free 16-byte reads
constexpr uint32_t kOffScale = kStages * kTile;      // float [stages][8][20]
constexpr uint32_t kOffPref = kOffScale + kStages * 4 * 8 * kScalePitch;
constexpr uint32_t kOffWarp = kOffPref + 4 * (fg8::kColsMaxE + 4);
constexpr uint32_t kSmemBytes = kOffWarp + 4 * 36;

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

// -s by the FMA pipe
FG8_DEV float negated(float s) {
    float d;
    asm("fma.rn.f32 %0, %1, 0fBF800000, 0f80000000;" : "=f"(d) : "f"(s));
    return d;
}

__global__ void __launch_bounds__(kThreads, kCtasPerSm) requant_columns(const Args a) {
    extern __shared__ __align__(128) uint8_t smem[];
    float* s_scale = reinterpret_cast<float*>(smem + kOffScale);
    int32_t* s_pref = reinterpret_cast<int32_t*>(smem + kOffPref);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int word = lane & 3, group = lane >> 2;   // columns 16 warp + 4 word .., tokens 16 group ..

    fg8::tile_prefix(a.offsets, a.E, s_pref, reinterpret_cast<int32_t*>(smem + kOffWarp));
    if (blockIdx.x == 0)
        for (int e = tid; e <= a.E; e += kThreads) a.offsets_out[e] = 128 * s_pref[e];
    const int ncb = (int)(a.K / 128);
    const int tiles = (int)min((int64_t)s_pref[a.E], a.P / 128);
    const int64_t items = (int64_t)tiles * ncb;
    const int64_t i0 = items * blockIdx.x / gridDim.x;
    int left = (int)(items * (blockIdx.x + 1) / gridDim.x - i0);   // items to go
    if (left == 0) return;
    int tile = (int)(i0 / ncb), cb = (int)(i0 % ncb);

    // What a thread gathers: 16 bytes of rows tid / 8, 32, 64 and 96 further on, and
    // (the first 128) a row's scale.  Chunk c of row r stands at c ^ (r / 16 mod 8):
    // the 8 token groups that a warp reads together are on different banks.
    const uint8_t* src[4];
    const float* src_scale = nullptr;
    uint32_t src_ok = 0;   // bits 0..3: the rows exist (padding: zeros); bit 4: the scale's
    int ahead_tile = tile, ahead_cb = cb, ahead = left, ahead_stage = 0;
    auto find_sources = [&](int t, int c) {   // for item (t, c) and the ones after it in the tile
        const fg8::RowTile rt = fg8::find_tile(t, s_pref, a.offsets, a.E, (int)a.R);
        auto source = [&](int r) {
            if (r >= rt.n_in) return (int64_t)-1;
            const int64_t v = a.row_token ? (int64_t)a.row_token[rt.row0 + r] : (int64_t)rt.row0 + r;
            if (v >= 0 && v < a.T) return v;
            fg8::set_status(a.status, FG8_ERR_INVALID_ARG);
            return (int64_t)-1;
        };
        src_ok = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t v = source((tid >> 3) + 32 * j);
            src_ok |= (uint32_t)(v >= 0) << j;
            src[j] = a.xq + max(v, (int64_t)0) * a.K + 128 * (int64_t)c + 16 * (tid & 7);
        }
        if (tid < 128) {
            const int64_t v = source(tid);
            src_ok |= (uint32_t)(v >= 0) << 4;
            src_scale = a.sx + (int64_t)c * a.T + max(v, (int64_t)0);
        }
    };
    const uint32_t sbase = fg8::tma::smem_u32(smem);
    auto issue = [&]() {   // the next item of the CTA's range, if there is one
        if (ahead > 0) {
            --ahead;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = (tid >> 3) + 32 * j;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                 sbase + ahead_stage * kTile + 128 * r + 16 * ((tid & 7) ^ (r >> 4))),
                             "l"(src[j]), "r"(src_ok >> j & 1u ? 16u : 0u)
                             : "memory");
                src[j] += 128;
            }
            if (tid < 128) {
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(
                                 sbase + kOffScale + 4 * (ahead_stage * 8 * kScalePitch + (tid >> 4) * kScalePitch + (tid & 15))),
                             "l"(src_scale), "r"(src_ok & 16u ? 4u : 0u)
                             : "memory");
                src_scale += a.T;
            }
            if (++ahead_stage == kStages) ahead_stage = 0;
            if (++ahead_cb == ncb) {
                ahead_cb = 0;
                ++ahead_tile;
                if (ahead > 0) find_sources(ahead_tile, 0);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    find_sources(tile, cb);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue();

    const int col0 = 16 * warp + 4 * word;
    uint8_t* out = a.xqT + ((int64_t)128 * cb + col0) * a.P + 128 * (int64_t)tile + 16 * group;
    for (int st = 0; left > 0; --left) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
        __syncthreads();   // this item is there, and the stage of the item before has been read
        issue();
        float4 sc[kRows / 4];
#pragma unroll
        for (int i = 0; i < kRows / 4; ++i)
            sc[i] = reinterpret_cast<const float4*>(s_scale + (st * 8 + group) * kScalePitch)[i];
        const uint32_t in_addr = sbase + st * kTile + kRows * group * 128 + 16 * (warp ^ group) + 4 * word;
        // 16 tokens x 4 columns, negated
        float2 x[kRows][2];
        float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const float2 v0 = fg8::e4m3x2_at(in_addr + 128 * i), v1 = fg8::e4m3x2_at(in_addr + 128 * i + 2);
            const float s = i % 4 == 0 ? sc[i / 4].x : i % 4 == 1 ? sc[i / 4].y : i % 4 == 2 ? sc[i / 4].z : sc[i / 4].w;
            const float ns = negated(s);
            x[i][0] = __fmul2_rn(v0, make_float2(ns, ns));
            x[i][1] = __fmul2_rn(v1, make_float2(ns, ns));
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            m[0] = fmaxf(m[0], fabsf(x[i][0].x));
            m[1] = fmaxf(m[1], fabsf(x[i][0].y));
            m[2] = fmaxf(m[2], fabsf(x[i][1].x));
            m[3] = fmaxf(m[3], fabsf(x[i][1].y));
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1)
#pragma unroll
            for (int c = 0; c < 4; ++c) m[c] = fmaxf(m[c], __shfl_xor_sync(0xffffffffu, m[c], o));
        // scale and reciprocal: lane group g works out column g mod 4 and hands it round
        const float mine = group & 2 ? (group & 1 ? m[3] : m[2]) : (group & 1 ? m[1] : m[0]);
        const float s_mine = fg8::tile_scale_fast(mine);
        // reciprocal 0: the quotient's residual would leave the normal range, these
        // codes take the division
        const float r_mine = s_mine >= fg8::kCorrectedMin ? -__frcp_rn(s_mine) : 0.f;
        if (group < 4) a.saT[(int64_t)tile * a.K + 128 * cb + col0 + group] = s_mine;
        float s[4], r[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            s[c] = __shfl_sync(0xffffffffu, s_mine, 4 * c + word);
            r[c] = __shfl_sync(0xffffffffu, r_mine, 4 * c + word);
        }
        if (!__any_sync(0xffffffffu, r_mine == 0.f)) {
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const float2 s2 = make_float2(s[2 * p], s[2 * p + 1]), nr = make_float2(r[2 * p], r[2 * p + 1]);
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    const float2 z0 = __fmul2_rn(x[i][p], nr);
                    x[i][p] = __ffma2_rn(__ffma2_rn(z0, s2, x[i][p]), nr, z0);
                }
            }
        } else {
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                const float sc_ = c == 0 ? s[0] : c == 1 ? s[1] : c == 2 ? s[2] : s[3];
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    const float v = c & 1 ? (c & 2 ? x[i][1].y : x[i][0].y) : (c & 2 ? x[i][1].x : x[i][0].x);
                    const float z = __fdiv_rn(-v, sc_);
                    if (c == 0) x[i][0].x = z;
                    if (c == 1) x[i][0].y = z;
                    if (c == 2) x[i][1].x = z;
                    if (c == 3) x[i][1].y = z;
                }
            }
        }
        // 16 tokens of a column are 16 bytes
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            uint32_t q[4];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                float z[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) z[i] = c & 1 ? x[4 * h + i][c >> 1].y : x[4 * h + i][c >> 1].x;
                q[h] = __byte_perm(fg8::cvt_e4m3x2(z[0], z[1]), fg8::cvt_e4m3x2(z[2], z[3]), 0x5410);
            }
            *reinterpret_cast<uint4*>(out + c * a.P) = make_uint4(q[0], q[1], q[2], q[3]);
        }
        if (++st == kStages) st = 0;
        if (++cb == ncb) {
            cb = 0;
            ++tile;
            out = a.xqT + (int64_t)col0 * a.P + 128 * (int64_t)tile + 16 * group;
        } else {
            out += 128 * a.P;
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
    const int64_t most = (R / 128 + E) * (K / 128);
    if (R / 128 + E > INT32_MAX) return FG8_ERR_UNSUPPORTED;
    int64_t grid = (int64_t)kCtasPerSm * fg8h::num_sms();
    if (grid > most) grid = most;
    if (most / grid > INT32_MAX) return FG8_ERR_UNSUPPORTED;
    requant_columns<<<(unsigned)grid, kThreads, kSmemBytes, (cudaStream_t)stream>>>(a);
    return fg8h::launch_status();
}
