// gate.cu -- the combine's gate weights per routed row, and the router's gradient.
//
// Forward (fg8_unpermute_combine's weights, DeepSeek-V3 summary sec. 2.1): a
// token's kept slots have affinities a_j with sum S, and weights w_j = a_j / S
// (normalize) or a_j.  Backward: with g_j = dL/dw_j,
//     dL/da_j = (g_j - sum_i w_i g_i) / S          (normalize; 0 where S = 0)
//             = g_j                                 (otherwise)
// and, since a_j = sigmoid(u[id_j]), dL/du[id_j] += dL/da_j * a_j (1 - a_j);
// the selection itself and the selection bias have no gradient.
//
// Both are bound by launch and load latency (8192 tokens x 8 slots: 0.26 MB of
// maps, 4 MB of partial dots, 8 MB of logit gradients).  A token is held by a
// group of KG lanes (a power of two >= k), one slot a lane, so the loads of all
// slots are in flight together; the ordered sums run over shuffles, which keeps
// the slot order of fg8_unpermute_combine (bit-equal weights) and makes the
// results independent of the launch shape.  Both calls together take 8.5 us on a
// B200 for those 8192 tokens (256 experts, 16 blocks of dots; 14 MB of data, 2.2 us
// at the copy rate) and 4.6 us for 333 tokens x 6 slots: two launches and the
// dependent loads map -> dots.  With KG = 16 for every k: 9.9 and 4.8 us.
#include <type_traits>

#include "fg8_common.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kMaxSlots = 16;
constexpr unsigned kFull = 0xffffffffu;

// sum over the group's kept slots in slot order, the same value in every lane
template <int KG>
FG8_DEV float ordered_sum(float v, bool kept, int k) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < KG; ++j) {
        const float vj = __shfl_sync(kFull, v, j, KG);
        const bool kj = __shfl_sync(kFull, (int)kept, j, KG) != 0;
        if (j < k && kj) s = __fadd_rn(s, vj);
    }
    return s;
}

template <int KG>
__global__ void __launch_bounds__(kThreads)
gate_weights(const int32_t* __restrict__ token_row, const float* __restrict__ affinity, int64_t T,
             int k, int normalize, int64_t R, float* __restrict__ row_w) {
    const int64_t gt = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / KG;   // token
    const int j = threadIdx.x & (KG - 1);
    int32_t row = -1;
    float a = 0.f;
    if (gt < T && j < k) {
        row = token_row[gt * k + j];
        a = affinity[gt * k + j];
    }
    const bool kept = row >= 0 && row < R;
    const float sum = ordered_sum<KG>(a, kept, k);
    if (kept) row_w[row] = !normalize ? a : (sum != 0.f ? __fdiv_rn(a, sum) : 0.f);
}

template <int KG>
__global__ void __launch_bounds__(kThreads)
gate_backward(const float* __restrict__ dot, int nb, int64_t R, const int32_t* __restrict__ token_row,
              const int32_t* __restrict__ ids, const float* __restrict__ affinity, int64_t T, int k,
              int E, int normalize, float* __restrict__ daff, float* __restrict__ dlogits) {
    const int64_t gt = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / KG;
    const int lane = threadIdx.x & 31, j = lane & (KG - 1);
    const bool slot = gt < T && j < k;
    int32_t row = -1, id = -1;
    float a = 0.f;
    if (slot) {
        row = token_row[gt * k + j];
        a = affinity[gt * k + j];
        if (dlogits) id = ids[gt * k + j];
    }
    if (dlogits) {
        // this warp's token rows of dlogits are one contiguous range: zeros
        // first (while the loads above are in flight), the slots' values after
        // the warp barrier below
        const int64_t t0 = ((int64_t)blockIdx.x * kThreads + (threadIdx.x & ~31)) / KG;
        const int64_t t1 = min(T, t0 + 32 / KG);
        if (t0 < t1) {
            float* p = dlogits + t0 * E;
            const int64_t n = (t1 - t0) * E;
            const int64_t head = min(n, (int64_t)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / 4);
            if (lane < head) p[lane] = 0.f;
            const int64_t n4 = (n - head) / 4;
            float4* p4 = reinterpret_cast<float4*>(p + head);
            for (int64_t i = lane; i < n4; i += 32) p4[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            const int64_t tail = head + 4 * n4;
            if (lane < n - tail) p[tail + lane] = 0.f;
        }
    }
    const bool kept = row >= 0 && row < R;
    float g = 0.f;
    if (kept) {
        const float* d = dot + row;
        int b = 0;
        for (; b + 8 <= nb; b += 8) {   // eight loads in flight, added in block order
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __ldg(d + (int64_t)(b + i) * R);
#pragma unroll
            for (int i = 0; i < 8; ++i) g += v[i];
        }
        for (; b < nb; ++b) g += __ldg(d + (int64_t)b * R);
    }
    float da = g;
    if (normalize) {
        const float sum = ordered_sum<KG>(a, kept, k);
        const float w = sum != 0.f ? __fdiv_rn(a, sum) : 0.f;
        const float mean = ordered_sum<KG>(w * g, kept, k);
        da = sum != 0.f ? __fdiv_rn(g - mean, sum) : 0.f;
    }
    if (!kept) da = 0.f;
    if (slot) daff[gt * k + j] = da;
    if (dlogits) {
        __syncwarp();   // the zeros are in place
        const float v = kept ? da * (a * (1.0f - a)) : 0.f;   // a dropped slot's affinity may be anything
        // an expert named by several slots gets their sum, in slot order, from the first of them
        float total = 0.f;
        bool first = true;
#pragma unroll
        for (int i = 0; i < KG; ++i) {
            const float vi = __shfl_sync(kFull, v, i, KG);
            const int32_t ii = __shfl_sync(kFull, id, i, KG);
            if (i < k && ii == id) {
                total += vi;
                if (i < j) first = false;
            }
        }
        if (slot && first && id >= 0 && id < E) dlogits[gt * E + id] = total;
    }
}

template <class F>
fg8_status by_slots(int k, F go) {
    if (k <= 1) return go(std::integral_constant<int, 1>());
    if (k <= 2) return go(std::integral_constant<int, 2>());
    if (k <= 4) return go(std::integral_constant<int, 4>());
    if (k <= 8) return go(std::integral_constant<int, 8>());
    return go(std::integral_constant<int, 16>());
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

}  // namespace

extern "C" fg8_status fg8_gate_weights(const int32_t* token_row, const float* affinity, int64_t T,
                                       int k, int normalize, int64_t R, float* row_w,
                                       fg8_stream_t stream) {
    if (T < 0 || R < 0 || k < 1 || k > kMaxSlots || (normalize != 0 && normalize != 1))
        return FG8_ERR_INVALID_ARG;
    if (T == 0 || R == 0) return FG8_OK;
    if (!token_row || !affinity || !row_w) return FG8_ERR_INVALID_ARG;
    if (!aligned4(token_row) || !aligned4(affinity) || !aligned4(row_w)) return FG8_ERR_INVALID_ARG;
    if (R > INT32_MAX || T > INT32_MAX / k) return FG8_ERR_UNSUPPORTED;
    return by_slots(k, [&](auto kg) {
        constexpr int KG = decltype(kg)::value;
        const int64_t grid = (T * KG + kThreads - 1) / kThreads;
        gate_weights<KG><<<(unsigned)grid, kThreads, 0, (cudaStream_t)stream>>>(token_row, affinity, T, k,
                                                                               normalize, R, row_w);
        return fg8h::launch_status();
    });
}

extern "C" fg8_status fg8_gate_backward(const float* gate_dot, int nb, int64_t R,
                                        const int32_t* token_row, const int32_t* topk_ids,
                                        const float* affinity, int64_t T, int k, int E, int normalize,
                                        float* daffinity, float* dlogits, fg8_stream_t stream) {
    if (T < 0 || R < 0 || nb < 1 || E < 1 || k < 1 || k > kMaxSlots || (normalize != 0 && normalize != 1))
        return FG8_ERR_INVALID_ARG;
    if (T == 0) return FG8_OK;
    if (!token_row || !affinity || !daffinity || (R > 0 && !gate_dot) || (dlogits && !topk_ids))
        return FG8_ERR_INVALID_ARG;
    if (!aligned4(gate_dot) || !aligned4(token_row) || !aligned4(topk_ids) || !aligned4(affinity) ||
        !aligned4(daffinity) || !aligned4(dlogits))
        return FG8_ERR_INVALID_ARG;
    if (R > INT32_MAX || T > INT32_MAX / k) return FG8_ERR_UNSUPPORTED;
    return by_slots(k, [&](auto kg) {
        constexpr int KG = decltype(kg)::value;
        const int64_t grid = (T * KG + kThreads - 1) / kThreads;
        gate_backward<KG><<<(unsigned)grid, kThreads, 0, (cudaStream_t)stream>>>(
            gate_dot, nb, R, token_row, topk_ids, affinity, T, k, E, normalize, daffinity, dlogits);
        return fg8h::launch_status();
    });
}
