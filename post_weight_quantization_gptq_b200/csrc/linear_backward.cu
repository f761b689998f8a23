// What surrounds the gradient product of the layers with an epilogue:
//   slopes   linear  dP = dY * act'(pre),  dbias[n] = sum_t dP[t][n]
//            gated   dG = dY * U * act'(G),  dU = dY * act(G)
//            in fp32 from the saved bf16 pre-activations, rounded to bf16 once
//            (the tensor cores read them as 16-bit operands); the bias sums
//            take the unrounded values.
//   scatter  dX[t][perm[k]] = dXq[t][k], a token row at a time through shared
//            memory, so that HBM sees rows in order on both sides.
// Both are bound by HBM: every value is read and written once.  Bias sums are
// two-step (token slabs, then slabs in order) instead of atomic adds, so that
// they have the same bits every call.
#include "activation.cuh"
#include "common.cuh"
#include "kernels.h"

namespace gptq {
namespace {

constexpr int kCols = 256;      // columns per CTA: 32 lanes x 8
constexpr int kRows = 8;        // token rows in flight per CTA
constexpr int kMaxSlabs = 256;  // token slabs of the bias sums
constexpr int kSlab = 8;        // tokens of one, at least

// Tokens per CTA: kSlab, or as many as leave at most kMaxSlabs slabs.
int64_t slab_tokens(int64_t n_tok) {
    const int64_t least = (n_tok + kMaxSlabs - 1) / kMaxSlabs;
    return least <= kSlab ? kSlab : (least + kRows - 1) / kRows * kRows;
}
int64_t slabs(int64_t n_tok) { return (n_tok + slab_tokens(n_tok) - 1) / slab_tokens(n_tok); }

__device__ __forceinline__ void get8(const uint16_t* p, float (&v)[8], int count) {
    if (count == 8 && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
        const uint4 q = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(w[j] << 16);
            v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < count ? bf16_to_float(p[j]) : 0.f;
    }
}
// dP rows start on 16 bytes and c is a multiple of 8
__device__ __forceinline__ void put8(uint16_t* p, const float (&v)[8], int count) {
    if (count == 8) {
        *reinterpret_cast<uint4*>(p) = make_uint4(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]),
                                                  f32x2_to_bf16x2(v[4], v[5]), f32x2_to_bf16x2(v[6], v[7]));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < count) p[j] = f32_to_bf16_bits(v[j]);
    }
}

// (act(x), act'(x)) of eight values (one branch on the activation).
template <bool VALUE>
__device__ __forceinline__ void slopes8(const float (&x)[8], float (&value)[8], float (&slope)[8], int act) {
    auto each = [&](int which) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            slope[j] = activate_slope(x[j], which);
            if constexpr (VALUE) value[j] = activate(x[j], which);
        }
    };
    switch (act) {
        case GPTQ_ACT_RELU: each(GPTQ_ACT_RELU); break;
        case GPTQ_ACT_GELU: each(GPTQ_ACT_GELU); break;
        case GPTQ_ACT_GELU_TANH: each(GPTQ_ACT_GELU_TANH); break;
        case GPTQ_ACT_SILU: each(GPTQ_ACT_SILU); break;
        default: each(GPTQ_ACT_NONE); break;
    }
}

// The outputs may be the inputs themselves: a thread reads its eight entries
// of all of them before it writes.  A warp takes 256 columns of a token.
__global__ void __launch_bounds__(256) gated_slopes_kernel(const __grid_constant__ BackwardCall c, int chunks) {
    const int lane = threadIdx.x & 31;
    const int64_t total = c.n_tok * chunks;
    for (int64_t e = blockIdx.x * 8ll + (threadIdx.x >> 5); e < total; e += gridDim.x * 8ll) {
        const int64_t t = e / chunks, n = (e - t * chunks) * kCols + 8 * lane;
        const int count = static_cast<int>(c.d_row - n < 8 ? c.d_row - n : 8);
        if (count <= 0) continue;
        float dy[8], g[8], u[8], value[8], slope[8];
        get8(c.dY + t * c.lddy + n, dy, count);
        get8(c.pre[0] + t * c.ldpre[0] + n, g, count);
        get8(c.pre[1] + t * c.ldpre[1] + n, u, count);
        slopes8<true>(g, value, slope, c.act);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            u[j] = dy[j] * u[j] * slope[j];
            g[j] = dy[j] * value[j];
        }
        put8(c.dP[0] + t * c.lddp[0] + n, u, count);
        put8(c.dP[1] + t * c.lddp[1] + n, g, count);
    }
}

// A CTA takes a slab of tokens of 256 columns and leaves the columns' sums.
__global__ void __launch_bounds__(256) slopes_kernel(const __grid_constant__ BackwardCall c, float* bias_part, int64_t slab) {
    __shared__ float sums[kRows][kCols + 8];
    const int lane = threadIdx.x & 31, r = threadIdx.x >> 5;
    const int64_t n = blockIdx.x * static_cast<int64_t>(kCols) + 8 * lane;
    const int count = static_cast<int>(c.d_row - n < 8 ? c.d_row - n : 8);
    const int64_t t1 = (blockIdx.y + 1) * slab < c.n_tok ? (blockIdx.y + 1) * slab : c.n_tok;
    float sum[8] = {};
    if (count > 0) {
#pragma unroll 2
        for (int64_t t = blockIdx.y * slab + r; t < t1; t += kRows) {
            float dy[8];
            get8(c.dY + t * c.lddy + n, dy, count);
            if (c.act != GPTQ_ACT_NONE) {
                float p[8], slope[8];
                get8(c.pre[0] + t * c.ldpre[0] + n, p, count);
                slopes8<false>(p, p, slope, c.act);
#pragma unroll
                for (int j = 0; j < 8; ++j) dy[j] *= slope[j];
            }
            if (c.dP[0] != nullptr) put8(c.dP[0] + t * c.lddp[0] + n, dy, count);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j] += dy[j];
        }
    }
    if (bias_part == nullptr) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) sums[r][8 * lane + j] = sum[j];
    __syncthreads();
    const int64_t col = blockIdx.x * static_cast<int64_t>(kCols) + threadIdx.x;
    if (col < c.d_row) {
        float v = 0.f;
#pragma unroll
        for (int q = 0; q < kRows; ++q) v += sums[q][threadIdx.x];
        bias_part[blockIdx.y * c.d_row + col] = v;
    }
}

// dbias[n] = the slabs' sums: 32 columns per CTA, eight chains of slabs each,
// joined in a fixed order.
__global__ void __launch_bounds__(256) bias_sum_kernel(const float* __restrict__ part, int slabs, int64_t d_row,
                                                       float* __restrict__ dbias) {
    __shared__ float sums[8][32];
    const int col = threadIdx.x & 31, chain = threadIdx.x >> 5;
    const int64_t n = blockIdx.x * 32ll + col;
    float v = 0.f;
    if (n < d_row)
        for (int s = chain; s < slabs; s += 8) v += part[s * d_row + n];
    sums[chain][col] = v;
    __syncthreads();
    if (chain == 0 && n < d_row) {
#pragma unroll
        for (int q = 1; q < 8; ++q) v += sums[q][col];
        dbias[n] = v;
    }
}

constexpr int kScatterThreads = 512;
constexpr int kScatterSmem = 220 * 1024;

// One token row at a time: its values go to their columns in shared memory and
// leave in order.  The permutation is staged once per CTA as 16-bit indices
// (kSmall: d_col <= 65536 and both fit), entries outside [0, d_col) read as k.
template <bool kSmall>
__global__ void __launch_bounds__(kScatterThreads) scatter_kernel(const uint16_t* __restrict__ dXq, int64_t n_tok,
                                                                  int K, const int32_t* __restrict__ perm,
                                                                  uint16_t* __restrict__ dX, int64_t lddx) {
    extern __shared__ __align__(16) uint16_t sm[];
    if constexpr (!kSmall) {
        for (int64_t t = blockIdx.x; t < n_tok; t += gridDim.x)
            for (int k = threadIdx.x; k < K; k += kScatterThreads) {
                int col = __ldg(perm + k);
                if (col < 0 || col >= K) col = k;
                dX[t * lddx + col] = dXq[t * K + k];
            }
        return;
    }
    uint16_t* idx = sm;        // [K]
    uint16_t* row = sm + K;    // [K]
    stage_permutation(idx, perm, K, kScatterThreads);
    for (int k = 8 * threadIdx.x; k < K; k += 8 * kScatterThreads)
        *reinterpret_cast<uint4*>(row + k) = make_uint4(0, 0, 0, 0);
    const int chunks = K / 8;
    for (int64_t t = blockIdx.x; t < n_tok; t += gridDim.x) {
        __syncthreads();   // the row buffer has been written out (first: idx is there)
        const uint4* src = reinterpret_cast<const uint4*>(dXq + t * K);
        for (int c = threadIdx.x; c < chunks; c += kScatterThreads) {
            const uint4 v = src[c], ix = reinterpret_cast<const uint4*>(idx)[c];
            const uint32_t vw[4] = {v.x, v.y, v.z, v.w}, iw[4] = {ix.x, ix.y, ix.z, ix.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                row[iw[j] & 0xFFFFu] = static_cast<uint16_t>(vw[j]);
                row[iw[j] >> 16] = static_cast<uint16_t>(vw[j] >> 16);
            }
        }
        __syncthreads();
        uint16_t* out = dX + t * lddx;
        if ((reinterpret_cast<uintptr_t>(out) & 15) == 0) {
            for (int c = threadIdx.x; c < chunks; c += kScatterThreads)
                reinterpret_cast<uint4*>(out)[c] = reinterpret_cast<const uint4*>(row)[c];
        } else {
            for (int k = threadIdx.x; k < K; k += kScatterThreads) out[k] = row[k];
        }
    }
}

}  // namespace

size_t bias_partial_bytes(int64_t n_tok, int64_t d_row) {
    return static_cast<size_t>(slabs(n_tok)) * d_row * sizeof(float);
}

// The most of any batch of up to n_tok tokens.
size_t most_bias_partial_bytes(int64_t n_tok, int64_t d_row) {
    const int64_t s = (n_tok + kSlab - 1) / kSlab;
    return static_cast<size_t>(s < kMaxSlabs ? s : kMaxSlabs) * d_row * sizeof(float);
}

gptq_status launch_slopes(const BackwardCall& c, float* bias_part, int64_t* launches, cudaStream_t stream) {
    const bool gated = c.mat[1].packed != nullptr;
    if (!gated && c.dP[0] == nullptr && bias_part == nullptr) return GPTQ_OK;   // dY is the gradient
    const int64_t ns = slabs(c.n_tok), chunks = (c.d_row + kCols - 1) / kCols;
    if (gated) {
        const int64_t want = (c.n_tok * chunks + 7) / 8, most = 8 * num_sms();
        gated_slopes_kernel<<<static_cast<unsigned>(want < most ? want : most), 256, 0, stream>>>(
            c, static_cast<int>(chunks));
    } else {
        slopes_kernel<<<dim3(static_cast<unsigned>(chunks), static_cast<unsigned>(ns)), 256, 0, stream>>>(
            c, bias_part, slab_tokens(c.n_tok));
    }
    if (cudaGetLastError() != cudaSuccess) return GPTQ_ERR_CUDA;
    ++*launches;
    if (bias_part != nullptr) {
        bias_sum_kernel<<<static_cast<unsigned>((c.d_row + 31) / 32), 256, 0, stream>>>(
            bias_part, static_cast<int>(ns), c.d_row, c.dbias);
        if (cudaGetLastError() != cudaSuccess) return GPTQ_ERR_CUDA;
        ++*launches;
    }
    return GPTQ_OK;
}

gptq_status launch_scatter(const uint16_t* dXq, int64_t n_tok, int d_col, const int32_t* perm, uint16_t* dX,
                           int64_t lddx, cudaStream_t stream) {
    const size_t smem = static_cast<size_t>(d_col) * 4;
    if (d_col <= 65536 && smem <= kScatterSmem) {
        auto kern = scatter_kernel<true>;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kScatterSmem) != cudaSuccess)
            return GPTQ_ERR_CUDA;
        int per_sm = 0;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kScatterThreads, smem) != cudaSuccess)
            return GPTQ_ERR_CUDA;
        const int64_t resident = static_cast<int64_t>(per_sm > 0 ? per_sm : 1) * num_sms();
        kern<<<static_cast<int>(n_tok < resident ? n_tok : resident), kScatterThreads, smem, stream>>>(
            dXq, n_tok, d_col, perm, dX, lddx);
    } else {
        const int64_t want = 4 * num_sms();
        scatter_kernel<false><<<static_cast<int>(n_tok < want ? n_tok : want), kScatterThreads, 0, stream>>>(
            dXq, n_tok, d_col, perm, dX, lddx);
    }
    return cudaGetLastError() == cudaSuccess ? GPTQ_OK : GPTQ_ERR_CUDA;
}

}  // namespace gptq
