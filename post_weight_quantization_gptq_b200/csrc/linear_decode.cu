// A few tokens through packed layers, with the epilogue of the layer:
//   linear  Y[t][n] = act( sum_k X[t][perm[k]] W[n][k] + bias[n] ) + residual[t][n]
//   gated   Y[t][n] = act( sum_k X[t][perm[k]] Wg[n][k] ) * sum_k X[t][perm[k]] Wu[n][k]
// with W[n][k] = s[k/g][n] (q[n][k] - z[k/g][n]) in fp32, Y rounded once to bf16.
//
// Mathematics.  Per group the scale and zero point leave the sum,
//   sum_k x_k s (q_k - z) = s ( sum_k x_k (c + q_k) - (c + z) sum_k x_k ),
// and c + q_k is built without a conversion: a code's bits ORed into the
// mantissa of bf16 128 (0x4300, one unit per code step) give 128 + q exactly;
// an 8-bit code is two of them, 128 + its low half and 2048 + 16 its high half
// (0x4500, steps of 16).  The sums run on the tensor cores (m16n8k16, 16 weight
// rows by 8 tokens, exact products of bf16 values, fp32 sums), the plain token
// sum through one more tile of ones, whose result lands in the registers that
// need it.  c <= 2176 costs log2(c / |q - z|) bits of the 24, far below the
// output's 8.
//
// Bound: the packed layer is read once for up to 32 tokens, so HBM; below
// about 10 MB the launch and the length of one warp's chain.  Which 16 codes meet in an instruction
// is free as long as X agrees, so a lane reads 32 consecutive codes of a row
// in one or two vector loads (the lanes of a row 128 codes together) and
// needs 7 shift / logic instructions per 8 codes.
//
// Work split: a warp owns 32 weight rows (gated: 16 of each matrix) and every
// kth block of 128 codes; the warps of a CTA, and of a cluster of CTAs, split
// K so that a layer of few rows still fills the GPU.  Partial sums meet in
// shared memory, across the cluster through distributed shared memory, in a
// fixed order (no atomics).  More tokens put more warps on different rows of
// one CTA, which share the tokens' loads in L1.
#include <cooperative_groups.h>

#include "activation.cuh"
#include "common.cuh"
#include "kernels.h"

namespace cg = cooperative_groups;

namespace gptq {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kTiles = 2;            // 16-row weight tiles per warp
constexpr int kBlock = 128;          // codes per row and step of a warp
constexpr int kMaxTok = 32;          // tokens per launch

// How groups lie in a block of 128 codes: a block lies in one group; a group
// is 32 or 64 codes; a group is 8 or 16 codes.
enum GroupMode { kWide, kNarrow, kTiny };

struct Args {
    PackedMatrix mat[2];
    const uint16_t* X;   // quantization order, rows 16-byte aligned
    int64_t ldx;
    int n_tok, K, N, g;
    int64_t words;       // packed words per row
    const float* bias;
    const uint16_t* residual;
    int64_t ldr;
    uint16_t* Y;
    int64_t ldy;
    int act;
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A token row's 16 bytes.  Coherent (the gather before this kernel may still
// run when it starts) and cached in L1 (other warps of the CTA read them too).
__device__ __forceinline__ uint4 load_x(const uint16_t* p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// A lane's 32 consecutive codes of one row (BITS words).
template <int BITS>
__device__ __forceinline__ void load_codes(const uint32_t* p, uint32_t (&w)[BITS]) {
    if constexpr (BITS == 2) {
        const uint2 v = __ldcs(reinterpret_cast<const uint2*>(p));
        w[0] = v.x; w[1] = v.y;
    } else if constexpr (BITS == 3) {
        w[0] = __ldcs(p); w[1] = __ldcs(p + 1); w[2] = __ldcs(p + 2);
    } else {
#pragma unroll
        for (int q = 0; q < BITS / 4; ++q) {
            const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p) + q);
            w[4 * q] = v.x; w[4 * q + 1] = v.y; w[4 * q + 2] = v.z; w[4 * q + 3] = v.w;
        }
    }
}

// Eight consecutive codes (a unit) as the words the pair extraction reads:
// code i's bits at STEP * i of the low half, code i + 4's of the high half
// (8-bit codes keep two words, codes 0..3 and 4..7).
template <int BITS>
struct Unit {
    uint32_t v[BITS == 8 ? 2 : 1];
};

template <int BITS>
__device__ __forceinline__ Unit<BITS> unit_of(const uint32_t (&w)[BITS], int j) {
    Unit<BITS> u;
    if constexpr (BITS == 4) {
        u.v[0] = w[j];
    } else if constexpr (BITS == 2) {
        u.v[0] = __byte_perm(w[j >> 1], 0, (j & 1) ? 0x4342 : 0x4140);
    } else if constexpr (BITS == 3) {
        const uint32_t b = j == 0 ? w[0]
                         : j == 1 ? __funnelshift_r(w[0], w[1], 24)
                         : j == 2 ? __funnelshift_r(w[1], w[2], 16) : (w[2] >> 8);
        u.v[0] = (b & 0xFFFu) | ((b & 0xFFF000u) << 4);
    } else {
        u.v[0] = w[2 * j];
        u.v[1] = w[2 * j + 1];
    }
    return u;
}

// Codes i and i + 4 of the unit as bf16 128 + q (8 bits: 128 + the low half;
// the high half as 2048 + 16 h by pair_high).
template <int BITS>
__device__ __forceinline__ uint32_t pair_low(const Unit<BITS>& u, int i) {
    if constexpr (BITS == 8) {
        const uint32_t p = __byte_perm(u.v[0], u.v[1], 0x0400 + 0x0101 * i);
        return (p & 0x000F000Fu) | 0x43004300u;
    } else {
        constexpr uint32_t kMask = ((1u << BITS) - 1u) * 0x00010001u;
        return ((u.v[0] >> (BITS * i)) & kMask) | 0x43004300u;
    }
}
__device__ __forceinline__ uint32_t pair_high(const Unit<8>& u, int i) {
    const uint32_t p = __byte_perm(u.v[0], u.v[1], 0x0400 + 0x0101 * i);
    return ((p >> 4) & 0x000F000Fu) | 0x45004500u;
}

// Lane t of a quad holds units 4t .. 4t+3; afterwards unit 4j + t for j = 0..3
// (a 4 x 4 transposition across the quad in two exchange steps).
template <int W>
__device__ __forceinline__ void quad_transpose(uint32_t (&v)[4][W], int t) {
#pragma unroll
    for (int x = 0; x < W; ++x) {
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
            const uint32_t send = (t & 1) ? v[j][x] : v[j + 1][x];
            const uint32_t got = __shfl_xor_sync(0xffffffffu, send, 1);
            if (t & 1) v[j][x] = got; else v[j + 1][x] = got;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t send = (t & 2) ? v[j][x] : v[j + 2][x];
            const uint32_t got = __shfl_xor_sync(0xffffffffu, send, 2);
            if (t & 2) v[j][x] = got; else v[j + 2][x] = got;
        }
    }
}

// WR: row groups of a CTA (its other warps split K).  Cluster ranks (y) split K too.
template <int BITS, int MODE, int NT, bool GATED, int WR>
__global__ void __launch_bounds__(kThreads, NT >= 4 || (BITS == 8 && NT >= 2) ? 1 : 2)
    decode_kernel(const Args a) {
    constexpr int WK = kWarps / WR;
    constexpr int kRows = 16 * kTiles * WR;         // weight rows of the CTA
    constexpr int kTok = 8 * NT;
    constexpr int kPitch = kRows + 4;
    constexpr float kOff = BITS == 8 ? 2176.f : 128.f;
    __shared__ float red[WK][kTok][kPitch];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wr = warp % WR, wk = warp / WR;
    const int g8 = lane >> 2, t = lane & 3;
    const int n0 = blockIdx.x * (GATED ? 16 * WR : kRows);   // the CTA's first output
    const int ranks = gridDim.y, rank = blockIdx.y;
    const int nblk = (a.K + kBlock - 1) / kBlock;
    const int step = WK * ranks;

    // the lane's rows: tile m, row g8 and g8 + 8 (clamped: surplus rows are
    // computed from the last row and dropped)
    const uint32_t* base[kTiles][2];
    int row[kTiles][2];
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = GATED ? n0 + 16 * wr + g8 + 8 * h : n0 + 32 * wr + 16 * m + g8 + 8 * h;
            row[m][h] = min(r, a.N - 1);
            base[m][h] = a.mat[GATED ? m : 0].packed + row[m][h] * a.words + t * BITS;
        }

    float acc[kTiles][NT][4];
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
#pragma unroll
        for (int q = 0; q < NT; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][q][i] = 0.f;

    uint32_t nxt[kTiles][2][BITS];
    auto fetch = [&](int b) {
        const bool in = b < nblk && b * kBlock + 32 * t < a.K;
#pragma unroll
        for (int m = 0; m < kTiles; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (in) {
                    load_codes<BITS>(base[m][h] + static_cast<int64_t>(b) * (4 * BITS), nxt[m][h]);
                } else {
#pragma unroll
                    for (int i = 0; i < BITS; ++i) nxt[m][h][i] = 0;
                }
            }
    };
    const int blocks_per_group = a.g / kBlock;   // kWide with more than one group
    int b = rank * WK + wk;
    fetch(b);
    pdl_wait();   // X may come from the gather launched before this kernel

    for (; b < nblk; b += step) {
        uint32_t cur[kTiles][2][BITS];
#pragma unroll
        for (int m = 0; m < kTiles; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < BITS; ++i) cur[m][h][i] = nxt[m][h][i];
        fetch(b + step);

        constexpr int UW = BITS == 8 ? 2 : 1;
        uint32_t un[kTiles][2][4][UW];
#pragma unroll
        for (int m = 0; m < kTiles; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const Unit<BITS> u = unit_of<BITS>(cur[m][h], j);
#pragma unroll
                    for (int x = 0; x < UW; ++x) un[m][h][j][x] = u.v[x];
                }
                if constexpr (MODE != kWide) quad_transpose<UW>(un[m][h], t);
            }

        float c[kTiles][NT][4], cs[NT][4];
        auto clear = [&]() {
#pragma unroll
            for (int q = 0; q < NT; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    cs[q][i] = 0.f;
#pragma unroll
                    for (int m = 0; m < kTiles; ++m) c[m][q][i] = 0.f;
                }
        };
        // the 32 codes that step j of the quad covers; `mask` keeps this
        // lane's codes (all ones) or drops them (a group of 8 or 16 codes)
        auto products = [&](int j, const uint32_t (&xb)[NT][4], uint32_t mask) {
            const uint32_t one = 0x3F803F80u & mask;
#pragma unroll
            for (int m = 0; m < kTiles; ++m) {
                Unit<BITS> u0, u1;
#pragma unroll
                for (int x = 0; x < UW; ++x) {
                    u0.v[x] = un[m][0][j][x];
                    u1.v[x] = un[m][1][j][x];
                }
#pragma unroll
                for (int p = 0; p < 4; p += 2) {
                    const uint32_t a0 = pair_low<BITS>(u0, p) & mask, a1 = pair_low<BITS>(u1, p) & mask;
                    const uint32_t a2 = pair_low<BITS>(u0, p + 1) & mask, a3 = pair_low<BITS>(u1, p + 1) & mask;
#pragma unroll
                    for (int q = 0; q < NT; ++q) mma_bf16(c[m][q], a0, a1, a2, a3, xb[q][p], xb[q][p + 1]);
                    if constexpr (BITS == 8) {
                        const uint32_t h0 = pair_high(u0, p) & mask, h1 = pair_high(u1, p) & mask;
                        const uint32_t h2 = pair_high(u0, p + 1) & mask, h3 = pair_high(u1, p + 1) & mask;
#pragma unroll
                        for (int q = 0; q < NT; ++q) mma_bf16(c[m][q], h0, h1, h2, h3, xb[q][p], xb[q][p + 1]);
                    }
                }
            }
#pragma unroll
            for (int q = 0; q < NT; ++q)
#pragma unroll
                for (int p = 0; p < 4; p += 2) mma_bf16(cs[q], one, one, one, one, xb[q][p], xb[q][p + 1]);
        };
        // the finished group's sums enter the outputs
        auto fold = [&](int group) {
#pragma unroll
            for (int m = 0; m < kTiles; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const PackedMatrix& mt = a.mat[GATED ? m : 0];
                    const int64_t at = static_cast<int64_t>(group) * a.N + row[m][h];
                    const float s = __ldg(mt.scales + at);
                    const float z = kOff + static_cast<float>(__ldg(mt.zeros + at));
#pragma unroll
                    for (int q = 0; q < NT; ++q)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            acc[m][q][2 * h + i] = fmaf(s, fmaf(-z, cs[q][i], c[m][q][2 * h + i]), acc[m][q][2 * h + i]);
                }
        };
        // the tokens' values of step j, paired like the codes
        auto tokens = [&](int j, uint32_t (&xb)[NT][4]) {
            const int k = b * kBlock + 8 * (MODE == kWide ? 4 * t + j : 4 * j + t);
#pragma unroll
            for (int q = 0; q < NT; ++q) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (8 * q + g8 < a.n_tok && k < a.K) v = load_x(a.X + (8 * q + g8) * a.ldx + k);
                xb[q][0] = __byte_perm(v.x, v.z, 0x5410);
                xb[q][1] = __byte_perm(v.x, v.z, 0x7632);
                xb[q][2] = __byte_perm(v.y, v.w, 0x5410);
                xb[q][3] = __byte_perm(v.y, v.w, 0x7632);
            }
        };

        if constexpr (MODE == kWide) {
            clear();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t xb[NT][4];
                tokens(j, xb);
                products(j, xb, 0xffffffffu);
            }
            fold(a.g >= a.K ? 0 : b / blocks_per_group);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = b * kBlock + 32 * j;
                if (k >= a.K) break;   // the same for every lane
                uint32_t xb[NT][4];
                tokens(j, xb);
                if constexpr (MODE == kNarrow) {
                    clear();
                    products(j, xb, 0xffffffffu);
                    fold(k / a.g);
                } else {
                    for (int sub = 0; sub < 32 / a.g; ++sub) {
                        clear();
                        products(j, xb, t * 8 / a.g == sub ? 0xffffffffu : 0u);
                        fold(k / a.g + sub);
                    }
                }
            }
        }
    }

    // ---- partial sums of the K slices: within the CTA, then the cluster
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
#pragma unroll
        for (int q = 0; q < NT; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                red[wk][8 * q + 2 * t + (i & 1)][(wr * kTiles + m) * 16 + g8 + 8 * (i >> 1)] = acc[m][q][i];
    __syncthreads();
    for (int e = threadIdx.x; e < kTok * kRows; e += kThreads) {
        const int tok = e / kRows, r = e % kRows;
        float v = red[0][tok][r];
#pragma unroll
        for (int w = 1; w < WK; ++w) v += red[w][tok][r];
        red[0][tok][r] = v;   // each entry has one owner
    }
    cg::cluster_group cluster = cg::this_cluster();
    if (ranks > 1) cluster.sync(); else __syncthreads();
    constexpr int kOut = GATED ? 16 * WR : kRows;
    for (int e = rank * kThreads + threadIdx.x; e < kTok * kOut; e += ranks * kThreads) {
        const int tok = e / kOut, o = e % kOut, n = n0 + o;
        if (tok >= a.n_tok || n >= a.N) continue;
        // gated: o = 16 wr + r lies in tile (wr, 0), its partner in tile (wr, 1)
        const int r = GATED ? (o >> 4) * 32 + (o & 15) : o;
        float v = 0.f, u = 0.f;
        for (int k = 0; k < ranks; ++k) {
            const float* p = ranks > 1 ? cluster.map_shared_rank(&red[0][tok][r], k) : &red[0][tok][r];
            v += p[0];
            if constexpr (GATED) u += p[16];
        }
        float y;
        if constexpr (GATED) {
            y = activate(v, a.act) * u;
        } else {
            if (a.bias != nullptr) v += a.bias[n];
            y = activate(v, a.act);
            if (a.residual != nullptr)
                y += bf16_to_float(a.residual[tok * a.ldr + n]);
        }
        a.Y[tok * a.ldy + n] = f32_to_bf16_bits(y);
    }
    if (ranks > 1) cluster.sync();   // no CTA leaves while its sums are read
}

// Xq[t][k] = X[t][perm[k]] (perm entries outside [0, K) read as k), 8 values
// per thread; K is a multiple of 8.
__global__ void __launch_bounds__(256) gather_rows_kernel(const uint16_t* __restrict__ X, int64_t ldx,
                                                          int n_tok, int K,
                                                          const int32_t* __restrict__ perm,
                                                          uint16_t* __restrict__ Xq) {
    pdl_trigger();
    const int chunks = K / 8;
    for (int e = blockIdx.x * 256 + threadIdx.x; e < n_tok * chunks; e += gridDim.x * 256) {
        const int tok = e / chunks, c = e - tok * chunks;
        const uint16_t* xr = X + tok * ldx;
        uint32_t v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int k = 8 * c + i;
            int col = perm != nullptr ? __ldg(perm + k) : k;
            if (col < 0 || col >= K) col = k;
            v[i] = __ldg(xr + col);
        }
        reinterpret_cast<uint4*>(Xq + static_cast<int64_t>(tok) * K)[c] =
            make_uint4(v[0] | (v[1] << 16), v[2] | (v[3] << 16), v[4] | (v[5] << 16), v[6] | (v[7] << 16));
    }
}

template <int BITS, int MODE, int NT, bool GATED, int WR>
cudaError_t launch_one(const Args& a, bool pdl, cudaStream_t stream) {
    const int per = (GATED ? 16 : 32) * WR;
    const int tiles = (a.N + per - 1) / per;
    const int nblk = (a.K + kBlock - 1) / kBlock;
    // split K over a cluster while there are fewer than two CTAs per SM and a
    // warp keeps at least two blocks
    int ranks = 1;
    while (ranks < 8 && tiles * ranks < 2 * num_sms() && nblk >= 4 * ranks * (kWarps / WR)) ranks *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(tiles, ranks);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (ranks > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim = {1, static_cast<unsigned>(ranks), 1};
        ++n;
    }
    if (pdl) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, decode_kernel<BITS, MODE, NT, GATED, WR>, a);
}

template <int BITS, int MODE, bool GATED>
cudaError_t launch_tokens(const Args& a, bool pdl, cudaStream_t stream) {
    if (a.n_tok <= 8) return launch_one<BITS, MODE, 1, GATED, 1>(a, pdl, stream);
    if (a.n_tok <= 16) return launch_one<BITS, MODE, 2, GATED, 2>(a, pdl, stream);
    return launch_one<BITS, MODE, 4, GATED, 4>(a, pdl, stream);
}

template <int BITS, bool GATED>
cudaError_t launch_mode(const Args& a, bool pdl, cudaStream_t stream) {
    if (a.g >= a.K || a.g % kBlock == 0) return launch_tokens<BITS, kWide, GATED>(a, pdl, stream);
    if (a.g >= 32) return launch_tokens<BITS, kNarrow, GATED>(a, pdl, stream);
    return launch_tokens<BITS, kTiny, GATED>(a, pdl, stream);
}

template <bool GATED>
cudaError_t launch_bits(const Args& a, int bits, bool pdl, cudaStream_t stream) {
    switch (bits) {
        case 2: return launch_mode<2, GATED>(a, pdl, stream);
        case 3: return launch_mode<3, GATED>(a, pdl, stream);
        case 4: return launch_mode<4, GATED>(a, pdl, stream);
        default: return launch_mode<8, GATED>(a, pdl, stream);
    }
}

}  // namespace

size_t linear_decode_workspace_bytes(int64_t n_tok, int64_t d_col) {
    const int64_t t = n_tok < kMaxTok ? n_tok : kMaxTok;
    return ((static_cast<size_t>(t) * d_col * 2 + 255) / 256) * 256;
}

gptq_status launch_linear_decode(const LinearCall& c, cudaStream_t stream) {
    const bool gated = c.mat[1].packed != nullptr;
    const bool gather = needs_gather(c.X, c.ldx, c.perm);
    Args a = {};
    a.mat[0] = c.mat[0];
    a.mat[1] = c.mat[1];
    a.K = static_cast<int>(c.d_col);
    a.N = static_cast<int>(c.d_row);
    a.g = (c.group == -1 || c.group > a.K) ? a.K : c.group;
    a.words = c.d_col * c.bits / 32;
    a.bias = c.bias;
    a.ldr = c.ldr;
    a.ldy = c.ldy;
    a.act = c.act;
    int64_t launches = 0;
    for (int64_t t0 = 0; t0 < c.n_tok; t0 += kMaxTok) {
        a.n_tok = static_cast<int>(c.n_tok - t0 < kMaxTok ? c.n_tok - t0 : kMaxTok);
        a.X = c.X + t0 * c.ldx;
        a.ldx = c.ldx;
        if (gather) {
            uint16_t* xq = static_cast<uint16_t*>(c.ws);
            const int64_t work = (static_cast<int64_t>(a.n_tok) * (a.K / 8) + 255) / 256;
            const int blocks = static_cast<int>(work < 8 * num_sms() ? work : 8 * num_sms());
            gather_rows_kernel<<<blocks, 256, 0, stream>>>(a.X, a.ldx, a.n_tok, a.K, c.perm, xq);
            if (cudaGetLastError() != cudaSuccess) return GPTQ_ERR_CUDA;
            a.X = xq;
            a.ldx = c.d_col;
            ++launches;
        }
        a.residual = c.residual == nullptr ? nullptr : c.residual + t0 * c.ldr;
        a.Y = c.Y + t0 * c.ldy;
        const cudaError_t e = gated ? launch_bits<true>(a, c.bits, gather, stream)
                                    : launch_bits<false>(a, c.bits, gather, stream);
        if (e != cudaSuccess) return GPTQ_ERR_CUDA;
        ++launches;
    }
    count_launches(launches);
    return GPTQ_OK;
}

}  // namespace gptq
