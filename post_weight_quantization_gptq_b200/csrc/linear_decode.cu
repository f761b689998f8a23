// A few tokens through packed layers, with the epilogue of the layer:
//   linear  Y[t][n] = act( sum_k X[t][perm[k]] W[n][k] + bias[n] ) + residual[t][n]
//   gated   Y[t][n] = act( sum_k X[t][perm[k]] Wg[n][k] ) * sum_k X[t][perm[k]] Wu[n][k]
// with W[n][k] = s[k/g][n] (q[n][k] - z[k/g][n]) in fp32, Y rounded once to bf16.
//
// Mathematics.  Per group the scale and zero point leave the sum,
//   sum_k x_k s (q_k - z) = s ( sum_k x_k q_k - z sum_k x_k ),
// and a code needs no conversion: the bf16 bit patterns 0 .. 255 are the
// numbers p 2^-133 (subnormal, then the first binade, evenly spaced), so a
// code masked out of its word, wherever in the low byte of a half word it
// lies, is q 2^(j - 133) for its bit position j.  The tokens are multiplied by
// 2^(64 - j) to match (exact), which keeps a group's two sums, 2^-69 of their
// value, in fp32's normal range; they are scaled back before s enters, so that
// the outputs' sums have fp32's whole range (scaled back at the end, results
// below 2^-57 lost bits to fp32's subnormal range).  The sums run on the tensor
// cores (m16n8k16, 16 weight rows by 8 tokens, exact products, fp32 sums), the
// plain token sum through one more tile whose codes are all 1, so that it lands
// in the registers that need it.  Tokens of magnitude 2^64 and more may
// overflow; below 2^-57 the products x q and x z lose relative precision (2^-80
// absolute, times s).
//
// Bound: the packed layer is read once for up to 32 tokens, so HBM; below
// about 10 MB the launch and the length of one warp's chain.  A large layer
// saturates no unit (8192 x 16384, one token: 40 % of HBM, 49 % of the issue
// slots and of the ALU pipe while the SMs are busy, which is three quarters of
// the time): what is left is few warps per SM, CTAs that do not fill the last
// round, and the first loads and joins at its ends.  Instructions per code still
// count.  Which 16 codes meet in an instruction is free as long as the tokens
// agree, so a lane takes 8 consecutive codes of two rows and masks them out with
// 5 shift / logic instructions (7 where each pair is brought to the low bits and
// completed to 128 + q); weights and tokens arrive by TMA, which costs the warps
// nothing (per-thread asynchronous copies took 258 of 448 instructions per 4096
// codes).
//
// Work split: a warp owns 16 MT weight rows (gated: half of them of each
// matrix) and every kth block of 128 codes, with a ring of blocks of its own in
// shared memory that its lane 0 refills -- no barrier between warps, no
// producer.  The warps of a CTA, and of a cluster of CTAs, split K so that a
// layer of few rows still fills the GPU.  Partial sums meet in shared memory,
// across the cluster through distributed shared memory, in a fixed order (no
// atomics).  Every wait is bounded (GPTQ_ERR_TIMEOUT).
#include <cuda.h>
#include <cooperative_groups.h>

#include "activation.cuh"
#include "common.cuh"
#include "f32x2.cuh"
#include "kernels.h"

namespace cg = cooperative_groups;

namespace gptq {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kBlock = 128;          // codes per row and step of a warp
constexpr int kMaxTok = 32;          // tokens per launch
constexpr int kMaxDepth = 8;         // blocks of a warp's ring
// Shared memory of two and of one CTA per SM: all of the 228 KB less 1 KB for
// each CTA.  (With 112 KB the rings of groups of 64 at five to eight tokens missed two
// blocks by 1 KB and ran with one CTA: 8192 x 8192 34.9 us, now 17.1.)
constexpr int kSmemTwo = 113 * 1024, kSmemOne = kMaxDynamicSmem;

// How groups lie in a block of 128 codes: a block lies in one group; a group
// is 32 or 64 codes; a group is 8 or 16 codes.
enum GroupMode { kWide, kNarrow, kTiny };

struct Args {
    PackedMatrix mat[2];
    int n_tok, K, N, g;
    const float* bias;
    const uint16_t* residual;
    int64_t ldr;
    uint16_t* Y;
    int64_t ldy;
    int act;
    int gathered;            // the tokens are written by the kernel launched just before
    int depth;               // blocks of the ring
    int slot_bytes;          // of one: weights, then tokens
    int red_at;              // where the partial sums lie in shared memory, after the rings
    int ngb_log2;            // groups per block (kNarrow, kTiny)
    int blocks_per_group;    // (kWide)
    uint32_t group_magic;    // block / blocks_per_group = high word of block * group_magic; 0: divide
    int32_t* status;
    uint64_t probe_ns;
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight consecutive codes (a unit): one word, two at 8 bits.  The words of
// three and two bits hold codes 0..3 from bit 0 and codes 4..7 from bit 16.
template <int BITS>
struct Unit {
    uint32_t v[BITS == 8 ? 2 : 1];
};

// Where unit 4j + t lies in the 128 codes of a row: a byte offset from the
// start of row 0 of an 8-row group (16 BITS bytes per row, groups on 1024-byte
// boundaries or, at 3 bits, anywhere).  The copy's swizzle permutes a row's
// 16-byte pieces by its number, so that the 32 lanes' reads (rows g8 = 0..7,
// t = 0..3) meet 32 banks.
template <int BITS>
__device__ __forceinline__ uint32_t unit_offset(int j, int g8, int t) {
    if constexpr (BITS == 4) return g8 * 64 + ((j ^ (g8 >> 1)) << 4) + 4 * t;                        // 64-byte swizzle
    else if constexpr (BITS == 2) return g8 * 32 + (((j >> 1) ^ (g8 >> 2)) << 4) + 8 * (j & 1) + 2 * t;  // 32-byte
    else if constexpr (BITS == 3) return g8 * 48 + 12 * j + 4 * ((3 * t) >> 2);                      // none
    else return g8 * 128 + (((2 * j + (t >> 1)) ^ g8) << 4) + 8 * (t & 1);                           // 128-byte
}
template <int BITS>
__device__ __forceinline__ Unit<BITS> load_unit(const uint8_t* at, int t) {
    Unit<BITS> u;
    if constexpr (BITS == 4) {
        u.v[0] = *reinterpret_cast<const uint32_t*>(at);
    } else if constexpr (BITS == 2) {
        u.v[0] = __byte_perm(*reinterpret_cast<const uint16_t*>(at), 0, 0x4140);
    } else if constexpr (BITS == 3) {   // 24 bits of two words (the fourth unit: of one)
        const uint32_t* w = reinterpret_cast<const uint32_t*>(at);
        const uint32_t v = __funnelshift_r(w[0], w[t == 3 ? 0 : 1], (24 * t) & 31);
        u.v[0] = __byte_perm(v, v << 4, 0x7610);
    } else {
        const uint2 v = *reinterpret_cast<const uint2*>(at);
        u.v[0] = v.x;
        u.v[1] = v.y;
    }
    return u;
}

// The unit's codes as four words of two bf16 patterns: word i holds codes i and
// i + 4 (8 bits: words 0, 1 codes 0 | 2 and 1 | 3, words 2, 3 codes 4 | 6 and
// 5 | 7), at bit position shift_of(i) of the half words.
template <int BITS>
__device__ __forceinline__ uint32_t pair_of(const Unit<BITS>& u, int i) {
    if constexpr (BITS == 8) {
        return (i & 1) ? __byte_perm(u.v[i >> 1], 0, 0x4341) : (u.v[i >> 1] & 0x00FF00FFu);
    } else if constexpr (BITS == 2) {
        return u.v[0] & (0x00030003u << (2 * i));
    } else {
        // two codes fit the low byte: the upper pairs after one shift
        const uint32_t v = i < 2 ? u.v[0] : u.v[0] >> (2 * BITS);
        return v & (((1u << BITS) - 1u) * 0x00010001u << (i & 1 ? BITS : 0));
    }
}
template <int BITS>
__host__ __device__ constexpr int shift_of(int i) {
    return BITS == 8 ? 0 : BITS == 2 ? 2 * i : (i & 1) * BITS;
}
// 2^e as a pair of bf16
__host__ __device__ constexpr uint32_t bf16x2_pow2(int e) { return static_cast<uint32_t>(127 + e) << 7 | static_cast<uint32_t>(127 + e) << 23; }
constexpr int kScaleUp = 64;                 // of the tokens
constexpr float kScaleBack = 0x1p69f;        // 2^(133 - 64)

// Eight consecutive token values as the four words that meet the unit's.
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <int BITS>
__device__ __forceinline__ void token_pairs(uint4 v, uint32_t (&x)[4]) {
    if constexpr (BITS == 8) {
        x[0] = __byte_perm(v.x, v.y, 0x5410);
        x[1] = __byte_perm(v.x, v.y, 0x7632);
        x[2] = __byte_perm(v.z, v.w, 0x5410);
        x[3] = __byte_perm(v.z, v.w, 0x7632);
    } else {
        x[0] = __byte_perm(v.x, v.z, 0x5410);
        x[1] = __byte_perm(v.x, v.z, 0x7632);
        x[2] = __byte_perm(v.y, v.w, 0x5410);
        x[3] = __byte_perm(v.y, v.w, 0x7632);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = mul_bf16x2(x[i], bf16x2_pow2(kScaleUp - shift_of<BITS>(i)));
}

__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the newest n groups of this thread have landed
__device__ __forceinline__ void cp_wait(int n) {
    switch (n) {
        case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
        case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
        case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
        case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
        case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
        case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
        case 6: asm volatile("cp.async.wait_group 6;" ::: "memory"); break;
        default: asm volatile("cp.async.wait_group 7;" ::: "memory"); break;
    }
}

// NT tiles of 8 tokens, MT tiles of 16 weight rows per warp.
template <int BITS, int NT, int MT>
struct Shape {
    static constexpr int kRows = 16 * MT;                    // weight rows of the CTA
    static constexpr int kRowBytes = 16 * BITS;              // 128 codes
    static constexpr int kWBytes = kRows * kRowBytes;        // of a block
    static constexpr int kPitch = kRows + 4;                 // of the partial sums
    static constexpr int kHead = 1024;                       // barriers
};

template <int BITS, int MODE, int NT, int MT, bool GATED>
__global__ void __launch_bounds__(kThreads, NT * MT >= 8 ? 1 : 2)
    decode_kernel(const __grid_constant__ CUtensorMap tmw0, const __grid_constant__ CUtensorMap tmw1,
                  const __grid_constant__ CUtensorMap tmx, const __grid_constant__ Args a) {
    using S = Shape<BITS, NT, MT>;
    constexpr int kRows = S::kRows;
    constexpr int kTilesM = GATED ? MT / 2 : MT;             // tiles of one matrix
    constexpr int kOut = 16 * kTilesM;                       // outputs of the CTA
    extern __shared__ __align__(1024) uint8_t sm[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm);        // [kWarps][kMaxDepth]
    uint64_t* never = bars + kWarps * kMaxDepth;             // (timeout probe)
    int* abort_word = reinterpret_cast<int*>(never + 1);
    int* stopped = abort_word + 1;                           // [kWarps]: lane 0's first block that did not come
    volatile int* abort = abort_word;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g8 = lane >> 2, t = lane & 3;
    const int ranks = gridDim.y, rank = blockIdx.y;
    const int nblk = (a.K + kBlock - 1) / kBlock;
    const int first = rank * kWarps + warp, stride = ranks * kWarps;
    const int steps = nblk > first ? (nblk - first + stride - 1) / stride : 0;   // blocks of this warp, per tile
    const int tiles = (a.N + kOut - 1) / kOut;               // the CTA's: blockIdx.x, + gridDim.x, ...
    const int mine = (tiles - static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
    const int items = mine * steps;                          // blocks of this warp in all
    const int depth = a.depth;
    const int ngb_log2 = MODE == kWide ? 0 : a.ngb_log2;     // groups per block
    const int groups = (a.K + a.g - 1) / a.g;
    uint64_t* full = bars + warp * kMaxDepth;
    const int half_bytes = a.n_tok * 128;                    // 64 codes of the tokens
    const uint8_t* ring_p = sm + S::kHead + warp * depth * a.slot_bytes;
    const uint32_t ring = smem_u32(ring_p);
    const int sc_bytes = 2 * kRows * 4 << ngb_log2;          // a block's scales, then zero points
    uint8_t* sc_ring = sm + S::kHead + kWarps * depth * a.slot_bytes + warp * depth * sc_bytes;

    // The ring runs on through the CTA's tiles: (next_s, next_n0) is the block to
    // load next, of the tile of outputs from next_n0 on.
    int next_s = 0, next_n0 = blockIdx.x * kOut;
    // lane 0: a block's weights, and its tokens
    auto load_weights = [&](int s, int n0, int slot) {
        const int x = (first + s * stride) * (4 * BITS);
        const uint32_t dst = ring + slot * a.slot_bytes;
        mbar_arrive_expect_tx(&full[slot], S::kWBytes + 2 * half_bytes);
        if constexpr (GATED) {
            tma_load_2d_at(dst, &tmw0, &full[slot], x, n0);
            tma_load_2d_at(dst + S::kWBytes / 2, &tmw1, &full[slot], x, n0);
        } else {
            tma_load_2d_at(dst, &tmw0, &full[slot], x, n0);
        }
    };
    auto load_tokens = [&](int s, int slot) {
        const int x = (first + s * stride) * kBlock;
        const uint32_t dst = ring + slot * a.slot_bytes + S::kWBytes;
        tma_load_2d_at(dst, &tmx, &full[slot], x, 0);
        tma_load_2d_at(dst + half_bytes, &tmx, &full[slot], x + 64, 0);
    };
    // the warp: the scales and zero points of a block's groups, [group][row]
    // (4 bytes each: their rows in memory have any alignment)
    constexpr int kOwn = (kRows + 31) / 32;                  // rows per lane
    const float* sc_src[kOwn];
    int64_t z_off[kOwn];                                     // bytes from there to the zero point
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        const int r = lane + 32 * i;
        const PackedMatrix& m = a.mat[GATED && r >= kOut ? 1 : 0];
        sc_src[i] = m.scales + r % kOut;
        z_off[i] = reinterpret_cast<const char*>(m.zeros) - reinterpret_cast<const char*>(m.scales);
    }
    auto load_scales = [&](int s, int n0, int slot) {
        const int b = first + s * stride;
        const uint32_t dst = smem_u32(sc_ring) + slot * sc_bytes + 4 * lane;
        for (int q = 0; q < (1 << ngb_log2); ++q) {
            // kWide: block / blocks per group, as a multiplication where that is exact
            const int gi = MODE != kWide ? (b << ngb_log2) + q
                         : a.group_magic != 0 ? static_cast<int>(__umulhi(b, a.group_magic)) : b / a.blocks_per_group;
            const int64_t off = static_cast<int64_t>(gi) * a.N + n0;
#pragma unroll
            for (int i = 0; i < kOwn; ++i) {
                const bool in = n0 + (lane + 32 * i) % kOut < a.N && gi < groups;
                const char* src = reinterpret_cast<const char*>(in ? sc_src[i] + off : a.mat[0].scales);
                if (kRows % 32 == 0 || lane + 32 * i < kRows) {
                    cp4(dst + 4 * (q * kRows + 32 * i), src, in);
                    cp4(dst + 4 * (q * kRows + 32 * i) + sc_bytes / 2, in ? src + z_off[i] : src, in);
                }
            }
        }
    };

    if (lane == 0) {
        for (int d = 0; d < depth; ++d) mbar_init(&full[d], 1);
        stopped[warp] = 0;
        if (warp == 0) {
            mbar_init(never, 1);
            *abort_word = 0;
        }
        fence_barrier_init();
        fence_async_smem();
        if (warp == 0) {
            tma_prefetch_desc(&tmw0);
            tma_prefetch_desc(&tmx);
        }
    }
    // a warp's barriers are its own: its copies need not wait for the others
    auto advance = [&]() {
        if (++next_s == steps) {
            next_s = 0;
            next_n0 += gridDim.x * kOut;
        }
    };
    const int ahead = min(depth, items);
    for (int d = 0; d < depth; ++d) {
        if (d < ahead) {
            if (lane == 0) {
                load_weights(next_s, next_n0, d);
                if (!a.gathered) load_tokens(next_s, d);
            }
            load_scales(next_s, next_n0, d);
            advance();
        }
        cp_commit();
    }
    if (a.gathered) {
        pdl_wait();   // the tokens come from the kernel before; weights and scales do not
        if (lane == 0)
            for (int d = 0; d < ahead; ++d) load_tokens(d % steps, d);
    }
    __syncthreads();   // the abort word is set up

    float acc[MT][NT][4];

    // Where a lane reads in a slot (slots lie on 1024-byte boundaries).  Column
    // g8 of a token tile stands for token (g8 >> 1) | (g8 & 1) << 2, so that
    // neighbouring columns are four rows apart, which the copy's 128-byte
    // swizzle puts half the banks away; a column past the last token repeats
    // that and is dropped.
    uint32_t w_off[4], x_off[NT][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        w_off[j] = unit_offset<BITS>(j, g8, t);
#pragma unroll
        for (int q = 0; q < NT; ++q) {
            const int tok = min(8 * q + ((g8 >> 1) | (g8 & 1) << 2), a.n_tok - 1);
            const uint32_t at = S::kWBytes + (j >> 1) * half_bytes + tok * 128;
            x_off[q][j] = at + (((4 * (j & 1) + t) ^ ((at >> 7) & 7)) << 4);
        }
    }

    int slot = 0;
    uint32_t phase = 0;
    bool ok = true;
    int done = 0;   // blocks consumed
    if (a.probe_ns != 0 && warp == 0) ok = wait_probe(never, a.probe_ns, abort);
    float* red = reinterpret_cast<float*>(sm + a.red_at);    // [kWarps][n_tok][kPitch]
    cg::cluster_group cluster = cg::this_cluster();
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int n0 = tile * kOut;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int q = 0; q < NT; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][q][i] = 0.f;
    for (int s = 0; s < steps; ++s, ++done) {
        // a lane whose wait runs out stays with its warp, whatever it then reads
        if (ok && !mbar_wait_short(&full[slot], phase, abort)) {
            ok = false;
            if (lane == 0) stopped[warp] = done;
        }
        cp_wait(depth - 1);
        __syncwarp();
        const int b = first + s * stride;
        const uint8_t* at = ring_p + slot * a.slot_bytes;

        // c += the 32 codes of step j of tile m times the tokens; `mask` keeps
        // this lane's codes (all ones) or drops them (a group of 8 or 16 codes)
        auto units = [&](int m, int j, Unit<BITS> (&u)[2]) {
            u[0] = load_unit<BITS>(at + w_off[j] + 16 * m * S::kRowBytes, t);
            u[1] = load_unit<BITS>(at + w_off[j] + (16 * m + 8) * S::kRowBytes, t);
        };
        auto product = [&](const Unit<BITS> (&u)[2], const uint32_t (&xb)[NT][4], uint32_t mask, float (&c)[NT][4]) {
#pragma unroll
            for (int p = 0; p < 4; p += 2) {
                const uint32_t a0 = pair_of<BITS>(u[0], p) & mask, a1 = pair_of<BITS>(u[1], p) & mask;
                const uint32_t a2 = pair_of<BITS>(u[0], p + 1) & mask, a3 = pair_of<BITS>(u[1], p + 1) & mask;
#pragma unroll
                for (int q = 0; q < NT; ++q) mma_bf16(c[q], a0, a1, a2, a3, xb[q][p], xb[q][p + 1]);
            }
        };
        // the same with codes of 1
        auto total = [&](const uint32_t (&xb)[NT][4], uint32_t mask, float (&c)[NT][4]) {
#pragma unroll
            for (int p = 0; p < 4; p += 2) {
                const uint32_t o0 = (0x00010001u << shift_of<BITS>(p)) & mask;
                const uint32_t o1 = (0x00010001u << shift_of<BITS>(p + 1)) & mask;
#pragma unroll
                for (int q = 0; q < NT; ++q) mma_bf16(c[q], o0, o0, o1, o1, xb[q][p], xb[q][p + 1]);
            }
        };
        auto clear = [&](float (&c)[NT][4]) {
#pragma unroll
            for (int q = 0; q < NT; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i) c[q][i] = 0.f;
        };
        // the finished sums of tile m and the block's group enter the outputs, two
        // tokens at a time: sum - z total, scaled back (exact), times s (in scalar
        // instructions the scaling cost 8192 x 8192 with groups of 32 6 % at 32
        // tokens; packed, 3 %)
        const float* sc = reinterpret_cast<const float*>(sc_ring + slot * sc_bytes) + g8;
        const int32_t* zc = reinterpret_cast<const int32_t*>(sc) + (kRows << ngb_log2);
        auto fold = [&](int m, int grp, const float (&c)[NT][4], const float (&cs)[NT][4]) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float sv = sc[grp * kRows + m * 16 + 8 * h];
                const float z = -static_cast<float>(zc[grp * kRows + m * 16 + 8 * h]);
                const uint64_t s2 = pk2(sv, sv), z2 = pk2(z, z), back = pk2(kScaleBack, kScaleBack);
#pragma unroll
                for (int q = 0; q < NT; ++q) {
                    float* v = acc[m][q] + 2 * h;
                    const uint64_t sum = fma2(z2, pk2(cs[q][0], cs[q][1]), pk2(c[q][2 * h], c[q][2 * h + 1]));
                    unpk2(fma2(s2, mul2(sum, back), pk2(v[0], v[1])), v[0], v[1]);
                }
            }
        };
        // the tokens' values of step j (unit 4j + t), paired like the codes
        auto tokens = [&](int j, uint32_t (&xb)[NT][4]) {
#pragma unroll
            for (int q = 0; q < NT; ++q) {
                const uint4 v = *reinterpret_cast<const uint4*>(at + x_off[q][j]);
                token_pairs<BITS>(v, xb[q]);
            }
        };
        const int left = a.K - b * kBlock;   // codes from this block on

        if constexpr (MODE == kTiny) {
            // groups of 8 or 16: the lanes of a quad hold different ones
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (32 * j >= left) break;   // the same for every lane
                uint32_t xb[NT][4];
                tokens(j, xb);
                Unit<BITS> u[MT][2];
#pragma unroll
                for (int m = 0; m < MT; ++m) units(m, j, u[m]);
                for (int sub = 0; sub < 32 / a.g; ++sub) {
                    const uint32_t mask = t * 8 / a.g == sub ? 0xffffffffu : 0u;
                    float cs[NT][4];
                    clear(cs);
                    total(xb, mask, cs);
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        float c[NT][4];
                        clear(c);
                        product(u[m], xb, mask, c);
                        fold(m, 32 * j / a.g + sub, c, cs);
                    }
                }
            }
        } else {
            float c[MT][NT][4], cs[NT][4];
            const bool g32 = a.g == 32;   // (kNarrow) a group ends with each step, else with every second
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t xb[NT][4];
                tokens(j, xb);
                if (j == 0 || (MODE == kNarrow && (j == 2 || g32))) {
                    clear(cs);
#pragma unroll
                    for (int m = 0; m < MT; ++m) clear(c[m]);
                }
                total(xb, 0xffffffffu, cs);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    Unit<BITS> u[2];
                    units(m, j, u);
                    product(u, xb, 0xffffffffu, c[m]);
                    if constexpr (MODE == kNarrow) {
                        // (groups past the last column have no scale: K is a multiple of 64)
                        if ((g32 || (j & 1)) && 32 * j < left) fold(m, g32 ? j : j >> 1, c[m], cs);
                    } else {
                        if (j == 3) fold(m, 0, c[m], cs);
                    }
                }
            }
        }
        __syncwarp();   // every lane has read the slot
        if (done + depth < items) {
            if (lane == 0 && ok) {
                load_weights(next_s, next_n0, slot);
                load_tokens(next_s, slot);
            }
            load_scales(next_s, next_n0, slot);
            advance();
        }
        cp_commit();
        if (++slot == depth) {
            slot = 0;
            phase ^= 1u;
        }
    }
    // ---- partial sums of the K slices: within the CTA, then the cluster (whose
    // CTAs have one tile each)
    if (a.red_at == S::kHead) __syncthreads();   // the sums take the place of the rings
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int q = 0; q < NT; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int col = 2 * t + (i & 1), tk = 8 * q + ((col >> 1) | (col & 1) << 2);   // its token, as above
                if (tk < a.n_tok) red[(warp * a.n_tok + tk) * S::kPitch + m * 16 + g8 + 8 * (i >> 1)] = acc[m][q][i];
            }
    __syncthreads();
    if (ranks > 1) {
        for (int e = threadIdx.x; e < a.n_tok * kRows; e += kThreads) {
            const int tk = e / kRows, r = e % kRows;
            float v = red[tk * S::kPitch + r];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) v += red[(w * a.n_tok + tk) * S::kPitch + r];
            red[tk * S::kPitch + r] = v;   // each entry has one owner
        }
        cluster.sync();
    }
    for (int e = rank * kThreads + threadIdx.x; e < a.n_tok * kOut; e += ranks * kThreads) {
        const int tk = e / kOut, r = e % kOut, n = n0 + r;
        if (n >= a.N) continue;
        float v = 0.f, u = 0.f;
        if (ranks > 1) {
            for (int k = 0; k < ranks; ++k) {
                const float* p = cluster.map_shared_rank(red + tk * S::kPitch + r, k);
                v += p[0];
                if constexpr (GATED) u += p[kOut];
            }
        } else {
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float* p = red + (w * a.n_tok + tk) * S::kPitch + r;
                v += p[0];
                if constexpr (GATED) u += p[kOut];
            }
        }
        float y;
        if constexpr (GATED) {
            y = activate(v, a.act) * u;
        } else {
            if (a.bias != nullptr) v += a.bias[n];
            y = activate(v, a.act);
            if (a.residual != nullptr) y += bf16_to_float(a.residual[tk * a.ldr + n]);
        }
        a.Y[tk * a.ldy + n] = f32_to_bf16_bits(y);
    }
    if (ranks > 1) cluster.sync();   // no CTA leaves while its sums are read
    else if (tile + static_cast<int>(gridDim.x) < tiles) __syncthreads();   // the sums are rewritten
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!ok && lane == 0) {
        // never leave with copies in flight (bounded): from that block on, as far as
        // they were issued
        volatile int no_abort = 0;
        const int from = stopped[warp];
        for (int i = from; i < items && i < from + depth; ++i)
            if (!mbar_wait(&full[i % depth], (i / depth) & 1u, &no_abort)) break;
    }
    if (threadIdx.x == 0 && *abort) report(a.status, GPTQ_ERR_TIMEOUT);
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

// What a launch needs beside Args: the tokens' buffer and the code width.
struct Launch {
    const uint16_t* X;
    int64_t ldx;
    cudaStream_t stream;
};

// A block in the rings of a CTA's warps: weights and tokens, scales and zero points.
template <class S>
int ring_block_bytes(int n_tok, int groups) {
    return kWarps * ((S::kWBytes + n_tok * 256 + 1023) / 1024 * 1024 + S::kRows * 8 * groups);
}

template <int BITS, int MODE, int NT, int MT, bool GATED>
cudaError_t launch_one(Args a, const Launch& l) {
    using S = Shape<BITS, NT, MT>;
    auto kern = decode_kernel<BITS, MODE, NT, MT, GATED>;
    constexpr int kOut = GATED ? S::kRows / 2 : S::kRows;
    const int tiles = (a.N + kOut - 1) / kOut;
    const int nblk = (a.K + kBlock - 1) / kBlock;
    // split K over a cluster while all CTAs still run in one wave (two per SM) and
    // every warp keeps at least two blocks
    int ranks = 1;
    while (ranks < 8 && tiles * ranks <= num_sms() && nblk >= 4 * ranks * kWarps) ranks *= 2;
    const int steps = (nblk + kWarps * ranks - 1) / (kWarps * ranks);
    const int ngb = MODE == kWide ? 1 : kBlock / a.g;
    for (a.ngb_log2 = 0; (1 << a.ngb_log2) < ngb; ++a.ngb_log2) {}
    const uint64_t bpg = a.g >= a.K ? nblk : a.g / kBlock;   // (kWide only)
    a.blocks_per_group = static_cast<int>(bpg);
    // magic = ceil(2^32 / bpg) overshoots by e / bpg with e < bpg: exact below
    // block nblk if nblk e < 2^32 (a block's number itself where bpg is 1)
    const uint64_t magic = bpg > 1 ? ((uint64_t{1} << 32) + bpg - 1) / bpg : 0;
    a.group_magic = bpg > 1 && nblk * (magic * bpg - (uint64_t{1} << 32)) < (uint64_t{1} << 32)
                        ? static_cast<uint32_t>(magic) : 0;
    a.probe_ns = take_wait_probe(kProbeDecode);
    a.slot_bytes = (S::kWBytes + a.n_tok * 256 + 1023) / 1024 * 1024;
    const int per = ring_block_bytes<S>(a.n_tok, ngb);
    const int sums = kWarps * a.n_tok * S::kPitch * 4;       // the warps' partial sums
    const int per_sm = NT * MT >= 8 ? 1 : 2, room = (per_sm == 1 ? kSmemOne : kSmemTwo) - S::kHead;
    // More tiles than CTAs run at a time: these go through the tiles in turn, their
    // rings running on, if the partial sums leave the rings two blocks (2 x
    // 11008 x 4096 at one token 17.6 against 19.4 us).  Otherwise the sums take
    // the rings' place after a CTA's only tile.
    const int wave = per_sm * num_sms();
    const bool turns = tiles > wave && room - sums >= 2 * per;
    const int grid = turns ? wave : tiles;
    const int items = steps * (turns ? (tiles + wave - 1) / wave : 1);
    int depth = (turns ? room - sums : room) / per;
    if (depth < 2) depth = (kSmemOne - S::kHead) / per;      // one CTA per SM then
    if (depth < 1) return cudaErrorInvalidConfiguration;
    a.depth = depth > kMaxDepth ? kMaxDepth : depth;
    if (a.depth > items) a.depth = items;
    a.red_at = turns ? S::kHead + a.depth * per : S::kHead;
    const int smem = turns || a.depth * per < sums ? a.red_at + sums : S::kHead + a.depth * per;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemOne);
    if (e != cudaSuccess) return e;
    constexpr Swz kSwz = BITS == 8 ? Swz::k128 : BITS == 4 ? Swz::k64 : BITS == 2 ? Swz::k32 : Swz::kNone;
    const uint64_t words = static_cast<uint64_t>(a.K) * BITS / 32;
    CUtensorMap tw[2], tx;
    // the packed words move as raw 32-bit elements (the map's fp32 type only sizes them)
    for (int m = 0; m < (GATED ? 2 : 1); ++m)
        if (!make_tmap_2d(&tw[m], false, a.mat[m].packed, words, a.N, words, 4 * BITS, kOut, kSwz))
            return cudaErrorInvalidValue;
    if (!GATED) tw[1] = tw[0];
    if (!make_tmap_2d(&tx, true, l.X, a.K, a.n_tok, l.ldx, 64, a.n_tok, Swz::k128)) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, ranks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = l.stream;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (ranks > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim = {1, static_cast<unsigned>(ranks), 1};
        ++n;
    }
    if (a.gathered) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kern, tw[0], tw[1], tx, a);
}

template <int BITS, int MODE, bool GATED>
cudaError_t launch_tokens(const Args& a, const Launch& l) {
    // Eight tokens: 64 weight rows per CTA from 4096 rows on (the tokens' work and
    // a block's fixed work are shared by twice the weights: 8192 x 4096 at one
    // token 8.4 against 11.9 us with 32 rows), fewer where 32 rows are needed to
    // fill the GPU or where 64 leave no two blocks in the rings of two CTAs per SM
    // (8192 x 8192, eight tokens: 8 bits in groups of 64 18.5 against 27.4, 4 bits in groups of 32
    // 19.8 against 27.7 us).
    constexpr int kMany = MODE == kTiny || BITS == 8 ? 2 : 4;
    if (a.n_tok <= 8 && (GATED ? 2 : 1) * static_cast<int64_t>(a.N) >= 4096 &&
        2 * ring_block_bytes<Shape<BITS, 1, kMany>>(a.n_tok, MODE == kWide ? 1 : kBlock / a.g) <= kSmemTwo - 1024)
        return launch_one<BITS, MODE, 1, kMany, GATED>(a, l);
    if (a.n_tok <= 8) return launch_one<BITS, MODE, 1, 2, GATED>(a, l);
    // 9 to 16: 32 rows, two CTAs per SM; 64 rows run with one (8192 x 8192 at 16
    // tokens 25.8 against 21.0 us, in groups of 32 33.2 against 27.1; ahead where
    // the tiles go round several times, 2 x 28672 x 8192 104.9 against 115.2).
    if (a.n_tok <= 16) return launch_one<BITS, MODE, 2, 2, GATED>(a, l);
    // (wide codes or tiny groups: 64 rows would not leave room for two blocks)
    return launch_one<BITS, MODE, 4, MODE == kTiny || BITS == 8 ? 2 : 4, GATED>(a, l);
}

template <int BITS, bool GATED>
cudaError_t launch_mode(const Args& a, const Launch& l) {
    if (a.g >= a.K || a.g % kBlock == 0) return launch_tokens<BITS, kWide, GATED>(a, l);
    if (a.g >= 32) return launch_tokens<BITS, kNarrow, GATED>(a, l);
    return launch_tokens<BITS, kTiny, GATED>(a, l);
}

template <bool GATED>
cudaError_t launch_bits(const Args& a, int bits, const Launch& l) {
    switch (bits) {
        case 2: return launch_mode<2, GATED>(a, l);
        case 3: return launch_mode<3, GATED>(a, l);
        case 4: return launch_mode<4, GATED>(a, l);
        default: return launch_mode<8, GATED>(a, l);
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
    a.status = c.status;
    a.bias = c.bias;
    a.ldr = c.ldr;
    a.ldy = c.ldy;
    a.act = c.act;
    int64_t launches = 0;
    for (int64_t t0 = 0; t0 < c.n_tok; t0 += kMaxTok) {
        a.n_tok = static_cast<int>(c.n_tok - t0 < kMaxTok ? c.n_tok - t0 : kMaxTok);
        Launch l = {c.X + t0 * c.ldx, c.ldx, stream};
        if (gather) {
            uint16_t* xq = static_cast<uint16_t*>(c.ws);
            const int64_t work = (static_cast<int64_t>(a.n_tok) * (a.K / 8) + 255) / 256;
            const int blocks = static_cast<int>(work < 8 * num_sms() ? work : 8 * num_sms());
            gather_rows_kernel<<<blocks, 256, 0, stream>>>(l.X, l.ldx, a.n_tok, a.K, c.perm, xq);
            if (cudaGetLastError() != cudaSuccess) return GPTQ_ERR_CUDA;
            l.X = xq;
            l.ldx = c.d_col;
            ++launches;
        }
        a.residual = c.residual == nullptr ? nullptr : c.residual + t0 * c.ldr;
        a.Y = c.Y + t0 * c.ldy;
        a.gathered = gather;
        const cudaError_t e = gated ? launch_bits<true>(a, c.bits, l) : launch_bits<false>(a, c.bits, l);
        if (e != cudaSuccess) return GPTQ_ERR_CUDA;
        ++launches;
    }
    count_launches(launches);
    return GPTQ_OK;
}

}  // namespace gptq
