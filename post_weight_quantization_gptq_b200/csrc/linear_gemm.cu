// Many tokens through packed layers on the 5th-generation tensor cores, with
// the epilogue of the layer, and the gradient with respect to the tokens:
//   linear    Y = act(Xq W^T + bias) + residual          (Xq[t][k] = X[t][perm[k]])
//   gated     Y = act(Xq Wg^T) * (Xq Wu^T)
//   backward  dXq = dP W  (linear),  dXq = dG Wg + dU Wu  (gated)
// with the 16-bit weights W[n][k] = bf16( fp32(s[k/g][n]) * (q[n][k] - z[k/g][n]) ):
// products of two bf16 values are exact, sums are fp32, outputs are rounded to
// bf16 once.
//
// One kernel for the three, in two sizes: a CTA with a tile of 128 tokens x 256
// columns, and a pair of CTAs (cta_group::2) with 512 x 256.  It sweeps the
// contraction in stages of 64:
//   warp 0      TMA: the stage's tokens (128 x 64 bf16, 128-byte swizzle)
//   warp 2      TMA: the stage's packed words, in a ring of their own
//   warp 1      tensor memory and the MMAs (kind::f16, M 128, N 256, K 16)
//   warps 3..   dequantize the stage's 256 x 64 weights into a bf16 tile in
//               shared memory, one thread per 64 codes of one weight row; teams
//               of eight warps take the stages in turn and keep a stage's weights
//               in registers until their buffer is free, so that hand-overs
//               (waits, fence, arrivals) and MMAs hide behind arithmetic (0.64 us
//               per stage of 128 tokens; 0.77 with the buffer waited for first).
//               After the sweep they drain the accumulators through the epilogue
// linear    the tile's columns are 256 weight rows n, the stage 64 of their k:
//           the weight tile is K-major.
// gated     the columns are 128 rows of the gate and the same 128 of the up
//           matrix, so a thread finds both products of an output in its own
//           tensor-memory lane and the gate product never leaves the chip.
// backward  the columns are 256 k, the stage 64 weight rows n: a thread still
//           writes 64 codes of one row as 128 bytes, which now is the MN-major
//           layout of the same tile; the two matrices of the gated form are two
//           sweeps into one accumulator.
// Dequantization is arithmetic on two pipes (see weights8).  A pair's tile whose
// second 256 tokens lie past the end skips their loads and MMAs.
//
// Tiles that do not fill the last wave of SMs split the contraction: their
// partial tiles go to the workspace and a second kernel adds them in order and
// runs the epilogue.  No atomics: same bits every call.  Every wait is bounded
// (GPTQ_ERR_TIMEOUT).
#include <cuda.h>

#include "activation.cuh"
#include "common.cuh"
#include "f32x2.cuh"
#include "kernels.h"

namespace gptq {
namespace {

enum Mode { kLinear, kGated, kBack };

constexpr int TM = 128;                       // tokens per tile of a single CTA
constexpr int TN = 256;                       // tile columns (MMA N)
constexpr int BK = 64;                        // contraction per stage
constexpr int kAStages = 4;
constexpr int kABytes = TM * BK * 2;          // 16 KB: a stage's tokens
constexpr int kBBytes = TN * BK * 2;          // 32 KB: one dequantized tile
constexpr int kTeams = 2;                     // of 8 dequantizing warps, on alternate stages
constexpr int kTeamWarps = 8;
// One dequantized tile per team: the warps hold the next in registers, and the
// shared memory serves the packed words, whose loads have the longer way (four
// tiles and two to four stages: 13000 x 4096 gated, 112 tokens 50.6 us at 4 bits
// and 70.1 at 8, now 48.2 and 48.0).
constexpr int kBBufs = kTeams;
constexpr int kMaxPStages = 6;
constexpr int kDeqWarps = kTeams * kTeamWarps;
constexpr int kThreads = 32 * (3 + kDeqWarps);
constexpr uint32_t kTmemCols = 256;
// SMs of the device this library is built for.  It only shapes the plan (split
// contractions, partial tiles): with fewer SMs a call is as right and takes more
// waves, and a workspace's size does not depend on the current device.
constexpr int kSms = 148;
constexpr int kMinStages = 4;                 // least stages of a split tile's part (8: 4096 x 1024, 128 tokens 16.6 us, now 14.7)
constexpr int kMaxSplit = 16;

// Packed words of a stage.  A box of the tensor map is 64 codes wide (16 bytes
// or more) except at 3 bits, where 64 codes are 24 bytes: its boxes hold 128
// codes, two stages of the forward sweep.
template <int BITS, int MODE>
struct Geom {
    static constexpr int kBoxCodes = BITS == 3 ? 128 : 64;
    static constexpr int kBoxWords = kBoxCodes * BITS / 32;
    static constexpr int kRowBytes = kBoxWords * 4;
    static constexpr bool kPairs = BITS == 3 && MODE != kBack;   // a slot serves two stages
    static constexpr int kSlot = MODE == kBack ? 64 * TN * BITS / 8 : TN * kRowBytes;
    static constexpr int kPStages = kPairs ? 4 : 6;
    static constexpr int kSmem = kAStages * kABytes + kBBufs * kBBytes + kPStages * kSlot + 1024 + 256;
    // a parity wait is only right for the phase after the last one seen, so a
    // team has to meet every phase of a slot or buffer: stages it shares with
    // the other team come back to it
    static_assert(kPStages % kTeams == 0 && kBBufs % kTeams == 0, "rings of whole rounds of the teams");
};

struct Bars {
    uint64_t afull[kAStages], aempty[kAStages];
    uint64_t pfull[kMaxPStages], pempty[kMaxPStages];
    uint64_t bfull[kBBufs], bempty[kBBufs];
    uint64_t acc_full, drain;
    uint64_t never;                             // (timeout probe)
    uint32_t tmem;
    int abort;
};
static_assert(sizeof(Bars) <= 256, "their share of kSmem");

struct Args {
    PackedMatrix mat[2];
    int n_tok, N;        // rows and columns of the output
    int nk;              // stages of the whole contraction
    int nk1;             // backward: stages of the first matrix
    int d_row, d_col, g;
    int tiles_n;
    int full, split, per;   // whole tiles; parts of the others and their stages
    int part_rows;          // tokens of a partial tile
    int tile_tokens;        // 128, or 512 per pair of CTAs
    float* part;
    const float* bias;
    int act;
    const uint16_t* residual;
    int64_t ldr;
    uint16_t* pre[2];
    int64_t ldpre[2];
    uint16_t* Y;
    int64_t ldy;
    int32_t* status;
    uint64_t probe_ns;
};

// ------------------------------------------------------------- epilogue
// Sixteen consecutive bf16 values per lane (32 bytes, the sector that L2 moves),
// `count` of them valid (0: none).  Called by whole warps.  Rows on 32- or
// 16-byte boundaries move in one or two accesses per lane; for any other
// alignment the warp goes through its 1 KB of shared memory, so that 16 lanes
// write (read) the 16 values of a row together: alone, a lane's 2-byte stores
// are as many sector writes (a gated 72 x 775 tile with its products saved took
// 35 us).
__device__ __forceinline__ int vector_bytes(const void* p, int count) {
    // 32, 16 or 0 for the warp
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    if (__all_sync(0xffffffffu, count == 0 || (count == 16 && (at & 31) == 0))) return 32;
    return __all_sync(0xffffffffu, count == 0 || (count == 16 && (at & 15) == 0)) ? 16 : 0;
}
__device__ __forceinline__ void store16(uint16_t* p, const float (&v)[16], int count, uint8_t* scratch) {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = f32x2_to_bf16x2(v[2 * j], v[2 * j + 1]);
    const int bytes = vector_bytes(p, count);
    if (bytes == 32) {
        if (count > 0)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
                         "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                         : "memory");
        return;
    }
    if (bytes == 16) {
        if (count > 0) {
            reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
            reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
        return;
    }
    const int lane = threadIdx.x & 31;
    __syncwarp();
    reinterpret_cast<uint4*>(scratch)[2 * lane] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(scratch)[2 * lane + 1] = make_uint4(w[4], w[5], w[6], w[7]);
    __syncwarp();
#pragma unroll 4
    for (int i = 0; i < 16; ++i) {
        const int owner = 2 * i + (lane >> 4), idx = lane & 15;
        uint16_t* q = reinterpret_cast<uint16_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(p), owner));
        if (idx < __shfl_sync(0xffffffffu, count, owner)) q[idx] = reinterpret_cast<const uint16_t*>(scratch)[owner * 16 + idx];
    }
    __syncwarp();
}
__device__ __forceinline__ void load16(const uint16_t* p, uint32_t (&w)[8], int count, uint8_t* scratch) {
    const int bytes = vector_bytes(p, count);
    if (bytes == 32) {
        if (count > 0)
            asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                         : "l"(p)
                         : "memory");
        return;
    }
    if (bytes == 16) {
        if (count > 0) {
            const uint4 x = reinterpret_cast<const uint4*>(p)[0], y = reinterpret_cast<const uint4*>(p)[1];
            w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
            w[4] = y.x; w[5] = y.y; w[6] = y.z; w[7] = y.w;
        }
        return;
    }
    const int lane = threadIdx.x & 31;
    uint16_t got[16];   // all loads in flight together
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int owner = 2 * i + (lane >> 4), idx = lane & 15;
        const uint16_t* q = reinterpret_cast<const uint16_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(p), owner));
        const bool in = idx < __shfl_sync(0xffffffffu, count, owner);
        got[i] = in ? q[idx] : static_cast<uint16_t>(0);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) reinterpret_cast<uint16_t*>(scratch)[(2 * i + (lane >> 4)) * 16 + (lane & 15)] = got[i];
    __syncwarp();
    const uint4 x = reinterpret_cast<const uint4*>(scratch)[2 * lane], y = reinterpret_cast<const uint4*>(scratch)[2 * lane + 1];
    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    w[4] = y.x; w[5] = y.y; w[6] = y.z; w[7] = y.w;
    __syncwarp();
}

// Sixteen consecutive outputs of token t from column n on (a multiple of 16): v
// their sums (gated: of the gate, u of the up matrix), r the residual's words.
// count: of the 16 that exist (0: a token or column past the end).
__device__ __forceinline__ int valid16(const Args& a, int t, int n) {
    return t < a.n_tok && n < a.N ? min(16, a.N - n) : 0;
}
template <int MODE>
__device__ __forceinline__ void load_residual(const Args& a, int t, int n, uint32_t (&r)[8], uint8_t* scratch) {
    if constexpr (MODE == kLinear) {
        if (a.residual != nullptr) load16(a.residual + t * a.ldr + n, r, valid16(a, t, n), scratch);
    }
}
template <int MODE>
__device__ __forceinline__ void emit16(const Args& a, int t, int n, float (&v)[16], const float (&u)[16],
                                       const uint32_t (&r)[8], uint8_t* scratch) {
    const int count = valid16(a, t, n);
    if constexpr (MODE == kLinear) {
        if (a.bias != nullptr) {
            if (count == 16 && (reinterpret_cast<uintptr_t>(a.bias) & 15) == 0) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 b = __ldg(reinterpret_cast<const float4*>(a.bias + n) + j);
                    v[4 * j] += b.x; v[4 * j + 1] += b.y; v[4 * j + 2] += b.z; v[4 * j + 3] += b.w;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (j < count) v[j] += __ldg(a.bias + n + j);
            }
        }
        if (a.pre[0] != nullptr) store16(a.pre[0] + t * a.ldpre[0] + n, v, count, scratch);
        activate_all(v, a.act);
        if (a.residual != nullptr) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[2 * j] += __uint_as_float(r[j] << 16);
                v[2 * j + 1] += __uint_as_float(r[j] & 0xFFFF0000u);
            }
        }
    } else if constexpr (MODE == kGated) {
        if (a.pre[0] != nullptr) store16(a.pre[0] + t * a.ldpre[0] + n, v, count, scratch);
        if (a.pre[1] != nullptr) store16(a.pre[1] + t * a.ldpre[1] + n, u, count, scratch);
        activate_all(v, a.act);
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] *= u[j];
    }
    store16(a.Y + t * a.ldy + n, v, count, scratch);
}

// ------------------------------------------------------- dequantization
// The NW words (32 or 64 codes) of a thread's stage; 3-bit rows lie on 8-byte
// boundaries (4-byte for 32 codes), the others on whole vectors.
template <int BITS, int NW>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[NW]) {
    if constexpr (BITS == 3) {
#pragma unroll
        for (int q = 0; q < NW; ++q) w[q] = reinterpret_cast<const uint32_t*>(p)[q];
    } else if constexpr (NW == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x;
        w[1] = v.y;
    } else {
#pragma unroll
        for (int q = 0; q < NW / 4; ++q) {
            const uint4 v = reinterpret_cast<const uint4*>(p)[q];
            w[4 * q] = v.x; w[4 * q + 1] = v.y; w[4 * q + 2] = v.z; w[4 * q + 3] = v.w;
        }
    }
}

// A group's parameters as the arithmetic below takes them.  A code at bits
// BITS p .. of a word (p = 0 .. 3) is masked there and ORed with the exponent of
// 2^23: the float 2^23 + q 2^(BITS p), no shift.  Less 2^23 + z 2^(BITS p) that
// is (q - z) 2^(BITS p) exactly, and times s 2^-(BITS p) it is the fp32 product
// s (q - z), rounded once.  8-bit codes are put at bit 0 by a byte permute.
template <int BITS>
struct Group {
    static constexpr int kPairs = BITS == 8 ? 1 : 2;
    uint64_t off[kPairs], scale[kPairs];   // positions (0, 1) and (2, 3)
    __device__ __forceinline__ void set(float s, float z) {
        constexpr float kBase = 8388608.f;
        if constexpr (BITS == 8) {
            off[0] = pk2(kBase + z, kBase + z);
            scale[0] = pk2(s, s);
        } else {
            constexpr float k1 = 1 << BITS, k2 = 1 << (2 * BITS), k3 = 1 << (3 * BITS);
            off[0] = pk2(kBase + z, fmaf(z, k1, kBase));
            off[1] = pk2(fmaf(z, k2, kBase), fmaf(z, k3, kBase));
            scale[0] = pk2(s, s * (1.f / k1));
            scale[1] = pk2(s * (1.f / k2), s * (1.f / k3));
        }
    }
};

// Codes 8c .. 8c+7 of a thread's words as four bf16x2 weights: per 8 codes 8 masks
// and a shift, 4 packings and 8 packed fp32 operations on the other pipe (a
// table look-up by byte permutes takes 23 on the first, which runs 64 lanes per
// cycle and bound the sweep).
template <int BITS, int NW>
__device__ __forceinline__ void weights8(const uint32_t (&w)[NW], int c, const Group<BITS>& g, uint32_t (&o)[4]) {
    constexpr uint32_t kMagic = 0x4B000000u;
    uint64_t f[4];
    if constexpr (BITS == 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t x = w[2 * c + (i >> 1)];
            const int b = 2 * (i & 1);
            f[i] = pk2(__uint_as_float(__byte_perm(x, kMagic, 0x7440 + b)), __uint_as_float(__byte_perm(x, kMagic, 0x7441 + b)));
        }
    } else {
        uint32_t v;   // the 8 codes from bit 0 on
        if constexpr (BITS == 4) {
            v = w[c];
        } else if constexpr (BITS == 2) {
            v = (c & 1) ? w[c >> 1] >> 16 : w[c >> 1];
        } else {
            const int b = (24 * c) >> 5, sh = (24 * c) & 31;
            v = sh <= 8 ? (w[b] >> sh) : __funnelshift_r(w[b], w[b + 1 < NW ? b + 1 : NW - 1], sh);
        }
        const uint32_t u = v >> (4 * BITS);
        constexpr uint32_t kMask = (1u << BITS) - 1u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t x = i < 2 ? v : u;
            const int at = 2 * BITS * (i & 1);
            f[i] = pk2(__uint_as_float((x & (kMask << at)) | kMagic),
                       __uint_as_float((x & (kMask << (at + BITS))) | kMagic));
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        unpk2(mul2(sub2(f[i], g.off[i % Group<BITS>::kPairs]), g.scale[i % Group<BITS>::kPairs]), lo, hi);
        o[i] = f32x2_to_bf16x2(lo, hi);
    }
}

// A CTA's accumulators (tokens t0 .. and t0 + step .. in the two halves) through
// the epilogue, or into partial tile `slot` (whose rows start `row0` before t0).
// WARPS / 4 warps share a lane quarter's chunks of 16 columns.
template <int MODE, int WARPS>
__device__ __forceinline__ void drain_tile(const Args& a, uint32_t tmem, int slot, int halves, int t0, int step,
                                           int n0, int warp, int lane, int row0, uint8_t* smem) {
    const int q = warp & 3;           // tensor-memory lane quarter of this warp
    const int side = (warp - 3) >> 2;
    uint8_t* scratch = smem + (warp - 3) * 1024;   // of the rings, which the sweep has left
    const int chunks = MODE == kGated && slot < 0 ? TN / 32 : TN / 16;
#pragma unroll 1
    for (int e = side; e < halves * chunks; e += WARPS / 4) {
        const int h = e / chunks, c = e % chunks;
        const int t = t0 + h * step + 32 * q + lane;
        const uint32_t at = tmem + (static_cast<uint32_t>(32 * q) << 16) + h * TN + c * 16;
        float v[16], u[16];
        uint32_t r[8] = {};
        if (slot < 0) load_residual<MODE>(a, t, n0 + c * 16, r, scratch);
        tmem_ld16(at, v);
        if constexpr (MODE == kGated) {
            if (slot < 0) tmem_ld16(at + TN / 2, u);
        }
        if (t < a.n_tok && slot >= 0) {
            float* p = a.part + (static_cast<int64_t>(slot) * a.part_rows + (t - t0 + row0)) * TN + c * 16;
#pragma unroll
            for (int x = 0; x < 2; ++x)   // 32 bytes each (the workspace is 256-byte aligned)
                asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p + 8 * x),
                             "f"(v[8 * x]), "f"(v[8 * x + 1]), "f"(v[8 * x + 2]), "f"(v[8 * x + 3]), "f"(v[8 * x + 4]),
                             "f"(v[8 * x + 5]), "f"(v[8 * x + 6]), "f"(v[8 * x + 7])
                             : "memory");
        }
        __syncwarp();
        if (slot < 0) emit16<MODE>(a, t, n0 + c * 16, v, u, r, scratch);
    }
}

// GPT: groups in a thread's 64 codes (1 where g is a multiple of 64 or one group
// spans the row).
template <int BITS, int GPT, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    packed_gemm_kernel(const __grid_constant__ CUtensorMap tma0, const __grid_constant__ CUtensorMap tma1,
                       const __grid_constant__ CUtensorMap tmp0, const __grid_constant__ CUtensorMap tmp1,
                       const __grid_constant__ Args a) {
    using G = Geom<BITS, MODE>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint8_t* bbuf = smem + kAStages * kABytes;
    uint8_t* pbuf = bbuf + kBBufs * kBBytes;
    Bars* bars = reinterpret_cast<Bars*>(pbuf + G::kPStages * G::kSlot);
    volatile int* abort = &bars->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // this CTA's tile and its part of the contraction
    int tile = blockIdx.x, k0 = 0, k1 = a.nk, slot = -1;
    if (tile >= a.full) {
        slot = tile - a.full;
        tile = a.full + slot / a.split;
        k0 = (slot % a.split) * a.per;
        k1 = min(a.nk, k0 + a.per);
    }
    const int t0 = (tile / a.tiles_n) * TM;
    const int n0 = (tile % a.tiles_n) * (MODE == kGated ? TN / 2 : TN);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kAStages; ++s) {
            mbar_init(&bars->afull[s], 1);
            mbar_init(&bars->aempty[s], 1);
        }
        for (int s = 0; s < G::kPStages; ++s) {
            mbar_init(&bars->pfull[s], 1);
            mbar_init(&bars->pempty[s], G::kPairs ? 2 * kTeamWarps : kTeamWarps);
        }
        for (int b = 0; b < kBBufs; ++b) {
            mbar_init(&bars->bfull[b], kTeamWarps);
            mbar_init(&bars->bempty[b], 1);
        }
        mbar_init(&bars->acc_full, 1);
        mbar_init(&bars->drain, 1);
        mbar_init(&bars->never, 1);
        bars->abort = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tma0);
        tma_prefetch_desc(&tmp0);
    }
    if (warp == 1) {
        tmem_alloc(&bars->tmem, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem;

    if (warp == 0) {
        // ------------------------------------------------ TMA: tokens
        if (lane == 0) {
            int i = 0;
            for (int it = k0; it < k1 && !*abort; ++it, ++i) {
                const int st = i % kAStages;
                if (!mbar_wait_short(&bars->aempty[st], ((i / kAStages) & 1u) ^ 1u, abort)) break;
                const bool second = MODE == kBack && it >= a.nk1;
                const CUtensorMap* map = second ? &tma1 : &tma0;
                const int x = (second ? it - a.nk1 : it) * BK;
                mbar_arrive_expect_tx(&bars->afull[st], kABytes);
                tma_load_2d(smem + st * kABytes, map, &bars->afull[st], x, t0);
            }
            // never leave with copies in flight (bounded even when aborting)
            volatile int no_abort = 0;
            for (int j = 0; j < min(i, kAStages); ++j) {
                const int i2 = i - 1 - j;
                if (!mbar_wait_short(&bars->afull[i2 % kAStages], (i2 / kAStages) & 1u, &no_abort)) {
                    *abort = 1;
                    break;
                }
            }
        }
    } else if (warp == 2) {
        // ------------------------------------------------ TMA: packed words
        if (lane == 0) {
            constexpr int kStep = G::kPairs ? 2 : 1;
            int i = 0;
            for (int it = k0; it < k1 && !*abort; it += kStep, ++i) {
                const int ps = i % G::kPStages;
                if (!mbar_wait_short(&bars->pempty[ps], ((i / G::kPStages) & 1u) ^ 1u, abort)) break;
                uint8_t* dst = pbuf + ps * G::kSlot;
                mbar_arrive_expect_tx(&bars->pfull[ps], G::kSlot);
                if constexpr (MODE == kBack) {
                    const bool second = it >= a.nk1;
                    const int row = (second ? it - a.nk1 : it) * BK;
                    constexpr int kBoxes = TN / G::kBoxCodes;
                    for (int c = 0; c < kBoxes; ++c)
                        tma_load_2d(dst + c * (BK * G::kRowBytes), second ? &tmp1 : &tmp0, &bars->pfull[ps],
                                    (n0 / G::kBoxCodes + c) * G::kBoxWords, row);
                } else {
                    const int x = (it / kStep) * G::kBoxWords;
                    tma_load_2d(dst, &tmp0, &bars->pfull[ps], x, n0);
                    tma_load_2d(dst + 128 * G::kRowBytes, MODE == kGated ? &tmp1 : &tmp0, &bars->pfull[ps], x,
                                MODE == kGated ? n0 : n0 + 128);
                }
            }
            volatile int no_abort = 0;
            for (int j = 0; j < min(i, G::kPStages); ++j) {
                const int i2 = i - 1 - j;
                if (!mbar_wait_short(&bars->pfull[i2 % G::kPStages], (i2 / G::kPStages) & 1u, &no_abort)) {
                    *abort = 1;
                    break;
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        if (lane == 0) {
            constexpr uint32_t kIdesc = instr_desc(/*bf16*/ 1, /*A K-major*/ 0, /*B*/ MODE == kBack ? 1 : 0, 128, TN);
            bool ok = wait_probe(&bars->never, a.probe_ns, abort);
            for (int i = 0; ok && i < k1 - k0; ++i) {
                const int st = i % kAStages, b = i % kBBufs;
                if (!mbar_wait_short(&bars->afull[st], (i / kAStages) & 1u, abort) ||
                    !mbar_wait_short(&bars->bfull[b], (i / kBBufs) & 1u, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t am = smem_u32(smem + st * kABytes);
                const uint32_t bm = smem_u32(bbuf + b * kBBytes);
#pragma unroll
                for (int kk = 0; kk < BK / 16; ++kk) {
                    // K-major: 32 bytes of each row; MN-major: two atoms of 8
                    // weight rows, boxes of 64 columns 8 KB apart
                    const uint64_t bd = MODE == kBack ? smem_desc(bm + kk * 2048, 8192, 1024, 2)
                                                      : smem_desc(bm + kk * 32, 16, 1024, 2);
                    mma_f16_ss(tmem, smem_desc(am + kk * 32, 16, 1024, 2), bd, kIdesc, (i > 0 || kk > 0) ? 1u : 0u);
                }
                mma_commit(&bars->aempty[st]);
                mma_commit(&bars->bempty[b]);
            }
            if (ok) mma_commit(&bars->acc_full);
            mma_commit(&bars->drain);
            volatile int no_abort = 0;
            if (!mbar_wait_short(&bars->drain, 0, &no_abort)) *abort = 1;
        }
    } else {
        // ------------------------------------------------ dequantize
        const int j = (threadIdx.x - 96) & 255;   // the thread's 128 bytes of the weight tile
        const int team = (threadIdx.x - 96) >> 8; // which stages it takes
        // forward: weight row `wrow` of matrix `mi`; backward: row 64 it + (j & 63),
        // columns n0 + 64 (j >> 6) on
        const int mi = MODE == kGated ? j >> 7 : 0;
        const int wrow = n0 + (MODE == kGated ? (j & 127) : j);
        const int kcol = n0 + 64 * (j >> 6);
        const int groups = (a.d_col + a.g - 1) / a.g;
        // this stage's scales and zero points, and the next one's: loaded a stage
        // ahead and first touched then (even the conversion to float would wait)
        float s[GPT] = {}, s_nx[GPT];
        int z[GPT] = {}, z_nx[GPT];
        const int span = GPT == 1 ? a.g / BK : 1;              // stages per group (forward)
        int gi = GPT == 1 && MODE != kBack ? (k0 + team) / span : 0, rem = GPT == 1 && MODE != kBack ? (k0 + team) % span : 0;
        const int back_group = GPT == 1 ? kcol / a.g : kcol / 64 * GPT;
        auto fetch = [&](int it) {
#pragma unroll
            for (int q = 0; q < GPT; ++q) {
                int group, row, m;
                bool in;
                if constexpr (MODE == kBack) {
                    m = it >= a.nk1 ? 1 : 0;
                    row = (m ? it - a.nk1 : it) * BK + (j & 63);
                    group = back_group + q;
                    in = it < k1 && row < a.d_row && kcol < a.d_col;
                } else {
                    m = mi;
                    row = wrow;
                    group = GPT == 1 ? gi : it * GPT + q;
                    in = it < k1 && row < a.d_row && group < groups;
                }
                s_nx[q] = 0.f;   // rows and columns past the layer: weights 0
                z_nx[q] = 0;
                if (in) {
                    const int64_t at = static_cast<int64_t>(group) * a.d_row + row;
                    s_nx[q] = __ldg(a.mat[m].scales + at);
                    z_nx[q] = __ldg(a.mat[m].zeros + at);
                }
            }
            if constexpr (GPT == 1 && MODE != kBack) {   // the group of the team's next stage
                rem += kTeams;
                while (rem >= span) {
                    rem -= span;
                    ++gi;
                }
            }
        };
        fetch(k0 + team);
        Group<BITS> grp;
        uint32_t dst_off[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) dst_off[c] = j * 128 + ((c ^ (j & 7)) << 4);
        // a lane whose wait runs out stays with its warp, writes what it has and
        // reports nothing more
        bool ok = true;
        for (int it = k0 + team, i = team; it < k1; it += kTeams, i += kTeams) {
            const int pi = G::kPairs ? i >> 1 : i;
            const int ps = pi % G::kPStages, b = i % kBBufs;
#pragma unroll
            for (int q = 0; q < GPT; ++q) {
                s[q] = s_nx[q];
                z[q] = z_nx[q];
            }
            fetch(it + kTeams);
            if constexpr (GPT == 1) grp.set(s[0], static_cast<float>(z[0]));
            ok = ok && mbar_wait_short(&bars->pfull[ps], (pi / G::kPStages) & 1u, abort);
            const uint8_t* src = pbuf + ps * G::kSlot;
            if constexpr (BITS != 3) {
                src += j * G::kRowBytes;
            } else if constexpr (MODE == kBack) {
                src += (j >> 7) * (BK * G::kRowBytes) + (j & 63) * G::kRowBytes + ((j >> 6) & 1) * (G::kRowBytes / 2);
            } else {
                src += j * G::kRowBytes + (i & 1) * (G::kRowBytes / 2);
            }
            uint32_t w[2 * BITS];
            load_words<BITS>(src, w);
            // the stage's weights wait in registers for their buffer, so that the
            // arithmetic overlaps the MMAs that still read it
            uint32_t o[8][4];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                if constexpr (GPT > 1) {
                    if (c % (8 / GPT) == 0) grp.set(s[c / (8 / GPT)], static_cast<float>(z[c / (8 / GPT)]));
                }
                weights8<BITS>(w, c, grp, o[c]);
            }
            ok = ok && mbar_wait_short(&bars->bempty[b], ((i / kBBufs) & 1u) ^ 1u, abort);
            const uint32_t tile_at = smem_u32(bbuf + b * kBBytes);
#pragma unroll
            for (int c = 0; c < 8; ++c) sts128_u(tile_at + dst_off[c], make_uint4(o[c][0], o[c][1], o[c][2], o[c][3]));
            fence_async_smem();
            // one arrival per warp (arrivals on a barrier are serialized)
            __syncwarp();
            if (lane == 0 && ok) {
                mbar_arrive(&bars->bfull[b]);
                // the slot's words have been used (their loads completed) before it may be refilled
                mbar_arrive(&bars->pempty[ps]);
            }
        }
        // ------------------------------------------------ drain: tensor memory -> output
        if (warp_agree(ok && mbar_wait_short(&bars->acc_full, 0, abort))) {
            tc_fence_after();
            drain_tile<MODE, kDeqWarps>(a, tmem, slot, 1, t0, 0, n0, warp, lane, 0, smem);
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, kTmemCols);
    if (threadIdx.x == 0 && bars->abort) report(a.status, GPTQ_ERR_TIMEOUT);
}

// ------------------------------------------------------------ pairs of CTAs
// The same product by two CTAs of a cluster (cta_group::2): a tile of 512 tokens
// x 256 columns, MMAs of M 256 (128 tokens of each CTA) and N 256, of whose
// weight rows each CTA dequantizes and holds 128 (gated: one the gate's, the
// other the up matrix's; backward: 128 of the columns k).  Against two single
// CTAs the weight tile is dequantized, written and read once instead of twice:
// 120 KB of shared memory traffic per CTA and stage instead of 176, at 128 bytes
// per cycle the difference between 940 and 1375 cycles for 1024 of MMAs.
// Roles as above, a dequantizing thread with 32 codes of one of the CTA's 128
// rows (a hand-over between the CTAs takes longer than one inside a CTA, so a
// stage's arithmetic has to be short: four teams of four warps, 64 codes each,
// took 0.73 us per stage of 256 tokens).  The teams of both CTAs report a stage to
// rank 0's barrier, and one thread of rank 1 its tokens' arrival.  A thread
// meets every phase of a barrier that it waits on, in order: a parity wait for
// phase n returns at once while phase n - 1 is still open.
constexpr int PM = 512;                       // tokens per pair and tile
constexpr int kPairBBytes = 128 * BK * 2;     // 16 KB: a CTA's half of the weight tile
constexpr int kHalfBytes = 128 * BK * 2;      // 16 KB: 128 tokens of a stage
constexpr int kPairTeams = 2;                 // of 8 warps (three gained nothing)
constexpr int kPairDeqWarps = kPairTeams * kTeamWarps;
constexpr int kPairThreads = 32 * (3 + kPairDeqWarps);
constexpr int kPairBBufs = 4;
constexpr int kPairUnits = 8;                 // of them in the ring: 4 stages of 256 tokens per CTA, 8 of 128
constexpr uint32_t kPairTmemCols = 512;
template <int BITS, int MODE>
struct PairGeom {
    static constexpr int kBoxWords = Geom<BITS, MODE>::kBoxWords;
    static constexpr int kRowBytes = Geom<BITS, MODE>::kRowBytes;
    static constexpr bool kPairs = Geom<BITS, MODE>::kPairs;
    static constexpr int kSlot = Geom<BITS, MODE>::kSlot / 2;
    static constexpr int kPStages = BITS == 8 || kPairs ? 4 : 8;
    static constexpr int kBBufs = kPairBBufs;
    static constexpr int kSmem = kPairUnits * kHalfBytes + kBBufs * kPairBBytes + kPStages * kSlot + 1024 + 512;
    static_assert(kPStages % kPairTeams == 0 && kBBufs % kPairTeams == 0, "rings of whole rounds of the teams");
};
struct PairBars {
    uint64_t afull[kPairUnits], aempty[kPairUnits];
    uint64_t peer[kPairUnits];                  // rank 0's: rank 1's tokens have landed
    uint64_t pfull[8], pempty[8];
    uint64_t ready[kPairBBufs], bempty[kPairBBufs];               // ready: rank 0's, arrivals of both CTAs
    uint64_t acc_full, drain;
    uint64_t never;                             // (timeout probe)
    uint32_t tmem;
    int abort;
};
static_assert(sizeof(PairBars) <= 512, "their share of kSmem");

template <int BITS, int GPT, int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    pair_gemm_kernel(const __grid_constant__ CUtensorMap tma0, const __grid_constant__ CUtensorMap tma1,
                     const __grid_constant__ CUtensorMap tmp0, const __grid_constant__ CUtensorMap tmp1,
                     const __grid_constant__ Args a) {
    using G = PairGeom<BITS, MODE>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint8_t* bbuf = smem + kPairUnits * kHalfBytes;
    uint8_t* pbuf = bbuf + G::kBBufs * kPairBBytes;
    PairBars* bars = reinterpret_cast<PairBars*>(pbuf + G::kPStages * G::kSlot);
    volatile int* abort = &bars->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_rank());

    int tile = blockIdx.x >> 1, k0 = 0, k1 = a.nk, slot = -1;
    if (tile >= a.full) {
        slot = tile - a.full;
        tile = a.full + slot / a.split;
        k0 = (slot % a.split) * a.per;
        k1 = min(a.nk, k0 + a.per);
    }
    const int t0 = (tile / a.tiles_n) * PM + 128 * rank;     // this CTA's tokens: t0 .. and t0 + 256 ..
    const int n0 = (tile % a.tiles_n) * (MODE == kGated ? TN / 2 : TN);
    const int halves = (tile / a.tiles_n) * PM + 256 < a.n_tok ? 2 : 1;
    const int depth = kPairUnits / halves, abytes = halves * kHalfBytes;   // of the tokens' ring

    if (threadIdx.x == 0) {
        for (int s = 0; s < kPairUnits; ++s) {
            mbar_init(&bars->afull[s], 1);
            mbar_init(&bars->aempty[s], 1);
            mbar_init(&bars->peer[s], 1);
        }
        for (int s = 0; s < G::kPStages; ++s) {
            mbar_init(&bars->pfull[s], 1);
            mbar_init(&bars->pempty[s], G::kPairs ? 2 * kTeamWarps : kTeamWarps);
        }
        for (int b = 0; b < G::kBBufs; ++b) {
            mbar_init(&bars->ready[b], 2 * kTeamWarps);
            mbar_init(&bars->bempty[b], 1);
        }
        mbar_init(&bars->acc_full, 1);
        mbar_init(&bars->drain, 1);
        mbar_init(&bars->never, 1);
        bars->abort = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tma0);
        tma_prefetch_desc(&tmp0);
    }
    if (warp == 1) {
        tmem_alloc_pair(&bars->tmem, kPairTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();   // both CTAs' barriers are there
    tc_fence_after();
    const uint32_t tmem = bars->tmem;

    if (warp == 0) {
        // ------------------------------------------------ TMA: tokens
        if (lane == 0) {
            int i = 0;
            for (int it = k0; it < k1 && !*abort; ++it, ++i) {
                const int st = i % depth;
                if (!mbar_wait_short(&bars->aempty[st], ((i / depth) & 1u) ^ 1u, abort)) break;
                const bool second = MODE == kBack && it >= a.nk1;
                const CUtensorMap* map = second ? &tma1 : &tma0;
                const int x = (second ? it - a.nk1 : it) * BK;
                mbar_arrive_expect_tx(&bars->afull[st], halves * kHalfBytes);
                for (int h = 0; h < halves; ++h)
                    tma_load_2d(smem + st * abytes + h * kHalfBytes, map, &bars->afull[st], x, t0 + 256 * h);
            }
            // never leave with copies in flight (bounded even when aborting)
            volatile int no_abort = 0;
            for (int j = 0; j < min(i, depth); ++j) {
                const int i2 = i - 1 - j;
                if (!mbar_wait_short(&bars->afull[i2 % depth], (i2 / depth) & 1u, &no_abort)) {
                    *abort = 1;
                    break;
                }
            }
        }
    } else if (warp == 2) {
        // ------------------------------------------------ TMA: packed words
        if (lane == 0) {
            constexpr int kStep = G::kPairs ? 2 : 1;
            const CUtensorMap* own = MODE == kGated && rank == 1 ? &tmp1 : &tmp0;
            const int row0 = MODE == kGated ? n0 : n0 + 128 * rank;
            int i = 0;
            for (int it = k0; it < k1 && !*abort; it += kStep, ++i) {
                const int ps = i % G::kPStages;
                if (!mbar_wait_short(&bars->pempty[ps], ((i / G::kPStages) & 1u) ^ 1u, abort)) break;
                uint8_t* dst = pbuf + ps * G::kSlot;
                mbar_arrive_expect_tx(&bars->pfull[ps], G::kSlot);
                if constexpr (MODE == kBack) {
                    const bool second = it >= a.nk1;
                    const int row = (second ? it - a.nk1 : it) * BK;
                    constexpr int kBoxCodes = Geom<BITS, MODE>::kBoxCodes, kBoxes = 128 / kBoxCodes;
                    for (int c = 0; c < kBoxes; ++c)
                        tma_load_2d(dst + c * (BK * G::kRowBytes), second ? &tmp1 : &tmp0, &bars->pfull[ps],
                                    (row0 / kBoxCodes + c) * G::kBoxWords, row);
                } else {
                    tma_load_2d(dst, own, &bars->pfull[ps], (it / kStep) * G::kBoxWords, row0);
                }
            }
            volatile int no_abort = 0;
            for (int j = 0; j < min(i, G::kPStages); ++j) {
                const int i2 = i - 1 - j;
                if (!mbar_wait_short(&bars->pfull[i2 % G::kPStages], (i2 / G::kPStages) & 1u, &no_abort)) {
                    *abort = 1;
                    break;
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer (for both CTAs)
        if (lane == 0 && rank == 0) {
            constexpr uint32_t kIdesc = instr_desc(/*bf16*/ 1, /*A K-major*/ 0, /*B*/ MODE == kBack ? 1 : 0, 256, TN);
            bool ok = wait_probe(&bars->never, a.probe_ns, abort);
            for (int i = 0; ok && i < k1 - k0; ++i) {
                const int st = i % depth, b = i % G::kBBufs;
                if (!mbar_wait_short(&bars->afull[st], (i / depth) & 1u, abort) ||
                    !mbar_wait_cluster(&bars->peer[st], (i / depth) & 1u, abort) ||
                    !mbar_wait_cluster(&bars->ready[b], (i / G::kBBufs) & 1u, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t am = smem_u32(smem + st * abytes);
                const uint32_t bm = smem_u32(bbuf + b * kPairBBytes);
                for (int h = 0; h < halves; ++h)
#pragma unroll
                    for (int kk = 0; kk < BK / 16; ++kk) {
                        // as in the single-CTA kernel, each CTA with its 128 rows of both
                        const uint64_t bd = MODE == kBack ? smem_desc(bm + kk * 2048, 8192, 1024, 2)
                                                          : smem_desc(bm + kk * 32, 16, 1024, 2);
                        mma_f16_ss_pair(tmem + h * TN, smem_desc(am + h * kHalfBytes + kk * 32, 16, 1024, 2), bd, kIdesc,
                                        (i > 0 || kk > 0) ? 1u : 0u);
                    }
                mma_commit_pair(&bars->aempty[st]);
                mma_commit_pair(&bars->bempty[b]);
            }
            if (ok) mma_commit_pair(&bars->acc_full);
            mma_commit_pair(&bars->drain);
            volatile int no_abort = 0;
            if (!mbar_wait_short(&bars->drain, 0, &no_abort)) *abort = 1;
        } else if (lane == 0) {
            // rank 1: passes its tokens' arrival on, in order
            bool ok = true;
            for (int i = 0; i < k1 - k0 && ok; ++i) {
                const int st = i % depth;
                ok = mbar_wait_short(&bars->afull[st], (i / depth) & 1u, abort);
                if (ok) mbar_arrive_cluster(&bars->peer[st], 0);
            }
            // the last arrivals that rank 0's MMAs send here have to land before this CTA leaves
            volatile int no_abort = 0;
            if (!mbar_wait_short(&bars->drain, 0, &no_abort)) *abort = 1;
            for (int d = 0; ok && d < depth && d < k1 - k0; ++d) {
                const int i = k1 - k0 - 1 - d;
                mbar_wait_short(&bars->aempty[i % depth], (i / depth) & 1u, abort);
            }
            for (int d = 0; ok && d < G::kBBufs && d < k1 - k0; ++d) {
                const int i = k1 - k0 - 1 - d;
                mbar_wait_short(&bars->bempty[i % G::kBBufs], (i / G::kBBufs) & 1u, abort);
            }
        }
    } else {
        // ------------------------------------------------ dequantize
        const int j = (threadIdx.x - 96) & 127;          // 128 bytes of the CTA's half of the tile,
        const int part = ((threadIdx.x - 96) >> 7) & 1;  // and which 32 of their 64 codes
        const int team = (threadIdx.x - 96) >> 8;
        const int mi = MODE == kGated ? rank : 0;
        const int wrow = n0 + (MODE == kGated ? 0 : 128 * rank) + j;             // forward
        const int kcol = n0 + 128 * rank + 64 * (j >> 6);                        // backward
        const int groups = (a.d_col + a.g - 1) / a.g;
        constexpr int TG = GPT == 1 ? 1 : GPT / 2;                               // groups in 32 codes
        float s[TG] = {}, s_nx[TG];
        int z[TG] = {}, z_nx[TG];
        const int span = GPT == 1 ? a.g / BK : 1;
        int gi = GPT == 1 && MODE != kBack ? (k0 + team) / span : 0, rem = GPT == 1 && MODE != kBack ? (k0 + team) % span : 0;
        const int back_group = GPT == 1 ? kcol / a.g : kcol / 64 * GPT + part * TG;
        auto fetch = [&](int it) {
#pragma unroll
            for (int q = 0; q < TG; ++q) {
                int group, row, m;
                bool in;
                if constexpr (MODE == kBack) {
                    m = it >= a.nk1 ? 1 : 0;
                    row = (m ? it - a.nk1 : it) * BK + (j & 63);
                    group = back_group + q;
                    in = it < k1 && row < a.d_row && kcol < a.d_col;
                } else {
                    m = mi;
                    row = wrow;
                    group = GPT == 1 ? gi : it * GPT + part * TG + q;
                    in = it < k1 && row < a.d_row && group < groups;
                }
                s_nx[q] = 0.f;   // rows and columns past the layer: weights 0
                z_nx[q] = 0;
                if (in) {
                    const int64_t at = static_cast<int64_t>(group) * a.d_row + row;
                    s_nx[q] = __ldg(a.mat[m].scales + at);
                    z_nx[q] = __ldg(a.mat[m].zeros + at);
                }
            }
            if constexpr (GPT == 1 && MODE != kBack) {   // the group of the team's next stage
                rem += kPairTeams;
                while (rem >= span) {
                    rem -= span;
                    ++gi;
                }
            }
        };
        fetch(k0 + team);
        Group<BITS> grp;
        uint32_t dst_off[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) dst_off[c] = j * 128 + (((4 * part + c) ^ (j & 7)) << 4);
        // a lane whose wait runs out stays with its warp, writes what it has and
        // reports nothing more
        bool ok = true;
        for (int it = k0 + team, i = team; it < k1; it += kPairTeams, i += kPairTeams) {
            const int pi = G::kPairs ? i >> 1 : i;
            const int ps = pi % G::kPStages, b = i % G::kBBufs;
#pragma unroll
            for (int q = 0; q < TG; ++q) {
                s[q] = s_nx[q];
                z[q] = z_nx[q];
            }
            fetch(it + kPairTeams);
            if constexpr (TG == 1) grp.set(s[0], static_cast<float>(z[0]));
            ok = ok && mbar_wait_short(&bars->pfull[ps], (pi / G::kPStages) & 1u, abort);
            const uint8_t* src = pbuf + ps * G::kSlot + part * (4 * BITS);
            if constexpr (BITS != 3) {
                src += j * G::kRowBytes;
            } else if constexpr (MODE == kBack) {
                src += (j & 63) * G::kRowBytes + (j >> 6) * (G::kRowBytes / 2);
            } else {
                src += j * G::kRowBytes + (i & 1) * (G::kRowBytes / 2);
            }
            uint32_t w[BITS];
            load_words<BITS>(src, w);
            uint32_t o[4][4];   // wait in registers for their buffer, as above
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if constexpr (TG > 1) {
                    if (c % (4 / TG) == 0) grp.set(s[c / (4 / TG)], static_cast<float>(z[c / (4 / TG)]));
                }
                weights8<BITS>(w, c, grp, o[c]);
            }
            ok = ok && mbar_wait_short(&bars->bempty[b], ((i / G::kBBufs) & 1u) ^ 1u, abort);
            const uint32_t tile_at = smem_u32(bbuf + b * kPairBBytes);
#pragma unroll
            for (int c = 0; c < 4; ++c) sts128_u(tile_at + dst_off[c], make_uint4(o[c][0], o[c][1], o[c][2], o[c][3]));
            fence_async_smem();
            __syncwarp();
            if (lane == 0 && ok) {
                mbar_arrive_cluster(&bars->ready[b], 0);
                mbar_arrive(&bars->pempty[ps]);
            }
        }
        // ------------------------------------------------ drain: tensor memory -> output
        if (warp_agree(ok && mbar_wait_short(&bars->acc_full, 0, abort))) {
            tc_fence_after();
            drain_tile<MODE, kPairDeqWarps>(a, tmem, slot, halves, t0, 256, n0, warp, lane, 128 * rank, smem);
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync_all();   // no CTA leaves while the pair's MMAs or arrivals may touch it
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, kPairTmemCols);
    if (threadIdx.x == 0 && bars->abort) report(a.status, GPTQ_ERR_TIMEOUT);
}

// The split tiles: their parts added in order, then the epilogue.  One thread
// per 16 outputs of a token.
template <int MODE>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ Args a, int split_tiles) {
    constexpr int kOut = MODE == kGated ? TN / 2 : TN;
    __shared__ __align__(16) uint8_t scratch_all[8 * 1024];
    uint8_t* scratch = scratch_all + (threadIdx.x >> 5) * 1024;
    const int64_t per_tile = static_cast<int64_t>(a.part_rows) * (kOut / 16);
    const int64_t total = per_tile * split_tiles;
    // whole warps go round together
    for (int64_t first = blockIdx.x * 256ll + (threadIdx.x & ~31); first < total; first += gridDim.x * 256ll) {
        const int64_t e = first + (threadIdx.x & 31);
        const int i = static_cast<int>(e / per_tile), x = static_cast<int>(e % per_tile);
        const int row = x / (kOut / 16), c = (x % (kOut / 16)) * 16;
        const int tile = a.full + i;
        const int n = (tile % a.tiles_n) * kOut + c;
        const int t = e < total ? (tile / a.tiles_n) * a.tile_tokens + row : a.n_tok;   // (past the end: nothing)
        uint32_t r[8] = {};
        load_residual<MODE>(a, t, n, r, scratch);
        float v[16] = {}, u[16] = {};
        if (valid16(a, t, n) > 0) {
            const float* p = a.part + (static_cast<int64_t>(i) * a.split * a.part_rows + row) * TN + c;
#pragma unroll 4
            for (int k = 0; k < a.split; ++k, p += static_cast<int64_t>(a.part_rows) * TN) {
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const float4 q = __ldcs(reinterpret_cast<const float4*>(p) + y);
                    v[4 * y] += q.x; v[4 * y + 1] += q.y; v[4 * y + 2] += q.z; v[4 * y + 3] += q.w;
                    if constexpr (MODE == kGated) {
                        const float4 w = __ldcs(reinterpret_cast<const float4*>(p + TN / 2) + y);
                        u[4 * y] += w.x; u[4 * y + 1] += w.y; u[4 * y + 2] += w.z; u[4 * y + 3] += w.w;
                    }
                }
            }
        }
        __syncwarp();
        emit16<MODE>(a, t, n, v, u, r, scratch);
    }
}

// Tiles of the output, how many of them run whole, and into how many parts of
// `per` stages each of the others is split.
struct Plan {
    bool pair;      // pairs of CTAs with tiles of 512 tokens
    int tile_tokens, tiles_n, tiles_t, full, split, per, part_rows;
    size_t part_bytes;
};

// Pairs of CTAs from here on.  A pair's stage of 512 tokens takes 0.93 us on two
// SMs, one of up to 256 tokens still 0.8; a single CTA's of 128 takes 0.66, so
// two of those serve 256 tokens better.
constexpr int kPairTokens = 257;

Plan make_plan(int64_t n_tok, int64_t N, int nk, bool gated, bool pairs) {
    Plan p;
    const int out = gated ? TN / 2 : TN;
    p.tiles_n = static_cast<int>((N + out - 1) / out);
    p.pair = n_tok >= kPairTokens;
    p.tile_tokens = p.pair ? PM : TM;
    const int slots = p.pair ? kSms / 2 : kSms;
    p.tiles_t = static_cast<int>((n_tok + p.tile_tokens - 1) / p.tile_tokens);
    const int64_t tiles = static_cast<int64_t>(p.tiles_n) * p.tiles_t;
    p.full = static_cast<int>(tiles);
    p.split = 1;
    p.per = nk;
    p.part_rows = static_cast<int>(n_tok < p.tile_tokens ? n_tok : p.tile_tokens);
    p.part_bytes = 0;
    const int rest = static_cast<int>(tiles % slots);
    int split = rest > 0 ? slots / rest : 1;
    if (split > kMaxSplit) split = kMaxSplit;
    if (split > nk / kMinStages) split = nk / kMinStages;
    if (split > 1) {
        int per = (nk + split - 1) / split;
        if (pairs) per = (per + 1) / 2 * 2;   // a packed slot serves two stages
        split = (nk + per - 1) / per;
        if (split > 1) {
            p.full = static_cast<int>(tiles) - rest;
            p.split = split;
            p.per = per;
            p.part_bytes = static_cast<size_t>(rest) * split * p.part_rows * TN * sizeof(float);
        }
    }
    return p;
}

// Most bytes of partial tiles that any batch of up to n_tok tokens leaves, at
// either kind of packed slot.  They go up and down with the tokens: a part's rows
// grow up to a tile, and how many tiles the last wave holds repeats itself after
// `slots` rows of tiles.
size_t most_part_bytes(int64_t n_tok, int64_t N, int nk, bool gated) {
    size_t most = 0;
    auto take = [&](int64_t n) {
        for (const bool pairs : {false, true}) {
            const size_t b = make_plan(n < n_tok ? n : n_tok, N, nk, gated, pairs).part_bytes;
            if (b > most) most = b;
        }
    };
    for (int64_t n = TM; n - TM < n_tok && n < kPairTokens; n += TM) take(n);
    for (int64_t n = PM; n - PM < n_tok && n <= static_cast<int64_t>(PM) * (kSms / 2 + 1) && n_tok >= kPairTokens; n += PM)
        take(n);
    return most;
}

template <int BITS, int GPT, int MODE>
cudaError_t launch_one(const CUtensorMap (&ta)[2], const CUtensorMap (&tp)[2], const Args& a, int units,
                       cudaStream_t stream) {
    const bool pair = a.tile_tokens == PM;
    auto kern = pair ? pair_gemm_kernel<BITS, GPT, MODE> : packed_gemm_kernel<BITS, GPT, MODE>;
    const int smem = pair ? PairGeom<BITS, MODE>::kSmem : Geom<BITS, MODE>::kSmem;
    static_assert(PairGeom<BITS, MODE>::kSmem <= 227 * 1024 && Geom<BITS, MODE>::kSmem <= 227 * 1024,
                  "shared memory per CTA");
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kern<<<pair ? 2 * units : units, pair ? kPairThreads : kThreads, smem, stream>>>(ta[0], ta[1], tp[0], tp[1], a);
    return cudaGetLastError();
}

template <int BITS, int MODE>
cudaError_t launch_groups(const CUtensorMap (&ta)[2], const CUtensorMap (&tp)[2], const Args& a, int units,
                          cudaStream_t stream) {
    const int g = a.g;
    if (g % 64 == 0 || g >= a.d_col) return launch_one<BITS, 1, MODE>(ta, tp, a, units, stream);
    if (g == 32) return launch_one<BITS, 2, MODE>(ta, tp, a, units, stream);
    if (g == 16) return launch_one<BITS, 4, MODE>(ta, tp, a, units, stream);
    return launch_one<BITS, 8, MODE>(ta, tp, a, units, stream);
}

template <int MODE>
gptq_status run(Args a, const CUtensorMap (&ta)[2], const uint32_t* const (&packed)[2], int bits, bool pairs,
                void* part, int64_t* launches, cudaStream_t stream) {
    const Plan p = make_plan(a.n_tok, a.N, a.nk, MODE == kGated, pairs);
    a.tiles_n = p.tiles_n;
    a.full = p.full; a.split = p.split; a.per = p.per; a.part_rows = p.part_rows;
    a.tile_tokens = p.tile_tokens;
    a.part = static_cast<float*>(part);
    a.probe_ns = take_wait_probe(p.pair ? kProbePair : kProbeSingle);
    const int rest = p.tiles_n * p.tiles_t - p.full;
    const int units = p.full + rest * p.split;
    // the packed words move as raw 32-bit elements (the map's fp32 type only sizes them)
    const uint64_t words = static_cast<uint64_t>(a.d_col) * bits / 32;
    const uint32_t box = static_cast<uint32_t>((bits == 3 ? 128 : 64) * bits / 32);
    CUtensorMap tp[2];
    for (int m = 0; m < 2; ++m)
        if (!make_tmap_2d(&tp[m], false, packed[m], words, a.d_row, words, box, MODE == kBack ? BK : 128, Swz::kNone))
            return GPTQ_ERR_INVALID_ARG;
    cudaError_t e;
    switch (bits) {
        case 2: e = launch_groups<2, MODE>(ta, tp, a, units, stream); break;
        case 3: e = launch_groups<3, MODE>(ta, tp, a, units, stream); break;
        case 4: e = launch_groups<4, MODE>(ta, tp, a, units, stream); break;
        default: e = launch_groups<8, MODE>(ta, tp, a, units, stream); break;
    }
    if (e != cudaSuccess) return GPTQ_ERR_CUDA;
    ++*launches;
    if (rest > 0) {
        const int64_t work = static_cast<int64_t>(rest) * a.part_rows * ((MODE == kGated ? TN / 2 : TN) / 16);
        const int64_t want = (work + 255) / 256;
        join_kernel<MODE><<<static_cast<int>(want < 16 * kSms ? want : 16 * kSms), 256, 0, stream>>>(a, rest);
        if (cudaGetLastError() != cudaSuccess) return GPTQ_ERR_CUDA;
        ++*launches;
    }
    return GPTQ_OK;
}

size_t round256(size_t b) { return (b + 255) / 256 * 256; }

}  // namespace

size_t linear_gemm_workspace_bytes(int64_t n_tok, int64_t d_col, int64_t d_row, bool gated) {
    return round256(most_part_bytes(n_tok, d_row, static_cast<int>(d_col / BK), gated)) +
           round256(static_cast<size_t>(n_tok) * d_col * 2);
}

namespace {
// A call's workspace: its partial tiles, then the gathered tokens.
size_t gemm_part_bytes(const LinearCall& c) {
    return round256(make_plan(c.n_tok, c.d_row, static_cast<int>(c.d_col / BK), c.mat[1].packed != nullptr, c.bits == 3)
                        .part_bytes);
}
}  // namespace

size_t linear_gemm_call_bytes(const LinearCall& c) {
    return gemm_part_bytes(c) +
           (needs_gather(c.X, c.ldx, c.perm) ? round256(static_cast<size_t>(c.n_tok) * c.d_col * 2) : 0);
}

gptq_status launch_linear_gemm(const LinearCall& c, cudaStream_t stream) {
    const bool gated = c.mat[1].packed != nullptr;
    int64_t launches = 0;
    const uint16_t* A = c.X;
    int64_t lda = c.ldx;
    if (needs_gather(c.X, c.ldx, c.perm)) {
        uint16_t* xq = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(c.ws) + gemm_part_bytes(c));
        if (launch_gather_bf16(c.X, c.ldx, c.n_tok, static_cast<int>(c.d_col), c.perm, xq, stream) != cudaSuccess)
            return GPTQ_ERR_CUDA;
        A = xq;
        lda = c.d_col;
        ++launches;
    }
    CUtensorMap ta[2];
    if (!make_tmap_2d(&ta[0], true, A, c.d_col, c.n_tok, lda, BK, 128, Swz::k128)) return GPTQ_ERR_INVALID_ARG;
    ta[1] = ta[0];
    Args a = {};
    a.mat[0] = c.mat[0];
    a.mat[1] = c.mat[1];
    a.n_tok = static_cast<int>(c.n_tok);
    a.N = static_cast<int>(c.d_row);
    a.d_row = static_cast<int>(c.d_row);
    a.d_col = static_cast<int>(c.d_col);
    a.nk = a.nk1 = a.d_col / BK;
    a.g = (c.group == -1 || c.group > a.d_col) ? a.d_col : c.group;
    a.bias = c.bias;
    a.act = c.act;
    a.residual = c.residual; a.ldr = c.ldr;
    for (int m = 0; m < 2; ++m) {
        a.pre[m] = c.pre[m];
        a.ldpre[m] = c.ldpre[m];
    }
    a.Y = c.Y; a.ldy = c.ldy;
    a.status = c.status;
    const uint32_t* packed[2] = {c.mat[0].packed, gated ? c.mat[1].packed : c.mat[0].packed};
    const gptq_status s = gated ? run<kGated>(a, ta, packed, c.bits, c.bits == 3, c.ws, &launches, stream)
                                : run<kLinear>(a, ta, packed, c.bits, c.bits == 3, c.ws, &launches, stream);
    count_launches(launches);
    return s;
}

// ---- gradients: the slopes (linear_backward.cu), then dXq = dP W here, then
// the columns back in the input's order.
namespace {
int back_stages(int64_t d_row, bool gated) { return static_cast<int>((d_row + BK - 1) / BK) * (gated ? 2 : 1); }

// A call's workspace: its partial tiles, the partial bias gradients, dXq (with a
// permutation).
struct BackwardSpace {
    size_t at_bias, at_dxq, total;
};
BackwardSpace backward_space(const BackwardCall& c) {
    const Plan p = make_plan(c.n_tok, c.d_col, back_stages(c.d_row, c.mat[1].packed != nullptr), false, false);
    BackwardSpace w;
    w.at_bias = round256(p.part_bytes);
    w.at_dxq = w.at_bias + (c.dbias != nullptr ? round256(bias_partial_bytes(c.n_tok, c.d_row)) : 0);
    w.total = w.at_dxq + (c.perm != nullptr ? round256(static_cast<size_t>(c.n_tok) * c.d_col * 2) : 0);
    return w;
}
}  // namespace

size_t linear_backward_workspace_bytes(int64_t n_tok, int64_t d_col, int64_t d_row, bool gated) {
    return round256(most_part_bytes(n_tok, d_col, back_stages(d_row, gated), false)) +
           (gated ? 0 : round256(most_bias_partial_bytes(n_tok, d_row))) +
           round256(static_cast<size_t>(n_tok) * d_col * 2);
}

size_t linear_backward_call_bytes(const BackwardCall& c) { return backward_space(c).total; }

gptq_status launch_linear_backward(const BackwardCall& c, cudaStream_t stream) {
    const bool gated = c.mat[1].packed != nullptr;
    int64_t launches = 0;
    uint8_t* ws = static_cast<uint8_t*>(c.ws);
    const BackwardSpace w = backward_space(c);
    float* bias_part = c.dbias == nullptr ? nullptr : reinterpret_cast<float*>(ws + w.at_bias);
    uint16_t* dxq = c.perm == nullptr ? nullptr : reinterpret_cast<uint16_t*>(ws + w.at_dxq);
    gptq_status s = launch_slopes(c, bias_part, &launches, stream);
    if (s != GPTQ_OK) return s;
    CUtensorMap ta[2];
    for (int m = 0; m < 2; ++m) {
        // the gradient of the products: dPre / dGate, dUp, or dY itself
        const int k = gated ? m : 0;
        const uint16_t* D = c.dP[k] != nullptr ? c.dP[k] : c.dY;
        const int64_t ld = c.dP[k] != nullptr ? c.lddp[k] : c.lddy;
        if (!make_tmap_2d(&ta[m], true, D, c.d_row, c.n_tok, ld, BK, 128, Swz::k128)) return GPTQ_ERR_INVALID_ARG;
    }
    Args a = {};
    a.mat[0] = c.mat[0];
    a.mat[1] = gated ? c.mat[1] : c.mat[0];
    a.n_tok = static_cast<int>(c.n_tok);
    a.N = a.d_col = static_cast<int>(c.d_col);
    a.d_row = static_cast<int>(c.d_row);
    a.nk = back_stages(c.d_row, gated);
    a.nk1 = back_stages(c.d_row, false);
    a.g = (c.group == -1 || c.group > a.d_col) ? a.d_col : c.group;
    a.Y = c.perm != nullptr ? dxq : c.dX;
    a.ldy = c.perm != nullptr ? c.d_col : c.lddx;
    a.status = c.status;
    const uint32_t* packed[2] = {a.mat[0].packed, a.mat[1].packed};
    s = run<kBack>(a, ta, packed, c.bits, false, ws, &launches, stream);
    if (s == GPTQ_OK && c.perm != nullptr) {
        s = launch_scatter(dxq, c.n_tok, static_cast<int>(c.d_col), c.perm, c.dX, c.lddx, stream);
        ++launches;
    }
    count_launches(launches);
    return s;
}

}  // namespace gptq
