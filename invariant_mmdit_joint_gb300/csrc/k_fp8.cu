// Projections in 8-bit floating point: rows rounded to codes of 8 bits (e4m3
// or e5m2) with one power-of-two scale for each 128 of them, and the product of
// two such operands.
//
//   quantise   block of 128 along a row (or 128 x 128): scale 2^e, e the
//              smallest (>= -126) with max |x| <= 448 * 2^e (57344 for e5m2);
//              code = x * 2^-e rounded to nearest, ties to even. Powers of two
//              lose nothing but the code's own rounding, and are what the tensor
//              core's block scale takes (one byte, e + 127).
//   product    d[t, f] = sum_k a[t, k] b[f, k] (+ bias[f]): K in chunks of 512
//              (4 blocks), a chunk's sum in the tensor core's fp32 accumulator,
//              the chunks added in ascending order in fp32, one rounding of d.
//
// fp8_quant_kernel: one CTA per 128 x 128 tile of x, read once; writes the codes
// of its rows' blocks, of its columns' blocks (the transposed operand that a sum
// over rows needs), or both, and the columns' sums (a bias gradient).
// fp8_quant_rows_kernel: the rows' blocks alone. Both bound by HBM.
//
// The products: tcgen05.mma kind::mxf8f6f4 with block scales. The features (b's
// rows) are the rows of an accumulator, the tokens (a's rows) its columns, so
// that a call with few tokens takes a narrow accumulator and reads each weight
// once. Warps: 0 TMA producer, 1 MMA issuer and TMEM owner (the whole warp runs
// the loop, one elected lane issues: in a loop of one lane the operands are moved
// to uniform registers one by one, which took as long as the products), 2 scale
// loader (gathers four blocks' bytes a row into the 128 x 4 layout that tcgen05.cp
// spreads over TMEM), 4 .. 11 the sums of the chunks and the output. Every
// accumulator starts a chunk anew; the chunks meet in fp32 registers or shared
// memory, always in ascending order: a token's bytes do not depend on the kernel
// that computed them. Every wait is bounded. A kernel that starts early (griddepcontrol) is alive while the one before
// it writes what it reads: its loads are ordinary ones, which the wait orders; read-only loads (ld.global.nc) are for
// memory that nobody writes while the kernel lives.
//   fp8_gemm_pair_kernel  CTA pairs, 256 features x 224 tokens: 3.1 PFLOP/s (8704
//       tokens, 2560 -> 7680: 110 us); without the output 3.9. Bound by the tensor
//       pipe (76% active), and by shared memory's port while the output passes.
//   fp8_gemm_few_kernel   up to 64 tokens, 128 features x 16 or 64 tokens, the chunks
//       shared out over a cluster. Bound by latency: launch, first loads, join.
#include "rlk_device.cuh"
#include "rlk_internal.h"
#include "rlk_sm100.cuh"
#include "rlk_tmap.h"

#include <algorithm>
#include <atomic>

RLK_DEFINE_STRICT_PROBE(probe_fp8_tu)

namespace rlk {
namespace {

using namespace sm100;

// ------------------------------------------------------------------ quantise
constexpr int kTile = 128;          // rows and columns of a quantise CTA
constexpr int kQuantThreads = 256;  // 16 row groups x 16 column groups of 8
constexpr int kRowsTile = 64;       // rows of a CTA of the kernel for blocks along rows alone

struct QuantItem {
    const void* x;
    uint8_t *q, *q_scale, *qt, *qt_scale;
    float* part;  // column sums of each row tile [row_tiles, cols], or null
    long long x_stride;
    int rows, cols, ldq, lds, ldqt, ldst;
    int col_tiles, tile0;  // tiles of the item: tile0 + row tile * col_tiles + column tile
    bool square;
};
struct QuantArgs {
    QuantItem item[kFp8MaxItems];
    int n;
};

// Exponent of the block's scale: the smallest e >= -126 with top <= 1.75 * 2^(e + room).
__device__ __forceinline__ int scale_exponent(float top, int room) {
    const int e = (int)((__float_as_uint(top) + 0x1FFFFFu) >> 23) - 127 - room;
    return max(e, -126);
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

template <bool kE5m2>
__device__ __forceinline__ uint32_t code2(float lo, float hi) {  // two codes, lo in the low byte
    uint16_t r;
    if (kE5m2)
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
template <bool kE5m2>
__device__ __forceinline__ uint2 code8(const float (&v)[8]) {
    return make_uint2(code2<kE5m2>(v[0], v[1]) | code2<kE5m2>(v[2], v[3]) << 16,
                      code2<kE5m2>(v[4], v[5]) | code2<kE5m2>(v[6], v[7]) << 16);
}

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {  // of magnitudes; passes over NaN
    const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
}

// Eight neighbouring values of a row as they are stored: 16 bytes of bf16, 32 of fp32.
template <bool kFp32>
struct Eight {
    uint32_t w[kFp32 ? 8 : 4];
    __device__ __forceinline__ void load(const void* x, long long at) {
        if (kFp32) {
            const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(x) + at);
            const uint4 a = p[0], b = p[1];
            w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
            w[kFp32 ? 4 : 0] = b.x, w[kFp32 ? 5 : 1] = b.y, w[kFp32 ? 6 : 2] = b.z, w[kFp32 ? 7 : 3] = b.w;
        } else {
            const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at);
            w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (uint32_t& k : w) k = 0;
    }
    __device__ __forceinline__ float get(int j) const {
        return kFp32 ? __uint_as_float(w[kFp32 ? j : 0]) : (j & 1) ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1]);
    }
    // Largest magnitude but for NaN. An infinity takes the code of NaN and no part in its block's scale: it is made
    // a NaN here, before anything else looks at it.
    __device__ __forceinline__ float top() {
        float m = top_once();
        if (m == INFINITY) {
            if (kFp32) {
#pragma unroll
                for (uint32_t& k : w)
                    if ((k & 0x7fffffffu) == 0x7f800000u) k = 0x7fffffffu;
            } else {
#pragma unroll
                for (uint32_t& k : w) {
                    if ((k & 0x7fffu) == 0x7f80u) k |= 0x7fffu;
                    if ((k & 0x7fff0000u) == 0x7f800000u) k |= 0x7fff0000u;
                }
            }
            m = top_once();
        }
        return m;
    }

   private:
    __device__ __forceinline__ float top_once() const {
        if (kFp32) {
            float m = 0.0f;
#pragma unroll
            for (const uint32_t k : w) m = fmaxf(m, fabsf(__uint_as_float(k)));
            return m;
        }
        uint32_t m = w[0] & 0x7fff7fffu;
#pragma unroll
        for (int k = 1; k < 4; ++k) m = max_bf16x2(m, w[k] & 0x7fff7fffu);
        return fmaxf(fmaxf(bf16_lo(m), bf16_hi(m)), 0.0f);
    }
};

template <bool kFp32, bool kE5m2>
__device__ __forceinline__ uint2 codes_of(const Eight<kFp32>& v, float s) {
    const uint64_t s2 = f2_pack(s, s);
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; j += 2) f2_unpack(mul_f2(f2_pack(v.get(j), v.get(j + 1)), s2), y[j], y[j + 1]);
    return code8<kE5m2>(y);
}

__device__ __forceinline__ const QuantItem& item_of(const QuantArgs& a, int& tile) {
    int i = 0;
    while (i + 1 < a.n && (int)blockIdx.x >= a.item[i + 1].tile0) ++i;
    tile = blockIdx.x - a.item[i].tile0;
    return a.item[i];
}

// Blocks along the rows alone: 8 lanes a block, each with two runs of eight columns; two rows a thread, no shared memory
// (bound by instructions: 16 lanes with one run each and the same work beside it took 13.5 of them a value and 14.0 us
// for 8704 rows of 2560; 12.0 so, HBM's floor 9.9).
template <bool kFp32, bool kE5m2>
__global__ void __launch_bounds__(kQuantThreads) fp8_quant_rows_kernel(const __grid_constant__ QuantArgs a) {
    constexpr int kRoom = kE5m2 ? 15 : 8, kRows = kRowsTile / 32;
    asm volatile("griddepcontrol.launch_dependents;");  // (the product of few tokens starts on its weights)
    int tile;
    const QuantItem& it = item_of(a, tile);
    const int cg = threadIdx.x & 7, rg = threadIdx.x >> 3;
    const int r0 = (tile / it.col_tiles) * kRowsTile + rg, block = tile % it.col_tiles, col = block * kTile + 8 * cg;
    const bool near = col < it.cols, far = col + 64 < it.cols;
    Eight<kFp32> v[kRows][2];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const bool live = r0 + 32 * i < it.rows;
        const long long at = (long long)(r0 + 32 * i) * it.x_stride + col;
        if (live && near)
            v[i][0].load(it.x, at);
        else
            v[i][0].clear();
        if (live && far)
            v[i][1].load(it.x, at + 64);
        else
            v[i][1].clear();
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        float m = fmaxf(v[i][0].top(), v[i][1].top());
#pragma unroll
        for (int k = 4; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
        const int row = r0 + 32 * i, e = scale_exponent(m, kRoom);
        if (row >= it.rows) continue;
        const float s = power_of_two(-e);
        uint8_t* const q = it.q + (long long)row * it.ldq + col;
        if (near) *reinterpret_cast<uint2*>(q) = codes_of<kFp32, kE5m2>(v[i][0], s);
        if (far) *reinterpret_cast<uint2*>(q + 64) = codes_of<kFp32, kE5m2>(v[i][1], s);
        if (cg == 0) it.q_scale[(long long)row * it.lds + block] = (uint8_t)(e + 127);
    }
}

struct QuantSmem {
    float row_top[kTile];
    float col[16][kTile];  // the row groups' column maxima, then their column sums
    float col_top[kTile];
    uint8_t t[kTile * kTile];  // codes of columns: 128 bytes a column, 8-byte chunk g at g ^ (column / 8)
};

// Blocks along the columns (and along the rows, or of 128 x 128), column sums: a 128 x 128 tile a CTA, eight rows of
// eight columns a thread, kept as they were loaded (8704 x 2560 both ways: 18.8 us cold, HBM's floor
// 13.2; 65% of the issue slots).
template <bool kFp32, bool kE5m2>
__global__ void __launch_bounds__(kQuantThreads) fp8_quant_kernel(const __grid_constant__ QuantArgs a) {
    __shared__ __align__(16) QuantSmem sm;
    constexpr int kRoom = kE5m2 ? 15 : 8;
    asm volatile("griddepcontrol.launch_dependents;");
    int tile;
    const QuantItem& it = item_of(a, tile);
    const int tid = threadIdx.x, lane = tid & 31;
    const int cg = tid & 15, rg = tid >> 4;
    const int r0 = (tile / it.col_tiles) * kTile, c0 = (tile % it.col_tiles) * kTile;
    const int col = c0 + 8 * cg;
    const bool col_live = col < it.cols, sums = it.part != nullptr;
    Eight<kFp32> v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = r0 + 8 * rg + i;
        if (row < it.rows && col_live)
            v[i].load(it.x, (long long)row * it.x_stride + col);
        else
            v[i].clear();
    }
    float sum[8];
    if (sums) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            sum[j] = v[0].get(j);
#pragma unroll
            for (int i = 1; i < 8; ++i) sum[j] += v[i].get(j);
        }
    }
    float tops[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) tops[i] = v[i].top();
    // rows over their 16 lanes, halves traded: lane k of a group ends with row k / 2
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool up = lane & 8;
        const float give = up ? tops[i] : tops[i + 4], keep = up ? tops[i + 4] : tops[i];
        tops[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, 8));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const bool up = lane & 4;
        const float give = up ? tops[i] : tops[i + 2], keep = up ? tops[i + 2] : tops[i];
        tops[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, 4));
    }
    {
        const bool up = lane & 2;
        const float give = up ? tops[0] : tops[1], keep = up ? tops[1] : tops[0];
        tops[0] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, 2));
        tops[0] = fmaxf(tops[0], __shfl_xor_sync(0xffffffffu, tops[0], 1));
    }
    if ((lane & 1) == 0) sm.row_top[8 * rg + ((lane & 15) >> 1)] = tops[0];
    if (!it.square) {
        if (kFp32) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float m = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i].get(j)));
                sm.col[rg][8 * cg + j] = m;
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t m = 0;  // (zero magnitudes: NaN never stays)
#pragma unroll
                for (int i = 0; i < 8; ++i) m = max_bf16x2(m, v[i].w[k] & 0x7fff7fffu);
                *reinterpret_cast<float2*>(&sm.col[rg][8 * cg + 2 * k]) = make_float2(bf16_lo(m), bf16_hi(m));
            }
        }
    }
    __syncthreads();
    if (it.square) {  // one scale for the tile
        if (tid < 32) {
            float m = fmaxf(fmaxf(sm.row_top[lane], sm.row_top[lane + 32]), fmaxf(sm.row_top[lane + 64], sm.row_top[lane + 96]));
#pragma unroll
            for (int k = 16; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
            __syncwarp();
            for (int k = 0; k < 4; ++k) sm.row_top[lane + 32 * k] = sm.col_top[lane + 32 * k] = m;
        }
    } else if (tid < kTile) {
        float m = sm.col[0][tid];
#pragma unroll
        for (int k = 1; k < 16; ++k) m = fmaxf(m, sm.col[k][tid]);
        sm.col_top[tid] = m;
    }
    __syncthreads();
    if (sums) {
#pragma unroll
        for (int j = 0; j < 8; ++j) sm.col[rg][8 * cg + j] = sum[j];
    }
    if (it.q != nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = r0 + 8 * rg + i;
            const float s = power_of_two(-scale_exponent(sm.row_top[8 * rg + i], kRoom));
            if (row < it.rows && col_live)
                *reinterpret_cast<uint2*>(it.q + (long long)row * it.ldq + col) = codes_of<kFp32, kE5m2>(v[i], s);
        }
        if (tid < kTile && r0 + tid < it.rows)
            it.q_scale[(long long)(r0 + tid) * it.lds + c0 / kTile] = (uint8_t)(scale_exponent(sm.row_top[tid], kRoom) + 127);
    }
    if (it.qt != nullptr) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float s = power_of_two(-scale_exponent(sm.col_top[8 * cg + j], kRoom));
            const uint64_t s2 = f2_pack(s, s);
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; i += 2) f2_unpack(mul_f2(f2_pack(v[i].get(j), v[i + 1].get(j)), s2), y[i], y[i + 1]);
            *reinterpret_cast<uint2*>(sm.t + (8 * cg + j) * kTile + ((rg ^ cg) << 3)) = code8<kE5m2>(y);
        }
        if (tid < kTile && c0 + tid < it.cols)
            it.qt_scale[(long long)(c0 + tid) * it.ldst + r0 / kTile] = (uint8_t)(scale_exponent(sm.col_top[tid], kRoom) + 127);
    }
    __syncthreads();
    if (it.qt != nullptr) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = tid + k * kQuantThreads, c = i >> 3, g = i & 7, x = c >> 3;
            uint4 w = *reinterpret_cast<const uint4*>(sm.t + c * kTile + (((2 * g) ^ (x & ~1)) << 3));
            if (x & 1) w = make_uint4(w.z, w.w, w.x, w.y);
            // (a row's codes past it.rows are zeros, up to the row's padded length)
            if (c0 + c < it.cols && r0 + 16 * g < it.rows)
                *reinterpret_cast<uint4*>(it.qt + (long long)(c0 + c) * it.ldqt + r0 + 16 * g) = w;
        }
    }
    if (sums && tid < kTile && c0 + tid < it.cols) {
        float a = sm.col[0][tid];
#pragma unroll
        for (int k = 1; k < 16; ++k) a += sm.col[k][tid];
        it.part[(long long)(r0 / kTile) * it.cols + c0 + tid] = a;
    }
}

// A launch that may set itself up while the one before it ends: its kernel waits (griddepcontrol.wait) before it reads
// or writes. The kernels that round are launched plainly (so launched they took SMs from the products before them: a
// training step at 1024^2 447 -> 477 us).
template <typename Args>
cudaError_t launch_after(void (*kernel)(Args), int grid, int threads, int smem, cudaStream_t s, const Args& a) {
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)grid);
    c.blockDim = dim3((unsigned)threads);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    c.attrs = &attr;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, a);
}

struct FoldItem {
    const float* part;
    float* out;
    int tiles, cols, block0;
};
struct FoldArgs {
    FoldItem item[kFp8MaxItems];
    int n;
};
constexpr int kFoldThreads = 256, kFoldCols = 32, kFoldRuns = kFoldThreads / kFoldCols;

// Column sums: every 8th row tile in ascending order, then these 8 runs.
__global__ void __launch_bounds__(kFoldThreads) fp8_fold_kernel(const __grid_constant__ FoldArgs a) {
    __shared__ float sm[kFoldRuns][kFoldCols];
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int i = 0;
    while (i + 1 < a.n && (int)blockIdx.x >= a.item[i + 1].block0) ++i;
    const FoldItem& it = a.item[i];
    const int cc = threadIdx.x % kFoldCols, run = threadIdx.x / kFoldCols;
    const int c = (blockIdx.x - it.block0) * kFoldCols + cc;
    float s = 0.0f;
    if (c < it.cols) {
        const float* p = it.part + c;
#pragma unroll 4
        for (int t = run; t < it.tiles; t += kFoldRuns) s += p[(long long)t * it.cols];
    }
    sm[run][cc] = s;
    __syncthreads();
    if (run > 0 || c >= it.cols) return;
#pragma unroll
    for (int k = 1; k < kFoldRuns; ++k) s += sm[k][cc];
    it.out[c] = s;
}

// ------------------------------------------------------------------ product
constexpr int kBK = 128;        // bytes of a row in a stage: one scale block
constexpr int kChunkBlocks = 4; // blocks whose products share an accumulator
constexpr int kFBytes = 128 * kBK;
constexpr int kThreads = 384;
constexpr int kWarpTma = 0, kWarpMma = 1, kWarpScale = 2, kWarpEpilogue = 4;
constexpr int kScaleRing = 6;  // chunks whose scales are at hand: gathering one takes longer than its products
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kWaitLimitNs = 2000000000ull;

__device__ int g_status_fp8;

// A call with few tokens: NT columns (16 or 64) of an accumulator for each chunk of K, all at hand until the end. kRaw:
// the tokens come as bf16 rows and are rounded here, by the warps that have nothing to do until then.
template <int NT, bool kRaw>
struct Few {
    static constexpr int kStageBytes = kFBytes + (kRaw ? 0 : NT * kBK);
    static constexpr int kStages = NT == 16 ? 5 : 4;
    static constexpr int kSlots = kRaw ? 3 : NT == 16 ? 11 : 3;  // chunks a CTA takes
    static constexpr int kScaleCol = kSlots * NT;               // two sets of 8 columns, 16 apart
    static constexpr uint32_t kTmemCols = 256;                  // two CTAs an SM
    static constexpr int kSumBytes = 128 * NT * 4;              // a chunk's sums, in the stages' place when these are done
    static constexpr int kSumsBytes = kSlots * kSumBytes > kStages * kStageBytes ? kSlots * kSumBytes : kStages * kStageBytes;
    static constexpr int kTokenBytes = kRaw ? kSlots * kChunkBlocks * NT * kBK : 0;  // their codes, for all of the CTA's K
    static constexpr int kSmemBytes = kSumsBytes + kTokenBytes + kSlots * 1024 + 1024;
    // (a third CTA on an SM would wait for TMEM, perhaps while its cluster waits for it)
    static_assert(kScaleCol + 32 <= (int)kTmemCols && 2 * kSmemBytes <= 226 * 1024 && 3 * kSmemBytes > 228 * 1024, "");
};

struct GemmItem {
    CUtensorMap map_f, map_t;  // features [n, k], box 128 x 128; tokens [m, k], box 128 x NT (a pair's CTA: half)
    CUtensorMap map_d;         // pairs: d [m, n], box of 32 features
    const uint8_t *sf, *st;
    const uint16_t* bias;
    const void* rows;  // bf16 tokens [m, k] to be rounded (few tokens), or null
    void* d;
    long long d_stride;
    int k, ldsf, ldst, m, n, blocks, tiles_f, tile0;
    uint32_t idesc;  // formats of the operands
    bool fp32, accumulate;
};
struct GemmArgs {
    GemmItem item[kFp8MaxItems];
    int n, tiles, ctas;  // ctas: of a cluster that shares K out (few tokens)
};

// Instruction descriptor of kind::mxf8f6f4 with e8m0 scales, without the
// formats and the scale bytes' places.
constexpr uint32_t idesc_mx(int M, int N) {
    return (1u << 23) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// D[tmem] (+)= (A * 2^sa)[smem] * (B * 2^sb)[smem]; A, B 8-bit, K = 32, one scale a row.
__device__ __forceinline__ void mma_mx(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t sa,
                                       uint32_t sb, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(
            d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_mx_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t sa,
                                            uint32_t sb, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(
            d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
}
// 32 rows of 16 bytes from shared memory to 4 TMEM columns, repeated in every lane quarter.
__device__ __forceinline__ void tmem_copy_scales(uint32_t taddr, uint64_t sdesc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n" ::"r"(taddr), "l"(sdesc) : "memory");
}
__device__ __forceinline__ void tmem_copy_scales_pair(uint32_t taddr, uint64_t sdesc) {  // in both CTAs
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n" ::"r"(taddr), "l"(sdesc) : "memory");
}
__device__ __forceinline__ void fail(volatile int* abort_flag) {
    *abort_flag = 1;
    atomicOr(&g_status_fp8, 1);
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, kWaitLimitNs));
}

__device__ __forceinline__ bool warp_wait_cluster(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    return __all_sync(0xffffffffu, mbar_wait_cluster(bar, parity, abort_flag, kWaitLimitNs));
}

struct TileAt {
    int item, f0, t0;
};
// A lane's four rows' scale words of atom i (0 features, then tokens) from block kb on.
__device__ __forceinline__ void gather_scales(uint32_t (&w)[4], const GemmItem& g, int i, const TileAt& at, int kb, int lane) {
    const int r0 = i == 0 ? at.f0 : at.t0 + 128 * (i - 1), rows = i == 0 ? g.n : g.m;
    const uint8_t* p = i == 0 ? g.sf : g.st;
    const int ld = i == 0 ? g.ldsf : g.ldst;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int r = r0 + 32 * c + lane;
        w[c] = r < rows ? *reinterpret_cast<const uint32_t*>(p + (long long)r * ld + kb) : 0x7f7f7f7fu;
    }
}
__device__ __forceinline__ void put_scales(uint32_t dst, const uint32_t (&w)[4]) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
}
// A chunk's sums from TMEM, added to those of the chunks before: 32 columns a wait, the last 16 by themselves.
template <int kHalf>
__device__ __forceinline__ void add_chunk(float (&acc)[kHalf], uint32_t taddr, bool first) {
#pragma unroll
    for (int c = 0; c + 32 <= kHalf; c += 32) {
        uint32_t r[32];
        tmem_ld32(taddr + c, r);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) acc[c + i] = first ? __uint_as_float(r[i]) : acc[c + i] + __uint_as_float(r[i]);
    }
    if (kHalf % 32 != 0) {
        constexpr int c = kHalf / 32 * 32;
        uint32_t r[16];
        tmem_ld16(taddr + c, r);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[c + i] = first ? __uint_as_float(r[i]) : acc[c + i] + __uint_as_float(r[i]);
    }
}

// Allows a kernel its shared memory, at its first launch on a device.
template <auto kKernel>
cudaError_t smem_once(int bytes) {
    static std::atomic<uint64_t> done;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && (done.load() >> dev & 1) != 0)) return e;
    e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kKernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (e == cudaSuccess && dev < 64) done |= 1ull << dev;
    return e;
}

// ---- few tokens ----
__device__ __forceinline__ float4 load_cluster(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// 128 features x NT tokens a cluster, the chunks of K shared out over its CTAs (rank r: chunks r * share ..), so that a
// few tokens' weights stream through many SMs. Each CTA leaves its chunks' sums in shared memory; then each adds up a
// part of the features over all chunks in ascending order: the sums and bytes of any other number of CTAs or tokens.
// Before it waits for the kernel that rounds the tokens, a CTA has its weights fetched to L2.
// (16 bf16 tokens rounded here: one launch for two.)
template <int NT, bool kRaw>
__global__ void __launch_bounds__(kThreads, 2) fp8_gemm_few_kernel(const __grid_constant__ GemmArgs a) {
    using C = Few<NT, kRaw>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * C::kStages + C::kSlots + 1];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;

    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int ctas = a.ctas, rank = blockIdx.x % ctas, t = blockIdx.x / ctas;
    int item = 0;
    while (item + 1 < a.n && t >= a.item[item + 1].tile0) ++item;
    const GemmItem& g = a.item[item];
    TileAt at;
    at.item = item;
    at.f0 = (t - g.tile0) % g.tiles_f * 128;
    at.t0 = (t - g.tile0) / g.tiles_f * NT;
    const int chunks = (g.blocks + kChunkBlocks - 1) / kChunkBlocks, share = (chunks + ctas - 1) / ctas;
    const int c0 = min(rank * share, chunks), n_chunks = min(share, chunks - c0);
    const int b0 = c0 * kChunkBlocks, n_blocks = min(g.blocks - min(b0, g.blocks), n_chunks * kChunkBlocks);

    const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
    auto stage_f = [&](int st) { return sbase + st * C::kStageBytes; };
    auto stage_t = [&](int st) { return sbase + st * C::kStageBytes + kFBytes; };
    const uint32_t tokens = sbase + C::kSumsBytes, scales = tokens + C::kTokenBytes;
    const uint32_t bar_full = smem_u32(&bars[0]), bar_empty = bar_full + 8 * C::kStages;
    const uint32_t bar_scale = bar_empty + 8 * C::kStages, bar_acc = bar_scale + 8 * C::kSlots;

    if (tid == 0) {
        abort_flag = 0;
        for (int i = 0; i < C::kStages; ++i) mbar_init(bar_full + 8 * i, 1), mbar_init(bar_empty + 8 * i, 1);
        for (int i = 0; i < C::kSlots; ++i) mbar_init(bar_scale + 8 * i, kRaw ? 9 : 1);
        mbar_init(bar_acc, 1);
        fence_barrier_init();
    }
    if (warp == kWarpMma) {
        tmem_alloc(smem_u32(&tmem_slot), C::kTmemCols);
        tmem_relinquish();
    }
    if (warp == kWarpTma && lane == 0)
        for (int kb = 0; kb < n_blocks; ++kb)
            asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(&g.map_f)),
                         "r"((b0 + kb) * kBK), "r"(at.f0)
                         : "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;

    if (warp == kWarpTma) {
        if (lane == 0) {
            bool ok = true;
            int it = 0;
            for (; it < n_blocks; ++it) {
                const int st = it % C::kStages;
                const uint32_t use = it / C::kStages;
                if (use > 0 && !mbar_wait(bar_empty + 8 * st, (use - 1) & 1, &abort_flag, kWaitLimitNs)) {
                    ok = false;
                    break;
                }
                mbar_expect_tx(bar_full + 8 * st, C::kStageBytes);
                tma_load_2d(stage_f(st), &g.map_f, bar_full + 8 * st, (b0 + it) * kBK, at.f0);
                if (!kRaw) tma_load_2d(stage_t(st), &g.map_t, bar_full + 8 * st, (b0 + it) * kBK, at.t0);
            }
            if (!ok) fail(&abort_flag);
            for (int u = max(0, it - C::kStages); u < it; ++u)
                mbar_wait_drain(bar_full + 8 * (u % C::kStages), (u / C::kStages) & 1, kWaitLimitNs);
        }
    } else if (warp == kWarpMma) {
        const uint64_t f0 = sdesc_sw128(stage_f(0), 16, 1024), t0 = sdesc_sw128(kRaw ? tokens : stage_t(0), 16, 1024);
        const uint64_t s0 = sdesc_noswizzle(scales, 0, 128);
        uint32_t st = 0, phase = 0;
        bool ok = true;
        for (int c = 0; ok && c < n_chunks; ++c) {
            if (!warp_wait(bar_scale + 8 * c, 0, &abort_flag)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t sa = tmem + C::kScaleCol + (c & 1) * 16, sb = sa + 4, acc = tmem + c * NT;
            if (elect_one()) {
                tmem_copy_scales(sa, s0 + (c * 1024 >> 4));
                tmem_copy_scales(sb, s0 + ((c * 1024 + 512) >> 4));
            }
            const int n = min(kChunkBlocks, n_blocks - c * kChunkBlocks);
            uint32_t id = g.idesc;
            for (int kb = 0; kb < n; ++kb) {
                if (!warp_wait(bar_full + 8 * st, phase, &abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t f = f0 + st * (C::kStageBytes >> 4);
                const uint64_t tk = t0 + (kRaw ? (c * kChunkBlocks + kb) * (NT * kBK >> 4) : st * (C::kStageBytes >> 4));
                if (elect_one()) {
#pragma unroll
                    for (int j = 0; j < kBK / 32; ++j) mma_mx(acc, f + 2 * j, tk + 2 * j, id, sa, sb, j > 0 || kb > 0 ? 1u : 0u);
                    mma_commit(bar_empty + 8 * st);
                }
                if (++st == C::kStages) st = 0, phase ^= 1;
                id += (1u << 29) | (1u << 4);  // the next block's scale bytes
            }
        }
        if (elect_one()) {
            if (!ok) fail(&abort_flag);
            mma_commit(bar_acc);
        }
    } else if (warp == kWarpScale) {
        for (int c = 0; c < n_chunks; ++c) {
            uint32_t w[2][4];
#pragma unroll
            for (int i = 0; i < (kRaw ? 1 : 2); ++i) gather_scales(w[i], g, i, at, b0 + c * kChunkBlocks, lane);
#pragma unroll
            for (int i = 0; i < (kRaw ? 1 : 2); ++i) put_scales(scales + c * 1024 + 512 * i + 16 * lane, w[i]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_scale + 8 * c);
        }
    } else if (kRaw && warp >= kWarpEpilogue) {
        // two tokens a warp, 16 lanes each: a block's 128 values to codes at once, a chunk's four loaded together
        const bool e5m2 = g.idesc >> 10 & 1;
        const int row = 2 * (warp - kWarpEpilogue) + (lane >> 4), cg = lane & 15;
        for (int c = 0; c < n_chunks; ++c) {
            Eight<false> v[kChunkBlocks];
#pragma unroll
            for (int b = 0; b < kChunkBlocks; ++b) {
                const int col = (b0 + c * kChunkBlocks + b) * kBK + 8 * cg;
                if (row < g.m && col < g.k)
                    v[b].load(g.rows, (long long)row * g.k + col);
                else
                    v[b].clear();
            }
#pragma unroll
            for (int b = 0; b < kChunkBlocks; ++b) {
                float m = v[b].top();
#pragma unroll
                for (int k = 8; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
                const int e = scale_exponent(m, e5m2 ? 15 : 8);
                const float s = power_of_two(-e);
                const uint2 q = e5m2 ? codes_of<false, true>(v[b], s) : codes_of<false, false>(v[b], s);
                asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(tokens + (c * kChunkBlocks + b) * (NT * kBK) + row * kBK +
                                                                      (((cg >> 1) ^ (row & 7)) << 4) + (cg & 1) * 8),
                             "r"(q.x), "r"(q.y)
                             : "memory");
                if (cg == 0)
                    asm volatile("st.shared.u8 [%0], %1;" ::"r"(scales + c * 1024 + 512 + row * 16 + b), "r"(e + 127) : "memory");
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_scale + 8 * c);
        }
    }
    __syncwarp();
    // every product done, every stage read: their place takes the sums, [chunk][token][feature]
    if (!warp_wait(bar_acc, 0, &abort_flag) && lane == 0) fail(&abort_flag);
    tc_fence_after();
    __syncthreads();
    if (warp >= kWarpEpilogue) {
        const int quarter = warp & 3, f = 32 * quarter + lane;
        for (int c = (warp - kWarpEpilogue) >> 2; c < n_chunks * (NT / 16); c += 2) {  // 16 columns each
            uint32_t r[16];
            tmem_ld16(tmem + ((uint32_t)(quarter * 32) << 16) + 16 * c, r);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i)
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(sbase + ((16 * c + i) * 128 + f) * 4), "r"(r[i]) : "memory");
        }
    }
    tc_fence_before();
    if (ctas > 1)
        cluster_sync_all();
    else
        __syncthreads();
    // four features of one token a thread
    const int quads = 32 / ctas, first = rank * (128 / ctas), count = min(NT, g.m - at.t0);
    for (int e = tid; e < quads * count; e += kThreads) {
        const int i = first + 4 * (e % quads), tk = e / quads, f = at.f0 + i;
        if (f >= g.n) continue;
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        int w = 0, l = 0;
        for (int c = 0; c < chunks; c += 4) {
            float4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (c + j >= chunks) break;
                const uint32_t from = sbase + ((l * NT + tk) * 128 + i) * 4;
                v[j] = load_cluster(ctas > 1 ? map_rank(from, w) : from);
                if (++l == share) l = 0, ++w;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (c + j >= chunks) break;
                sum = c + j == 0 ? v[j] : make_float4(sum.x + v[j].x, sum.y + v[j].y, sum.z + v[j].z, sum.w + v[j].w);
            }
        }
        if (g.bias != nullptr) {
            const uint2 b = *reinterpret_cast<const uint2*>(g.bias + f);
            sum = make_float4(sum.x + bf16_lo(b.x), sum.y + bf16_hi(b.x), sum.z + bf16_lo(b.y), sum.w + bf16_hi(b.y));
        }
        const long long to = (long long)(at.t0 + tk) * g.d_stride + f;
        if (g.fp32) {
            float4* d = reinterpret_cast<float4*>(static_cast<float*>(g.d) + to);
            if (g.accumulate) {
                const float4 o = *d;
                sum = make_float4(o.x + sum.x, o.y + sum.y, o.z + sum.z, o.w + sum.w);
            }
            *d = sum;
        } else {
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(g.d) + to) = make_uint2(pack_bf16(sum.x, sum.y), pack_bf16(sum.z, sum.w));
        }
    }
    if (ctas > 1) cluster_sync_all();  // nobody leaves while another reads its sums
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

// ---- the wide product: CTA pairs ----
constexpr int kPairTokens = 224;  // columns of the accumulator: two of them and the scales fill TMEM
struct Pair {
    static constexpr int kTBytes = kPairTokens / 2 * kBK;  // a CTA's half of the tokens
    static constexpr int kBlockBytes = kFBytes + kTBytes;
    static constexpr int kStageBlocks = 2;  // scale blocks of a stage: a wait and a commit for eight products
    static constexpr int kStageBytes = kStageBlocks * kBlockBytes;
    static constexpr int kStages = 3;
    static constexpr int kAtoms = 2, kScaleBytes = 512 * (1 + kAtoms);
    static constexpr int kHalf = kPairTokens / 2, kScaleCol = 2 * kPairTokens;
    static constexpr int kOutTokens = kHalf / 2;           // tokens an epilogue warp hands to TMA at once in bf16
    static constexpr int kOutBytes = kOutTokens * 32 * 2;  // its buffer; half as many tokens in fp32
    static constexpr int kSmemBytes = kStages * kStageBytes + kScaleRing * kScaleBytes + 8 * kOutBytes + 1024;
    static_assert(kOutBytes % 128 == 0 && kOutTokens % 2 == 0 && kSmemBytes <= 227 * 1024, "");
    static_assert(kBlockBytes % 1024 == 0 && kTBytes % 1024 == 0 && kScaleCol + 32 <= 512 && kChunkBlocks % kStageBlocks == 0, "");
};

// A warp's 32 features (lane: f) over kHalf tokens from t on: + bias, rounded, by way of its buffer in shared memory to
// TMA, which cuts off what is past the matrix. Each pass waits until the one before it has left the buffer.
template <bool kFp32>
__device__ __forceinline__ void store_pair(const GemmItem& g, const float (&acc)[Pair::kHalf], uint32_t buffer, int f, int t) {
    constexpr int kTokens = kFp32 ? Pair::kOutTokens / 2 : Pair::kOutTokens;
    const int lane = threadIdx.x & 31, f0 = f - lane;
    if (f0 >= g.n) return;
    const float b = f < g.n && g.bias != nullptr ? __uint_as_float((uint32_t)g.bias[f] << 16) : 0.0f;
#pragma unroll
    for (int j = 0; j < Pair::kHalf; j += kTokens) {
        if (t + j >= g.m) break;
        bulk_wait_read_all();  // (the lane that stored; nothing to wait for in the others)
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kTokens; i += 2) {
            const float v0 = acc[j + i] + b, v1 = acc[j + i + 1] + b;
            if (kFp32) {
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(buffer + i * 128 + lane * 4), "f"(v0) : "memory");
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(buffer + i * 128 + 128 + lane * 4), "f"(v1) : "memory");
            } else {
                const uint32_t w = pack_bf16(v0, v1);
                asm volatile("st.shared.u16 [%0], %1;" ::"r"(buffer + i * 64 + lane * 2), "h"((uint16_t)w) : "memory");
                asm volatile("st.shared.u16 [%0], %1;" ::"r"(buffer + i * 64 + 64 + lane * 2), "h"((uint16_t)(w >> 16)) : "memory");
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            if (kFp32 && g.accumulate)
                tma_add_2d(&g.map_d, buffer, f0, t + j);
            else
                tma_store_2d(&g.map_d, buffer, f0, t + j);
            bulk_commit_group();
        }
    }
}

// 256 features x 224 tokens a cluster of two CTAs: each has 128 features' codes and half of the tokens', so that a
// product reads half the tokens' bytes from each SM's shared memory. The first CTA issues; both load, and both read
// out their 128 features.
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) fp8_gemm_pair_kernel(const __grid_constant__ GemmArgs a) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * Pair::kStages + 2 * kScaleRing + 5];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;

    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t rank = cluster_rank();
    const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
    const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
    auto stage_f = [&](int st) { return sbase + st * Pair::kStageBytes; };
    auto stage_t = [&](int st) { return sbase + st * Pair::kStageBytes + kFBytes; };
    auto scales = [&](int g) { return sbase + Pair::kStages * Pair::kStageBytes + g * Pair::kScaleBytes; };
    // of these the first CTA waits on its own full, sfull and free, both on theirs of the others
    const uint32_t bar_full = smem_u32(&bars[0]), bar_empty = bar_full + 8 * Pair::kStages;
    const uint32_t bar_sfull = bar_empty + 8 * Pair::kStages, bar_sempty = bar_sfull + 8 * kScaleRing;
    const uint32_t bar_acc = bar_sempty + 8 * kScaleRing, bar_free = bar_acc + 16, bar_drain = bar_free + 16;

    if (tid == 0) {
        abort_flag = 0;
        for (int i = 0; i < Pair::kStages; ++i) mbar_init(bar_full + 8 * i, 1), mbar_init(bar_empty + 8 * i, 1);
        for (int i = 0; i < kScaleRing; ++i) mbar_init(bar_sfull + 8 * i, 2), mbar_init(bar_sempty + 8 * i, 1);
        for (int i = 0; i < 2; ++i) mbar_init(bar_acc + 8 * i, 1), mbar_init(bar_free + 8 * i, 16);
        mbar_init(bar_drain, 1);
        fence_barrier_init();
    }
    if (warp == kWarpMma) {
        tmem_alloc_pair(smem_u32(&tmem_slot), kTmemCols);
        tmem_relinquish_pair();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");  // (the kernels before it round what it reads)
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;

    auto tile = [&](int t) {
        TileAt r;
        r.item = 0;
        while (r.item + 1 < a.n && t >= a.item[r.item + 1].tile0) ++r.item;
        const int l = t - a.item[r.item].tile0;
        r.f0 = (l % a.item[r.item].tiles_f) * 256 + 128 * rank;
        r.t0 = (l / a.item[r.item].tiles_f) * kPairTokens;
        return r;
    };

    if (warp == kWarpTma) {
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int n = 0, t; ok && (t = tile_of_turn(n, first, step)) < a.tiles; ++n) {
                const TileAt at = tile(t);
                const GemmItem& g = a.item[at.item];
                for (int kb = 0; kb < g.blocks; kb += Pair::kStageBlocks, ++it) {
                    const int st = it % Pair::kStages;
                    const uint32_t use = it / Pair::kStages;
                    if (use > 0 && !mbar_wait(bar_empty + 8 * st, (use - 1) & 1, &abort_flag, kWaitLimitNs)) {
                        ok = false;
                        break;
                    }
                    // (the bytes of both CTAs; the second one's may be counted before this)
                    if (rank == 0) mbar_expect_tx(bar_full + 8 * st, 2 * Pair::kStageBytes);
#pragma unroll
                    for (int b = 0; b < Pair::kStageBlocks; ++b) {  // (zeros past the row's end)
                        tma_load_2d_pair(stage_f(st) + b * Pair::kBlockBytes, &g.map_f, bar_full + 8 * st, (kb + b) * kBK, at.f0);
                        tma_load_2d_pair(stage_t(st) + b * Pair::kBlockBytes, &g.map_t, bar_full + 8 * st, (kb + b) * kBK,
                                         at.t0 + Pair::kHalf * rank);
                    }
                }
            }
            if (!ok) fail(&abort_flag);
            // drain: every stage issued here has landed (counted on the first CTA's barriers) or been consumed
            if (rank == 0) {
                for (uint32_t u = it < Pair::kStages ? 0 : it - Pair::kStages; u < it; ++u)
                    mbar_wait_drain(bar_full + 8 * (u % Pair::kStages), (u / Pair::kStages) & 1, kWaitLimitNs);
            } else if (ok) {
                for (uint32_t u = it < Pair::kStages ? 0 : it - Pair::kStages; u < it; ++u)
                    mbar_wait_drain(bar_empty + 8 * (u % Pair::kStages), (u / Pair::kStages) & 1, kWaitLimitNs);
            }
        }
    } else if (warp == kWarpMma) {
        if (rank == 0) {
            // (the whole warp runs the loop, one lane issues; the issuing thread has about a hundred cycles a product: descriptors are sums of what is at hand)
            const uint64_t f0 = sdesc_sw128(stage_f(0), 16, 1024), t0 = sdesc_sw128(stage_t(0), 16, 1024);
            const uint64_t s0 = sdesc_noswizzle(scales(0), 0, 128);
            uint32_t chunks = 0;  // of all tiles
            for (int n = 0, t; (t = tile_of_turn(n, first, step)) < a.tiles; ++n) chunks += (a.item[tile(t).item].blocks + kChunkBlocks - 1) / kChunkBlocks;
            uint32_t st = 0, phase = 0, chunk = 0;
            bool ok = true;
            auto copy_scales = [&](uint32_t c) {  // a chunk's, one chunk ahead of its products
                const uint32_t ring = c % kScaleRing;
                if (!warp_wait_cluster(bar_sfull + 8 * ring, (c / kScaleRing) & 1, &abort_flag)) return false;
                tc_fence_after();
                const uint32_t sa = tmem + Pair::kScaleCol + (c & 1) * 16;
                if (elect_one())
#pragma unroll
                for (int i = 0; i < 1 + Pair::kAtoms; ++i)
                    tmem_copy_scales_pair(sa + 4 * i, s0 + ((ring * Pair::kScaleBytes + 512 * i) >> 4));
                return true;
            };
            if (chunks > 0) ok = copy_scales(0);
            for (int n = 0, t; ok && (t = tile_of_turn(n, first, step)) < a.tiles; ++n) {
                const GemmItem& g = a.item[tile(t).item];
                const int blocks = g.blocks;
                for (int kb = 0; ok && kb < blocks; ++chunk) {
                    const int buf = chunk & 1;
                    const uint32_t use = chunk >> 1;
                    if (use > 0 && !warp_wait_cluster(bar_free + 8 * buf, (use - 1) & 1, &abort_flag)) {
                        ok = false;
                        break;
                    }
                    const uint32_t acc = tmem + buf * kPairTokens;
                    const uint32_t sa = tmem + Pair::kScaleCol + buf * 16, sb = sa + 4;
                    const int start = kb, end = min(kb + kChunkBlocks, blocks);
                    uint32_t id = g.idesc;
                    while (kb < end) {
                        if (!warp_wait(bar_full + 8 * st, phase, &abort_flag)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t f = f0 + st * (Pair::kStageBytes >> 4), tk = t0 + st * (Pair::kStageBytes >> 4);
                        const bool new_sum = kb == start, two = kb + 1 < end;
                        if (elect_one()) {
#pragma unroll
                            for (int b = 0; b < Pair::kStageBlocks; ++b) {
                                if (b > 0 && !two) break;
#pragma unroll
                                for (int j = 0; j < kBK / 32; ++j)  // (each block's scale bytes are one further)
                                    mma_mx_pair(acc, f + ((b * Pair::kBlockBytes) >> 4) + 2 * j, tk + ((b * Pair::kBlockBytes) >> 4) + 2 * j,
                                                id + b * ((1u << 29) | (1u << 4)), sa, sb, b > 0 || j > 0 || !new_sum ? 1u : 0u);
                            }
                            mma_commit_pair(bar_empty + 8 * st);
                        }
                        kb += two ? 2 : 1;
                        id += 2 * ((1u << 29) | (1u << 4));
                        if (++st == Pair::kStages) st = 0, phase ^= 1;
                        if (new_sum && chunk + 1 < chunks && !copy_scales(chunk + 1)) {
                            ok = false;
                            break;
                        }
                    }
                    if (ok && elect_one()) {
                        mma_commit_pair(bar_sempty + 8 * (chunk % kScaleRing));
                        mma_commit_pair(bar_acc + 8 * buf);
                    }
                }
            }
            if (elect_one()) {
                if (!ok) fail(&abort_flag);
                mma_commit_pair(bar_drain);
            }
        }
        if (lane == 0) mbar_wait_drain(bar_drain, 0, kWaitLimitNs);  // (in both: the last thing that arrives here)
    } else if (warp == kWarpScale) {
        uint32_t chunk = 0;
        bool ok = true;
        for (int n = 0, t; ok && (t = tile_of_turn(n, first, step)) < a.tiles; ++n) {
            const TileAt at = tile(t);
            const GemmItem& g = a.item[at.item];
            for (int kb = 0; kb < g.blocks; kb += kChunkBlocks, ++chunk) {
                const int ring = chunk % kScaleRing;
                const uint32_t use = chunk / kScaleRing;
                uint32_t w[1 + Pair::kAtoms][4];
#pragma unroll
                for (int i = 0; i < 1 + Pair::kAtoms; ++i) gather_scales(w[i], g, i, at, kb, lane);
                if (use > 0 && !warp_wait(bar_sempty + 8 * ring, (use - 1) & 1, &abort_flag)) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int i = 0; i < 1 + Pair::kAtoms; ++i) put_scales(scales(ring) + 512 * i + 16 * lane, w[i]);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(map_rank(bar_sfull + 8 * ring, 0));
            }
        }
        if (!ok && lane == 0) fail(&abort_flag);
    } else if (warp >= kWarpEpilogue) {
        const int quarter = warp & 3, half = (warp - kWarpEpilogue) >> 2;
        const uint32_t at0 = tmem + ((uint32_t)(quarter * 32) << 16) + half * Pair::kHalf;
        const uint32_t buffer = scales(kScaleRing) + (warp - kWarpEpilogue) * Pair::kOutBytes;
        uint32_t chunk = 0;
        bool ok = true;
        for (int n = 0, t; ok && (t = tile_of_turn(n, first, step)) < a.tiles; ++n) {
            const TileAt at = tile(t);
            const GemmItem& g = a.item[at.item];
            float acc[Pair::kHalf];
            for (int kb = 0; kb < g.blocks; kb += kChunkBlocks, ++chunk) {
                const int buf = chunk & 1;
                if (!warp_wait(bar_acc + 8 * buf, (chunk >> 1) & 1, &abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                add_chunk<Pair::kHalf>(acc, at0 + buf * kPairTokens, kb == 0);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(map_rank(bar_free + 8 * buf, 0));
            }
            const int f = at.f0 + 32 * quarter + lane, tk = at.t0 + half * Pair::kHalf;
            if (ok && g.fp32) store_pair<true>(g, acc, buffer, f, tk);
            if (ok && !g.fp32) store_pair<false>(g, acc, buffer, f, tk);
        }
        bulk_wait_all();
        if (!ok && lane == 0) fail(&abort_flag);
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // the other CTA's products, commits and arrivals reach this one's memory until here
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, kTmemCols);
    }
}

cudaError_t launch_pair(GemmArgs& a, int sms, cudaStream_t s) {
    std::stable_sort(a.item, a.item + a.n, [](const GemmItem& x, const GemmItem& y) { return x.blocks > y.blocks; });
    a.tiles = 0;
    for (int i = 0; i < a.n; ++i) {
        GemmItem& g = a.item[i];
        g.tiles_f = (g.n + 255) / 256;
        g.tile0 = a.tiles;
        g.idesc |= idesc_mx(256, kPairTokens);
        a.tiles += g.tiles_f * ((g.m + kPairTokens - 1) / kPairTokens);
    }
    cudaError_t e = smem_once<fp8_gemm_pair_kernel>(Pair::kSmemBytes);
    if (e != cudaSuccess) return e;
    // clusters that fit at once: more would wait for the first to end
    static std::atomic<int> fit[64];
    int dev = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    int pairs = dev < 64 ? fit[dev].load() : 0;
    if (pairs == 0) {
        cudaLaunchConfig_t c{};
        c.gridDim = dim3(2 * (sms / 2));
        c.blockDim = dim3(kThreads);
        c.dynamicSmemBytes = Pair::kSmemBytes;
        if ((e = cudaOccupancyMaxActiveClusters(&pairs, fp8_gemm_pair_kernel, &c)) != cudaSuccess) return e;
        if (pairs < 1) return cudaErrorLaunchOutOfResources;
        if (dev < 64) fit[dev].store(pairs);
    }
    timing_begin(kKFp8Gemm, s);
    e = launch_after(fp8_gemm_pair_kernel, 2 * (a.tiles < pairs ? a.tiles : pairs), kThreads, Pair::kSmemBytes, s, a);
    timing_end(kKFp8Gemm, s);
    return e;
}

// The CTAs that share a tile's K: enough for two an SM of all the tiles, at most one a chunk, and enough for each CTA's
// TMEM (0: it is not).
template <int NT, bool kRaw>
int few_ctas(const rlk_fp8_product* p, int n, int sms) {
    constexpr int kSlots = Few<NT, kRaw>::kSlots;
    long long tiles = 0, chunks = 1;
    for (int i = 0; i < n; ++i) {
        if (p[i].m == 0 || p[i].n == 0) continue;
        tiles += (p[i].n + 127) / 128 * ((p[i].m + NT - 1) / NT);
        const long long c = (p[i].k + 128 * kChunkBlocks - 1) / (128 * kChunkBlocks);
        chunks = c > chunks ? c : chunks;
    }
    int ctas = 1;
    while (ctas < 8 && (chunks > (long long)ctas * kSlots || (2 * ctas <= chunks && 2 * ctas * tiles <= 2 * sms))) ctas *= 2;
    return chunks <= (long long)ctas * kSlots ? ctas : 0;
}

template <int NT, bool kRaw>
cudaError_t launch_few(GemmArgs& a, int ctas, cudaStream_t s) {
    a.tiles = 0;
    a.ctas = ctas;
    for (int i = 0; i < a.n; ++i) {
        GemmItem& g = a.item[i];
        g.tiles_f = (g.n + 127) / 128;
        g.tile0 = a.tiles;
        g.idesc |= idesc_mx(128, NT);
        a.tiles += g.tiles_f * ((g.m + NT - 1) / NT);
    }
    cudaError_t e = smem_once<fp8_gemm_few_kernel<NT, kRaw>>(Few<NT, kRaw>::kSmemBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)(a.tiles * ctas));
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = Few<NT, kRaw>::kSmemBytes;
    c.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = attr;
    c.numAttrs = 2;
    timing_begin(kKFp8Gemm, s);
    e = cudaLaunchKernelEx(&c, fp8_gemm_few_kernel<NT, kRaw>, a);
    timing_end(kKFp8Gemm, s);
    return e;
}

// codes [rows, k] with rows ld bytes apart, box 128 x box_rows
bool codes_map(CUtensorMap* m, const void* base, long long rows, long long k, long long ld, int box_rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld};
    const cuuint32_t box[2] = {kBK, (cuuint32_t)box_rows};
    return tmap::encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, box);
}

}  // namespace

// fp32 input 1, e5m2 2, blocks along the rows alone 4
static int quant_kind(const rlk_fp8_quant& e) {
    return (e.x_dtype == RLK_FP32 ? 1 : 0) | (e.format == RLK_E5M2 ? 2 : 0) |
           (e.qt == nullptr && e.square == 0 && e.col_sum == nullptr ? 4 : 0);
}

// The items of one kind (input type, format, rows alone or a tile's work) in one launch.
static cudaError_t launch_quant_kind(const rlk_fp8_quant* q, int n, int kind, cudaStream_t s) {
    QuantArgs a;
    a.n = 0;
    int tiles = 0;
    const bool fp32 = kind & 1, e5m2 = kind & 2, rows_alone = kind & 4;
    for (int i = 0; i < n; ++i) {
        const rlk_fp8_quant& e = q[i];
        if (e.rows == 0 || kind != quant_kind(e)) continue;
        QuantItem& it = a.item[a.n++];
        it.x = e.x;
        it.q = static_cast<uint8_t*>(e.q);
        it.q_scale = e.q_scale;
        it.qt = static_cast<uint8_t*>(e.qt);
        it.qt_scale = e.qt_scale;
        it.part = e.col_sum != nullptr ? static_cast<float*>(e.workspace) : nullptr;
        it.x_stride = e.x_stride;
        it.rows = (int)e.rows;
        it.cols = (int)e.cols;
        it.ldq = (int)rlk_fp8_row_bytes(e.cols);
        it.lds = (int)rlk_fp8_scale_row_bytes(e.cols);
        it.ldqt = (int)rlk_fp8_row_bytes(e.rows);
        it.ldst = (int)rlk_fp8_scale_row_bytes(e.rows);
        it.col_tiles = (int)((e.cols + 127) / 128);
        it.tile0 = tiles;
        it.square = e.square != 0;
        const long long tall = rows_alone ? kRowsTile : kTile;
        tiles += (int)((e.rows + tall - 1) / tall) * it.col_tiles;
    }
    if (tiles == 0) return cudaSuccess;
    void (*const kernel)(QuantArgs) =
        rows_alone ? (fp32 ? (e5m2 ? fp8_quant_rows_kernel<true, true> : fp8_quant_rows_kernel<true, false>)
                           : (e5m2 ? fp8_quant_rows_kernel<false, true> : fp8_quant_rows_kernel<false, false>))
                   : (fp32 ? (e5m2 ? fp8_quant_kernel<true, true> : fp8_quant_kernel<true, false>)
                           : (e5m2 ? fp8_quant_kernel<false, true> : fp8_quant_kernel<false, false>));
    timing_begin(kKFp8Quant, s);
    kernel<<<tiles, kQuantThreads, 0, s>>>(a);
    timing_end(kKFp8Quant, s);
    return cudaGetLastError();
}

cudaError_t launch_fp8_quant(const rlk_fp8_quant* q, int n, cudaStream_t s) {
    FoldArgs f;
    f.n = 0;
    int blocks = 0;
    unsigned kinds = 0;
    for (int i = 0; i < n; ++i) {
        const rlk_fp8_quant& e = q[i];
        if (e.rows > 0) kinds |= 1u << quant_kind(e);
        if (e.col_sum == nullptr) continue;
        f.item[f.n++] = FoldItem{static_cast<const float*>(e.workspace), e.col_sum, (int)((e.rows + 127) / 128), (int)e.cols, blocks};
        blocks += ((int)e.cols + kFoldCols - 1) / kFoldCols;
    }
    cudaError_t e = cudaSuccess;
    for (int kind = 0; kind < 8 && e == cudaSuccess; ++kind)
        if (kinds >> kind & 1) e = launch_quant_kind(q, n, kind, s);
    if (e != cudaSuccess || blocks == 0) return e;
    timing_begin(kKFp8Fold, s);
    e = launch_after(fp8_fold_kernel, blocks, kFoldThreads, 0, s, f);
    timing_end(kKFp8Fold, s);
    return e;
}

cudaError_t launch_fp8_gemm(const rlk_fp8_product* p, int n, cudaStream_t s) {
    GemmArgs a;
    a.n = 0;
    long long most = 0;
    for (int i = 0; i < n; ++i) most = most < p[i].m ? p[i].m : most;
    int dev = 0, sms = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (err != cudaSuccess) return err;
    // The accumulator's columns: the narrowest that takes every token, if K is not too long for it, else 224 (64 for 100 to
    // 1000 tokens, all tiles at once, took as long as pairs: 2560 -> 2560 with 300 tokens 13.0 us for 11.7, 512 -> 1024 with
    // 1000 7.5 for 7.9).
    int nt = kPairTokens, ctas = 0;
    const bool raw = p[0].a_rows != 0;  // (16 tokens at most, of 12288 values at most)
    if (most <= 64) {
        nt = most <= 16 ? 16 : 64;
        ctas = raw ? few_ctas<16, true>(p, n, sms) : nt == 16 ? few_ctas<16, false>(p, n, sms) : few_ctas<64, false>(p, n, sms);
        if (ctas == 0) nt = kPairTokens;
    }
    if (raw && nt != 16) return cudaErrorInvalidValue;
    for (int i = 0; i < n; ++i) {
        const rlk_fp8_product& e = p[i];
        if (e.m == 0 || e.n == 0) continue;
        GemmItem& g = a.item[a.n++];
        const long long ld = rlk_fp8_row_bytes(e.k);
        if (!codes_map(&g.map_f, e.b, e.n, e.k, ld, 128) || (!raw && !codes_map(&g.map_t, e.a, e.m, e.k, ld, nt == kPairTokens ? nt / 2 : nt)))
            return cudaErrorInvalidValue;
        if (nt == kPairTokens) {
            const bool fp32 = e.d_dtype == RLK_FP32;
            const cuuint64_t dims[2] = {(cuuint64_t)e.n, (cuuint64_t)e.m};
            const cuuint64_t strides[1] = {(cuuint64_t)e.d_stride * (fp32 ? 4 : 2)};
            const cuuint32_t box[2] = {32, (cuuint32_t)(fp32 ? Pair::kOutTokens / 2 : Pair::kOutTokens)};
            if (!tmap::encode(&g.map_d, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, e.d, dims,
                              strides, box, CU_TENSOR_MAP_SWIZZLE_NONE))
                return cudaErrorInvalidValue;
        }
        g.sf = e.b_scale;
        g.st = e.a_scale;
        g.bias = static_cast<const uint16_t*>(e.bias);
        g.rows = raw ? e.a : nullptr;
        g.k = (int)e.k;
        g.d = e.d;
        g.d_stride = e.d_stride;
        g.ldsf = g.ldst = (int)rlk_fp8_scale_row_bytes(e.k);
        g.m = (int)e.m;
        g.n = (int)e.n;
        g.blocks = (int)((e.k + 127) / 128);
        // (the features are the instruction's A)
        g.idesc = (e.b_format == RLK_E5M2 ? 1u << 7 : 0u) | (e.a_format == RLK_E5M2 ? 1u << 10 : 0u);
        g.fp32 = e.d_dtype == RLK_FP32;
        g.accumulate = e.accumulate != 0;
    }
    if (a.n == 0) return cudaSuccess;
    return raw        ? launch_few<16, true>(a, ctas, s)
           : nt == 16 ? launch_few<16, false>(a, ctas, s)
           : nt == 64 ? launch_few<64, false>(a, ctas, s)
                      : launch_pair(a, sms, s);
}

int read_and_clear_status_fp8(cudaStream_t s) {
    int v = 0, zero = 0;
    if (cudaMemcpyFromSymbolAsync(&v, g_status_fp8, sizeof(int), 0, cudaMemcpyDeviceToHost, s) != cudaSuccess) return -1;
    if (cudaMemcpyToSymbolAsync(g_status_fp8, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s) != cudaSuccess) return -1;
    if (cudaStreamSynchronize(s) != cudaSuccess) return -1;
    return v;
}

}  // namespace rlk
